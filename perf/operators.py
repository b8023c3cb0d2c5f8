"""The token mixers beside Kimi Delta Attention, as they are timed.

Six operators, each in the form for prompts and the form for one new token per sequence:

  conv_prefill, conv_step      short causal depthwise convolution with an optional SiLU
  ssm_prefill, ssm_step        selective state space scan: one decay per head and token, state [n, p]
  window_prefill, window_step  attention with a sliding window and a few first tokens that stay
                               visible, over a ring cache of fixed size

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (decay
exponents in 64); with ``own`` true it calls the library.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64        # tokens per block of the plain scan
QBLOCK = 256      # queries per block of the plain window attention


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a short ragged prompt batch in fp32, continuing from a kept history: launch-bound
        {"name": "conv_prefill small f32", "op": "conv_prefill", "B": 3, "T": 200, "D": 1000, "W": 4, "silu": True,
         "state": True, "ragged": True, "dtype": "f32"},
        # a whole layer's prompt batch: x, B and C of 56 heads of 128 inside the projection's rows
        {"name": "conv_prefill wide", "op": "conv_prefill", "B": 4, "T": 8192, "D": 7424, "W": 4, "silu": True,
         "state": False, "ragged": False, "dtype": "bf16"},
        # one user, one token: latency
        {"name": "conv_step one", "op": "conv_step", "N": 1, "D": 7424, "W": 4, "silu": True, "dtype": "bf16"},
        # a serving batch of 256 sequences
        {"name": "conv_step batch", "op": "conv_step", "N": 256, "D": 7424, "W": 4, "silu": True, "dtype": "bf16"},
        # one long prompt of odd length, few heads: the sequence itself has to fill the GPU
        {"name": "ssm_prefill long", "op": "ssm_prefill", "B": 1, "T": 20001, "H": 16, "G": 1, "n": 128, "p": 64,
         "gated": True, "state": True, "ragged": False, "dtype": "bf16"},
        # model width: 56 heads of 128, four prompts
        {"name": "ssm_prefill wide", "op": "ssm_prefill", "B": 4, "T": 16384, "H": 56, "G": 1, "n": 128, "p": 128,
         "gated": True, "state": False, "ragged": False, "dtype": "bf16"},
        # one user, one token, fp32
        {"name": "ssm_step one f32", "op": "ssm_step", "N": 1, "H": 56, "G": 1, "n": 128, "p": 64, "gated": True,
         "dtype": "f32"},
        # a serving batch: 256 sequences of 56 heads of 128
        {"name": "ssm_step batch", "op": "ssm_step", "N": 256, "H": 56, "G": 8, "n": 128, "p": 128, "gated": True,
         "dtype": "bf16"},
        # ragged pieces of prompts continued from their caches (chunked prefill), odd sizes
        {"name": "window_prefill ragged", "op": "window_prefill", "B": 5, "T": 333, "H": 8, "Hkv": 2, "d": 64,
         "window": 200, "sinks": 3, "cache": True, "ragged": True, "dtype": "bf16"},
        # one prompt at model width
        {"name": "window_prefill wide", "op": "window_prefill", "B": 1, "T": 16384, "H": 56, "Hkv": 8, "d": 128,
         "window": 4096, "sinks": 4, "cache": True, "ragged": False, "dtype": "bf16"},
        # one user, one token: few rows, a long axis
        {"name": "window_step one", "op": "window_step", "N": 1, "H": 56, "Hkv": 8, "d": 128, "window": 4096,
         "sinks": 4, "dtype": "bf16"},
        # a serving batch
        {"name": "window_step batch", "op": "window_step", "N": 64, "H": 56, "Hkv": 8, "d": 128, "window": 4096,
         "sinks": 4, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prefill", "conv_step", "ssm_prefill", "ssm_prefill", "ssm_step", "window_prefill",
                     "window_prefill", "window_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "conv_prefill":
        D = _log(rng, 16, 8192)
        T = _log(rng, 1, 16384)
        B = max(1, min(_log(rng, 1, 64), (60 << 20) // (D * T)))
        return {"op": op, "B": B, "T": T, "D": D, "W": rng.choice([2, 3, 4, 4]), "silu": rng.random() < 0.7,
                "state": rng.random() < 0.5, "ragged": rng.random() < 0.5, "dtype": dtype}
    if op == "conv_step":
        return {"op": op, "N": _log(rng, 1, 1024), "D": _log(rng, 16, 8192), "W": rng.choice([2, 3, 4, 4]),
                "silu": rng.random() < 0.7, "dtype": dtype}
    G = rng.choice([1, 1, 2, 4])
    H = G * _log(rng, 1, 14)
    n, p = rng.choice([64, 128]), rng.choice([64, 128])
    if op == "ssm_prefill":
        T = _log(rng, 1, 32768 if dtype == "bf16" else 4096)
        B = max(1, min(_log(rng, 1, 16), (3 << 20 if dtype == "bf16" else 1 << 18) // (H * T)))
        return {"op": op, "B": B, "T": T, "H": H, "G": G, "n": n, "p": p, "gated": rng.random() < 0.6,
                "state": rng.random() < 0.5, "ragged": rng.random() < 0.5, "dtype": dtype}
    if op == "ssm_step":
        return {"op": op, "N": max(1, min(_log(rng, 1, 512), 14000 // H)), "H": H, "G": G, "n": n, "p": p,
                "gated": rng.random() < 0.6, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    d = rng.choice([64, 128])
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, 4, 16])
    if op == "window_prefill":
        T = _log(rng, 1, 16384 if dtype == "bf16" else 2048)
        B = max(1, min(_log(rng, 1, 16), (3 << 30) // (H * T * (window + QBLOCK))))
        return {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "window": window, "sinks": sinks,
                "cache": rng.random() < 0.7, "ragged": rng.random() < 0.5, "dtype": dtype}
    return {"op": op, "N": max(1, min(_log(rng, 1, 256), (64 << 12) // window)), "H": H, "Hkv": Hkv, "d": d,
            "window": window, "sinks": sinks, "dtype": dtype}


# ----------------------------------------------------------------------------------------- inputs
def _rows(width):
    """Length of a projection's rows: whole 16-byte groups, as a program pads them."""
    return -(-width // 8) * 8


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32) * (hi - lo) + lo

    op = case["op"]
    s = {"op": op, "dtype": dt}
    if op.endswith("prefill"):
        B, T = case["B"], case["T"]
        s["lens"] = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32) if case["ragged"] else None
    if op in ("conv_prefill", "conv_step"):
        D, W = case["D"], case["W"]
        # x is a slice of the input projection's rows, after the gate's columns and before the steps'
        lead = _rows(D // 2)
        row = _rows(lead + D + 8)
        s["w"] = uniform(-W ** -0.5, W ** -0.5, D, W).to(dt)
        s["bias"] = uniform(-0.2, 0.2, D).to(dt)
        s["silu"] = case["silu"]
        if op == "conv_prefill":
            s["x"] = normal(B, T, row)[:, :, lead:lead + D]
            s["state"] = normal(B, W - 1, D) if case["state"] else None
            # rows past a sequence's end keep what the buffer holds
            s["y"] = torch.zeros(B, T, D, dtype=dt, device=dev)
        else:
            s["x"] = normal(case["N"], row)[:, lead:lead + D]
            s["state"] = normal(case["N"], W - 1, D)
    elif op in ("ssm_prefill", "ssm_step"):
        H, G, n, p = case["H"], case["G"], case["n"], case["p"]
        lead = (B, T) if op == "ssm_prefill" else (case["N"],)
        # x, B and C are slices of the convolution's rows; z and the raw steps of the projection's
        xbc = normal(*lead, H * p + 2 * G * n)
        proj = normal(*lead, _rows(H * p + H))
        s["x"] = xbc[..., :H * p].unflatten(-1, (H, p))
        s["Bm"] = xbc[..., H * p:H * p + G * n].unflatten(-1, (G, n))
        s["Cm"] = xbc[..., H * p + G * n:].unflatten(-1, (G, n))
        s["z"] = proj[..., :H * p].unflatten(-1, (H, p)) if case["gated"] else None
        s["dt"] = proj[..., H * p:H * p + H]
        s["A"] = -uniform(1.0, 16.0, H)
        s["D"] = uniform(0.5, 1.5, H)
        # steps between about 0.001 and 0.1 where the projection gives zero
        step = torch.exp(uniform(math.log(0.001), math.log(0.1), H))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        if op == "ssm_prefill":
            s["S"] = normal(B, H, n, p, dtype=torch.float32) if case["state"] else None
            s["y"] = torch.zeros(B, T, H, p, dtype=dt, device=dev)
        else:
            s["S"] = normal(case["N"], H, n, p, dtype=torch.float32)
    else:
        H, Hkv, d, window, sinks = (case[k] for k in ("H", "Hkv", "d", "window", "sinks"))
        s["window"], s["sinks"], s["scale"] = window, sinks, d ** -0.5
        lead = (B, T) if op == "window_prefill" else (case["N"],)
        # q, k and v side by side in one projection's rows
        qkv = normal(*lead, (H + 2 * Hkv) * d)
        s["q"] = qkv[..., :H * d].unflatten(-1, (H, d))
        s["k"] = qkv[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
        s["v"] = qkv[..., (H + Hkv) * d:].unflatten(-1, (Hkv, d))
        rows = lead[0]
        if op == "window_step" or case["cache"]:
            s["k_cache"] = normal(rows, sinks + window, Hkv, d)
            s["v_cache"] = normal(rows, sinks + window, Hkv, d)
        else:
            s["k_cache"] = s["v_cache"] = None
        # tokens each sequence has behind it: none, some, or far more than the window
        before = torch.randint(0, 2 * (sinks + window), (rows,), generator=g, device=dev, dtype=torch.int32)
        if op == "window_step":
            s["pos"] = before + window   # in service: the ring has usually filled
        else:
            s["start"] = before if case["cache"] and case["ragged"] else None
            s["o"] = torch.zeros(rows, T, H, d, dtype=dt, device=dev)
    return s


# -------------------------------------------------------------------------------------------- run
def run(s):
    if own:
        return _own(s)
    return {"conv_prefill": _conv_prefill, "conv_step": _conv_step, "ssm_prefill": _ssm_prefill,
            "ssm_step": _ssm_step, "window_prefill": _window_prefill, "window_step": _window_step}[s["op"]](s)


def _own(s):
    import chunked_gated_delta_13_amd as kda
    op = s["op"]
    if op == "conv_prefill":
        return kda.conv_prefill(s["x"], s["w"], s["bias"], s["state"], lens=s["lens"], silu=s["silu"], y=s["y"])
    if op == "conv_step":
        return kda.conv_step(s["x"], s["w"], s["state"], s["bias"], silu=s["silu"]), s["state"]
    if op == "ssm_prefill":
        return kda.ssm_prefill(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], D=s["D"], z=s["z"],
                               dt_bias=s["dt_bias"], lens=s["lens"], y=s["y"])
    if op == "ssm_step":
        return kda.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], D=s["D"], z=s["z"],
                            dt_bias=s["dt_bias"]), s["S"]
    if op == "window_prefill":
        o = kda.window_prefill(s["q"], s["k"], s["v"], s["window"], s["sinks"], scale=s["scale"],
                               k_cache=s["k_cache"], v_cache=s["v_cache"], start=s["start"], lens=s["lens"], o=s["o"])
    else:
        o = kda.window_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], s["window"], s["sinks"],
                            scale=s["scale"])
    return o, s["k_cache"], s["v_cache"]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _alive(lens, B, T, device):
    """[B, T] truth values: token t of sequence b exists."""
    if lens is None:
        return torch.ones(B, T, dtype=torch.bool, device=device)
    return torch.arange(T, device=device)[None] < lens[:, None]


def _conv_prefill(s):
    x, w = s["x"], s["w"].float()
    B, T, D = x.shape
    W = w.shape[1]
    past = x.new_zeros(B, W - 1, D) if s["state"] is None else s["state"]
    whole = torch.cat([past, x], 1)
    y = (whole.float().unfold(1, W, 1) * w).sum(-1) + s["bias"].float()
    y = _silu(y) if s["silu"] else y
    alive = _alive(s["lens"], B, T, x.device)
    s["y"].copy_(torch.where(alive[..., None], y, s["y"].float()))
    end = alive.sum(1)
    at = end[:, None] + torch.arange(W - 1, device=x.device)   # the last W - 1 rows before the end
    return s["y"], torch.gather(whole, 1, at[..., None].expand(B, W - 1, D))


def _conv_step(s):
    whole = torch.cat([s["state"], s["x"][:, None]], 1)
    y = (whole.float() * s["w"].float().t()).sum(1) + s["bias"].float()
    y = _silu(y) if s["silu"] else y
    s["state"].copy_(whole[:, 1:])
    return y.to(s["dtype"]), s["state"]


def _ssm_prefill(s):
    """Blocks of CHUNK tokens: inside a block by its decay-weighted C B^T, between blocks by the
    products of the decays.  Exponents are summed in 64 bits."""
    x, A = s["x"].float(), s["A"]
    B, T, H, p = x.shape
    G, n = s["Bm"].shape[-2:]
    R, nc = H // G, -(-T // CHUNK)
    alive = _alive(s["lens"], B, T, x.device)
    step = _softplus(s["dt"].float() + s["dt_bias"]) * alive[..., None]

    def blocks(v):   # [B, T, ...] -> [B, nc, CHUNK, ...], zeros behind the end
        v = torch.cat([v, v.new_zeros(B, nc * CHUNK - T, *v.shape[2:])], 1)
        return v.unflatten(1, (nc, CHUNK))

    live = alive[..., None, None]
    xb = blocks(torch.where(live, x, 0.0)).permute(0, 1, 3, 2, 4)                    # [B, nc, H, L, p]
    bb = blocks(torch.where(live, s["Bm"].float(), 0.0)).permute(0, 1, 3, 2, 4)      # [B, nc, G, L, n]
    cb = blocks(torch.where(live, s["Cm"].float(), 0.0)).permute(0, 1, 3, 2, 4)
    db = blocks(step).permute(0, 1, 3, 2)                                            # [B, nc, H, L]
    cum = (db.double() * A.double()[:, None]).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf)).float()
    mix = torch.matmul(cb, bb.transpose(-1, -2).contiguous())                        # [B, nc, G, L, L]
    mix = mix[:, :, :, None] * (decay * db[..., None, :]).unflatten(2, (G, R))
    y = torch.matmul(mix.flatten(2, 3), xb)
    late = torch.exp(cum[..., -1:] - cum).float() * db
    inc = torch.matmul(bb.transpose(-1, -2).contiguous()[:, :, :, None], (late[..., None] * xb).unflatten(2, (G, R)))
    inc = inc.flatten(2, 3)                                                          # [B, nc, H, n, p]
    first = inc.new_zeros(B, 1, H, n, p) if s["S"] is None else s["S"][:, None]
    inc = torch.cat([first, inc], 1)
    tot = torch.cat([cum.new_zeros(B, 1, H), cum[..., -1]], 1).cumsum(1).permute(0, 2, 1)   # [B, H, nc + 1]
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp((tot[..., :, None] - tot[..., None, :]).masked_fill(~low, -math.inf)).float()
    states = torch.matmul(carry, inc.permute(0, 2, 1, 3, 4).flatten(-2)).unflatten(-1, (n, p))   # after c blocks
    entry = states[:, :, :-1].permute(0, 2, 1, 3, 4).unflatten(2, (G, R))
    y = y + torch.matmul(cb[:, :, :, None], entry).flatten(2, 3) * torch.exp(cum).float()[..., None]
    y = y + s["D"][:, None, None] * xb
    y = y.permute(0, 1, 3, 2, 4).flatten(1, 2)[:, :T]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["y"].copy_(torch.where(live, y, s["y"].float()))
    return s["y"], states[:, :, -1].contiguous()


def _ssm_step(s):
    S, x = s["S"], s["x"].float()
    R = x.shape[1] // s["Bm"].shape[1]
    step = _softplus(s["dt"].float() + s["dt_bias"])
    b = s["Bm"].float().repeat_interleave(R, 1)
    c = s["Cm"].float().repeat_interleave(R, 1)
    S.mul_(torch.exp(step * s["A"])[..., None, None]).add_(b[..., None] * (step[..., None] * x)[..., None, :])
    y = (c[..., None] * S).sum(-2) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["dtype"]), S


def _window_prefill(s):
    """Blocks of QBLOCK queries against the keys of their band, and against the first tokens."""
    q, k, v, window, sinks = s["q"], s["k"], s["v"], s["window"], s["sinks"]
    B, T, H, d = q.shape
    Hkv = k.shape[2]
    R, dev = H // Hkv, q.device
    start = torch.zeros(B, dtype=torch.int64, device=dev) if s["start"] is None else s["start"].long()
    alive = _alive(s["lens"], B, T, dev)
    nb = -(-T // QBLOCK)
    pad = nb * QBLOCK - T

    def pick(rows, at):   # rows [B, m, Hkv, d] by at [B, j]
        return torch.gather(rows, 1, at[..., None, None].expand(*at.shape, Hkv, d))

    def keys(new, cache):
        """fp32 rows of the positions start - window ... start + T - 1 (+ padding), and of 0 ... sinks - 1."""
        new_f = new.float()
        tail = new_f.new_zeros(B, pad, Hkv, d)
        back = start[:, None] - window + torch.arange(window, device=dev)
        first = torch.arange(sinks, device=dev).expand(B, sinks)
        here = pick(new_f, (first - start[:, None]).clamp(0, T - 1))
        if cache is None:
            return torch.cat([new_f.new_zeros(B, window, Hkv, d), new_f, tail], 1), here
        past = pick(cache, sinks + (back - sinks).remainder(window)).float()
        firsts = torch.where((first < start[:, None])[..., None, None], cache[:, :sinks].float(), here)
        return torch.cat([past, new_f, tail], 1), firsts

    kk, k0 = keys(k, s["k_cache"])
    vv, v0 = keys(v, s["v_cache"])
    band = window + QBLOCK
    qp = torch.cat([q.float(), q.new_zeros(B, pad, H, d, dtype=torch.float32)], 1)
    qb = qp.view(B, nb, QBLOCK, Hkv, R, d).permute(0, 1, 3, 4, 2, 5).reshape(B, nb, Hkv, R * QBLOCK, d) * s["scale"]
    kb = kk.unfold(1, band, QBLOCK).contiguous()                        # [B, nb, Hkv, d, band]
    vb = vv.unfold(1, band, QBLOCK).transpose(-1, -2).contiguous()      # [B, nb, Hkv, band, d]
    qpos = start[:, None, None] + torch.arange(nb * QBLOCK, device=dev).view(nb, QBLOCK)   # [B, nb, QBLOCK]
    kpos = (start[:, None, None] - window + torch.arange(nb, device=dev)[:, None] * QBLOCK
            + torch.arange(band, device=dev))                                              # [B, nb, band]
    gap = qpos[..., :, None] - kpos[..., None, :]
    see = (gap >= 0) & (gap < window) & (kpos >= sinks)[..., None, :]
    see0 = qpos[..., None] >= torch.arange(sinks, device=dev)
    scores = torch.cat([torch.matmul(qb, kb), torch.matmul(qb, k0.permute(0, 2, 3, 1).contiguous()[:, None])], -1)
    see = torch.cat([see, see0], -1)[:, :, None, None]                                     # [B, nb, 1, 1, Q, keys]
    scores = scores.unflatten(-2, (R, QBLOCK)).masked_fill_(~see, -math.inf)
    scores = torch.exp_(scores.sub_(scores.amax(-1, keepdim=True))).flatten(-3, -2)
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores[..., :band], vb) + torch.matmul(scores[..., band:], v0.permute(0, 2, 1, 3).contiguous()[:, None])
    out = (out / total).unflatten(-2, (R, QBLOCK)).permute(0, 1, 4, 2, 3, 5).reshape(B, nb * QBLOCK, H, d)[:, :T]
    s["o"].copy_(torch.where(alive[..., None, None], out, s["o"].float()))
    if s["k_cache"] is not None:
        # the newest token of each slot, where there is one among the new ones
        last = start + alive.sum(1) - 1
        slot = torch.arange(sinks + window, device=dev)
        ring = last[:, None] - (last[:, None] - slot).remainder(window)
        newest = torch.where(slot < sinks, slot, ring)
        fresh = (newest >= start[:, None]) & (newest <= last[:, None]) & ((slot < sinks) | (newest >= sinks))
        at = (newest - start[:, None]).clamp(0, T - 1)
        for cache, new in ((s["k_cache"], k), (s["v_cache"], v)):
            cache.copy_(torch.where(fresh[..., None, None], pick(new, at), cache))
    return s["o"], s["k_cache"], s["v_cache"]


def _window_step(s):
    q, window, sinks = s["q"].float(), s["window"], s["sinks"]
    N, H, d = q.shape
    Hkv = s["k"].shape[1]
    pos = s["pos"].long()
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks).remainder(window))
    row = torch.arange(N, device=q.device)
    s["k_cache"][row, slot] = s["k"]
    s["v_cache"][row, slot] = s["v"]
    seen = torch.arange(sinks + window, device=q.device) <= pos[:, None]   # slots fill in order
    qg = q.view(N, Hkv, H // Hkv, d) * s["scale"]
    scores = torch.matmul(qg, s["k_cache"].float().permute(0, 2, 3, 1).contiguous())
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    scores = torch.exp(scores - scores.amax(-1, keepdim=True))
    out = torch.matmul(scores, s["v_cache"].float().permute(0, 2, 1, 3).contiguous()) / scores.sum(-1, keepdim=True)
    return out.view(N, H, d).to(s["dtype"]), s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("conv_prefill", "conv_step"):
        D, W = case["D"], case["W"]
        if op == "conv_step":
            return {"bytes": e * (case["N"] * D * 2 * W + D * (W + 1)), "flops": 2 * case["N"] * D * W}
        rows = case["B"] * case["T"] * (0.5 if case["ragged"] else 1)
        keep = case["B"] * (W - 1) * D * (2 if case["state"] else 1)
        return {"bytes": e * (rows * 2 * D + keep + D * (W + 1)), "flops": 2 * rows * D * W}
    if op in ("ssm_prefill", "ssm_step"):
        H, G, n, p = case["H"], case["G"], case["n"], case["p"]
        per = e * (H * p * (3 if case["gated"] else 2) + 2 * G * n + H)
        if op == "ssm_step":
            N = case["N"]
            return {"bytes": N * (per + 8 * H * n * p), "flops": 5 * N * H * n * p}
        rows = case["B"] * case["T"] * (0.5 if case["ragged"] else 1)
        # per token and head in blocks of 64: the causal half of C B^T and of its product with x,
        # the read of the state and its update
        flops = rows * H * (CHUNK * (n + p) + 4 * n * p)
        return {"bytes": rows * per + case["B"] * 4 * H * n * p * (2 if case["state"] else 1), "flops": flops}
    H, Hkv, d, window, sinks = (case[k] for k in ("H", "Hkv", "d", "window", "sinks"))
    if op == "window_step":
        N, slots = case["N"], sinks + window
        return {"bytes": N * e * (2 * slots * Hkv * d + 2 * H * d + 2 * Hkv * d), "flops": 4 * N * H * d * slots}
    share = 0.5 if case["ragged"] else 1
    rows = case["B"] * case["T"] * share
    T = case["T"] * share
    # visible keys over all queries: a ramp up to the window when nothing lies before, then the window
    full = window + sinks
    if case["cache"] and case["ragged"]:
        pairs = rows * min(full, full * 0.75 + T / 2)
    elif T <= full:
        pairs = case["B"] * T * (T + 1) / 2
    else:
        pairs = case["B"] * (full * (full + 1) / 2 + (T - full) * full)
    kept = case["B"] * min(T, full) * 2 * Hkv * d if case["cache"] else 0
    past = case["B"] * full * 0.75 * 2 * Hkv * d if case["cache"] and case["ragged"] else 0
    return {"bytes": e * (rows * (2 * H * d + 2 * Hkv * d) + kept + past), "flops": 4 * pairs * H * d}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, token by token (scan) or head by head (attention)."""
    s = prepare(case, seed)
    f = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    op = case["op"]
    if op in ("conv_prefill", "conv_step"):
        return _exact_conv(f, op == "conv_step")
    if op in ("ssm_prefill", "ssm_step"):
        return _exact_ssm(f, op == "ssm_step")
    if op == "window_step":
        f = dict(f, q=f["q"][:, None], k=f["k"][:, None], v=f["v"][:, None], start=f["pos"], lens=None, o=None)
        o, kc, vc = _exact_window(f)
        return o[:, 0], kc, vc
    return _exact_window(f)


def _exact_conv(f, step):
    x = f["x"][:, None] if step else f["x"]
    B, T, D = x.shape
    W = f["w"].shape[1]
    lens = [T] * B if step or f["lens"] is None else f["lens"].tolist()
    state = torch.zeros(B, W - 1, D, dtype=torch.float64, device=x.device) if f["state"] is None else f["state"]
    y = torch.zeros(B, T, D, dtype=torch.float64, device=x.device)
    kept = torch.empty_like(state)
    for b in range(B):
        line = torch.cat([state[b], x[b, :lens[b]]])
        acc = f["bias"].expand(lens[b], D).clone()
        for j in range(W):
            acc += line[j:j + lens[b]] * f["w"][:, j]
        y[b, :lens[b]] = acc * torch.sigmoid(acc) if f["silu"] else acc
        kept[b] = line[lens[b]:]
    return (y[:, 0] if step else y), kept


def _exact_ssm(f, step):
    x, dt, bm, cm = ((f[k][:, None] if step else f[k]) for k in ("x", "dt", "Bm", "Cm"))
    B, T, H, p = x.shape
    G, n = bm.shape[-2:]
    if B * T * H * n * p > 1 << 37:
        return None   # longer than a check may take
    lens = None if step else f["lens"]
    delta = torch.nn.functional.softplus(dt + f["dt_bias"].to(torch.float64), threshold=700)
    decay = torch.exp(delta * f["A"])
    S = torch.zeros(B, G, H // G, n, p, dtype=torch.float64, device=x.device)
    if f["S"] is not None:
        S += f["S"].view_as(S)
    y = torch.zeros(B, T, H, p, dtype=torch.float64, device=x.device)
    u = (delta[..., None] * x).view(B, T, G, H // G, 1, p)
    decay = decay.view(B, T, G, H // G, 1, 1)
    bm, cm = bm[:, :, :, None, :, None], cm[:, :, :, None, None, :]
    for t in range(T):
        new = torch.addcmul(decay[:, t] * S, bm[:, t], u[:, t])
        S = new if lens is None else torch.where((lens > t).view(B, 1, 1, 1, 1), new, S)
        y[:, t] = torch.matmul(cm[:, t], S).view(B, H, p)
    y = y + f["D"][:, None] * x
    if f["z"] is not None:
        z = f["z"][:, None] if step else f["z"]
        y = y * z * torch.sigmoid(z)
    if lens is not None:
        y = torch.where((torch.arange(T, device=x.device)[None] < lens[:, None])[..., None, None], y, 0.0)
    return (y[:, 0] if step else y), S.reshape(B, H, n, p)


def _exact_window(f):
    q, k, v, window, sinks = f["q"], f["k"], f["v"], f["window"], f["sinks"]
    B, T, H, d = q.shape
    R, dev = H // k.shape[2], q.device
    lens = [T] * B if f["lens"] is None else f["lens"].tolist()
    start = [0] * B if f["start"] is None else f["start"].tolist()
    out = torch.zeros(B, T, H, d, dtype=torch.float64, device=dev)
    kc, vc = (None if f[c] is None else f[c].clone() for c in ("k_cache", "v_cache"))

    def slots(p):
        return torch.where(p < sinks, p, sinks + (p - sinks) % window)

    for b in range(B):
        if not lens[b]:
            continue
        s0, m = start[b], lens[b]
        old = torch.cat([torch.arange(min(sinks, s0)), torch.arange(max(sinks, s0 - window), max(sinks, s0))]).to(dev)
        new = torch.arange(s0, s0 + m, device=dev)
        at = torch.cat([old, new])
        kb = k[b, :m] if not len(old) else torch.cat([f["k_cache"][b, slots(old)], k[b, :m]])
        vb = v[b, :m] if not len(old) else torch.cat([f["v_cache"][b, slots(old)], v[b, :m]])
        gap = new[:, None] - at
        hidden = (gap < 0) | ((gap >= window) & (at >= sinks))
        for h in range(H):
            w = torch.matmul(q[b, :m, h], kb[:, h // R].t().contiguous()) * f["scale"]
            w = torch.softmax(w.masked_fill_(hidden, -math.inf), -1)
            out[b, :m, h] = torch.matmul(w, vb[:, h // R].contiguous())
        if kc is not None:
            keep = new[(new < sinks) | (new >= s0 + m - window)]
            kc[b, slots(keep)] = k[b, keep - s0]
            vc[b, slots(keep)] = v[b, keep - s0]
    return out, kc, vc
