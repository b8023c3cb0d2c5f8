"""The layers beside Kimi Delta Attention that a hybrid model's user needs next, as they are timed.

Five operators:

  delta_prefill, delta_step   the gated delta rule with one decay per head and token, key heads shared by
                              groups of value heads: prompts in chunks, and one token
  attn_prefill                causal attention over packed prompts of different lengths; the queries of a
                              sequence are the last ones of its keys (a prompt run in pieces has more keys)
  cache_write, cache_read     keys and values into a paged cache of 4 bits an element and back: blocks of 32
                              channels share a power of two, elements are 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign
  attn_step                   attention of one token (or a few drafted ones) per sequence over that cache

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (decay exponents in
64); with ``own`` true it calls the library.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64          # tokens per block of the plain delta rule
BLOCK = 32          # channels that share a power of two in the cache
SCORES = 1 << 30    # scores of one block of queries of the plain attention


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a short ragged batch in fp32, continued from kept states: launches and chains of a few chunks
        {"name": "delta_prefill ragged f32", "op": "delta_prefill", "B": 3, "T": 301, "H": 8, "Hk": 4, "dk": 64, "dv": 64,
         "state": True, "ragged": True, "dtype": "f32"},
        # one long prompt of odd length, few heads: the sequence itself has to fill the GPU
        {"name": "delta_prefill long", "op": "delta_prefill", "B": 1, "T": 20001, "H": 16, "Hk": 16, "dk": 128, "dv": 128,
         "state": True, "ragged": False, "dtype": "bf16"},
        # model width: 56 heads of 128 over 28 key heads, four prompts
        {"name": "delta_prefill wide", "op": "delta_prefill", "B": 4, "T": 16384, "H": 56, "Hk": 28, "dk": 128, "dv": 128,
         "state": False, "ragged": False, "dtype": "bf16"},
        # one user, one token, fp32
        {"name": "delta_step one f32", "op": "delta_step", "N": 1, "H": 56, "Hk": 28, "dk": 128, "dv": 128, "dtype": "f32"},
        # a serving batch: 256 sequences of 56 heads of 128
        {"name": "delta_step batch", "op": "delta_step", "N": 256, "H": 56, "Hk": 28, "dk": 128, "dv": 128, "dtype": "bf16"},
        # pieces of prompts behind the tokens that were read back from their caches (chunked prefill)
        {"name": "attn_prefill pieces", "op": "attn_prefill", "B": 5, "most": 1500, "least": 77, "new": 130, "H": 8, "Hkv": 2,
         "d": 64, "dtype": "bf16"},
        # a short packed batch in fp32, a prompt of one token in it
        {"name": "attn_prefill packed f32", "op": "attn_prefill", "B": 6, "most": 2000, "least": 1, "new": 0, "H": 16, "Hkv": 4,
         "d": 128, "dtype": "f32"},
        # model width: packed prompts, the longest of 16384 tokens
        {"name": "attn_prefill wide", "op": "attn_prefill", "B": 4, "most": 16384, "least": 333, "new": 0, "H": 56, "Hkv": 8,
         "d": 128, "dtype": "bf16"},
        # pieces of five prompts are kept, and their whole prefixes read back for the attention: odd sizes
        {"name": "cache pieces f32", "op": "cache", "B": 5, "most": 700, "least": 40, "new": 111, "Hkv": 2, "d": 64, "page": 16,
         "dtype": "f32"},
        # a layer's long prompts at model width, kept and read back
        {"name": "cache wide", "op": "cache", "B": 4, "most": 16384, "least": 8000, "new": 16384, "Hkv": 8, "d": 128, "page": 64,
         "dtype": "bf16"},
        # one user, one token behind a long context: few rows, a long axis
        {"name": "attn_step one", "op": "attn_step", "N": 1, "m": 1, "most": 32777, "least": 32777, "H": 56, "Hkv": 8, "d": 128,
         "page": 64, "dtype": "bf16"},
        # a serving batch of 64 sequences of different lengths
        {"name": "attn_step batch", "op": "attn_step", "N": 64, "m": 1, "most": 16384, "least": 1000, "H": 56, "Hkv": 8, "d": 128,
         "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_prefill", "delta_prefill", "delta_step", "attn_prefill", "attn_prefill", "cache", "attn_step",
                     "attn_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("delta"):
        Hk = _log(rng, 1, 28)
        H = Hk * rng.choice([1, 1, 2, 2, 3, 4])
        dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        if op == "delta_step":
            return {"op": op, "N": max(1, min(_log(rng, 1, 512), 14000 // H)), "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype}
        T = _log(rng, 1, 20000 if dtype == "bf16" else 4096)
        B = max(1, min(_log(rng, 1, 16), (3 << 20 if dtype == "bf16" else 1 << 18) // (H * T)))
        return {"op": op, "B": B, "T": T, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "state": rng.random() < 0.6,
                "ragged": rng.random() < 0.5, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "attn_prefill":
        most = _log(rng, 1, 16384 if dtype == "bf16" else 3000)
        B = max(1, min(_log(rng, 1, 32), (3 << 30) // (H * most * most)))
        return {"op": op, "B": B, "most": most, "least": _log(rng, 1, most), "new": rng.choice([0, 0, _log(rng, 1, most)]), "H": H,
                "Hkv": Hkv, "d": d, "dtype": dtype}
    if op == "cache":
        most = _log(rng, 1, 16384)
        B = max(1, min(_log(rng, 1, 64), (24 << 20) // (Hkv * d * most)))
        return {"op": op, "B": B, "most": most, "least": _log(rng, 1, most), "new": _log(rng, 1, most), "Hkv": Hkv, "d": d,
                "page": page, "dtype": dtype}
    most = _log(rng, 1, 65536)
    m = rng.choice([1, 1, 1, 2, 4])
    N = max(1, min(_log(rng, 1, 256), (400 << 20) // (Hkv * d * most)))
    return {"op": op, "N": N, "m": m, "most": max(most, m), "least": max(m, _log(rng, 1, most)), "H": H, "Hkv": Hkv, "d": d,
            "page": page, "dtype": dtype}


# ----------------------------------------------------------------------------------------- inputs
def _lengths(count, most, least):
    """`count` lengths between `least` and `most`, evenly spaced over their logarithm."""
    if count == 1:
        return [most]
    return [max(1, round(least * (most / least) ** (i / (count - 1)))) for i in range(count)]


def _counts(case):
    """Tokens of each sequence behind the call, and the new ones among them, in the order of the case."""
    total = _lengths(case["B"], case["most"], case["least"])
    if not case["new"]:
        return total, total
    return total, [min(n, t) for n, t in zip(_lengths(case["B"], case["new"], max(1, case["new"] // 10)), reversed(total))][::-1]


def _shuffled(g, *lists):
    at = torch.randperm(len(lists[0]), generator=g, device="cuda").tolist()
    return [[x[i] for i in at] for x in lists]


def _sums(lengths):
    """[0, l0, l0 + l1, ...] as int32 on the device."""
    return torch.tensor([0] + lengths, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


def _page_table(g, lengths, page):
    """Pages for these lengths, in any order of a pool that holds some more, and how many the pool has."""
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + 3
    at = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(need), dtype=torch.int32, device="cuda")
    used = 0
    for b, n in enumerate(need):
        table[b, :n] = at[used:used + n]
        used += n
    return table, pool


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
    if op.startswith("delta"):
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        lead = (case["B"], case["T"]) if op == "delta_prefill" else (case["N"],)
        # q, k and v side by side in the convolution's rows, q and k normalised in place
        rows = normal(*lead, 2 * Hk * dk + H * dv)
        qk = rows[..., :2 * Hk * dk].unflatten(-1, (2 * Hk, dk))
        qk.copy_(qk.float() / qk.float().square().sum(-1, keepdim=True).sqrt())
        qk[..., :Hk, :].mul_(dk ** -0.5)
        s["q"], s["k"] = qk[..., :Hk, :], qk[..., Hk:, :]
        s["v"] = rows[..., 2 * Hk * dk:].unflatten(-1, (H, dv))
        # log decays -A softplus(a + bias): steps between about 0.001 and 0.1 where a is zero, A from 1 to 16
        step = torch.exp(uniform(math.log(0.001), math.log(0.1), H))
        raw = normal(*lead, H, dtype=torch.float32) + step + torch.log(-torch.expm1(-step))
        s["g"] = -uniform(1.0, 16.0, H) * torch.log1p(torch.exp(raw))
        s["beta"] = torch.sigmoid(normal(*lead, H, dtype=torch.float32))
        s["lens"] = None
        if op == "delta_prefill":
            if case["ragged"]:
                lens, = _shuffled(g, _lengths(case["B"], case["T"], max(1, case["T"] // 8)))
                s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
            s["S"] = normal(case["B"], H, dk, dv, dtype=torch.float32) if case["state"] else None
            # rows past a sequence's end keep what the buffer holds
            s["o"] = torch.zeros(*lead, H, dv, dtype=dt, device=dev)
        else:
            s["S"] = normal(case["N"], H, dk, dv, dtype=torch.float32)
        return s
    Hkv, d = case["Hkv"], case["d"]
    # a few channels of the keys are larger than the others, as positions' encodings leave them
    wide = torch.exp(normal(Hkv, d, std=0.5, dtype=torch.float32))
    if op == "attn_prefill":
        H = case["H"]
        s["nk"], s["nq"] = _shuffled(g, *_counts(case))
        s["cu_q"], s["cu_k"], s["scale"] = _sums(s["nq"]), _sums(s["nk"]), d ** -0.5
        if case["new"]:
            s["q"], k, v = normal(sum(s["nq"]), H, d), normal(sum(s["nk"]), Hkv, d), normal(sum(s["nk"]), Hkv, d)
        else:   # slices of one projection's rows
            rows = normal(sum(s["nq"]), H + 2 * Hkv, d)
            s["q"], k, v = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
        k.mul_(wide.to(dt))
        s["k"], s["v"] = k, v
        return s
    if op == "cache":
        total, new = _shuffled(g, *_counts(case))
        s["pages"], pool = _page_table(g, total, case["page"])
        s["start"] = torch.tensor([t - n for t, n in zip(total, new)], dtype=torch.int32, device=dev)
        s["cu_new"], s["cu_all"], s["total"] = _sums(new), _sums(total), sum(total)
        rows = normal(sum(new), 2 * Hkv, d)
        s["k"], s["v"] = rows[:, :Hkv], rows[:, Hkv:]
        s["k"].mul_(wide.to(dt))
    else:
        lens, = _shuffled(g, _lengths(case["N"], case["most"], case["least"]))
        s["pages"], pool = _page_table(g, lens, case["page"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"], s["scale"] = normal(case["N"], case["m"], case["H"], d), d ** -0.5
    s["d"], s["page"] = d, case["page"]
    # what the caches hold: earlier tokens, quantised
    for name, by in (("k_cache", wide), ("v_cache", None)):
        x = normal(pool, Hkv, case["page"], d, dtype=torch.bfloat16)
        codes, exps = _quantise(x if by is None else x * by[:, None].to(torch.bfloat16))
        s[name] = torch.cat([codes.flatten(2), exps.flatten(2)], -1)
    return s


# ------------------------------------------------------------------------------------ the 4-bit form
def _quantise(x):
    """x [..., d] in blocks of 32: elements [..., d / 2] bytes (even channels in the low half) and exponents
    [..., d / 32] bytes.  A block's power of two is the smallest from 2^-125 on with max |x| <= 7 2^e."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    most = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(most)                      # most = m 2^e, m in [1/2, 1); 7 = 0.875 * 2^3
    e = torch.where(most == 0, -125, e - torch.where(m <= 0.875, 3, 2)).clamp(min=-125)
    y = x.abs() * torch.exp2(-e.float())
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5)
            + (x.signbit() * 8)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).squeeze(-1).to(torch.uint8)


def _values(rows, d):
    """fp32 values of cache rows: elements [..., d / 2] followed by exponents [..., d / 32]."""
    codes, exps = rows[..., :d // 2], rows[..., d // 2:]
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=rows.device)
    return grid[code.int()] * torch.exp2(exps.float() - 127).repeat_interleave(BLOCK, -1)


def _pool_rows(cache, page, d):
    """The pool as views of its rows' elements [pages, Hkv, page, d / 2] and exponents [pages, Hkv, page, d / 32]."""
    n = page * d // 2
    return cache[..., :n].unflatten(-1, (page, d // 2)), cache[..., n:].unflatten(-1, (page, d // BLOCK))


def _places(cu, start, n, pages, page):
    """Page and row of each of n packed tokens."""
    i = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), i, right=True)
    at = i - cu[b] + (0 if start is None else start[b])
    return pages[b, at // page].long(), at % page


# -------------------------------------------------------------------------------------------- run
def run(s):
    if own:
        return _own(s)
    return {"delta_prefill": _delta_prefill, "delta_step": _delta_step, "attn_prefill": _attn_prefill, "cache": _cache,
            "attn_step": _attn_step}[s["op"]](s)


def _own(s):
    import chunked_gated_delta_13_amd as kda
    op = s["op"]
    if op == "delta_prefill":
        return kda.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], lens=s["lens"], o=s["o"])
    if op == "delta_step":
        return kda.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"]), s["S"]
    if op == "attn_prefill":
        return kda.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"])
    if op == "cache":
        kda.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["cu_new"], s["start"])
        return kda.cache_read(s["k_cache"], s["v_cache"], s["pages"], s["cu_all"], s["total"], s["d"], dtype=s["dtype"])
    return kda.attn_step(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lens"], scale=s["scale"])


def _delta_prefill(s):
    """Blocks of CHUNK tokens: inside a block by the inverse of I + A, A its decay-weighted beta K K^T, from
    block to block by the state.  Exponents are summed in 64 bits."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, T, Hk, dk = q.shape
    H, dv = v.shape[-2:]
    R, nc, dev = H // Hk, -(-T // CHUNK), q.device
    live = torch.ones(B, T, 1, dtype=torch.bool, device=dev)
    if s["lens"] is not None:
        live = (torch.arange(T, device=dev)[None] < s["lens"][:, None])[..., None]

    def blocks(x):   # [B, T, heads, w] -> [B, nc, heads, CHUNK, w], zeros behind the end
        x = torch.where(live[..., None], x, 0)
        x = torch.cat([x, x.new_zeros(B, nc * CHUNK - T, *x.shape[2:])], 1)
        return x.unflatten(1, (nc, CHUNK)).transpose(2, 3)

    qb, kb, vb = blocks(q), blocks(k), blocks(v)
    beta = blocks(s["beta"][..., None])
    cum = blocks(s["g"][..., None].double()).cumsum(-2)                                   # [B, nc, H, L, 1]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp((cum - cum.transpose(-1, -2)).masked_fill(~low, -math.inf)).float()
    kt = kb.transpose(-1, -2).contiguous()

    def per_head(x):   # key heads to value heads
        return x.repeat_interleave(R, 2) if R > 1 else x

    A = per_head(torch.matmul(kb, kt)) * decay * beta
    A = A.tril_(-1)
    mix = per_head(torch.matmul(qb, kt)) * decay
    # the inverse of I + A, from blocks of one token on: [[X, 0], [-Y L X, Y]]
    inv = torch.eye(CHUNK, device=dev).expand(A.shape).contiguous()
    for n in (1, 2, 4, 8, 16, 32):
        m = CHUNK // (2 * n)

        def part(t, i, j):   # block (i, j) of each pair of blocks on the diagonal
            t = t.unflatten(-1, (m, 2, n)).unflatten(-4, (m, 2, n))
            return t.diagonal(dim1=-6, dim2=-3)[..., i, :, j, :, :].permute(0, 1, 2, 5, 3, 4).contiguous()

        new = -torch.matmul(part(inv, 1, 1), torch.matmul(part(A, 1, 0), part(inv, 0, 0)))
        inv.unflatten(-1, (m, 2, n)).unflatten(-4, (m, 2, n)).diagonal(dim1=-6, dim2=-3)[..., 1, :, 0, :, :].copy_(
            new.permute(0, 1, 2, 4, 5, 3))
    kh, qh, grow = per_head(kb), per_head(qb), torch.exp(cum).float()
    u0 = torch.matmul(inv, beta * vb)                                                     # from zero states
    w = torch.matmul(inv, beta * grow * kh)                                               # U = u0 - w S
    late = (torch.exp(cum[..., -1:, :] - cum).float() * kh).transpose(-1, -2).contiguous()
    qg, last = grow * qh, grow[..., -1:, :]
    S = q.new_zeros(B, H, dk, dv) if s["S"] is None else s["S"]
    o = []
    for c in range(nc):
        u = u0[:, c] - torch.matmul(w[:, c], S)
        o.append(torch.matmul(qg[:, c], S) + torch.matmul(mix[:, c], u))
        S = last[:, c] * S + torch.matmul(late[:, c], u)
    o = torch.stack(o, 1).transpose(2, 3).flatten(1, 2)[:, :T]
    s["o"].copy_(torch.where(live[..., None], o, s["o"].float()))
    return s["o"], S


def _delta_step(s):
    S = s["S"]
    R = S.shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(R, 1) for n in ("q", "k"))
    S.mul_(torch.exp(s["g"])[..., None, None])
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S.add_(k[..., None] * u[..., None, :])
    return (q[..., None] * S).sum(-2).to(s["dtype"]), S


def _attn_prefill(s):
    """The packed sequences as a padded batch, a block of queries at a time."""
    q, k, v, nq, nk = s["q"], s["k"], s["v"], s["nq"], s["nk"]
    B, (H, d), Hkv, dev = len(nq), q.shape[1:], k.shape[1], q.device
    Q, K, R = max(nq), max(nk), H // Hkv

    def padded(x, cu, n):
        at = cu[:-1, None].long() + torch.arange(n, device=dev)
        return x[at.clamp(max=x.shape[0] - 1)]

    kk = padded(k, s["cu_k"], K).float().permute(0, 2, 3, 1).contiguous()                 # [B, Hkv, d, K]
    vv = padded(v, s["cu_k"], K).float().permute(0, 2, 1, 3).contiguous()
    qq = padded(q, s["cu_q"], Q).float() * s["scale"]
    back = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])            # keys before the first query
    out = torch.empty(q.shape, dtype=torch.float32, device=dev)
    step = max(1, SCORES // (B * H * K))
    for q0 in range(0, Q, step):
        q1 = min(Q, q0 + step)
        most = max(min(b, q1) + c - b for b, c in zip(nq, nk))
        qb = qq[:, q0:q1].unflatten(2, (Hkv, R)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, R * (q1 - q0), d)
        w = torch.matmul(qb, kk[..., :most].contiguous()).unflatten(2, (R, q1 - q0))
        i = torch.arange(q0, q1, device=dev)
        see = torch.arange(most, device=dev) <= (back[:, None] + i)[..., None]
        w.masked_fill_(~see[:, None, None], -math.inf)
        w = torch.exp_(w.sub_(w.amax(-1, keepdim=True))).flatten(2, 3)
        ob = torch.matmul(w, vv[:, :, :most]) / w.sum(-1, keepdim=True)
        ob = ob.unflatten(2, (R, q1 - q0)).permute(0, 3, 1, 2, 4).flatten(2, 3)           # [B, q, H, d]
        inside = i < (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
        at = (s["cu_q"][:-1, None] + i)[inside]
        out[at.long()] = ob[inside]
    return out.to(s["dtype"])


def _cache(s):
    d, page = s["d"], s["page"]
    where, row = _places(s["cu_new"], s["start"], s["k"].shape[0], s["pages"], page)
    from_, row_ = _places(s["cu_all"], None, s["total"], s["pages"], page)
    outs = []
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        codes, exps = _quantise(x)
        c, e = _pool_rows(cache, page, d)
        c[where, :, row] = codes
        e[where, :, row] = exps
        outs.append(_values(torch.cat([c[from_, :, row_], e[from_, :, row_]], -1), d).to(s["dtype"]))
    return tuple(outs)


def _attn_step(s):
    q, d, page = s["q"].float(), s["d"], s["page"]
    N, m, H, _ = q.shape
    K = s["pages"].shape[1] * page
    Hkv = s["k_cache"].shape[1]

    def rows(cache):   # [N, Hkv, K, d] in fp32
        c, e = _pool_rows(cache, page, d)
        at = s["pages"].long()
        r = torch.cat([c[at], e[at]], -1)                                                 # [N, pages, Hkv, page, bytes]
        return _values(r.transpose(1, 2).flatten(2, 3), d)

    qg = (q * s["scale"]).unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [N, Hkv, m R, d]
    w = torch.matmul(qg, rows(s["k_cache"]).transpose(-1, -2).contiguous()).unflatten(2, (m, H // Hkv))
    limit = s["lens"][:, None] - m + 1 + torch.arange(m, device=q.device)
    see = torch.arange(K, device=q.device) < limit[..., None]                             # [N, m, K]
    w = w.masked_fill(~see[:, None, :, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True)).flatten(2, 3)
    o = torch.matmul(w, rows(s["v_cache"])) / w.sum(-1, keepdim=True)
    return o.unflatten(2, (m, H // Hkv)).permute(0, 2, 1, 3, 4).reshape(N, m, H, d).to(s["dtype"])


# ------------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("delta"):
        H, Hk, dk, dv = (case[k] for k in ("H", "Hk", "dk", "dv"))
        row = e * (2 * Hk * dk + 2 * H * dv) + 8 * H
        if op == "delta_step":
            return {"bytes": case["N"] * (row + 8 * H * dk * dv), "flops": 7 * case["N"] * H * dk * dv}
        B, T = case["B"], case["T"]
        tokens = sum(_lengths(B, T, max(1, T // 8))) if case["ragged"] else B * T
        # per token and head in blocks of 64: the causal halves of K K^T, Q K^T, the inverse's and the scores'
        # products, the two reads of the state and its update
        flops = tokens * H * (CHUNK * (2 * dk + 2 * dv) + 6 * dk * dv)
        return {"bytes": tokens * row + B * 4 * H * dk * dv * (2 if case["state"] else 1), "flops": flops}
    Hkv, d = case["Hkv"], case["d"]
    packed = d / 2 + d / BLOCK
    if op == "attn_prefill":
        nk, nq = _counts(case)
        pairs = sum(q * (k - q) + q * (q + 1) / 2 for q, k in zip(nq, nk))
        return {"bytes": e * d * (2 * case["H"] * sum(nq) + 2 * Hkv * sum(nk)), "flops": 4 * pairs * case["H"] * d}
    if op == "cache":
        total, new = _counts(case)
        return {"bytes": 2 * Hkv * (sum(new) + sum(total)) * (e * d + packed), "flops": 0}
    lens = _lengths(case["N"], case["most"], case["least"])
    pairs = sum(case["m"] * n - case["m"] * (case["m"] - 1) / 2 for n in lens)
    return {"bytes": 2 * Hkv * sum(lens) * packed + 2 * e * case["N"] * case["m"] * case["H"] * d,
            "flops": 4 * pairs * case["H"] * d}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, token by token (delta rule) or sequence by sequence and head by head."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "delta_step":
        t = {k: (x[:, None] if k in ("q", "k", "v", "g", "beta") else x) for k, x in s.items()}
        o, S = _exact_delta(t)
        return o[:, 0], S
    if op == "delta_prefill":
        return _exact_delta(s)
    if op == "attn_prefill":
        return _exact_attn(s["q"].double(), s["k"].double(), s["v"].double(), s["cu_q"].tolist(), s["cu_k"].tolist(), s["scale"])
    if op == "cache":
        return _exact_cache(s)
    N, m, H, d = s["q"].shape
    lens, out = s["lens"].tolist(), []
    for b in range(N):
        kk, vv = (_exact_rows(c, s["pages"][b], s["page"], d)[:lens[b]] for c in (s["k_cache"], s["v_cache"]))
        out.append(_exact_attn(s["q"][b].double(), kk, vv, [0, m], [0, lens[b]], s["scale"]))
    return torch.stack(out)


def _exact_delta(s):
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    B, T, Hk, dk = q.shape
    H, dv = v.shape[-2:]
    if B * T * H * dk * dv > 1 << 37:
        return None   # longer than a check may take
    alpha, beta = torch.exp(s["g"].double()), s["beta"].double()
    S = torch.zeros(B, Hk, H // Hk, dk, dv, dtype=torch.float64, device=q.device)
    if s["S"] is not None:
        S += s["S"].double().view_as(S)
    o = torch.zeros(B, T, H, dv, dtype=torch.float64, device=q.device)
    lens = s["lens"]
    q, k = q[:, :, :, None, None], k[:, :, :, None, None]                                 # [B, T, Hk, 1, 1, dk]
    for t in range(T):
        P = alpha[:, t].view(B, Hk, -1, 1, 1) * S
        u = beta[:, t].view(B, Hk, -1, 1, 1) * (v[:, t].view(B, Hk, -1, 1, dv) - torch.matmul(k[:, t], P))
        P = torch.addcmul(P, k[:, t].transpose(-1, -2), u)
        S = P if lens is None else torch.where((lens > t).view(B, 1, 1, 1, 1), P, S)
        o[:, t] = torch.matmul(q[:, t], S).view(B, H, dv)
    if lens is not None:
        o = torch.where((torch.arange(T, device=q.device)[None] < lens[:, None])[..., None, None], o, 0.0)
    return o, S.reshape(B, H, dk, dv)


def _exact_attn(q, k, v, cu_q, cu_k, scale):
    out = torch.zeros_like(q)
    R = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(q.shape[1]):
            kh, vh = (x[cu_k[b]:cu_k[b + 1], h // R].contiguous() for x in (k, v))
            w = torch.matmul(q[cu_q[b]:cu_q[b + 1], h], kh.t().contiguous()) * scale
            w.masked_fill_(torch.ones(n, m, dtype=torch.bool, device=q.device).triu(m - n + 1), -math.inf)
            out[cu_q[b]:cu_q[b + 1], h] = torch.matmul(torch.softmax(w, -1), vh)
    return out


def _exact_rows(cache, pages, page, d):
    """Values [tokens, Hkv, d] of a sequence's pages, from the bits of each element: sign, two of exponent, one
    of fraction."""
    flat = cache[pages.long()]                                                            # [pages, Hkv, bytes]
    split = page * d // 2
    byte = flat[..., :split].unflatten(-1, (page, d // 2)).long()
    code = torch.stack([byte % 16, byte // 16], -1).flatten(-2)
    sign, power, half = 1 - 2 * (code // 8), code // 2 % 4, (code % 2).double()
    value = torch.where(power == 0, half / 2, (1 + half / 2) * 2.0 ** (power - 1).double()) * sign
    scale = 2.0 ** (flat[..., split:].unflatten(-1, (page, d // BLOCK)).double() - 127)
    value = value.unflatten(-1, (-1, BLOCK)) * scale[..., None]
    return value.flatten(-2).permute(0, 2, 1, 3).flatten(0, 1)


def _exact_cache(s):
    """Each new block by search: the power of two, then the nearest of the fifteen values, the even one of two."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=s["k"].device)
    cu_new, cu_all, start, outs = s["cu_new"].tolist(), s["cu_all"].tolist(), s["start"].tolist(), []
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        x = x.double().unflatten(-1, (-1, BLOCK))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -130))) - 4
        for _ in range(4):
            e = torch.where(top > 7 * 2.0 ** e, e + 1, e)
        e = e.clamp(min=-125)
        gap = ((x.abs() / 2.0 ** e)[..., None] - grid).abs()
        gap = gap + torch.tensor([0, 1, 0, 1, 0, 1, 0, 1], device=grid.device) * 1e-13    # ties to the even code
        x = (grid[gap.argmin(-1)] * torch.where(x < 0, -1.0, 1.0) * 2.0 ** e).flatten(-2)
        out = []
        for b in range(len(start)):
            out.append(_exact_rows(cache, s["pages"][b], s["page"], s["d"])[:start[b]])
            out.append(x[cu_new[b]:cu_new[b + 1]])
            assert start[b] + cu_new[b + 1] - cu_new[b] == cu_all[b + 1] - cu_all[b]
        outs.append(torch.cat(out))
    return tuple(outs)
