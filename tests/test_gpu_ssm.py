"""The state space scan on the device against its definition in 64 bits.

Tolerances.  With m the sum of the absolute values of all terms behind an element (the recurrence run
on absolute values), u = 2^-24 and h the half step of the input type:
* every fp32 sum of K terms is off by at most 2 K u m (matrix cores may truncate); a token's terms pass
  through at most T + n + 128 additions, three products each in the update of the bf16 form;
* exponents are sums of up to 64 numbers reaching c, off by at most 8 u c, and as much again in the
  factors they become; softplus, silu and the exponentials add at most 32 u;
* outputs of the bf16 form: C B^T weights and the state as an operand are rounded to bf16 once each,
  2 h m at most together with the result's own rounding h |y|.
So |S - ref| <= k m with k = u (6 (T + n + 128) + 32 c), and |y - ref| <= (h' + k) m + h |y| with
h' = h (1 + h) for bf16 and 0 for fp32.  rel-L2 keeps the library's bars (bf16 1e-2, fp32 1e-4).
"""
import numpy as np
import pytest
import torch

from tests import mixers_reference as ref
from tests.parity import rel_l2

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BAR = {"bf16": 1e-2, "f32": 1e-4}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _inputs(B, T, H, G, n, p, dtype, seed, *, S0=True, gated=True, skip=True, strong=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    i = {"x": rnd(B, T, H, p).to(dt), "dt": rnd(B, T, H).to(dt), "Bm": rnd(B, T, G, n).to(dt), "Cm": rnd(B, T, G, n).to(dt),
         "A": -torch.rand(H, generator=g) * 15 - 1,
         "dt_bias": rnd(H) * (1.0 if strong else 0.3) + (1.0 if strong else -4.0)}
    i["S0"] = rnd(B, H, n, p) if S0 else None
    i["z"] = rnd(B, T, H, p).to(dt) if gated else None
    i["D"] = rnd(H) if skip else None
    return i


def _cuda(i):
    return {k: None if v is None else v.cuda() for k, v in i.items()}


def _check(i, y, S, lens, dtype):
    T, n = i["x"].shape[1], i["Bm"].shape[-1]
    want, mag, S_ref, S_mag, c = ref.ssm(**i, lens=lens)
    k = ref.U32 * (6 * (T + n + 128) + 32 * c)
    h = ref.half_step(DT[dtype]) if dtype == "bf16" else 0.0
    if S is not None:
        d = np.abs(ref.f64(S) - S_ref)
        assert (d <= k * S_mag + 1e-30).all(), float((d / (k * S_mag + 1e-30)).max())
        assert rel_l2(S, S_ref) <= 1e-4
    live = ~np.isnan(want)
    g = ref.f64(y)
    d = np.abs(g - want)[live]
    tol = ((h * (1 + h) + k) * mag + ref.half_step(DT[dtype]) * np.abs(want))[live] + 1e-30
    assert (d <= tol).all(), float((d / tol).max())
    if live.any():
        assert rel_l2(g[live], want[live]) <= BAR[dtype]


# B, T, H, G, n, p, dtype, S0, gated, skip, strong, lens, seg_len
CASES = [
    (1, 1, 1, 1, 64, 64, "bf16", True, True, True, False, None, 0),
    (2, 63, 2, 1, 128, 64, "bf16", False, True, True, False, None, 0),
    (1, 64, 2, 2, 64, 128, "bf16", True, False, False, False, None, 0),
    (2, 65, 3, 1, 128, 128, "bf16", True, True, True, False, None, 0),
    (1, 65, 3, 1, 128, 128, "f32", True, True, True, False, None, 0),
    (3, 200, 4, 2, 128, 128, "bf16", True, True, True, False, [0, 200, 129], 0),
    (3, 200, 4, 4, 128, 64, "bf16", True, True, False, True, [1, 64, 300], 64),   # 300 is clamped to T
    (2, 333, 2, 1, 64, 64, "bf16", False, False, True, True, [333, -2], 128),     # -2 is clamped to 0
    (1, 520, 6, 2, 128, 128, "bf16", True, True, True, False, None, 64),
    (2, 150, 2, 1, 64, 64, "f32", True, True, True, True, [150, 70], 64),
    (1, 190, 2, 1, 64, 128, "f32", True, True, True, False, None, 128),
    (1, 190, 2, 2, 128, 64, "f32", False, False, False, False, None, 64),
    (1, 2500, 1, 1, 128, 64, "bf16", True, True, True, False, None, 0),           # split by the plan
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])) + f"-seg{c[-1]}")
def test_ssm_prefill_matches_definition(case):
    kda = _kda()
    B, T, H, G, n, p, dtype, S0, gated, skip, strong, lens, seg = case
    print("ssm_prefill", case, flush=True)
    i = _inputs(B, T, H, G, n, p, dtype, 11, S0=S0, gated=gated, skip=skip, strong=strong)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    y = torch.full((B, T, H, p), 5.0, dtype=DT[dtype], device="cuda")
    S = torch.full((B, H, n, p), float("nan"), device="cuda")
    kda.ssm_prefill(**_cuda(i), lens=None if ln is None else ln.cuda(), seg_len=seg, y=y, S_T=S)
    torch.cuda.synchronize()
    _check(i, y, S, ln, dtype)
    for b, m in enumerate(ref.lens_of(ln, B, T)):
        assert bool((y[b, m:] == 5.0).all())


def test_ssm_prefill_automatic_plan_splits():
    kda = _kda()
    assert kda.ssm_workspace_bytes(1, 2500, 1, 1, 128, 64) > 0
    assert kda.ssm_workspace_bytes(1, 64, 1, 1, 128, 64) == 0


@pytest.mark.parametrize("seg", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prefill_slices_in_place_and_nan_in_the_padding(dtype, seg):
    """x, B and C cut from one buffer's rows, z and dt from another's, NaN in every row behind a
    sequence's end; the state updated in place."""
    kda = _kda()
    B, T, H, G, n, p = 2, 230, 3, 1, 64, 64
    dt = DT[dtype]
    lens = torch.tensor([230, 97], dtype=torch.int32)
    i = _inputs(B, T, H, G, n, p, dtype, 12)
    nan = float("nan")
    xbc = torch.full((B, T, H * p + 2 * G * n), nan, dtype=dt)
    zdt = torch.full((B, T, H * p + 8), nan, dtype=dt)
    for b in range(B):
        m = int(lens[b])
        xbc[b, :m] = torch.cat([i[k][b, :m].flatten(1) for k in ("x", "Bm", "Cm")], 1)
        zdt[b, :m, :H * p] = i["z"][b, :m].flatten(1)
        zdt[b, :m, H * p:H * p + H] = i["dt"][b, :m]
    xbc, zdt = xbc.cuda(), zdt.cuda()
    d = _cuda(i)
    S = d["S0"].clone()
    y, S2 = kda.ssm_prefill(xbc[..., :H * p].unflatten(-1, (H, p)), zdt[..., H * p:H * p + H], d["A"],
                            xbc[..., H * p:H * p + n].unflatten(-1, (G, n)), xbc[..., H * p + n:].unflatten(-1, (G, n)), S,
                            D=d["D"], z=zdt[..., :H * p].unflatten(-1, (H, p)), dt_bias=d["dt_bias"], lens=lens.cuda(),
                            seg_len=seg, S_T=S)
    torch.cuda.synchronize()
    assert S2 is S
    _check(i, y, S, lens, dtype)


def test_ssm_prefill_without_state_and_empty_calls():
    kda = _kda()
    i = _cuda(_inputs(2, 70, 2, 1, 64, 64, "bf16", 13))
    y0, S = kda.ssm_prefill(**i)
    y1, none = kda.ssm_prefill(**i, return_state=False)
    assert none is None and torch.equal(y0, y1)
    e = {k: (v[:, :0] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in i.items()}
    y, S = kda.ssm_prefill(**e)
    assert y.shape == (2, 0, 2, 64) and torch.equal(S, i["S0"])
    y, S = kda.ssm_prefill(**dict(e, S0=None))
    assert bool((S == 0).all())
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    y, S = kda.ssm_prefill(**i, lens=lens, y=torch.full_like(i["x"], 3.0), seg_len=64)
    assert torch.equal(S, i["S0"]) and bool((y == 3.0).all())


def test_ssm_prefill_two_runs_give_the_same_bits_and_streams_are_kept():
    kda = _kda()
    i = _cuda(_inputs(1, 1000, 2, 1, 128, 128, "bf16", 14))
    y0, S0 = kda.ssm_prefill(**i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, S1 = kda.ssm_prefill(**i)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(S0, S1)


@pytest.mark.parametrize("N,H,G,n,p,dtype", [(1, 1, 1, 64, 64, "bf16"), (5, 6, 2, 128, 64, "bf16"), (3, 7, 1, 64, 128, "f32"),
                                             (9, 5, 5, 128, 128, "bf16"), (2, 56, 8, 128, 64, "f32")])
def test_ssm_step_matches_definition(N, H, G, n, p, dtype):
    kda = _kda()
    print("ssm_step", N, H, G, n, p, dtype, flush=True)
    i = _inputs(N, 1, H, G, n, p, dtype, 15)
    d = {k: (v[:, 0] if v is not None and k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in _cuda(i).items()}
    S = d.pop("S0").clone()
    y = kda.ssm_step(**d, S=S)
    torch.cuda.synchronize()
    _check(i, y[:, None], S, None, dtype)


def test_conv_and_scan_prompt_then_tokens_equal_the_whole():
    """A layer's path: projection rows -> convolution -> scan for a prompt, then token by token, against
    the definition of the whole sequence (and KDA's own convolution input stays usable beside it)."""
    kda = _kda()
    B, T, more, H, G, n, p, W = 2, 100, 4, 2, 1, 64, 64, 4
    g = torch.Generator().manual_seed(16)
    width, gate = H * p + 2 * G * n, H * p
    row = gate + width + 8
    rows = torch.randn(B, T + more, row, generator=g)
    w, bias = torch.randn(width, W, generator=g) * 0.5, torch.randn(width, generator=g) * 0.1
    i = _inputs(B, T + more, H, G, n, p, "f32", 17)
    conv, _, _, _ = ref.conv(rows[..., gate:gate + width], w, bias, None, None, True)
    conv = torch.from_numpy(conv)
    full = {"x": conv[..., :H * p].unflatten(-1, (H, p)), "Bm": conv[..., H * p:H * p + n].unflatten(-1, (G, n)),
            "Cm": conv[..., H * p + n:].unflatten(-1, (G, n)), "z": rows[..., :gate].unflatten(-1, (H, p)),
            "dt": rows[..., gate + width:gate + width + H]}
    full.update({k: i[k] for k in ("A", "D", "dt_bias", "S0")})
    r, wd, bd = rows.cuda(), w.cuda(), bias.cuda()
    c = {k: i[k].cuda() for k in ("A", "D", "dt_bias")}
    S = i["S0"].cuda()

    def mixer(part, conv_call, scan_call):
        u = conv_call(part[..., gate:gate + width])
        return scan_call(u[..., :H * p].unflatten(-1, (H, p)), part[..., gate + width:gate + width + H], c["A"],
                         u[..., H * p:H * p + n].unflatten(-1, (G, n)), u[..., H * p + n:].unflatten(-1, (G, n)), S,
                         D=c["D"], z=part[..., :gate].unflatten(-1, (H, p)), dt_bias=c["dt_bias"])

    hist = torch.empty(B, W - 1, width, device="cuda")
    y, S = mixer(r[:, :T], lambda x: kda.conv_prefill(x.contiguous(), wd, bd, state_out=hist)[0],
                 lambda *a, **k: kda.ssm_prefill(*[v.contiguous() for v in a], **{m: v.contiguous() for m, v in k.items()}))
    ys = [y]
    for t in range(T, T + more):
        ys.append(mixer(r[:, t], lambda x: kda.conv_step(x, wd, hist, bd), kda.ssm_step)[:, None])
    torch.cuda.synchronize()
    want, _, S_ref, _, _ = ref.ssm(**full)
    assert rel_l2(torch.cat(ys, 1), want) <= 1e-5 and rel_l2(S, S_ref) <= 1e-5
