"""The gated delta rule on the device against its definition in 64 bits.

Tolerances.  u = 2^-24, h the half step of the output's type, N the largest norm of a head's state over the prompt
(its entry state among them).  With decays and beta |k|^2 <= 1 every token's transition is a contraction, so an error of
the state does not grow.  On the state's path (K S0, the inverse, its product, the update) each stage sums at most dk + C = 192
products of 24-bit factors; their roundings are independent, with a deviation of sqrt(192) u / sqrt(3) of the norm of
what they sum, five such stages one after the other: five deviations together are 5 sqrt(5) sqrt(192 / 3) u =
90 u = 5.4e-6.  So |S_T - ref|_F <= 90 u N, and an fp32 output, one more sum with |q|, is off by 90 u |q| N + h |o|.
With bf16 inputs an output is formed from the state at the entry of its block of 64 rounded once, from the weights
w_ij = 2^(c_i - c_j) (q_i . k_j) rounded once, and from u_j in 16 bits: (h (1 + h) + 2^-16) (2^(c_i) |S0|^T |q_i| + sum_j |w_ij| |u_j|)
more.  One token is a single sum over dk terms: 2 (dk + 8) u of the terms' absolute values.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U90 = 90 * ref.U32


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _inputs(seed, dtype, B, T, H, Hk, dk, dv, strong=False):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = rnd(B, T, 2 * Hk * dk + H * dv)
    qk = rows[..., :2 * Hk * dk].view(B, T, 2 * Hk, dk)
    qk /= qk.norm(dim=-1, keepdim=True) * 1.01        # (|k| stays at most 1 after its rounding)
    rows = rows.to(DT[dtype])
    decay = -torch.rand(B, T, H, generator=g) * (60.0 if strong else 0.3)
    if strong:
        decay[torch.rand(B, T, H, generator=g) < 0.6] = -0.01
        decay[torch.rand(B, T, H, generator=g) < 0.05] = -float("inf")
        decay[torch.rand(B, T, H, generator=g) < 0.05] = 0.0
    return rows, decay, torch.rand(B, T, H, generator=g), rnd(B, H, dk, dv)


def _split(rows, H, Hk, dk, dv):
    n = Hk * dk
    return rows[..., :n].unflatten(-1, (Hk, dk)), rows[..., n:2 * n].unflatten(-1, (Hk, dk)), rows[..., 2 * n:].unflatten(-1, (H, dv))


def _norms(q, k, v, g, beta, S0, lens, chunk):
    """The recurrence in 64 bits, with the state's largest norm per head and the terms of each output."""
    q, k, v, g, beta = (ref.f64(t) for t in (q, k, v, g, beta))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    S = np.zeros((B, H, dk, dv)) if S0 is None else ref.f64(S0).copy()
    o, terms = np.full(v.shape, np.nan), np.full(v.shape, np.nan)
    top = np.sqrt((S ** 2).sum((2, 3)))
    for b in range(B):
        for t in range(T if lens is None else lens[b]):
            kk, qq = np.repeat(k[b, t], H // Hk, 0), np.repeat(q[b, t], H // Hk, 0)
            a = np.exp(g[b, t])[:, None, None]
            if t % chunk == 0:
                first, us, ks, cs = S[b].copy(), [], [], []
            S[b] = a * S[b]
            w = beta[b, t][:, None] * (v[b, t] - np.einsum("hk,hkv->hv", kk, S[b]))
            S[b] += kk[:, :, None] * w[:, None]
            first = a * first                              # 2^(c_i) S0
            cs = [a[:, :, 0] * c for c in cs] + [np.ones((H, 1))]
            us.append(np.abs(w))
            ks.append(kk)
            o[b, t] = np.einsum("hk,hkv->hv", qq, S[b])
            terms[b, t] = np.einsum("hk,hkv->hv", np.abs(qq), np.abs(first))
            for c, kj, uj in zip(cs, ks, us):
                terms[b, t] += c * np.abs((qq * kj).sum(-1, keepdims=True)) * uj
            top[b] = np.maximum(top[b], np.sqrt((S[b] ** 2).sum((1, 2))))
    return o, terms, S, top, np.sqrt((q ** 2).sum(-1))


def _check(o, S, q, k, v, g, beta, S0, lens, dtype, more=1.0):
    want, terms, S_ref, top, nq = _norms(q, k, v, g, beta, S0, lens, 64)
    h = ref.half_step(DT[dtype])
    R = v.shape[2] // q.shape[2]
    tol = more * U90 * (np.repeat(nq, R, 2) * top[:, None])[..., None] + h * np.abs(want) + 1e-37
    if dtype == "bf16":
        tol = tol + (h * (1 + h) + 2.0 ** -16) * terms
    live = ~np.isnan(want)
    err = np.abs(ref.f64(o) - want)
    assert np.isfinite(ref.f64(o)[live]).all() and (err[live] <= tol[live]).all(), float((err / tol)[live].max())
    if S is not None:
        off = np.sqrt(((ref.f64(S) - S_ref) ** 2).sum((2, 3)))
        assert (off <= more * U90 * top + 1e-37).all(), float((off / (more * U90 * top + 1e-37)).max())


# B, T, H, Hk, dk, dv, dtype, state, lens, seg_len, strong decays
CASES = [
    (1, 1, 1, 1, 64, 64, "bf16", False, None, 0, False),
    (2, 63, 2, 1, 128, 128, "bf16", True, None, 0, False),
    (1, 64, 3, 3, 64, 128, "bf16", True, None, 0, False),
    (2, 130, 4, 2, 128, 64, "bf16", True, [130, 65], 0, False),
    (3, 200, 6, 2, 64, 64, "bf16", False, [0, 200, 1], 0, True),
    (2, 150, 2, 2, 128, 128, "f32", True, [150, 33], 0, False),
    (1, 97, 4, 1, 64, 128, "f32", False, None, 0, True),
    (2, 31, 2, 1, 128, 64, "f32", True, None, 0, False),
    (2, 333, 2, 1, 128, 128, "bf16", True, [333, 100], 64, False),       # split; a segment without tokens
    (1, 400, 4, 4, 64, 128, "bf16", False, None, 128, False),
    (2, 260, 2, 2, 128, 64, "f32", True, [200, 64], 64, False),
    (1, 300, 2, 1, 64, 64, "f32", False, None, 128, True),
    (1, 300, 3, 1, 128, 128, "bf16", True, None, 192, True),
    (150, 70, 2, 1, 64, 128, "bf16", True, None, 0, False),              # enough heads for 128 columns a workgroup
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])) + f"-{c[9]}-{int(c[10])}")
def test_delta_prefill_matches_definition(case):
    kda = _kda()
    B, T, H, Hk, dk, dv, dtype, state, lens, seg, strong = case
    print("delta_prefill", case, flush=True)
    rows, g, beta, S0 = _inputs(1, dtype, B, T, H, Hk, dk, dv, strong)
    for b, n in enumerate(lens or []):                       # padding holds NaN
        rows[b, n:], g[b, n:], beta[b, n:] = float("nan"), float("nan"), float("nan")
    args = (*_split(rows, H, Hk, dk, dv), g, beta)
    S0 = S0 if state else None
    o = torch.full((B, T, H, dv), 9.0, dtype=DT[dtype], device="cuda")
    need = kda.delta_workspace_bytes(B, T, H, Hk, dk, dv, DT[dtype], seg)
    assert (need > 0) == (seg > 0) or seg == 0
    ws = torch.full((max(1, need // 4),), float("nan"), device="cuda")
    dr = rows.cuda()
    got, S_T = kda.delta_prefill(*_split(dr, H, Hk, dk, dv), g.cuda(), beta.cuda(), None if S0 is None else S0.cuda(), seg_len=seg, o=o,
                                 lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"), workspace=ws)
    torch.cuda.synchronize()
    assert got is o
    _check(o, S_T, *args, S0, lens, dtype)
    for b, n in enumerate(lens or []):
        assert bool((o[b, n:] == 9.0).all())


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("f32", 64, 128), ("bf16", 64, 64)])
def test_delta_prefill_split_with_dead_and_living_segments(dtype, dk, dv):
    """Segments over which decays leave nothing of a state (their transitions are not formed, and their own states are run
    from where it matters), others that keep it, in any order, and more of them than a wave has lanes."""
    kda = _kda()
    B, T, H, Hk, seg = 2, 70 * 64 + 5, 2, 1, 64
    rows, g, beta, S0 = _inputs(8, dtype, B, T, H, Hk, dk, dv)
    g = g * 0.1                                              # about 2^-1 a segment
    for b, h, s in ((0, 0, 3), (0, 0, 4), (0, 0, 6), (0, 1, 0), (1, 0, 68), (1, 1, 1), (1, 1, 3), (1, 1, 5)):
        g[b, s * seg + 20:s * seg + 40, h] = -6.0            # 2^-173
    g[1, 64 * 64:64 * 64 + 64, 1] = -1.4                     # 2^-129 over a whole segment
    dr = rows.cuda()
    o, S_T = kda.delta_prefill(*_split(dr, H, Hk, dk, dv), g.cuda(), beta.cuda(), S0.cuda(), seg_len=seg)
    torch.cuda.synchronize()
    _check(o, S_T, *_split(rows, H, Hk, dk, dv), g, beta, S0, None, dtype)


@pytest.mark.parametrize("dtype,seg", [("bf16", 0), ("bf16", 64), ("f32", 0)])
def test_delta_prefill_of_near_parallel_keys(dtype, seg):
    """Keys in groups of near-parallel vectors, beta up to 1 and hardly any decay: A's entries lie near beta, the inverse
    has large alternating ones.  The transitions are contractions still; the inverse's own conditioning is counted by
    what the definition's results change under one rounding to fp32 of k, v, beta and g (largest of three draws), for each of
    the 64 tokens of a block."""
    kda = _kda()
    B, T, H, Hk, dk, dv = 1, 200, 4, 2, 128, 64
    g0 = torch.Generator().manual_seed(5)
    rows, g, beta, S0 = _inputs(2, dtype, B, T, H, Hk, dk, dv)
    q, k, v = _split(rows, H, Hk, dk, dv)
    base = torch.randn(B, T // 8, 1, Hk, dk, generator=g0).expand(B, T // 8, 8, Hk, dk).reshape(B, T, Hk, dk)
    near = base / base.norm(dim=-1, keepdim=True) + 0.02 * torch.randn(B, T, Hk, dk, generator=g0) / dk ** 0.5
    k.copy_(near / near.norm(dim=-1, keepdim=True) / 1.01)
    g = g * 0.01
    _, _, S_ref, top, _ = _norms(q, k, v, g, beta, S0, None, 64)
    sigma = 0.0
    for i in range(3):
        p = torch.Generator().manual_seed(i)
        off = lambda t: t.double() * (1 + ref.U32 * (2 * torch.rand(t.shape, generator=p, dtype=torch.float64) - 1))  # noqa: E731
        _, _, S2, _, _ = _norms(q, off(k), off(v), off(g), off(beta), S0, None, 64)
        sigma = max(sigma, float((np.sqrt(((S2 - S_ref) ** 2).sum((2, 3))) / top).max()))
    dr = rows.cuda()
    o, S_T = kda.delta_prefill(*_split(dr, H, Hk, dk, dv), g.cuda(), beta.cuda(), S0.cuda(), seg_len=seg)
    torch.cuda.synchronize()
    print("sigma", sigma, flush=True)
    _check(o, S_T, q, k, v, g, beta, S0, None, dtype, more=1 + 64 * sigma / U90)


@pytest.mark.parametrize("N,H,Hk,dk,dv,dtype", [(1, 1, 1, 64, 64, "bf16"), (3, 6, 2, 128, 128, "bf16"), (2, 4, 4, 64, 128, "f32"),
                                                (5, 3, 1, 128, 64, "f32"), (9, 56, 28, 128, 128, "bf16")])
def test_delta_step_matches_definition(N, H, Hk, dk, dv, dtype):
    kda = _kda()
    print("delta_step", N, H, Hk, dk, dv, dtype, flush=True)
    rows, g, beta, S = _inputs(3, dtype, N, 1, H, Hk, dk, dv, strong=True)
    args = (*_split(rows, H, Hk, dk, dv), g, beta)
    want, mag, S_ref, M = lref.delta(*args, S)
    Sd, dr = S.cuda(), rows.cuda()
    o = torch.full((N, H, dv), 9.0, dtype=DT[dtype], device="cuda")
    kda.delta_step(*(t[:, 0] for t in _split(dr, H, Hk, dk, dv)), g[:, 0].cuda(), beta[:, 0].cuda(), Sd, o=o)
    torch.cuda.synchronize()
    e = 2 * (dk + 8) * ref.U32
    assert (np.abs(ref.f64(Sd) - S_ref) <= e * M + 1e-37).all()
    assert (np.abs(ref.f64(o) - want[:, 0]) <= 2 * e * mag[:, 0] + ref.half_step(DT[dtype]) * np.abs(want[:, 0]) + 1e-37).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prompt_in_pieces_then_tokens(dtype):
    """Pieces that hand their state on, then tokens, against the whole in one: the state of every boundary."""
    kda = _kda()
    B, T, H, Hk, dk, dv = 2, 203, 4, 2, 128, 128
    rows, g, beta, S0 = _inputs(4, dtype, B, T, H, Hk, dk, dv)
    dr, gd, bd, S = rows.cuda(), g.cuda(), beta.cuda(), S0.cuda()
    at, outs = 0, []
    for n in (1, 64, 100, 35):
        part = slice(at, at + n)
        o, S2 = kda.delta_prefill(*_split(dr[:, part].contiguous(), H, Hk, dk, dv), gd[:, part].contiguous(), bd[:, part].contiguous(), S, S_T=S)
        assert S2 is S
        outs.append(o)
        at += n
    for t in range(at, T):
        outs.append(kda.delta_step(*(x[:, t] for x in _split(dr, H, Hk, dk, dv)), gd[:, t].contiguous(), bd[:, t].contiguous(), S)[:, None])
    torch.cuda.synchronize()
    # blocks begin elsewhere than in one call: a rounded entry state of either is within the terms below, twice
    o = torch.cat(outs, 1)
    want, terms, S_ref, top, nq = _norms(*_split(rows, H, Hk, dk, dv), g, beta, S0, None, 1)
    off = np.sqrt(((ref.f64(S) - S_ref) ** 2).sum((2, 3)))
    assert (off <= U90 * top).all()
    if dtype == "f32":
        assert (np.abs(ref.f64(o) - want) <= U90 * (np.repeat(nq, H // Hk, 2) * top[:, None])[..., None] + 1e-37).all()


def test_no_tokens_and_no_state():
    kda = _kda()
    rows, g, beta, S0 = _inputs(6, "bf16", 2, 5, 2, 1, 64, 128)
    q, k, v = (t.cuda() for t in _split(rows, 2, 1, 64, 128))
    o, S = kda.delta_prefill(q[:, :0], k[:, :0], v[:, :0], g[:, :0].cuda(), beta[:, :0].cuda(), S0.cuda())
    _, Z = kda.delta_prefill(q[:, :0], k[:, :0], v[:, :0], g[:, :0].cuda(), beta[:, :0].cuda())
    a, none = kda.delta_prefill(q, k, v, g.cuda(), beta.cuda(), S0.cuda(), return_state=False)
    b, _ = kda.delta_prefill(q, k, v, g.cuda(), beta.cuda(), S0.cuda())
    torch.cuda.synchronize()
    assert o.shape == (2, 0, 2, 128) and torch.equal(S.cpu(), S0) and not Z.any() and none is None and torch.equal(a, b)


def test_a_value_that_is_no_number_stays_in_its_sequence_and_head():
    kda = _kda()
    B, T, H, Hk, dk, dv = 2, 200, 4, 2, 64, 64
    rows, g, beta, S0 = _inputs(7, "bf16", B, T, H, Hk, dk, dv)
    bad = rows.clone()
    _split(bad, H, Hk, dk, dv)[1][1, 100, 0] = float("nan")    # a key of sequence 1, heads 0 and 1
    res = [kda.delta_prefill(*_split(r.cuda(), H, Hk, dk, dv), g.cuda(), beta.cuda(), S0.cuda(), seg_len=64) for r in (rows, bad)]
    torch.cuda.synchronize()
    (o, S), (p, Q) = res
    assert torch.equal(o[0], p[0]) and torch.equal(S[0], Q[0])
    assert torch.equal(o[1, :, 2:], p[1, :, 2:]) and torch.equal(S[1, 2:], Q[1, 2:])
    assert torch.equal(o[1, :64], p[1, :64]) and torch.isnan(Q[1, :2]).any()
