"""Causal attention over packed prompts on the device against its definition in 64 bits.

Tolerance.  u = 2^-24, h the half step of the input type.  A score is a sum of d products off by at most
2 (d + 8) u a, with a = scale * sum |q k|; scaling and the exponential's argument add 8 u a, so a
probability is off by at most e = u (2 d + 32) a + 40 u relative, numerator and denominator alike.  With
bf16 inputs it is rounded once (h) as an operand.  Sums over K keys add 4 K u.  With m = sum p |v|:
|o - ref| <= (2 e + h' + 4 K u) m + h |o|, h' = h (1 + h) for bf16 and 0 for fp32.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _draw(seed, dtype, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype])


def _sums(lengths, first=0):
    return np.cumsum([first] + list(lengths)).tolist()


def _inside(got, want, mag, a, d, keys, dtype):
    g, live = ref.f64(got), ~np.isnan(want)
    h = ref.half_step(DT[dtype])
    e = ref.U32 * ((2 * d + 32) * a[..., None] + 40)
    tol = (2 * e + (h * (1 + h) if dtype == "bf16" else 0) + 4 * keys * ref.U32) * mag + h * np.abs(want) + 1e-37
    err = np.abs(g - want)[live]
    assert np.isfinite(g[live]).all() and (err <= tol[live]).all(), float((err / tol[live]).max())


# queries and keys of each sequence (keys None: as many), H, Hkv, d, dtype, rows before the first sequence and behind the last
CASES = [
    ([1], None, 1, 1, 64, "bf16", 0, 0),
    ([64], None, 2, 1, 64, "bf16", 0, 0),
    ([65, 1, 0, 63], None, 4, 2, 128, "bf16", 0, 3),
    ([200], None, 3, 1, 128, "f32", 0, 0),                       # 3 rows a query: tiles end inside a query
    ([130, 7, 300], None, 8, 8, 128, "bf16", 2, 5),
    ([0, 0, 5, 0], None, 5, 1, 64, "f32", 0, 0),
    ([33, 20, 1], [200, 20, 65], 7, 1, 128, "bf16", 0, 0),       # pieces behind earlier keys
    ([33, 40, 3], [10, 39, 0], 4, 2, 64, "bf16", 1, 1),          # more queries than keys: the first see none
    ([70, 66], [2, 500], 2, 2, 128, "f32", 0, 0),
    ([1] * 70, [i % 9 for i in range(70)], 2, 1, 64, "bf16", 0, 0),   # more sequences than lanes of a wave
    ([2] * 130 + [90], None, 16, 2, 64, "bf16", 0, 0),
    ([200, 250], None, 56, 8, 128, "bf16", 0, 0),                # 64 rows a workgroup, one group of waves
    ([200, 20, 230], [210, 20, 900], 28, 4, 64, "bf16", 0, 2),
    ([130, 70], None, 24, 12, 64, "bf16", 0, 0),                 # kv heads in sets of four, and of eight
    ([90, 40, 3], None, 16, 16, 128, "f32", 0, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join([str(len(c[0])), str(sum(c[0]))] + [str(x) for x in c[2:6]]))
def test_attn_prefill_matches_definition(case):
    kda = _kda()
    nq, nk, H, Hkv, d, dtype, lead, tail = case
    print("attn_prefill", case, flush=True)
    cu_q = _sums(nq, lead)
    cu_k = cu_q if nk is None else _sums(nk, lead)
    Nq, Nk = cu_q[-1] + tail, cu_k[-1] + tail
    q, k, v = _draw(1, dtype, Nq, H, d), _draw(2, dtype, Nk, Hkv, d), _draw(3, dtype, Nk, Hkv, d)
    want, mag, a = lref.attn_prefill(q, k, v, cu_q, cu_k, d ** -0.5)
    for t, c in ((q, cu_q), (k, cu_k), (v, cu_k)):              # rows of no sequence hold NaN
        t[:c[0]], t[c[-1]:] = float("nan"), float("nan")
    o = torch.full((Nq, H, d), 9.0, dtype=DT[dtype], device="cuda")
    dev = lambda c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    got = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), dev(cu_q), None if nk is None else dev(cu_k), o=o)
    torch.cuda.synchronize()
    assert got is o
    _inside(o, want, mag, a, d, max(nk or nq), dtype)
    assert bool((o[:lead] == 9.0).all()) and bool((o[cu_q[-1]:] == 9.0).all())
    empty = np.isnan(want) | (mag == 0)
    assert (ref.f64(o)[empty & ~np.isnan(want)] == 0).all()     # none visible: zeros


@pytest.mark.parametrize("H,Hkv,d,dtype", [(56, 8, 128, "bf16"), (14, 2, 64, "bf16"), (16, 4, 128, "f32"), (6, 6, 64, "f32")])
def test_attn_prefill_of_long_prompts(H, Hkv, d, dtype):
    """128 rows a workgroup (bf16), many tiles of keys: some queries of every sequence against the definition."""
    kda = _kda()
    nq = [1500, 1, 700, 2222]
    print("attn_prefill long", H, Hkv, d, dtype, flush=True)
    cu = _sums(nq)
    rows = _draw(1, dtype, cu[-1], H + 2 * Hkv, d)                # slices of one projection's rows
    q, k, v = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
    dr = rows.cuda()
    o = kda.attn_prefill(dr[:, :H], dr[:, H:H + Hkv], dr[:, H + Hkv:], torch.tensor(cu, dtype=torch.int32, device="cuda"), scale=0.2)
    torch.cuda.synchronize()
    o = ref.f64(o)
    qq, kk, vv = ref.f64(q), ref.f64(k), ref.f64(v)
    for b, n in enumerate(nq):
        s = slice(cu[b], cu[b + 1])
        at = sorted({0, n // 3, n // 2, n - 2, n - 1, 63, 64, 127, 128} & set(range(n)))
        want, mag, a = lref.attend(qq[s][at], kk[s], vv[s], 0.2, [i + 1 for i in at])
        _inside(torch.from_numpy(o[s][at]), want, mag, a, d, n, dtype)


# few queries over many keys: ranges of keys, some of them without any
SPLITS = [
    ([1], [3000], 2, 1, 128, "bf16"),
    ([5, 3], [2000, 70], 4, 2, 64, "f32"),
    ([40, 33, 0, 17], [900, 40, 2000, 1], 4, 2, 128, "bf16"),
    ([64, 20], [100, 9000], 2, 1, 64, "bf16"),
    ([6, 9], [4, 1500], 3, 3, 128, "f32"),                        # queries that see none
]


@pytest.mark.parametrize("case", SPLITS, ids=lambda c: "-".join([str(sum(c[0])), str(sum(c[1]))] + [str(x) for x in c[2:]]))
def test_attn_prefill_split_over_ranges_matches_definition(case):
    """As above, with the smallest workspace; the same call without the split has the same bounds."""
    from chunked_gated_delta_13_amd import _lib
    kda = _kda()
    nq, nk, H, Hkv, d, dtype = case
    print("attn_prefill split", case, flush=True)
    cu_q, cu_k = _sums(nq, 1), _sums(nk)
    Nq, Nk = cu_q[-1] + 2, cu_k[-1]
    q, k, v = _draw(1, dtype, Nq, H, d), _draw(2, dtype, Nk, Hkv, d), _draw(3, dtype, Nk, Hkv, d)
    want, mag, a = lref.attn_prefill(q, k, v, cu_q, cu_k, d ** -0.5)
    q, k, v, cq, ck = q.cuda(), k.cuda(), v.cuda(), *(torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    need = kda.attn_prefill_workspace_bytes(len(nq), Nq, Nk, H, Hkv, d, DT[dtype])
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    o = torch.full((Nq, H, d), 9.0, dtype=DT[dtype], device="cuda")
    one = o.clone()
    kda.attn_prefill(q, k, v, cq, ck, o=o, workspace=ws)
    p = lambda t: t.data_ptr()  # noqa: E731
    st = _lib.load().kda_attn_prefill(p(q), p(k), p(v), p(cq), p(ck), p(one), len(nq), Nq, Nk, H, Hkv, d, d ** -0.5, H * d, Hkv * d,
                                      Hkv * d, _lib.KDA_BF16 if dtype == "bf16" else _lib.KDA_F32, None, 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for t in (o, one):
        _inside(t, want, mag, a, d, max(nk), dtype)
        assert bool((t[:1] == 9.0).all()) and bool((t[cu_q[-1]:] == 9.0).all())
        assert (ref.f64(t)[~np.isnan(want) & (mag == 0)] == 0).all()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f32")])
def test_maxima_that_rise_late(d, dtype):
    """Keys whose scores grow along the sequence, by far more than the exponentials' range: the running maximum has
    to follow, in whole tiles too.  Scores of 300 are held to 2^-24 of their size (the bounds count that)."""
    kda = _kda()
    n, H = 500, 2
    print("rising maxima", d, dtype, flush=True)
    q, v = torch.ones(n, H, d, dtype=DT[dtype]), _draw(3, dtype, n, 1, d)
    k = (torch.linspace(-300, 300, n)[:, None, None] / d).expand(n, 1, d).to(DT[dtype]).contiguous()
    want, mag, a = lref.attn_prefill(q, k, v, [0, n], [0, n], 1.0)
    o = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=1.0)
    torch.cuda.synchronize()
    _inside(o, want, mag, a, d, n, dtype)


def test_sequence_ends_outside_the_tensor_are_clamped():
    """Device values that no correct program sends: nothing is read or written outside the tensors, and the sequences
    that they leave are answered.  Rows of the others are open, so only those are compared."""
    kda = _kda()
    q, k, v = _draw(1, "bf16", 40, 2, 64), _draw(2, "bf16", 40, 1, 64), _draw(3, "bf16", 40, 1, 64)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    i32 = lambda *c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    a = kda.attn_prefill(q, k, v, i32(0, 15, 40))
    b = kda.attn_prefill(q, k, v, i32(-7, 15, 2 ** 31 - 1))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_a_value_that_is_no_number_stays_in_its_sequence():
    kda = _kda()
    q, k, v = (_draw(i, "bf16", 300, 2, 64).cuda() for i in (1, 2, 3))
    cu = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    want = kda.attn_prefill(q, k, v, cu)
    for t, x in ((k, float("nan")), (v, float("inf"))):
        t[150] = x
    got = kda.attn_prefill(q, k, v, cu)
    torch.cuda.synchronize()
    assert torch.equal(got[:100], want[:100]) and torch.equal(got[200:], want[200:])
    assert torch.isnan(got[150:200].float()).all()
