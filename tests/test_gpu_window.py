"""Window attention on the device against its definition in 64 bits.

Tolerance.  u = 2^-24, h the half step of the input type.  A score is a sum of d products off by at most
2 (d + 8) u a, with a = scale * sum |q k|; scaling and the exponential's argument add 8 u a, so a
probability is off by at most e = u (2 d + 32) a + 40 u relative, numerator and denominator alike.  With
bf16 inputs it is rounded once (h) as an operand.  Sums over K keys add 4 K u.  With m = sum p |v|:
|o - ref| <= (2 e + h' + 4 K u) m + h |o|, h' = h (1 + h) for bf16 and 0 for fp32.
"""
import numpy as np
import pytest
import torch

from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _inside(got, want, mag, a, d, keys, dtype):
    g, live = ref.f64(got), ~np.isnan(want)
    h = ref.half_step(DT[dtype])
    e = ref.U32 * ((2 * d + 32) * a[..., None] + 40)
    tol = (2 * e + (h * (1 + h) if dtype == "bf16" else 0) + 4 * keys * ref.U32) * mag + h * np.abs(want) + 1e-37
    err = np.abs(g - want)[live]
    assert np.isfinite(g[live]).all() and (err <= tol[live]).all(), float((err / tol[live]).max())


def _draw(seed, dtype, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype])


def _caches(rows, win, sinks, Hkv, d, dtype, before, seed):
    """Ring caches after `before` tokens of each sequence; rows no token has reached hold NaN."""
    kc = torch.full((rows, sinks + win, Hkv, d), float("nan"), dtype=DT[dtype])
    vc = kc.clone()
    for b, n in enumerate(before):
        m = min(int(n), sinks + win)
        kc[b, :m] = _draw(seed + b, dtype, m, Hkv, d)
        vc[b, :m] = _draw(seed + 50 + b, dtype, m, Hkv, d)
    return kc, vc


# B, T, H, Hkv, d, window, sinks, dtype, start, lens
CASES = [
    (1, 1, 1, 1, 64, 1, 0, "bf16", None, None),
    (1, 64, 2, 1, 64, 1, 0, "bf16", None, None),              # every token sees itself only
    (2, 130, 4, 2, 128, 16, 4, "bf16", None, None),
    (1, 200, 3, 1, 128, 500, 4, "bf16", None, None),          # window longer than the prompt
    (1, 200, 3, 1, 128, 63, 3, "f32", None, None),
    (3, 150, 2, 2, 64, 40, 0, "bf16", [0, 17, 400], [150, 0, 77]),
    (3, 150, 7, 1, 64, 70, 5, "bf16", [3, 80, 1000], [149, 200, 1]),     # 200 is clamped; a start inside the sinks
    (2, 33, 8, 2, 128, 200, 16, "bf16", [100, 5000], [33, 30]),
    (2, 140, 2, 1, 64, 33, 70, "f32", [0, 69], [140, 139]),   # more sinks than a tile and than the window
    (2, 70, 2, 2, 128, 7, 1, "f32", [2**31 - 200, 0], [70, -1]),         # far positions; -1 is clamped to 0
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])))
def test_window_prefill_matches_definition(case):
    kda = _kda()
    B, T, H, Hkv, d, win, sinks, dtype, start, lens = case
    print("window_prefill", case, flush=True)
    q, k, v = _draw(1, dtype, B, T, H, d), _draw(2, dtype, B, T, Hkv, d), _draw(3, dtype, B, T, Hkv, d)
    st = None if start is None else torch.tensor(start, dtype=torch.int32)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    kc, vc = _caches(B, win, sinks, Hkv, d, dtype, [0] * B if start is None else start, 10)
    want, mag, a, kc_ref, vc_ref = ref.window(q, k, v, win, sinks, d ** -0.5, kc, vc, st, ln)
    for b, m in enumerate(ref.lens_of(ln, B, T)):            # padding holds NaN
        for t in (q, k, v):
            t[b, m:] = float("nan")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    kd, vd = kc.cuda(), vc.cuda()
    o = torch.full((B, T, H, d), 9.0, dtype=DT[dtype], device="cuda")
    kda.window_prefill(dev(q), dev(k), dev(v), win, sinks, k_cache=kd, v_cache=vd, start=dev(st), lens=dev(ln), o=o)
    torch.cuda.synchronize()
    _inside(o, want, mag, a, d, win + sinks, dtype)
    for b, m in enumerate(ref.lens_of(ln, B, T)):
        assert bool((o[b, m:] == 9.0).all())
    assert np.array_equal(ref.f64(kd), kc_ref, equal_nan=True) and np.array_equal(ref.f64(vd), vc_ref, equal_nan=True)
    if start is None:   # without caches: the same outputs
        o2 = torch.full_like(o, 9.0)
        kda.window_prefill(dev(q), dev(k), dev(v), win, sinks, lens=dev(ln), o=o2)
        torch.cuda.synchronize()
        assert torch.equal(o, o2)


# few queries over long windows: ranges of keys, some of them without any
SPLITS = [
    (1, 1, 2, 1, 128, 1000, 4, "bf16", [5000], None),
    (1, 5, 4, 2, 64, 777, 0, "f32", [2000], None),
    (3, 40, 4, 2, 128, 600, 5, "bf16", [0, 3, 9000], [40, 33, 17]),      # two rings that have hardly begun
    (4, 70, 2, 1, 64, 500, 16, "bf16", [10, 700, 100, 2000], [0, 1, 70, 64]),
    (2, 65, 3, 3, 128, 260, 1, "f32", [400, 0], [65, 2]),
    (1, 700, 1, 1, 64, 1000, 0, "bf16", None, None),                     # no earlier tokens
]


@pytest.mark.parametrize("case", SPLITS, ids=lambda c: "-".join(map(str, c[:8])))
def test_window_prefill_split_over_ranges_matches_definition(case):
    """As above, with the smallest workspace; the same call without the split has the same bounds."""
    from chunked_gated_delta_13_amd import _lib
    kda = _kda()
    B, T, H, Hkv, d, win, sinks, dtype, start, lens = case
    print("window_prefill split", case, flush=True)
    q, k, v = _draw(1, dtype, B, T, H, d), _draw(2, dtype, B, T, Hkv, d), _draw(3, dtype, B, T, Hkv, d)
    st = None if start is None else torch.tensor(start, dtype=torch.int32)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    kc, vc = _caches(B, win, sinks, Hkv, d, dtype, [0] * B if start is None else start, 10)
    want, mag, a, kc_ref, vc_ref = ref.window(q, k, v, win, sinks, d ** -0.5, kc, vc, st, ln)
    for b, m in enumerate(ref.lens_of(ln, B, T)):
        for t in (q, k, v):
            t[b, m:] = float("nan")
    need = kda.window_prefill_workspace_bytes(B, T, H, Hkv, d, win, sinks, DT[dtype], continued=start is not None)
    assert need > 0 and need % 16 == 0
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    qd, kd, vd, sd, ld = dev(q), dev(k), dev(v), dev(st), dev(ln)
    for split in (True, False):
        kcd, vcd = kc.cuda(), vc.cuda()
        o = torch.full((B, T, H, d), 9.0, dtype=DT[dtype], device="cuda")
        if split:
            room = torch.full((need // 4 + 64,), float("nan"), device="cuda")
            kda.window_prefill(qd, kd, vd, win, sinks, k_cache=kcd, v_cache=vcd, start=sd, lens=ld, o=o,
                               workspace=room[:need // 4])
        else:
            ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
            _lib.check(_lib.load().kda_window_prefill(
                ptr(qd), ptr(kd), ptr(vd), ptr(kcd), ptr(vcd), ptr(sd), ptr(ld), ptr(o), B, T, H, Hkv, d, win, sinks, d ** -0.5,
                H * d, Hkv * d, Hkv * d, 0 if dtype == "bf16" else 1, None, 0, torch.cuda.current_stream().cuda_stream), "window")
        torch.cuda.synchronize()
        _inside(o, want, mag, a, d, win + sinks, dtype)
        for b, m in enumerate(ref.lens_of(ln, B, T)):
            assert bool((o[b, m:] == 9.0).all())
        assert np.array_equal(ref.f64(kcd), kc_ref, equal_nan=True) and np.array_equal(ref.f64(vcd), vc_ref, equal_nan=True)
    assert bool(torch.isnan(room[need // 4:]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_prefill_slices_scale_and_large_scores(dtype):
    """q, k and v cut from one projection's rows; scores up to several hundred."""
    kda = _kda()
    B, T, H, Hkv, d, win, sinks = 2, 100, 4, 2, 64, 48, 2
    qkv = _draw(5, dtype, B, T, (H + 2 * Hkv) * d, std=3.0)
    cut = lambda t: (t[..., :H * d].unflatten(-1, (H, d)), t[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d)),  # noqa: E731
                     t[..., (H + Hkv) * d:].unflatten(-1, (Hkv, d)))
    q, k, v = cut(qkv)
    want, mag, a, _, _ = ref.window(q, k, v, win, sinks, 1.5)
    o = kda.window_prefill(*cut(qkv.cuda()), win, sinks, scale=1.5)
    torch.cuda.synchronize()
    _inside(o, want, mag, a, d, win + sinks, dtype)


@pytest.mark.parametrize("dtype,H,Hkv,d,win,sinks", [("bf16", 4, 2, 128, 50, 4), ("f32", 6, 1, 64, 30, 0)])
def test_window_pieces_then_tokens_equal_the_whole(dtype, H, Hkv, d, win, sinks):
    """A prompt in uneven pieces through the cache, then token by token, against the definition of the
    whole sequence; the caches end as the definition's."""
    kda = _kda()
    B, total = 2, 180
    q, k, v = _draw(6, dtype, B, total, H, d), _draw(7, dtype, B, total, Hkv, d), _draw(8, dtype, B, total, Hkv, d)
    kc = torch.full((B, sinks + win, Hkv, d), float("nan"), dtype=DT[dtype])
    want, mag, a, kc_ref, vc_ref = ref.window(q, k, v, win, sinks, d ** -0.5, kc, kc)
    kd, vd = kc.cuda(), kc.cuda()
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    outs, at = [], 0
    for n in (3, 70, 1, 65, 30):
        start = torch.full((B,), at, dtype=torch.int32, device="cuda")
        outs.append(kda.window_prefill(*(t[:, at:at + n].contiguous() for t in (q, k, v)), win, sinks, k_cache=kd, v_cache=vd,
                                       start=start))
        at += n
    pos = torch.full((B,), at, dtype=torch.int32, device="cuda")
    while at < total:
        outs.append(kda.window_step(q[:, at], k[:, at], v[:, at], kd, vd, pos, win, sinks)[:, None])
        pos += 1
        at += 1
    torch.cuda.synchronize()
    _inside(torch.cat(outs, 1), want, mag, a, d, win + sinks, dtype)
    assert np.array_equal(ref.f64(kd), kc_ref) and np.array_equal(ref.f64(vd), vc_ref)


# N, H, Hkv, d, window, sinks, dtype, pos
STEPS = [
    (1, 1, 1, 64, 1, 0, "bf16", [0]),
    (4, 8, 2, 128, 100, 4, "bf16", [0, 3, 4, 103]),            # first token, last sink, first ring row, ring full
    (3, 7, 1, 64, 300, 0, "bf16", [299, 300, 100000]),
    (2, 20, 1, 128, 150, 3, "bf16", [77, 2**31 - 2]),          # more than 16 heads on one kv head; a far position
    (1, 14, 2, 128, 4096, 4, "bf16", [9000]),                  # split over ranges
    (1, 14, 2, 128, 4096, 4, "bf16", [700]),                   # split, with ranges that no token has reached
    (2, 4, 2, 64, 2000, 16, "f32", [5000, 10]),
    (5, 3, 3, 128, 31, 1, "f32", [0, 1, 31, 32, 33]),
]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c[:7])))
def test_window_step_matches_definition(case):
    kda = _kda()
    N, H, Hkv, d, win, sinks, dtype, pos = case
    print("window_step", case, flush=True)
    q, k, v = _draw(1, dtype, N, H, d), _draw(2, dtype, N, Hkv, d), _draw(3, dtype, N, Hkv, d)
    kc, vc = _caches(N, win, sinks, Hkv, d, dtype, pos, 20)
    p = torch.tensor(pos, dtype=torch.int32)
    want, mag, a, kc_ref, vc_ref = ref.window(q[:, None], k[:, None], v[:, None], win, sinks, d ** -0.5, kc, vc, p)
    kd, vd = kc.cuda(), vc.cuda()
    o = kda.window_step(q.cuda(), k.cuda(), v.cuda(), kd, vd, p.cuda(), win, sinks, o=torch.full((N, H, d), float("nan"),
                        dtype=DT[dtype], device="cuda"))
    torch.cuda.synchronize()
    _inside(o, want[:, 0], mag[:, 0], a[:, 0], d, win + sinks, dtype)
    assert np.array_equal(ref.f64(kd), kc_ref, equal_nan=True) and np.array_equal(ref.f64(vd), vc_ref, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("win", [300, 1500])
def test_window_scores_below_the_range_of_fp32_have_no_weight(dtype, win):
    """A run of keys whose products with the query are -inf in fp32 (-6e41): their exponentials are 0, also
    where they fill a whole tile, and the other keys' scores of 0 weigh their values equally.  Weights are 1
    exactly, so what is off is the sum (a rounding per key and per join) and the output's rounding."""
    kda = _kda()
    d, far = 64, 200
    q = torch.full((1, 1, d), 1e20, dtype=DT[dtype])
    kc = torch.zeros(1, win, 1, d, dtype=DT[dtype])
    kc[:, :far] = -1e20
    vc = _draw(4, dtype, 1, win, 1, d)
    v = _draw(5, dtype, 1, 1, d)
    see = torch.cat([vc[:, far:win - 1, 0], v], 1).double()
    want, mag = see.mean(1, keepdim=True).numpy(), see.abs().mean(1, keepdim=True).numpy()
    tol = ref.half_step(DT[dtype]) * np.abs(want) + (win + 16) * ref.U32 * mag
    zero = torch.zeros(1, 1, d, dtype=DT[dtype])
    o = kda.window_step(q.cuda(), zero.cuda(), v.cuda(), kc.cuda(), vc.cuda(),
                        torch.tensor([win - 1], dtype=torch.int32, device="cuda"), win)
    ks = torch.cat([kc[:, :win - 1], zero[:, None]], 1).cuda()
    vs = torch.cat([vc[:, :win - 1], v[:, None]], 1).cuda()
    p = kda.window_prefill(q[:, None].expand(1, win, 1, d).contiguous().cuda(), ks, vs, win)
    torch.cuda.synchronize()
    for name, got in (("step", o), ("prompt", p[:, -1])):
        err = np.abs(ref.f64(got) - want)
        assert (err <= tol).all(), (name, float((err / tol).max()))


def test_window_step_splits_where_rows_are_few():
    kda = _kda()
    assert kda.window_step_workspace_bytes(1, 14, 2, 128, 4096, 4) > 0
    assert kda.window_step_workspace_bytes(512, 14, 2, 128, 4096, 4) == 0


def test_window_empty_calls():
    kda = _kda()
    e = torch.empty(2, 0, 4, 64, device="cuda")
    assert kda.window_prefill(e, e[:, :, :2], e[:, :, :2], 8).shape == (2, 0, 4, 64)
    z = torch.empty(0, 4, 64, device="cuda")
    c = torch.empty(0, 8, 2, 64, device="cuda")
    assert kda.window_step(z, z[:, :2], z[:, :2], c, c.clone(), torch.empty(0, dtype=torch.int32, device="cuda"), 8).shape == (0, 4, 64)
