"""Window attention where many queries run: the kernel of 128 queries per workgroup (bf16, as many
workgroups as compute units or more), and running maxima that have to be raised in a tile that every
query sees whole.  The reference is the definition in 64 bits on the device, head by head.

Tolerance as for the small cases: with u = 2^-24, h the half step of the input type, a = scale * sum |q k|
at its largest, m = sum p |v| and K keys: a probability is off by e = u (2 d + 32) a + 40 u relative, in
numerator and denominator, and by h' = h (1 + h) as a bf16 operand; |o - ref| <= (2 e + h' + 4 K u) m + h |o|.
"""
import pytest
import torch

from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _r(seed, dtype, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dtype])


def _check(q, k, v, win, sinks, scale, kc, vc, start, lens, o, dtype, before=None):
    """o against the definition, sequence by sequence and head by head; rows behind the end against `before`."""
    B, T, H, d = q.shape
    R = H // k.shape[2]
    h = ref.half_step(DT[dtype])
    worst = 0.0
    for b in range(B):
        s, m = (0 if start is None else start[b]), (T if lens is None else min(max(lens[b], 0), T))
        if before is not None:
            assert torch.equal(o[b, m:], before[b, m:])
        if m == 0:
            continue
        new = torch.arange(s, s + m, device="cuda")
        old = torch.cat([torch.arange(min(sinks, s)), torch.arange(max(sinks, s - win + 1), max(sinks, s))]).cuda()
        at = torch.cat([old, new])
        row = torch.where(old < sinks, old, sinks + (old - sinks) % win)
        keys = [torch.cat(([c[b, row].double()] if len(old) else []) + [t[b, :m].double()]) for c, t in ((kc, k), (vc, v))]
        gap = new[:, None] - at
        see = (gap >= 0) & ((gap < win) | (at < sinks))
        count = float(see.sum(1).max())
        for i in range(H):
            qi, ki, vi = q[b, :m, i].double(), keys[0][:, i // R].contiguous(), keys[1][:, i // R].contiguous()
            w = (qi @ ki.t().contiguous() * scale).masked_fill(~see, -torch.inf)
            p = torch.softmax(w, -1)
            want, mag = p @ vi, p @ vi.abs()
            a = (qi.abs() @ ki.abs().t().contiguous() * scale).masked_fill(~see, 0).amax(-1, keepdim=True)
            e = ref.U32 * ((2 * d + 32) * a + 40)
            tol = (2 * e + (h * (1 + h) if dtype == "bf16" else 0) + 4 * count * ref.U32) * mag + h * want.abs() + 1e-37
            got = o[b, :m, i].double()
            assert bool(torch.isfinite(got).all())
            worst = max(worst, float(((got - want).abs() / tol).max()))
    print("worst share of the tolerance", worst, flush=True)
    assert worst <= 1


def _wide(B, T, H):
    """The plan's rule for 128 queries per workgroup."""
    return B * H * -(-T // 128) >= torch.cuda.get_device_properties(0).multi_processor_count


# B, T, H, Hkv, d, window, sinks, start, lens
WIDE = [
    (4, 300, 32, 4, 128, 150, 4, [0, 3, 400, 5000], [300, 0, 129, 257]),
    (4, 300, 32, 8, 64, 150, 4, [2, 77, 0, 100000], [299, 128, 1, 300]),
    (2, 200, 64, 64, 64, 500, 0, None, None),               # a window longer than the prompt, a kv head per head
    (1, 1000, 40, 8, 128, 700, 70, None, None),             # most tiles whole; more first tokens than a tile
    (4, 130, 64, 1, 128, 1, 0, None, [130, 64, 65, 129]),   # every token sees itself only
    (2, 513, 28, 7, 64, 64, 1, [64, 65], None),             # a window of one tile
    (1, 2500, 16, 2, 128, 1024, 4, [1500], None),           # a long piece over a full ring
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c[:7])))
def test_wide_prompt_matches_definition(case):
    kda = _kda()
    B, T, H, Hkv, d, win, sinks, start, lens = case
    print("window_prefill wide", case, flush=True)
    assert _wide(B, T, H)
    q, k, v = _r(1, "bf16", B, T, H, d), _r(2, "bf16", B, T, Hkv, d), _r(3, "bf16", B, T, Hkv, d)
    kc, vc = (torch.full((B, sinks + win, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b, n in enumerate(start or []):                     # rows that no token has reached hold NaN
        n = min(n, sinks + win)
        kc[b, :n], vc[b, :n] = _r(10 + b, "bf16", n, Hkv, d), _r(20 + b, "bf16", n, Hkv, d)
    kc0, vc0 = kc.clone(), vc.clone()
    for b, m in enumerate(lens or []):                      # and so do the rows behind a sequence's end
        for t in (q, k, v):
            t[b, m:] = float("nan")
    i32 = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    before = _r(4, "bf16", B, T, H, d)
    o = before.clone()
    kda.window_prefill(q, k, v, win, sinks, k_cache=kc, v_cache=vc, start=i32(start), lens=i32(lens), o=o)
    torch.cuda.synchronize()
    _check(q, k, v, win, sinks, d ** -0.5, kc0, vc0, start, lens, o, "bf16", before)
    for b in range(B):                                      # the rings as a token-by-token writer leaves them
        s, m = (0 if start is None else start[b]), (T if lens is None else lens[b])
        for c, c0, t in ((kc, kc0, k), (vc, vc0, v)):
            p = torch.arange(s, s + m, device="cuda")
            keep = (p < sinks) | (p >= s + m - win)
            row = torch.where(p < sinks, p, sinks + (p - sinks) % win)[keep]
            want = c0[b].clone()
            want[row] = t[b, :m][keep]
            assert torch.equal(c[b].nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype,B,T,H,Hkv,d", [("bf16", 1, 700, 8, 2, 128), ("bf16", 1, 700, 8, 2, 64), ("f32", 1, 500, 2, 1, 64),
                                               ("f32", 1, 500, 2, 1, 128), ("bf16", 2, 700, 32, 4, 128), ("bf16", 2, 700, 32, 4, 64)])
def test_running_maximum_is_raised_inside_whole_tiles(dtype, B, T, H, Hkv, d):
    """Scores that rise by 12 to several hundred at keys late in the prompt, in tiles that all queries of a wave
    see whole: taken with the maximum at hand, their exponentials reach from e^12 past fp32's range.  Later keys
    fall back to ordinary scores."""
    kda = _kda()
    win, sinks, scale = 300, 2, d ** -0.5
    assert _wide(B, T, H) == (B == 2)
    q, k, v = _r(1, dtype, B, T, H, d), _r(2, dtype, B, T, Hkv, d), _r(3, dtype, B, T, Hkv, d)
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    # (position, score): within one tile, in the next tiles, and past 88, where exponentials leave fp32
    for at, score in ((150, 12.0), (200, 14.0), (201, 30.0), (260, 45.0), (300, 80.0), (333, 300.0), (390, 500.0), (470, 505.0)):
        k[:, at, :, 0] = score / (4.0 * scale)
    o = kda.window_prefill(q, k, v, win, sinks)
    torch.cuda.synchronize()
    _check(q, k, v, win, sinks, scale, None, None, None, None, o, dtype)


def test_negative_counts_of_earlier_tokens_count_as_none():
    kda = _kda()
    B, T, H, Hkv, d, win, sinks = 2, 40, 4, 2, 64, 20, 3
    q, k, v = _r(1, "bf16", B, T, H, d), _r(2, "bf16", B, T, Hkv, d), _r(3, "bf16", B, T, Hkv, d)
    got = []
    for n in (0, -1, -2 ** 31):
        kc, vc = (torch.full((B, sinks + win, Hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        before = torch.full((B,), n, dtype=torch.int32, device="cuda")
        o = kda.window_prefill(q, k, v, win, sinks, k_cache=kc, v_cache=vc, start=before)
        kc1, vc1 = kc.clone(), vc.clone()
        s = kda.window_step(q[:, 0], k[:, 0], v[:, 0], kc1, vc1, before, win, sinks)
        got.append((o, kc, vc, s, kc1, vc1))
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
