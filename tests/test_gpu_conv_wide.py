"""The short convolution at sizes where a thread walks 8 or 16 tokens and where outputs go past the caches,
against its definition in 64 bits on the device.  Tolerance as for the small cases: with m the sum of the
absolute values of W + 1 terms, |y - ref| <= (1.1 (W + 1) m + 10 |ref|) 2^-24 + half_step |ref|.
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


# B, T, D, W, dtype, tile, streamed, state, lens
WIDE = [
    (2, 9000, 1024, 4, "bf16", 8, False, True, [9000, 4501]),
    (2, 16400, 1024, 4, "bf16", 16, False, True, [16391, 9001]),
    (2, 16400, 1024, 3, "bf16", 16, False, False, None),
    (1, 4200, 1001, 4, "bf16", 16, False, True, [4189]),         # rows off 16 bytes: one channel per thread
    (2, 16500, 520, 2, "f32", 16, False, True, [3, 16499]),
    (3, 16500, 2048, 4, "bf16", 16, True, True, [16500, 2, 8200]),
    (2, 13000, 2048, 4, "f32", 16, True, True, [12987, 13000]),
    (1, 110000, 1001, 4, "bf16", 16, True, False, None),         # large, but rows off 16 bytes
]


def _tile(B, T, D, dtype):
    """Tokens per thread by the launch's rule: 16, halved while fewer than 64 x 4096 threads have work."""
    v = 16 // DT[dtype].itemsize
    groups, tile = (D // v if D % v == 0 else D), 16
    while tile > 4 and groups * B * -(-T // tile) < 64 * 4096:
        tile //= 2
    return tile


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c[:6])) + ("-streamed" if c[6] else ""))
def test_wide_conv_prefill_matches_definition(case):
    kda = _kda()
    B, T, D, W, dtype, tile, streamed, has_state, lens = case
    print("conv_prefill wide", case, flush=True)
    assert _tile(B, T, D, dtype) == tile and (B * T * D * DT[dtype].itemsize > 192 << 20) == streamed
    x, w, bias = _r(1, dtype, B, T, D), _r(2, dtype, D, W) * 0.5, _r(3, dtype, D)
    state = _r(4, dtype, B, W - 1, D) if has_state else None
    for b, m in enumerate(lens or []):
        x[b, m:] = float("nan")
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    y = torch.full((B, T, D), 7.0, dtype=DT[dtype], device="cuda")
    _, kept = kda.conv_prefill(x, w, bias, state, lens=ln, y=y)
    torch.cuda.synchronize()
    worst = 0.0
    for b in range(B):
        m = T if lens is None else lens[b]
        assert bool((y[b, m:] == 7.0).all())
        line = torch.cat([torch.zeros(W - 1, D, dtype=DT[dtype], device="cuda") if state is None else state[b], x[b, :m]])
        assert torch.equal(kept[b], line[m:])
        for lo in range(0, m, 8192):
            part = line[lo:min(lo + 8192, m) + W - 1].double()
            n = part.shape[0] - (W - 1)
            terms = [part[j:j + n] * w[:, j].double() for j in range(W)] + [bias.double().expand(n, D)]
            acc, mag = sum(terms), sum(t.abs() for t in terms)
            want = acc * torch.sigmoid(acc)
            tol = (1.1 * (W + 1) * mag + 10 * want.abs()) * ref.U32 + ref.half_step(DT[dtype]) * want.abs() + 1e-37
            worst = max(worst, float(((y[b, lo:lo + n].double() - want).abs() / tol).max()))
    print("worst share of the tolerance", worst, flush=True)
    assert worst <= 1
