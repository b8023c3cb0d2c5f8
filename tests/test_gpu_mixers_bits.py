"""How many bits the token mixers' bf16 forms keep where inputs make a lost bit visible."""
import numpy as np
import pytest
import torch

from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _draw(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


@pytest.mark.parametrize("N,H,Hkv,d,win,sinks,pos", [(6, 8, 2, 64, 5, 0, 40), (3, 20, 1, 128, 37, 3, 100), (1, 14, 2, 128, 3000, 4, 9000)])
def test_window_step_keeps_sixteen_bits_of_a_probability(N, H, Hkv, d, win, sinks, pos):
    """Values of one size and either sign, so that an output is a small difference of large terms: probabilities
    rounded to 8 bits would show in it.  With u = 2^-24, a = scale * sum |q k| and m = sum p |v|: a probability
    is off by e = u (2 d + 32) a + 40 u relative, numerator and denominator alike, and by 2^-8 of 2^-8 as two
    bf16 parts; sums over K keys add 4 K u; the result is rounded once (2^-8 |o|)."""
    kda = _kda()
    q, k, v = _draw(1, N, H, d), _draw(2, N, Hkv, d), _draw(3, N, Hkv, d).sign()
    kc, vc = _draw(4, N, win + sinks, Hkv, d), _draw(5, N, win + sinks, Hkv, d).sign()
    p = torch.full((N,), pos, dtype=torch.int32)
    want, mag, a, _, _ = ref.window(q[:, None], k[:, None], v[:, None], win, sinks, d ** -0.5, kc, vc, p)
    o = kda.window_step(q.cuda(), k.cuda(), v.cuda(), kc.cuda(), vc.cuda(), p.cuda(), win, sinks)
    torch.cuda.synchronize()
    want, mag, a = want[:, 0], mag[:, 0], a[:, 0, :, None]
    e = ref.U32 * ((2 * d + 32) * a + 40)
    tol = (2 * e + 2.0 ** -16 + 4 * (win + sinks) * ref.U32) * mag + ref.half_step(BF16) * np.abs(want)
    worst = float((np.abs(ref.f64(o) - want) / tol).max())
    print("worst share of the tolerance", worst, flush=True)
    assert worst <= 1
