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


@pytest.mark.parametrize("n,p,T", [(64, 64, 64), (64, 128, 64), (128, 128, 128)])
def test_ssm_decay_between_near_tokens_behind_strong_ones(n, p, T):
    """40 tokens of each chunk decay by the most there is (2^-160 each), so that sums of exponents pass 6400 where
    fp32 numbers lie 2^-11 apart; the decays between the weak tokens after them are differences of such sums.  One
    token j has an input, and y_i = e^{c_i - c_j} dt_j (C_i . B_j) x_j.  Rounding the weight and the output to bf16
    (half step h = 2^-8 each) hides an exponent's error in one number, so it is looked for as a factor common to
    N = 32768 heads of independent B and C: f = sum(y y_ref) / sum(y_ref^2).  Relative roundings are at most h,
    with mean 0 and at most h / sqrt(3) of deviation each; C . B is near normal, whose sum(t^4) / sum(t^2)^2 is 3 / N:
    f is off by h sqrt(2 / N) of deviation at most, and by 40 u for softplus and the exponentials, where the
    exponent itself (up to 20 here) is off by 2 u of its size.  Tolerance: five deviations."""
    kda = _kda()
    B, H, strong = 32, 1024, 40
    N = B * H
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    dt = torch.full((T,), 30.0)
    weak = torch.arange(T) % 64 >= strong
    dt[weak] = torch.linspace(-5.0, -4.0, int(weak.sum()))
    dt = dt.to(BF16)
    A = -16.0
    d = np.logaddexp(0.0, ref.f64(dt))
    a = np.maximum(d * A / np.log(2.0), -160.0)
    first = T - 64
    c = np.cumsum(a[first:])
    # the weak token whose sum is furthest off in fp32, and those after it
    off = np.abs(c.astype(np.float32) - c)
    j = strong + int(np.argmax(off[strong:60]))
    x = torch.zeros(B, T, H, p, dtype=BF16, device="cuda")
    x[:, first + j] = 1.0
    Bm, Cm = rnd(B, T, H, n), rnd(B, T, H, n)
    y, _ = kda.ssm_prefill(x, dt.cuda().expand(B, H, T).transpose(1, 2).contiguous(), torch.full((H,), A, device="cuda"), Bm, Cm,
                           return_state=False, seg_len=(T + 63) // 64 * 64)
    torch.cuda.synchronize()
    tol = 5 * 2.0 ** -8 * (2 / N) ** 0.5 + 80 * ref.U32
    worst = 0.0
    for i in range(j, 64):
        dot = (Cm[:, first + i].double() * Bm[:, first + j].double()).sum(-1)
        want = float(np.exp2(c[i] - c[j]) * d[first + j]) * dot
        got = y[:, first + i, :, :].double().mean(-1)
        f = float((got * want).sum() / (want * want).sum())
        worst = max(worst, abs(f - 1))
    print("worst", worst, "tolerance", tol, flush=True)
    assert worst <= tol
