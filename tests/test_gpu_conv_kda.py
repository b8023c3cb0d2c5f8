"""The short convolution in front of Kimi Delta Attention: q, k and v of a projection's rows each pass through
one of their own, for a prompt (convolution, then chunk_prefill) and token by token (conv_step, then
decode_step), against the definition of the convolution and the oracle's recurrence in 64 bits.

Both bounds are the library's for KDA (rel-L2 1e-2 and max-abs 3e-2 in bf16, 1e-4 and 1e-3 in fp32): the inputs
of the recurrence are the convolution's outputs as the device rounded them, which are checked on their own.
"""
import numpy as np
import pytest
import torch

import oracle
from tests import mixers_reference as ref
from tests.parity import assert_close

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_convolved_inputs_feed_the_prompt_and_the_tokens_of_kda(dtype, d):
    import chunked_gated_delta_13_amd as kda
    B, T, more, H, W = 2, 150, 5, 3, 4
    dt, width = DT[dtype], 3 * d
    g = torch.Generator().manual_seed(31)
    rows = torch.randn(B, T + more, 3 * width + 8, generator=g).to(dt)      # q, k, v side by side, and a tail
    w = [(torch.randn(width, W, generator=g) * 0.5).to(dt) for _ in range(3)]
    log_alpha = -torch.rand(B, T + more, H, d, generator=g) * 0.3
    beta = torch.rand(B, T + more, H, generator=g)
    S0 = torch.randn(B, H, d, d, generator=g) * 0.02

    def unit(t):   # KDA takes normalised q and k
        return (t.float() / t.float().norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt)

    dr, dw = rows.cuda(), [t.cuda() for t in w]
    cut = lambda t, i: t[..., i * width:(i + 1) * width]  # noqa: E731
    la, be, S = log_alpha.cuda(), beta.cuda(), S0.cuda()
    hist, conv = [], []
    for i in range(3):
        y, s = kda.conv_prefill(cut(dr[:, :T].contiguous(), i), dw[i])
        hist.append(s)
        conv.append([y])
    q, k, v = (c[0].unflatten(-1, (H, d)) for c in conv)
    o, S = kda.chunk_prefill(unit(q), unit(k), v, la[:, :T].contiguous(), be[:, :T].contiguous(), S, S_T=S)
    outs = [o]
    for t in range(T, T + more):
        tok = [kda.conv_step(cut(dr[:, t], i), dw[i], hist[i]) for i in range(3)]
        for c, y in zip(conv, tok):
            c.append(y[:, None])
        q, k, v = (y.unflatten(-1, (H, d)) for y in tok)
        outs.append(kda.decode_step(unit(q), unit(k), v, la[:, t].contiguous(), be[:, t].contiguous(), S)[:, None])
    torch.cuda.synchronize()
    conv = [torch.cat(c, 1) for c in conv]
    for i in range(3):
        want, mag, kept, _ = ref.conv(cut(rows, i), w[i], None, None, None, True)
        tol = (1.1 * (W + 1) * mag + 10 * np.abs(want)) * ref.U32 + ref.half_step(dt) * np.abs(want) + 1e-37
        assert (np.abs(ref.f64(conv[i]) - want) <= tol).all()
        assert np.array_equal(ref.f64(hist[i]), kept)
    q, k, v = (c.cpu().unflatten(-1, (H, d)) for c in conv)
    o_ref, S_ref = oracle.prefill(unit(q), unit(k), v, log_alpha, beta, S0)[:2]
    assert_close("o", torch.cat(outs, 1), o_ref, dtype)
    assert_close("S", S, S_ref, dtype)
