"""Sizes at which the layers' kernels take forms that small tests do not reach: 128 state columns a workgroup in fp32 (whole and
in segments), 64 rows a workgroup of d = 64 in one group of waves; and fp32 attention at the lower end of the range."""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref
from tests import test_gpu_attn as attn
from tests import test_gpu_delta as delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hk,lens", [(70, 1, False), (97, 2, True)])
def test_delta_in_fp32_with_enough_heads_for_whole_states(T, Hk, lens):
    """140 states of 128 x 128: a workgroup holds one whole."""
    kda = delta._kda()
    B, H, d = 70, 2, 128
    print("delta f32 wide", T, Hk, lens, flush=True)
    rows, g, beta, S0 = delta._inputs(31, "f32", B, T, H, Hk, d, d)
    lens = [T, 0, 1, 33, 32, 64] * 11 + [T] * 4 if lens else None
    dr = rows.cuda()
    o, S_T = kda.delta_prefill(*delta._split(dr, H, Hk, d, d), g.cuda(), beta.cuda(), S0.cuda(),
                               lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    delta._check(o, S_T, *delta._split(rows, H, Hk, d, d), g, beta, S0, lens, "f32")


def test_delta_in_fp32_segments_of_whole_states():
    """71 segments of four states of 128 x 128, some of which leave nothing of a state."""
    kda = delta._kda()
    B, T, H, Hk, d, seg = 2, 70 * 64 + 5, 2, 1, 128, 64
    print("delta f32 wide segments", flush=True)
    rows, g, beta, S0 = delta._inputs(32, "f32", B, T, H, Hk, d, d)
    g = g * 0.1
    for b, h, s in ((0, 0, 3), (0, 0, 4), (0, 0, 6), (0, 1, 0), (1, 0, 68), (1, 1, 1), (1, 1, 3), (1, 1, 5)):
        g[b, s * seg + 20:s * seg + 40, h] = -6.0            # 2^-173
    dr = rows.cuda()
    o, S_T = kda.delta_prefill(*delta._split(dr, H, Hk, d, d), g.cuda(), beta.cuda(), S0.cuda(), seg_len=seg)
    torch.cuda.synchronize()
    delta._check(o, S_T, *delta._split(rows, H, Hk, d, d), g, beta, S0, None, "f32")


@pytest.mark.parametrize("case", [
    ([200, 250], None, 56, 8, 64, "bf16", 0, 0),
    ([200, 20, 230], [210, 20, 900], 56, 8, 64, "bf16", 1, 2),
    ([450, 3], [100, 640], 56, 8, 64, "bf16", 0, 0),         # queries without keys
], ids=lambda c: "-".join([str(sum(c[0])), str(c[1] is None)]))
def test_attn_prefill_of_64_rows_in_one_group_of_waves(case):
    attn.test_attn_prefill_matches_definition(case)


def test_attention_in_fp32_below_the_parts_range():
    """Values from 2^-125 to 2^-60: three bf16 parts hold 24 bits of a value or 2^-126, whichever is more."""
    kda = attn._kda()
    n, H, d = 200, 2, 64
    q, k, v = attn._draw(1, "f32", n, H, d), attn._draw(2, "f32", n, 1, d), attn._draw(3, "f32", n, 1, d)
    v = v.sign() * (1 + v.abs().frac()) * torch.exp2(torch.linspace(-125, -60, d).round())
    want, mag, a = lref.attn_prefill(q, k, v, [0, n], [0, n], 0.2)
    o = kda.attn_prefill(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=0.2)
    torch.cuda.synchronize()
    # products of parts and outputs below 2^-126 may count as nothing too: n of each of the six, and one
    e = ref.U32 * ((2 * d + 32) * a[..., None] + 40)
    assert (np.abs(ref.f64(o) - want) <= (2 * e + 4 * n * ref.U32) * mag + (1 + 6 * n + 1) * 2.0 ** -126).all()
