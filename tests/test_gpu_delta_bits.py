"""The gated delta rule's bf16 outputs on the device, held to what two bf16 parts of every factor leave (delta_bits.py); the
state's part of the tolerance is that of test_gpu_delta.py."""
import numpy as np
import pytest
import torch

from tests import mixers_reference as ref
from tests.delta_bits import SHARE
from tests.test_gpu_delta import CASES, U90, _inputs, _kda, _norms, _split

pytestmark = pytest.mark.gpu


def _held(o, want, terms, top, nq, R):
    tol = U90 * (np.repeat(nq, R, 2) * top[:, None])[..., None] + SHARE * terms + ref.half_step(torch.bfloat16) * np.abs(want) + 1e-37
    live = ~np.isnan(want)
    err = np.abs(ref.f64(o) - want)
    assert np.isfinite(ref.f64(o)[live]).all() and (err[live] <= tol[live]).all(), float((err / tol)[live].max())


@pytest.mark.parametrize("case", [c for c in CASES if c[6] == "bf16" and c[0] < 100], ids=lambda c: "-".join(map(str, c[:6])) + f"-{c[9]}-{int(c[10])}")
def test_outputs_from_two_parts_of_every_factor(case):
    kda = _kda()
    B, T, H, Hk, dk, dv, dtype, state, lens, seg, strong = case
    print("bits", case, flush=True)
    rows, g, beta, S0 = _inputs(21, dtype, B, T, H, Hk, dk, dv, strong)
    args = (*_split(rows, H, Hk, dk, dv), g, beta)
    S0 = S0 if state else None
    dr = rows.cuda()
    o, _ = kda.delta_prefill(*_split(dr, H, Hk, dk, dv), g.cuda(), beta.cuda(), None if S0 is None else S0.cuda(), seg_len=seg,
                             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want, terms, _, top, nq = _norms(*args, S0, lens, 64)
    _held(o, want, terms, top, nq, H // Hk)


def test_outputs_of_a_prompt_in_pieces_then_tokens():
    """Each piece against the definition from the state that it was handed, then tokens, single sums over dk terms."""
    kda = _kda()
    B, T, H, Hk, dk, dv = 2, 203, 4, 2, 128, 128
    rows, g, beta, S0 = _inputs(22, "bf16", B, T, H, Hk, dk, dv)
    dr, gd, bd, S, at = rows.cuda(), g.cuda(), beta.cuda(), S0.cuda(), 0
    for n in (1, 64, 100, 35, 1, 1, 1):
        part = slice(at, at + n)
        had = S.cpu()
        q, k, v = (x[:, part].contiguous() for x in _split(dr, H, Hk, dk, dv))
        if n == 1 and at > 0:
            o = kda.delta_step(q[:, 0], k[:, 0], v[:, 0], gd[:, at].contiguous(), bd[:, at].contiguous(), S)[:, None]
        else:
            o, _ = kda.delta_prefill(q, k, v, gd[:, part].contiguous(), bd[:, part].contiguous(), S, S_T=S)
        torch.cuda.synchronize()
        want, terms, _, top, nq = _norms(*(x[:, part] for x in _split(rows, H, Hk, dk, dv)), g[:, part], beta[:, part], had, None, 64)
        _held(o, want, terms, top, nq, H // Hk)
        at += n
    assert at == T
