"""The gated delta rule where updates expand, in segments: a split may only take as forgotten what the transitions
themselves have shrunk to nothing, not what the decays alone would.

Tolerances.  u = 2^-24, N the largest norm of a head's state.  As in test_gpu_delta.py an error of 90 u N arises over a
block; the transitions below grow nothing over any range of tokens by more than the state itself grows, so over T
tokens the state is off by at most T 90 u N, the rounding of the decays (log(1/2) and log(1/4) in fp32: 2^-25 of them) included.
Outputs of bf16 inputs: factors in two bf16 parts (2^-16 each) and the product of two second parts left out (2^-8 2^-8): 3 2^-16
of the terms' absolute values, and the output's own rounding.
"""
import numpy as np
import pytest
import torch

from tests import mixers_reference as ref
from tests.test_gpu_delta import DT, U90, _inputs, _kda, _norms, _split

pytestmark = pytest.mark.gpu

T, D = 2000, 64


def _pattern(name):
    """log2 of the decays and beta of T tokens, whose keys have length one along the first axis."""
    t = np.arange(T)
    if name == "alternating":          # every token: half of the state, its first row to minus twice itself
        return np.full(T, -1.0), np.full(T, 3.0)
    if name == "turns":                # 32 tokens to a quarter each, 32 tokens to minus four times each: a block ends where it began
        return np.where(t % 64 < 32, -2.0, 0.0), np.where(t % 64 < 32, 0.0, 5.0)
    if name == "late":                 # 2^-180 over each 192 tokens, the last 64 of which take 2^64 back
        return np.where(t % 192 < 180, -1.0, 0.0), np.where(t % 192 >= 128, 3.0, 0.5)
    raise ValueError(name)


def _held(o, S, q, k, v, g, beta, S0, dtype, more):
    want, terms, S_ref, top, nq = _norms(q, k, v, g, beta, S0, None, 64)
    off = np.sqrt(((ref.f64(S) - S_ref) ** 2).sum((2, 3)))
    assert (off <= more * U90 * top).all(), float((off / (more * U90 * top)).max())
    tol = more * U90 * (np.repeat(nq, v.shape[2] // q.shape[2], 2) * top[:, None])[..., None] + ref.half_step(DT[dtype]) * np.abs(want)
    if dtype == "bf16":
        tol = tol + 3 * 2.0 ** -16 * (1 + 2.0 ** -8) * terms
    err = np.abs(ref.f64(o) - want)
    assert (err <= tol + 1e-37).all(), float((err / (tol + 1e-37)).max())


@pytest.mark.parametrize("values", [False, True], ids=["state", "values"])
@pytest.mark.parametrize("seg", [0, 64, 192, 2048])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["alternating", "turns", "late"])
def test_a_split_keeps_what_updates_have_grown(name, dtype, seg, values):
    kda = _kda()
    print("growth", name, dtype, seg, values, flush=True)
    log2, beta = _pattern(name)
    g = torch.from_numpy(log2 * np.log(2.0)).float()[None, :, None]
    beta = torch.from_numpy(beta).float()[None, :, None]
    k, v = torch.zeros(1, T, 1, D, dtype=DT[dtype]), torch.zeros(1, T, 1, D, dtype=DT[dtype])
    k[..., 0] = 1.0
    if values:                         # a few, which later tokens carry on
        for at in (5, 62, 133):
            v[:, at::192, :, ::3] = 1.0
    S0 = torch.ones(1, 1, D, D)
    need = kda.delta_workspace_bytes(1, T, 1, 1, D, D, DT[dtype], seg)
    assert (need > 0) == (seg < T)     # the library's own choice is a split too
    o, S = kda.delta_prefill(k.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), S0.cuda(), seg_len=seg)
    torch.cuda.synchronize()
    _held(o, S, k, k, v, g, beta, S0, dtype, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_has_grown_before_the_decays_of_its_segment(dtype):
    """A segment of 320 tokens: 96 that double the first row, 224 that decay to 2^-130 together, so that 2^-34 of its entry
    state is left there; the next one's tokens take 2^34 back.  Each step only scales the row (and turns its sign), so its
    relative error is at most that of T steps, however large it was in between."""
    kda = _kda()
    print("growth before", dtype, flush=True)
    t = np.arange(T)
    beta = np.where((t >= 1600) & (t < 1696) | (t >= 1920) & (t < 1954), 3.0, 0.0)
    g = torch.from_numpy(np.where((t >= 1696) & (t < 1920), -130 / 224 * np.log(2.0), 0.0)).float()[None, :, None]
    beta = torch.from_numpy(beta).float()[None, :, None]
    k, v = torch.zeros(1, T, 1, D, dtype=DT[dtype]), torch.zeros(1, T, 1, D, dtype=DT[dtype])
    k[..., 0] = 1.0
    S0 = torch.ones(1, 1, D, D)
    o, S = kda.delta_prefill(k.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), S0.cuda(), seg_len=320)
    torch.cuda.synchronize()
    left = np.exp(ref.f64(g).sum() + 130 * np.log(2.0))       # +-1 but for the decays' rounding
    assert np.abs(ref.f64(S[0, 0, 0]) - left).max() <= T * U90


@pytest.mark.parametrize("dtype,dk,dv,seg", [("bf16", 128, 128, 0), ("bf16", 64, 128, 64), ("f32", 128, 64, 0), ("f32", 64, 64, 128)])
def test_updates_at_the_edge_of_expanding(dtype, dk, dv, seg):
    """beta up to 2 and keys of length one but for their rounding, so that single updates expand a little: segments that
    leave nothing beside others that do.  The tolerance counts how far one rounding to fp32 of k, v, beta and g moves the
    definition's own state (the largest of three draws), for each of the 64 tokens of a block."""
    kda = _kda()
    B, n, H, Hk = 2, 64 * 20 + 9, 2, 1
    print("edge", dtype, dk, dv, seg, flush=True)
    rows, g, beta, S0 = _inputs(11, dtype, B, n, H, Hk, dk, dv)
    q, k, v = _split(rows, H, Hk, dk, dv)
    k.copy_(k.float() / k.float().norm(dim=-1, keepdim=True))
    beta = beta + (beta > 0.5).float()                       # below 1/2, or from 3/2 to 2
    g = g * 0.1
    for b, h, s in ((0, 0, 3), (0, 0, 4), (0, 1, 0), (1, 0, 18), (1, 1, 7), (1, 1, 9)):
        g[b, s * 64 + 20:s * 64 + 50, h] = -4.0              # 2^-173
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
    _held(o, S_T, q, k, v, g, beta, S0, dtype, 1 + 64 * sigma / U90)
