"""The short convolution on the device against its definition in 64 bits.

Tolerance.  A sum of W <= 4 products and a bias runs as one chain of fused multiply-adds: at most
W + 1 fp32 roundings of partial sums no larger than the terms' absolute sum m.  SiLU has a slope of at
most 1.1, and its exponential, addition, reciprocal and product add at most 8 half steps of the result
(the exponential's argument is off by half a step relative: |v| e^-|v| <= 0.37 more of a half step).
The result is rounded once more: |got - ref| <= (1.1 (W + 1) m + 10 |ref|) 2^-24 + half_step |ref|.
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


def _draw(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _inside(got, want, mag, W, dtype):
    g, live = ref.f64(got), ~np.isnan(want)
    tol = (1.1 * (W + 1) * mag + 10 * np.abs(want)) * ref.U32 + ref.half_step(dtype) * np.abs(want) + 1e-37
    bad = np.abs(g - want)[live] > tol[live]
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - want) / tol)[live].max()))


# B, T, D, W, dtype, silu, bias, state, lens (None, or per sequence)
CASES = [
    (1, 1, 8, 4, "bf16", True, True, True, None),
    (2, 2, 64, 4, "bf16", True, True, True, None),            # fewer tokens than taps
    (2, 2, 64, 4, "bf16", True, True, False, None),
    (3, 65, 200, 3, "bf16", False, True, True, [65, 0, 1]),   # an empty sequence and a one-token one
    (4, 130, 1000, 4, "bf16", True, False, True, [130, 2, 77, 200]),   # 200 is clamped to T
    (2, 300, 77, 2, "bf16", True, True, True, [299, 3]),      # odd rows: no 16-byte groups
    (1, 1025, 7, 4, "f32", True, True, True, None),
    (3, 40, 132, 4, "f32", True, True, True, [-5, 40, 39]),   # -5 is clamped to 0
    (2, 5000, 256, 4, "f32", False, False, False, [5000, 4097]),
    (1, 70000, 16, 4, "bf16", True, True, True, None),        # long
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_conv_prefill_matches_definition(case):
    kda = _kda()
    B, T, D, W, dtype, act, has_bias, has_state, lens = case
    print("conv_prefill", case, flush=True)
    dt = DT[dtype]
    x = _draw((B, T, D), 1, dt)
    w, bias = _draw((D, W), 2, dt, 0.5), _draw((D,), 3, dt, 0.2) if has_bias else None
    state = _draw((B, W - 1, D), 4, dt) if has_state else None
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    want, mag, kept, ls = ref.conv(x, w, bias, state, ln, act)
    y = torch.full((B, T, D), 7.0, dtype=dt, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got, st = kda.conv_prefill(dev(x), dev(w), dev(bias), dev(state), lens=dev(ln), silu=act, y=y)
    torch.cuda.synchronize()
    assert got is y
    _inside(got, want, mag, W, dt)
    assert np.array_equal(ref.f64(st), kept)
    for b in range(B):
        assert bool((got[b, ls[b]:] == 7.0).all())   # rows behind the end stay


@pytest.mark.parametrize("dtype,D,row,lead", [("bf16", 256, 520, 8), ("bf16", 256, 519, 5), ("f32", 60, 130, 3)])
def test_conv_prefill_rows_of_a_projection_and_state_in_place(dtype, D, row, lead):
    """x cut out of wider rows (16-byte aligned and not), NaN around it and in padded rows; the
    history updated in place."""
    kda = _kda()
    dt = DT[dtype]
    B, T, W = 3, 97, 4
    lens = torch.tensor([97, 2, 50], dtype=torch.int32)
    wide = torch.full((B, T, row), float("nan"), dtype=dt)
    x = _draw((B, T, D), 5, dt)
    wide[:, :, lead:lead + D] = x
    for b in range(B):
        wide[b, lens[b]:] = float("nan")
    w, bias, state = _draw((D, W), 6, dt, 0.5), _draw((D,), 7, dt), _draw((B, W - 1, D), 8, dt)
    want, mag, kept, _ = ref.conv(x, w, bias, state, lens, True)
    s = state.cuda()
    got, st = kda.conv_prefill(wide.cuda()[:, :, lead:lead + D], w.cuda(), bias.cuda(), s, lens=lens.cuda(), state_out=s)
    torch.cuda.synchronize()
    assert st is s and np.array_equal(ref.f64(s), kept)
    _inside(got, want, mag, W, dt)


@pytest.mark.parametrize("N,D,W,dtype", [(1, 8, 4, "bf16"), (5, 77, 3, "bf16"), (300, 136, 4, "bf16"), (3, 50, 2, "f32"),
                                         (2, 4096, 4, "f32")])
def test_conv_step_matches_definition_and_continues_a_prompt(N, D, W, dtype):
    """Tokens one by one after a prompt equal the whole sequence at once, bit for bit, and the
    definition within its tolerance."""
    kda = _kda()
    dt = DT[dtype]
    T, more = 6, 5
    x = _draw((N, T + more, D), 9, dt)
    w, bias = _draw((D, W), 10, dt, 0.5), _draw((D,), 11, dt)
    want, mag, kept, _ = ref.conv(x, w, bias, None, None, True)
    xd, wd, bd = x.cuda(), w.cuda(), bias.cuda()
    y0, s = kda.conv_prefill(xd[:, :T].contiguous(), wd, bd)
    steps = [kda.conv_step(xd[:, T + i], wd, s, bd) for i in range(more)]
    whole, _ = kda.conv_prefill(xd, wd, bd)
    torch.cuda.synchronize()
    got = torch.cat([y0, torch.stack(steps, 1)], 1)
    assert torch.equal(got, whole)
    _inside(got, want, mag, W, dt)
    assert np.array_equal(ref.f64(s), kept)


def test_conv_empty_calls():
    kda = _kda()
    w = torch.ones(16, 4, device="cuda")
    s = torch.randn(2, 3, 16, device="cuda")
    y, so = kda.conv_prefill(torch.empty(2, 0, 16, device="cuda"), w, None, s)
    assert y.shape == (2, 0, 16) and torch.equal(so, s)
    _, so = kda.conv_prefill(torch.empty(2, 0, 16, device="cuda"), w)
    assert bool((so == 0).all())
    y, so = kda.conv_prefill(torch.empty(0, 5, 16, device="cuda"), w)
    assert y.shape == (0, 5, 16) and so.shape == (0, 3, 16)
    assert kda.conv_step(torch.empty(0, 16, device="cuda"), w, torch.empty(0, 3, 16, device="cuda")).shape == (0, 16)
