"""Refusals of the token mixers' C entry points on the host (no GPU needed, no kernel is launched).

Fake, never-dereferenced pointer values are used, so the calls that pass them are skipped where a GPU
is present.
"""
import ctypes

import pytest

import chunked_gated_delta_13_amd as kda
from chunked_gated_delta_13_amd import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 4
BF16, F32 = 0, 1
BIG = 1 << 40   # fake, well-separated, 16-byte-aligned addresses


def _at(i):
    return BIG * (i + 1)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.fixture
def host_only():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake pointers are only passed where no GPU exists")


def _vp(x):
    return ctypes.c_void_p(x)


def _conv(lib, x=_at(0), w=_at(1), bias=_at(2), s_in=_at(3), lens=_at(4), y=_at(5), s_out=_at(6), B=2, T=10, D=64,
          W=4, stride=64, silu=1, dt=BF16):
    return lib.kda_conv_prefill(_vp(x), _vp(w), _vp(bias), _vp(s_in), _vp(lens), _vp(y), _vp(s_out), B, T, D, W,
                                stride, silu, dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-1), INVALID), (dict(W=0), INVALID),
    (dict(dt=9), INVALID), (dict(stride=63), INVALID), (dict(stride=-64), INVALID),
    (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(B=60000, T=1 << 30, D=1 << 20, stride=1 << 20), INVALID),      # more bytes than an address space holds
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=_at(0) + 1), INVALID), (dict(w=_at(1) + 1), INVALID), (dict(y=_at(5) + 1), INVALID),
    (dict(lens=_at(4) + 2), INVALID), (dict(s_out=_at(6) + 1), INVALID),
    (dict(y=_at(0)), INVALID), (dict(y=_at(0) + 2 * 10 * 64 * 2 - 2), INVALID),   # over x, over its last element
    (dict(stride=100, y=_at(0) + 2 * (64 + 10)), INVALID),                # in a gap between x's rows
    (dict(s_out=_at(3) + 2), INVALID), (dict(s_out=_at(5)), INVALID), (dict(y=_at(3)), INVALID),
])
def test_conv_prefill_refusals(lib, host_only, kw, expect):
    assert _conv(lib, **kw) == expect


def test_conv_prefill_noops(lib):
    none = dict(x=None, w=None, bias=None, s_in=None, lens=None, y=None, s_out=None)
    assert _conv(lib, B=0, **none) == OK
    assert _conv(lib, D=0, stride=0, **none) == OK


def _cstep(lib, x=_at(0), w=_at(1), bias=_at(2), s=_at(3), y=_at(4), N=2, D=64, W=4, stride=64, dt=F32):
    return lib.kda_conv_step(_vp(x), _vp(w), _vp(bias), _vp(s), _vp(y), N, D, W, stride, 1, dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(W=5), UNSUPPORTED), (dict(dt=2), INVALID), (dict(stride=10), INVALID),
    (dict(s=None), INVALID), (dict(y=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(s=_at(3) + 2), INVALID), (dict(y=_at(3)), INVALID), (dict(y=_at(0)), INVALID), (dict(s=_at(0)), INVALID),
    (dict(N=65536), UNSUPPORTED),
])
def test_conv_step_refusals(lib, host_only, kw, expect):
    assert _cstep(lib, **kw) == expect


def test_conv_step_noops(lib):
    assert _cstep(lib, N=0, x=None, w=None, bias=None, s=None, y=None) == OK


def test_conv_binding_refuses_what_it_cannot_run():
    import torch
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="HIP device"):
        kda.conv_prefill(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        kda.conv_step(x[:, 0], w, torch.zeros(2, 3, 8))
