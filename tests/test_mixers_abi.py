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


def _ssm(lib, B=2, T=200, H=4, G=2, n=128, p=64, dt=BF16, seg=0, ws=None, ws_bytes=0, strides=None, **ptr):
    q = dict(x=_at(0), dt_=_at(1), A=_at(2), Bm=_at(3), Cm=_at(4), D=_at(5), z=_at(6), bias=_at(7), S0=_at(8), lens=_at(9),
             y=_at(10), S_T=_at(11))
    q.update(ptr)
    st = strides or (H * p, H, G * n, G * n, H * p)
    return lib.kda_ssm_prefill(*[_vp(v) for v in q.values()], B, T, H, G, n, p, *st, dt, seg, _vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID),
    (dict(dt=5), INVALID), (dict(n=0), INVALID), (dict(n=96), UNSUPPORTED), (dict(p=32), UNSUPPORTED),
    (dict(seg=-64), INVALID), (dict(seg=100), INVALID),
    (dict(B=1 << 20, H=1 << 10, G=1), UNSUPPORTED), (dict(B=1 << 30, T=1 << 30, H=1 << 20, G=1), INVALID),
    (dict(x=None), INVALID), (dict(dt_=None), INVALID), (dict(A=None), INVALID), (dict(Bm=None), INVALID),
    (dict(Cm=None), INVALID), (dict(y=None), INVALID),
    (dict(x=_at(0) + 8), INVALID), (dict(Bm=_at(3) + 2), INVALID), (dict(z=_at(6) + 8), INVALID),
    (dict(dt_=_at(1) + 1), INVALID), (dict(A=_at(2) + 2), INVALID), (dict(y=_at(10) + 8), INVALID),
    (dict(S0=_at(8) + 4), INVALID), (dict(lens=_at(9) + 1), INVALID),
    (dict(strides=(255, 4, 256, 256, 256)), INVALID),      # shorter than a row
    (dict(strides=(260, 4, 256, 256, 256)), INVALID),      # rows off 16-byte boundaries
    (dict(strides=(256, 3, 256, 256, 256)), INVALID),
    (dict(strides=(256, 4, 256, 256, 0)), INVALID),
    (dict(strides=(1 << 23, 4, 256, 256, 256)), UNSUPPORTED),   # 64 rows past 32-bit offsets
    (dict(y=_at(0)), INVALID), (dict(y=_at(11)), INVALID), (dict(y=_at(8)), INVALID), (dict(S_T=_at(3)), INVALID),
    (dict(S_T=_at(8) + 64), INVALID), (dict(S_T=_at(2)), INVALID),
    (dict(seg=64), WORKSPACE), (dict(seg=64, ws=_at(12), ws_bytes=100), WORKSPACE),
    (dict(seg=64, ws=_at(12) + 8, ws_bytes=1 << 30), INVALID), (dict(seg=64, ws=_at(0), ws_bytes=1 << 30), INVALID),
    (dict(seg=64, ws=_at(11), ws_bytes=1 << 30), INVALID),
])
def test_ssm_prefill_refusals(lib, host_only, kw, expect):
    assert _ssm(lib, **kw) == expect


@pytest.mark.parametrize("kw", [dict(B=1 << 20, T=1, H=8, G=1), dict(B=1 << 11, T=1 << 16, H=8, G=1, seg=64)])
def test_ssm_refuses_more_units_than_a_launch_holds(lib, host_only, kw):
    assert _ssm(lib, **kw) == UNSUPPORTED
    assert lib.kda_ssm_prefill_workspace_bytes(kw["B"], kw["T"], kw["H"], 1, 128, 64, BF16, kw.get("seg", 0)) == 0


def test_ssm_step_refuses_more_units_than_a_launch_holds(lib, host_only):
    assert _sstep(lib, N=1 << 20, H=8, G=1) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(B=65535, T=1, H=512, Hkv=1), dict(B=1, T=1 << 28, H=4, Hkv=1),
                                dict(B=1, T=1 << 20, H=1, Hkv=1 << 0, window=1 << 28, sinks=1 << 28, d=128)])
def test_window_prefill_refuses_more_than_a_launch_holds(lib, host_only, kw):
    assert _window(lib, **kw) == UNSUPPORTED


def test_window_step_refuses_more_units_than_a_launch_holds(lib, host_only):
    assert _wstep(lib, N=65535, H=512, Hkv=1) == UNSUPPORTED
    assert lib.kda_window_step_workspace_bytes(65535, 512, 1, 64, 20, 4, F32) == 0


def test_ssm_workspace(lib):
    need = lib.kda_ssm_prefill_workspace_bytes
    assert need(2, 200, 4, 2, 128, 64, BF16, 64) == 8 * 4 * (128 * 64 * 4 + 4)   # 8 heads, 4 segments
    assert need(2, 200, 4, 2, 128, 64, BF16, 256) == 0
    assert need(2, 200, 4, 3, 128, 64, BF16, 64) == 0                             # a refused shape
    assert need(2, 0, 4, 2, 128, 64, BF16, 64) == 0


def test_ssm_noops(lib):
    none = {k: None for k in ("x", "dt_", "A", "Bm", "Cm", "D", "z", "bias", "S0", "lens", "y", "S_T")}
    assert _ssm(lib, B=0, **none) == OK
    assert _ssm(lib, H=0, G=0, **none) == OK


def _sstep(lib, N=2, H=4, G=2, n=128, p=64, dt=F32, strides=None, **ptr):
    q = dict(x=_at(0), dt_=_at(1), A=_at(2), Bm=_at(3), Cm=_at(4), D=_at(5), z=_at(6), bias=_at(7), S=_at(8), y=_at(9))
    q.update(ptr)
    st = strides or (H * p, H, G * n, G * n, H * p)
    return lib.kda_ssm_step(*[_vp(v) for v in q.values()], N, H, G, n, p, *st, dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(G=3), INVALID), (dict(n=32), UNSUPPORTED), (dict(dt=2), INVALID),
    (dict(S=None), INVALID), (dict(y=None), INVALID), (dict(x=None), INVALID), (dict(S=_at(8) + 4), INVALID),
    (dict(y=_at(8)), INVALID), (dict(S=_at(0)), INVALID), (dict(strides=(256, 4, 255, 256, 256)), INVALID),
    (dict(N=1 << 24), UNSUPPORTED),
])
def test_ssm_step_refusals(lib, host_only, kw, expect):
    assert _sstep(lib, **kw) == expect


def test_ssm_binding_refuses_what_it_cannot_run():
    import torch
    x, b = torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 1, 64)
    with pytest.raises(ValueError, match="HIP device"):
        kda.ssm_prefill(x, x[..., 0], torch.zeros(2), b, b)
    with pytest.raises(ValueError, match="HIP device"):
        kda.ssm_step(x[:, 0], x[:, 0, :, 0], torch.zeros(2), b[:, 0], b[:, 0], torch.zeros(2, 2, 64, 64))


def _window(lib, B=2, T=50, H=4, Hkv=2, d=64, window=20, sinks=4, scale=0.125, dt=BF16, strides=None, ws=None,
            ws_bytes=0, **ptr):
    q = dict(q=_at(0), k=_at(1), v=_at(2), kc=_at(3), vc=_at(4), start=_at(5), lens=_at(6), o=_at(7))
    q.update(ptr)
    st = strides or (H * d, Hkv * d, Hkv * d)
    return lib.kda_window_prefill(*[_vp(x) for x in q.values()], B, T, H, Hkv, d, window, sinks, scale, *st, dt, _vp(ws), ws_bytes,
                                  None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(dt=3), INVALID), (dict(d=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(B=65536), UNSUPPORTED), (dict(window=1 << 29), UNSUPPORTED),
    (dict(B=65535, T=1 << 29, H=4), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(kc=None, vc=None), INVALID),     # start without caches
    (dict(q=_at(0) + 8), INVALID), (dict(v=_at(2) + 2), INVALID), (dict(o=_at(7) + 4), INVALID),
    (dict(kc=_at(3) + 8), INVALID), (dict(start=_at(5) + 2), INVALID), (dict(lens=_at(6) + 1), INVALID),
    (dict(strides=(255, 128, 128)), INVALID), (dict(strides=(260, 128, 128)), INVALID), (dict(strides=(256, 127, 128)), INVALID),
    (dict(o=_at(0)), INVALID), (dict(o=_at(3)), INVALID), (dict(vc=_at(3)), INVALID), (dict(kc=_at(1)), INVALID),
    (dict(vc=_at(5)), INVALID),
])
def test_window_prefill_refusals(lib, host_only, kw, expect):
    assert _window(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws=_at(8), ws_bytes=64), WORKSPACE), (dict(ws=_at(8) + 4, ws_bytes=1 << 30), INVALID),
    (dict(ws=_at(3), ws_bytes=1 << 30), INVALID), (dict(ws=_at(7) + 16, ws_bytes=1 << 30), INVALID),
])
def test_window_prefill_workspace_refusals(lib, host_only, kw, expect):
    assert _window(lib, window=5000, **kw) == expect


def test_window_prefill_workspace(lib):
    need = lib.kda_window_prefill_workspace_bytes
    per = 2 * 50 * 4 * (64 + 4) * 4
    assert need(2, 50, 4, 2, 64, 5000, 4, BF16, 1) % per == 0 and need(2, 50, 4, 2, 64, 5000, 4, BF16, 1) >= 2 * per
    assert need(2, 50, 4, 2, 64, 5000, 4, BF16, 0) == 0           # 50 keys at most
    assert need(64, 4096, 8, 2, 64, 5000, 4, BF16, 1) == 0        # enough queries
    assert need(0, 50, 4, 2, 64, 5000, 4, BF16, 1) == 0 and need(2, 0, 4, 2, 64, 5000, 4, BF16, 1) == 0
    assert need(2, 50, 4, 3, 64, 5000, 4, BF16, 1) == 0           # refused shapes need nothing


def test_window_noops(lib):
    none = {x: None for x in ("q", "k", "v", "kc", "vc", "start", "lens", "o")}
    assert _window(lib, B=0, **none) == OK
    assert _window(lib, H=0, Hkv=0, **none) == OK
    assert _window(lib, T=0, **none) == OK


def _wstep(lib, N=2, H=4, Hkv=2, d=64, window=20, sinks=4, scale=0.125, dt=F32, strides=None, ws=None, ws_bytes=0, **ptr):
    q = dict(q=_at(0), k=_at(1), v=_at(2), kc=_at(3), vc=_at(4), pos=_at(5), o=_at(6))
    q.update(ptr)
    st = strides or (H * d, Hkv * d, Hkv * d)
    return lib.kda_window_step(*[_vp(x) for x in q.values()], N, H, Hkv, d, window, sinks, scale, *st, dt, _vp(ws), ws_bytes,
                               None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(Hkv=3), INVALID), (dict(window=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(dt=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(pos=None), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(o=_at(0)), INVALID), (dict(o=_at(4)), INVALID),
    (dict(vc=_at(3) + 16), INVALID), (dict(pos=_at(5) + 2), INVALID), (dict(strides=(255, 128, 128)), INVALID),
    (dict(window=5000), WORKSPACE), (dict(window=5000, ws=_at(7), ws_bytes=64), WORKSPACE),
    (dict(window=5000, ws=_at(7) + 4, ws_bytes=1 << 30), INVALID), (dict(window=5000, ws=_at(3), ws_bytes=1 << 30), INVALID),
])
def test_window_step_refusals(lib, host_only, kw, expect):
    assert _wstep(lib, **kw) == expect


def test_window_step_noop_and_workspace(lib):
    assert _wstep(lib, N=0, q=None, k=None, v=None, kc=None, vc=None, pos=None, o=None) == OK
    need = lib.kda_window_step_workspace_bytes
    assert need(1, 8, 2, 128, 100, 4, BF16) == 0 and need(0, 8, 2, 128, 5000, 4, BF16) == 0
    assert need(1, 8, 3, 128, 5000, 4, BF16) == 0
    per = 8 * (128 + 4) * 4
    assert need(1, 8, 2, 128, 5000, 4, BF16) % per == 0 and need(1, 8, 2, 128, 5000, 4, BF16) >= 2 * per


def test_window_binding_refuses_what_it_cannot_run():
    import torch
    q = torch.zeros(2, 5, 2, 64)
    with pytest.raises(ValueError, match="HIP device"):
        kda.window_prefill(q, q, q, 4)
    with pytest.raises(ValueError, match="HIP device"):
        kda.window_step(q[:, 0], q[:, 0], q[:, 0], q, q, torch.zeros(2, dtype=torch.int32), 4)


def test_binding_refuses_sizes_past_32_bits():
    """What the C integers would cut off is refused before the call."""
    with pytest.raises(ValueError, match="32 bits"):
        kda.window_step_workspace_bytes(1, 8, 2, 128, 2 ** 32 + 20)
    with pytest.raises(ValueError, match="32 bits"):
        kda.ssm_workspace_bytes(1, 100, 1, 1, 64, 64, seg_len=-2 ** 32 + 64)
    assert kda.window_step_workspace_bytes(1, 8, 2, 128, 2 ** 31 - 1) == 0


def test_binding_refuses_what_is_no_tensor():
    with pytest.raises(TypeError, match="x must be a tensor"):
        kda.conv_step(None, None, None)
    with pytest.raises(TypeError, match="x must be a tensor"):
        kda.ssm_prefill([1.0], None, None, None, None)
    with pytest.raises(TypeError, match="q must be a tensor"):
        kda.window_prefill(3, None, None, 4)
