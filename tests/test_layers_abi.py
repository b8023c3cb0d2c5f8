"""Refusals of the C entry points of the packed attention, the 4-bit cache and the gated delta rule on the host (no GPU
needed, no kernel is launched).  Fake, never-dereferenced pointer values are used, so the calls that pass them are
skipped where a GPU is present.
"""
import ctypes

import pytest

import chunked_gated_delta_13_amd as kda
from chunked_gated_delta_13_amd import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BF16, F32 = 0, 1
BIG = 1 << 40   # fake, well-separated, 16-byte-aligned addresses
NAN, INF = float("nan"), float("inf")


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


def _attn(lib, q=_at(0), k=_at(1), v=_at(2), cq=_at(3), ck=_at(4), o=_at(5), B=2, Nq=10, Nk=30, H=4, Hkv=2, d=64, scale=0.1, qs=256,
          ks=128, vs=128, dt=BF16, ws=None, wb=0):
    return lib.kda_attn_prefill(_vp(q), _vp(k), _vp(v), _vp(cq), _vp(ck), _vp(o), B, Nq, Nk, H, Hkv, d, scale, qs, ks, vs, dt, _vp(ws), wb,
                                None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(Nq=-1), INVALID), (dict(Nk=-1), INVALID), (dict(H=-1), INVALID), (dict(d=0), INVALID),
    (dict(dt=9), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(H=1 << 17, Hkv=1 << 17), UNSUPPORTED), (dict(Nq=1 << 30, Nk=1 << 30), UNSUPPORTED),
    (dict(B=1 << 23), UNSUPPORTED), (dict(Nk=(1 << 30) + 1, ks=128), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(scale=2.4e38), INVALID),
    (dict(ck=None), INVALID),                                             # as many keys as queries without cu_k
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cq=None), INVALID), (dict(o=None), INVALID),
    (dict(qs=255), INVALID), (dict(qs=260), INVALID), (dict(ks=127), INVALID), (dict(vs=132), INVALID),
    (dict(q=_at(0) + 8), INVALID), (dict(o=_at(5) + 2), INVALID), (dict(cq=_at(3) + 2), INVALID), (dict(ck=_at(4) + 1), INVALID),
    (dict(o=_at(0)), INVALID), (dict(o=_at(1)), INVALID), (dict(o=_at(3)), INVALID), (dict(o=_at(2) - 16), INVALID),
    (dict(ws=_at(6) + 4, wb=1 << 30), INVALID),
])
def test_attn_prefill_refusals(lib, host_only, kw, expect):
    assert _attn(lib, **kw) == expect


def test_attn_prefill_workspace(lib, host_only):
    need = lib.kda_attn_prefill_workspace_bytes(1, 8, 4000, 4, 2, 64, BF16)
    assert need > 0
    many = dict(B=1, Nq=8, Nk=4000)
    assert _attn(lib, ws=_at(6), wb=need - 1, **many) == WORKSPACE
    assert _attn(lib, ws=_at(5), wb=need, **many) == INVALID              # over the outputs
    assert _attn(lib, ws=_at(1) + 16, wb=need, **many) == INVALID         # over the keys
    assert lib.kda_attn_prefill_workspace_bytes(1, 100000, 100000, 56, 8, 128, BF16) == 0
    assert lib.kda_attn_prefill_workspace_bytes(1, 8, 4000, 4, 3, 64, BF16) == 0


def test_attn_prefill_noops(lib):
    none = dict(q=None, k=None, v=None, cq=None, ck=None, o=None)
    assert _attn(lib, B=0, Nq=30, **none) == OK
    assert _attn(lib, Nq=0, Nk=0, **none) == OK
    assert _attn(lib, H=0, Hkv=0, Nq=30, **none) == OK


def _write(lib, k=_at(0), v=_at(1), kc=_at(2), vc=_at(3), pg=_at(4), cu=_at(5), st=_at(6), B=2, N=10, Hkv=2, d=64, n_pages=9, max_pages=3,
           page=16, ks=128, vs=128, dt=BF16):
    return lib.kda_cache_write(_vp(k), _vp(v), _vp(kc), _vp(vc), _vp(pg), _vp(cu), _vp(st), B, N, Hkv, d, n_pages, max_pages, page, ks, vs,
                               dt, None)


def _read(lib, kc=_at(2), vc=_at(3), pg=_at(4), cu=_at(5), st=_at(6), k=_at(0), v=_at(1), B=2, N=10, Hkv=2, d=64, n_pages=9, max_pages=3,
          page=16, dt=BF16):
    return lib.kda_cache_read(_vp(kc), _vp(vc), _vp(pg), _vp(cu), _vp(st), _vp(k), _vp(v), B, N, Hkv, d, n_pages, max_pages, page, dt, None)


BOTH = [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(page=0), INVALID), (dict(page=-16), INVALID), (dict(page=24), INVALID), (dict(page=8), UNSUPPORTED),
    (dict(page=1 << 17), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED), (dict(d=0), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(dt=2), INVALID), (dict(cu=None), INVALID),                      # one token each: N == B
    (dict(N=1 << 27, Hkv=2), UNSUPPORTED), (dict(Hkv=1 << 16), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(pg=None), INVALID),
    (dict(k=_at(0) + 2), INVALID), (dict(v=_at(1) + 8), INVALID), (dict(kc=_at(2) + 4), INVALID), (dict(pg=_at(4) + 2), INVALID),
    (dict(cu=_at(5) + 1), INVALID), (dict(st=_at(6) + 2), INVALID),
    (dict(kc=_at(0)), INVALID), (dict(v=_at(2)), INVALID),
]


@pytest.mark.parametrize("kw,expect", BOTH + [
    (dict(vc=_at(2)), INVALID), (dict(kc=_at(4)), INVALID), (dict(ks=127), INVALID), (dict(vs=132), INVALID), (dict(kc=_at(1) + 2 * 128 * 9), INVALID),
])
def test_cache_write_refusals(lib, host_only, kw, expect):
    assert _write(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", BOTH + [(dict(v=_at(0) + 16), INVALID), (dict(k=_at(4)), INVALID)])
def test_cache_read_refusals(lib, host_only, kw, expect):
    assert _read(lib, **kw) == expect


def test_cache_noops(lib):
    none = dict(k=None, v=None, kc=None, vc=None, pg=None, cu=None, st=None)
    for call in (_write, _read):
        assert call(lib, B=0, N=0, **none) == OK
        assert call(lib, Hkv=0, N=2, **none) == OK


def _step(lib, q=_at(0), kc=_at(1), vc=_at(2), pg=_at(3), ln=_at(4), o=_at(5), N=2, m=1, H=4, Hkv=2, d=64, n_pages=9, max_pages=30, page=16,
          scale=0.1, qs=256, dt=BF16, ws=_at(6), wb=1 << 30):
    return lib.kda_attn_step(_vp(q), _vp(kc), _vp(vc), _vp(pg), _vp(ln), _vp(o), N, m, H, Hkv, d, n_pages, max_pages, page, scale, qs, dt,
                             _vp(ws), wb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(m=-1), INVALID), (dict(H=-1), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dt=7), INVALID), (dict(page=48), INVALID), (dict(page=8), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED),
    (dict(N=1 << 20, m=100), UNSUPPORTED), (dict(N=1 << 24, H=2, Hkv=2), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID),
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(pg=None), INVALID), (dict(ln=None), INVALID),
    (dict(o=None), INVALID), (dict(qs=255), INVALID), (dict(qs=260), INVALID), (dict(q=_at(0) + 8), INVALID), (dict(o=_at(5) + 8), INVALID),
    (dict(ln=_at(4) + 2), INVALID), (dict(kc=_at(1) + 8), INVALID), (dict(ws=_at(6) + 8), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wb=0), WORKSPACE), (dict(o=_at(0)), INVALID), (dict(o=_at(1)), INVALID), (dict(o=_at(4)), INVALID), (dict(ws=_at(1)), INVALID),
    (dict(ws=_at(5)), INVALID),
])
def test_attn_step_refusals(lib, host_only, kw, expect):
    assert _step(lib, **kw) == expect


def test_attn_step_noops_and_sizes(lib):
    none = dict(q=None, kc=None, vc=None, pg=None, ln=None, o=None, ws=None, wb=0)
    assert _step(lib, N=0, **none) == OK
    assert _step(lib, m=0, **none) == OK
    assert _step(lib, H=0, Hkv=0, **none) == OK
    size = lib.kda_attn_step_workspace_bytes
    assert size(1, 1, 8, 2, 128, 8, 16, BF16) == 0                        # one slot of keys
    assert size(1, 1, 8, 2, 128, 1000, 16, BF16) > 0 and size(1, 1, 8, 3, 128, 1000, 16, BF16) == 0


def _delta(lib, q=_at(0), k=_at(1), v=_at(2), g=_at(3), b=_at(4), S0=_at(5), ln=_at(6), o=_at(7), S=_at(8), B=2, T=300, H=4, Hk=2, dk=64, dv=128,
           qs=128, ks=128, vs=512, dt=BF16, seg=0, ws=_at(9), wb=1 << 30):
    return lib.kda_delta_prefill(_vp(q), _vp(k), _vp(v), _vp(g), _vp(b), _vp(S0), _vp(ln), _vp(o), _vp(S), B, T, H, Hk, dk, dv, qs, ks, vs, dt,
                                 seg, _vp(ws), wb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(Hk=-1), INVALID), (dict(Hk=3), INVALID), (dict(Hk=0), INVALID),
    (dict(dk=0), INVALID), (dict(dk=32), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(dt=5), INVALID), (dict(seg=-64), INVALID),
    (dict(seg=100), INVALID), (dict(B=1 << 19), UNSUPPORTED), (dict(B=60000, T=1 << 30, H=1 << 14, Hk=1), INVALID),
    (dict(B=1 << 17, T=1 << 12, seg=64, wb=0), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(b=None), INVALID),
    (dict(o=None), INVALID), (dict(qs=127), INVALID), (dict(ks=132), INVALID), (dict(vs=511), INVALID), (dict(q=_at(0) + 8), INVALID),
    (dict(g=_at(3) + 2), INVALID), (dict(b=_at(4) + 1), INVALID), (dict(ln=_at(6) + 2), INVALID), (dict(S0=_at(5) + 4), INVALID),
    (dict(S=_at(8) + 8), INVALID), (dict(o=_at(7) + 2), INVALID), (dict(S=_at(5) + 16), INVALID), (dict(o=_at(5)), INVALID),
    (dict(o=_at(2)), INVALID), (dict(S=_at(3)), INVALID), (dict(S=_at(7)), INVALID),
    (dict(seg=64, ws=None), WORKSPACE), (dict(seg=64, wb=100), WORKSPACE), (dict(seg=64, ws=_at(9) + 4), INVALID),
    (dict(seg=64, ws=_at(5)), INVALID), (dict(seg=64, ws=_at(0)), INVALID),
])
def test_delta_prefill_refusals(lib, host_only, kw, expect):
    assert _delta(lib, **kw) == expect


def _dstep(lib, q=_at(0), k=_at(1), v=_at(2), g=_at(3), b=_at(4), S=_at(5), o=_at(6), N=2, H=4, Hk=2, dk=64, dv=128, qs=128, ks=128, vs=512,
           dt=F32):
    return lib.kda_delta_step(_vp(q), _vp(k), _vp(v), _vp(g), _vp(b), _vp(S), _vp(o), N, H, Hk, dk, dv, qs, ks, vs, dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INVALID), (dict(Hk=3), INVALID), (dict(dk=96), UNSUPPORTED), (dict(dt=3), INVALID), (dict(N=1 << 19), UNSUPPORTED),
    (dict(S=None), INVALID), (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(o=None), INVALID), (dict(qs=127), INVALID),
    (dict(S=_at(5) + 4), INVALID), (dict(S=_at(2)), INVALID), (dict(o=_at(5)), INVALID), (dict(o=_at(0)), INVALID),
])
def test_delta_step_refusals(lib, host_only, kw, expect):
    assert _dstep(lib, **kw) == expect


def test_delta_noops_and_sizes(lib):
    none = dict(q=None, k=None, v=None, g=None, b=None, S0=None, ln=None, o=None, S=None, ws=None, wb=0)
    assert _delta(lib, B=0, **none) == OK
    assert _delta(lib, H=0, Hk=0, **none) == OK
    assert _delta(lib, T=0, **none) == OK
    assert _dstep(lib, N=0, q=None, k=None, v=None, g=None, b=None, S=None, o=None) == OK
    assert _dstep(lib, H=0, Hk=0, q=None, k=None, v=None, g=None, b=None, S=None, o=None) == OK
    size = lib.kda_delta_prefill_workspace_bytes
    assert size(2, 300, 4, 2, 64, 128, BF16, 64) == 8 * 4 * (5 * 64 * 128 + 4 * 64 * 64) + 8 * 4 * 4
    assert size(2, 300, 4, 2, 64, 128, BF16, 320) == 0 and size(2, 300, 4, 3, 64, 128, BF16, 64) == 0


def test_workspace_queries_of_the_package():
    import torch
    for size, args in ((kda.attn_prefill_workspace_bytes, (1, 8, 4000, 4, 2, 64)), (kda.attn_step_workspace_bytes, (1, 1, 8, 2, 128, 1000, 16)),
                       (kda.delta_workspace_bytes, (1, 20000, 2, 1, 64, 64))):
        assert size(*args) == size(*args, dtype=torch.bfloat16) > 0
        with pytest.raises(TypeError, match="bfloat16 or float32"):
            size(*args, dtype=torch.float16)
        with pytest.raises(ValueError, match="32 bits"):
            size(2 ** 40, *args[1:])
    assert kda.cache_page_bytes(128, 64) == 64 * 68 and kda.cache_page_bytes(64, 16) == 16 * 34
