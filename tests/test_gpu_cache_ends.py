"""Sequence ends that lie outside the packed tensor: writing to the 4-bit cache and reading it back clamp them as the
attention of prompts does, so that a call is, to the bit, the call with the clamped ends.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref
from tests.test_gpu_cache import DT, _draw, _i32, _kda, _pool, _table

pytestmark = pytest.mark.gpu

N = 40
ENDS = [(-7, 15, 2 ** 31 - 1), (-7, -3, N), (-2 ** 31, 15, N), (-2 ** 31, -2 ** 31, 2 ** 31 - 1), (N + 5, N + 9, 2 ** 31 - 1), (3, 9, 9)]


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("cu", ENDS, ids=lambda c: "_".join(map(str, c)))
def test_ends_outside_the_tensor_are_clamped(cu, dtype, d):
    kda = _kda()
    print("ends", cu, dtype, d, flush=True)
    Hkv, page, start = 2, 16, [5, 0]
    clamped = np.clip(cu, 0, N)
    new = np.diff(clamped).tolist()
    table, n_pages = _table([N + 5, N], page, 1)
    k, v = _draw(1, dtype, N, Hkv, d), _draw(2, dtype, N, Hkv, d)
    pools, rows = [], []
    for c in (cu, clamped):
        kc, vc = _pool(n_pages, Hkv, d, page, 3), _pool(n_pages, Hkv, d, page, 4)
        kda.cache_write(k.cuda(), v.cuda(), kc, vc, _i32(table), _i32(c), _i32(start))
        ko = torch.full((N, Hkv, d), 9.0, dtype=DT[dtype], device="cuda")
        vo = ko.clone()
        kda.cache_read(kc, vc, _i32(table), _i32(c), N, d, _i32(start), dtype=DT[dtype], k=ko, v=vo)
        torch.cuda.synchronize()
        pools.append((kc, vc))
        rows.append((ko, vo))
    for a, b in zip(pools[0] + rows[0], pools[1] + rows[1]):
        assert torch.equal(a, b)
    for c, o, x in zip(pools[0], rows[0], (k, v)):
        want, _ = lref.quantise(ref.f64(x))
        inside = np.zeros(N, bool)
        for b, n in enumerate(new):
            at = slice(clamped[b], clamped[b + 1])
            inside[at] = True
            got = lref.rows_of(c, table[b], start[b] + n, page, d)[start[b]:]
            assert np.array_equal(got, want[at]) and np.array_equal(ref.f64(o[at]), want[at])
        assert (ref.f64(o)[~inside] == 9.0).all()
