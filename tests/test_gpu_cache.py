"""The 4-bit paged cache on the device: what is written and read back is held to the bit, the attention over it to its
definition in 64 bits over the values that the cache stands for.

Tolerance of the attention.  u = 2^-24.  Every cached value is exact, and so are queries (fp32 ones as three bf16
parts), so a score is a sum of d products (3 d in fp32) off by at most 2 (3 d + 8) u a, with a = scale * sum |q k|; scaling
and the exponential's argument add 8 u a: a probability is off by at most e = u (6 d + 32) a + 40 u relative,
numerator and denominator alike, and by 2^-8 of 2^-8 (2^-24 in fp32) as bf16 parts.  Sums over K keys add 4 K u.  With
m = sum p |v|: |o - ref| <= (2 e + p + 4 K u) m + h |o|, p = 2^-16 or 2^-24, h the half step of the output.
"""
import numpy as np
import pytest
import torch

from tests import layers_reference as lref
from tests import mixers_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kda():
    import chunked_gated_delta_13_amd as kda
    kda.load_library()
    return kda


def _draw(seed, dtype, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype])


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(n_pages, Hkv, d, page, seed):
    """Bytes as a pool may hold them before anything is written: NaN exponents among them."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (n_pages, Hkv, page * (d // 2 + d // 32)), generator=g, dtype=torch.uint8).cuda()


def _table(lengths, page, seed, more=2, bad=-1):
    """Pages in any order; entries that no token needs hold `bad`."""
    need = [-(-n // page) for n in lengths]
    n_pages = sum(need) + more
    at = np.random.RandomState(seed).permutation(n_pages)
    table = np.full((len(lengths), max(need + [1]) + 1), bad)
    used = 0
    for b, n in enumerate(need):
        table[b, :n] = at[used:used + n]
        used += n
    return table, n_pages


def _hard(seed, dtype, n, Hkv, d):
    """Rows whose blocks differ in size by 2^40, with ties, zeros, negative zeros and single large channels."""
    x = _draw(seed, "f32", n, Hkv, d)
    g = torch.Generator().manual_seed(seed + 1)
    x = x.unflatten(-1, (-1, 32)) * torch.exp2(torch.randint(-20, 21, (n, Hkv, d // 32, 1), generator=g).float())
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -1.25, -5.0, 6.0, 0.0, -0.0, 6.5])
    x[0, :, 0, :16], x[0, :, 0, 16:] = ties, 0.0
    x[-1] = 0.0
    x[n // 2, :, -1, 5] = 1e6
    return x.flatten(-2).to(DT[dtype])


# new tokens, tokens before them, Hkv, d, page, dtype
ROWS = [
    ([1], [0], 1, 64, 16, "bf16"),
    ([17, 0, 5, 40], [15, 3, 0, 16], 2, 128, 16, "bf16"),
    ([100, 33], [7, 64], 3, 64, 32, "f32"),
    ([5, 300, 1], [1000, 0, 128], 8, 128, 128, "bf16"),
    ([2] * 67, [i % 40 for i in range(67)], 1, 128, 16, "f32"),   # more sequences than lanes of a wave
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join([str(len(c[0])), str(sum(c[0]))] + [str(x) for x in c[2:]]))
def test_cache_rows_to_the_bit(case):
    kda = _kda()
    new, before, Hkv, d, page, dtype = case
    print("cache rows", case, flush=True)
    total = [a + b for a, b in zip(new, before)]
    table, n_pages = _table(total, page, 1)
    kc, vc = _pool(n_pages, Hkv, d, page, 2), _pool(n_pages, Hkv, d, page, 3)
    cu0 = np.cumsum([0] + before)
    kda.cache_write(_hard(6, dtype, int(cu0[-1]) + 1, Hkv, d).cuda(), _hard(7, dtype, int(cu0[-1]) + 1, Hkv, d).cuda(), kc, vc,
                    _i32(table), _i32(cu0))
    old = [lref.rows_of(c, table[b], n, page, d) for c in (kc, vc) for b, n in enumerate(before)]
    lead, tail = 3, 2                                             # rows of no sequence
    cu = np.cumsum([lead] + new)
    N = int(cu[-1]) + tail
    row = 2 * Hkv + 1
    rows = torch.cat([_hard(4, dtype, N, Hkv, d), _hard(14, dtype, N, Hkv, d), _draw(5, dtype, N, 1, d)], 1)
    k, v = rows[:, :Hkv], rows[:, Hkv:2 * Hkv]
    rows_d = rows.cuda()
    kb, vb = kc.clone(), vc.clone()
    kda.cache_write(rows_d[:, :Hkv], rows_d[:, Hkv:2 * Hkv], kc, vc, _i32(table), _i32(cu), _i32(before))
    torch.cuda.synchronize()
    assert rows.shape[1] == row
    for i, (c, x, c0) in enumerate(((kc, k, kb), (vc, v, vb))):
        x, _ = lref.quantise(ref.f64(x))
        touched = np.zeros(c.shape, bool)
        for b in range(len(new)):
            got = lref.rows_of(c, table[b], total[b], page, d)
            assert np.array_equal(got[:before[b]], old[i * len(new) + b], equal_nan=True)   # earlier tokens stay
            assert np.array_equal(got[before[b]:], x[cu[b]:cu[b + 1]])
            for p in range(before[b], total[b]):
                r = p % page
                touched[table[b, p // page], :, r * (d // 2):(r + 1) * (d // 2)] = True
                at = page * (d // 2) + r * (d // 32)
                touched[table[b, p // page], :, at:at + d // 32] = True
        assert np.array_equal(c.cpu().numpy()[~touched], c0.cpu().numpy()[~touched])        # and so does all else
    # back, from the first position on and from the new ones on, in both types
    for dt in DT.values():
        all_cu = np.cumsum([1] + total)
        ko = torch.full((int(all_cu[-1]) + 1, Hkv, d), 9.0, dtype=dt, device="cuda")
        vo = ko.clone()
        kda.cache_read(kc, vc, _i32(table), _i32(all_cu), ko.shape[0], d, dtype=dt, k=ko, v=vo)
        kn, vn = kda.cache_read(kc, vc, _i32(table), _i32(cu), N, d, _i32(before), dtype=dt)
        torch.cuda.synchronize()
        for o, n, c in ((ko, kn, kc), (vo, vn, vc)):
            assert bool((o[:1] == 9.0).all()) and bool((o[-1:] == 9.0).all()) and o.dtype == dt == n.dtype
            for b in range(len(new)):
                want = lref.rows_of(c, table[b], total[b], page, d)
                assert np.array_equal(ref.f64(o[all_cu[b]:all_cu[b + 1]]), want, equal_nan=True)
                assert np.array_equal(ref.f64(n[cu[b]:cu[b + 1]]), want[before[b]:], equal_nan=True)


def test_sizes_at_the_ends_of_the_range():
    """Blocks from the smallest numbers to the largest, and infinities and NaN."""
    kda = _kda()
    tops = [0.0, 1e-45, 2.0 ** -149, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126, 2.0 ** -123, 1e-30, 1.0, 7.0, 7.0000005, 1e20, 2.0 ** 95,
            6 * 2.0 ** 95, 7 * 2.0 ** 95, 1e30, 3.4e38, float("inf"), -float("inf"), float("nan")]
    n = len(tops)
    x = torch.linspace(-1, 1, 64).repeat(n, 1, 1) * torch.tensor([t if np.isfinite(t) else 1.0 for t in tops])[:, None, None]
    for i, t in enumerate(tops):
        x[i, 0, 40] = t
    table = [[1, 0, -1]]
    kc, vc = _pool(2, 1, 64, 16, 1), _pool(2, 1, 64, 16, 2)
    kda.cache_write(x.cuda(), (-x).cuda(), kc, vc, _i32(table), _i32([0, n]))
    k, v = kda.cache_read(kc, vc, _i32(table), _i32([0, n]), n, 64, dtype=torch.float32)
    torch.cuda.synchronize()
    want, _ = lref.quantise(ref.f64(x))
    assert np.array_equal(ref.f64(k), want, equal_nan=True) and np.array_equal(ref.f64(v), -want, equal_nan=True)
    assert np.isnan(want[-3:, 0, 32:]).all() and np.isfinite(want[-3:, 0, :32]).all()


def test_one_token_each_and_entries_outside_the_pool():
    """Without cu a row of the table has one token.  Entries outside the pool and positions past the table are neither
    written nor followed: they read back as zeros, and the pool keeps what it held."""
    kda = _kda()
    N, Hkv, d, page = 7, 2, 128, 16
    table = np.array([[0, 1], [2, 3], [4, 99], [-5, 5], [6, 2 ** 31 - 1], [7, 7], [-2 ** 31, -1]])
    start = [0, 16, 16, 3, 31, 32, 5]          # the last but one lies past the table
    kc, vc = _pool(8, Hkv, d, page, 1), _pool(8, Hkv, d, page, 2)
    kb = kc.clone()
    k, v = _draw(1, "bf16", N, Hkv, d), _draw(2, "bf16", N, Hkv, d)
    kda.cache_write(k.cuda(), v.cuda(), kc, vc, _i32(table), None, _i32(start))
    ko, vo = kda.cache_read(kc, vc, _i32(table), None, N, d, _i32(start))
    torch.cuda.synchronize()
    has = np.array([True, True, False, False, False, False, False])
    for o, x in ((ko, k), (vo, v)):
        want, _ = lref.quantise(ref.f64(x))
        assert np.array_equal(ref.f64(o)[has], want[has]) and (ref.f64(o)[~has] == 0).all()
    same = (kc == kb).all(-1).all(-1).cpu().numpy()
    assert same[[1, 2, 4, 5, 6, 7]].all() and not same[[0, 3]].any()
    # negative starts count as 0
    kda.cache_write(k[:1].cuda(), v[:1].cuda(), kc, vc, _i32(table[:1]), None, _i32([-9]))
    torch.cuda.synchronize()
    assert np.array_equal(lref.rows_of(kc, table[0], 1, page, d), lref.quantise(ref.f64(k[:1]))[0])


def _inside(got, want, mag, a, d, keys, dtype):
    g, h = ref.f64(got), ref.half_step(DT[dtype])
    e = ref.U32 * ((6 * d + 32) * a[..., None] + 40)
    tol = (2 * e + (2.0 ** -16 if dtype == "bf16" else 2.0 ** -24) + 4 * keys * ref.U32) * mag + h * np.abs(want) + 1e-37
    err = np.abs(g - want)
    assert np.isfinite(g).all() and (err <= tol).all(), float((err / tol).max())


def _filled(kda, lens, Hkv, d, page, dtype, seed):
    """Caches that hold lens tokens of each sequence, written by the library, in pools of random bytes."""
    table, n_pages = _table(lens, page, seed, bad=10 ** 6)
    kc, vc = _pool(n_pages, Hkv, d, page, seed + 1), _pool(n_pages, Hkv, d, page, seed + 2)
    cu = np.cumsum([0] + lens)
    k, v = _draw(seed + 3, dtype, int(cu[-1]), Hkv, d), _draw(seed + 4, dtype, int(cu[-1]), Hkv, d)
    kda.cache_write(k.cuda(), v.cuda(), kc, vc, _i32(table), _i32(cu))
    return table, kc, vc


# lens, m, H, Hkv, d, page, dtype
STEPS = [
    ([1], 1, 1, 1, 64, 16, "bf16"),
    ([0, 5, 16, 17, 33], 1, 4, 2, 128, 16, "bf16"),
    ([130, 128, 127, 1], 1, 7, 1, 128, 32, "f32"),
    ([700, 3, 0, 1000], 1, 20, 1, 64, 64, "bf16"),               # more heads of a group than a matrix tile's rows
    ([2, 50, 300, 129], 4, 14, 2, 128, 64, "bf16"),              # drafted tokens, more of them than the first has
    ([1, 0, 200], 3, 6, 6, 64, 16, "f32"),
    ([5000, 64], 2, 8, 2, 128, 128, "bf16"),
    ([30 + 3 * i for i in range(70)], 1, 2, 1, 64, 16, "bf16"),  # more sequences than lanes of a wave
    ([40, 90], 9, 8, 2, 64, 32, "f32"),                          # 36 rows: three matrix tiles
    ([900 + 7 * i for i in range(40)], 1, 16, 8, 64, 32, "bf16"),   # a few slots each, joined by one wave a row
    ([500 + 11 * i for i in range(30)], 2, 12, 6, 128, 16, "f32"),
]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join([str(len(c[0])), str(max(c[0]))] + [str(x) for x in c[1:]]))
def test_attn_step_matches_definition(case):
    kda = _kda()
    lens, m, H, Hkv, d, page, dtype = case
    print("attn_step", case, flush=True)
    N = len(lens)
    table, kc, vc = _filled(kda, lens, Hkv, d, page, dtype, 1)
    rows = _draw(9, dtype, N, m, H + 3, d)
    q = rows[:, :, 1:1 + H]
    qd = rows.cuda()[:, :, 1:1 + H]
    want, mag, a = np.zeros((N, m, H, d)), np.zeros((N, m, H, d)), np.zeros((N, m, H))
    for b in range(N):
        kk, vv = (lref.rows_of(c, table[b], lens[b], page, d) for c in (kc, vc))
        want[b], mag[b], a[b] = lref.attend(ref.f64(q[b]), kk, vv, d ** -0.5, [lens[b] - m + 1 + t for t in range(m)])
    need = kda.attn_step_workspace_bytes(N, m, H, Hkv, d, table.shape[1], page, DT[dtype])
    ws = torch.full((max(1, need // 4),), float("nan"), device="cuda")
    o = torch.full((N, m, H, d), 9.0, dtype=DT[dtype], device="cuda")
    kda.attn_step(qd, kc, vc, _i32(table), _i32(lens), o=o, workspace=ws)
    torch.cuda.synchronize()
    _inside(o, want, mag, a, d, max(lens), dtype)
    assert (ref.f64(o)[mag == 0] == 0).all()
    if m == 1:
        o3 = kda.attn_step(qd[:, 0], kc, vc, _i32(table), _i32(lens))
        torch.cuda.synchronize()
        assert o3.shape == (N, H, d) and torch.equal(o3, o[:, 0])


def test_attn_step_lengths_and_pages_outside():
    """Lengths past the table count as what it holds, negative ones as none; tokens on an entry outside the pool are
    not seen, wherever they lie."""
    kda = _kda()
    Hkv, H, d, page, n = 2, 4, 64, 16, 64
    lens = [n, n, n, n]
    table, kc, vc = _filled(kda, lens, Hkv, d, page, "bf16", 1)
    q = _draw(9, "bf16", 4, H, d)
    table = table[:, :4]
    cut = table.copy()
    cut[1, 0], cut[2, 2], cut[3] = 10 ** 9, -7, -1
    said = [2 ** 31 - 1, 50, 64, 64]
    o = kda.attn_step(q.cuda(), kc, vc, _i32(cut), _i32(said))
    none = kda.attn_step(q.cuda(), kc, vc, _i32(table), _i32([-1, -2 ** 31, 0, 0]))
    torch.cuda.synchronize()
    for b, seen in enumerate([range(64), range(16, 50), [*range(32), *range(48, 64)], []]):
        kk, vv = (lref.rows_of(c, table[b], n, page, d)[list(seen)] for c in (kc, vc))
        want, mag, a = lref.attend(ref.f64(q[b:b + 1]), kk, vv, d ** -0.5, [len(kk)])
        _inside(o[b:b + 1], want, mag, a, d, n, "bf16")
    assert bool((o[3] == 0).all()) and bool((none == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_step_maxima_that_rise_late(dtype):
    """Keys whose scores grow along the sequence, by far more than the exponentials' range."""
    kda = _kda()
    n, H, d, page = 600, 3, 64, 16
    table, n_pages = _table([n], page, 1)
    kc, vc = _pool(n_pages, 1, d, page, 1), _pool(n_pages, 1, d, page, 2)
    k = torch.linspace(-40, 40, n)[:, None, None].expand(n, 1, d).contiguous()
    v = _draw(3, "f32", n, 1, d)
    kda.cache_write(k.cuda(), v.cuda(), kc, vc, _i32(table), _i32([0, n]))
    q = torch.ones(1, H, d, dtype=DT[dtype])
    kk, vv = (lref.rows_of(c, table[0], n, page, d) for c in (kc, vc))
    want, mag, a = lref.attend(ref.f64(q[0])[None], kk, vv, 0.1, [n])
    o = kda.attn_step(q.cuda(), kc, vc, _i32(table), _i32([n]), scale=0.1)
    torch.cuda.synchronize()
    _inside(o, want, mag, a, d, n, dtype)


def test_a_prompt_in_pieces_and_its_tokens():
    """Pieces of three prompts through write, read back and attention, then tokens: each against the definition over the
    values that the cache stands for (a piece's own keys among them, as the next piece reads them)."""
    kda = _kda()
    H, Hkv, d, page, N = 6, 2, 128, 16, 3
    pieces, tokens = [[40, 1, 17], [0, 30, 100], [25, 2, 60]], 3
    most = [sum(p[b] for p in pieces) + tokens for b in range(N)]
    table, n_pages = _table(most, page, 1)
    kc, vc = _pool(n_pages, Hkv, d, page, 2), _pool(n_pages, Hkv, d, page, 3)
    pages, have = _i32(table), [0] * N
    for i, new in enumerate(pieces):
        cu = np.cumsum([0] + new)
        rows = _draw(10 + i, "bf16", int(cu[-1]), H + 2 * Hkv, d)
        r = rows.cuda()
        start = _i32(have)
        have = [a + b for a, b in zip(have, new)]
        cu_k = np.cumsum([0] + have)
        kda.cache_write(r[:, H:H + Hkv], r[:, H + Hkv:], kc, vc, pages, _i32(cu), start)
        k, v = kda.cache_read(kc, vc, pages, _i32(cu_k), int(cu_k[-1]), d)
        o = kda.attn_prefill(r[:, :H], k, v, _i32(cu), _i32(cu_k))
        torch.cuda.synchronize()
        want, mag, a = lref.attn_prefill(rows[:, :H], k, v, cu.tolist(), cu_k.tolist(), d ** -0.5)
        h = ref.half_step(torch.bfloat16)
        e = ref.U32 * ((2 * d + 32) * a[..., None] + 40)
        tol = (2 * e + h * (1 + h) + 4 * max(have) * ref.U32) * mag + h * np.abs(want) + 1e-37
        assert (np.abs(ref.f64(o) - want) <= tol).all()
        for b in range(N):
            assert np.array_equal(ref.f64(k[cu_k[b]:cu_k[b + 1]]), lref.rows_of(kc, table[b], have[b], page, d))
    for t in range(tokens):
        rows = _draw(20 + t, "bf16", N, H + 2 * Hkv, d)
        r = rows.cuda()
        kda.cache_write(r[:, H:H + Hkv], r[:, H + Hkv:], kc, vc, pages, None, _i32(have))
        have = [n + 1 for n in have]
        o = kda.attn_step(r[:, :H], kc, vc, pages, _i32(have))
        torch.cuda.synchronize()
        for b in range(N):
            kk, vv = (lref.rows_of(c, table[b], have[b], page, d) for c in (kc, vc))
            want, mag, a = lref.attend(ref.f64(rows[b:b + 1, :H]), kk, vv, d ** -0.5, [have[b]])
            _inside(o[b:b + 1], want, mag, a, d, have[b], "bf16")


def test_pool_past_32_bits():
    """Pages that begin past 2^32 bytes of the pool."""
    kda = _kda()
    Hkv, d, page = 8, 128, 128
    size = kda.cache_page_bytes(d, page)
    n_pages = (1 << 32) // (Hkv * size) + 3
    kc, vc = (torch.zeros(n_pages, Hkv, size, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = _i32([[n_pages - 1, 0], [1, n_pages - 2]])
    near = _i32([[2, 0], [1, 3]])
    k, v, q = _draw(1, "bf16", 400, Hkv, d).cuda(), _draw(2, "bf16", 400, Hkv, d).cuda(), _draw(3, "bf16", 2, Hkv, d).cuda()
    cu, lens, got = _i32([0, 200, 400]), _i32([200, 200]), []
    for t in (table, near):
        kda.cache_write(k, v, kc, vc, t, cu)
        got.append((*kda.cache_read(kc, vc, t, cu, 400, d), kda.attn_step(q, kc, vc, t, lens)))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
