"""Plain float64 definitions of the full-attention layer's parts and of the gated delta rule, on the CPU (tests only).

Each follows its formula and shares no code with the library.  Beside a result comes the sum of the absolute
values of the terms behind it, for tolerances that count roundings.
"""
import numpy as np

from tests.mixers_reference import f64

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def attend(q, k, v, scale, sees):
    """One sequence: q [n, H, d], k, v [m, Hkv, d], query i sees the first sees[i] keys.  (o, |terms|, largest
    scale * sum |q k|)."""
    n, H, d = q.shape
    R = H // k.shape[1]
    o, mag, a = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, H))
    for i in range(n):
        m = max(0, min(int(sees[i]), k.shape[0]))
        if m == 0:
            continue
        for h in range(H):
            kk, vv = k[:m, h // R], v[:m, h // R]
            w = scale * (kk @ q[i, h])
            a[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            p = np.exp(w - w.max())
            p /= p.sum()
            o[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
    return o, mag, a


def attn_prefill(q, k, v, cu_q, cu_k, scale):
    """(o, |terms|, a): rows outside the sequences are NaN."""
    q, k, v = f64(q), f64(k), f64(v)
    o, mag, a = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.zeros(q.shape[:2])
    for b in range(len(cu_q) - 1):
        s, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n, m = s.stop - s.start, t.stop - t.start
        o[s], mag[s], a[s] = attend(q[s], k[t], v[t], scale, [i + m - n + 1 for i in range(n)])
    return o, mag, a


def quantise(x):
    """x [..., d] (float64) as the values that the cache's 4-bit form stands for, by search, and the exponents."""
    x = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(x).max(-1, keepdims=True)
    e = np.full(top.shape, -125.0)
    for n in range(-125, 96):
        e = np.where((top > 7 * 2.0 ** e) & (n < 95), e + 1, e)
    gap = np.abs(np.abs(x)[..., None] / 2.0 ** e[..., None] - GRID) + 1e-12 * (np.arange(8) % 2)   # ties to even
    y = GRID[gap.argmin(-1)] * np.sign(x) * 2.0 ** e
    y = np.where(np.isfinite(top), y, np.nan)
    return y.reshape(*y.shape[:-2], -1), np.where(np.isfinite(top), e + 127, 255)[..., 0]


def rows_of(cache, table, n, page, d):
    """Values [n, Hkv, d] of a sequence's first n positions, from the bytes of one pool; NaN where a table entry
    lies outside the pool or the table ends."""
    pool = cache.cpu().numpy()
    out = np.full((n, pool.shape[1], d), np.nan)
    for i in range(n):
        at = i // page
        if at >= len(table) or not 0 <= table[at] < pool.shape[0]:
            continue
        p, r = pool[table[at]], i % page
        byte = p[:, r * (d // 2):(r + 1) * (d // 2)]
        code = np.stack([byte & 15, byte >> 4], -1).reshape(pool.shape[1], d)
        exps = p[:, page * (d // 2) + r * (d // 32):page * (d // 2) + (r + 1) * (d // 32)].astype(np.float64)
        scale = np.where(exps == 255, np.nan, 2.0 ** (exps - 127))
        out[i] = GRID[code & 7] * np.where(code & 8, -1, 1) * np.repeat(scale, 32, -1)
    return out


def delta(q, k, v, g, beta, S0=None, lens=None):
    """The gated delta rule: (o, |terms| of o, S_T, |terms| of S_T).  o rows behind a sequence's end are NaN."""
    q, k, v, g, beta, S0 = (f64(t) for t in (q, k, v, g, beta, S0))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    S = np.zeros((B, H, dk, dv)) if S0 is None else S0.copy()
    M = np.abs(S)
    o, mag = np.full(v.shape, np.nan), np.full(v.shape, np.nan)
    for b in range(B):
        for t in range(T if lens is None else lens[b]):
            kk, qq = (np.repeat(x[b, t], H // Hk, 0) for x in (k, q))
            P, N = (np.exp(g[b, t])[:, None, None] * x for x in (S[b], M[b]))
            u = beta[b, t][:, None] * (v[b, t] - np.einsum("hk,hkv->hv", kk, P))
            w = np.abs(beta[b, t])[:, None] * (np.abs(v[b, t]) + np.einsum("hk,hkv->hv", np.abs(kk), N))
            S[b] = P + kk[:, :, None] * u[:, None]
            M[b] = N + np.abs(kk)[:, :, None] * w[:, None]
            o[b, t] = np.einsum("hk,hkv->hv", qq, S[b])
            mag[b, t] = np.einsum("hk,hkv->hv", np.abs(qq), M[b])
    return o, mag, S, M
