"""Plain float64 definitions of the token mixers beside KDA, on the CPU (tests only).

Each follows its formula token by token and shares no code with the library.  Beside a result comes
the sum of the absolute values of the terms behind it, for tolerances that count roundings.
"""
import numpy as np
import torch

U32 = 2.0 ** -24     # half a step of fp32, relative


def half_step(dtype):
    """A rounding to `dtype` is off by at most this much, relative to the value."""
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def silu(x):
    return x * sigmoid(x)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def lens_of(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens.tolist()]


def conv(x, w, bias, state, lens, act):
    """(y, |terms|, state_out, lens): y rows behind a sequence's end are NaN."""
    x, w, bias, state = f64(x), f64(w), f64(bias), f64(state)
    B, T, D = x.shape
    W = w.shape[1]
    ls = lens_of(lens, B, T)
    y, mag = np.full((B, T, D), np.nan), np.full((B, T, D), np.nan)
    kept = np.zeros((B, W - 1, D))
    for b in range(B):
        line = np.concatenate([np.zeros((W - 1, D)) if state is None else state[b], x[b, :ls[b]]])
        for t in range(ls[b]):
            terms = [line[t + j] * w[:, j] for j in range(W)] + ([bias] if bias is not None else [])
            v = sum(terms)
            y[b, t], mag[b, t] = (silu(v) if act else v), sum(abs(u) for u in terms)
        kept[b] = line[ls[b]:]
    return y, mag, kept, ls


def ssm(x, dt, A, Bm, Cm, S0=None, D=None, z=None, dt_bias=None, lens=None):
    """(y, |terms| of y, S_T, |terms| of S_T, largest exponent of a 64-token chunk).  y rows behind a
    sequence's end are NaN."""
    x, dt, A, Bm, Cm, S0, D, z, dt_bias = (f64(t) for t in (x, dt, A, Bm, Cm, S0, D, z, dt_bias))
    B, T, H, p = x.shape
    G, n = Bm.shape[2:]
    ls = lens_of(lens, B, T)
    S = np.zeros((B, H, n, p)) if S0 is None else S0.copy()
    M = np.abs(S)
    y, mag = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    cmax = 0.0
    for b in range(B):
        c = 0.0
        for t in range(ls[b]):
            d = softplus(dt[b, t] + (0 if dt_bias is None else dt_bias))
            c = np.abs(d * A) + (0.0 if t % 64 == 0 else c)
            cmax = max(cmax, float(c.max()))
            k = np.repeat(Bm[b, t], H // G, 0)[:, :, None]
            q = np.repeat(Cm[b, t], H // G, 0)[:, :, None]
            e = np.exp(d * A)[:, None, None]
            u = d[:, None, None] * k * x[b, t][:, None, :]
            S[b] = e * S[b] + u
            M[b] = e * M[b] + np.abs(u)
            skip = 0 if D is None else D[:, None] * x[b, t]
            gate = 1 if z is None else silu(z[b, t])
            y[b, t] = ((S[b] * q).sum(1) + skip) * gate
            mag[b, t] = ((M[b] * np.abs(q)).sum(1) + np.abs(skip)) * np.abs(gate)
    return y, mag, S, M, cmax


def ring_row(p, sinks, window):
    return p if p < sinks else sinks + (p - sinks) % window


def window(q, k, v, win, sinks, scale, k_cache=None, v_cache=None, start=None, lens=None):
    """(o, |terms|, largest scale * sum |q k| per query, k_cache, v_cache): o rows behind a sequence's end
    are NaN; the caches are copies with the new tokens written."""
    q, k, v, kc, vc = (f64(t) for t in (q, k, v, k_cache, v_cache))
    B, T, H, d = q.shape
    Hkv = k.shape[2]
    ls = lens_of(lens, B, T)
    st = [0] * B if start is None else [int(n) for n in start.tolist()]
    o, mag, a = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.zeros((B, T, H))
    kc2, vc2 = (None if c is None else c.copy() for c in (kc, vc))
    for b in range(B):
        s = st[b]
        for i in range(ls[b]):
            t = s + i
            see = sorted(set(range(min(sinks, t + 1))) | set(range(max(0, t - win + 1), t + 1)))
            at = [(None, j - s) if j >= s else (ring_row(j, sinks, win), None) for j in see]
            kk = np.stack([k[b, n] if n is not None else kc[b, c] for c, n in at])     # [keys, Hkv, d]
            vv = np.stack([v[b, n] if n is not None else vc[b, c] for c, n in at])
            for h in range(H):
                g = h // (H // Hkv)
                w = scale * (kk[:, g] @ q[b, i, h])
                a[b, i, h] = scale * (np.abs(kk[:, g]) @ np.abs(q[b, i, h])).max()
                p = np.exp(w - w.max())
                p /= p.sum()
                o[b, i, h] = p @ vv[:, g]
                mag[b, i, h] = p @ np.abs(vv[:, g])
        if kc is not None:
            for i in range(ls[b]):
                row = ring_row(s + i, sinks, win)
                kc2[b, row], vc2[b, row] = k[b, i], v[b, i]
    return o, mag, a, kc2, vc2
