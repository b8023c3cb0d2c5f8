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
