"""How exact the gated delta rule's bf16 outputs are, for tests on the device and for a model of them on the CPU.

A block's outputs are o_i = 2^(c_i) S0^T q_i + sum_j w_ij u_j with w_ij = 2^(c_i - c_j) (q_i . k_j).  S0, w and u enter
as two bf16 parts each: a part leaves 2^-8 of what it rounds, two leave 2^-16, and the product of the second parts of w
and u, left out, is 2^-8 2^-8 of the term.  Exponents are differences of two fp32 sums of at most 128 where a weight is not
below 2^-128, so off by 128 2^-24, which is 2^-17 ln 2 of the weight; the exponential itself is good to 2^-22.  Together at
most (3 2^-16 (1 + 2^-8) + 2^-17) of terms = 2^(c_i) |S0|^T |q_i| + sum_j |w_ij| |u_j|, where a factor rounded once
would leave 2^-8 of them.
"""
import numpy as np
import torch

SHARE = 3 * 2.0 ** -16 * (1 + 2.0 ** -8) + 2.0 ** -17


def parts(x, n):
    """x (float64) in n bf16 parts, the first one largest."""
    out = []
    for _ in range(n):
        p = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
        out.append(p)
        x = x - p
    return out


def block(q, k, v, g, beta, S0):
    """One head's block in 64 bits: c [C], weights [C, C], u [C, dv], entry state decayed to each token [C, dk, dv]."""
    C = len(g)
    c = np.cumsum(g)
    S, u = S0.copy(), np.zeros(v.shape)
    for t in range(C):
        S = np.exp(g[t]) * S
        u[t] = beta[t] * (v[t] - S.T @ k[t])
        S = S + np.outer(k[t], u[t])
    w = np.tril(np.exp(np.minimum(c[:, None] - c[None], 0)) * (q @ k.T))
    return c, w, u


def outputs(q, k, v, g, beta, S0, n_state=2, n_weights=2, n_u=2):
    """The block's outputs from factors of so many parts, the exact ones, and the terms' absolute values."""
    c, w, u = block(q, k, v, g, beta, S0)
    grow = np.exp(c)[:, None]
    want = grow * (q @ S0) + w @ u
    terms = grow * (np.abs(q) @ np.abs(S0)) + np.abs(w) @ np.abs(u)
    got = grow * sum(q @ p for p in parts(S0, n_state))
    for i, a in enumerate(parts(w, n_weights)):
        for j, b in enumerate(parts(u, n_u)):
            if i + j < 2:
                got = got + a @ b
    return got, want, terms
