"""What stands beside KDA in a hybrid model: short causal convolution, selective state space scan, attention with a
sliding window and a few first tokens that stay visible, causal attention over packed prompts, a paged cache of 4 bits
an element with the attention over it, and the gated delta rule with one decay per head.

Signatures and their documentation; checks and marshalling are in csrc/binding (``_mixers.so``), since a
token of these operators keeps the device busy for a few microseconds only.  Inputs may be slices of a
projection's rows: tokens of one tensor lie a fixed stride apart and the elements of a token are
contiguous.  Outputs and states are contiguous.  Calls run on the current stream of the tensors' device.
Like KDA's own calls they form no gradients: results are detached, also where an input requires one.
Tensors without memory of their own (inside torch.vmap, torch.func or a fake tensor mode) are refused.
"""
from __future__ import annotations

import ctypes
import os

from . import _lib

_INT_MAX = 2 ** 31 - 1
# the library's entry points in the order in which the binding takes them
_ENTRIES = ("kda_conv_prefill", "kda_conv_step", "kda_ssm_prefill_workspace_bytes", "kda_ssm_prefill", "kda_ssm_step",
            "kda_window_prefill_workspace_bytes", "kda_window_prefill", "kda_window_step_workspace_bytes", "kda_window_step",
            "kda_attn_prefill_workspace_bytes", "kda_attn_prefill", "kda_cache_write", "kda_cache_read",
            "kda_attn_step_workspace_bytes", "kda_attn_step",
            "kda_delta_prefill_workspace_bytes", "kda_delta_prefill", "kda_delta_step")
_native = None


def _load():
    """The binding, bound to the loaded library (once).  Like the library it has to be built."""
    global _native
    if _native is None:
        lib = _lib.load()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mixers.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(python chunked_gated_delta_13_amd/build.py)")
        from . import _mixers
        _mixers.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _ENTRIES), _lib.check)
        _native = _mixers
    return _native


def _code(dt):
    import torch
    if dt is None or dt == torch.bfloat16:
        return _lib.KDA_BF16
    if dt == torch.float32:
        return _lib.KDA_F32
    raise TypeError(f"inputs must be bfloat16 or float32, got {dt}")


def _fits(*sizes):
    """Sizes are 32-bit numbers at the library's entry points."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX:
        raise ValueError(f"sizes must fit 32 bits, got {max(sizes, key=abs)}")


def conv_prefill(x, w, bias=None, state=None, *, lens=None, silu=True, y=None, state_out=None,
                 return_state=True):
    """Short causal depthwise convolution of a prompt batch.  Returns (y, state_out).

    x [B, T, D] (rows may be strided), w [D, W] with W 2, 3 or 4, bias [D]; ``state`` [B, W-1, D] are
    the inputs before the first token (None = zeros), ``state_out`` the last W-1 inputs of each
    sequence (may be ``state`` itself; None when return_state is False).  ``lens`` (int32 [B]) gives
    the tokens of each sequence of a padded batch; rows of y behind them are left as they were.  Widths
    of whole 16-byte groups of channels run about half again as fast as others.
    """
    return (_native or _load()).conv_prefill(x, w, bias, state, lens, silu, y, state_out, return_state)


def conv_step(x, w, state, bias=None, *, silu=True, y=None):
    """The convolution for one new token of N sequences: x [N, D] (rows may be strided), ``state``
    [N, W-1, D] shifted in place.  Returns y [N, D]."""
    return (_native or _load()).conv_step(x, w, state, bias, silu, y)


def ssm_workspace_bytes(B, T, H, G, n, p, dtype=None, seg_len=0):
    """Device workspace bytes of ssm_prefill for this shape on the current device (dtype None = bfloat16)."""
    _fits(B, T, H, G, n, p, seg_len)
    return int(_lib.load().kda_ssm_prefill_workspace_bytes(B, T, H, G, n, p, _code(dtype), seg_len))


def ssm_prefill(x, dt, A, Bm, Cm, S0=None, *, D=None, z=None, dt_bias=None, lens=None, seg_len=0, y=None,
                S_T=None, return_state=True, workspace=None):
    """Selective state space scan of a prompt batch.  Returns (y, S_T).

    x, z [B, T, H, p]; dt [B, T, H] raw steps (softplus(dt + dt_bias) is applied); A, D, dt_bias [H]
    fp32; Bm, Cm [B, T, G, n]; S0, S_T [B, H, n, p] fp32 (S_T may be S0; None when return_state is False).
    x, dt, Bm, Cm and z may be slices of a projection's rows.  ``lens`` (int32 [B]) gives the tokens of
    each sequence of a padded batch; rows of y behind them are left as they were.  ``seg_len`` forces the
    tokens per segment of the sequence split (0 = the library's choice).
    """
    return (_native or _load()).ssm_prefill(x, dt, A, Bm, Cm, S0, D, z, dt_bias, lens, seg_len, y, S_T, return_state,
                                            workspace)


def ssm_step(x, dt, A, Bm, Cm, S, *, D=None, z=None, dt_bias=None, y=None):
    """One token of the scan for N sequences: x, z [N, H, p], dt [N, H], Bm, Cm [N, G, n]; ``S``
    [N, H, n, p] is updated in place.  Returns y [N, H, p]."""
    return (_native or _load()).ssm_step(x, dt, A, Bm, Cm, S, D, z, dt_bias, y)


def window_prefill_workspace_bytes(B, T, H, Hkv, d, window, sinks=0, dtype=None, continued=False):
    """Device workspace bytes of window_prefill for this shape on the current device (dtype None = bfloat16);
    ``continued`` where the call is given ``start``."""
    _fits(B, T, H, Hkv, d, window, sinks)
    return int(_lib.load().kda_window_prefill_workspace_bytes(B, T, H, Hkv, d, window, sinks, _code(dtype), int(continued)))


def window_prefill(q, k, v, window, sinks=0, *, scale=None, k_cache=None, v_cache=None, start=None, lens=None,
                   o=None, workspace=None):
    """Attention of a prompt batch with a sliding window and ``sinks`` first tokens that stay visible: the
    query at position t sees key j <= t where t - j < window or j < sinks.  Returns o [B, T, H, d].

    q [B, T, H, d]; k, v [B, T, Hkv, d] with Hkv dividing H (all may be slices of a projection's rows).
    ``k_cache`` / ``v_cache`` [B, sinks + window, Hkv, d] are the sequences' ring caches: earlier tokens
    (``start`` [B] int32 of them, None = 0) are read from them and the new ones that stay visible are
    written to them.  ``lens`` (int32 [B]) gives the new tokens of each sequence of a padded batch; rows
    of o behind them are left as they were.  ``scale`` defaults to d ** -0.5.  Few queries over a long
    window are run as ranges of keys, in ``workspace`` if it is large enough, else in a new one.
    """
    return (_native or _load()).window_prefill(q, k, v, window, sinks, scale, k_cache, v_cache, start, lens, o,
                                               workspace)


def window_step_workspace_bytes(N, H, Hkv, d, window, sinks=0, dtype=None):
    """Device workspace bytes of window_step for this shape on the current device (dtype None = bfloat16)."""
    _fits(N, H, Hkv, d, window, sinks)
    return int(_lib.load().kda_window_step_workspace_bytes(N, H, Hkv, d, window, sinks, _code(dtype)))


def window_step(q, k, v, k_cache, v_cache, pos, window, sinks=0, *, scale=None, o=None, workspace=None):
    """The same attention for one new token of N sequences over their ring caches, which receive the
    token's k and v: q [N, H, d], k, v [N, Hkv, d], ``pos`` (int32 [N]) the tokens before it (negative values
    count as 0).  Returns o."""
    return (_native or _load()).window_step(q, k, v, k_cache, v_cache, pos, window, sinks, scale, o, workspace)


def attn_prefill_workspace_bytes(B, Nq, Nk, H, Hkv, d, dtype=None):
    """Device workspace bytes of attn_prefill for B sequences of Nq queries and Nk keys together on the current
    device (dtype None = bfloat16)."""
    _fits(B, Nq, Nk, H, Hkv, d)
    return int(_lib.load().kda_attn_prefill_workspace_bytes(B, Nq, Nk, H, Hkv, d, _code(dtype)))


def attn_prefill(q, k, v, cu_q, cu_k=None, *, scale=None, o=None, workspace=None):
    """Causal attention over packed prompts of different lengths.  Returns o [Nq, H, d].

    q [Nq, H, d]; k, v [Nk, Hkv, d] with Hkv dividing H (all may be slices of a projection's rows): the tokens
    of sequence b are the rows from ``cu_q[b]`` up to ``cu_q[b + 1]`` (int32 [B + 1], on the device, not
    decreasing), its keys those from ``cu_k[b]`` on (None = ``cu_q``).  Its queries are its last tokens: with nq
    queries and nk keys, query i sees the keys j <= i + nk - nq, and one that sees none gets zeros.  A prompt run
    in pieces has its earlier keys in front, as cache_read returns them.  Rows of o outside the sequences are left as
    they were.  ``scale`` defaults to d ** -0.5.  Few queries over many keys are run as ranges of keys, in
    ``workspace`` if it is large enough, else in a new one.
    """
    return (_native or _load()).attn_prefill(q, k, v, cu_q, cu_k, scale, o, workspace)


def cache_page_bytes(d, page):
    """Bytes of one page of ``page`` tokens of one kv head with d channels in the 4-bit cache: 4.25 bits an element.
    k_cache and v_cache are uint8 tensors [n_pages, Hkv, cache_page_bytes(d, page)]."""
    return page * (d // 2 + d // 32)


def cache_write(k, v, k_cache, v_cache, pages, cu=None, start=None):
    """Keys and values of packed tokens into a paged cache of 4 bits an element, in place.

    k, v [N, Hkv, d] (may be slices of a projection's rows); ``k_cache`` / ``v_cache`` uint8 [n_pages, Hkv,
    cache_page_bytes(d, page)], ``page`` a power of two from 16 on; ``pages`` int32 [B, max_pages]: the page of each
    ``page`` positions of a sequence.  Sequence b's tokens are the rows from ``cu[b]`` up to ``cu[b + 1]`` (int32
    [B + 1]; None: one token each, N = B), the first one at position ``start[b]`` (int32 [B], None = 0; negative values
    count as 0).  32 channels share a power of two, an element is one of 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign.
    Tokens past the table, or on an entry outside the pool, are not written.  No two tokens of a call may share a
    place.
    """
    return (_native or _load()).cache_write(k, v, k_cache, v_cache, pages, cu, start)


def cache_read(k_cache, v_cache, pages, cu, tokens, d, start=None, *, dtype=None, k=None, v=None):
    """Keys and values of the cache as packed rows, for the attention of a prompt's next piece.  Returns (k, v)
    [tokens, Hkv, d] in ``dtype`` (None = bfloat16, which holds every value).

    Row i of sequence b (the rows from ``cu[b]`` up to ``cu[b + 1]``; cu None: one token each) is position
    ``start[b]`` + i - cu[b] (start None = 0).  Positions without a page are zeros; rows outside the sequences are left as
    they were.
    """
    return (_native or _load()).cache_read(k_cache, v_cache, pages, cu, tokens, d, start, dtype, k, v)


def attn_step_workspace_bytes(N, m, H, Hkv, d, max_pages, page, dtype=None):
    """Device workspace bytes of attn_step for this shape on the current device (dtype None = bfloat16)."""
    _fits(N, m, H, Hkv, d, max_pages, page)
    return int(_lib.load().kda_attn_step_workspace_bytes(N, m, H, Hkv, d, max_pages, page, _code(dtype)))


def attn_step(q, k_cache, v_cache, pages, lens, *, scale=None, o=None, workspace=None):
    """Attention of the newest token of N sequences over the 4-bit cache, or of their m newest ones (drafted
    tokens to be verified).  Returns o, shaped like q.

    q [N, H, d] or [N, m, H, d] (may be slices of a projection's rows); caches and ``pages`` as for cache_write,
    which has written the new tokens too; ``lens`` int32 [N]: the tokens of each sequence in the cache, at most
    what its table holds.  Query t sees the first lens - m + 1 + t of them; one that sees none gets zeros, and tokens on
    a table's entry outside the pool are not seen.  ``scale`` defaults to d ** -0.5.
    """
    return (_native or _load()).attn_step(q, k_cache, v_cache, pages, lens, scale, o, workspace)


def delta_workspace_bytes(B, T, H, Hk, dk, dv, dtype=None, seg_len=0):
    """Device workspace bytes of delta_prefill for this shape on the current device (dtype None = bfloat16)."""
    _fits(B, T, H, Hk, dk, dv, seg_len)
    return int(_lib.load().kda_delta_prefill_workspace_bytes(B, T, H, Hk, dk, dv, _code(dtype), seg_len))


def delta_prefill(q, k, v, g, beta, S0=None, *, lens=None, seg_len=0, o=None, S_T=None, return_state=True, workspace=None):
    """The gated delta rule of a prompt batch, one decay per head and token.  Returns (o, S_T).

        S <- e^g S + beta k (v - e^g S^T k)^T,    o = S^T q

    q, k [B, T, Hk, dk]; v [B, T, H, dv] (all may be slices of a projection's rows), key head h Hk // H serves value head h;
    g, beta [B, T, H] fp32, g the natural log of the decay (at most 0, not bounded below); S0, S_T [B, H, dk, dv] fp32
    (S_T may be S0; None when return_state is False).  As in chunk_prefill, q and k are taken as they are (callers
    normalise and scale them), and beta too.  ``lens`` (int32 [B]) gives the tokens of each sequence of a padded batch; rows of o behind
    them are left as they were.  ``seg_len`` forces the tokens per segment of the sequence split (a multiple of 64; 0 = the
    library's choice).  The result does not depend on it beyond rounding: a split takes as forgotten only what the transitions
    behind it, e^g max(1, |1 - beta |k|^2|) each, have shrunk to less than 2^-126.
    """
    return (_native or _load()).delta_prefill(q, k, v, g, beta, S0, lens, seg_len, o, S_T, return_state, workspace)


def delta_step(q, k, v, g, beta, S, *, o=None):
    """One token of the gated delta rule for N sequences: q, k [N, Hk, dk], v [N, H, dv], g, beta [N, H] fp32; ``S``
    [N, H, dk, dv] is updated in place.  Returns o [N, H, dv]."""
    return (_native or _load()).delta_step(q, k, v, g, beta, S, o)
