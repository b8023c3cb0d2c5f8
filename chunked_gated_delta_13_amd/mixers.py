"""Token mixers beside KDA: short causal convolution, selective state space scan, and attention with a
sliding window and a few first tokens that stay visible.

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
            "kda_window_prefill_workspace_bytes", "kda_window_prefill", "kda_window_step_workspace_bytes", "kda_window_step")
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
