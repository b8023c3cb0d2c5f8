"""Token mixers beside KDA: short causal convolution (further operators of this kind follow the
same rules).

Argument marshalling only, like the rest of the binding.  Inputs may be slices of a projection's
rows: tokens of one tensor lie a fixed stride apart and the elements of a token are contiguous.
Outputs and states are contiguous.
"""
from __future__ import annotations

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.KDA_BF16, torch.float32: _lib.KDA_F32}


def _code(dt):
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"inputs must be bfloat16 or float32, got {dt}")
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(name, t, dtype, shape, device):
    """A contiguous tensor of exactly this type, shape and device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(name, t, dtype, shape, device, lead):
    """Checks a tensor whose first `lead` axes are rows and whose other axes are contiguous inside a
    row; returns the stride between rows in elements."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    width = 1
    for size, stride in zip(reversed(shape[lead:]), reversed(t.stride()[lead:])):
        if size > 1 and stride != width:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        width *= size
    if lead == 1:
        return t.stride(0) if shape[0] > 1 else width
    step = t.stride(1) if shape[1] > 1 else (t.stride(0) if shape[0] > 1 else width)
    if shape[0] > 1 and shape[1] > 0 and t.stride(0) != step * shape[1]:
        raise ValueError(f"{name}: sequence b must start at row b * T of evenly spaced rows")
    return step


def _device(t, where):
    if t.device.type != "cuda":
        raise ValueError(f"{where} runs on a HIP device; got a tensor on {t.device}")
    return t.device


def _call(fn, dev, *args):
    """The library call on the current stream of the tensors' device, with that device current."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if dev.index == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        _lib.check(st, fn.__name__)


def conv_prefill(x, w, bias=None, state=None, *, lens=None, silu=True, y=None, state_out=None,
                 return_state=True):
    """Short causal depthwise convolution of a prompt batch.  Returns (y, state_out).

    x [B, T, D] (rows may be strided), w [D, W] with W 2, 3 or 4, bias [D]; ``state`` [B, W-1, D] are
    the inputs before the first token (None = zeros), ``state_out`` the last W-1 inputs of each
    sequence (may be ``state`` itself; None when return_state is False).  ``lens`` (int32 [B]) gives
    the tokens of each sequence of a padded batch; rows of y behind them are left as they were.
    """
    dev = _device(x, "conv_prefill")
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [B, T, D] and w [D, W]")
    B, T, D = x.shape
    W = w.shape[1]
    dt = x.dtype
    code = _code(dt)
    x_stride = _rows("x", x, dt, x.shape, dev, 2)
    _check("w", w, dt, (D, W), dev)
    if bias is not None:
        _check("bias", bias, dt, (D,), dev)
    keep = (B, W - 1, D)
    if state is not None:
        _check("state", state, dt, keep, dev)
    if lens is not None:
        _check("lens", lens, torch.int32, (B,), dev)
    if y is None:
        y = torch.empty((B, T, D), dtype=dt, device=dev)
    else:
        _check("y", y, dt, (B, T, D), dev)
    if state_out is not None:
        _check("state_out", state_out, dt, keep, dev)
    elif return_state:
        state_out = torch.empty(keep, dtype=dt, device=dev)
    _call(_lib.load().kda_conv_prefill, dev, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lens), _ptr(y),
          _ptr(state_out), B, T, D, W, x_stride, int(bool(silu)), code)
    return y, state_out


def conv_step(x, w, state, bias=None, *, silu=True, y=None):
    """The convolution for one new token of N sequences: x [N, D] (rows may be strided), ``state``
    [N, W-1, D] shifted in place.  Returns y [N, D]."""
    dev = _device(x, "conv_step")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [N, D] and w [D, W]")
    N, D = x.shape
    W = w.shape[1]
    dt = x.dtype
    code = _code(dt)
    x_stride = _rows("x", x, dt, x.shape, dev, 1)
    _check("w", w, dt, (D, W), dev)
    if bias is not None:
        _check("bias", bias, dt, (D,), dev)
    _check("state", state, dt, (N, W - 1, D), dev)
    if y is None:
        y = torch.empty((N, D), dtype=dt, device=dev)
    else:
        _check("y", y, dt, (N, D), dev)
    _call(_lib.load().kda_conv_step, dev, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(y), N, D, W, x_stride,
          int(bool(silu)), code)
    return y
