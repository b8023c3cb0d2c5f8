"""Token mixers beside KDA: short causal convolution, selective state space scan, and attention with a
sliding window and a few first tokens that stay visible.

Argument marshalling only, like the rest of the binding.  Inputs may be slices of a projection's
rows: tokens of one tensor lie a fixed stride apart and the elements of a token are contiguous.
Outputs and states are contiguous.
"""
from __future__ import annotations

import functools

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


def _refuse(name, t, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _check(name, t, dtype, shape, device):
    """A contiguous tensor of exactly this type, shape and device."""
    if not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _refuse(name, t, dtype, shape, device)


def _rows(name, t, dtype, shape, device, lead):
    """Checks a tensor whose first `lead` axes are rows and whose other axes (one or two) are contiguous
    inside a row; returns the stride between rows in elements."""
    if not (t.dtype is dtype and t.shape == shape and t.device == device):
        _refuse(name, t, dtype, shape, device)
    stride = t.stride()
    width = shape[-1]
    inner = stride[-1] == 1 or width <= 1
    if len(stride) - lead == 2:
        inner = inner and (stride[-2] == width or shape[-2] <= 1)
        width *= shape[-2]
    if not inner and width > 0:
        raise ValueError(f"{name}: the elements of a token must be contiguous")
    if lead == 1:
        return stride[0] if shape[0] > 1 else width
    B, T = shape[0], shape[1]
    step = stride[1] if T > 1 else (stride[0] if B > 1 else width)
    if B > 1 and T > 0 and stride[0] != step * T:
        raise ValueError(f"{name}: sequence b must start at row b * T of evenly spaced rows")
    return step


_INT_MAX = 2 ** 31 - 1


def _fits(*sizes):
    """Sizes are 32-bit numbers at the library's entry points."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX:
        raise ValueError(f"sizes must fit 32 bits, got {max(sizes, key=abs)}")


def _workspace(workspace, need, dev):
    """The caller's workspace if it is large enough, else a new one; returns it and its bytes."""
    if workspace is None:
        return (None, 0) if need == 0 else (torch.empty(need, dtype=torch.uint8, device=dev), need)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    size = workspace.numel() * workspace.element_size()
    return (torch.empty(need, dtype=torch.uint8, device=dev), need) if size < need else (workspace, size)


def _hip(t, where):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{where} runs on a HIP device; got a tensor on {dev}")
    return dev


# the current stream of a device as a number, without a stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, dev, *args):
    """The library call on the current stream of the tensors' device, with that device current."""
    index = dev.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
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
    dev = _hip(x, "conv_prefill")
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
    _fits(B, T, D, W)
    keep = (B, W - 1, D)
    if state is not None:
        _check("state", state, dt, keep, dev)
    if lens is not None:
        _check("lens", lens, torch.int32, (B,), dev)
    if y is None:
        y = x.new_empty((B, T, D))
    else:
        _check("y", y, dt, (B, T, D), dev)
    if state_out is not None:
        _check("state_out", state_out, dt, keep, dev)
    elif return_state:
        state_out = x.new_empty(keep)
    _call(_lib.load().kda_conv_prefill, dev, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lens), _ptr(y),
          _ptr(state_out), B, T, D, W, x_stride, int(bool(silu)), code)
    return y, state_out


def conv_step(x, w, state, bias=None, *, silu=True, y=None):
    """The convolution for one new token of N sequences: x [N, D] (rows may be strided), ``state``
    [N, W-1, D] shifted in place.  Returns y [N, D]."""
    dev = _hip(x, "conv_step")
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
    _fits(N, D, W)
    _check("state", state, dt, (N, W - 1, D), dev)
    if y is None:
        y = x.new_empty((N, D))
    else:
        _check("y", y, dt, (N, D), dev)
    _call(_lib.load().kda_conv_step, dev, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(y), N, D, W, x_stride,
          int(bool(silu)), code)
    return y


def _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, lead):
    """Checks of the scan's inputs; returns the sizes and the row strides (x, dt, B, C, z)."""
    dev, ty = x.device, x.dtype
    rows = x.shape[:lead]
    H, p = x.shape[lead:]
    if Bm.dim() != lead + 2:
        raise ValueError("Bm must have one axis of groups and one of state channels after the tokens")
    G, n = Bm.shape[lead:]
    xs = _rows("x", x, ty, x.shape, dev, lead)
    ds = _rows("dt", dt, ty, (*rows, H), dev, lead)
    bs = _rows("Bm", Bm, ty, (*rows, G, n), dev, lead)
    cs = _rows("Cm", Cm, ty, (*rows, G, n), dev, lead)
    zs = 0
    if z is not None:
        zs = _rows("z", z, ty, x.shape, dev, lead)
    _check("A", A, torch.float32, (H,), dev)
    if D is not None:
        _check("D", D, torch.float32, (H,), dev)
    if dt_bias is not None:
        _check("dt_bias", dt_bias, torch.float32, (H,), dev)
    return (H, G, n, p), (xs, ds, bs, cs, zs)


@functools.lru_cache(maxsize=1024)
def _ssm_bytes(device, *shape):   # a plan depends on the shape and the device's compute units only
    with torch.cuda.device(device):
        return int(_lib.load().kda_ssm_prefill_workspace_bytes(*shape))


def ssm_workspace_bytes(B, T, H, G, n, p, dtype=torch.bfloat16, seg_len=0):
    """Device workspace bytes of ssm_prefill for this shape on the current device."""
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
    dev = _hip(x, "ssm_prefill")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, p]")
    B, T = x.shape[:2]
    ty = x.dtype
    code = _code(ty)
    (H, G, n, p), strides = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    _fits(B, T, H, G, n, p, seg_len)
    state = (B, H, n, p)
    if S0 is not None:
        _check("S0", S0, torch.float32, state, dev)
    if lens is not None:
        _check("lens", lens, torch.int32, (B,), dev)
    if y is None:
        y = x.new_empty((B, T, H, p))
    else:
        _check("y", y, ty, (B, T, H, p), dev)
    if S_T is not None:
        _check("S_T", S_T, torch.float32, state, dev)
    elif return_state:
        S_T = torch.empty(state, dtype=torch.float32, device=dev)
    lib = _lib.load()
    need = _ssm_bytes(dev.index, B, T, H, G, n, p, code, seg_len)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    _call(lib.kda_ssm_prefill, dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias),
          _ptr(S0), _ptr(lens), _ptr(y), _ptr(S_T), B, T, H, G, n, p, *strides, code, seg_len, _ptr(workspace),
          ws_bytes)
    return y, S_T


def ssm_step(x, dt, A, Bm, Cm, S, *, D=None, z=None, dt_bias=None, y=None):
    """One token of the scan for N sequences: x, z [N, H, p], dt [N, H], Bm, Cm [N, G, n]; ``S``
    [N, H, n, p] is updated in place.  Returns y [N, H, p]."""
    dev = _hip(x, "ssm_step")
    if x.dim() != 3:
        raise ValueError("x must be [N, H, p]")
    N = x.shape[0]
    ty = x.dtype
    code = _code(ty)
    (H, G, n, p), strides = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 1)
    _fits(N, H, G, n, p)
    _check("S", S, torch.float32, (N, H, n, p), dev)
    if y is None:
        y = x.new_empty((N, H, p))
    else:
        _check("y", y, ty, (N, H, p), dev)
    _call(_lib.load().kda_ssm_step, dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
          _ptr(dt_bias), _ptr(S), _ptr(y), N, H, G, n, p, *strides, code)
    return y


def _window_inputs(q, k, v, lead):
    dev, ty = q.device, q.dtype
    rows = q.shape[:lead]
    H, d = q.shape[lead:]
    if k.dim() != lead + 2:
        raise ValueError("k must have one axis of heads and one of channels after the tokens")
    Hkv = k.shape[lead]
    kv = (*rows, Hkv, d)
    return (H, Hkv, d), (_rows("q", q, ty, q.shape, dev, lead), _rows("k", k, ty, kv, dev, lead),
                         _rows("v", v, ty, kv, dev, lead))


def window_prefill(q, k, v, window, sinks=0, *, scale=None, k_cache=None, v_cache=None, start=None, lens=None,
                   o=None):
    """Attention of a prompt batch with a sliding window and ``sinks`` first tokens that stay visible: the
    query at position t sees key j <= t where t - j < window or j < sinks.  Returns o [B, T, H, d].

    q [B, T, H, d]; k, v [B, T, Hkv, d] with Hkv dividing H (all may be slices of a projection's rows).
    ``k_cache`` / ``v_cache`` [B, sinks + window, Hkv, d] are the sequences' ring caches: earlier tokens
    (``start`` [B] int32 of them, None = 0) are read from them and the new ones that stay visible are
    written to them.  ``lens`` (int32 [B]) gives the new tokens of each sequence of a padded batch; rows
    of o behind them are left as they were.  ``scale`` defaults to d ** -0.5.
    """
    dev = _hip(q, "window_prefill")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d]")
    B, T = q.shape[:2]
    ty = q.dtype
    code = _code(ty)
    (H, Hkv, d), strides = _window_inputs(q, k, v, 2)
    _fits(B, T, H, Hkv, d, window, sinks)
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache come together")
    if k_cache is not None:
        _check("k_cache", k_cache, ty, (B, sinks + window, Hkv, d), dev)
        _check("v_cache", v_cache, ty, (B, sinks + window, Hkv, d), dev)
    if start is not None:
        _check("start", start, torch.int32, (B,), dev)
    if lens is not None:
        _check("lens", lens, torch.int32, (B,), dev)
    if o is None:
        o = q.new_empty((B, T, H, d))
    else:
        _check("o", o, ty, (B, T, H, d), dev)
    _call(_lib.load().kda_window_prefill, dev, _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(start),
          _ptr(lens), _ptr(o), B, T, H, Hkv, d, window, sinks, max(d, 1) ** -0.5 if scale is None else scale, *strides, code)
    return o


@functools.lru_cache(maxsize=1024)
def _window_bytes(device, *shape):
    with torch.cuda.device(device):
        return int(_lib.load().kda_window_step_workspace_bytes(*shape))


def window_step_workspace_bytes(N, H, Hkv, d, window, sinks=0, dtype=torch.bfloat16):
    """Device workspace bytes of window_step for this shape on the current device."""
    _fits(N, H, Hkv, d, window, sinks)
    return int(_lib.load().kda_window_step_workspace_bytes(N, H, Hkv, d, window, sinks, _code(dtype)))


def window_step(q, k, v, k_cache, v_cache, pos, window, sinks=0, *, scale=None, o=None, workspace=None):
    """The same attention for one new token of N sequences over their ring caches, which receive the
    token's k and v: q [N, H, d], k, v [N, Hkv, d], ``pos`` (int32 [N]) the tokens before it.  Returns o."""
    dev = _hip(q, "window_step")
    if q.dim() != 3:
        raise ValueError("q must be [N, H, d]")
    N = q.shape[0]
    ty = q.dtype
    code = _code(ty)
    (H, Hkv, d), strides = _window_inputs(q, k, v, 1)
    _fits(N, H, Hkv, d, window, sinks)
    _check("k_cache", k_cache, ty, (N, sinks + window, Hkv, d), dev)
    _check("v_cache", v_cache, ty, (N, sinks + window, Hkv, d), dev)
    _check("pos", pos, torch.int32, (N,), dev)
    if o is None:
        o = q.new_empty((N, H, d))
    else:
        _check("o", o, ty, (N, H, d), dev)
    lib = _lib.load()
    need = _window_bytes(dev.index, N, H, Hkv, d, window, sinks, code)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    _call(lib.kda_window_step, dev, _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos), _ptr(o), N, H,
          Hkv, d, window, sinks, max(d, 1) ** -0.5 if scale is None else scale, *strides, code, _ptr(workspace), ws_bytes)
    return o
