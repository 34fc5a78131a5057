"""Binding of linear attention with a decay for each head (include/selscan.h:
selscan_linattn_fwd, selscan_linattn_bwd, selscan_linattn_step): argument
marshalling only, as in ``selscan.py``."""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from functools import lru_cache

from . import selscan as _s
from .selscan import LinattnOptions, _check, _dtype_code, _ptr, _torch

_NO_CONTEXT = nullcontext()


def _dense(t, name, shape, dtype, device):
    """Pointer of a required dense operand; the checks in the order in which
    they are cheap (a decode step's call is bound by its host time)."""
    if t is not None and t.shape == shape and t.dtype is dtype and t.is_contiguous() \
            and t.device == device:
        return t.data_ptr()
    return _ptr(t, name, shape, dtype, device)  # says what is wrong


def _raw_stream(device):
    """Handle of the device's current stream."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(device.index) if get else torch.cuda.current_stream(device).cuda_stream


def _on(device, stream, tensors):
    """Context in which allocations and the launch belong to ``stream`` (None:
    the device's current one; a torch stream or a raw handle) on ``device``,
    whatever the current device is. ``tensors`` stay out of the allocator's
    hands until a given stream is done with them."""
    torch = _torch()
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return _NO_CONTEXT
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _rows(t, name, shape, dtype, device):
    """Pointer and elements between tokens of a [batch, L, heads, dim] operand
    whose heads are contiguous within a token and whose tokens are evenly
    spaced over the batch (a dense tensor, or a slice of a projection)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_cuda \
            and t.is_contiguous():
        return t.data_ptr(), 0
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    B, L, H, d = shape
    sb, sl, sh, sd = t.stride()
    row = sl if L > 1 else sb if B > 1 else H * d
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or row < H * d \
            or (B > 1 and L > 1 and sb != L * row):
        raise ValueError(f"{name}: heads must be contiguous within a token and tokens evenly "
                         f"spaced over the batch (strides {t.stride()}); call .contiguous()")
    return t.data_ptr(), row


@lru_cache(maxsize=512)
def _workspace(entry, device_index, *sizes):
    """Workspace bytes for these sizes (they depend on the device's SM count)."""
    torch = _torch()
    with torch.cuda.device(device_index):
        return int(getattr(_s.load_library(), entry)(*sizes))


def _operands(q, k, v, log_decay, initial_state, seqlens):
    """Checked sizes, dtype code and options of a call over whole sequences."""
    torch = _torch()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and k must be [batch, L, qk_heads, dk] and v [batch, L, heads, dv]")
    B, L, Hq, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    qp, qs = _rows(q, "q", (B, L, Hq, dk), dt, dev)
    kp, ks = _rows(k, "k", (B, L, Hq, dk), dt, dev)
    vp, vs = _rows(v, "v", (B, L, H, dv), dt, dev)
    per_token, per_head = _decays(log_decay, (B, L, H), H, dt, dev)
    opts = LinattnOptions(
        per_token, per_head,
        _ptr(initial_state, "initial_state", (B, H, dk, dv), torch.float32, dev, required=False),
        _ptr(seqlens, "seqlens", (B,), torch.int32, dev, required=False), qs, ks, vs)
    return (B, L, Hq, H, dk, dv), code, (qp, kp, vp), opts


def _scale(scale, dk):
    """The given scale or dk^−1/2 (a dk of zero is refused with the other sizes)."""
    return float(scale) if scale is not None else dk ** -0.5 if dk else 1.0


def _decays(log_decay, shape, heads, dtype, device):
    """The pair of pointers (decays per token, decays per head)."""
    if log_decay is None:
        return None, None
    if log_decay.dim() == 1:
        return None, _dense(log_decay, "log_decay", (heads,), _torch().float32, device)
    return _dense(log_decay, "log_decay", shape, dtype, device), None


def selscan_linattn_fwd(q, k, v, log_decay=None, scale=None, initial_state=None, seqlens=None,
                        y=None, final_state=None, return_final_state=False, stream=None):
    """Linear attention with a decay for each head (C ABI
    ``selscan_linattn_fwd``): S_t = exp(g_t)·S_{t−1} + k_t v_tᵀ, y_t =
    scale·S_tᵀ q_t.

    q, k: [batch, L, qk_heads, dk]; v: [batch, L, heads, dv] (heads a multiple
    of qk_heads: neighbouring heads share a query and a key; dk, dv ≤ 128;
    float32 or bfloat16, dense or slices of one projection). log_decay: g as
    [batch, L, heads] of q's dtype, or [heads] float32 (a fixed decay for each
    head), or None (no decay); −inf resets. scale: None for dk^−1/2.
    initial_state: [batch, heads, dk, dv] float32, may be final_state itself.
    seqlens: [batch] int32 on the GPU, the rows' lengths (tokens behind them are
    not used and get y = 0). Returns y [batch, L, heads, dv] (or (y,
    final_state))."""
    torch = _torch()
    sizes, code, ptrs, opts = _operands(q, k, v, log_decay, initial_state, seqlens)
    B, L, Hq, H, dk, dv = sizes
    dev = q.device
    scale = _scale(scale, dk)
    with _on(dev, stream, (q, k, v, log_decay, initial_state, seqlens, y, final_state)):
        if y is None:
            y = torch.empty_like(v, memory_format=torch.contiguous_format)
        if final_state is None and return_final_state:
            final_state = torch.empty(B, H, dk, dv, device=dev, dtype=torch.float32)
        nbytes = _workspace("selscan_linattn_workspace_bytes", dev.index, *sizes, code)
        ws = torch.empty(nbytes, device=dev, dtype=torch.uint8) if nbytes else None
        _check(_s.load_library().selscan_linattn_fwd(
            *ptrs, scale, ctypes.byref(opts), _dense(y, "y", (B, L, H, dv), q.dtype, dev),
            _ptr(final_state, "final_state", (B, H, dk, dv), torch.float32, dev, required=False),
            *sizes, code, ws.data_ptr() if nbytes else None, nbytes,
            _raw_stream(dev)))
    return (y, final_state) if return_final_state else y


def selscan_linattn_bwd(q, k, v, log_decay=None, scale=None, initial_state=None, seqlens=None,
                        dy=None, dfinal_state=None, stream=None):
    """Gradient of ``selscan_linattn_fwd`` for the loss Σ dy·y + Σ
    dfinal_state·final_state (C ABI ``selscan_linattn_bwd``). Inputs as for the
    forward; dy: [batch, L, heads, dv] of q's dtype; dfinal_state: [batch,
    heads, dk, dv] float32 or None. Returns a dict: dq, dk, dv (q's dtype,
    dense), dlog_decay ([batch, L, heads]; None unless log_decay has that shape:
    a decay given by head is a constant) and dh0 (the initial state's, float32;
    None without one)."""
    torch = _torch()
    sizes, code, ptrs, opts = _operands(q, k, v, log_decay, initial_state, seqlens)
    B, L, Hq, H, dk, dv = sizes
    dev, dt = q.device, q.dtype
    scale = _scale(scale, dk)
    with _on(dev, stream, (q, k, v, log_decay, initial_state, seqlens, dy, dfinal_state)):
        out = dict(
            dq=torch.empty(B, L, Hq, dk, device=dev, dtype=dt),
            dk=torch.empty(B, L, Hq, dk, device=dev, dtype=dt),
            dv=torch.empty(B, L, H, dv, device=dev, dtype=dt),
            # by the argument: an empty tensor's pointer is NULL
            dlog_decay=torch.empty(B, L, H, device=dev, dtype=dt)
            if log_decay is not None and log_decay.dim() == 3 else None,
            dh0=None if initial_state is None
            else torch.empty(B, H, dk, dv, device=dev, dtype=torch.float32))
        nbytes = _workspace("selscan_linattn_bwd_workspace_bytes", dev.index, *sizes, code)
        ws = torch.empty(nbytes, device=dev, dtype=torch.uint8) if nbytes else None
        _check(_s.load_library().selscan_linattn_bwd(
            *ptrs, scale, ctypes.byref(opts), _dense(dy, "dy", (B, L, H, dv), dt, dev),
            _ptr(dfinal_state, "dfinal_state", (B, H, dk, dv), torch.float32, dev, required=False),
            *(None if out[n] is None else out[n].data_ptr()
              for n in ("dq", "dk", "dv", "dlog_decay", "dh0")),
            *sizes, code, ws.data_ptr() if nbytes else None, nbytes,
            _raw_stream(dev)))
    return out


def selscan_linattn_step(state, q, k, v, log_decay=None, scale=None, y=None, stream=None):
    """One token of ``selscan_linattn_fwd``, in place on ``state`` [batch,
    heads, dk, dv] float32 (C ABI ``selscan_linattn_step``). q, k: [batch,
    qk_heads, dk]; v: [batch, heads, dv]; log_decay: [batch, heads] of q's
    dtype, or [heads] float32, or None. Returns y [batch, heads, dv]."""
    torch = _torch()
    if state.dim() != 4 or q.dim() != 3 or not q.is_cuda:
        if state.dim() == 4 and q.dim() == 3:
            raise ValueError("q must be a CUDA tensor")
        raise ValueError("state must be [batch, heads, dk, dv] and q [batch, qk_heads, dk]")
    B, H, dk, dv = state.shape
    Hq = q.shape[1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    scale = _scale(scale, dk)
    per_token, per_head = _decays(log_decay, (B, H), H, dt, dev)
    with _on(dev, stream, (state, q, k, v, log_decay, y)):
        if y is None:
            y = torch.empty_like(v)
        _check(_s.load_library().selscan_linattn_step(
            _dense(state, "state", (B, H, dk, dv), torch.float32, dev),
            _dense(q, "q", (B, Hq, dk), dt, dev), _dense(k, "k", (B, Hq, dk), dt, dev),
            _dense(v, "v", (B, H, dv), dt, dev), per_token, per_head, scale,
            _dense(y, "y", (B, H, dv), dt, dev), B, Hq, H, dk, dv, code,
            _raw_stream(dev)))
    return y
