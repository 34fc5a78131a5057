"""Binding of the block-norm junction (include/selscan.h:
selscan_block_norm_fwd, selscan_block_norm_bwd): argument marshalling only, as
in ``selscan.py``."""
from __future__ import annotations

import ctypes

from . import selscan as _s
from .linattn import _dense, _on, _raw_stream
from .selscan import BlockNormOptions, _check, _dtype_code, _ptr, _torch

GATES = {"before": 1, "after": 2}


def _flat(t, name, shape, dtype, device):
    """Pointer and elements between rows of a [..., dim] operand with evenly
    spaced rows."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_cuda \
            and t.is_contiguous():
        return t.data_ptr(), 0
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    dim = shape[-1]
    # rows evenly spaced: every leading stride is the next one times its size
    row = None
    span = 1
    for n, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if row is None:
            row = st
        elif st != row * span:
            row = -1
            break
        span *= n
    if (dim > 1 and t.stride(-1) != 1) or (row is not None and row < dim):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced (strides "
                         f"{t.stride()}); call .contiguous()")
    return t.data_ptr(), 0 if row is None else row


def _options(x, z, weight, residual, res_scale, next_weight, groups, eps, gate, want_f32):
    torch = _torch()
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    shape, dev, dt = x.shape, x.device, x.dtype
    dim = shape[-1]
    code = _dtype_code(x)
    if gate not in GATES:
        raise ValueError(f"gate must be one of {list(GATES)}")
    rt = dt
    if residual is not None:
        rt = residual.dtype
        if rt not in (dt, torch.float32):
            raise TypeError(f"residual has dtype {rt}, expected {dt} or float32")
    elif want_f32:
        rt = torch.float32
    f32 = torch.float32
    xp, xs = _flat(x, "x", shape, dt, dev)
    zp, zs = (None, 0) if z is None else _flat(z, "z", shape, dt, dev)
    row = (dim,)
    opts = BlockNormOptions(
        zp, xs, zs, None if weight is None else _dense(weight, "weight", row, f32, dev),
        None if residual is None else _dense(residual, "residual", shape, rt, dev),
        None if res_scale is None else _dense(res_scale, "res_scale", row, f32, dev),
        None if next_weight is None else _dense(next_weight, "next_weight", row, f32, dev),
        groups, 0 if z is None else GATES[gate], int(rt == f32), eps)
    rows = x.numel() // dim if dim else 0
    return xp, opts, rt, rows, dim, code


def selscan_block_norm_fwd(x, z=None, weight=None, residual=None, res_scale=None,
                           next_weight=None, groups=1, eps=1e-5, gate="after", out=None, y=None,
                           out_f32=False, stream=None):
    """What stands between two blocks, in one pass (C ABI
    ``selscan_block_norm_fwd``): u = RMSNorm(x)·weight, gated by silu(z) (gate
    "after" the norm or "before" it); out = residual + res_scale·u; y =
    RMSNorm(out)·next_weight.

    x, z: [..., dim] float32 or bfloat16 with evenly spaced rows; weight,
    res_scale, next_weight: [dim] float32, each optional; residual: x's shape,
    x's dtype or float32; groups: groups of the first norm. Returns (out, y):
    out has the residual's dtype (without one x's, or float32 with
    ``out_f32``) and may be given as the residual itself; y is None without
    next_weight."""
    torch = _torch()
    xp, opts, rt, rows, dim, code = _options(x, z, weight, residual, res_scale, next_weight,
                                             groups, eps, gate, out_f32)
    dev = x.device
    with _on(dev, stream, (x, z, weight, residual, res_scale, next_weight, out, y)):
        if out is None:
            out = torch.empty_like(x, dtype=rt, memory_format=torch.contiguous_format)
        if y is None and next_weight is not None:
            y = torch.empty_like(x, memory_format=torch.contiguous_format)
        _check(_s.load_library().selscan_block_norm_fwd(
            xp, ctypes.byref(opts), _dense(out, "out", x.shape, rt, dev),
            None if y is None else _dense(y, "y", x.shape, x.dtype, dev), rows, dim, code,
            _raw_stream(dev)))
    return out, y


def selscan_block_norm_bwd(x, z=None, weight=None, residual=None, res_scale=None,
                           next_weight=None, groups=1, eps=1e-5, gate="after", dout=None, dy=None,
                           out_f32=False, stream=None):
    """Gradient of ``selscan_block_norm_fwd`` for the loss Σ dout·out + Σ dy·y
    (C ABI ``selscan_block_norm_bwd``). Inputs as for the forward; dout: out's
    shape and dtype or None; dy: x's shape and dtype, with next_weight. Returns
    a dict: dx, dz, dresidual, dweight, dres_scale, dnext_weight (the weights'
    float32; None where the input was None)."""
    torch = _torch()
    xp, opts, rt, rows, dim, code = _options(x, z, weight, residual, res_scale, next_weight,
                                             groups, eps, gate, out_f32)
    dev, f32 = x.device, torch.float32
    with _on(dev, stream, (x, z, weight, residual, res_scale, next_weight, dout, dy)):
        def like(t, dtype):
            return None if t is None else torch.empty_like(
                t, dtype=dtype, memory_format=torch.contiguous_format)

        out = dict(dx=like(x, x.dtype), dz=like(z, x.dtype), dresidual=like(residual, rt),
                   dweight=like(weight, f32), dres_scale=like(res_scale, f32),
                   dnext_weight=like(next_weight, f32))
        nbytes = int(_s.load_library().selscan_block_norm_bwd_workspace_bytes(rows, dim))
        ws = torch.empty(nbytes, device=dev, dtype=torch.uint8) if nbytes else None
        _check(_s.load_library().selscan_block_norm_bwd(
            xp, ctypes.byref(opts),
            None if dout is None else _dense(dout, "dout", x.shape, rt, dev),
            None if dy is None else _dense(dy, "dy", x.shape, x.dtype, dev),
            *(None if t is None else t.data_ptr() for t in out.values()), rows, dim, code,
            ws.data_ptr() if nbytes else None, nbytes,
            _raw_stream(dev)))
    return out
