"""Layer norm of rows and its gradients (Python binding of the ``kda_layer_norm_*`` entry points of
include/kda.h).

Argument marshalling only: torch provides device memory and the current CUDA stream; all arithmetic
runs in libkda.so's kernels, and there is no CPU fallback. Every call enqueues on the current stream
of its tensors' device.
"""

from __future__ import annotations

import ctypes

import torch

from .decay import _F32, _ROPE_TYPES, _call, _p, _typed, _want, _written
from .kda import _check, load_library


def _rows(x, name):
    """Rows, width and row stride of a [..., width] tensor whose rows are contiguous and evenly apart."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a [..., width] tensor")
    if x.dtype not in _ROPE_TYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    width = x.shape[-1]
    if width < 1:
        raise ValueError(f"{name} must have at least one column")
    rows = x.numel() // width
    if rows == 0 or x.is_contiguous():
        return rows, width, width
    if width > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    stride, count = None, 1
    for size, st in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * count:
            raise ValueError(f"{name}: rows must be evenly apart")
        count *= size
    return rows, width, width if stride is None else stride


def kda_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None):
    """Layer norm over the last dimension, y = (x - mean) rstd weight + bias with rstd = 1 / sqrt(var + eps):
    returns (y, mean, rstd), the last two FP32 of x's shape without its last dimension, for the backward.
    x [..., width] BF16, FP16 or FP32, rows contiguous and evenly apart (columns of a wider tensor, say); weight, bias FP32
    [width] or None. ``out``: a contiguous tensor for y, which may be x."""
    lib = load_library()
    rows, width, stride = _rows(x, "x")
    dev = x.device
    if weight is not None:
        _want(weight, "weight", _F32, (width,), dev)
    if bias is not None:
        _want(bias, "bias", _F32, (width,), dev)
    y = out
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _want(y, "out", x.dtype, x.shape, dev)
    mean = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    _call(lib.kda_layer_norm_fwd, dev, x.data_ptr(), _ROPE_TYPES[x.dtype], _p(weight), _p(bias), rows, width, stride, eps,
          y.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    if out is not None:
        _written((y,))
    return y, mean, rstd


def kda_layer_norm_bwd(dy, x, weight, mean, rstd, bias=True, out=None, workspace=None):
    """Gradients of kda_layer_norm_fwd from that of its output, dy, its inputs and its mean and rstd: returns
    (dx, dweight, dbias), the last two FP32 [width], summed over all rows; dweight is None where there is no
    weight, dbias where ``bias`` is false. ``out``: a contiguous tensor for dx, which may be dy or x (width up to
    12288, FP32 8192). ``workspace``: a uint8 tensor for the partial sums (kda_layer_norm_workspace_bytes); None
    takes one for the call."""
    lib = load_library()
    rows, width, stride = _rows(x, "x")
    dev = x.device
    _typed(dy, "dy", x.dtype, x.shape, dev)
    dy_stride = _rows(dy, "dy")[2]
    if weight is not None:
        _want(weight, "weight", _F32, (width,), dev)
    _want(mean, "mean", _F32, x.shape[:-1], dev)
    _want(rstd, "rstd", _F32, x.shape[:-1], dev)
    dx = out
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _want(dx, "out", x.dtype, x.shape, dev)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = torch.empty((width,), dtype=_F32, device=dev) if bias else None
    if workspace is None:
        if (dweight is not None or dbias is not None) and rows:
            n = ctypes.c_size_t(0)
            _check(lib.kda_layer_norm_workspace_bytes(rows, width, ctypes.byref(n)))
            workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    else:
        _want(workspace, "workspace", torch.uint8, workspace.shape, dev)
    _call(lib.kda_layer_norm_bwd, dev, dy.data_ptr(), x.data_ptr(), _ROPE_TYPES[x.dtype], _p(weight), mean.data_ptr(),
          rstd.data_ptr(), rows, width, dy_stride, stride, dx.data_ptr(), _p(dweight), _p(dbias), _p(workspace),
          0 if workspace is None else workspace.numel())
    if out is not None:
        _written((dx,))
    return dx, dweight, dbias
