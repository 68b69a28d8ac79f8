"""Layer norm and dropout of rows: argument checks and marshalling only.

Tensors are on the current CUDA device (ValueError if not), `stream` as in the
expert calls.  The backward pass is explicit: no call is part of autograd's graph.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Union

import torch

from ._lib import check, lib
from .experts import _DTYPE_CODE, _dtype, _on, _stream

_LOW64 = 2 ** 64 - 1
_LARGEST = torch.finfo(torch.float32).max


# Checks of shapes and types, which a program repeats call for call, are kept by those.
@functools.lru_cache(maxsize=1024)
def _rows(shape, stride, dtype, name: str, like=None):
    """Checks a [rows, width] matrix with contiguous rows (of shape `like`); returns its type code and row stride."""
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (name, dtype))
    if len(shape) != 2:
        raise ValueError("%s must be a 2-d torch tensor" % name)
    n, w = shape
    if w < 1 or (like is not None and shape != like):
        raise ValueError("%s must have shape %s, got %s" % (name, "(rows, width)" if like is None else tuple(like), tuple(shape)))
    s, c = stride
    if n <= 1:
        s = w
    if s < w or (c != 1 and w > 1):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return code, s


@functools.lru_cache(maxsize=1024)
def _params(width: int, weight, bias) -> int:
    """Checks a norm's rows' width and its parameters' types and shapes; returns their type code."""
    if width > 1 << 24:
        raise ValueError("rows of up to 2^24 elements are supported, got %d" % width)
    dtype = (weight or bias or (torch.float32,))[0]
    for name, given in (("weight", weight), ("bias", bias)):
        if given and (given[0] not in _DTYPE_CODE or tuple(given[1]) != (width,)):
            raise ValueError("%s must be a contiguous float32, float16 or bfloat16 tensor of %d elements" % (name, width))
        if given and given[0] != dtype:
            raise ValueError("weight and bias must have one type, got %s and %s" % (dtype, given[0]))
    return _DTYPE_CODE[dtype]


def _tensor(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a 2-d torch tensor" % name)


def _cuda(x, name: str) -> torch.device:
    device = x.device
    if device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor, is on %s" % (name, device))
    return device


def _there(t, name: str, device) -> int:
    if t.device != device:
        raise ValueError("%s must be on %s, is on %s" % (name, device, t.device))
    return t.data_ptr()


def _param(t, name: str, device) -> int:
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return _there(t, name, device)


def _eps(eps) -> float:
    eps = float(eps)
    if not 1e-24 <= eps <= _LARGEST:
        raise ValueError("eps must be in 1e-24 .. %g, got %r" % (_LARGEST, eps))
    return eps


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """[rows, width] in `dtype` (default x's): each row of x [rows, width] less its mean,
    over the root of its variance plus eps, times weight plus bias (each [width], of
    one type; None: ones, zeros).  Sums and statistics are fp32; x of any row stride;
    eps from 1e-24 to fp32's largest number."""
    if stream is not None:
        return _on(stream, layer_norm, x, weight, bias, eps, dtype)
    _tensor(x, "x")
    shape = x.shape
    code, stride = _rows(shape, x.stride(), x.dtype, "x")
    device = _cuda(x, "x")
    weight_ptr = bias_ptr = weight_is = bias_is = None
    if weight is not None:
        _tensor(weight, "weight")
        weight_is = weight.dtype, weight.shape
        weight_ptr = _param(weight, "weight", device)
    if bias is not None:
        _tensor(bias, "bias")
        bias_is = bias.dtype, bias.shape
        bias_ptr = _param(bias, "bias", device)
    param = _params(shape[1], weight_is, bias_is)
    eps = _eps(eps)
    dtype = dtype or x.dtype
    out_code = _dtype(dtype)
    y = torch.empty(shape, dtype=dtype, device=device)
    check(lib.emb_layer_norm(x.data_ptr(), code, stride, shape[0], shape[1], weight_ptr, bias_ptr, param, eps, y.data_ptr(), out_code,
                             _stream(device)), "emb_layer_norm")
    return y


@functools.lru_cache(maxsize=256)
def _grad_workspace(rows: int, width: int) -> int:
    n = ctypes.c_size_t()
    check(lib.emb_layer_norm_grad_workspace(rows, width, ctypes.byref(n)), "emb_layer_norm_grad_workspace")
    return n.value


def layer_norm_grad(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
                    need_x: bool = True, need_weight: bool = True, stream=None):
    """(grad_x in x's dtype, grad_weight and grad_bias [width] in weight's dtype, or float32
    without a weight) of layer_norm; None in the place of those that are not needed.
    The statistics are taken from x again."""
    if stream is not None:
        return _on(stream, layer_norm_grad, grad_y, x, weight, eps, need_x, need_weight)
    _tensor(x, "x")
    _tensor(grad_y, "grad_y")
    shape = x.shape
    code, stride = _rows(shape, x.stride(), x.dtype, "x")
    grad_code, grad_stride = _rows(grad_y.shape, grad_y.stride(), grad_y.dtype, "grad_y", shape)
    device = _cuda(x, "x")
    grad_ptr = _there(grad_y, "grad_y", device)
    rows, width = shape
    weight_ptr, weight_is, param_dtype = None, None, torch.float32
    if weight is not None:
        _tensor(weight, "weight")
        param_dtype = weight.dtype
        weight_is = param_dtype, weight.shape
        weight_ptr = _param(weight, "weight", device)
    param = _params(width, weight_is, None)
    eps = _eps(eps)
    grad_x = grad_weight = grad_bias = x_out = weight_out = bias_out = None
    if need_x:
        grad_x = torch.empty(shape, dtype=x.dtype, device=device)
        x_out = grad_x.data_ptr()
    if need_weight:
        grad_weight = torch.empty(width, dtype=param_dtype, device=device)
        grad_bias = torch.empty(width, dtype=param_dtype, device=device)
        weight_out, bias_out = grad_weight.data_ptr(), grad_bias.data_ptr()
    size = _grad_workspace(rows, width)
    ws = torch.empty(size, dtype=torch.uint8, device=device)   # torch's blocks start at 512 bytes
    check(lib.emb_layer_norm_grad(grad_ptr, grad_code, grad_stride, x.data_ptr(), code, stride, rows, width, weight_ptr, param, eps,
                                  x_out, weight_out, bias_out, ws.data_ptr(), size, _stream(device)), "emb_layer_norm_grad")
    return grad_x, grad_weight, grad_bias


def dropout(x: torch.Tensor, rate: float, seed: Union[int, torch.Tensor], offset: int = 0,
            residual: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """[rows, width] in `dtype` (default the residual's, else x's): x [rows, width] with a share `rate` of its
    elements dropped and the others divided by 1 - rate, plus `residual` (of the result's dtype).

    Which ones depends on seed, offset and the element's place (row * width + column)
    alone, so dropout_grad with the same ones drops the same, and nothing is stored.
    The rate counts in steps of 2^-16.  seed: an int, or an int64 CUDA tensor of one
    element, which the replays of a captured graph read anew.  offset: any number that
    sets one use of a seed apart from another (a layer's, a step's).  Of both the low
    64 bits are used."""
    if stream is not None:
        return _on(stream, dropout, x, rate, seed, offset, residual, dtype)
    _tensor(x, "x")
    shape = x.shape
    code, stride = _rows(shape, x.stride(), x.dtype, "x")
    device = _cuda(x, "x")
    rate = float(rate)
    if not 0.0 <= rate <= 1.0:
        raise ValueError("rate must be in 0 .. 1, got %r" % (rate,))
    dtype = dtype or (x if residual is None else residual).dtype
    out_code = _dtype(dtype)
    residual_ptr, residual_stride = None, 0
    if residual is not None:
        _tensor(residual, "residual")
        residual_code, residual_stride = _rows(residual.shape, residual.stride(), residual.dtype, "residual", shape)
        if residual_code != out_code:
            raise ValueError("residual must have the result's dtype %s, got %s" % (dtype, residual.dtype))
        residual_ptr = _there(residual, "residual", device)
    seed_ptr = None
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != device:
            raise ValueError("seed must be an int or an int64 tensor of one element on %s" % device)
        seed_ptr, seed = seed.data_ptr(), 0
    y = torch.empty(shape, dtype=dtype, device=device)
    check(lib.emb_dropout(x.data_ptr(), code, stride, shape[0], shape[1], rate, int(seed) & _LOW64, seed_ptr, int(offset) & _LOW64,
                          residual_ptr, residual_stride, y.data_ptr(), out_code, _stream(device)), "emb_dropout")
    return y


def dropout_grad(grad_y: torch.Tensor, rate: float, seed: Union[int, torch.Tensor], offset: int = 0,
                 dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Gradient of dropout's x, in `dtype` (default grad_y's), from the same rate, seed and
    offset; that of its residual is grad_y."""
    return dropout(grad_y, rate, seed, offset, None, dtype, stream)
