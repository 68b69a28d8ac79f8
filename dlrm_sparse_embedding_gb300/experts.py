"""Expert layer: tokens sorted by expert, their rows gathered, multiplied by
each expert's weights and added back, with the gradients.

Argument checks and marshalling only; the work is in libemb.so.  Tensors are on
the current CUDA device, calls run on the current torch stream or on `stream`,
and what they return is allocated for that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from ._lib import DTYPES, EmbExpertPlan, check, lib

_DTYPE_CODE = {torch.float32: DTYPES["f32"], torch.float16: DTYPES["f16"], torch.bfloat16: DTYPES["bf16"]}
MAX_EXPERTS = 1024
MAX_EXPERTS_PER_TOKEN = 64


def _on(stream):
    """Allocations belong to the stream that the call runs on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle(stream) -> int:
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _matrix(t, name: str, rows: int, width: Optional[int] = None, dtype=None, device=None) -> int:
    """Checks a [rows, width] matrix with contiguous rows; returns its row stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-d torch tensor" % name)
    if t.dtype not in _DTYPE_CODE:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    n, w = t.shape
    if n != rows or (width is not None and w != width) or w < 1:
        raise ValueError("%s must have shape (%d, %s), got %s" % (name, rows, width or "width", tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the plan on %s" % (name, t.device, device))
    s, c = t.stride()
    if n <= 1:
        s = w
    if (c != 1 and w > 1) or s < w:
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return s


def _dtype(dtype, default) -> torch.dtype:
    dtype = default if dtype is None else dtype
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be float32, float16 or bfloat16, got %s" % (dtype,))
    return dtype


class ExpertPlan:
    """Where each of a batch's assignments goes (see expert_sort).

    ``offsets`` int32 [E + 1], ``src`` int32 [T * k] and ``pos`` int32 [T, k]:
    expert e's rows are offsets[e] to offsets[e + 1], row p holds assignment
    src[p] = t * k + j, and token t's j-th expert has row pos[t, j] (-1: none).
    """

    __slots__ = ("offsets", "src", "pos", "tokens", "k", "experts", "device", "_c", "_ref")

    def __init__(self, offsets: torch.Tensor, src: torch.Tensor, pos: torch.Tensor):
        for t, name, dims in ((offsets, "offsets", 1), (src, "src", 1), (pos, "pos", 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
                raise ValueError("%s must be a contiguous %d-d int32 tensor" % (name, dims))
        for t, name in ((offsets, "offsets"), (src, "src"), (pos, "pos")):
            if not t.is_cuda or t.device != offsets.device:
                raise ValueError("%s must be a CUDA tensor on the plan's device" % name)
        T, k = pos.shape
        E = offsets.shape[0] - 1
        if not 1 <= k <= MAX_EXPERTS_PER_TOKEN or not 1 <= E <= MAX_EXPERTS:
            raise ValueError("a plan has 1 to %d experts and 1 to %d experts a token, got %d and %d"
                             % (MAX_EXPERTS, MAX_EXPERTS_PER_TOKEN, E, k))
        if src.shape[0] != T * k:
            raise ValueError("src holds %d assignments, pos %d" % (src.shape[0], T * k))
        self.offsets, self.src, self.pos = offsets, src, pos
        self.tokens, self.k, self.experts, self.device = T, k, E, offsets.device
        self._c = EmbExpertPlan(offsets.data_ptr(), src.data_ptr(), pos.data_ptr(), T, k, E)
        self._ref = ctypes.byref(self._c)

    @property
    def assignments(self) -> int:
        return self.tokens * self.k


def _plan(plan) -> ExpertPlan:
    if not isinstance(plan, ExpertPlan):
        raise ValueError("plan must be an ExpertPlan, got %s" % type(plan).__name__)
    return plan


def expert_sort(ids: torch.Tensor, num_experts: int, stream=None) -> ExpertPlan:
    """The plan of int32 or int64 ids [tokens, k] of experts in [0, num_experts).

    A stable sort: within an expert, assignments stay in order.  -1 marks an
    assignment without an expert; any other id outside the range is treated the
    same way and reported by dense_status()."""
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be an int32 or int64 tensor")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous [tokens, k], got %s" % (tuple(ids.shape),))
    if not ids.is_cuda:
        raise ValueError("ids must be a CUDA tensor")
    T, k = ids.shape
    E = int(num_experts)
    if not 1 <= k <= MAX_EXPERTS_PER_TOKEN or not 1 <= E <= MAX_EXPERTS:
        raise ValueError("1 to %d experts and 1 to %d experts a token are supported, got %d and %d"
                         % (MAX_EXPERTS, MAX_EXPERTS_PER_TOKEN, E, k))
    n = ctypes.c_size_t()
    check(lib.emb_expert_sort_workspace(T, k, E, ctypes.byref(n)), "emb_expert_sort_workspace")
    with _on(stream):
        i32 = dict(dtype=torch.int32, device=ids.device)
        plan = ExpertPlan(torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty((T, k), **i32))
        ws = torch.empty(n.value, dtype=torch.uint8, device=ids.device)   # torch's blocks start at 512 bytes
        check(lib.emb_expert_sort(ids.data_ptr(), ids.element_size(), plan._ref, ws.data_ptr(), n.value,
                                  _handle(stream)), "emb_expert_sort")
    return plan


def expert_dispatch(plan: ExpertPlan, x: torch.Tensor, dtype: Optional[torch.dtype] = None,
                    stream=None) -> torch.Tensor:
    """Rows [tokens * k, width] in expert order of x [tokens, width], in `dtype`
    (default x's); the rows after the last group are zero."""
    plan = _plan(plan)
    stride = _matrix(x, "x", plan.tokens, device=plan.device)
    dtype = _dtype(dtype, x.dtype)
    width = x.shape[1]
    with _on(stream):
        rows = torch.empty((plan.assignments, width), dtype=dtype, device=plan.device)
        check(lib.emb_expert_dispatch(plan._ref, x.data_ptr(), _DTYPE_CODE[x.dtype], stride, width, rows.data_ptr(),
                                      _DTYPE_CODE[dtype], _handle(stream)), "emb_expert_dispatch")
    return rows


def expert_dispatch_grad(plan: ExpertPlan, grad_rows: torch.Tensor, dtype: Optional[torch.dtype] = None,
                         stream=None) -> torch.Tensor:
    """Gradient [tokens, width] of expert_dispatch's x, in `dtype` (default grad_rows's)."""
    plan = _plan(plan)
    stride = _matrix(grad_rows, "grad_rows", plan.assignments, device=plan.device)
    dtype = _dtype(dtype, grad_rows.dtype)
    width = grad_rows.shape[1]
    with _on(stream):
        grad_x = torch.empty((plan.tokens, width), dtype=dtype, device=plan.device)
        check(lib.emb_expert_dispatch_grad(plan._ref, grad_rows.data_ptr(), _DTYPE_CODE[grad_rows.dtype], stride, width,
                                           grad_x.data_ptr(), _DTYPE_CODE[dtype], _handle(stream)),
              "emb_expert_dispatch_grad")
    return grad_x


def _weights(plan, weights) -> None:
    if (not isinstance(weights, torch.Tensor) or weights.dtype != torch.float32 or not weights.is_contiguous()
            or tuple(weights.shape) != (plan.tokens, plan.k)):
        raise ValueError("weights must be contiguous float32 [%d, %d]" % (plan.tokens, plan.k))
    if weights.device != plan.device:
        raise ValueError("weights is on %s, the plan on %s" % (weights.device, plan.device))


def expert_combine(plan: ExpertPlan, rows: torch.Tensor, weights: torch.Tensor, dtype: Optional[torch.dtype] = None,
                   stream=None) -> torch.Tensor:
    """[tokens, width]: each token's rows, weighted by float32 weights [tokens, k]
    and added in fp32, in `dtype` (default rows's)."""
    plan = _plan(plan)
    stride = _matrix(rows, "rows", plan.assignments, device=plan.device)
    _weights(plan, weights)
    dtype = _dtype(dtype, rows.dtype)
    width = rows.shape[1]
    with _on(stream):
        out = torch.empty((plan.tokens, width), dtype=dtype, device=plan.device)
        check(lib.emb_expert_combine(plan._ref, rows.data_ptr(), _DTYPE_CODE[rows.dtype], stride, weights.data_ptr(),
                                     width, out.data_ptr(), _DTYPE_CODE[dtype], _handle(stream)), "emb_expert_combine")
    return out


def expert_combine_grad(plan: ExpertPlan, grad_out: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                        stream=None):
    """(grad_rows in rows's dtype, grad_weights float32 [tokens, k]) of expert_combine."""
    plan = _plan(plan)
    stride = _matrix(rows, "rows", plan.assignments, device=plan.device)
    width = rows.shape[1]
    grad_stride = _matrix(grad_out, "grad_out", plan.tokens, width, device=plan.device)
    _weights(plan, weights)
    with _on(stream):
        grad_rows = torch.empty((plan.assignments, width), dtype=rows.dtype, device=plan.device)
        grad_weights = torch.empty((plan.tokens, plan.k), dtype=torch.float32, device=plan.device)
        check(lib.emb_expert_combine_grad(plan._ref, grad_out.data_ptr(), _DTYPE_CODE[grad_out.dtype], grad_stride,
                                          rows.data_ptr(), _DTYPE_CODE[rows.dtype], stride, weights.data_ptr(), width,
                                          grad_rows.data_ptr(), grad_weights.data_ptr(), _handle(stream)),
              "emb_expert_combine_grad")
    return grad_rows, grad_weights


def _linear(plan, t, name, width, dtype) -> int:
    s = _matrix(t, name, plan.assignments, width, dtype, plan.device)
    if s % 8 or t.data_ptr() % 16:
        raise ValueError("%s must be 16-byte aligned with a row stride that is a multiple of 8" % name)
    return s


def _weight(plan, weight):
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("weight must be a float16 or bfloat16 tensor")
    if weight.dim() != 3 or weight.shape[0] != plan.experts or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [%d, out, in], got %s" % (plan.experts, tuple(weight.shape)))
    _, N, K = weight.shape
    if N % 8 or K % 8 or N < 8 or K < 8 or weight.data_ptr() % 16:
        raise ValueError("weight's out and in widths must be multiples of 8 and its memory 16-byte aligned, got %s"
                         % (tuple(weight.shape),))
    if weight.device != plan.device:
        raise ValueError("weight is on %s, the plan on %s" % (weight.device, plan.device))
    return N, K


def expert_linear(plan: ExpertPlan, rows: torch.Tensor, weight: torch.Tensor, stream=None) -> torch.Tensor:
    """[tokens * k, out]: each expert's rows times the transpose of its own
    weight [out, in] of ``weight`` [E, out, in]; float16 or bfloat16, fp32 sums.
    Rows after the last group are not read; their products are zero."""
    plan = _plan(plan)
    N, K = _weight(plan, weight)
    stride = _linear(plan, rows, "rows", K, weight.dtype)
    with _on(stream):
        y = torch.empty((plan.assignments, N), dtype=weight.dtype, device=plan.device)
        check(lib.emb_expert_linear(plan._ref, rows.data_ptr(), stride, weight.data_ptr(), K, N,
                                    _DTYPE_CODE[weight.dtype], y.data_ptr(), _handle(stream)), "emb_expert_linear")
    return y


def expert_linear_grad(plan: ExpertPlan, grad_y: torch.Tensor, rows: Optional[torch.Tensor], weight: torch.Tensor,
                       need_rows: bool = True, need_weight: bool = True, stream=None):
    """(grad_rows, grad_weight) of expert_linear; None in the place of one that is not needed."""
    plan = _plan(plan)
    N, K = _weight(plan, weight)
    grad_stride = _linear(plan, grad_y, "grad_y", N, weight.dtype)
    code = _DTYPE_CODE[weight.dtype]
    grad_rows = grad_weight = None
    if need_weight:
        stride = _linear(plan, rows, "rows", K, weight.dtype)
    with _on(stream):
        if need_rows:
            grad_rows = torch.empty((plan.assignments, K), dtype=weight.dtype, device=plan.device)
            check(lib.emb_expert_linear_grad_rows(plan._ref, grad_y.data_ptr(), grad_stride, weight.data_ptr(), K, N,
                                                  code, grad_rows.data_ptr(), _handle(stream)),
                  "emb_expert_linear_grad_rows")
        if need_weight:
            grad_weight = torch.empty_like(weight)
            check(lib.emb_expert_linear_grad_weight(plan._ref, grad_y.data_ptr(), grad_stride, rows.data_ptr(), stride,
                                                    K, N, code, grad_weight.data_ptr(), _handle(stream)),
                  "emb_expert_linear_grad_weight")
    return grad_rows, grad_weight


def dense_status(stream=None) -> int:
    """Waits for the stream; returns and clears the device's sticky status of the
    expert calls and of orthogonalize (EMB_OK, EMB_ERR_KEY_RANGE, EMB_ERR_TIMEOUT)."""
    return int(lib.emb_dense_status(_handle(stream)))
