"""Expert layer: tokens sorted by expert, their rows gathered, multiplied by
each expert's weights and added back, with the gradients.

Argument checks and marshalling only; the work is in libemb.so.  Tensors are on
the current CUDA device (ValueError if not).  Every call takes `stream`: it runs
on that stream (default: the current one), and what it returns is allocated for
it.  The caller orders it after the work that makes its inputs; memory of inputs
that are freed meanwhile is not used again before the call's work is done.

As everywhere in this package, the backward pass is explicit: no call is part of
autograd's graph, and what one returns requires no gradient even where its
inputs do.  The *_grad calls give the gradients; code under autograd calls them
from a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._lib import DTYPES, EmbExpertPlan, check, lib

_DTYPE_CODE = {torch.float32: DTYPES["f32"], torch.float16: DTYPES["f16"], torch.bfloat16: DTYPES["bf16"]}
MAX_EXPERTS = 1024
MAX_EXPERTS_PER_TOKEN = 64
SORT_ALONE = 4096   # assignments up to which a sort leaves its workspace alone


def _on(stream, call, *args):
    """`call` on another stream: what it returns is allocated for that stream, and
    its inputs' memory is kept until that stream has passed the call."""
    with torch.cuda.stream(stream):
        result = call(*args)
    for arg in args:
        for t in (arg.offsets, arg.src, arg.pos) if isinstance(arg, ExpertPlan) else (arg,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result


def _stream(device: torch.device) -> int:
    """The current stream, as an address; `device`, the tensors', has to be the current one
    (the library's calls run there, whatever their arguments' addresses)."""
    current = torch._C._cuda_getDevice()
    if device.index != current:
        raise ValueError("the tensors are on %s, the current device is cuda:%d" % (device, current))
    return torch._C._cuda_getCurrentRawStream(current)


def _matrix(t, name: str, rows: int, device, width: Optional[int] = None):
    """Checks a [rows, width] matrix with contiguous rows on `device`; returns its
    address, type code, row stride and width."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-d torch tensor" % name)
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    n, w = t.shape
    if n != rows or w < 1 or (width is not None and w != width):
        raise ValueError("%s must have shape (%d, %s), got %s" % (name, rows, width or "width", tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s is on %s, the plan on %s" % (name, t.device, device))
    s, c = t.stride()
    if n <= 1:
        s = w
    if s < w or (c != 1 and w > 1):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return t.data_ptr(), code, s, w


def _dtype(dtype) -> int:
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError("dtype must be float32, float16 or bfloat16, got %s" % (dtype,))
    return code


def _indices(t, name: str, dims: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-d int32 tensor" % (name, dims))


class ExpertPlan:
    """Where each of a batch's assignments goes (see expert_sort).

    ``offsets`` int32 [E + 1], ``src`` int32 [T * k] and ``pos`` int32 [T, k]:
    expert e's rows are offsets[e] to offsets[e + 1], row p holds assignment
    src[p] = t * k + j, and token t's j-th expert has row pos[t, j] (-1: none).
    """

    __slots__ = ("offsets", "src", "pos", "tokens", "k", "experts", "assignments", "device", "_c", "_ref")

    def __init__(self, offsets: torch.Tensor, src: torch.Tensor, pos: torch.Tensor):
        _indices(offsets, "offsets", 1)
        _indices(src, "src", 1)
        _indices(pos, "pos", 2)
        device = offsets.device
        if not (offsets.is_cuda and src.device == device and pos.device == device):
            raise ValueError("offsets, src and pos must be CUDA tensors on one device, got %s, %s and %s"
                             % (device, src.device, pos.device))
        T, k = pos.shape
        E = offsets.shape[0] - 1
        if not 1 <= k <= MAX_EXPERTS_PER_TOKEN or not 1 <= E <= MAX_EXPERTS:
            raise ValueError("a plan has 1 to %d experts and 1 to %d experts a token, got %d and %d"
                             % (MAX_EXPERTS, MAX_EXPERTS_PER_TOKEN, E, k))
        if src.shape[0] != T * k:
            raise ValueError("src holds %d assignments, pos %d" % (src.shape[0], T * k))
        self._set(offsets, src, pos, T, k, E, device)

    def _set(self, offsets, src, pos, T, k, E, device):
        self.offsets, self.src, self.pos = offsets, src, pos
        self.tokens, self.k, self.experts, self.assignments, self.device = T, k, E, T * k, device
        self._c = EmbExpertPlan(offsets.data_ptr(), src.data_ptr(), pos.data_ptr(), T, k, E)
        self._ref = ctypes.byref(self._c)
        return self


def _plan(plan) -> ExpertPlan:
    if not isinstance(plan, ExpertPlan):
        raise ValueError("plan must be an ExpertPlan, got %s" % type(plan).__name__)
    return plan


@functools.lru_cache(maxsize=256)
def _sort_workspace(tokens: int, k: int, experts: int) -> int:
    n = ctypes.c_size_t()
    check(lib.emb_expert_sort_workspace(tokens, k, experts, ctypes.byref(n)), "emb_expert_sort_workspace")
    return n.value


@functools.lru_cache(maxsize=None)
def _untouched(device: torch.device) -> torch.Tensor:
    """The workspace of sorts that do not use theirs (an allocation takes 2 us of a small sort's 15)."""
    return torch.empty(_sort_workspace(1, 1, 1), dtype=torch.uint8, device=device)


def expert_sort(ids: torch.Tensor, num_experts: int, stream=None) -> ExpertPlan:
    """The plan of int32 or int64 ids [tokens, k] of experts in [0, num_experts).

    A stable sort: within an expert, assignments stay in order.  -1 marks an
    assignment without an expert; any other id outside the range is treated the
    same way and reported by dense_status()."""
    if stream is not None:
        return _on(stream, expert_sort, ids, num_experts)
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
    device, i32 = ids.device, torch.int32
    plan = ExpertPlan.__new__(ExpertPlan)._set(
        torch.empty(E + 1, dtype=i32, device=device), torch.empty(T * k, dtype=i32, device=device),
        torch.empty((T, k), dtype=i32, device=device), T, k, E, device)
    size = _sort_workspace(T, k, E)
    if T * k <= SORT_ALONE:
        ws = _untouched(device)
    else:
        ws = torch.empty(size, dtype=torch.uint8, device=device)   # torch's blocks start at 512 bytes
    check(lib.emb_expert_sort(ids.data_ptr(), ids.element_size(), plan._ref, ws.data_ptr(), size, _stream(device)),
          "emb_expert_sort")
    return plan


def expert_dispatch(plan: ExpertPlan, x: torch.Tensor, dtype: Optional[torch.dtype] = None,
                    stream=None) -> torch.Tensor:
    """Rows [tokens * k, width] in expert order of x [tokens, width], in `dtype`
    (default x's); the rows after the last group are zero."""
    if stream is not None:
        return _on(stream, expert_dispatch, plan, x, dtype)
    device = _plan(plan).device
    ptr, code, stride, width = _matrix(x, "x", plan.tokens, device)
    dtype = dtype or x.dtype
    out_code = _dtype(dtype)
    rows = torch.empty((plan.assignments, width), dtype=dtype, device=device)
    check(lib.emb_expert_dispatch(plan._ref, ptr, code, stride, width, rows.data_ptr(), out_code, _stream(device)),
          "emb_expert_dispatch")
    return rows


def expert_dispatch_grad(plan: ExpertPlan, grad_rows: torch.Tensor, dtype: Optional[torch.dtype] = None,
                         stream=None) -> torch.Tensor:
    """Gradient [tokens, width] of expert_dispatch's x, in `dtype` (default grad_rows's)."""
    if stream is not None:
        return _on(stream, expert_dispatch_grad, plan, grad_rows, dtype)
    device = _plan(plan).device
    ptr, code, stride, width = _matrix(grad_rows, "grad_rows", plan.assignments, device)
    dtype = dtype or grad_rows.dtype
    out_code = _dtype(dtype)
    grad_x = torch.empty((plan.tokens, width), dtype=dtype, device=device)
    check(lib.emb_expert_dispatch_grad(plan._ref, ptr, code, stride, width, grad_x.data_ptr(), out_code,
                                       _stream(device)), "emb_expert_dispatch_grad")
    return grad_x


def _weights(plan, weights) -> int:
    if (not isinstance(weights, torch.Tensor) or weights.dtype != torch.float32 or not weights.is_contiguous()
            or weights.shape != plan.pos.shape):
        raise ValueError("weights must be contiguous float32 [%d, %d]" % (plan.tokens, plan.k))
    if weights.device != plan.device:
        raise ValueError("weights is on %s, the plan on %s" % (weights.device, plan.device))
    return weights.data_ptr()


def expert_combine(plan: ExpertPlan, rows: torch.Tensor, weights: torch.Tensor, dtype: Optional[torch.dtype] = None,
                   stream=None) -> torch.Tensor:
    """[tokens, width]: each token's rows, weighted by float32 weights [tokens, k]
    and added in fp32, in `dtype` (default rows's)."""
    if stream is not None:
        return _on(stream, expert_combine, plan, rows, weights, dtype)
    device = _plan(plan).device
    ptr, code, stride, width = _matrix(rows, "rows", plan.assignments, device)
    weights_ptr = _weights(plan, weights)
    dtype = dtype or rows.dtype
    out_code = _dtype(dtype)
    out = torch.empty((plan.tokens, width), dtype=dtype, device=device)
    check(lib.emb_expert_combine(plan._ref, ptr, code, stride, weights_ptr, width, out.data_ptr(), out_code,
                                 _stream(device)), "emb_expert_combine")
    return out


def expert_combine_grad(plan: ExpertPlan, grad_out: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                        stream=None):
    """(grad_rows in rows's dtype, grad_weights float32 [tokens, k]) of expert_combine."""
    if stream is not None:
        return _on(stream, expert_combine_grad, plan, grad_out, rows, weights)
    device = _plan(plan).device
    ptr, code, stride, width = _matrix(rows, "rows", plan.assignments, device)
    grad_ptr, grad_code, grad_stride, _ = _matrix(grad_out, "grad_out", plan.tokens, device, width)
    weights_ptr = _weights(plan, weights)
    grad_rows = torch.empty((plan.assignments, width), dtype=rows.dtype, device=device)
    grad_weights = torch.empty((plan.tokens, plan.k), dtype=torch.float32, device=device)
    check(lib.emb_expert_combine_grad(plan._ref, grad_ptr, grad_code, grad_stride, ptr, code, stride, weights_ptr, width,
                                      grad_rows.data_ptr(), grad_weights.data_ptr(), _stream(device)),
          "emb_expert_combine_grad")
    return grad_rows, grad_weights


def _operand(plan, t, name, width, code):
    """_matrix for an operand of the products; returns its address and row stride."""
    ptr, c, stride, _ = _matrix(t, name, plan.assignments, plan.device, width)
    if c != code:
        raise ValueError("%s must have weight's dtype, got %s" % (name, t.dtype))
    if stride % 8 or ptr % 16:
        raise ValueError("%s must be 16-byte aligned with a row stride that is a multiple of 8" % name)
    return ptr, stride


def _weight(plan, weight):
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("weight must be a float16 or bfloat16 tensor")
    if weight.dim() != 3 or weight.shape[0] != plan.experts or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [%d, out, in], got %s" % (plan.experts, tuple(weight.shape)))
    _, N, K = weight.shape
    ptr = weight.data_ptr()
    if N % 8 or K % 8 or N < 8 or K < 8 or ptr % 16:
        raise ValueError("weight's out and in widths must be multiples of 8 and its memory 16-byte aligned, got %s"
                         % (tuple(weight.shape),))
    if weight.device != plan.device:
        raise ValueError("weight is on %s, the plan on %s" % (weight.device, plan.device))
    return ptr, _DTYPE_CODE[weight.dtype], N, K


def expert_linear(plan: ExpertPlan, rows: torch.Tensor, weight: torch.Tensor, stream=None) -> torch.Tensor:
    """[tokens * k, out]: each expert's rows times the transpose of its own
    weight [out, in] of ``weight`` [E, out, in]; float16 or bfloat16, fp32 sums.
    Rows after the last group are not read; their products are zero."""
    if stream is not None:
        return _on(stream, expert_linear, plan, rows, weight)
    device = _plan(plan).device
    weight_ptr, code, N, K = _weight(plan, weight)
    ptr, stride = _operand(plan, rows, "rows", K, code)
    y = torch.empty((plan.assignments, N), dtype=weight.dtype, device=device)
    check(lib.emb_expert_linear(plan._ref, ptr, stride, weight_ptr, K, N, code, y.data_ptr(), _stream(device)),
          "emb_expert_linear")
    return y


def expert_linear_grad(plan: ExpertPlan, grad_y: torch.Tensor, rows: Optional[torch.Tensor], weight: torch.Tensor,
                       need_rows: bool = True, need_weight: bool = True, stream=None):
    """(grad_rows, grad_weight) of expert_linear; None in the place of one that is not needed."""
    if stream is not None:
        return _on(stream, expert_linear_grad, plan, grad_y, rows, weight, need_rows, need_weight)
    device = _plan(plan).device
    weight_ptr, code, N, K = _weight(plan, weight)
    grad_ptr, grad_stride = _operand(plan, grad_y, "grad_y", N, code)
    if need_weight:
        ptr, stride = _operand(plan, rows, "rows", K, code)
    grad_rows = grad_weight = None
    if need_rows:
        grad_rows = torch.empty((plan.assignments, K), dtype=weight.dtype, device=device)
        check(lib.emb_expert_linear_grad_rows(plan._ref, grad_ptr, grad_stride, weight_ptr, K, N, code,
                                              grad_rows.data_ptr(), _stream(device)), "emb_expert_linear_grad_rows")
    if need_weight:
        grad_weight = torch.empty_like(weight)
        check(lib.emb_expert_linear_grad_weight(plan._ref, grad_ptr, grad_stride, ptr, stride, K, N, code,
                                                grad_weight.data_ptr(), _stream(device)),
              "emb_expert_linear_grad_weight")
    return grad_rows, grad_weight


def dense_status(stream=None) -> int:
    """Waits for the stream; returns and clears the device's sticky status of the
    expert calls and of orthogonalize (EMB_OK, EMB_ERR_KEY_RANGE, EMB_ERR_TIMEOUT).
    The stream, if given, is one of the current device's."""
    if stream is None:
        return int(lib.emb_dense_status(torch.cuda.current_stream().cuda_stream))
    current = torch._C._cuda_getDevice()
    if stream.device.index != current:
        raise ValueError("the stream is on %s, the current device is cuda:%d" % (stream.device, current))
    return int(lib.emb_dense_status(stream.cuda_stream))
