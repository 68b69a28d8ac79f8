"""Orthogonalised updates (Muon): argument checks and marshalling only.  Not part
of autograd's graph: the result requires no gradient even where the update does."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from ._lib import check, lib
from .experts import _DTYPE_CODE, _on, _stream

#: K. Jordan et al., "Muon" (2024)
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@functools.lru_cache(maxsize=256)
def _workspace(batch: int, rows: int, cols: int) -> int:
    n = ctypes.c_size_t()
    check(lib.emb_orthogonalize_workspace(batch, rows, cols, ctypes.byref(n)), "emb_orthogonalize_workspace")
    return n.value


def orthogonalize(update: torch.Tensor, steps: int = 5, coefficients: Tuple[float, float, float] = COEFFICIENTS,
                  eps: float = 1e-7, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bfloat16 [..., rows, cols]: each matrix of `update` (float32, float16 or
    bfloat16) with its singular values driven towards 1, by `steps` steps
    X <- a X + (b A + c A A) X, A = X X^T, from X = update / (|update|_F + eps).

    The steps' products take fp16 numbers, so the result is not fp32's: with the
    output's rounding to bf16 (1.7e-3 of the 2-norm) it is 2.1e-3 off after five
    steps, 3.4e-3 after eight and up to 2e-2 after 32 with the default coefficients,
    1.8e-3 with ones that converge.

    update: [rows, cols] or [batch, rows, cols] with contiguous rows, rows and
    cols up to 65536; steps 1 to 32.  out, if given, is contiguous bfloat16 of
    update's shape and may not overlap it."""
    if stream is not None:
        return _on(stream, orthogonalize, update, steps, coefficients, eps, out)
    if not isinstance(update, torch.Tensor) or update.dim() not in (2, 3):
        raise ValueError("update must be a 2-d or 3-d torch tensor")
    if update.dtype not in _DTYPE_CODE:
        raise ValueError("update must be float32, float16 or bfloat16, got %s" % update.dtype)
    if not update.is_cuda:
        raise ValueError("update must be a CUDA tensor")
    rows, cols = update.shape[-2:]
    batch = update.shape[0] if update.dim() == 3 else 1
    if not 1 <= rows <= 65536 or not 1 <= cols <= 65536 or batch > 65535:
        raise ValueError("matrices of 1 to 65536 rows and columns, 65535 at most, got %s" % (tuple(update.shape),))
    batch_stride = update.stride(0) if update.dim() == 3 and batch > 1 else 0
    row_stride = update.stride(-2) if rows > 1 else cols
    if (cols > 1 and update.stride(-1) != 1) or row_stride < cols:
        raise ValueError("update's rows must be contiguous and not overlap")
    if not 1 <= int(steps) <= 32:
        raise ValueError("steps must be in 1 .. 32, got %r" % (steps,))
    if len(coefficients) != 3:
        raise ValueError("coefficients are three numbers, got %r" % (coefficients,))
    if not float(eps) >= 0:
        raise ValueError("eps must not be negative, got %r" % (eps,))
    a, b, c = (float(v) for v in coefficients)
    size = _workspace(batch, rows, cols)
    if out is not None and (not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16 or out.shape != update.shape
                            or not out.is_contiguous() or out.device != update.device):
        raise ValueError("out must be contiguous bfloat16 %s on %s" % (tuple(update.shape), update.device))
    if out is None:
        out = torch.empty(update.shape, dtype=torch.bfloat16, device=update.device)
    ws = torch.empty(size, dtype=torch.uint8, device=update.device)   # torch's blocks start at 512 bytes
    check(lib.emb_orthogonalize(update.data_ptr(), _DTYPE_CODE[update.dtype], batch_stride, row_stride, batch, rows, cols,
                                int(steps), a, b, c, float(eps), out.data_ptr(), ws.data_ptr(), size,
                                _stream(update.device)), "emb_orthogonalize")
    return out
