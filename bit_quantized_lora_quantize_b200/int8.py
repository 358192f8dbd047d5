"""Thin Python binding of the linear layer on 8-bit integer weights of
``libqlora.so`` (formulas in include/qlora.h).

Every call runs on the tensors' device, on that device's current stream.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from .qlora import QloraError, lib
from .rows import DTYPES, _call, _matrix, _out, _typed


@dataclass
class PackedInt8:
    """A matrix [rows, cols] as 8-bit codes with one scale per row.  Rows of
    codes lie ``codes.stride(0)`` bytes apart, a multiple of 16."""

    codes: torch.Tensor  # int8 [rows, ld], ld >= cols; -127..127 (-128 only up to 131071 columns)
    scale: torch.Tensor  # float32 [rows]
    shape: tuple

    @property
    def ld(self) -> int:
        # a single row has no next one to lie at a stride
        return self.codes.stride(0) if self.codes.shape[0] > 1 else -(-self.codes.shape[1] // 16) * 16


def _packed(X: torch.Tensor, p: PackedInt8, what: str):
    """(rows, cols, ld) of a packed matrix on X's device."""
    rows, cols = p.shape
    c, s, dev = p.codes, p.scale, X.device
    shape = c.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < cols or c.dtype != torch.int8 or c.device != dev \
            or c.stride(1) != 1:
        raise ValueError(f"{what}.codes: int8 [{rows}, >= {cols}] with unit stride along rows expected on {dev}")
    _typed(X, (rows,), torch.float32, what + ".scale", s)
    return rows, cols, p.ld


def qlora_quantize_int8(X: torch.Tensor, out: PackedInt8 | None = None) -> PackedInt8:
    """Quantize the rows of a matrix (tokens, or a weight's output channels).
    `out`, if given, is a PackedInt8 of the same shape that is overwritten."""
    rows, cols, code = _matrix(X)
    if X.dim() != 2:
        raise ValueError("a matrix expected")
    if out is None:
        ld = -(-cols // 16) * 16
        out = PackedInt8(torch.empty(rows, ld, dtype=torch.int8, device=X.device),
                         torch.empty(rows, dtype=torch.float32, device=X.device), (rows, cols))
    elif tuple(out.shape) != (rows, cols) or out.codes.shape[1] < -(-cols // 16) * 16:
        raise ValueError("out does not hold a matrix of this shape")
    _, _, ld = _packed(X, out, "out")
    _call("qlora_quantize_int8", X.device, X.data_ptr(), rows, cols, code, out.codes.data_ptr(), ld,
          out.scale.data_ptr())
    return out


def qlora_int8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().qlora_int8_workspace_bytes(M, K, N))


def new_int8_workspace(M: int, K: int, N: int, device) -> torch.Tensor:
    """Workspace of the 8-bit products for these sizes."""
    nbytes = qlora_int8_workspace_bytes(M, K, N)
    if nbytes == 0:
        raise QloraError("qlora_int8_workspace_bytes", 3, f"M={M} K={K} N={N}")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:1024].zero_()  # status word and counters; the rest is written before it is read
    return ws


def _workspace(X: torch.Tensor, M: int, K: int, N: int, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is None:
        return new_int8_workspace(M, K, N, X.device)
    return _typed(X, (workspace.numel(),), torch.uint8, "workspace", workspace)


def qlora_matmul_int8(X: PackedInt8, W: PackedInt8, dtype: torch.dtype = torch.bfloat16,
                      workspace: torch.Tensor | None = None, Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M, N] of type `dtype` for quantized inputs [M, K] and a weight [N, K]."""
    c = X.codes
    if not c.is_cuda:
        raise ValueError("qlora kernels take CUDA tensors only (no CPU path)")
    M, K, ldx = _packed(c, X, "X")
    N, Kw, ldw = _packed(c, W, "W")
    if Kw != K:
        raise ValueError("W: [N, K] for inputs [M, K] expected")
    if dtype not in DTYPES:
        raise ValueError("bfloat16, float16 or float32 results expected")
    workspace = _workspace(c, M, K, N, workspace)
    Y = _out(c, (M, N), dtype, "Y", Y)
    _call("qlora_matmul_int8", c.device, c.data_ptr(), ldx, X.scale.data_ptr(), M, K, N, W.codes.data_ptr(), ldw,
          W.scale.data_ptr(), Y.data_ptr(), DTYPES[dtype], workspace.data_ptr(), workspace.numel())
    return Y


def qlora_linear_int8_fwd(X: torch.Tensor, W: PackedInt8, workspace: torch.Tensor | None = None,
                          Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M, N] of X's type for inputs [M, K], quantized per token on the way."""
    M, K, code = _matrix(X)
    if X.dim() != 2:
        raise ValueError("a matrix expected")
    N, Kw, ldw = _packed(X, W, "W")
    if Kw != K:
        raise ValueError("W: [N, K] for inputs [M, K] expected")
    workspace = _workspace(X, M, K, N, workspace)
    Y = _out(X, (M, N), X.dtype, "Y", Y)
    _call("qlora_linear_int8_fwd", X.device, X.data_ptr(), M, K, N, code, W.codes.data_ptr(), ldw, W.scale.data_ptr(),
          Y.data_ptr(), workspace.data_ptr(), workspace.numel())
    return Y


__all__ = ["PackedInt8", "qlora_quantize_int8", "qlora_int8_workspace_bytes", "new_int8_workspace",
           "qlora_matmul_int8", "qlora_linear_int8_fwd"]
