"""Thin Python binding of the row-wise operators of ``libqlora.so``: dropout
from a counter-based generator, layer norm, and the two fused with a residual
sum (formulas in include/qlora.h).

A tensor of any shape is a matrix whose rows run along its last dimension.
Every call runs on the tensors' device, on that device's current stream.
"""

from __future__ import annotations

import torch

from .qlora import QloraError, _check, _ptr, lib

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _call(name: str, dev: torch.device, *args) -> None:
    """The library call `name` on the current stream of `dev`."""
    f = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        status = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        _check(name, status)


def _matrix(X: torch.Tensor):
    """(rows, cols, dtype code) of the tensor that sets a call's sizes."""
    if not X.is_cuda:
        raise ValueError("qlora kernels take CUDA tensors only (no CPU path)")
    if X.dim() < 1 or not X.is_contiguous():
        raise ValueError("qlora kernels take contiguous tensors of at least one dimension")
    code = DTYPES.get(X.dtype)
    if code is None:
        raise ValueError("bfloat16, float16 or float32 tensors expected")
    cols = X.shape[-1]
    return (X.numel() // cols if cols else 0), cols, code


def _like(X: torch.Tensor, *ts: torch.Tensor | None) -> None:
    """Each tensor given matches X in shape, type and device and is contiguous."""
    for t in ts:
        if t is not None and (t.shape != X.shape or t.dtype != X.dtype or t.device != X.device
                              or not t.is_contiguous()):
            raise ValueError("contiguous tensors of one shape, type and device expected")


def _vector(X: torch.Tensor, n: int, t: torch.Tensor | None, what: str, *dtypes: torch.dtype) -> None:
    """The vector, if there is one, has n values of one of these types, where X is."""
    if t is not None and (t.numel() != n or t.dtype not in dtypes or t.device != X.device or not t.is_contiguous()):
        raise ValueError(f"{what}: {n} contiguous values on the inputs' device expected, of a supported type")


def _params(X: torch.Tensor, cols: int, weight, bias) -> int:
    """Type code of the norm's parameters."""
    _vector(X, cols, weight, "weight", X.dtype, torch.float32)
    _vector(X, cols, bias, "bias", X.dtype, torch.float32)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias of one type expected")
    given = weight if weight is not None else bias
    return DTYPES[X.dtype if given is None else given.dtype]


def _draws(X: torch.Tensor, seed: int, offset: int, offset_dev: torch.Tensor | None) -> int | None:
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset are unsigned 64-bit integers")
    if offset_dev is None:
        return None
    _vector(X, 1, offset_dev, "offset_dev", torch.int64, torch.uint64)
    return offset_dev.data_ptr()


def qlora_dropout_fwd(X: torch.Tensor, p: float, seed: int, offset: int = 0, residual: torch.Tensor | None = None,
                      Y: torch.Tensor | None = None, offset_dev: torch.Tensor | None = None) -> torch.Tensor:
    """Y = dropout(X) [+ residual].  The call uses rows * ceil(cols / 8)
    counters from `offset` (plus the value in the one-element int64 tensor
    `offset_dev`, read on the device)."""
    rows, cols, code = _matrix(X)
    if Y is None:
        Y = torch.empty_like(X)
    _like(X, residual, Y)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_dropout_fwd", X.device, _ptr(X), _opt(residual), _ptr(Y), rows, cols, code, p, seed, offset, dev)
    return Y


def qlora_dropout_bwd(dY: torch.Tensor, p: float, seed: int, offset: int = 0, dX: torch.Tensor | None = None,
                      offset_dev: torch.Tensor | None = None) -> torch.Tensor:
    """dX of the dropout drawn with the same p, seed and offset."""
    rows, cols, code = _matrix(dY)
    if dX is None:
        dX = torch.empty_like(dY)
    _like(dY, dX)
    dev = _draws(dY, seed, offset, offset_dev)
    _call("qlora_dropout_bwd", dY.device, _ptr(dY), _ptr(dX), rows, cols, code, p, seed, offset, dev)
    return dX


def qlora_layernorm_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().qlora_layernorm_workspace_bytes(rows, cols))


def new_layernorm_workspace(rows: int, cols: int, device) -> torch.Tensor:
    """Workspace of the layer norm's backward calls for these sizes."""
    nbytes = qlora_layernorm_workspace_bytes(rows, cols)
    if nbytes == 0:
        raise QloraError("qlora_layernorm_workspace_bytes", 3, f"rows={rows} cols={cols}")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the status word; the rest is written before it is read
    return ws


def _norm_workspace(X: torch.Tensor, rows: int, cols: int, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is None:
        return new_layernorm_workspace(rows, cols, X.device)
    if workspace.device != X.device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous uint8 tensor on the inputs' device expected")
    return workspace


def _stats_out(X: torch.Tensor, rows: int, mean, rstd):
    if mean is None:
        mean = torch.empty(rows, dtype=torch.float32, device=X.device)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=X.device)
    _vector(X, rows, mean, "mean", torch.float32)
    _vector(X, rows, rstd, "rstd", torch.float32)
    return mean, rstd


def _stats_in(X: torch.Tensor, rows: int, mean: torch.Tensor, rstd: torch.Tensor) -> None:
    if mean is None or rstd is None:
        raise ValueError("the mean and rstd of the forward are needed")
    _vector(X, rows, mean, "mean", torch.float32)
    _vector(X, rows, rstd, "rstd", torch.float32)


def _param_grads(X: torch.Tensor, cols: int, wanted: bool, dweight, dbias):
    if wanted and dweight is None:
        dweight = torch.empty(cols, dtype=torch.float32, device=X.device)
    if wanted and dbias is None:
        dbias = torch.empty(cols, dtype=torch.float32, device=X.device)
    _vector(X, cols, dweight, "dweight", torch.float32)
    _vector(X, cols, dbias, "dbias", torch.float32)
    return dweight, dbias


def qlora_layernorm_fwd(X: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                        eps: float = 1e-5, Y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                        rstd: torch.Tensor | None = None):
    """(Y, mean, rstd) of the layer norm of each row; weight and bias have X's
    type or float32, None stands for 1 and 0."""
    rows, cols, code = _matrix(X)
    wcode = _params(X, cols, weight, bias)
    if Y is None:
        Y = torch.empty_like(X)
    _like(X, Y)
    mean, rstd = _stats_out(X, rows, mean, rstd)
    _call("qlora_layernorm_fwd", X.device, _ptr(X), _opt(weight), _opt(bias), _ptr(Y), _ptr(mean), _ptr(rstd), rows,
          cols, code, wcode, eps)
    return Y, mean, rstd


def qlora_layernorm_bwd(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        dX: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                        dbias: torch.Tensor | None = None, param_grads: bool = True):
    """(dX, dweight, dbias); the parameters' gradients are float32, and None
    with ``param_grads=False`` unless their tensors are given."""
    rows, cols, code = _matrix(X)
    wcode = _params(X, cols, weight, None)
    if dX is None:
        dX = torch.empty_like(X)
    _like(X, dY, dX)
    _stats_in(X, rows, mean, rstd)
    dweight, dbias = _param_grads(X, cols, param_grads, dweight, dbias)
    workspace = _norm_workspace(X, rows, cols, workspace)
    _call("qlora_layernorm_bwd", X.device, _ptr(dY), _ptr(X), _ptr(mean), _ptr(rstd), _opt(weight), _ptr(dX),
          _opt(dweight), _opt(dbias), rows, cols, code, wcode, _ptr(workspace), workspace.numel())
    return dX, dweight, dbias


def qlora_dropout_add_layernorm_fwd(X: torch.Tensor, residual: torch.Tensor, p: float, seed: int, offset: int = 0,
                                    weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                                    eps: float = 1e-5, offset_dev: torch.Tensor | None = None,
                                    Y: torch.Tensor | None = None, Z: torch.Tensor | None = None,
                                    mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """(Y, Z, mean, rstd): Z = residual + dropout(X) and its layer norm Y."""
    rows, cols, code = _matrix(X)
    wcode = _params(X, cols, weight, bias)
    if Y is None:
        Y = torch.empty_like(X)
    if Z is None:
        Z = torch.empty_like(X)
    _like(X, residual, Y, Z)
    mean, rstd = _stats_out(X, rows, mean, rstd)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_dropout_add_layernorm_fwd", X.device, _ptr(X), _ptr(residual), _opt(weight), _opt(bias), _ptr(Z),
          _ptr(Y), _ptr(mean), _ptr(rstd), rows, cols, code, wcode, eps, p, seed, offset, dev)
    return Y, Z, mean, rstd


def qlora_dropout_add_layernorm_bwd(dY: torch.Tensor, dZ: torch.Tensor | None, Z: torch.Tensor, mean: torch.Tensor,
                                    rstd: torch.Tensor, p: float, seed: int, offset: int = 0,
                                    weight: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                    offset_dev: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                                    dresidual: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                                    dbias: torch.Tensor | None = None, param_grads: bool = True):
    """(dX, dresidual, dweight, dbias) of the fused call drawn with the same
    p, seed and offset; dZ is the gradient that reaches Z past the norm."""
    rows, cols, code = _matrix(Z)
    wcode = _params(Z, cols, weight, None)
    if dX is None:
        dX = torch.empty_like(Z)
    if dresidual is None:
        dresidual = torch.empty_like(Z)
    _like(Z, dY, dZ, dX, dresidual)
    _stats_in(Z, rows, mean, rstd)
    dev = _draws(Z, seed, offset, offset_dev)
    dweight, dbias = _param_grads(Z, cols, param_grads, dweight, dbias)
    workspace = _norm_workspace(Z, rows, cols, workspace)
    _call("qlora_dropout_add_layernorm_bwd", Z.device, _ptr(dY), _opt(dZ), _ptr(Z), _ptr(mean), _ptr(rstd),
          _opt(weight), _ptr(dX), _ptr(dresidual), _opt(dweight), _opt(dbias), rows, cols, code, wcode, p, seed,
          offset, dev, _ptr(workspace), workspace.numel())
    return dX, dresidual, dweight, dbias


__all__ = ["qlora_dropout_fwd", "qlora_dropout_bwd", "qlora_layernorm_workspace_bytes", "new_layernorm_workspace",
           "qlora_layernorm_fwd", "qlora_layernorm_bwd", "qlora_dropout_add_layernorm_fwd",
           "qlora_dropout_add_layernorm_bwd"]
