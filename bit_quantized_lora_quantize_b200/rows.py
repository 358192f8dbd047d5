"""Thin Python binding of the row-wise operators of ``libqlora.so``: dropout
from a counter-based generator, layer norm, the two fused with a residual sum,
and the linear whose adapter sees dropped inputs (formulas in include/qlora.h).

A tensor of any shape is a matrix whose rows run along its last dimension.
Every call runs on the tensors' device, on that device's current stream.
Outputs passed in share no memory with the inputs or with one another.
"""

from __future__ import annotations

import torch

from .qlora import PackedNF4, QloraError, _check, lib, packed_sizes, qlora_workspace_bytes

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


_functions: dict = {}


def _call(name: str, dev: torch.device, *args) -> None:
    """The library call `name` on the current stream of `dev`."""
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    index = dev.index
    if index == _current_device():
        status = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(index))
    if status:
        _check(name, status)


# A small kernel runs for less time than torch.cuda.current_stream takes to
# build its object: ask for the handle itself where torch has that call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _matrix(X: torch.Tensor):
    """(rows, cols, dtype code) of the tensor that sets a call's sizes."""
    if not X.is_cuda:
        raise ValueError("qlora kernels take CUDA tensors only (no CPU path)")
    shape = X.shape
    if not shape or not X.is_contiguous():
        raise ValueError("qlora kernels take contiguous tensors of at least one dimension")
    code = DTYPES.get(X.dtype)
    if code is None:
        raise ValueError("bfloat16, float16 or float32 tensors expected")
    cols = shape[-1]
    if len(shape) == 2:
        return shape[0], cols, code
    return (X.numel() // cols if cols else 0), cols, code


def _like(X: torch.Tensor, *ts: torch.Tensor | None) -> None:
    """Each tensor given matches X in shape, type and device and is contiguous."""
    shape, dtype, dev = X.shape, X.dtype, X.device
    for t in ts:
        if t is not None and (t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous()):
            raise ValueError("contiguous tensors of one shape, type and device expected")


def _vector(X: torch.Tensor, n: int, t: torch.Tensor | None, what: str, *dtypes: torch.dtype) -> None:
    """The vector, if there is one, has n values of one of these types, where X is."""
    if t is not None and (t.dtype not in dtypes or t.numel() != n or t.device != X.device or not t.is_contiguous()):
        raise ValueError(f"{what}: {n} contiguous values on the inputs' device expected, of a supported type")


def _params(X: torch.Tensor, cols: int, weight, bias) -> int:
    """Type code of the norm's parameters: X's type or float32, one for both."""
    given = weight if weight is not None else bias
    if given is None:
        return DTYPES[X.dtype]
    dtype, dev = given.dtype, X.device
    if dtype != X.dtype and dtype != torch.float32:
        raise ValueError("weight and bias: the inputs' type or float32 expected")
    for t in (weight, bias):
        if t is not None and (t.dtype != dtype or t.numel() != cols or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"weight and bias: {cols} contiguous values of one type on the inputs' device expected")
    return DTYPES[dtype]


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
    _like(X, residual, Y)
    if Y is None:
        Y = torch.empty_like(X)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_dropout_fwd", X.device, X.data_ptr(), _opt(residual), Y.data_ptr(), rows, cols, code, p, seed,
          offset, dev)
    return Y


def qlora_dropout_bwd(dY: torch.Tensor, p: float, seed: int, offset: int = 0, dX: torch.Tensor | None = None,
                      offset_dev: torch.Tensor | None = None) -> torch.Tensor:
    """dX of the dropout drawn with the same p, seed and offset."""
    rows, cols, code = _matrix(dY)
    _like(dY, dX)
    if dX is None:
        dX = torch.empty_like(dY)
    dev = _draws(dY, seed, offset, offset_dev)
    _call("qlora_dropout_bwd", dY.device, dY.data_ptr(), dX.data_ptr(), rows, cols, code, p, seed, offset, dev)
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


# torch.empty_strided takes two thirds of torch.empty's time on the host, and
# short calls are bound by that.
def _vector_of(dev: torch.device, n: int) -> torch.Tensor:
    return torch.empty_strided((n,), (1,), dtype=torch.float32, device=dev)


def _two(X: torch.Tensor, n: int):
    """Two float32 vectors of n values."""
    first = _vector_of(X.device, n)
    return first, torch.empty_like(first)


def _stats_out(X: torch.Tensor, rows: int, mean, rstd):
    if mean is None and rstd is None:
        return _two(X, rows)
    if mean is None:
        mean = _vector_of(X.device, rows)
    if rstd is None:
        rstd = _vector_of(X.device, rows)
    _vector(X, rows, mean, "mean", torch.float32)
    _vector(X, rows, rstd, "rstd", torch.float32)
    return mean, rstd


def _stats_in(X: torch.Tensor, rows: int, mean: torch.Tensor, rstd: torch.Tensor) -> None:
    if mean is None or rstd is None:
        raise ValueError("the mean and rstd of the forward are needed")
    _vector(X, rows, mean, "mean", torch.float32)
    _vector(X, rows, rstd, "rstd", torch.float32)


def _param_grads(X: torch.Tensor, cols: int, wanted: bool, dweight, dbias):
    if wanted and dweight is None and dbias is None:
        return _two(X, cols)
    if wanted and dweight is None:
        dweight = _vector_of(X.device, cols)
    if wanted and dbias is None:
        dbias = _vector_of(X.device, cols)
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
    else:
        _like(X, Y)
    mean, rstd = _stats_out(X, rows, mean, rstd)
    _call("qlora_layernorm_fwd", X.device, X.data_ptr(), _opt(weight), _opt(bias), Y.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), rows, cols, code, wcode, eps)
    return Y, mean, rstd


def qlora_layernorm_bwd(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        dX: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                        dbias: torch.Tensor | None = None, param_grads: bool = True):
    """(dX, dweight, dbias); the parameters' gradients are float32, and None
    with ``param_grads=False`` unless their tensors are given."""
    rows, cols, code = _matrix(X)
    wcode = _params(X, cols, weight, None)
    _like(X, dY, dX)
    if dX is None:
        dX = torch.empty_like(X)
    _stats_in(X, rows, mean, rstd)
    dweight, dbias = _param_grads(X, cols, param_grads, dweight, dbias)
    workspace = _norm_workspace(X, rows, cols, workspace)
    _call("qlora_layernorm_bwd", X.device, dY.data_ptr(), X.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
          _opt(weight), dX.data_ptr(), _opt(dweight), _opt(dbias), rows, cols, code, wcode, workspace.data_ptr(),
          workspace.numel())
    return dX, dweight, dbias


def qlora_dropout_add_layernorm_fwd(X: torch.Tensor, residual: torch.Tensor, p: float, seed: int, offset: int = 0,
                                    weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                                    eps: float = 1e-5, offset_dev: torch.Tensor | None = None,
                                    Y: torch.Tensor | None = None, Z: torch.Tensor | None = None,
                                    mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """(Y, Z, mean, rstd): Z = residual + dropout(X) and its layer norm Y."""
    rows, cols, code = _matrix(X)
    wcode = _params(X, cols, weight, bias)
    _like(X, residual, Y, Z)
    if Y is None:
        Y = torch.empty_like(X)
    if Z is None:
        Z = torch.empty_like(X)
    mean, rstd = _stats_out(X, rows, mean, rstd)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_dropout_add_layernorm_fwd", X.device, X.data_ptr(), residual.data_ptr(), _opt(weight), _opt(bias),
          Z.data_ptr(), Y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, cols, code, wcode, eps, p, seed, offset,
          dev)
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
    _like(Z, dY, dZ, dX, dresidual)
    if dX is None:
        dX = torch.empty_like(Z)
    if dresidual is None:
        dresidual = torch.empty_like(Z)
    _stats_in(Z, rows, mean, rstd)
    dev = _draws(Z, seed, offset, offset_dev)
    dweight, dbias = _param_grads(Z, cols, param_grads, dweight, dbias)
    workspace = _norm_workspace(Z, rows, cols, workspace)
    _call("qlora_dropout_add_layernorm_bwd", Z.device, dY.data_ptr(), _opt(dZ), Z.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), _opt(weight), dX.data_ptr(), dresidual.data_ptr(), _opt(dweight), _opt(dbias), rows, cols,
          code, wcode, p, seed, offset, dev, workspace.data_ptr(), workspace.numel())
    return dX, dresidual, dweight, dbias


# ---------------------------------------------------------------- linear with adapter dropout
def qlora_dropout_workspace_bytes(M: int, K: int, N: int, r: int) -> int:
    return int(lib().qlora_dropout_workspace_bytes(M, K, N, r))


def new_dropout_workspace(M: int, K: int, N: int, r: int, device) -> torch.Tensor:
    """Workspace of the linear calls with adapter dropout for these sizes."""
    nbytes = qlora_dropout_workspace_bytes(M, K, N, r)
    if nbytes == 0:
        raise QloraError("qlora_dropout_workspace_bytes", 3, f"M={M} K={K} N={N} r={r}")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    # what the plain calls keep; the rest, of M x K values, is written before it is read
    ws[:qlora_workspace_bytes(M, K, N, r)].zero_()
    return ws


def _linear(X: torch.Tensor, W: PackedNF4, A: torch.Tensor, B: torch.Tensor, workspace: torch.Tensor | None):
    """(M, K, N, r, workspace) of a linear call, its inputs checked."""
    if not X.is_cuda:
        raise ValueError("qlora kernels take CUDA tensors only (no CPU path)")
    if X.dim() != 2 or len(W.shape) != 2 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("matrices expected")
    (M, K), N, r = X.shape, W.shape[0], A.shape[1]
    if W.shape[1] != K:
        raise ValueError("W: [N, K] for inputs [M, K] expected")
    if workspace is None:
        workspace = new_dropout_workspace(M, K, N, r, X.device)
    nc, nb, nb2 = packed_sizes(N * K)
    bf16, u8 = torch.bfloat16, torch.uint8
    _all_typed(X.device, ((X, (M, K), bf16, "X"), (A, (K, r), bf16, "A"), (B, (r, N), bf16, "B"),
                          (W.codes, (nc,), u8, "W.codes"), (W.absmax_q, (nb,), u8, "W.absmax_q"),
                          (W.absmax_scale, (nb2 + (W.dq == "centred_fp8"),), torch.float32, "W.absmax_scale"),
                          (workspace, (workspace.numel(),), u8, "workspace")))
    return M, K, N, r, workspace


def _all_typed(dev: torch.device, given) -> None:
    """Each (tensor, shape, type, name) is as it says, contiguous and on `dev`."""
    for t, shape, dtype, what in given:
        if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: contiguous {dtype} of shape {tuple(shape)} on {dev} expected")


def _typed(X: torch.Tensor, shape: tuple, dtype: torch.dtype, what: str, t: torch.Tensor) -> torch.Tensor:
    _all_typed(X.device, ((t, shape, dtype, what),))
    return t


def _out(X: torch.Tensor, shape: tuple, dtype: torch.dtype, what: str, t: torch.Tensor | None) -> torch.Tensor:
    if t is None:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=X.device)
    return _typed(X, shape, dtype, what, t)


def qlora_linear_fwd_dropout(X: torch.Tensor, W: PackedNF4, A: torch.Tensor, B: torch.Tensor, scale: float, p: float,
                             seed: int, offset: int = 0, workspace: torch.Tensor | None = None,
                             Y: torch.Tensor | None = None, T_save: torch.Tensor | None = None,
                             offset_dev: torch.Tensor | None = None):
    """(Y, T_save) for Y = X W'^T + (s dropout(X) A) B; the draws are those of
    ``qlora_dropout_fwd(X, p, seed, offset)``."""
    M, K, N, r, workspace = _linear(X, W, A, B, workspace)
    Y = _out(X, (M, N), torch.bfloat16, "Y", Y)
    T_save = _out(X, (M, r), torch.float32, "T_save", T_save)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_linear_fwd_dropout", X.device, X.data_ptr(), M, K, N, W.codes.data_ptr(), W.absmax_q.data_ptr(),
          W.absmax_scale.data_ptr(), W.code_value, A.data_ptr(), B.data_ptr(), r, scale, p, seed, offset, dev,
          Y.data_ptr(), T_save.data_ptr(), workspace.data_ptr(), workspace.numel())
    return Y, T_save


def qlora_linear_bwd_dropout(dY: torch.Tensor, X: torch.Tensor, T_save: torch.Tensor, W: PackedNF4, A: torch.Tensor,
                             B: torch.Tensor, scale: float, p: float, seed: int, offset: int = 0,
                             workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                             dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                             offset_dev: torch.Tensor | None = None):
    """(dX, dA, dB) of the forward drawn with the same p, seed and offset."""
    M, K, N, r, workspace = _linear(X, W, A, B, workspace)
    _all_typed(X.device, ((dY, (M, N), torch.bfloat16, "dY"), (T_save, (M, r), torch.float32, "T_save")))
    dX = _out(X, (M, K), torch.bfloat16, "dX", dX)
    dA = _out(X, (K, r), torch.float32, "dA", dA)
    dB = _out(X, (r, N), torch.float32, "dB", dB)
    dev = _draws(X, seed, offset, offset_dev)
    _call("qlora_linear_bwd_dropout", X.device, dY.data_ptr(), X.data_ptr(), T_save.data_ptr(), M, K, N,
          W.codes.data_ptr(), W.absmax_q.data_ptr(), W.absmax_scale.data_ptr(), W.code_value, A.data_ptr(),
          B.data_ptr(), r, scale, p, seed, offset, dev, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return dX, dA, dB


__all__ = ["qlora_dropout_fwd", "qlora_dropout_bwd", "qlora_layernorm_workspace_bytes", "new_layernorm_workspace",
           "qlora_layernorm_fwd", "qlora_layernorm_bwd", "qlora_dropout_add_layernorm_fwd",
           "qlora_dropout_add_layernorm_bwd", "qlora_dropout_workspace_bytes", "new_dropout_workspace",
           "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout"]
