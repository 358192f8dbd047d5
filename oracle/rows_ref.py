"""Oracle for the row-wise operators: dropout from a counter-based generator,
layer norm and its gradients, the two fused with a residual sum.

TEST INFRASTRUCTURE ONLY (see the package header).  numpy, float64; the
generator in Python's own integers' arithmetic on uint64 arrays.

The QLoRA pages have no counterpart: these are the usual definitions.  The
generator is Philox4x32-10 as published (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", SC 2011), pinned to that
paper's known-answer vectors.
"""

from __future__ import annotations

import numpy as np

_M32 = np.uint64(0xFFFFFFFF)
_S32 = np.uint64(32)


def philox4x32(counter, key) -> np.ndarray:
    """Ten rounds over a counter of four 32-bit words (arrays or numbers) with
    a key of two; returns uint32 [..., 4]."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k = [int(w) for w in key]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> _S32) ^ c[1] ^ np.uint64(k[0]), p1 & _M32, (p0 >> _S32) ^ c[3] ^ np.uint64(k[1]), p0 & _M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(np.broadcast_arrays(*c), axis=-1).astype(np.uint32)


def dropout_keep(rows: int, cols: int, p: float, seed: int, offset: int = 0) -> np.ndarray:
    """bool [rows, cols]: which elements stay."""
    groups = -(-cols // 8)
    n = np.arange(rows * groups, dtype=np.uint64) + np.uint64(offset & 0xFFFFFFFFFFFFFFFF)  # modulo 2^64
    words = philox4x32((n & _M32, n >> _S32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))
    draws = np.empty((rows * groups, 8), dtype=np.int64)
    draws[:, 0::2] = words & np.uint32(0xFFFF)
    draws[:, 1::2] = words >> np.uint32(16)
    return draws.reshape(rows, groups * 8)[:, :cols] >= round(65536 * p)


def dropout_gain(p: float) -> float:
    t = round(65536 * p)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def dropout(X, p: float, seed: int, offset: int = 0, residual=None) -> np.ndarray:
    """keep * (X * gain) + residual, dropped elements selected away."""
    X = np.asarray(X, dtype=np.float64)
    y = np.where(dropout_keep(*X.shape, p, seed, offset), X * dropout_gain(p), 0.0)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def layernorm(X, weight=None, bias=None, eps: float = 1e-5):
    """(Y, mean, rstd)."""
    X = np.asarray(X, dtype=np.float64)
    mean = X.mean(axis=1)
    d = X - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layernorm_grads(dY, X, mean, rstd, weight=None):
    """(dX, dweight, dbias) for the given statistics."""
    dY, X = np.asarray(dY, dtype=np.float64), np.asarray(X, dtype=np.float64)
    h = (X - np.asarray(mean, dtype=np.float64)[:, None]) * np.asarray(rstd, dtype=np.float64)[:, None]
    g = dY if weight is None else dY * weight
    dx = (g - g.mean(axis=1)[:, None] - h * (g * h).mean(axis=1)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    return dx, (dY * h).sum(axis=0), dY.sum(axis=0)
