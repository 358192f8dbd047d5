"""Oracle for the 8-bit integer linear: quantization by rows and the product.

TEST INFRASTRUCTURE ONLY (see the package header).  numpy; whole numbers in
int64, quotients in float64, which tells every quotient of two float32 values
from the halves between whole numbers up to 127 (they differ from a half by
at least 2^-25 or not at all).

The QLoRA pages have no counterpart: symmetric absmax quantization with a
scale per token and per output channel, the usual definition.
"""

from __future__ import annotations

import numpy as np


def quantize_int8(X):
    """(codes int8 [rows, cols], scale float32 [rows]) of float32 values."""
    X = np.asarray(X, dtype=np.float32)
    top = np.abs(X).max(axis=1)  # NaN where a row holds one
    with np.errstate(invalid="ignore", over="ignore"):
        scale = (top / np.float32(127)).astype(np.float32)
    codes = np.zeros(X.shape, dtype=np.int8)
    for i in range(X.shape[0]):
        if np.isfinite(scale[i]) and scale[i] > 0:
            q = np.rint(X[i].astype(np.float64) / float(scale[i]))  # ties to even
            codes[i] = np.clip(q, -127, 127).astype(np.int8)
    return codes, scale


def matmul_int8(xq, sx, wq, sw):
    """float64 [M, N]; the sums in whole numbers (float64 products are exact
    below 2^53)."""
    total = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    return total * np.asarray(sx, dtype=np.float64)[:, None] * np.asarray(sw, dtype=np.float64)[None, :]
