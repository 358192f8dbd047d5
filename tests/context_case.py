"""Runs calls that opt in to large shared memory in two contexts of one device,
one after the other, through the C ABI and the driver API alone; exits 0 when
every call succeeds and both contexts' outputs agree bit for bit.  Run by
test_gpu_contexts.py in a process of its own."""

import ctypes
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_quantized_lora_quantize_b200 import qlora  # noqa: E402

cuda = ctypes.CDLL("libcuda.so.1")
P, SIZE = ctypes.c_void_p, ctypes.c_size_t
cuda.cuMemAlloc_v2.argtypes = [ctypes.POINTER(P), SIZE]
cuda.cuMemcpyHtoD_v2.argtypes = [P, P, SIZE]
cuda.cuMemcpyDtoH_v2.argtypes = [P, P, SIZE]
cuda.cuMemsetD8_v2.argtypes = [P, ctypes.c_ubyte, SIZE]


def ok(status):
    assert status == 0, f"driver call -> {status}"


def alloc(nbytes):
    p = P()
    ok(cuda.cuMemAlloc_v2(ctypes.byref(p), nbytes))
    ok(cuda.cuMemsetD8_v2(p, 0, nbytes))
    return p


def up(a):
    p = alloc(a.nbytes)
    ok(cuda.cuMemcpyHtoD_v2(p, a.ctypes.data, a.nbytes))
    return p


def down(p, nbytes):
    out = np.empty(nbytes, dtype=np.uint8)
    ok(cuda.cuMemcpyDtoH_v2(out.ctypes.data, p, nbytes))
    return out


def bf16(rng, *shape):
    return (rng.normal(size=shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def calls(L):
    """A pair GEMM, the norm's ring kernel and the 8-bit product; their outputs."""
    rng = np.random.default_rng(0)
    M, K, N, r = 300, 256, 264, 8
    nb = N * K // 64
    X, A, B = (up(bf16(rng, *s)) for s in ((M, K), (K, r), (r, N)))
    codes, aq = up(rng.integers(0, 256, N * K // 2, dtype=np.uint8)), up(rng.integers(1, 256, nb, dtype=np.uint8))
    sc = up(rng.random(-(-nb // 256)).astype(np.float32))
    Y, T, nws = alloc(M * N * 2), alloc(M * r * 4), L.qlora_workspace_bytes(M, K, N, r)
    status = [L.qlora_linear_fwd(X, M, K, N, codes, aq, sc, A, B, r, 0.5, Y, T, alloc(nws), nws, None)]
    mean, rstd = up(rng.random(M).astype(np.float32)), up(rng.random(M).astype(np.float32))
    dX, dw, db, nln = alloc(M * K * 2), alloc(K * 4), alloc(K * 4), L.qlora_layernorm_workspace_bytes(M, K)
    status.append(L.qlora_layernorm_bwd(X, up(bf16(rng, M, K)), mean, rstd, None, dX, dw, db, M, K, 0, 0, alloc(nln), nln,
                                        None))
    wq, ws, n8 = up(rng.integers(-127, 128, (N, K), dtype=np.int8)), up(rng.random(N).astype(np.float32)), \
        L.qlora_int8_workspace_bytes(M, K, N)
    Y8 = alloc(M * N * 2)
    status.append(L.qlora_linear_int8_fwd(X, M, K, N, 0, wq, K, ws, Y8, alloc(n8), n8, None))
    assert status == [0, 0, 0], f"{status} {L.qlora_last_cuda_error()}"
    ok(cuda.cuCtxSynchronize())
    return [down(p, n) for p, n in ((Y, M * N * 2), (T, M * r * 4), (dX, M * K * 2), (dw, K * 4), (db, K * 4),
                                    (Y8, M * N * 2))]


def main():
    ok(cuda.cuInit(0))
    dev, first, second = ctypes.c_int(), P(), P()
    ok(cuda.cuDeviceGet(ctypes.byref(dev), 0))
    ok(cuda.cuDevicePrimaryCtxRetain(ctypes.byref(first), dev))
    ok(cuda.cuCtxPushCurrent_v2(first))
    L = qlora.lib()
    one = calls(L)
    ok(cuda.cuCtxCreate_v2(ctypes.byref(second), 0, dev))  # now current
    two = calls(L)
    ok(cuda.cuCtxPopCurrent_v2(ctypes.byref(P())))
    again = calls(L)
    assert one[0].any() and one[2].any() and one[5].any()
    for a, b, c in zip(one, two, again):
        assert np.array_equal(a, b) and np.array_equal(a, c)


if __name__ == "__main__":
    main()
    print("contexts ok")
