"""Host-side refusals of the 8-bit integer linear (fake pointers are never
read)."""

import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from bit_quantized_lora_quantize_b200 import build as qbuild

FAKE = 1 << 20
BF16, FP32 = 0, 2


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def test_quantize_validation(L):
    def call(x=FAKE, rows=4, cols=30, dt=BF16, codes=FAKE, ld=32, scale=FAKE):
        return L.qlora_quantize_int8(x, rows, cols, dt, codes, ld, scale, None)
    assert call(x=None) == 1 and call(codes=None) == 1 and call(scale=None) == 1
    assert call(rows=0) == 1 and call(cols=0) == 1 and call(dt=7) == 1
    assert call(ld=16) == 1 and call(ld=40) == 1  # too short, not a multiple of 16
    assert call(x=FAKE + 1) == 2 and call(codes=FAKE + 8) == 2 and call(scale=FAKE + 2) == 2
    assert call(rows=1 << 31) == 3


def test_product_validation(L):
    need = L.qlora_int8_workspace_bytes(4, 30, 8)
    assert need > 256

    def mm(x=FAKE, ldx=32, M=4, K=30, N=8, w=FAKE, ldw=32, y=FAKE, dt=BF16, ws=FAKE, nb=need):
        return L.qlora_matmul_int8(x, ldx, FAKE, M, K, N, w, ldw, FAKE, y, dt, ws, nb, None)
    assert mm(x=None) == 1 and mm(w=None) == 1 and mm(y=None) == 1 and mm(dt=3) == 1
    assert mm(M=0) == 1 and mm(K=-1) == 1 and mm(N=0) == 1
    assert mm(ldx=24) == 1 and mm(ldw=16) == 1
    assert mm(K=133145, ldx=133152, ldw=133152) == 3 and mm(M=1 << 31) == 3 and mm(N=(1 << 31) - 1) == 3
    assert mm(x=FAKE + 4) == 2 and mm(y=FAKE + 1) == 2 and mm(dt=FP32, y=FAKE + 2) == 2 and mm(ws=FAKE + 8) == 2
    assert mm(ws=None) == 4 and mm(nb=need - 1) == 4

    def lin(x=FAKE, M=4, K=30, N=8, dt=BF16, ldw=32, y=FAKE, ws=FAKE, nb=need):
        return L.qlora_linear_int8_fwd(x, M, K, N, dt, FAKE, ldw, FAKE, y, ws, nb, None)
    assert lin(x=None) == 1 and lin(y=None) == 1 and lin(M=0) == 1 and lin(dt=-1) == 1 and lin(ldw=31) == 1
    assert lin(x=FAKE + 1) == 2 and lin(K=1 << 20, ldw=1 << 20) == 3 and lin(ws=None) == 4 and lin(nb=0) == 4


def test_workspace_bytes(L):
    assert L.qlora_int8_workspace_bytes(0, 8, 8) == 0 and L.qlora_int8_workspace_bytes(1, 133145, 8) == 0
    with pytest.raises(q.QloraError):
        q.new_int8_workspace(1, 0, 8, "cpu")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 16)
    w = q.PackedInt8(torch.zeros(4, 16, dtype=torch.int8), torch.ones(4), (4, 16))
    for call in (lambda: q.qlora_quantize_int8(x), lambda: q.qlora_linear_int8_fwd(x, w),
                 lambda: q.qlora_matmul_int8(w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_overlapping_tensors_are_refused(L):
    """Rows of codes count from the first row to the end of the last."""
    X, C, S = FAKE, FAKE + 65536, FAKE + 2 * 65536

    def quant(codes=C, scale=S, ld=32):
        return L.qlora_quantize_int8(X, 4, 30, BF16, codes, ld, scale, None)
    assert quant(codes=X) == 1 and quant(codes=X + 224) == 1 and quant(scale=X + 236) == 1
    assert quant(scale=C + 124) == 1 and quant(codes=X - 96) == 1 and quant(codes=X - 320, ld=112) == 1
    need = L.qlora_int8_workspace_bytes(4, 30, 8)
    ws = FAKE + 3 * 65536

    def mm(y, w=C):
        return L.qlora_matmul_int8(X, 32, S, 4, 30, 8, w, 32, S + 4096, y, BF16, ws, need, None)
    assert mm(X + 124) == 1 and mm(C + 252) == 1 and mm(S - 62) == 1 and mm(S + 4096 + 30) == 1

    def lin(y):
        return L.qlora_linear_int8_fwd(X, 4, 30, 8, BF16, C, 32, S, y, ws, need, None)
    assert lin(X) == 1 and lin(X + 238) == 1 and lin(C + 252) == 1 and lin(S + 30) == 1 and lin(X - 62) == 1
