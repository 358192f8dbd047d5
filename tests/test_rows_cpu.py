"""Host-side refusals of the row-wise operators: every invalid call returns
its status before anything is launched (fake pointers are never read)."""

import ctypes

import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from bit_quantized_lora_quantize_b200 import build as qbuild

FAKE = 1 << 20
BF16, FP16, FP32 = 0, 1, 2
WS = 1 << 40


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def test_dropout_validation(L):
    def call(x=FAKE, res=None, y=FAKE, rows=4, cols=8, dt=BF16, p=0.1, dev=None):
        return L.qlora_dropout_fwd(x, res, y, rows, cols, dt, p, 1, 2, dev, None)
    assert call(x=None) == 1 and call(y=None) == 1
    assert call(rows=0) == 1 and call(cols=0) == 1 and call(rows=-1) == 1
    assert call(dt=3) == 1 and call(dt=-1) == 1
    assert call(p=-0.01) == 1 and call(p=1.01) == 1 and call(p=float("nan")) == 1
    assert call(x=FAKE + 1) == 2 and call(dt=FP32, y=FAKE + 2) == 2 and call(res=FAKE + 1) == 2
    assert call(dev=FAKE + 4) == 2
    assert call(rows=1 << 31) == 3 and call(cols=1 << 31) == 3 and call(rows=1 << 30, cols=1 << 30) == 3
    assert L.qlora_dropout_bwd(None, FAKE, 4, 8, BF16, 0.1, 1, 2, None, None) == 1
    assert L.qlora_dropout_bwd(FAKE, FAKE, 4, 8, BF16, 2.0, 1, 2, None, None) == 1


def test_layernorm_validation(L):
    def fwd(x=FAKE, w=FAKE, b=FAKE, y=FAKE, m=FAKE, rows=4, cols=8, dt=BF16, wdt=BF16, eps=1e-5):
        return L.qlora_layernorm_fwd(x, w, b, y, m, FAKE, rows, cols, dt, wdt, ctypes.c_float(eps), None)
    assert fwd(x=None) == 1 and fwd(y=None) == 1
    assert fwd(rows=0) == 1 and fwd(cols=-8) == 1
    assert fwd(dt=5) == 1 and fwd(wdt=5) == 1
    assert fwd(wdt=FP16) == 3 and fwd(dt=FP32, wdt=BF16) == 3
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("inf")) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(x=FAKE + 1) == 2 and fwd(w=FAKE + 1) == 2 and fwd(wdt=FP32, b=FAKE + 2) == 2 and fwd(m=FAKE + 2) == 2
    assert fwd(rows=1 << 31) == 3

    def bwd(dy=FAKE, x=FAKE, m=FAKE, r=FAKE, dx=FAKE, dw=FAKE, rows=4, cols=8, ws=FAKE, nb=WS):
        return L.qlora_layernorm_bwd(dy, x, m, r, FAKE, dx, dw, FAKE, rows, cols, BF16, BF16, ws, nb, None)
    assert bwd(dy=None) == 1 and bwd(x=None) == 1 and bwd(m=None) == 1 and bwd(r=None) == 1 and bwd(dx=None) == 1
    assert bwd(rows=0) == 1 and bwd(cols=1 << 31) == 3
    assert bwd(ws=None) == 4 and bwd(nb=L.qlora_layernorm_workspace_bytes(4, 8) - 1) == 4
    assert bwd(ws=FAKE + 8) == 2 and bwd(dw=FAKE + 2) == 2 and bwd(dy=FAKE + 1) == 2


def test_fused_validation(L):
    def fwd(x=FAKE, res=FAKE, z=FAKE, p=0.1, dev=None):
        return L.qlora_dropout_add_layernorm_fwd(x, res, FAKE, FAKE, z, FAKE, FAKE, FAKE, 4, 8, BF16, BF16,
                                                 ctypes.c_float(1e-5), p, 1, 2, dev, None)
    assert fwd(x=None) == 1 and fwd(res=None) == 1 and fwd(z=None) == 1 and fwd(p=1.5) == 1
    assert fwd(dev=FAKE + 1) == 2 and fwd(z=FAKE + 1) == 2 and fwd(res=FAKE + 1) == 2

    def bwd(dy=FAKE, dz=None, dx=FAKE, dres=FAKE, p=0.1, dev=None, ws=FAKE, nb=WS):
        return L.qlora_dropout_add_layernorm_bwd(dy, dz, FAKE, FAKE, FAKE, FAKE, dx, dres, FAKE, FAKE, 4, 8, BF16, BF16,
                                                 p, 1, 2, dev, ws, nb, None)
    assert bwd(dy=None) == 1 and bwd(dx=None) == 1 and bwd(dres=None) == 1 and bwd(p=-1.0) == 1
    assert bwd(dz=FAKE + 1) == 2 and bwd(dev=FAKE + 4) == 2 and bwd(ws=None) == 4 and bwd(nb=16) == 4


def test_linear_dropout_validation(L):
    need = L.qlora_dropout_workspace_bytes(16, 256, 256, 8)
    assert need >= L.qlora_workspace_bytes(16, 256, 256, 8) + 16 * 256 * 2
    assert L.qlora_dropout_workspace_bytes(16, 250, 256, 8) == 0

    def fwd(x=FAKE, K=256, r=8, code=0, s=1.0, p=0.1, dev=None, ws=FAKE, nb=need):
        return L.qlora_linear_fwd_dropout(x, 16, K, 256, FAKE, FAKE, FAKE, code, FAKE, FAKE, r, ctypes.c_float(s), p, 1,
                                          2, dev, FAKE, FAKE, ws, nb, None)
    assert fwd(x=None) == 1 and fwd(p=1.01) == 1 and fwd(p=float("nan")) == 1 and fwd(s=float("inf")) == 1
    assert fwd(s=3e38, p=0.9) == 1  # the gain carries the scale past float32
    assert fwd(code=9) == 1 and fwd(r=0) == 1
    assert fwd(x=FAKE + 2) == 2 and fwd(dev=FAKE + 4) == 2
    assert fwd(K=250) == 3 and fwd(r=257) == 3
    assert fwd(ws=None) == 4 and fwd(nb=need - 1) == 4

    def bwd(dy=FAKE, t=FAKE, s=1.0, p=0.1, dev=None, nb=need):
        return L.qlora_linear_bwd_dropout(dy, FAKE, t, 16, 256, 256, FAKE, FAKE, FAKE, 0, FAKE, FAKE, 8,
                                          ctypes.c_float(s), p, 1, 2, dev, FAKE, FAKE, FAKE, FAKE, nb, None)
    assert bwd(dy=None) == 1 and bwd(t=None) == 1 and bwd(p=-0.1) == 1 and bwd(s=float("nan")) == 1
    assert bwd(dev=FAKE + 1) == 2 and bwd(nb=need - 1) == 4


def test_workspace_sizes(L):
    assert L.qlora_layernorm_workspace_bytes(0, 8) == 0 and L.qlora_layernorm_workspace_bytes(8, 0) == 0
    assert L.qlora_layernorm_workspace_bytes(1, 8) >= 256
    with pytest.raises(q.QloraError):
        q.new_layernorm_workspace(0, 8, "cpu")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 8)
    for call in (lambda: q.qlora_dropout_fwd(x, 0.1, 1), lambda: q.qlora_dropout_bwd(x, 0.1, 1),
                 lambda: q.qlora_layernorm_fwd(x),
                 lambda: q.qlora_layernorm_bwd(x, x, torch.zeros(2), torch.zeros(2)),
                 lambda: q.qlora_dropout_add_layernorm_fwd(x, x, 0.1, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_overlapping_tensors_are_refused(L):
    """4 rows of 8 bf16 values take 64 bytes: an output may begin where an
    input ends, not before."""
    X, Y, Z, R = (FAKE + i * 4096 for i in range(4))

    def drop(y, res=None, rows=4):
        return L.qlora_dropout_fwd(X, res, y, rows, 8, BF16, 0.1, 1, 2, None, None)
    assert drop(X) == 1 and drop(X + 62) == 1 and drop(X - 62) == 1 and drop(R + 2, res=R) == 1
    assert L.qlora_dropout_bwd(X, X, 4, 8, BF16, 0.1, 1, 2, None, None) == 1

    def norm(y=Y, m=Z, r=R, w=None):
        return L.qlora_layernorm_fwd(X, w, None, y, m, r, 4, 8, BF16, FP32, ctypes.c_float(1e-5), None)
    assert norm(y=X) == 1 and norm(m=X + 60) == 1 and norm(r=Z + 12) == 1 and norm(w=Y + 60) == 1

    def norm_bwd(dx=Y, dw=Z, db=R):
        return L.qlora_layernorm_bwd(X, X + 4096 * 8, X + 4096 * 9, X + 4096 * 10, None, dx, dw, db, 4, 8, BF16, BF16,
                                     X + 4096 * 11, WS, None)
    assert norm_bwd(dx=X) == 1 and norm_bwd(dx=X + 4096 * 8 + 32) == 1
    assert norm_bwd(db=Z) == 1 and norm_bwd(dw=Y + 60) == 1 and norm_bwd(dw=X + 4096 * 9 + 12) == 1

    def fused(z=Z, y=Y, res=R):
        return L.qlora_dropout_add_layernorm_fwd(X, res, None, None, z, y, None, None, 4, 8, BF16, BF16,
                                                 ctypes.c_float(1e-5), 0.1, 1, 2, None, None)
    assert fused(z=Y) == 1 and fused(z=R) == 1 and fused(y=X) == 1 and fused(res=Z + 62) == 1

    def fused_bwd(dx=Z, dres=R, dz=None):
        return L.qlora_dropout_add_layernorm_bwd(X, dz, Y, X + 4096 * 9, X + 4096 * 10, None, dx, dres, None, None, 4, 8,
                                                 BF16, BF16, 0.1, 1, 2, None, X + 4096 * 11, WS, None)
    assert fused_bwd(dx=R) == 1 and fused_bwd(dx=X) == 1 and fused_bwd(dres=Y + 2) == 1 and fused_bwd(dz=Z) == 1
