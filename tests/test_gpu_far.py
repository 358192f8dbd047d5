"""The row operators and the linears on tensors of over 2^32 elements: the last
rows come out as they do alone or by the formula, so no offset is cut short.
About 35 GB on the device at most."""

import pytest
import torch

import bit_quantized_lora_quantize_b200 as q

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROWS, TAIL = 530_000, 4
HALF = 2.0 ** -8  # half a step of bf16, relative


def far(rows, cols, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x.normal_(generator=g)
    return x


def close(got, want, slack):
    """One rounding to bf16 of a float32 value that is off by `slack`."""
    got, want = got.double(), want.double()
    bound = (want.abs() + slack) * HALF + slack
    assert bool(((got - want).abs() <= bound).all())


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cols", [8192, 8191])
def test_dropout_and_quantization(cols):
    X = far(ROWS, cols)
    assert X.numel() > 1 << 32
    first = (ROWS - TAIL) * -(-cols // 8)  # the tail's first counter
    tail = X[-TAIL:].clone()
    Y = q.qlora_dropout_fwd(X, 0.3, 9, 5)
    assert torch.equal(Y[-TAIL:], q.qlora_dropout_fwd(tail, 0.3, 9, 5 + first))
    del Y
    P, alone = q.qlora_quantize_int8(X), q.qlora_quantize_int8(tail)
    assert torch.equal(P.codes[-TAIL:], alone.codes) and torch.equal(P.scale[-TAIL:], alone.scale)


@pytest.mark.parametrize("cols", [8192, 8191])
def test_norms(cols):
    X, R = far(ROWS, cols), far(ROWS, cols, 1)
    Y, Z, mean, rstd = q.qlora_dropout_add_layernorm_fwd(X, R, 0.3, 9, 5)
    first = (ROWS - TAIL) * -(-cols // 8)
    assert torch.equal(Z[-TAIL:], q.qlora_dropout_fwd(X[-TAIL:].clone(), 0.3, 9, 5 + first,
                                                      residual=R[-TAIL:].clone()))
    z = Z[-TAIL:].double()
    m, v = z.mean(1, keepdim=True), z.var(1, unbiased=False, keepdim=True)
    r = (v + 1e-5).rsqrt()
    h = (z - m) * r
    # a float32 sum of n terms is off by at most n 2^-24 of the terms' magnitudes
    n24 = cols * 2.0 ** -24
    close(Y[-TAIL:], h, n24 * float((z.abs().mean() * r.max() + h.abs().max())))
    del Y, R
    dY = X
    ws = q.new_layernorm_workspace(ROWS, cols, "cuda")
    dX, dR, dw, db = q.qlora_dropout_add_layernorm_bwd(dY, None, Z, mean, rstd, 0.3, 9, 5, workspace=ws)
    d = dY[-TAIL:].double()
    dz = r * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
    slack = n24 * float(r.max() * (d.abs().max() + d.abs().mean() + h.abs().max() * (d * h).abs().mean() * 3))
    close(dR[-TAIL:], dz, slack)
    keep = q.qlora_dropout_fwd(torch.ones_like(dX[-TAIL:]), 0.3, 9, 5 + first) != 0
    assert bool((dX[-TAIL:][~keep] == 0).all())
    gain = 65536 / (65536 - round(65536 * 0.3))
    close(dX[-TAIL:], torch.where(keep, dz * gain, 0.0), gain * slack)
    assert bool(dw.isfinite().all() and db.isfinite().all())


@pytest.mark.parametrize("N", [65536, 65531])
def test_int8_product(N):
    M, K = 66_000, 48
    X = far(M, K)
    W = q.qlora_quantize_int8(far(N, K, 1))
    Y = q.qlora_linear_int8_fwd(X, W)
    assert Y.numel() > 1 << 32
    assert torch.equal(Y[-TAIL:], q.qlora_linear_int8_fwd(X[-TAIL:].clone(), W))
    last = q.PackedInt8(W.codes[-8:].contiguous(), W.scale[-8:].contiguous(), (8, K))
    assert torch.equal(Y[:, -8:], q.qlora_linear_int8_fwd(X, last))


def test_linear_with_adapter_dropout():
    M, K, N, r, p = 66_000, 65536, 64, 8, 0.3
    X = far(M, K)
    W = q.qlora_quantize_nf4(far(N, K, 1) * 0.05)
    A, B = far(K, r, 2) * 0.01, far(r, N, 3) * 0.1
    first = (M - TAIL) * (K // 8)
    tail, dY = X[-TAIL:].clone(), far(M, N, 4)
    Y, T = q.qlora_linear_fwd_dropout(X, W, A, B, 2.0, p, 9, 5)
    y, t = q.qlora_linear_fwd_dropout(tail, W, A, B, 2.0, p, 9, 5 + first)
    # the same products, summed in orders that may differ: a step of bf16, and
    # float32 sums of K terms apart by K 2^-23 of the terms' magnitudes
    mags = tail.double().abs().mean() * A.double().abs().mean() * K * 2.0 / (1 - p)
    assert float((T[-TAIL:] - t).abs().max()) <= K * 2.0 ** -23 * float(mags)
    close(Y[-TAIL:], y, float(y.abs().max()) * HALF + K * 2.0 ** -23 * float(y.abs().max()))
    dX, dA, dB = q.qlora_linear_bwd_dropout(dY, X, T, W, A, B, 2.0, p, 9, 5)
    dx, _, _ = q.qlora_linear_bwd_dropout(dY[-TAIL:].clone(), tail, t, W, A, B, 2.0, p, 9, 5 + first)
    close(dX[-TAIL:], dx, float(dx.abs().max()) * 2 * HALF)
    assert bool(dA.isfinite().all() and dB.isfinite().all())


def test_adapter_dropout_rows_past_one_grid():
    """More 64-row blocks than a grid's second dimension holds: the rows of the
    second launch come out bit for bit as they do alone (every row's sums are
    taken in the same order at any M)."""
    edge = 65535 * 64
    M, K, N, r, p, cut = edge + 300, 64, 64, 8, 0.3, edge - 200
    X, dY, T = far(M, K), far(M, N, 1), torch.randn(M, r, device="cuda")
    W = q.qlora_quantize_nf4(far(N, K, 2) * 0.05)
    A, B = far(K, r, 3) * 0.01, far(r, N, 4) * 0.1
    dX, _, _ = q.qlora_linear_bwd_dropout(dY, X, T, W, A, B, 2.0, p, 9, 5)
    alone, _, _ = q.qlora_linear_bwd_dropout(dY[cut:].clone(), X[cut:].clone(), T[cut:].clone(), W, A, B, 2.0, p, 9,
                                             5 + cut * (K // 8))
    assert torch.equal(dX[cut:], alone)
    first, _, _ = q.qlora_linear_bwd_dropout(dY[:512].clone(), X[:512].clone(), T[:512].clone(), W, A, B, 2.0, p, 9, 5)
    assert torch.equal(dX[:512], first)
