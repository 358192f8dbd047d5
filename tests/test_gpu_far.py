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


@pytest.mark.parametrize("cols", [8192, 8191])
def test_norm_parameter_gradients(cols):
    """Sums over every row whose terms mostly have one sign, so that rows left out,
    taken twice or read elsewhere show: the 5712 rows past 2^32 elements are
    1.1 % of each sum.  A column's sum is a chain over a block's rows (one row
    slot at these widths), then over slots and blocks; h takes two roundings."""
    X = far(ROWS, cols)
    X += 1.0
    _, mean, rstd = q.qlora_layernorm_fwd(X)
    _, dw, db = q.qlora_layernorm_bwd(X, X, mean, rstd)
    want = torch.zeros(4, cols, dtype=torch.float64, device="cuda")  # sums and sums of magnitudes
    for i in range(0, ROWS, 8192):
        x = X[i:i + 8192].double()
        t = x * ((x - mean[i:i + 8192, None]) * rstd[i:i + 8192, None])
        want += torch.stack([t.sum(0), t.abs().sum(0), x.sum(0), x.abs().sum(0)])
    blocks = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    slack = (-(-ROWS // blocks) + 16 + 20 + 8 + 5 + 4) * 1.01 * 2.0 ** -24
    assert bool(((dw - want[0]).abs() <= slack * want[1]).all())
    assert bool(((db - want[2]).abs() <= slack * want[3]).all())
    assert float((0.005 * want[0] / want[1]).min()) > slack  # rows left out would show


def test_adapter_gradients():
    """dA and dB of the linear with adapter dropout over 66000 rows of 65536
    columns, all terms positive: 0.7 % of each sum lies past 2^32 elements.  A
    tensor-core sum of n products is off by at most (n / 8 + 8) 2^-23 of their
    magnitudes, the bf16 pairs by 2^-16, U by its own sum."""
    M, K, N, r, p = 66_000, 65536, 64, 8, 0.3
    X, dY = far(M, K).abs_(), far(M, N, 4).abs_()
    W = q.qlora_quantize_nf4(far(N, K, 1) * 0.05)
    A, B = far(K, r, 2) * 0.01, far(r, N, 3).abs_() * 0.1
    T = torch.rand(M, r, device="cuda")
    _, dA, dB = q.qlora_linear_bwd_dropout(dY, X, T, W, A, B, 2.0, p, 9, 5)
    acc = lambda n: (n / 8 + 8) * 2.0 ** -23  # noqa: E731
    gain = 65536 / (65536 - round(65536 * p))
    u = 2.0 * gain * (dY.double() @ B.double().t())
    want = torch.zeros(K, r, dtype=torch.float64, device="cuda")
    for i in range(0, M, 4096):
        x = X[i:i + 4096]
        kept = q.qlora_dropout_fwd(torch.ones_like(x), p, 9, 5 + i * (K // 8)) != 0
        want += torch.where(kept, x, 0).double().t() @ u[i:i + 4096]
    slack = 1.01 * (acc(2 * M) + acc(N) + 2.0 ** -16 + 2.0 ** -22)
    assert bool(((dA - want).abs() <= slack * want).all())
    want = T.double().t() @ dY.double()
    assert bool(((dB - want).abs() <= slack * want).all())
    assert slack < 0.006
