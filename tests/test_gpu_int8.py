"""The 8-bit integer linear on the GPU: codes and scales bit for bit against
the oracle, products within the roundings of the epilogue.

The sums are whole numbers and exact.  Y takes one rounding of the sum to
float32, two float32 products (u = 2^-24 each) and one rounding to its type."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from oracle import matmul_int8, quantize_int8
from tests.helpers import f32, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(rows, cols, dtype, seed, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.empty(rows * cols + pad, dtype=dtype, device=DEV)
    buf[pad:] = (torch.randn(rows * cols, generator=g) * std).to(dtype).to(DEV)
    return buf[pad:].view(rows, cols)


def packed(rows, cols, seed, full=False):
    """Random codes with scales; `full` puts every code at +-127."""
    r = np.random.default_rng(seed)
    codes = r.choice([-127, 127], (rows, cols)) if full else r.integers(-127, 128, (rows, cols))
    ld = -(-cols // 16) * 16 + 16 * (seed % 2)
    buf = torch.full((rows, ld), 99, dtype=torch.int8, device=DEV)  # columns past the end are not read
    buf[:, :cols] = torch.from_numpy(codes.astype(np.int8)).to(DEV)
    scale = torch.from_numpy((0.001 + 0.01 * r.random(rows)).astype(np.float32)).to(DEV)
    return q.PackedInt8(buf, scale, (rows, cols)), codes, scale.double().cpu().numpy()


def check(Y, ref, name="Y"):
    half = torch.finfo(Y.dtype).eps / 2 if Y.dtype != torch.float32 else 0.0
    tiny = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}[Y.dtype]
    bad = ~(np.abs(f64(Y) - ref) <= 1.001 * (half + 3 * U) * np.abs(ref) + tiny)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}"


# ------------------------------------------------------------------ codes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 16, 0), (3, 7, 0), (16, 256, 0), (5, 257, 1), (300, 1000, 0),
                                           (1, 8192, 0), (310, 4096, 1), (40, 11003, 0), (300, 8192, 0), (2, 32768, 0),
                                           (2, 33001, 0)])
def test_codes_and_scales(dtype, rows, cols, pad):
    X = rand(rows, cols, TYPES[dtype], rows + cols, pad=pad)
    ld = -(-cols // 16) * 16 + 32
    out = q.PackedInt8(torch.full((rows, ld), 55, dtype=torch.int8, device=DEV),
                       torch.empty(rows, dtype=torch.float32, device=DEV), (rows, cols))
    assert q.qlora_quantize_int8(X, out=out) is out
    codes, scale = quantize_int8(f32(X))
    got = out.codes.cpu().numpy()
    np.testing.assert_array_equal(got[:, :cols], codes)
    np.testing.assert_array_equal(out.scale.cpu().numpy(), scale)
    end = -(-cols // 16) * 16
    assert (got[:, cols:end] == 0).all() and (got[:, end:] == 55).all()


def test_codes_at_the_borders():
    """Quotients on a half and one float32 step to either side of it, tiny and
    huge scales, zeros, rows with an infinity or a NaN."""
    rows = []
    for top in (127.0, 1.0, 3e38, 1e-20, 2e-38, 1e-42, 7e-45, 1e-45):
        s = np.float32(np.float32(top) / np.float32(127))
        h = ((np.arange(64) + 0.5) * float(s)).astype(np.float32)
        x = np.concatenate([h, np.nextafter(h, np.float32(np.inf)), np.nextafter(h, np.float32(0)), -h])
        x = np.clip(x, -np.float32(top), np.float32(top)).astype(np.float32)
        x[0] = top
        rows.append(x)
    X = np.stack(rows + [np.zeros(256, np.float32)] * 3)
    X[-2, 3], X[-1, 200] = np.inf, np.nan
    got = q.qlora_quantize_int8(torch.from_numpy(X).to(DEV))
    codes, scale = quantize_int8(X)
    np.testing.assert_array_equal(got.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(got.scale.cpu().numpy(), scale)


# ------------------------------------------------------------------ products
SHAPES = [(1, 1, 1), (1, 16, 8), (1, 128, 128), (1, 4096, 1000), (1, 8192, 8192), (2, 1000, 4099), (8, 11008, 256),
          (16, 256, 256), (17, 777, 300), (33, 4096, 4096), (64, 8192, 512), (65, 640, 129), (128, 5000, 1024),
          (129, 128, 16), (200, 100, 260), (300, 11003, 4099), (512, 2048, 2048), (257, 4096, 20000), (3000, 512, 136)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_product(M, K, N, dtype):
    X, xq, sx = packed(M, K, M + K)
    W, wq, sw = packed(N, K, N + 1)
    ws = q.new_int8_workspace(M, K, N, DEV)
    ws[1024:].fill_(77)
    Y = torch.full((M, N), float("nan"), dtype=TYPES[dtype], device=DEV)
    for _ in range(2):
        assert q.qlora_matmul_int8(X, W, TYPES[dtype], workspace=ws, Y=Y) is Y
        assert q.qlora_check_status(ws) == 0
        check(Y, matmul_int8(xq, sx, wq, sw))
    assert not ws[256:1024].any()  # the counters are back at zero


@pytest.mark.parametrize("M,N", [(1, 256), (100, 128), (300, 136)])
def test_deepest_sums_stay_exact(M, N):
    """K at the limit with every code at +-127: sums up to 2^31 - 1."""
    K = 133144
    X, xq, _ = packed(M, K, 1, full=True)
    W, wq, _ = packed(N, K, 3, full=True)
    W.codes[0] = X.codes[0, :W.codes.shape[1]] if W.codes.shape[1] <= X.codes.shape[1] else W.codes[0]
    wq = W.codes[:, :K].cpu().numpy()
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    Y = q.qlora_matmul_int8(q.PackedInt8(X.codes, one(M), (M, K)), q.PackedInt8(W.codes, one(N), (N, K)), torch.float32)
    check(Y, matmul_int8(xq, np.ones(M), wq, np.ones(N)))
    assert abs(float(Y.max()) - 127 * 127 * K) <= 128


@pytest.mark.parametrize("M,K,N", [(1, 1000, 512), (7, 4096, 4096), (100, 555, 300), (400, 1024, 768),
                                   (150, 999, 1001)])
@pytest.mark.parametrize("dtype", TYPES)
def test_linear_from_floats(M, K, N, dtype):
    t = TYPES[dtype]
    X, Wf = rand(M, K, t, 1), rand(N, K, torch.bfloat16, 2, std=0.02)
    if M > 2:
        X[1] = 0
    W = q.qlora_quantize_int8(Wf)
    ws = q.new_int8_workspace(M, K, N, DEV)
    Y = q.qlora_linear_int8_fwd(X, W, workspace=ws)
    assert q.qlora_check_status(ws) == 0
    (xq, sx), (wq, sw) = quantize_int8(f32(X)), quantize_int8(f32(Wf))
    check(Y, matmul_int8(xq, sx, wq, sw))
    # the two steps apart give the same bits
    assert torch.equal(Y, q.qlora_matmul_int8(q.qlora_quantize_int8(X), W, t, workspace=ws))


def test_a_bad_token_stays_alone():
    for M in (5, 200):
        X, W = rand(M, 512, torch.bfloat16, 1), q.qlora_quantize_int8(rand(300, 512, torch.bfloat16, 2))
        clean = q.qlora_linear_int8_fwd(X, W)
        X[3, 17] = float("inf")
        got = q.qlora_linear_int8_fwd(X, W)
        assert got[3].isnan().all()
        keep = torch.arange(M) != 3
        assert torch.equal(got[keep], clean[keep])


def test_single_rows_need_no_stride():
    """One row of codes of any length: there is no next row to be apart from."""
    X, xq, sx = packed(1, 777, 2)
    W, wq, sw = packed(1, 777, 4)
    for M_codes, N_codes in ((X.codes[:, :777], W.codes[:, :777]), (X.codes, W.codes)):
        Y = q.qlora_matmul_int8(q.PackedInt8(M_codes, X.scale, (1, 777)), q.PackedInt8(N_codes, W.scale, (1, 777)))
        check(Y, matmul_int8(xq, sx, wq, sw))


def test_one_workspace_for_several_sizes():
    ws = q.new_int8_workspace(128, 4096, 4096, DEV)
    for M, K, N in ((100, 4096, 4096), (1, 2048, 1000), (16, 4096, 300), (128, 1000, 4096), (1, 4096, 4096)):
        X, xq, sx = packed(M, K, M)
        W, wq, sw = packed(N, K, N)
        check(q.qlora_matmul_int8(X, W, workspace=ws), matmul_int8(xq, sx, wq, sw))


def test_captured_token_step_on_a_side_stream():
    W = q.qlora_quantize_int8(rand(1000, 768, torch.bfloat16, 2))
    X = rand(2, 768, torch.bfloat16, 1)
    ws = q.new_int8_workspace(2, 768, 1000, DEV)
    Y = torch.empty(2, 1000, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.qlora_linear_int8_fwd(X, W, workspace=ws, Y=Y)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            q.qlora_linear_int8_fwd(X, W, workspace=ws, Y=Y)
    for seed in (5, 6):
        X.copy_(rand(2, 768, torch.bfloat16, seed))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, q.qlora_linear_int8_fwd(X, W))
    assert q.qlora_check_status(ws) == 0


@pytest.mark.parametrize("M,N", [(1, 40), (100, 130)])
def test_deepest_sums_of_the_lowest_code(M, N):
    """-128 everywhere: sums of 2^14 K fit 32 bits up to K = 131071."""
    K = 131071
    low = lambda n: q.PackedInt8(torch.full((n, K + 1), -128, dtype=torch.int8, device=DEV),  # noqa: E731
                                 torch.ones(n, device=DEV), (n, K))
    Y = q.qlora_matmul_int8(low(M), low(N), torch.float32)
    assert (Y == float(np.float32(128 * 128 * K))).all()
