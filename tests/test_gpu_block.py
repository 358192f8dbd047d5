"""The operators in a row, as a block uses them: a fine-tuning step of one
sub-layer (norm, 4-bit linear with adapter dropout, residual dropout and the
next norm, and back), and the serving step on an 8-bit weight.

The oracle runs the same chain in float64 from the same inputs, each stage on
the GPU's own result of the stage before it (as the backward of a real step
does with what was saved), so every stage is held to its own bound: the
linear's outputs to 2e-2 of their RMS like its other parity tests, the
row-wise outputs to one rounding of their type and what their sums are off by."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from bit_quantized_lora_quantize_b200 import synthetic
from oracle import (dropout, dropout_gain, dropout_keep, layernorm, layernorm_grads, matmul_int8, quantize_int8)
from tests.helpers import assert_close_rms, f32, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H = 2.0 ** -8   # half a bf16 step
# A row sum is off by at most 72 u of its terms' magnitudes (u = 2^-24: chains of
# 32, then 40 in the tree), so a mean by 2^-17.8 of their mean, which is below 1
# here; the few float32 roundings of a formula add u each.
E = 2.0 ** -16


def near(got, ref, name, extra=0.0):
    err = np.abs(f64(got) - ref)
    bound = H * np.abs(ref) + E * (1 + np.abs(ref)) + extra
    assert (err <= bound).all(), f"{name}: {err.max():.3e}"


def step(case, Wp, w1, b1, w2, b2, R, G, ws, wn, p, seed):
    """Forward and backward of the sub-layer; everything it computes."""
    X, A, B = case
    H1, m1, r1 = q.qlora_layernorm_fwd(X, w1, b1)
    L, T = q.qlora_linear_fwd_dropout(H1, Wp, A, B, 0.25, p, seed, 0, workspace=ws)
    Y, Z, m2, r2 = q.qlora_dropout_add_layernorm_fwd(L, R, p, seed, 1 << 20, w2, b2)
    dL, dR, dw2, db2 = q.qlora_dropout_add_layernorm_bwd(G, None, Z, m2, r2, p, seed, 1 << 20, w2, workspace=wn)
    dH1, dA, dB = q.qlora_linear_bwd_dropout(dL, H1, T, Wp, A, B, 0.25, p, seed, 0, workspace=ws)
    dX, dw1, db1 = q.qlora_layernorm_bwd(dH1, X, m1, r1, w1, workspace=wn)
    return H1, L, T, Y, Z, dL, dR, dw2, db2, dH1, dA, dB, dX, dw1, db1, m1, r1, m2, r2


def inputs(M=200, K=512, N=512, r=16):
    case = synthetic.linear_case(M, K, N, r, 0.25, seed=17)
    g = torch.Generator().manual_seed(3)
    vec = lambda n, m: (m + 0.2 * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)  # noqa: E731
    R = torch.randn(M, N, generator=g).to(torch.bfloat16).to(DEV)
    G = torch.randn(M, N, generator=g).to(torch.bfloat16).to(DEV)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    return (tuple(t.to(DEV) for t in (case.X, case.A, case.B)), Wp, vec(K, 1), vec(K, 0), vec(N, 1), vec(N, 0), R, G,
            q.new_dropout_workspace(M, K, N, r, DEV), q.new_layernorm_workspace(M, max(K, N), DEV))


def test_fine_tuning_step():
    args, p, seed = inputs(), 0.1, 99
    (X, A, B), Wp, w1, b1, w2, b2, R, G, ws, wn = args
    (H1, L, T, Y, Z, dL, dR, dw2, db2, dH1, dA, dB, dX, dw1, db1, m1, r1, m2, r2) = step(*args, p, seed)
    assert q.qlora_check_status(ws) == 0 and q.qlora_check_status(wn) == 0
    W = f64(q.qlora_dequantize_nf4(Wp))
    near(H1, layernorm(f64(X), f64(w1), f64(b1))[0], "first norm")
    h, a, b = f64(H1), f64(A), f64(B)
    hd = dropout(h, p, seed)
    assert_close_rms(f64(T), 0.25 * hd @ a, "T")
    assert_close_rms(f64(L), h @ W.T + 0.25 * hd @ a @ b, "linear")
    near(Z, dropout(f64(L), p, seed, 1 << 20, f64(R)), "residual sum")
    near(Y, layernorm(f64(Z), f64(w2), f64(b2))[0], "second norm")
    dz, ew2, eb2 = layernorm_grads(f64(G), f64(Z), f64(m2), f64(r2), f64(w2))
    near(dR, dz, "dresidual")
    near(dL, dropout(dz, p, seed, 1 << 20), "dlinear")
    assert_close_rms(f64(dw2), ew2, "dweight 2", 1e-5)
    assert_close_rms(f64(db2), eb2, "dbias 2", 1e-5)
    d, U = f64(dL), 0.25 * f64(dL) @ b.T
    keep = dropout_keep(*h.shape, p, seed)
    assert_close_rms(f64(dH1), d @ W + np.where(keep, dropout_gain(p) * (U @ a.T), 0), "dX of the linear")
    assert_close_rms(f64(dA), hd.T @ U, "dA")
    assert_close_rms(f64(dB), f64(T).T @ d, "dB")
    dx, ew1, eb1 = layernorm_grads(f64(dH1), f64(X), f64(m1), f64(r1), f64(w1))
    near(dX, dx, "dX", E * np.abs(dx).max())
    assert_close_rms(f64(dw1), ew1, "dweight 1", 1e-5)
    assert_close_rms(f64(db1), eb1, "dbias 1", 1e-5)


def test_step_in_a_graph_and_on_two_streams():
    """The same bits from a replayed graph, and from two streams at once with a
    workspace each."""
    args = inputs()
    ref = step(*args, 0.1, 99)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(*args, 0.1, 99)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, ref))
    other = list(args)
    other[8], other[9] = q.new_dropout_workspace(200, 512, 512, 16, DEV), q.new_layernorm_workspace(200, 512, DEV)
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for k, a in enumerate((args, other)):
            with torch.cuda.stream(streams[k]):
                got[k] = step(*a, 0.1, 99)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_serving_step(M):
    """Norm and 8-bit linear of a decode or prompt step, eager, captured and on
    two streams at once."""
    K, N = 2048, 1500
    g = torch.Generator().manual_seed(M)
    X = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).to(DEV)
    Wf = (0.02 * torch.randn(N, K, generator=g)).to(torch.bfloat16)
    W = q.qlora_quantize_int8(Wf.to(DEV))
    ws = [q.new_int8_workspace(M, K, N, DEV) for _ in range(2)]

    def run(k=0):
        Hn, _, _ = q.qlora_layernorm_fwd(X, w)
        return Hn, q.qlora_linear_int8_fwd(Hn, W, workspace=ws[k])

    Hn, Y = run()
    near(Hn, layernorm(f64(X), f64(w))[0], "norm")
    (xq, sx), (wq, sw) = quantize_int8(f32(Hn)), quantize_int8(f32(Wf))
    near(Y, matmul_int8(xq, sx, wq, sw), "Y")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured[1], Y)
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = run(k)[1]
    torch.cuda.synchronize()
    assert torch.equal(got[0], Y) and torch.equal(got[1], Y)
    assert q.qlora_check_status(ws[0]) == 0 and q.qlora_check_status(ws[1]) == 0
