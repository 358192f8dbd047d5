"""Dropout and layer norm on the GPU against the float64 oracle.

Tolerances are derived, not fitted.  u = 2^-24 is half a step of float32 and
eps/2 = torch.finfo(t).eps / 2 half a step of the output's type t, the one
rounding an output takes.  A sum of n terms that a thread adds in a chain of c
and the block then combines in a tree of depth d is off by at most
(c + d) u * sum|terms| to first order; c is at most 32 for rows held in
registers (32 columns per thread) and 8 * ceil(cols / 8192) for longer ones, d
at most 5 shuffles + 32 partial sums, so L = max(32, c) + 40 covers every row
sum.  The bounds below count those and the few roundings of each formula; a
factor of 1.01 covers the second-order terms."""

import math

import numpy as np
import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from oracle import dropout, dropout_keep, layernorm, layernorm_grads
from tests.helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# smallest step of a type: half of it bounds the rounding of subnormal values
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def out_err(ref, err, dtype):
    """Bound of a float32 result that is off by at most err, rounded once."""
    half = torch.finfo(dtype).eps / 2
    if dtype == torch.float32:
        return 1.01 * err + TINY[dtype]  # its last rounding is counted in err
    return 1.01 * (err + half * (np.abs(ref) + err)) + TINY[dtype]


def check(got, ref, bound, name):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][:3]} for {ref[bad][:3]}, bound {np.broadcast_to(bound, ref.shape)[bad][:3]}")


def rand(rows, cols, dtype, seed, mean=0.0, std=1.0, pad=0):
    """[rows, cols] values; pad > 0 shifts the start off its 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows * cols, generator=g) * std + mean).to(dtype)
    buf = torch.empty(rows * cols + pad, dtype=dtype, device=DEV)
    buf[pad:] = x.to(DEV)
    return buf[pad:].view(rows, cols)


def chain(cols):
    return max(32, 8 * math.ceil(cols / 8192)) + 40


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 8, 0), (3, 7, 0), (5, 256, 0), (16, 257, 1), (37, 1001, 0),
                                           (4, 4096, 3), (300, 8192, 0), (700, 4104, 0)])
@pytest.mark.parametrize("p,res", [(0.1, True), (0.6, False)])
def test_dropout(dtype, rows, cols, pad, p, res):
    t = TYPES[dtype]
    X, R = rand(rows, cols, t, 1, pad=pad), (rand(rows, cols, t, 2, pad=pad) if res else None)
    seed, offset = 0xDEADBEEF12345678, (1 << 32) - 5
    Y = q.qlora_dropout_fwd(X, p, seed, offset, residual=R)
    ref = dropout(f64(X), p, seed, offset, None if R is None else f64(R))
    # the gain is rounded once, the product and sum are one fused operation
    prod = np.abs(dropout(f64(X), p, seed, offset))
    check(Y, ref, out_err(ref, 2 * U * prod + U * np.abs(ref), t), "Y")
    dX = q.qlora_dropout_bwd(X, p, seed, offset)
    ref = dropout(f64(X), p, seed, offset)
    check(dX, ref, out_err(ref, 2 * U * np.abs(ref), t), "dX")
    np.testing.assert_array_equal(f64(dX)[~dropout_keep(rows, cols, p, seed, offset)], 0.0)


def test_dropout_drops_infinities_and_nan():
    X = torch.full((64, 96), float("inf"), device=DEV, dtype=torch.bfloat16)
    X[::2] = float("nan")
    R = torch.ones_like(X)
    keep = dropout_keep(64, 96, 0.5, 11)
    got = f64(q.qlora_dropout_fwd(X, 0.5, 11, residual=R))
    assert (got[~keep] == 1.0).all()
    assert np.isnan(got[0::2][keep[0::2]]).all() and np.isinf(got[1::2][keep[1::2]]).all()
    assert (f64(q.qlora_dropout_fwd(X, 1.0, 11, residual=R)) == 1.0).all()


def test_dropout_ends_and_shapes():
    X = rand(6, 40, torch.bfloat16, 3).view(2, 3, 40)
    assert torch.equal(q.qlora_dropout_fwd(X, 0.0, 5), X)
    assert not q.qlora_dropout_fwd(X, 1.0, 5).any()
    # leading dimensions are rows; each row starts a new counter
    whole = q.qlora_dropout_fwd(X, 0.4, 5, 100)
    assert torch.equal(whole[1], q.qlora_dropout_fwd(X[1], 0.4, 5, 100 + 3 * 5))
    # the counter wraps modulo 2^64
    top = (1 << 64) - 3
    got = q.qlora_dropout_fwd(torch.ones(1, 64, device=DEV), 0.5, 9, top) != 0
    np.testing.assert_array_equal(got.cpu().numpy(), dropout_keep(1, 64, 0.5, 9, top))


def test_dropout_replayed_graph_draws_anew():
    X = torch.ones(33, 100, device=DEV)
    at = torch.zeros(1, dtype=torch.int64, device=DEV)
    Y = torch.empty_like(X)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q.qlora_dropout_fwd(X, 0.3, 4, 7, Y=Y, offset_dev=at)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlora_dropout_fwd(X, 0.3, 4, 7, Y=Y, offset_dev=at)
    for n in (0, 1000, (1 << 40) + 1):
        at.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal((Y != 0).cpu().numpy(), dropout_keep(33, 100, 0.3, 4, 7 + n))


# ------------------------------------------------------------------ layer norm
def fwd_bounds(x, w, b, y, mean, rstd, dtype, cols):
    """(bound of Y, of mean, of rstd): the mean is off by L u mean|x|, each
    distance from it by that and one rounding, the variance by (L + 3) u of
    itself and by the mean's error squared, and rstd by half of the variance's
    error plus sqrt, division and the sum with eps (2 u each)."""
    L = chain(cols)
    ax = np.abs(x).mean(1)
    em = (L + 2) * U * ax
    rel = ((L + 5) / 2 + 6) * U + (em * rstd) ** 2
    hat = np.abs(x - mean[:, None]) * rstd[:, None]
    w = np.ones(cols) if w is None else np.abs(w)
    b = np.zeros(cols) if b is None else np.abs(b)
    eh = em[:, None] * rstd[:, None] + hat * (rel[:, None] + 2 * U)
    ey = eh * w + U * (hat * w + np.abs(y)) + U * b
    return out_err(y, ey, dtype), 1.01 * em + 1e-40, 1.01 * rel * rstd


FWD = [(1, 1), (3, 8), (5, 31), (2, 256), (9, 257), (300, 250), (40, 1000), (301, 1024), (300, 2048), (299, 768), (7, 2304),
       (310, 6400), (1, 4096),
       (300, 4096), (37, 5003), (1, 8192), (310, 8192), (300, 11008), (4, 22016), (300, 32768), (3, 32776),
       (2, 40001)]


@pytest.mark.parametrize("rows,cols", FWD)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                          ("fp32", "fp32")])
def test_layernorm_forward(rows, cols, dtype, wdtype):
    t = TYPES[dtype]
    X = rand(rows, cols, t, rows + cols, mean=0.3, std=2.0)
    w = rand(1, cols, TYPES[wdtype], 5, mean=1.0, std=0.3).view(-1)
    b = rand(1, cols, TYPES[wdtype], 6, std=0.3).view(-1)
    Y, mean, rstd = q.qlora_layernorm_fwd(X, w, b, 1e-5)
    y, m, r = layernorm(f64(X), f64(w), f64(b), 1e-5)
    by, bm, br = fwd_bounds(f64(X), f64(w), f64(b), y, m, r, t, cols)
    check(mean, m, bm, "mean")
    check(rstd, r, br, "rstd")
    check(Y, y, by, "Y")


@pytest.mark.parametrize("rows,cols,pad", [(7, 512, 1), (7, 513, 0), (2, 33000, 3)])
def test_layernorm_forward_without_parameters_and_unaligned(rows, cols, pad):
    X = rand(rows, cols, torch.bfloat16, 9, mean=-4.0, pad=pad)
    for w, b in ((None, None), (rand(1, cols, torch.bfloat16, 5).view(-1), None),
                 (None, rand(1, cols, torch.float32, 6).view(-1))):
        Y, mean, rstd = q.qlora_layernorm_fwd(X, w, b, 1e-3)
        w64, b64 = (None if v is None else f64(v) for v in (w, b))
        y, m, r = layernorm(f64(X), w64, b64, 1e-3)
        by, bm, br = fwd_bounds(f64(X), w64, b64, y, m, r, torch.bfloat16, cols)
        check(mean, m, bm, "mean")
        check(rstd, r, br, "rstd")
        check(Y, y, by, "Y")


def test_layernorm_far_from_zero():
    """A mean 1e4 times the spread: the squared distances are taken from the
    mean, so the variance keeps its digits."""
    X = rand(64, 4096, torch.float32, 1, mean=1e4, std=1.0)
    Y, mean, rstd = q.qlora_layernorm_fwd(X, eps=0.0)
    y, m, r = layernorm(f64(X), eps=0.0)
    by, bm, br = fwd_bounds(f64(X), None, None, y, m, r, torch.float32, 4096)
    check(mean, m, bm, "mean")
    check(rstd, r, br, "rstd")
    check(Y, y, by, "Y")


def test_layernorm_keeps_rows_apart():
    X = rand(40, 1000, torch.bfloat16, 2)
    clean = [v.clone() for v in q.qlora_layernorm_fwd(X)]
    X[7, 3] = float("nan")
    X[9, 999] = float("inf")
    X[11] = 0.5  # constant: variance 0
    Y, mean, rstd = q.qlora_layernorm_fwd(X)
    assert Y[7].isnan().all() and mean[9].isinf()
    assert not Y[11].any()
    flat = 1 / math.sqrt(float(np.float32(1e-5)))  # a root and a division, one rounding each
    assert abs(float(rstd[11]) - flat) <= 2.02 * U * flat
    rest = [i for i in range(40) if i not in (7, 9, 11)]
    for got, ref in zip((Y, mean, rstd), clean):
        assert torch.equal(got[rest], ref[rest])


def bwd_bounds(dy, x, mean, rstd, w, dx, rows, cols, dtype, extra=None):
    """h takes two roundings, g one; each row sum (L + 2) u of its terms; then
    three products, two sums and the one with dZ.  A column's sum runs over a
    chain of at most the rows of a block's slot, 16 slots and the blocks'
    partial sums (8 chains of at most 20, then 8)."""
    L = chain(cols) + 4
    h = np.abs(x - mean[:, None]) * rstd[:, None]
    g = np.abs(dy) if w is None else np.abs(dy * w)
    s1, s2 = g.mean(1)[:, None], (g * h).mean(1)[:, None]
    e = rstd[:, None] * U * (4 * g + (L + 4) * s1 + (L + 12) * h * s2) + 2 * U * np.abs(dx)
    if extra is not None:
        e = e + U * np.abs(extra)
    slots = max(1, 16 // max(1, 2 ** math.ceil(math.log2(max(1, cols / 512)))))
    length = math.ceil(rows / (slots * min(64, math.ceil(rows / slots)))) + 16 + 20 + 8 + 5
    return out_err(dx, e, dtype), 1.01 * length * U * (np.abs(dy) * h).sum(0), 1.01 * length * U * np.abs(dy).sum(0)


BWD = [(1, 1), (3, 8), (17, 31), (16, 256), (50, 257), (700, 250), (40, 1000), (2500, 1024), (333, 4096), (1, 8192),
       (60, 768), (33, 2304), (9, 2560), (20, 6400), (777, 5003), (700, 8192), (5, 8200),
       (130, 11008), (3, 22016), (2, 40001)]


@pytest.mark.parametrize("rows,cols", BWD)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp32"), ("fp16", "fp16"),
                                          ("fp32", "fp32")])
def test_layernorm_backward(rows, cols, dtype, wdtype):
    t = TYPES[dtype]
    X, dY = rand(rows, cols, t, rows, mean=0.3, std=2.0), rand(rows, cols, t, cols)
    w = rand(1, cols, TYPES[wdtype], 5, mean=1.0, std=0.3).view(-1)
    _, mean, rstd = q.qlora_layernorm_fwd(X, w)
    ws = q.new_layernorm_workspace(rows, cols, DEV)
    ws[256:].fill_(255)  # NaN: everything past the status word is written before it is read
    got = q.qlora_layernorm_bwd(dY, X, mean, rstd, w, workspace=ws)
    assert q.qlora_check_status(ws) == 0
    x, dy, m, r, wv = f64(X), f64(dY), f64(mean), f64(rstd), f64(w)
    refs = layernorm_grads(dy, x, m, r, wv)
    for name, a, ref, bound in zip(("dX", "dweight", "dbias"), got, refs,
                                   bwd_bounds(dy, x, m, r, wv, refs[0], rows, cols, t)):
        check(a, ref, bound, name)
    again = q.qlora_layernorm_bwd(dY, X, mean, rstd, w, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_layernorm_backward_variants():
    X, dY = rand(90, 768, torch.bfloat16, 1, pad=1), rand(90, 768, torch.bfloat16, 2)
    _, mean, rstd = q.qlora_layernorm_fwd(X)
    x, dy, m, r = f64(X), f64(dY), f64(mean), f64(rstd)
    dX, dw, db = q.qlora_layernorm_bwd(dY, X, mean, rstd)
    refs = layernorm_grads(dy, x, m, r)
    for a, ref, bound in zip((dX, dw, db), refs, bwd_bounds(dy, x, m, r, None, refs[0], 90, 768, torch.bfloat16)):
        check(a, ref, bound, "grad")
    only, none_w, none_b = q.qlora_layernorm_bwd(dY, X, mean, rstd, param_grads=False)
    assert none_w is None and none_b is None and torch.equal(only, dX)
    given = torch.full((768,), 7.0, device=DEV)
    _, dw1, db1 = q.qlora_layernorm_bwd(dY, X, mean, rstd, dweight=given, param_grads=False)
    assert dw1 is given and db1 is None and torch.equal(dw1, dw)


# ------------------------------------------------------------------ fused with the residual dropout
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (16, 256), (50, 257), (40, 1000), (333, 4096), (1, 8192),
                                       (370, 5003), (400, 8192), (5, 8200), (2, 33001)])
@pytest.mark.parametrize("dtype,wdtype,p", [("bf16", "fp32", 0.1), ("fp16", "fp16", 0.5), ("fp32", "fp32", 0.25),
                                            ("bf16", "bf16", 0.0)])
def test_dropout_add_layernorm(rows, cols, dtype, wdtype, p):
    t = TYPES[dtype]
    X, R = rand(rows, cols, t, 1, std=2.0), rand(rows, cols, t, 2, mean=0.3)
    dY, dZ = rand(rows, cols, t, 3), rand(rows, cols, t, 4)
    w = rand(1, cols, TYPES[wdtype], 5, mean=1.0, std=0.3).view(-1)
    b = rand(1, cols, TYPES[wdtype], 6, std=0.3).view(-1)
    seed, offset = 77, 1 << 33
    Y, Z, mean, rstd = q.qlora_dropout_add_layernorm_fwd(X, R, p, seed, offset, w, b)
    # the sum is the one that the dropout alone stores, the norm the norm alone of it
    assert torch.equal(Z, q.qlora_dropout_fwd(X, p, seed, offset, residual=R))
    for got, ref in zip((Y, mean, rstd), q.qlora_layernorm_fwd(Z, w, b)):
        assert torch.equal(got, ref)
    y, m, r = layernorm(f64(Z), f64(w), f64(b))
    by, bm, br = fwd_bounds(f64(Z), f64(w), f64(b), y, m, r, t, cols)
    check(mean, m, bm, "mean")
    check(rstd, r, br, "rstd")
    check(Y, y, by, "Y")
    ws = q.new_layernorm_workspace(rows, cols, DEV)
    for dz in (dZ, None):
        dX, dR, dw, db = q.qlora_dropout_add_layernorm_bwd(dY, dz, Z, mean, rstd, p, seed, offset, w, workspace=ws)
        assert q.qlora_check_status(ws) == 0
        z, dy, mm, rr, wv = f64(Z), f64(dY), f64(mean), f64(rstd), f64(w)
        dx, ew, eb = layernorm_grads(dy, z, mm, rr, wv)
        extra = 0.0 if dz is None else f64(dz)
        total = dx + extra
        norm_err, bw, bb = bwd_bounds(dy, z, mm, rr, wv, dx, rows, cols, torch.float32)
        err = norm_err + U * (np.abs(total) + norm_err)
        check(dR, total, out_err(total, err, t), "dresidual")
        dropped = dropout(total, p, seed, offset)
        gain = 65536 / (65536 - round(65536 * p))
        check(dX, dropped, out_err(dropped, gain * err + 2 * U * np.abs(dropped), t), "dX")
        assert not f64(dX)[~dropout_keep(rows, cols, p, seed, offset)].any()
        check(dw, ew, bw, "dweight")
        check(db, eb, bb, "dbias")


def test_gradient_against_differences():
    """The fused block's gradient of sum(Y * G) + sum(Z * H) along a random
    direction, against a difference of the float64 oracle's forward."""
    rows, cols, p, seed = 6, 96, 0.3, 5
    X, R, G, H, D = (rand(rows, cols, torch.float32, k) for k in range(5))
    w, b = rand(1, cols, torch.float32, 9, mean=1.0).view(-1), rand(1, cols, torch.float32, 8).view(-1)
    Y, Z, mean, rstd = q.qlora_dropout_add_layernorm_fwd(X, R, p, seed, 0, w, b)
    dX, dR, dw, db = q.qlora_dropout_add_layernorm_bwd(G, H, Z, mean, rstd, p, seed, 0, w)

    def loss(x, res, wv, bv):
        z = dropout(x, p, seed, 0, res)
        return float((layernorm(z, wv, bv)[0] * f64(G)).sum() + (z * f64(H)).sum())

    h, d = 1e-5, f64(D)
    base = [f64(v) for v in (X, R, w, b)]
    for k, grad, direction in ((0, dX, d), (1, dR, d), (2, dw, d[0]), (3, db, d[0])):
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + h * direction, base[k] - h * direction
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = float((f64(grad) * direction).sum())
        # the difference's own error is O(h^2) + O(2^-53 / h): below 1e-6 here
        assert abs(got - diff) <= 1e-5 * float(np.abs(f64(grad) * direction).sum()) + 1e-6


# ------------------------------------------------------------------ streams and graphs
def test_norm_on_a_side_stream_and_in_a_graph():
    X, dY = rand(300, 2048, torch.bfloat16, 1), rand(300, 2048, torch.bfloat16, 2)
    w = rand(1, 2048, torch.bfloat16, 3).view(-1)
    ref = q.qlora_layernorm_fwd(X, w)
    ref_b = q.qlora_layernorm_bwd(dY, X, ref[1], ref[2], w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = q.new_layernorm_workspace(300, 2048, DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = q.qlora_layernorm_fwd(X, w)
        got_b = q.qlora_layernorm_bwd(dY, X, got[1], got[2], w, workspace=ws)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + got_b, ref + ref_b))
    Y, mean, rstd = (torch.empty_like(v) for v in ref)
    dX, dw, db = (torch.empty_like(v) for v in ref_b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlora_layernorm_fwd(X, w, Y=Y, mean=mean, rstd=rstd)
        q.qlora_layernorm_bwd(dY, X, mean, rstd, w, workspace=ws, dX=dX, dweight=dw, dbias=db)
    X.copy_(rand(300, 2048, torch.bfloat16, 7))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    ref = q.qlora_layernorm_fwd(X, w)
    ref_b = q.qlora_layernorm_bwd(dY, X, ref[1], ref[2], w)
    assert all(torch.equal(a, b) for a, b in zip((Y, mean, rstd, dX, dw, db), ref + ref_b))


@pytest.mark.parametrize("rows,cols,pad", [(12000, 1000, 1), (6000, 2047, 5), (2000, 5003, 3), (12000, 520, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layernorm_backward_past_the_ring_unaligned(rows, cols, pad, dtype):
    """Tensors that start off a 16-byte boundary, with rows enough for every
    stage of the ring to be filled many times: the first stage once holds
    elements that ordinary stores put there."""
    t = TYPES[dtype]
    X, dY = rand(rows, cols, t, 1, mean=0.3, std=2.0, pad=pad), rand(rows, cols, t, 2, pad=pad)
    _, mean, rstd = q.qlora_layernorm_fwd(X)
    got = q.qlora_layernorm_bwd(dY, X, mean, rstd)
    x, dy, m, r = f64(X), f64(dY), f64(mean), f64(rstd)
    refs = layernorm_grads(dy, x, m, r)
    for name, a, ref, bound in zip(("dX", "dweight", "dbias"), got, refs,
                                   bwd_bounds(dy, x, m, r, None, refs[0], rows, cols, t)):
        check(a, ref, bound, name)
    assert all(torch.equal(a, b) for a, b in zip(got, q.qlora_layernorm_bwd(dY, X, mean, rstd)))


# ------------------------------------------------------------------ the plans of ordinary training calls
# Two rows per warp and step, one to sixteen row slots per block, rings that wrap.
@pytest.mark.parametrize("rows,cols,dtype", [(2500, 4096, "bf16"), (4096, 2048, "fp16"), (6000, 1024, "bf16"),
                                             (1500, 5120, "fp16"), (20000, 250, "bf16"), (12000, 257, "fp32")])
def test_layernorm_backward_of_many_rows(rows, cols, dtype):
    t = TYPES[dtype]
    X, dY = rand(rows, cols, t, 1, mean=0.3, std=2.0), rand(rows, cols, t, 2)
    w = rand(1, cols, torch.float32, 5, mean=1.0, std=0.3).view(-1)
    _, mean, rstd = q.qlora_layernorm_fwd(X, w)
    ws = q.new_layernorm_workspace(rows, cols, DEV)
    got = q.qlora_layernorm_bwd(dY, X, mean, rstd, w, workspace=ws)
    assert q.qlora_check_status(ws) == 0
    x, dy, m, r, wv = f64(X), f64(dY), f64(mean), f64(rstd), f64(w)
    refs = layernorm_grads(dy, x, m, r, wv)
    for name, a, ref, bound in zip(("dX", "dweight", "dbias"), got, refs,
                                   bwd_bounds(dy, x, m, r, wv, refs[0], rows, cols, t)):
        check(a, ref, bound, name)


@pytest.mark.parametrize("rows,cols,dtype", [(1500, 5120, "bf16"), (2500, 2560, "fp16"), (2500, 4096, "bf16"),
                                             (6000, 1000, "bf16"), (20000, 250, "fp16")])
@pytest.mark.parametrize("with_dz", [True, False])
def test_fused_backward_of_many_rows(rows, cols, dtype, with_dz):
    t, p, seed, offset = TYPES[dtype], 0.2, 77, 1 << 33
    Z, dY = rand(rows, cols, t, 1, mean=0.3, std=2.0), rand(rows, cols, t, 3)
    dZ = rand(rows, cols, t, 4) if with_dz else None
    w = rand(1, cols, t, 5, mean=1.0, std=0.3).view(-1)
    _, mean, rstd = q.qlora_layernorm_fwd(Z, w)
    dX, dR, dw, db = q.qlora_dropout_add_layernorm_bwd(dY, dZ, Z, mean, rstd, p, seed, offset, w)
    z, dy, m, r, wv = f64(Z), f64(dY), f64(mean), f64(rstd), f64(w)
    dx, ew, eb = layernorm_grads(dy, z, m, r, wv)
    total = dx if dZ is None else dx + f64(dZ)
    norm_err, bw, bb = bwd_bounds(dy, z, m, r, wv, dx, rows, cols, torch.float32)
    err = norm_err + U * (np.abs(total) + norm_err)
    check(dR, total, out_err(total, err, t), "dresidual")
    dropped = dropout(total, p, seed, offset)
    gain = 65536 / (65536 - round(65536 * p))
    check(dX, dropped, out_err(dropped, gain * err + 2 * U * np.abs(dropped), t), "dX")
    check(dw, ew, bw, "dweight")
    check(db, eb, bb, "dbias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,res", [(620, 8192, True), (620, 8192, False), (4877, 1000, True)])
def test_dropout_of_many_groups(dtype, rows, cols, res):
    """Sizes that take four groups of eight per thread, the last block in part."""
    t = TYPES[dtype]
    X, R = rand(rows, cols, t, 1), (rand(rows, cols, t, 2) if res else None)
    Y = q.qlora_dropout_fwd(X, 0.3, 5, 9, residual=R)
    ref = dropout(f64(X), 0.3, 5, 9, None if R is None else f64(R))
    prod = np.abs(dropout(f64(X), 0.3, 5, 9))
    check(Y, ref, out_err(ref, 2 * U * prod + U * np.abs(ref), t), "Y")
