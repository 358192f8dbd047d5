"""The linear with dropout on the adapter's inputs against the float64 oracle.

Bounds, to first order, with u = 2^-24 and h = 2^-8 (half a bf16 step):
a tensor-core sum of n products in float32 adds 16 of them per step and may
truncate at each, so it is off by at most (n / 8 + 8) 2^-23 sum|products|;
the rank-r intermediates enter later products as bf16 pairs, off by h^2 of
their size; Y is rounded once, dX twice."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_quantize_b200 as q
from bit_quantized_lora_quantize_b200 import synthetic
from oracle import dropout, dropout_gain, dropout_keep
from tests.helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, H = 2.0 ** -24, 2.0 ** -8


def acc(n, total):
    return (n / 8 + 8) * 2 * U * total


def check(got, ref, bound, name):
    bad = ~(np.abs(f64(got) - ref) <= 1.01 * bound + 1e-37)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, e.g. {f64(got)[bad][:3]} for {ref[bad][:3]}, "
                           f"bound {bound[bad][:3]}")


def reference(X, dY, Wd, A, B, T_save, s, p, seed, offset):
    """{name: (value, bound)} for the definition's five outputs."""
    M, K = X.shape
    N, r = Wd.shape[0], A.shape[1]
    keep, gain = dropout_keep(M, K, p, seed, offset), dropout_gain(p)
    xd = dropout(X, p, seed, offset)
    a = np.abs
    T = s * xd @ A
    eT = acc(K, abs(s) * (a(xd) @ a(A))) + 4 * U * a(T)
    Y = X @ Wd.T + T @ B
    eY = acc(K + 2 * r, a(X) @ a(Wd.T) + a(T) @ a(B)) + (eT + H * H * a(T)) @ a(B)
    Um = s * dY @ B.T
    eU = acc(N, abs(s) * (a(dY) @ a(B.T))) + 4 * U * a(Um)
    base = dY @ Wd
    eb = acc(N, a(dY) @ a(Wd))
    add = np.where(keep, gain * (Um @ A.T), 0.0)
    ea = gain * ((eU + H * H * a(Um)) @ a(A.T) + acc(2 * r, a(Um) @ a(A.T))) + 4 * U * a(add)
    dX = base + add
    eX = eb + ea + H * (a(base) + eb)
    dA = xd.T @ Um
    eA = a(xd.T) @ (eU + H * H * a(Um)) + acc(2 * M, a(xd.T) @ a(Um)) + 4 * U * a(dA)
    dB = T_save.T @ dY
    eB = H * H * a(T_save.T) @ a(dY) + acc(2 * M, a(T_save.T) @ a(dY))
    return {"Y": (Y, eY + H * (a(Y) + eY)), "T": (T, eT), "dX": (dX, eX + H * (a(dX) + eX)), "dA": (dA, eA),
            "dB": (dB, eB)}


def run(case, p, seed, offset, code="nf4", dq="linear8"):
    Wp = q.qlora_quantize_nf4(case.W.to(DEV), code=code, dq=dq)
    X, A, B, dY = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    ws = q.new_dropout_workspace(case.M, case.K, case.N, case.r, DEV)
    Y, T = q.qlora_linear_fwd_dropout(X, Wp, A, B, case.scale, p, seed, offset, workspace=ws)
    dX, dA, dB = q.qlora_linear_bwd_dropout(dY, X, T, Wp, A, B, case.scale, p, seed, offset, workspace=ws)
    assert q.qlora_check_status(ws) == 0
    Wd = f64(q.qlora_dequantize_nf4(Wp))  # bit-exact against its own oracle elsewhere
    ref = reference(f64(X), f64(dY), Wd, f64(A), f64(B), f64(T), case.scale, p, seed, offset)
    got = {"Y": Y, "T": T, "dX": dX, "dA": dA, "dB": dB}
    for name, (value, bound) in ref.items():
        check(got[name], value, bound, name)
    return got


@pytest.mark.parametrize("M,K,N,r", [(1, 64, 8, 1), (16, 256, 256, 8), (129, 320, 264, 12), (200, 64, 16, 64),
                                     (700, 576, 520, 72), (77, 1024, 1000, 130), (1100, 1984, 136, 16)])
@pytest.mark.parametrize("p", [0.1, 0.55])
def test_against_oracle(M, K, N, r, p):
    run(synthetic.linear_case(M, K, N, r, 0.5, seed=M + K + N + r), p, 0xABCDEF0123456789, (1 << 34) + 3)


@pytest.mark.parametrize("code,dq", [("fp4", "linear8"), ("int4", "linear8"), ("nf4", "centred_fp8")])
def test_every_code(code, dq):
    run(synthetic.linear_case(150, 256, 264, 8, 2.0, seed=3), 0.2, 5, 0, code, dq)


def test_without_dropout_equals_the_plain_calls():
    """p = 0 runs the same GEMMs on the same values: Y, T, dA and dB bit for
    bit; dX takes one more rounding."""
    case = synthetic.linear_case(300, 512, 520, 64, 0.25, seed=1)
    got = run(case, 0.0, 9, 0)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    X, A, B, dY = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    Y, T = q.qlora_linear_fwd(X, Wp, A, B, case.scale)
    dX, dA, dB = q.qlora_linear_bwd(dY, X, T, Wp, A, B, case.scale)
    for name, ref in (("Y", Y), ("T", T), ("dA", dA), ("dB", dB)):
        assert torch.equal(got[name], ref), name


def test_all_dropped_leaves_the_frozen_layer():
    case = synthetic.linear_case(140, 256, 264, 16, 0.25, seed=2)
    got = run(case, 1.0, 9, 0)
    assert not got["T"].any() and not got["dA"].any() and not got["dB"].any()


def test_infinite_inputs_that_are_dropped_leave_the_adapter_alone():
    """T and dA see the dropped inputs only; Y reads X itself."""
    M, K, p, seed = 160, 128, 0.5, 21
    case = synthetic.linear_case(M, K, 64, 8, 1.0, seed=4)
    keep = dropout_keep(M, K, p, seed)
    X = case.X.clone()
    X[5, np.flatnonzero(~keep[5])[0]] = float("inf")
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    A, B, dY = (t.to(DEV) for t in (case.A, case.B, case.dY))
    Y, T = q.qlora_linear_fwd_dropout(X.to(DEV), Wp, A, B, 1.0, p, seed)
    dX, dA, dB = q.qlora_linear_bwd_dropout(dY, X.to(DEV), T, Wp, A, B, 1.0, p, seed)
    assert torch.isfinite(T).all() and torch.isfinite(dA).all() and not torch.isfinite(Y[5]).all()
    assert torch.isfinite(Y[torch.arange(M) != 5]).all()


def test_captured_step_replays_with_new_draws():
    case = synthetic.linear_case(140, 256, 264, 16, 0.25, seed=6)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    X, A, B, dY = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    ws = q.new_dropout_workspace(case.M, case.K, case.N, case.r, DEV)
    at = torch.zeros(1, dtype=torch.int64, device=DEV)

    def step(**kw):
        Y, T = q.qlora_linear_fwd_dropout(X, Wp, A, B, 0.25, 0.3, 8, workspace=ws, **kw)
        return (Y, T, *q.qlora_linear_bwd_dropout(dY, X, T, Wp, A, B, 0.25, 0.3, 8, workspace=ws, **kw))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(offset_dev=at)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(offset_dev=at)
    for n in (0, 4480):
        at.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        ref = [q.qlora_linear_fwd_dropout(X, Wp, A, B, 0.25, 0.3, 8, n)[k] for k in (0, 1)]
        ref += q.qlora_linear_bwd_dropout(dY, X, ref[1], Wp, A, B, 0.25, 0.3, 8, n)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert q.qlora_check_status(ws) == 0


def test_gradients_against_differences():
    """Directional differences of sum(Y G) in float64 through the oracle's
    forward, for X, A and B."""
    M, K, N, r, s, p, seed = 12, 128, 64, 8, 1.0, 0.4, 3
    case = synthetic.linear_case(M, K, N, r, s, seed=8)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    X, A, B, G = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    _, T = q.qlora_linear_fwd_dropout(X, Wp, A, B, s, p, seed)
    grads = q.qlora_linear_bwd_dropout(G, X, T, Wp, A, B, s, p, seed)
    Wd = f64(q.qlora_dequantize_nf4(Wp))
    rng = np.random.default_rng(0)

    def loss(x, a, b):
        return float(((x @ Wd.T + s * dropout(x, p, seed) @ a @ b) * f64(G)).sum())

    base = [f64(v) for v in (X, A, B)]
    bounds = reference(*base[:1], f64(G), Wd, *base[1:], f64(T), s, p, seed, 0)
    for k, name in enumerate(("dX", "dA", "dB")):
        d = rng.normal(size=base[k].shape)
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + 1e-4 * d, base[k] - 1e-4 * d
        diff = (loss(*up) - loss(*down)) / 2e-4  # exact but for rounding: each argument enters linearly
        extra = float((np.abs(f64(T) - s * dropout(base[0], p, seed) @ base[1]).T @ np.abs(f64(G)) * np.abs(d)).sum()) \
            if name == "dB" else 0.0
        tol = 1.01 * float((bounds[name][1] * np.abs(d)).sum()) + extra + 1e-6 * abs(diff) + 1e-6
        assert abs(float((f64(grads[k]) * d).sum()) - diff) <= tol, name


@pytest.mark.parametrize("M,K,N,r,p", [(16, 256, 256, 8, 0.05), (150, 256, 264, 12, 0.1), (300, 512, 520, 64, 0.0),
                                       (700, 576, 136, 130, 0.5)])
def test_dx_is_rounded_once(M, K, N, r, p):
    """dX holds bf16 of one float32 sum: besides the float32 sums' own error
    (acc) it is within half a step, not a whole one."""
    case = synthetic.linear_case(M, K, N, r, 1.0, seed=M + r)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    X, A, B, dY = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    _, T = q.qlora_linear_fwd_dropout(X, Wp, A, B, 1.0, p, 77, 5)
    dX, _, _ = q.qlora_linear_bwd_dropout(dY, X, T, Wp, A, B, 1.0, p, 77, 5)
    a, dy, w, la, lb = np.abs, f64(dY), f64(q.qlora_dequantize_nf4(Wp)), f64(A), f64(B)
    u, gain = dy @ lb.T, dropout_gain(p)
    add = np.where(dropout_keep(M, K, p, 77, 5), gain * (u @ la.T), 0.0)
    ref = dy @ w + add
    eu = acc(N, a(dy) @ a(lb.T)) + (4 * U + H * H) * a(u)  # U's own sum, its scale and its bf16 pair
    err = acc(N, a(dy) @ a(w)) + gain * (eu @ a(la.T) + acc(2 * r, a(u) @ a(la.T))) + 4 * U * (a(add) + a(ref))
    check(dX, ref, err + H * (a(ref) + err), "dX")


@pytest.mark.parametrize("M,r", [(16, 8), (140, 13)])
def test_only_the_plain_part_of_the_workspace_needs_zeros(M, r):
    """Whatever lies behind the plain calls' bytes (NaN here) changes nothing."""
    case = synthetic.linear_case(M, 256, 264, r, 0.5, seed=5)
    Wp = q.qlora_quantize_nf4(case.W.to(DEV))
    X, A, B, dY = (t.to(DEV) for t in (case.X, case.A, case.B, case.dY))
    got = []
    for fill in (0, 255):
        ws = q.new_dropout_workspace(M, 256, 264, r, DEV)
        ws[q.qlora_workspace_bytes(M, 256, 264, r):].fill_(fill)
        Y, T = q.qlora_linear_fwd_dropout(X, Wp, A, B, 0.5, 0.2, 3, workspace=ws)
        got.append((Y, T, *q.qlora_linear_bwd_dropout(dY, X, T, Wp, A, B, 0.5, 0.2, 3, workspace=ws)))
        assert q.qlora_check_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
