"""Run one library call on a seeded synthetic case, a few times, for profiling.

    python -m bit_quantized_lora_quantize_b200.prof_case quantize --n 22016 --k 8192
    python -m bit_quantized_lora_quantize_b200.prof_case fwd --m 16 --n 8192 --k 8192
    python -m bit_quantized_lora_quantize_b200.prof_case bwd --m 4096 --n 4096 --k 4096
    python -m bit_quantized_lora_quantize_b200.prof_case adamw --n 9994240
    python -m bit_quantized_lora_quantize_b200.prof_case silu --m 8192 --n 11008
    python -m bit_quantized_lora_quantize_b200.prof_case dropout --m 8192 --n 11008
    python -m bit_quantized_lora_quantize_b200.prof_case norm-bwd --m 4096 --n 8192
    python -m bit_quantized_lora_quantize_b200.prof_case bwd-dropout --m 4096 --n 512 --k 8192
    python -m bit_quantized_lora_quantize_b200.prof_case int8 --m 1 --n 8192 --k 8192

Each case makes its inputs once, runs `--warmup` calls, then `--iters` calls
with a 256 MB buffer written between them (so the weight is read from HBM, not
from L2), and prints the mean device time per call measured with CUDA events.
A profiler attached to this process sees exactly the library's kernels plus
the flush writes.
"""

import argparse

import torch

from . import int8, rows, synthetic
from . import qlora as q


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("op", choices=["quantize", "dequantize", "fwd", "bwd", "adamw", "silu", "dropout", "norm-fwd",
                                   "norm-bwd", "block-fwd", "block-bwd", "fwd-dropout", "bwd-dropout", "int8"])
    ap.add_argument("--m", type=int, default=4096, help="tokens")
    ap.add_argument("--n", type=int, default=4096, help="weight rows (out features)")
    ap.add_argument("--k", type=int, default=4096, help="weight columns (in features)")
    ap.add_argument("--r", type=int, default=64)
    ap.add_argument("--scale", type=float, default=0.25)
    ap.add_argument("--p", type=float, default=0.1, help="dropout probability")
    ap.add_argument("--warmup", type=int, default=2)
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--seed", type=int, default=7)
    a = ap.parse_args(argv)

    dev = "cuda:0"
    torch.cuda.set_device(0)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    if a.op == "adamw":
        # a flat parameter vector of n (the block's adapters: 9994240)
        from . import paged
        opt = paged.PagedAdamW([(a.n, 0, 1)], dev, lr=2e-4, weight_decay=0.01)
        g = torch.randn(a.n, device=dev)
        call = lambda: opt.step(g)  # noqa: E731
    elif a.op == "silu":
        G = torch.randn(a.m, a.n, device=dev).to(torch.bfloat16)
        U = torch.randn(a.m, a.n, device=dev).to(torch.bfloat16)
        H = torch.empty_like(G)
        call = lambda: q.qlora_silu_gate_fwd(G, U, H)  # noqa: E731
    elif a.op in ("dropout", "norm-fwd", "norm-bwd", "block-fwd", "block-bwd"):
        X, R, w = (torch.randn(s, device=dev).to(torch.bfloat16) for s in ((a.m, a.n), (a.m, a.n), (a.n,)))
        _, mean, rstd = rows.qlora_layernorm_fwd(X, w)
        ws = rows.new_layernorm_workspace(a.m, a.n, dev)
        call = {"dropout": lambda: rows.qlora_dropout_fwd(X, a.p, a.seed),
                "norm-fwd": lambda: rows.qlora_layernorm_fwd(X, w, w),
                "norm-bwd": lambda: rows.qlora_layernorm_bwd(R, X, mean, rstd, w, workspace=ws),
                "block-fwd": lambda: rows.qlora_dropout_add_layernorm_fwd(X, R, a.p, a.seed, 0, w, w),
                "block-bwd": lambda: rows.qlora_dropout_add_layernorm_bwd(R, R, X, mean, rstd, a.p, a.seed, 0, w,
                                                                          workspace=ws)}[a.op]
    elif a.op == "int8":
        X = torch.randn(a.m, a.k, device=dev).to(torch.bfloat16)
        W8 = int8.qlora_quantize_int8(synthetic.weight_only(a.n, a.k, seed=a.seed).to(dev))
        ws = int8.new_int8_workspace(a.m, a.k, a.n, dev)
        call = lambda: int8.qlora_linear_int8_fwd(X, W8, workspace=ws)  # noqa: E731
    elif a.op in ("quantize", "dequantize"):
        W = synthetic.weight_only(a.n, a.k, seed=a.seed).to(dev)
        Wp = q.qlora_quantize_nf4(W)
        if a.op == "quantize":
            call = lambda: q.qlora_quantize_nf4(W, out=Wp)  # noqa: E731
        else:
            Wd = torch.empty_like(W)
            call = lambda: q.qlora_dequantize_nf4(Wp, out=Wd)  # noqa: E731
    else:
        case = synthetic.linear_case(a.m, a.k, a.n, a.r, a.scale, seed=a.seed)
        Wp = q.qlora_quantize_nf4(case.W.to(dev))
        X, A, B, dY = (t.to(dev) for t in (case.X, case.A, case.B, case.dY))
        ws = rows.new_dropout_workspace(a.m, a.k, a.n, a.r, dev)
        Y, T = q.qlora_linear_fwd(X, Wp, A, B, a.scale, workspace=ws)
        if a.op == "fwd-dropout":
            call = lambda: rows.qlora_linear_fwd_dropout(X, Wp, A, B, a.scale, a.p, a.seed, workspace=ws)  # noqa: E731
        elif a.op == "bwd-dropout":
            call = lambda: rows.qlora_linear_bwd_dropout(dY, X, T, Wp, A, B, a.scale, a.p, a.seed,  # noqa: E731
                                                         workspace=ws)
        elif a.op == "fwd":
            call = lambda: q.qlora_linear_fwd(X, Wp, A, B, a.scale, workspace=ws, Y=Y, T_save=T)  # noqa: E731
        else:
            call = lambda: q.qlora_linear_bwd(dY, X, T, Wp, A, B, a.scale, workspace=ws)  # noqa: E731
    for _ in range(a.warmup):
        call()
    torch.cuda.synchronize()
    total = 0.0
    for _ in range(a.iters):
        flush.zero_()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        call()
        e1.record()
        torch.cuda.synchronize()
        total += e0.elapsed_time(e1)
    print(f"{a.op} m={a.m} n={a.n} k={a.k} r={a.r}: {total / a.iters * 1e3:.1f} us per call")


if __name__ == "__main__":
    main()
