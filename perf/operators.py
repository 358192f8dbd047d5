"""Cases and plain forms of the operators around and beside the 4-bit LoRA
linear: dropout from a counter-based generator, layer norm, the two fused with
a residual sum, the linear whose adapter sees dropped inputs, and the product
in 8-bit integers.

``run`` computes a case either with elementary torch operations in float32 or
wider (``own`` false) or through the package's calls (``own`` true).  ``exact``
restates the same definitions in float64.

Random draws of the dropout: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011) with the 64-bit seed as
the key.  Row i of a [rows, cols] matrix takes counters
offset + i * ceil(cols / 8) + j for its groups of eight columns j; each 128-bit
output gives eight 16-bit draws, the low half of word 0 first.  An element is
dropped when its draw is below t = round(65536 p), and what is kept is
multiplied by c = 65536 / (65536 - t), so the mean is kept exactly.
"""

import math
import statistics

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a short evaluation batch of an odd-sized head, in float32: launch latency counts
        {"name": "dropout_short_odd", "op": "dropout", "rows": 37, "cols": 1001, "dtype": "fp32", "p": 0.5,
         "residual": True},
        # the gated intermediate of the 7B-shaped MLP over 8192 training tokens
        {"name": "dropout_mlp", "op": "dropout", "rows": 8192, "cols": 11008, "dtype": "bf16", "p": 0.05,
         "residual": False},
        # one token on its way through a decoder of width 8192
        {"name": "norm_token", "op": "norm_fwd", "rows": 1, "cols": 8192, "dtype": "bf16", "wdtype": "bf16"},
        # gradient of a norm with float32 parameters over a ragged batch in fp16
        {"name": "norm_ragged_bwd", "op": "norm_bwd", "rows": 777, "cols": 5003, "dtype": "fp16", "wdtype": "fp32"},
        # gradient of a norm of width 8192 over the 4096 tokens of a training step
        {"name": "norm_wide_bwd", "op": "norm_bwd", "rows": 4096, "cols": 8192, "dtype": "bf16", "wdtype": "bf16"},
        # the smallest configuration's tokens through residual dropout and norm, both ways, in float32
        {"name": "block_small", "op": "block", "rows": 16, "cols": 256, "dtype": "fp32", "wdtype": "fp32", "p": 0.1},
        # residual dropout and norm of the 65B-shaped block over 4096 tokens, both ways
        {"name": "block_wide", "op": "block", "rows": 4096, "cols": 8192, "dtype": "bf16", "wdtype": "fp32",
         "p": 0.1},
        # the smallest configured linear with adapter dropout: 16 tokens, 256 x 256, rank 8, both ways
        {"name": "lora_small", "op": "lora", "M": 16, "K": 256, "N": 256, "r": 8, "scale": 2.0, "p": 0.05},
        # the 7B-shaped attention projection over 8 sequences of 256 tokens with adapter dropout, both ways
        {"name": "lora_projection", "op": "lora", "M": 2048, "K": 4096, "N": 4096, "r": 64, "scale": 0.25, "p": 0.1},
        # one generated token through an 8-bit weight of the 65B shape
        {"name": "int8_token", "op": "int8", "M": 1, "K": 8192, "N": 8192, "dtype": "bf16"},
        # a ragged prompt through an 8-bit weight with odd depth and odd rows
        {"name": "int8_ragged", "op": "int8", "M": 300, "K": 11003, "N": 4099, "dtype": "fp16"},
        # 4096 prompt tokens through an 8-bit weight of the 65B shape
        {"name": "int8_tokens", "op": "int8", "M": 4096, "K": 8192, "N": 8192, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["dropout", "norm_fwd", "norm_bwd", "block", "lora", "int8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    p = rng.choice([0.05, 0.1, round(rng.uniform(0.0, 0.9), 3)])
    if op == "lora":
        return {"op": op, "M": _spread(rng, 1, 2048), "K": 64 * _spread(rng, 1, 64), "N": 8 * _spread(rng, 2, 512),
                "r": _spread(rng, 1, 64), "scale": rng.choice([0.25, 2.0]), "p": p}
    if op == "int8":
        return {"op": op, "M": _spread(rng, 1, 4096), "K": _spread(rng, 16, 8192), "N": _spread(rng, 16, 8192),
                "dtype": dtype}
    if op == "dropout":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 1, 5504), "dtype": dtype, "p": p,
                "residual": rng.random() < 0.5}
    case = {"op": op, "rows": _spread(rng, 1, 4096), "cols": _spread(rng, 32, 4096), "dtype": dtype,
            "wdtype": rng.choice([dtype, "fp32"])}
    if op == "block":
        case["p"] = p
    return case


def work(case):
    op = case["op"]
    if op == "lora":
        M, K, N, r = case["M"], case["K"], case["N"], case["r"]
        weight = N * K // 2 + -(-N * K // 64) + 4 * -(-N * K // 16384)
        # X, dY, A, B and the weight in; Y, dX (bf16), T, dA and dB (fp32) out
        nbytes = weight + 2 * (2 * M * K + 2 * M * N + K * r + r * N) + 4 * (M * r + K * r + r * N)
        return {"bytes": nbytes, "flops": 4 * M * N * K + 6 * M * r * (K + N)}
    if op == "int8":
        M, K, N, s = case["M"], case["K"], case["N"], SIZE[case["dtype"]]
        return {"bytes": s * M * K + N * K + 4 * N + s * M * N, "flops": 2 * M * N * K}
    n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
    if op == "dropout":
        return {"bytes": n * s * (3 if case["residual"] else 2), "flops": 2 * n}
    par = 2 * case["cols"] * SIZE[case["wdtype"]]
    if op == "norm_fwd":
        return {"bytes": 2 * n * s + par + 8 * case["rows"], "flops": 8 * n}
    if op == "norm_bwd":  # dY, X and the weight in; dX, the gradients of weight and bias out
        return {"bytes": 3 * n * s + par // 2 + 8 * case["cols"] + 8 * case["rows"], "flops": 12 * n}
    # block: X, residual, dY, dZ in; Y, Z, dX, dResidual out
    return {"bytes": 8 * n * s + par + 8 * case["cols"] + 8 * case["rows"], "flops": 24 * n}


# ------------------------------------------------------------------ inputs
def _hidden(g, rows, cols, dtype):
    """Hidden states as a decoder has them: normal values, a few wide columns, an offset."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    wide = 1.0 + 7.0 * (torch.rand(cols, generator=g, device=DEV) < 0.01)
    return (x * wide + 0.1).to(DTYPES[dtype])


def _levels():
    """The 16 levels of the 4-bit normal code: quantiles of eight positive and
    seven negative steps of the normal distribution, an exact zero, ends at 1."""
    inv = statistics.NormalDist().inv_cdf
    edge = 1.0 - 0.5 * (1.0 / 30.0 + 1.0 / 32.0)
    up = [inv(edge + (0.5 - edge) * i / 8) for i in range(8)]
    down = [-inv(edge + (0.5 - edge) * i / 7) for i in range(7)]
    v = sorted(up + down + [0.0])
    return [x / max(v) for x in v]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "seed": 0x9E3779B97F4A7C15 * (seed + 1) % (1 << 63), "offset": 1000 * seed}
    if op == "lora":
        M, K, N, r = case["M"], case["K"], case["N"], case["r"]
        s["X"], s["dY"] = _hidden(g, M, K, "bf16"), torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
        s["A"] = (0.01 * torch.randn(K, r, generator=g, device=DEV)).to(torch.bfloat16)
        s["B"] = (0.01 * torch.randn(r, N, generator=g, device=DEV)).to(torch.bfloat16)
        # a frozen weight as it comes off a checkpoint in the packed format
        nb = N * K // 64
        s["codes"] = torch.randint(0, 256, (N * K // 2,), generator=g, device=DEV, dtype=torch.uint8)
        s["absmax_q"] = torch.randint(90, 256, (nb,), generator=g, device=DEV, dtype=torch.uint8)
        s["absmax_scale"] = 0.06 + 0.02 * torch.rand(-(-nb // 256), generator=g, device=DEV)
        s["levels"] = torch.tensor(_levels(), dtype=torch.float32, device=DEV)
        return s
    if op == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        s["X"] = _hidden(g, M, K, case["dtype"])
        # a weight quantized once, by output channel; rows padded with zeros to 16 codes
        s["wcodes"] = torch.zeros(N, -(-K // 16) * 16, dtype=torch.int8, device=DEV)
        s["wcodes"][:, :K] = (40.0 * torch.randn(N, K, generator=g, device=DEV)).round().clamp(-127, 127).to(torch.int8)
        s["wscale"] = (0.06 + 0.02 * torch.rand(N, generator=g, device=DEV)) / 127
        return s
    rows, cols = case["rows"], case["cols"]
    s["X"] = _hidden(g, rows, cols, case["dtype"])
    if op == "dropout":
        s["residual"] = _hidden(g, rows, cols, case["dtype"]) if case["residual"] else None
        return s
    s["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(DTYPES[case["wdtype"]])
    s["bias"] = (0.2 * torch.randn(cols, generator=g, device=DEV)).to(DTYPES[case["wdtype"]])
    if op != "norm_fwd":
        s["dY"] = torch.randn(rows, cols, generator=g, device=DEV).to(DTYPES[case["dtype"]])
    if op == "norm_bwd":
        x = s["X"].double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
    if op == "block":
        s["residual"] = _hidden(g, rows, cols, case["dtype"])
        s["dZ"] = torch.randn(rows, cols, generator=g, device=DEV).to(DTYPES[case["dtype"]])
    return s


# ------------------------------------------------------------------ plain forms
def _philox_round(c, k):
    a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # products modulo 2^64; both halves are kept
    low = 0xFFFFFFFF
    return [(b >> 32 & low) ^ c[1] ^ k[0], b & low, (a >> 32 & low) ^ c[3] ^ k[1], a & low]


def _keep(rows, cols, p, seed, offset):
    """Truth values of the elements that stay."""
    groups = -(-cols // 8)
    n = offset + torch.arange(rows * groups, device=DEV, dtype=torch.int64)
    low = 0xFFFFFFFF
    c = [n & low, n >> 32 & low, torch.zeros_like(n), torch.zeros_like(n)]
    k = [seed & low, seed >> 32 & low]
    for _ in range(10):
        c = _philox_round(c, k)
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    c = torch.stack(c, 1)
    draws = torch.stack([c & 0xFFFF, c >> 16], 2).reshape(rows, groups * 8)[:, :cols]
    return draws >= round(65536 * p)


def _gain(p):
    t = round(65536 * p)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def _dropped(x, p, seed, offset):
    """Float32 values of dropout(x)."""
    keep = _keep(x.shape[0], x.shape[1], p, seed, offset)
    return torch.where(keep, x.float() * _gain(p), torch.zeros((), device=DEV))


def _norm(x, w, b):
    x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    return d * rstd * w.float() + b.float(), mean[:, 0], rstd[:, 0]


def _norm_grads(dy, x, mean, rstd, w):
    dy, h = dy.float(), (x.float() - mean[:, None]) * rstd[:, None]
    g = dy * w.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def _weight(s):
    """The bf16 weight that the packed codes stand for."""
    case = s["case"]
    code = torch.stack([s["codes"] >> 4, s["codes"] & 15], 1).reshape(-1).long()
    block = (s["absmax_q"].float() / 255) * s["absmax_scale"].repeat_interleave(256)[:s["absmax_q"].numel()]
    w = s["levels"][code].reshape(-1, 64) * block[:, None]
    return w.to(torch.bfloat16).float().reshape(case["N"], case["K"])


def _lora(s):
    case = s["case"]
    x, dy, a, b = s["X"].float(), s["dY"].float(), s["A"].float(), s["B"].float()
    w, scale = _weight(s), case["scale"]
    keep = _keep(case["M"], case["K"], case["p"], s["seed"], s["offset"])
    xd = torch.where(keep, x, 0.0) * _gain(case["p"])
    t = scale * (xd @ a)
    y = x @ w.T + t @ b
    u = scale * (dy @ b.T)
    dx = dy @ w + torch.where(keep, u @ a.T, 0.0) * _gain(case["p"])
    return y.to(torch.bfloat16), t, dx.to(torch.bfloat16), xd.T @ u, t.T @ dy


def _int8(s):
    x = s["X"].double()  # quotients next to a border between codes need more than 32 bits
    scale = (s["X"].float().abs().amax(1) / 127).double()
    code = torch.where(scale[:, None] > 0, (x / scale[:, None]).round(), 0.0).clamp(-127, 127)
    total = code @ s["wcodes"][:, :x.shape[1]].double().T
    return (total * scale[:, None] * s["wscale"].double()).to(s["X"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _run_own(s, case, op)
    if op == "dropout":
        y = _dropped(s["X"], case["p"], s["seed"], s["offset"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["X"].dtype)
    if op == "norm_fwd":
        y, mean, rstd = _norm(s["X"], s["weight"], s["bias"])
        return y.to(s["X"].dtype), mean, rstd
    if op == "norm_bwd":
        dx, dw, db = _norm_grads(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"])
        return dx.to(s["X"].dtype), dw, db
    if op == "block":
        dt = s["X"].dtype
        z = (_dropped(s["X"], case["p"], s["seed"], s["offset"]) + s["residual"].float()).to(dt)
        y, mean, rstd = _norm(z, s["weight"], s["bias"])
        dz, dw, db = _norm_grads(s["dY"], z, mean, rstd, s["weight"])
        dz = dz + s["dZ"].float()
        return y.to(dt), z, mean, rstd, _dropped(dz, case["p"], s["seed"], s["offset"]).to(dt), dz.to(dt), dw, db
    if op == "lora":
        return _lora(s)
    return _int8(s)


def _run_own(s, case, op):
    import bit_quantized_lora_quantize_b200 as q

    if op == "dropout":
        return q.qlora_dropout_fwd(s["X"], case["p"], s["seed"], s["offset"], residual=s["residual"])
    if op == "norm_fwd":
        return q.qlora_layernorm_fwd(s["X"], s["weight"], s["bias"], EPS)
    if op == "int8":
        if "W" not in s:  # the handle and the workspace that a program keeps for its weight
            s["W"] = q.PackedInt8(s["wcodes"], s["wscale"], (case["N"], case["K"]))
            s["ws"] = q.new_int8_workspace(case["M"], case["K"], case["N"], s["X"].device)
        return q.qlora_linear_int8_fwd(s["X"], s["W"], workspace=s["ws"])
    if op == "lora":
        if "W" not in s:
            s["W"] = q.PackedNF4(s["codes"], s["absmax_q"], s["absmax_scale"], (case["N"], case["K"]))
            s["ws"] = q.new_dropout_workspace(case["M"], case["K"], case["N"], case["r"], s["X"].device)
        y, t = q.qlora_linear_fwd_dropout(s["X"], s["W"], s["A"], s["B"], case["scale"], case["p"], s["seed"],
                                          s["offset"], workspace=s["ws"])
        dx, da, db = q.qlora_linear_bwd_dropout(s["dY"], s["X"], t, s["W"], s["A"], s["B"], case["scale"], case["p"],
                                                s["seed"], s["offset"], workspace=s["ws"])
        return y, t, dx, da, db
    if "ws" not in s:
        s["ws"] = q.new_layernorm_workspace(case["rows"], case["cols"], s["X"].device)
    if op == "norm_bwd":
        return q.qlora_layernorm_bwd(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"], workspace=s["ws"])
    y, z, mean, rstd = q.qlora_dropout_add_layernorm_fwd(s["X"], s["residual"], case["p"], s["seed"], s["offset"],
                                                         s["weight"], s["bias"], EPS)
    dx, dr, dw, db = q.qlora_dropout_add_layernorm_bwd(s["dY"], s["dZ"], z, mean, rstd, case["p"], s["seed"],
                                                       s["offset"], s["weight"], workspace=s["ws"])
    return y, z, mean, rstd, dx, dr, dw, db


# ------------------------------------------------------------------ definitions in 64 bits
def _kept64(rows, cols, p, seed, offset):
    """The multiplier of each element (0 or the gain), in numpy's unsigned 64-bit integers."""
    groups = (cols + 7) // 8
    word, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    n = np.arange(rows * groups, dtype=np.uint64) + np.uint64(offset)
    x0, x1 = n & word, n >> shift
    x2, x3 = np.zeros_like(n), np.zeros_like(n)
    k0, k1 = seed % 2**32, seed // 2**32
    for _ in range(10):
        m0, m1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (m1 >> shift) ^ x1 ^ np.uint64(k0), m1 & word, (m0 >> shift) ^ x3 ^ np.uint64(k1), m0 & word
        k0, k1 = (k0 + 0x9E3779B9) % 2**32, (k1 + 0xBB67AE85) % 2**32
    draws = np.stack([x0, x1, x2, x3], axis=1).astype("<u4").view("<u2").reshape(rows, groups * 8)[:, :cols]
    t = round(65536 * p)
    keep = torch.from_numpy(draws.astype(np.int32)).to(DEV) >= t
    return keep.double() * (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _stats64(x):
    mean = x.sum(1) / x.shape[1]
    var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
    return mean, 1.0 / torch.sqrt(var + EPS)


def _grads64(dy, x, mean, rstd, w):
    n = x.shape[1]
    hat = (x - mean[:, None]) * rstd[:, None]
    u = dy * w
    inner = u - (u.sum(1) / n)[:, None] - hat * ((u * hat).sum(1) / n)[:, None]
    return inner * rstd[:, None], torch.einsum("ij,ij->j", dy, hat), dy.sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "norm_fwd":
        mean, rstd = _stats64(f["X"])
        return torch.addcmul(f["bias"], (f["X"] - mean[:, None]) * rstd[:, None], f["weight"]), mean, rstd
    if op == "norm_bwd":
        return _grads64(f["dY"], f["X"], f["mean"], f["rstd"], f["weight"])
    if op == "int8":
        scale = (f["X"].abs().max(dim=1).values.float() / 127).double()
        ratio = f["X"] / torch.where(scale > 0, scale, 1.0)[:, None]
        low = torch.floor(ratio)
        up = (ratio - low > 0.5) | ((ratio - low == 0.5) & (low % 2 != 0))
        code = torch.clamp(low + up, -127, 127)
        w = s["wcodes"][:, :case["K"]].double() * f["wscale"][:, None]
        return torch.einsum("mk,nk->mn", code * scale[:, None], w)
    if op == "lora":
        m = _kept64(case["M"], case["K"], case["p"], s["seed"], s["offset"])
        nibble = torch.empty(s["codes"].numel(), 2, dtype=torch.int64, device=DEV)
        nibble[:, 0], nibble[:, 1] = s["codes"] // 16, s["codes"] % 16
        # the weight itself is defined by float32 steps and one bf16 rounding
        group = torch.arange(s["absmax_q"].numel(), device=DEV) // 256
        const = (s["absmax_q"].float() / 255.0) * s["absmax_scale"][group]
        w = (s["levels"][nibble.view(-1)] * const.repeat_interleave(64)).bfloat16().double().view(case["N"], case["K"])
        xm = f["X"] * m
        t = case["scale"] * (xm @ f["A"])
        u = case["scale"] * (f["dY"] @ f["B"].t())
        y = torch.addmm(t @ f["B"], f["X"], w.t())
        dx = torch.addmm((u @ f["A"].t()) * m, f["dY"], w)
        return y, t, dx, xm.t() @ u, t.t() @ f["dY"]
    m = _kept64(case["rows"], case["cols"], case["p"], s["seed"], s["offset"])
    z = f["X"] * m + (f["residual"] if "residual" in f else 0.0)
    if op == "dropout":
        return z
    # the sum is held in the inputs' type: what follows is defined on the rounded sum
    held = z.to(s["X"].dtype).double()
    mean, rstd = _stats64(held)
    y = torch.addcmul(f["bias"], (held - mean[:, None]) * rstd[:, None], f["weight"])
    dz, dw, db = _grads64(f["dY"], held, mean, rstd, f["weight"])
    total = dz + f["dZ"]
    return y, z, mean, rstd, total * m, total, dw, db
