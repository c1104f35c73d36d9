"""Cases of the gradient-clipping and 4-bit microscaled (MXFP4) operators.

Five operators: `clip` (global gradient norm over many tensors, gradients
scaled into other buffers), `adam` (the optimiser step over every parameter
group with the norm's clip factor), `quant` (a matrix to MXFP4 and back to
values), `linear` (a layer y = act(Q(x) Wq^T + b) with MXFP4 weights) and
`linear_bwd` (its gradients dx, dw, db).  With `own` false they run as
elementary torch operations in 32 bits; with `own` true as the calls a user
makes of the package.

MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 values along a row share
a power-of-two scale 2^(byte - 127), every value is a 4-bit E2M1 code (sign,
0 0.5 1 1.5 2 3 4 6), two codes a byte, the earlier one in the low half.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# Adam's constants as the package passes them (in 32 bits)
BETA1, BETA2, EPS, STEP, LR = 0.8999999761581421, 0.9990000128746033, 1.0000000036274937e-15, 1200, 0.00800000037997961


def listed():
    return [
        # the gradients of a tiny decoder (4 levels of 2^12 entries, its layers and biases): a call of a few microseconds
        {"name": "clip_tiny", "op": "clip", "big": 32768, "count": 14, "dtype": "f32", "max_norm": 0.1},
        # many half-precision tensors of odd sizes, views into one bucket at odd offsets
        {"name": "clip_bucket_f16", "op": "clip", "big": 33554432, "count": 300, "dtype": "f16", "max_norm": 0.5},
        # every group of the tiny decoder and 1,000 positions
        {"name": "adam_tiny", "op": "adam", "tables": 32768, "positions": 1000, "max_norm": 0.1},
        # the paper-scale tables (16 levels, 2^21 entries, 4 features) and the Stress scene's 8M positions
        {"name": "adam_paper", "op": "adam", "tables": 134217728, "positions": 8000000, "max_norm": 0.5},
        # an fp16 hash table (16 levels of 2^19 entries x 2 features) stored in 4 bits and read back
        {"name": "quant_table_f16", "op": "quant", "rows": 16, "cols": 1048576, "dtype": "f16", "transpose": False},
        # an odd fp32 activation matrix quantised along its long axis, as the weight gradient needs it
        {"name": "quant_columns_f32", "op": "quant", "rows": 30011, "cols": 250, "dtype": "f32", "transpose": True},
        # serving one token through a wide layer
        {"name": "linear_one", "op": "linear", "M": 1, "K": 4096, "N": 4096, "dtype": "f16", "relu": False},
        # the HexPlane deformation MLP's hidden layer over 300,000 Gaussians
        {"name": "linear_hexplane", "op": "linear", "M": 300000, "K": 256, "N": 256, "dtype": "f16", "relu": True},
        # a large square layer: the matrix cores' rate
        {"name": "linear_square", "op": "linear", "M": 8192, "K": 8192, "N": 8192, "dtype": "bf16", "relu": False},
        # training the HexPlane MLP's first layer (192 features) over 300,000 Gaussians
        {"name": "bwd_hexplane", "op": "linear_bwd", "M": 300000, "K": 192, "N": 256, "dtype": "f16", "relu": True},
        # its last layer (58 outputs), a small odd batch in fp32
        {"name": "bwd_odd_f32", "op": "linear_bwd", "M": 4099, "K": 250, "N": 58, "dtype": "f32", "relu": False},
        # a square layer's training step
        {"name": "bwd_square", "op": "linear_bwd", "M": 4096, "K": 4096, "N": 4096, "dtype": "bf16", "relu": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["clip", "adam", "quant", "linear", "linear", "linear_bwd", "linear_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "clip":
        return {"op": op, "big": _log(rng, 1000, 30_000_000), "count": _log(rng, 2, 300), "dtype": dtype,
                "max_norm": round(rng.uniform(0.01, 1.0), 3)}
    if op == "adam":
        return {"op": op, "tables": 8 * _log(rng, 500, 10_000_000), "positions": _log(rng, 1, 4_000_000),
                "max_norm": round(rng.uniform(0.01, 1.0), 3)}
    if op == "quant":
        rows = _log(rng, 1, 300_000)
        return {"op": op, "rows": rows, "cols": _log(rng, 1, min(1_000_000, 60_000_000 // rows)), "dtype": dtype,
                "transpose": rng.random() < 0.5}
    # layers: M rows (one token up to every Gaussian of a scene), K and N up to wide ones
    K, N = _log(rng, 8, 4096), _log(rng, 8, 4096)
    if rng.random() < 0.5:  # this framework's widths
        K, N = rng.choice([32, 64, 192, 256]), rng.choice([11, 56, 58, 64, 256])
    low = 1 if op == "linear" else 64
    M = _log(rng, low, max(low, min(300_000, 100_000_000 // (K + N), 130_000_000_000 // (K * N))))
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "relu": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _sizes(case):
    """Tensor sizes of a clip case: the large one, then ragged sizes from 1 to 200,000 spread over their logarithm."""
    out = [case["big"]]
    for i in range(case["count"] - 1):
        u = ((i + 1) * 0.6180339887498949) % 1.0
        out.append(max(1, int(200_000 ** u)) if case["big"] >= 1_000_000 else max(1, int(4096 ** u)))
    return out


# the other groups of a shared-trunk decoder: trunk weights and biases, the head's rows and biases per attribute
_MATS = (("w0", 64 * 32), ("b0", 64), ("w1", 64 * 64), ("b1", 64), ("head_w_scale", 3 * 64), ("head_b_scale", 3),
         ("head_w_rotation", 4 * 64), ("head_b_rotation", 4), ("head_w_color", 3 * 64), ("head_b_color", 3),
         ("head_w_opacity", 64), ("head_b_opacity", 1))


def _gradients(gen, n, touched=0.3):
    """A decoder's gradients: heavy-tailed, and zero for the table entries that no Gaussian touched."""
    g = torch.randn(n, generator=gen, device="cuda")
    g.mul_(torch.randn(n, generator=gen, device="cuda").mul_(0.7).exp_()).mul_(1e-3)
    return g.mul_(torch.rand(n, generator=gen, device="cuda").lt_(touched))


def _activations(gen, rows, cols, dtype):
    """Rows of different size, values of either sign."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    return x.mul_(torch.randn((rows, 1), generator=gen, device="cuda").mul_(0.5).exp_()).to(dtype)


def _weights(gen, n, k):
    return torch.randn((n, k), generator=gen, device="cuda").mul_(1.0 / math.sqrt(k))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    if op == "clip":
        sizes = _sizes(case)
        flat = _gradients(gen, sum(sizes)).to(DTYPES[case["dtype"]])
        s["flat"], s["out"] = flat, torch.empty_like(flat)
        s["grads"] = list(flat.split(sizes))
        s["outs"] = list(s["out"].split(sizes))
        if own:  # the list of tensors that a program clips step after step
            from implicit_attribute_decode_amd.pipeline import GradClip

            s["clip"] = GradClip(s["grads"], s["outs"])
    elif op == "adam":
        sizes = {"tables": case["tables"], **dict(_MATS)}
        s["p"], s["m"], s["v"], s["g"] = {}, {}, {}, {}
        for k, n in sizes.items():
            s["p"][k] = torch.randn(n, generator=gen, device="cuda").mul_(0.1)
            s["g"][k] = _gradients(gen, n, 0.1 if k == "tables" else 1.0)
            s["m"][k] = s["g"][k].flip(0).mul(0.3)
            s["v"][k] = s["m"][k].square().mul_(3.0).add_(s["g"][k].square(), alpha=0.01)
        n = case["positions"]
        s["xyzt"] = torch.randn((n, 4), generator=gen, device="cuda")
        s["p"]["positions"] = s["xyzt"][:, :3]
        s["g"]["positions"] = _gradients(gen, 3 * n, 0.5).view(n, 3)
        s["m"]["positions"] = s["g"]["positions"].flip(0).mul(0.3)
        s["v"]["positions"] = s["m"]["positions"].square().mul_(3.0).add_(s["g"]["positions"].square(), alpha=0.01)
        s["f16"] = s["p"]["tables"].half()  # the mirror that the decode reads
        if own:  # the optimiser that a training program keeps, at its step
            from implicit_attribute_decode_amd.pipeline import Adam

            groups = {k: {"param": p, "lr": LR, "f16": s["f16"].view(torch.int16) if k == "tables" else None}
                      for k, p in s["p"].items()}
            s["adam"] = Adam(groups, warmup=0, total=1_000_000_000, beta1=BETA1, beta2=BETA2, eps=EPS)
            s["adam"].state = {k: (s["m"][k], s["v"][k]) for k in groups}
            s["adam"].t = STEP - 1
        s["t"] = STEP - 1
    elif op == "quant":
        s["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["dtype"]])
    else:
        M, K, N, dt = case["M"], case["K"], case["N"], DTYPES[case["dtype"]]
        s["x"] = _activations(gen, M, K, dt)
        w = _weights(gen, N, K)
        if op == "linear":
            s["codes"], s["scales"] = _pack(w)
            s["bias"] = torch.randn(N, generator=gen, device="cuda").mul_(0.1)
        else:
            # the layer's weights in blocks along its outputs, which the input's gradient sums over
            s["codes"], s["scales"] = _pack(w.t().contiguous())
            s["dy"] = _activations(gen, M, N, dt).mul_(1e-2)
            s["y"] = torch.randn((M, N), generator=gen, device="cuda").relu_().to(dt) if case["relu"] else None
    return s


# ------------------------------------------------------- plain 4-bit forms


def _codes(x):
    """(signed E2M1 values q [rows, blocks, 32], block exponents e [rows, blocks, 1]) of rows of x: x ~ q 2^e."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    v = torch.nn.functional.pad(x.float(), (0, blocks * 32 - cols)).view(rows, blocks, 32)
    top = torch.frexp(v.abs().amax(-1, keepdim=True))[1] - 1  # floor(log2(largest magnitude))
    e = (top - 2).clamp_(-127, 125)
    u = v * torch.exp2(-e.float())
    a = u.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp_(max=6.0)
    return torch.copysign(q, u), e


def _quantized(x):
    """The values that rows of x have in MXFP4, in 32 bits."""
    q, e = _codes(x)
    return (q * torch.exp2(e.float())).view(x.shape[0], -1)[:, :x.shape[1]]


def _pack(x):
    """(codes [rows, 16 blocks] bytes, scales [rows, blocks] bytes) of rows of x."""
    q, e = _codes(x)
    a = q.abs()
    mag = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, a + 2.0, 0.5 * a + 4.0))
    c = (mag + 8.0 * torch.signbit(q)).to(torch.uint8).view(x.shape[0], -1)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), (e.squeeze(-1) + 127).to(torch.uint8).contiguous()


def _unpack(codes, scales, cols):
    """The 32-bit values that packed rows stand for."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 32)
    v = grid[c.int()] * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return v.view(codes.shape[0], -1)[:, :cols]


def _plain_clip(s):
    c = s["case"]
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt()
    factor = torch.where(norm > c["max_norm"], c["max_norm"] / norm, 1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * factor)
    return {"out": s["out"], "norm": norm, "factor": factor}


def _plain_adam(s):
    c = s["case"]
    s["t"] += 1
    t = s["t"]
    total = torch.stack([g.square().sum() for g in s["g"].values()]).sum()
    norm = total.sqrt()
    factor = torch.where(norm > c["max_norm"], c["max_norm"] / norm, 1.0)
    step, vs = LR / (1.0 - BETA1 ** t), 1.0 / (1.0 - BETA2 ** t)
    for k, p in s["p"].items():
        g, m, v = s["g"][k] * factor, s["m"][k], s["v"][k]
        m.mul_(BETA1).add_(g * (1.0 - BETA1))
        v.mul_(BETA2).add_(g * g * (1.0 - BETA2))
        p.sub_(step * m / ((v * vs).sqrt() + EPS))
    s["f16"].copy_(s["p"]["tables"])
    return {"p": s["p"], "m": s["m"], "v": s["v"], "f16": s["f16"], "norm": norm, "factor": factor}


def _plain_quant(s):
    c = s["case"]
    x = s["x"].t() if c["transpose"] else s["x"]
    return _quantized(x).to(s["x"].dtype)


def _plain_linear(s):
    c = s["case"]
    y = _quantized(s["x"]) @ _unpack(s["codes"], s["scales"], c["K"]).t() + s["bias"]
    return (y.relu_() if c["relu"] else y).to(s["x"].dtype)


def _plain_linear_bwd(s):
    c = s["case"]
    d = s["dy"].float()
    if s["y"] is not None:
        d = d * (s["y"] > 0)
    dx = _quantized(d) @ _unpack(s["codes"], s["scales"], c["N"]).t()
    dw = _quantized(d.t()) @ _quantized(s["x"].float().t()).t()
    return {"x": dx.to(s["x"].dtype), "weight": dw, "bias": d.sum(0)}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"clip": _plain_clip, "adam": _plain_adam, "quant": _plain_quant, "linear": _plain_linear,
                "linear_bwd": _plain_linear_bwd}[op](s)
    from implicit_attribute_decode_amd import pipeline as P

    if op == "clip":
        stats = s["clip"](c["max_norm"])
        return {"out": s["out"], "norm": stats[0], "factor": stats[1]}
    if op == "adam":
        stats = s["adam"].step(s["g"], max_norm=c["max_norm"])
        return {"p": s["p"], "m": s["m"], "v": s["v"], "f16": s["f16"], "norm": stats[0], "factor": stats[1]}
    if op == "quant":
        return P.mx4_quantize(s["x"], transpose=c["transpose"]).dequantize(s["x"].dtype)
    act = "relu" if c["relu"] else "none"
    if op == "linear":
        return P.mx4_linear(s["x"], P.Mx4Tensor(s["codes"], s["scales"], c["K"]), s["bias"], act)
    return P.mx4_linear_backward(s["dy"], s["x"], P.Mx4Tensor(s["codes"], s["scales"], c["N"]), y=s["y"])


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * BYTES[case["dtype"]], "flops": 3 * n}
    if op == "adam":
        n = case["tables"] + sum(k for _, k in _MATS) + 3 * case["positions"]
        return {"bytes": 28 * n + 2 * case["tables"], "flops": 16 * n}
    packed = lambda r, c: r * ((c + 31) // 32) * 17  # noqa: E731
    if op == "quant":
        n = case["rows"] * case["cols"]
        r, c = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        return {"bytes": 2 * n * BYTES[case["dtype"]] + packed(r, c), "flops": 4 * n}
    M, K, N, b = case["M"], case["K"], case["N"], BYTES[case["dtype"]]
    if op == "linear":
        return {"bytes": b * M * (K + N) + packed(N, K) + 4 * N, "flops": 2 * M * N * K}
    return {"bytes": b * M * (N * (2 if case["relu"] else 1) + 2 * K) + packed(K, N) + 4 * N * K + 4 * N,
            "flops": 4 * M * N * K}


# ------------------------------------------------ definitions in 64 bits


def _exact_mx4(x):
    """Values of rows of x (64-bit) in MXFP4, by the decision points between neighbouring codes: a tie goes to the even code."""
    rows, cols = x.shape
    out = torch.zeros((rows, (cols + 31) // 32 * 32), dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    b = out.view(rows, -1, 32)
    m = b.abs().max(-1, keepdim=True).values
    e = torch.where(m > 0, torch.floor(torch.log2(m)), torch.zeros_like(m))
    e = torch.where(torch.exp2(e) > m, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= m, e + 1, e)
    scale = torch.exp2((e - 2).clamp(min=-127))
    a = b.abs() / scale
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)[code.long()]
    return (value * scale * torch.sign(b)).view(rows, -1)[:, :cols]


def _exact_unpacked(codes, scales, cols):
    c = codes.long()
    c = torch.stack([c % 16, c // 16], -1).view(codes.shape[0], -1)
    exponent, mantissa = (c // 2) % 4, c % 2
    v = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
    v = torch.where(c >= 8, -v, v)
    return (v.view(codes.shape[0], -1, 32) * torch.exp2(scales.double() - 127).unsqueeze(-1)).view(c.shape)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g)
        factor = (case["max_norm"] / norm).clamp(max=1.0)
        return {"out": g * factor, "norm": norm, "factor": factor}
    if op == "adam":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["g"].values()]))
        factor = (case["max_norm"] / norm).clamp(max=1.0)
        out = {"p": {}, "m": {}, "v": {}, "norm": norm, "factor": factor}
        for k in s["p"]:
            g = s["g"][k].double() * factor
            m = BETA1 * s["m"][k].double() + (1 - BETA1) * g
            v = BETA2 * s["v"][k].double() + (1 - BETA2) * g ** 2
            upd = LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
            out["p"][k], out["m"][k], out["v"][k] = s["p"][k].double() - upd, m, v
        out["f16"] = out["p"]["tables"]
        return out
    if op == "quant":
        x = s["x"].double()
        return _exact_mx4(x.t() if case["transpose"] else x)
    x = s["x"].double()
    if op == "linear":
        w = _exact_unpacked(s["codes"], s["scales"], case["K"])
        y = torch.matmul(_exact_mx4(x), w.t().contiguous()) + s["bias"].double()
        return torch.clamp(y, min=0.0) if case["relu"] else y
    d = s["dy"].double()
    if s["y"] is not None:
        d = torch.where(s["y"] > 0, d, torch.zeros_like(d))
    wt = _exact_unpacked(s["codes"], s["scales"], case["N"])
    dw = torch.matmul(_exact_mx4(d.t()), _exact_mx4(x.t()).t().contiguous())
    return {"x": torch.matmul(_exact_mx4(d), wt.t().contiguous()), "weight": dw, "bias": d.sum(0)}
