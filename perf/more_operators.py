"""Cases of the code-table, dropout and group-scaled 4-bit operators.

Five operators: `embed` (rows of a table picked by index, scaled, with dropout
where asked; the table in 32 or 16 bits or in MXFP4), `embed_bwd` (the table's
gradient, the sum of the rows that picked each entry), `dropout` (a matrix
with values dropped by a counter-based generator), `q4_quant` (a matrix to
4-bit codes with group scales and back) and `q4_linear` (a layer
y = act(x Wq^T + b) with such weights and x as it is).  With `own` false they
run as elementary torch operations; with `own` true as the calls a user makes
of the package.

Dropout: value (r, c) of call `offset` under `seed` is kept where word c mod 4
of Philox4x32-10 (Salmon, Moraes, Dror & Shaw 2011) of the counter
(floor(c / 4), r, offset low, offset high) and the key (seed low, seed high) is
at least p 2^32 (rounded to a whole number), and then divided by 1 - p.

Group-scaled 4 bits: a group of 32, 64 or 128 values along a row has a scale s
and a zero z in 0..15 and stands for s (q - z), q in 0..15; two codes q a
byte, the earlier one in the low half.  One 32-bit word holds both: s as a
float32 whose lowest byte is zero, and z in that byte.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
OFFSET = 1200  # the call number a training program has reached


def listed():
    return [
        # one frame's cameras look up their codes (150 frames of 32 values): a call of a few microseconds
        {"name": "embed_codes", "op": "embed", "table": "f32", "V": 150, "D": 32, "n": 27, "out": "f16", "index": "i64",
         "order": "uniform", "scale": 1.0, "p": 0.0},
        # training: 300,000 rows out of 2^19 entries of 256 values, some far more often than others, with dropout
        {"name": "embed_drop", "op": "embed", "table": "bf16", "V": 524288, "D": 256, "n": 300000, "out": "bf16",
         "index": "i64", "order": "zipf", "scale": 16.0, "p": 0.1},
        # serving from a table kept in 4 bits
        {"name": "embed_mx4", "op": "embed", "table": "mx4", "V": 1048576, "D": 64, "n": 100003, "out": "f16",
         "index": "i32", "order": "uniform", "scale": 1.0, "p": 0.0},
        # the gradient of a table of many entries, each picked a few times and some thousands of times
        {"name": "bwd_tokens", "op": "embed_bwd", "V": 50021, "D": 512, "n": 131071, "dtype": "bf16", "index": "i64",
         "order": "zipf", "scale": 16.0, "p": 0.0},
        # the gradient of 150 frames' codes, from 300,000 Gaussians stored frame after frame, through dropout
        {"name": "bwd_codes", "op": "embed_bwd", "V": 150, "D": 64, "n": 300000, "dtype": "f32", "index": "i32",
         "order": "frames", "scale": 1.0, "p": 0.1},
        # dropout of the HexPlane MLP's hidden layer over 300,000 Gaussians
        {"name": "dropout_hexplane", "op": "dropout", "rows": 300000, "cols": 256, "dtype": "f16", "p": 0.1},
        # a small odd batch in fp32
        {"name": "dropout_odd_f32", "op": "dropout", "rows": 4099, "cols": 250, "dtype": "f32", "p": 0.5},
        # the weights of a wide layer to 4 bits and back
        {"name": "quant_square", "op": "q4_quant", "rows": 8192, "cols": 8192, "dtype": "bf16", "group": 128},
        # an odd layer's fp32 master weights
        {"name": "quant_odd_f32", "op": "q4_quant", "rows": 1000, "cols": 250, "dtype": "f32", "group": 32},
        # serving one token through a wide layer
        {"name": "q4_one", "op": "q4_linear", "M": 1, "K": 4096, "N": 4096, "dtype": "f16", "group": 128, "relu": False},
        # a few tokens at once through a wider one: the rate at which weights are read
        {"name": "q4_few", "op": "q4_linear", "M": 5, "K": 8192, "N": 16384, "dtype": "bf16", "group": 64, "relu": False},
        # many rows: the matrix cores' rate
        {"name": "q4_many", "op": "q4_linear", "M": 4096, "K": 4096, "N": 4096, "dtype": "bf16", "group": 128,
         "relu": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "embed_bwd", "dropout", "q4_quant", "q4_linear", "q4_linear", "q4_linear"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("embed", "embed_bwd"):
        D = _log(rng, 1, 1024)
        V = _log(rng, 1, min(1_000_000, 60_000_000 // D))
        n = _log(rng, 1, min(300_000, 60_000_000 // D))
        c = {"op": op, "V": V, "D": D, "n": n, "index": rng.choice(["i32", "i64"]),
             "order": rng.choice(["uniform", "zipf", "frames"]), "scale": rng.choice([1.0, round(math.sqrt(D), 3)]),
             "p": rng.choice([0.0, round(rng.uniform(0.01, 0.6), 3)])}
        if op == "embed":
            return {**c, "table": rng.choice(["f32", "f16", "bf16", "mx4"]), "out": dtype}
        return {**c, "dtype": dtype}
    if op == "dropout":
        rows = _log(rng, 1, 300_000)
        return {"op": op, "rows": rows, "cols": _log(rng, 1, min(8192, 60_000_000 // rows)), "dtype": dtype,
                "p": round(rng.uniform(0.01, 0.9), 3)}
    group = rng.choice([32, 64, 128])
    if op == "q4_quant":
        rows = _log(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": _log(rng, 1, min(16384, 60_000_000 // rows)), "dtype": dtype,
                "group": group}
    # layers: one token up to a batch of them, and K and N up to wide ones
    K, N = _log(rng, 8, 8192), _log(rng, 8, 8192)
    if rng.random() < 0.3:  # this framework's widths
        K, N = rng.choice([32, 64, 192, 256]), rng.choice([11, 56, 58, 64, 256])
    M = _log(rng, 1, 16) if rng.random() < 0.5 else _log(rng, 1, min(20_000, 30_000_000_000 // (K * N)))
    return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "group": group, "relu": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _indices(gen, case):
    """Indices of a call, one in fifty of them -1 (no entry: padding)."""
    n, V = case["n"], case["V"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["order"] == "frames":  # stored frame after frame
        i = torch.sort(u).values * V
    elif case["order"] == "zipf":  # as words are: the k-th most frequent about 1 / k as often, at places of no order
        i = torch.exp(u * math.log(V + 1.0)) - 1.0
        place = torch.randperm(V, generator=gen, device="cuda")
        i = place[i.long().clamp_(0, V - 1)]
    else:
        i = u * V
    i = i.long().clamp_(0, V - 1)
    i[torch.rand(n, generator=gen, device="cuda") < 0.02] = -1
    return i.to(torch.int32 if case["index"] == "i32" else torch.int64)


def _activations(gen, rows, cols, dtype):
    """Rows of different size, values of either sign."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    return x.mul_(torch.randn((rows, 1), generator=gen, device="cuda").mul_(0.5).exp_()).to(dtype)


def _weights(gen, n, k):
    w = torch.randn((n, k), generator=gen, device="cuda").mul_(1.0 / math.sqrt(k))
    return w.mul_(torch.randn((n, 1), generator=gen, device="cuda").mul_(0.3).exp_())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case), "seed": (int(seed) * 0x9E3779B97F4A7C15 + 0x123456789) % (1 << 62)}
    if op == "embed":
        V, D = case["V"], case["D"]
        s["index"] = _indices(gen, case)
        t = torch.randn((V, D), generator=gen, device="cuda").mul_(0.1)
        s["table"] = _mx4_pack(t) if case["table"] == "mx4" else t.to(DTYPES[case["table"]])
    elif op == "embed_bwd":
        s["index"] = _indices(gen, case)
        s["dy"] = _activations(gen, case["n"], case["D"], torch.float32).mul_(1e-2).to(DTYPES[case["dtype"]])
    elif op == "dropout":
        s["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["dtype"]])
    elif op == "q4_quant":
        s["w"] = _weights(gen, case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
    else:
        s["x"] = _activations(gen, case["M"], case["K"], DTYPES[case["dtype"]])
        s["codes"], s["words"] = _q4_pack(*_q4(_weights(gen, case["N"], case["K"]), case["group"]))
        s["bias"] = torch.randn(case["N"], generator=gen, device="cuda").mul_(0.1)
    if own:  # the handles that a program keeps
        from implicit_attribute_decode_amd import pipeline as P

        if op == "embed" and case["table"] == "mx4":
            s["table"] = P.Mx4Tensor(*s["table"], case["D"])
        if op == "q4_linear":
            s["q4"] = P.Q4Tensor(s["codes"], s["words"], case["K"], case["group"])
    return s


# ------------------------------------------------------------- plain forms


def _philox(c, key):
    """The four words (in 64-bit integers) of counters c, a list of four tensors of words."""
    m32 = 0xFFFFFFFF
    k0, k1 = key & m32, (key >> 32) & m32
    c0, c1, c2, c3 = c
    for _ in range(10):
        # the 64-bit products wrap to the right bits; the shift's copies of the sign are masked off
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & m32) ^ c1 ^ k0, b & m32, ((a >> 32) & m32) ^ c3 ^ k1, a & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return c0, c1, c2, c3


def _kept(rows, cols, p, seed, device):
    """[rows, cols] truth values: kept by dropout with probability 1 - p."""
    quads = (cols + 3) // 4
    r = torch.arange(rows, device=device).view(rows, 1).expand(rows, quads)
    q = torch.arange(quads, device=device).view(1, quads).expand(rows, quads)
    low, high = torch.full_like(q, OFFSET & 0xFFFFFFFF), torch.full_like(q, OFFSET >> 32)
    border = round(p * 2.0 ** 32)
    words = [w >= border for w in _philox([q, r, low, high], seed)]
    return torch.stack(words, -1).view(rows, 4 * quads)[:, :cols]


def _mx4_pack(x):
    """(codes, scales) of rows of x in MXFP4."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    v = torch.nn.functional.pad(x.float(), (0, blocks * 32 - cols)).view(rows, blocks, 32)
    e = (torch.frexp(v.abs().amax(-1, keepdim=True))[1] - 3).clamp_(-127, 125)
    u = v * torch.exp2(-e.float())
    a = u.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_(max=6.0)
    mag = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, a + 2.0, 0.5 * a + 4.0))
    c = (mag + 8.0 * torch.signbit(u)).to(torch.uint8).view(rows, -1)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), (e.squeeze(-1) + 127).to(torch.uint8).contiguous()


def _mx4_values(codes, scales, cols):
    """The 32-bit values that packed rows stand for."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 32)
    v = grid[c.int()] * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return v.view(codes.shape[0], -1)[:, :cols]


def _q4(w, group):
    """(q, z, s), [rows, groups, group or 1], of rows of w; in 64 bits, where borders between codes are decided exactly."""
    rows, cols = w.shape
    groups = (cols + group - 1) // group
    v = torch.nn.functional.pad(w.double(), (0, groups * group - cols)).view(rows, groups, group)
    lo, hi = v.amin(-1, keepdim=True).clamp_(max=0.0), v.amax(-1, keepdim=True).clamp_(min=0.0)
    s = (hi - lo) / 15.0
    m, e = torch.frexp(s)  # up to a whole number of 2^-16 of its power of two
    s = torch.ldexp(torch.ceil(m * 65536.0) / 65536.0, e)
    s = torch.where(hi > lo, s.clamp(min=2.0 ** -100), 0.0)
    d = torch.where(s > 0.0, s, 1.0)
    z = torch.round(-lo / d)
    return (torch.round(v / d) + z).clamp_(0.0, 15.0), z, s


def _q4_pack(q, z, s):
    """(codes bytes [rows, groups group / 2], words int32 [rows, groups rounded up to a multiple of 4])."""
    rows, groups, group = q.shape
    c = q.to(torch.uint8).view(rows, groups * group)
    words = s.float().view(torch.int32).view(rows, groups) | z.to(torch.int32).view(rows, groups)
    words = torch.nn.functional.pad(words, (0, -groups % 4))
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), words.contiguous()


def _q4_values(codes, words, cols, group):
    """The 32-bit values that packed rows stand for."""
    rows = codes.shape[0]
    q = torch.stack([codes & 15, codes >> 4], -1).view(rows, -1, group).float()
    w = words[:, :q.shape[1]].unsqueeze(-1)
    s = (w & ~255).view(torch.float32)
    return (s * (q - (w & 255).float())).view(rows, -1)[:, :cols]


def _plain_embed(s):
    c = s["case"]
    i = s["index"].long()
    there = ((i >= 0) & (i < c["V"])).unsqueeze(1)
    i = i.clamp(0, c["V"] - 1)
    rows = _mx4_values(s["table"][0][i], s["table"][1][i], c["D"]) if c["table"] == "mx4" else s["table"][i].float()
    rows = rows * (c["scale"] / (1.0 - c["p"]))
    if c["p"] > 0.0:
        there = there & _kept(c["n"], c["D"], c["p"], s["seed"], i.device)
    return torch.where(there, rows, 0.0).to(DTYPES[c["out"]])


def _plain_embed_bwd(s):
    c = s["case"]
    i = s["index"].long()
    there = (i >= 0) & (i < c["V"])
    d = s["dy"].float()
    if c["p"] > 0.0:
        d = torch.where(_kept(c["n"], c["D"], c["p"], s["seed"], i.device), d, 0.0)
    g = torch.zeros((c["V"] + 1, c["D"]), device=i.device)
    g.index_add_(0, torch.where(there, i, c["V"]), d)
    return g[:-1] * (c["scale"] / (1.0 - c["p"]))


def _plain_dropout(s):
    c = s["case"]
    y = s["x"].float() * (1.0 / (1.0 - c["p"]))
    return torch.where(_kept(c["rows"], c["cols"], c["p"], s["seed"], y.device), y, 0.0).to(s["x"].dtype)


def _plain_q4_quant(s):
    c = s["case"]
    q, z, scale = _q4(s["w"], c["group"])
    return (scale * (q - z)).view(c["rows"], -1)[:, :c["cols"]].to(s["w"].dtype)


def _plain_q4_linear(s):
    c = s["case"]
    y = s["x"].float() @ _q4_values(s["codes"], s["words"], c["K"], c["group"]).t() + s["bias"]
    return (y.relu_() if c["relu"] else y).to(s["x"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "dropout": _plain_dropout,
                "q4_quant": _plain_q4_quant, "q4_linear": _plain_q4_linear}[op](s)
    from implicit_attribute_decode_amd import pipeline as P

    drop = P.Dropout(c["p"], s["seed"], OFFSET) if c.get("p") else None
    if op == "embed":
        return P.embedding(s["table"], s["index"], scale=c["scale"], dtype=DTYPES[c["out"]], dropout=drop)
    if op == "embed_bwd":
        return P.embedding_backward(s["dy"], s["index"], c["V"], scale=c["scale"], dropout=drop)
    if op == "dropout":
        return drop(s["x"])
    if op == "q4_quant":
        return P.q4_quantize(s["w"], c["group"]).dequantize(s["w"].dtype)
    return P.q4_linear(s["x"], s["q4"], s["bias"], "relu" if c["relu"] else "none")


def work(case):
    op = case["op"]
    if op in ("embed", "embed_bwd"):
        n, V, D = case["n"], case["V"], case["D"]
        index = n * (8 if case["index"] == "i64" else 4)
        if op == "embed_bwd":
            return {"bytes": index + n * D * BYTES[case["dtype"]] + 4 * V * D, "flops": n * D}
        row = (D + 31) // 32 * 17 if case["table"] == "mx4" else D * BYTES[case["table"]]
        # rows picked again need not come from memory again: no more than the table, each row once
        return {"bytes": index + min(n, V) * row + n * D * BYTES[case["out"]], "flops": n * D}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * BYTES[case["dtype"]], "flops": n}
    packed = lambda r, k: r * ((k + case["group"] - 1) // case["group"]) * (case["group"] // 2 + 4)  # noqa: E731
    if op == "q4_quant":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * BYTES[case["dtype"]] + packed(case["rows"], case["cols"]), "flops": 4 * n}
    M, K, N = case["M"], case["K"], case["N"]
    return {"bytes": BYTES[case["dtype"]] * M * (K + N) + packed(N, K) + 4 * N, "flops": 2 * M * N * K}


# ------------------------------------------------ definitions in 64 bits


def _times(a, b):
    """(low, high) words of the product of words a (tensor) and b, from products of halves."""
    a0, a1, b0, b1 = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = a1 * b0 + ((a0 * b0) >> 16)
    low = (mid & 0xFFFF) + a0 * b1
    return ((low & 0xFFFF) << 16) | ((a0 * b0) & 0xFFFF), a1 * b1 + (mid >> 16) + (low >> 16)


def _exact_dropped(rows, cols, p, seed, device):
    """[rows, cols]: 1 / (1 - p) where kept, else 0, in 64 bits."""
    e = torch.arange(rows * ((cols + 3) // 4), device=device)
    state = [e % ((cols + 3) // 4), e // ((cols + 3) // 4), torch.zeros_like(e) + OFFSET % 2 ** 32,
             torch.zeros_like(e) + OFFSET // 2 ** 32]
    for i in range(10):
        low0, high0 = _times(state[0], 0xD2511F53)
        low1, high1 = _times(state[2], 0xCD9E8D57)
        keys = (seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        state = [high1 ^ state[1] ^ keys[0], low1, high0 ^ state[3] ^ keys[1], low0]
    dropped = torch.stack(state, 1).view(rows, -1)[:, :cols] < torch.round(torch.tensor(p * 2.0 ** 32, dtype=torch.float64))
    return (~dropped).double() / (1.0 - p)


def _exact_mx4(codes, scales, cols):
    c = codes.long()
    c = torch.stack([c % 16, c // 16], -1).view(codes.shape[0], -1)
    exponent, mantissa = (c // 2) % 4, c % 2
    v = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
    v = torch.where(c >= 8, -v, v)
    return (v.view(codes.shape[0], -1, 32) * torch.exp2(scales.double() - 127).unsqueeze(-1)).view(c.shape)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        i = s["index"].long()
        table = s["table"]
        if case["table"] == "mx4":
            table = _exact_mx4(table.codes, table.scales, case["D"]) if own else _exact_mx4(*table, case["D"])
        # an entry of zeros behind the last stands for every index that is none
        table = torch.cat([table.double(), torch.zeros((1, case["D"]), dtype=torch.float64, device=i.device)])
        out = table[torch.where((i < 0) | (i >= case["V"]), case["V"], i)] * case["scale"]
        return out * _exact_dropped(case["n"], case["D"], case["p"], s["seed"], i.device) if case["p"] else out
    if op == "embed_bwd":
        i = s["index"].long()
        d = s["dy"].double() * case["scale"]
        if case["p"]:
            d = d * _exact_dropped(case["n"], case["D"], case["p"], s["seed"], i.device)
        order = torch.argsort(i, stable=True)
        i, d = i[order], d[order]
        ends = torch.searchsorted(i, torch.arange(-1, case["V"], device=i.device), right=True)
        out = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=i.device)
        lengths = ends[1:] - ends[:-1]
        step = 0
        most = int(lengths.max())
        if most <= 4096:  # every entry's rows, one after the other
            while step < most:
                on = (lengths > step).nonzero().squeeze(1)
                out[on] += d[ends[:-1][on] + step]
                step += 1
            return out
        for v in (lengths > 0).nonzero().squeeze(1).tolist() if case["V"] <= 2000 else []:
            out[v] = d[int(ends[v]):int(ends[v + 1])].sum(0)
        return out if case["V"] <= 2000 else out.index_add_(0, i[ends[0]:], d[ends[0]:])
    if op == "dropout":
        return s["x"].double() * _exact_dropped(case["rows"], case["cols"], case["p"], s["seed"], s["x"].device)
    if op == "q4_quant":
        w, group = s["w"].double(), case["group"]
        out = torch.empty_like(w)
        for at in range(0, case["cols"], group):
            g = w[:, at:at + group]
            low, high = g.min(1, keepdim=True).values.clamp(max=0), g.max(1, keepdim=True).values.clamp(min=0)
            unit = (high - low) / 15
            power = torch.floor(torch.log2(torch.where(unit > 0, unit, 1.0)))
            power = power + (torch.exp2(power + 1) <= unit).double() - (torch.exp2(power) > unit).double()
            unit = torch.ceil(unit * torch.exp2(15 - power)) * torch.exp2(power - 15)
            unit = torch.where(high > low, unit.clamp(min=2.0 ** -100), torch.ones_like(unit))

            def nearest(a):  # ties to the even number
                f = torch.floor(a)
                return f + ((a - f > 0.5) | ((a - f == 0.5) & (f % 2 == 1))).double()

            zero = nearest(-low / unit)
            out[:, at:at + group] = unit * (torch.clamp(nearest(g / unit) + zero, 0, 15) - zero)
        return out
    codes, words, group = s["codes"].long(), s["words"].long() % 2 ** 32, case["group"]
    q = torch.stack([codes % 16, codes // 16], -1).view(case["N"], -1)
    each = words.repeat_interleave(group, dim=1)[:, :q.shape[1]]
    power, fraction = (each >> 23) % 256, (each % 2 ** 23) // 256 * 256
    scale = torch.where(power > 0, (1.0 + fraction.double() / 2 ** 23) * torch.exp2(power.double() - 127), 0.0)
    w = (scale * (q - each % 256))[:, :case["K"]]
    y = torch.matmul(s["x"].double(), w.t().contiguous()) + s["bias"].double()
    return torch.clamp(y, min=0.0) if case["relu"] else y
