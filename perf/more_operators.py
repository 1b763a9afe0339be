"""The rest of a training step's dense operators, as a user calls them, with
plain forms to measure them against:

  adamw   one AdamW step over many tensors at once, the two moments held in 32
          bits or in 8-bit floats that share an exponent in blocks of 256
  linear  a linear layer whose products are of 8-bit integers, one scale for
          each row (token, node) and each output channel; forward with prepared
          weights, or forward and backward with everything quantized on the way
  gnorm   group normalization of a batch of graphs (channels last, a graph's
          nodes are consecutive rows) with an activation, forward and backward

`run` computes a pass in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where `own` is true, through
quantized_gnn_message_gb300.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
BLOCK = 256  # values that share an exponent in the 8-bit moments
M32 = 0xFFFFFFFF
M64 = 0xFFFFFFFFFFFFFFFF

# ------------------------------------------------------------------ cases --


def listed():
    return [
        # the weights of the tiny two-layer stack (64 -> 64 -> 32, normalization, 300 classes): a call of a few
        # microseconds, where launches and host time are all there is
        dict(name="adamw-tiny", op="adamw", count=5, largest=9600, smallest=64, p="f32", g="f32", bits=32),
        # a model of many layers: weights, biases and normalization weights of every size between 1 and a million
        dict(name="adamw-many-8bit", op="adamw", count=200, largest=1048576, smallest=1, p="bf16", g="bf16", bits=8),
        # full-precision weights of a class head and its layers, fp32 moments, bf16 gradients
        dict(name="adamw-large-32bit", op="adamw", count=12, largest=33554432, smallest=1000, p="f32", g="bf16",
             bits=32),
        # node embeddings of a large graph (131,072 x 1,024 the largest table) with 8-bit moments
        dict(name="adamw-large-8bit", op="adamw", count=4, largest=134217728, smallest=65536, p="f32", g="f32", bits=8),
        # scores of one node over 10,007 classes: the form for single rows, which reads the weights and little else
        dict(name="linear-one-row", op="linear", mode="infer", n=1, k=1024, out=10007, dtype="f32", act=False, pad=0),
        # hidden layer of the large graph (2.45M nodes, 256 -> 256) with bias and ReLU
        dict(name="linear-2.4m-infer", op="linear", mode="infer", n=2449029, k=256, out=256, dtype="f32", act=True,
             pad=0),
        # a training step of a layer of odd sizes, padded rows
        dict(name="linear-odd-train", op="linear", mode="train", n=5003, k=1000, out=777, dtype="bf16", act=False,
             pad=3),
        # the largest: 16,384 rows of width 1,024 scored against 65,536 classes
        dict(name="linear-largest", op="linear", mode="infer", n=16384, k=1024, out=65536, dtype="bf16", act=False,
             pad=0),
        # evaluation of a small batch of molecules: 128 graphs of about 25 nodes
        dict(name="gnorm-molecules", op="gnorm", mode="infer", s=128, n=3201, d=64, groups=8, dtype="f32", act="silu",
             pad=0),
        # training on a batch of mid-size graphs: 4,096 graphs of about 150 nodes, 256 channels in 32 groups
        dict(name="gnorm-batch-train", op="gnorm", mode="train", s=4096, n=614400, d=256, groups=32, dtype="bf16",
             act="silu", pad=0),
        # odd widths: groups of 51 channels, padded rows, some graphs without nodes
        dict(name="gnorm-odd-train", op="gnorm", mode="train", s=1000, n=60001, d=255, groups=5, dtype="f16", act="none",
             pad=2),
        # one large graph as one segment: statistics over 2.45M nodes
        dict(name="gnorm-2.4m-train", op="gnorm", mode="train", s=1, n=2449029, d=256, groups=16, dtype="f32",
             act="silu", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "linear", "gnorm"])
    if op == "adamw":
        count = _log(rng, 1, 400)
        largest = _log(rng, 64, 134217728 if count < 6 else 134217728 * 4 // count)
        return dict(op=op, count=count, largest=largest, smallest=_log(rng, 1, largest),
                    p=rng.choice(["f32", "f32", "bf16", "f16"]), g=rng.choice(["f32", "bf16", "f16"]),
                    bits=rng.choice([8, 32]))
    if op == "linear":
        k = _log(rng, 16, 8192)
        out = _log(rng, 1, 65536)
        mode = rng.choice(["infer", "infer", "train"])
        top = 16384 * 1024 * 65536 // (3 if mode == "train" else 1)
        n = _log(rng, 1, max(1, min(2449029, top // (k * out), 2449029 * 256 // max(k, out))))
        return dict(op=op, mode=mode, n=n, k=k, out=out, dtype=rng.choice(["f32", "bf16", "f16"]),
                    act=mode == "infer" and rng.random() < 0.5, pad=rng.choice([0, 0, 1, 3, 8]))
    groups = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    d = groups * max(2, _log(rng, 16, 2048) // groups)
    n = _log(rng, 64, max(64, 2449029 * 256 // d // 2))
    mode = rng.choice(["infer", "train"])
    return dict(op=op, mode=mode, s=_log(rng, 1, max(1, n // 16)), n=n, d=d, groups=groups,
                dtype=rng.choice(["f32", "bf16", "f16"]),
                act=rng.choice(["none", "silu"] if mode == "train" else ["none", "relu", "silu"]),
                pad=rng.choice([0, 0, 1, 2, 8]))


# ----------------------------------------------------------------- inputs --


def _sizes(c):
    """`count` tensor sizes from `largest` down to `smallest`, even steps of the logarithm, not round."""
    r = (c["smallest"] / c["largest"]) ** (1.0 / max(1, c["count"] - 1))
    return [c["largest"] if i == 0 else max(1, int(c["largest"] * r ** i) - i % 3) for i in range(c["count"])]


def _matrix(n, d, pad, dtype, gen, mul=1.0, row_scale=False):
    """n x d values in a buffer of row pitch d + pad."""
    buf = torch.empty(n, d + pad, dtype=dtype, device=DEV)
    x = torch.randn(n, d, device=DEV, generator=gen)
    if row_scale:  # rows of different spread around different centres, as aggregated features are
        x.mul_(0.5 + 1.5 * torch.rand(n, 1, device=DEV, generator=gen))
        x.add_(torch.randn(n, 1, device=DEV, generator=gen))
    buf[:, :d] = x.mul_(mul)
    return buf[:, :d]


def _starts(sizes):
    """First rows of the tensors in the flat buffers, rows of BLOCK values, and the number of rows."""
    total = 0
    at = []
    for n in sizes:
        at.append(total)
        total += -(-n // BLOCK)
    return at, total


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case=dict(case), op=case["op"])
    if case["op"] == "adamw":
        # the tensors lie in flat buffers, each from a multiple of BLOCK values on, zeros between them
        st.update(seed=(seed * 0x9E3779B97F4A7C15 + 99) & M64, step=1000, sizes=_sizes(case))
        st["rows"], total = _starts(st["sizes"])
        start = torch.tensor(st["rows"], device=DEV) * BLOCK
        end = start + torch.tensor(st["sizes"], device=DEV)
        at = torch.arange(total * BLOCK, device=DEV)
        used = at < end[torch.searchsorted(start, at, right=True) - 1]
        scale = used * torch.exp(torch.randn(total * BLOCK, device=DEV, generator=gen))  # gradients of different spread
        del at
        normal = torch.randn(total * BLOCK, device=DEV, generator=gen)
        st["p"] = (0.05 * used * normal).to(TYPES[case["p"]])
        st["g"] = (0.01 * scale * normal.normal_(generator=gen)).to(TYPES[case["g"]])
        st["m"] = 0.003 * scale * normal.normal_(generator=gen)
        st["v"] = 1e-4 * scale.square() * (0.2 + normal.uniform_(generator=gen))
        if case["bits"] == 8:
            st["m"], st["me"] = _encode(st["m"].view(-1, BLOCK), None, True)
            st["v"], st["ve"] = _encode(st["v"].view(-1, BLOCK), None, False)
            st["m"], st["v"] = st["m"].view(-1), st["v"].view(-1)
        return st
    if case["op"] == "linear":
        n, k, out, t = case["n"], case["k"], case["out"], TYPES[case["dtype"]]
        st["x"] = _matrix(n, k, case["pad"], t, gen, row_scale=True)
        w = torch.randn(out, k, device=DEV, generator=gen).mul_(math.sqrt(1.0 / k))
        st["bias"] = 0.1 * torch.randn(out, device=DEV, generator=gen)
        if case["mode"] == "infer":  # the weights are quantized once, rows 16-byte aligned
            codes, st["sw"] = _quantize(w)
            st["wq"] = torch.zeros(out, (k + 15) // 16 * 16, dtype=torch.int8, device=DEV)[:, :k]
            st["wq"].copy_(codes)
        else:
            st["w"] = w
            st["dy"] = _matrix(n, out, case["pad"], t, gen, mul=0.25)
        return st
    s, n, d = case["s"], case["n"], case["d"]
    # graphs of different sizes, some of them empty where there are many
    cuts = torch.randint(0, n + 1, (s - 1,), device=DEV, generator=gen)
    even = torch.arange(1, s, device=DEV) * n // s
    cuts = torch.where(torch.rand(s - 1, device=DEV, generator=gen) < 0.02, cuts, even + (cuts - n // 2) // (2 * s))
    cuts = cuts.clamp(0, n).sort()[0]
    st["ptr"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), n)])
    st["max_rows"] = int((st["ptr"][1:] - st["ptr"][:-1]).max())  # the loader that put the batch together knows it
    st["x"] = _matrix(n, d, case["pad"], TYPES[case["dtype"]], gen, row_scale=True)
    st["gamma"] = 1.0 + 0.2 * torch.randn(d, device=DEV, generator=gen)
    st["beta"] = 0.2 * torch.randn(d, device=DEV, generator=gen)
    if case["mode"] == "train":
        st["dy"] = _matrix(n, d, case["pad"], TYPES[case["dtype"]], gen, mul=0.25)
    return st


# ------------------------------------------------------------ plain forms --

LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01


def _mix32(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & M32
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def _noise(seed, step, nblocks):
    """The library's counter hash over (seed and step, block, position), 32 bits."""
    s = (seed + step * 0x9E3779B97F4A7C15) & M64
    key = _mix32(torch.tensor((s ^ (s >> 32)) & M32, dtype=torch.int64, device=DEV))
    row = _mix32(torch.arange(nblocks, dtype=torch.int64, device=DEV) ^ key)
    col = (torch.arange(BLOCK, dtype=torch.int64, device=DEV) * 0x9E3779B9) & M32
    return _mix32((row[:, None] + col) & M32)


def _pow2(e):
    """2^e as fp32 for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _times_pow2(x, e):
    """x 2^e for whole e in [-254, 254], by two exact products."""
    h = e // 2
    return x * _pow2(h) * _pow2(e - h)


def _encode(x, noise, signed):
    """8-bit floats of blocks of values, with the block's exponent byte: the
    first moment as sign, 4 exponent bits and 3 of mantissa (torch's
    float8_e4m3fn), the second (never negative) as 4 and 4.  Values are scaled by
    a power of two that brings the block's largest, of exponent field e (at least
    16), to [2^7, 2^8) or [2^8, 2^9), and rounded down or up at random; without
    noise to the nearest.  A second moment that is not 0 never becomes 0."""
    kept = 3 if signed else 4
    e = (x.abs().view(torch.int32) >> 23).amax(1).clamp(min=16, max=254)
    y = _times_pow2(x.abs(), (127 + (7 if signed else 8) - e)[:, None])
    low = y < 2.0 ** -6
    bits = torch.where(low, y + 2.0 ** -6, y).view(torch.int32)
    drop = 23 - kept
    add = 1 << (drop - 1) if noise is None else ((noise >> 12) if signed else (noise & 0x7FFFF)).to(torch.int32)
    code = ((bits + add) >> drop) - torch.where(low, 121 << kept, 120 << kept).to(torch.int32)
    if signed:
        code = code | torch.where(x < 0, 128, 0).to(torch.int32)
    else:
        code = torch.where(x > 0, code.clamp(min=1, max=255), torch.zeros_like(code))
    return code.to(torch.uint8), e.to(torch.uint8)


def _decode(code, e, signed):
    """The fp32 values of 8-bit codes in blocks."""
    c = code.to(torch.int32)
    kept = 3 if signed else 4
    a = c & 127 if signed else c
    normal = ((a + (120 << kept)) << (23 - kept)).view(torch.float32)
    y = torch.where(a < (1 << kept), a.float() * 2.0 ** (-6 - kept), normal)
    y = _times_pow2(y, (e.to(torch.int32) - 127 - (7 if signed else 8))[:, None])
    return torch.where((c & 128) > 0, -y, y) if signed else y


def _plain_adamw(st):
    c = st["case"]
    st["step"] += 1
    p, g = st["p"].float().view(-1, BLOCK), st["g"].float().view(-1, BLOCK)
    m, v = st["m"].view(-1, BLOCK), st["v"].view(-1, BLOCK)
    if c["bits"] == 8:
        m, v = _decode(m, st["me"], True), _decode(v, st["ve"], False)
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    c1, c2 = 1.0 - BETA1 ** st["step"], 1.0 - BETA2 ** st["step"]
    p = p * (1.0 - LR * DECAY) - (LR / c1) * m / (torch.sqrt(v) / math.sqrt(c2) + ADAM_EPS)
    st["p"] = p.to(st["p"].dtype).view(-1)
    if c["bits"] == 8:
        noise = _noise(st["seed"], st["step"], p.shape[0])
        m, st["me"] = _encode(m, noise, True)
        v, st["ve"] = _encode(v, noise, False)
        st["m"], st["v"] = m.view(-1), v.view(-1)
        return {"p": st["p"], "m": _decode(m, st["me"], True).to(torch.bfloat16).view(-1),
                "v": _decode(v, st["ve"], False).to(torch.bfloat16).view(-1)}
    st["m"], st["v"] = m.view(-1), v.view(-1)
    return {"p": st["p"], "m": st["m"], "v": st["v"]}


def _quantize(x):
    """The scale of each row, its largest value / 127 as fp32 holds it, and the
    whole numbers in [-127, 127] of them that are nearest, decided in 64 bits: of
    millions of quotients many lie next to a half."""
    x = x.float()
    scale = (x.abs().amax(1).double() / 127.0).float()
    wide = scale.double()[:, None]
    return torch.round(torch.where(wide > 0, x / wide, torch.zeros_like(wide))).float(), scale


def _product(qa, sa, qb, sb):
    return (qa @ qb.t()) * sa[:, None] * sb


def _plain_linear(st):
    c = st["case"]
    t = st["x"].dtype
    if c["mode"] == "infer":
        qx, sx = _quantize(st["x"])
        y = _product(qx, sx, st["wq"].float(), st["sw"]) + st["bias"]
        return {"y": (torch.where(y > 0, y, torch.zeros_like(y)) if c["act"] else y).to(t)}
    x, w, dy = st["x"].float(), st["w"], st["dy"].float()
    y = _product(*_quantize(x), *_quantize(w)) + st["bias"]
    dx = _product(*_quantize(dy), *_quantize(w.t()))
    dw = _product(*_quantize(dy.t()), *_quantize(x.t()))
    return {"y": y.to(t), "dx": dx.to(t), "dw": dw, "dbias": dy.sum(0, dtype=torch.float64).float()}


def _plain_gnorm(st):
    c = st["case"]
    s, n, d, groups = c["s"], c["n"], c["d"], c["groups"]
    ptr = st["ptr"]
    seg = torch.searchsorted(ptr[1:], torch.arange(n, device=DEV), right=True)
    count = ((ptr[1:] - ptr[:-1]) * (d // groups)).clamp(min=1).float()[:, None]

    def mean_of(rows):
        """Over a segment's rows and a group's channels."""
        sums = torch.zeros(s, groups, dtype=torch.float64, device=DEV)
        sums.index_add_(0, seg, rows.view(n, groups, -1).sum(2, dtype=torch.float64))
        return sums.float() / count

    def spread(stat):
        return stat[seg][:, :, None]

    x = st["x"].float().view(n, groups, -1)
    mean = mean_of(x)
    x = x - spread(mean)
    rstd = 1.0 / torch.sqrt(mean_of(x * x) + EPS)
    xhat = (x * spread(rstd)).view(n, d)
    del x
    z = xhat * st["gamma"] + st["beta"]
    if c["act"] == "relu":
        y = torch.where(z > 0, z, torch.zeros_like(z))
    elif c["act"] == "silu":
        gate = 1.0 / (1.0 + torch.exp(-z))
        y = z * gate
    else:
        y = z
    out = {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}
    if c["mode"] == "infer":
        return out
    dz = st["dy"].float()
    if c["act"] == "silu":
        dz = dz * (gate * (1.0 + z * (1.0 - gate)))
        del gate
    del y, z
    out["dgamma"] = (dz * xhat).sum(0, dtype=torch.float64).float()
    out["dbeta"] = dz.sum(0, dtype=torch.float64).float()
    dz = dz * st["gamma"]
    a, b = mean_of(dz), mean_of(dz * xhat)
    dx = (dz.view(n, groups, -1) - spread(a) - xhat.view(n, groups, -1) * spread(b)) * spread(rstd)
    out["dx"] = dx.view(n, d).to(st["x"].dtype)
    return out


# -------------------------------------------------------------------- run --


def _views(st, name):
    """The tensors of a flat buffer: values, or, for the exponents, one of each block."""
    if name in ("me", "ve"):
        return [st[name][r:r - (-n // BLOCK)] for r, n in zip(st["rows"], st["sizes"])]
    return [st[name][r * BLOCK:r * BLOCK + n] for r, n in zip(st["rows"], st["sizes"])]


def run(st):
    c = st["case"]
    if own:
        import quantized_gnn_message_gb300 as q
        if c["op"] == "adamw":
            opt = st.get("opt")
            if opt is None:  # the optimizer that the program keeps, resumed at its step
                state = [_views(st, name) for name in ("m", "v")]
                if c["bits"] == 8:
                    state += [_views(st, name) for name in ("me", "ve")]
                opt = st["opt"] = q.AdamW(_views(st, "p"), LR, (BETA1, BETA2), ADAM_EPS, DECAY,
                                          state_bits=c["bits"], seed=st["seed"], state=state, step=st["step"],
                                          grads=_views(st, "g"))
            opt.step()
            if c["bits"] == 32:
                return {"p": st["p"], "m": st["m"], "v": st["v"]}
            return {"p": st["p"], "m": q.adam_moment(st["m"], st["me"], False, torch.bfloat16),
                    "v": q.adam_moment(st["v"], st["ve"], True, torch.bfloat16)}
        if c["op"] == "linear":
            if c["mode"] == "infer":
                return {"y": q.linear_i8(st["x"], st["wq"], st["sw"], st["bias"],
                                         act=q.ACT_RELU if c["act"] else q.ACT_NONE)}
            y = q.linear_i8(st["x"], *q.quantize_i8(st["w"]), st["bias"])
            dx, dw, dbias = q.linear_i8_bwd(st["dy"], st["x"], st["w"])
            return {"y": y, "dx": dx, "dw": dw, "dbias": dbias}
        act = {"none": q.ACT_NONE, "relu": q.ACT_RELU, "silu": q.ACT_SILU}[c["act"]]
        y, mean, rstd = q.group_norm_fwd(st["x"], c["groups"], st["ptr"], st["gamma"], st["beta"], EPS, act=act,
                                         max_rows=st["max_rows"])
        if c["mode"] == "infer":
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dgamma, dbeta = q.group_norm_bwd(st["dy"], st["x"], c["groups"], mean, rstd, st["ptr"], st["gamma"],
                                             st["beta"], act=act, max_rows=st["max_rows"])
        return {"y": y, "mean": mean, "rstd": rstd, "dgamma": dgamma, "dbeta": dbeta, "dx": dx}
    if c["op"] == "adamw":
        return _plain_adamw(st)
    return _plain_linear(st) if c["op"] == "linear" else _plain_gnorm(st)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        # weights and moments read and written, gradients read; 8-bit moments also returned as bf16 values
        moments = 2 * (1 + 1 + 2) + 2 * 2 / BLOCK if case["bits"] == 8 else 2 * (4 + 4)
        return {"bytes": int(n * (2 * SIZE[case["p"]] + SIZE[case["g"]] + moments)), "flops": 20 * n}
    e = SIZE[case["dtype"]]
    if case["op"] == "linear":
        n, k, out = case["n"], case["k"], case["out"]
        if case["mode"] == "infer":
            return {"bytes": e * n * (k + out) + k * out + 8 * out, "flops": 2 * n * k * out}
        return {"bytes": 2 * e * n * (k + out) + 8 * k * out + 8 * out, "flops": 6 * n * k * out}
    n, d, stats = case["n"], case["d"], 8 * case["s"] * (case["groups"] + 1)
    if case["mode"] == "infer":
        return {"bytes": 2 * n * d * e + stats + 8 * d, "flops": 10 * n * d}
    # x and dy read, y and dx written (x is read by both halves, counted once)
    return {"bytes": 4 * n * d * e + stats + 16 * d, "flops": 32 * n * d}


# ------------------------------------------------------------- 64 bits -----


def _hash64(seed, step, b0, b1):
    """Noise words of blocks b0..b1, by the definition: 32-bit words, modular products."""
    def fin(v):
        for shift, mul in ((16, 0x85EBCA6B), (13, 0xC2B2AE35)):
            v = torch.bitwise_xor(v, torch.div(v, 1 << shift, rounding_mode="floor"))
            v = torch.remainder(v * (mul & 0xFFFF) + torch.remainder(v * (mul >> 16), 1 << 16) * (1 << 16), 1 << 32)
        return torch.bitwise_xor(v, torch.div(v, 1 << 16, rounding_mode="floor"))
    s = (seed + step * 11400714819323198485) % (1 << 64)
    k = fin(torch.full((1,), (s % (1 << 32)) ^ (s // (1 << 32)), dtype=torch.int64, device=DEV))
    rows = fin(torch.bitwise_xor(torch.arange(b0, b1, dtype=torch.int64, device=DEV), k))
    cols = torch.remainder(torch.arange(BLOCK, dtype=torch.int64, device=DEV) * 2654435769, 1 << 32)
    return fin(torch.remainder(rows.unsqueeze(1) + cols.unsqueeze(0), 1 << 32))


def _value64(code, e, mantissa, top):
    """What a code stands for: (1 + f / 2^mantissa) 2^(x - 7), or f 2^(-6 - mantissa) where x is 0, times 2^(e - 127 - top)."""
    c = code.double()
    sign = 1.0
    if mantissa == 3:
        sign = 1.0 - 2.0 * (c >= 128)
        c = torch.remainder(c, 128)
    x, f = torch.div(c, 1 << mantissa, rounding_mode="floor"), torch.remainder(c, 1 << mantissa)
    y = torch.where(x > 0, (1.0 + f / (1 << mantissa)) * torch.pow(2.0, x - 7.0), f * 2.0 ** (-6 - mantissa))
    return sign * y * torch.pow(2.0, e.double() - 127 - top).repeat_interleave(BLOCK)


def _rounded64(x, u, mantissa, top):
    """Values on the grid of a block's codes, x / step + u rounded down, in 64 bits."""
    rows = x.view(-1, BLOCK)
    largest = rows.abs().amax(1, keepdim=True)
    scale = torch.pow(2.0, top - torch.floor(torch.log2(largest.clamp(min=2.0 ** -111))))
    y = rows.abs() * scale
    step = torch.pow(2.0, torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - mantissa)
    q = torch.floor(y / step + u) * step
    if mantissa == 4:
        q = torch.where(rows > 0, q.clamp(min=2.0 ** -10, max=31 * 2.0 ** 4), q)
    return (torch.sign(rows) * q / scale).view(-1)


def _quantize64(x):
    scale = (x.abs().amax(1).double() / 127).float().double()  # what the operator stores, codes are multiples of it
    return torch.round(x.double() / scale.clamp(min=1e-300)[:, None]), scale


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        out = {name: torch.empty(st["p"].numel(), dtype=torch.float64, device=DEV) for name in ("p", "m", "v")}
        step = st["step"] + 1
        piece = 1 << 16  # blocks at a time
        for b0 in range(0, out["p"].numel() // BLOCK, piece):
            b1 = min(b0 + piece, out["p"].numel() // BLOCK)
            at = slice(b0 * BLOCK, b1 * BLOCK)
            p, g, m, v = (st[name][at].double() for name in ("p", "g", "m", "v"))
            if case["bits"] == 8:
                m = _value64(st["m"][at], st["me"][b0:b1], 3, 7)
                v = _value64(st["v"][at], st["ve"][b0:b1], 4, 8)
            m = BETA1 * m + (1 - BETA1) * g
            v = BETA2 * v + (1 - BETA2) * g.square()
            hat = (m / (1 - BETA1 ** step)) / (torch.sqrt(v / (1 - BETA2 ** step)) + ADAM_EPS)
            out["p"][at] = p - LR * (DECAY * p + hat)
            if case["bits"] == 8:
                h = _hash64(st["seed"], step, b0, b1)
                m = _rounded64(m, torch.div(h, 1 << 12, rounding_mode="floor").double() / (1 << 20), 3, 7)
                v = _rounded64(v, torch.remainder(h, 1 << 19).double() / (1 << 19), 4, 8)
            out["m"][at], out["v"][at] = m, v
        return out
    if case["op"] == "linear":
        if case["mode"] == "infer":
            qx, sx = _quantize64(st["x"])
            y = torch.matmul(qx, st["wq"].double().T)
            y.mul_(sx[:, None]).mul_(st["sw"].double()).add_(st["bias"].double())
            return {"y": y.clamp_(min=0.0) if case["act"] else y}

        def product(a, b):
            (qa, sa), (qb, sb) = _quantize64(a), _quantize64(b)
            return torch.matmul(qa, qb.T) * torch.outer(sa, sb)
        x, w, dy = st["x"].double(), st["w"].double(), st["dy"].double()
        return {"y": product(x, w) + st["bias"].double(), "dx": product(dy, w.T), "dw": product(dy.T, x.T),
                "dbias": dy.sum(0)}
    n, d, groups, s = case["n"], case["d"], case["groups"], case["s"]
    length = st["ptr"][1:] - st["ptr"][:-1]
    seg = torch.repeat_interleave(torch.arange(s, device=DEV), length)
    gamma, beta = st["gamma"].double(), st["beta"].double()
    rows = max(1, (1 << 27) // d)
    cells = (length * (d // groups)).clamp(min=1).double()[:, None]

    def totals(of):
        """Sums of of(first row, last row) over segments and groups."""
        t = torch.zeros(s, groups, dtype=torch.float64, device=DEV)
        for r in range(0, n, rows):
            v = of(r, min(n, r + rows))
            t.index_add_(0, seg[r:r + rows], v.reshape(len(v), groups, d // groups).sum(2))
        return t / cells

    def wide(stat, r, e):
        return stat[seg[r:e]].repeat_interleave(d // groups, dim=1)

    mean = totals(lambda r, e: st["x"][r:e].double())
    var = totals(lambda r, e: (st["x"][r:e].double() - wide(mean, r, e)).square())
    rstd = torch.rsqrt(var + EPS)

    def parts(r, e):
        xhat = (st["x"][r:e].double() - wide(mean, r, e)) * wide(rstd, r, e)
        z = xhat * gamma + beta
        return xhat, z, torch.sigmoid(z)

    def outer(r, e):
        xhat, z, gate = parts(r, e)
        dz = st["dy"][r:e].double()
        return xhat, dz * (gate + z * gate * (1 - gate)) if case["act"] == "silu" else dz

    out = {"y": torch.empty(n, d, dtype=torch.float64, device=DEV), "mean": mean, "rstd": rstd}
    for r in range(0, n, rows):
        e = min(n, r + rows)
        xhat, z, gate = parts(r, e)
        out["y"][r:e] = z * gate if case["act"] == "silu" else z.clamp(min=0) if case["act"] == "relu" else z
    if case["mode"] == "infer":
        return out
    out["dgamma"] = torch.zeros(d, dtype=torch.float64, device=DEV)
    out["dbeta"] = torch.zeros(d, dtype=torch.float64, device=DEV)
    out["dx"] = torch.empty(n, d, dtype=torch.float64, device=DEV)
    for r in range(0, n, rows):
        xhat, dz = outer(r, min(n, r + rows))
        out["dgamma"] += (dz * xhat).sum(0)
        out["dbeta"] += dz.sum(0)
    a = totals(lambda r, e: outer(r, e)[1] * gamma)
    b = totals(lambda r, e: torch.mul(*outer(r, e)) * gamma)
    for r in range(0, n, rows):
        e = min(n, r + rows)
        xhat, dz = outer(r, e)
        out["dx"][r:e] = wide(rstd, r, e) * (dz * gamma - wide(a, r, e) - xhat * wide(b, r, e))
    return out
