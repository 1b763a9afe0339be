"""The training operators around the message-passing layers, as a user calls
them, with plain forms to measure them against:

  norm     layer normalization of node rows with the optional ReLU and dropout
           behind it, forward and backward (weight gradients included)
  dropout  counter-based dropout of features or of attention values; its
           backward is the same call on the gradient
  xent     softmax cross entropy of a linear classifier over many classes,
           loss and gradients, the logits never kept

`run` computes a pass in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where `own` is true, through
quantized_gnn_message_gb300.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
M32 = 0xFFFFFFFF

# ------------------------------------------------------------------ cases --


def listed():
    return [
        # the tiny GCN graph's hidden rows (1,024 nodes x 64): a call of a few
        # microseconds, where launches and host time are all there is
        dict(name="norm-tiny-train", op="norm", mode="train", n=1024, d=64, dtype="f32", act=False, p=0.5, pad=0),
        # evaluation pass of the 131k-node stack: normalization and ReLU, nothing kept for a backward pass
        dict(name="norm-131k-infer", op="norm", mode="infer", n=131072, d=256, dtype="f32", act=True, p=0.0, pad=0),
        # backward of normalization, ReLU and dropout over the large graph's hidden rows (2.45M x 256)
        dict(name="norm-2.4m-bwd", op="norm", mode="bwd", n=2449029, d=256, dtype="f32", act=True, p=0.5, pad=0),
        # wide rows in bf16, odd node count and width, padded row pitch: a training step without ReLU
        dict(name="norm-wide-train", op="norm", mode="train", n=30001, d=4099, dtype="bf16", act=False, p=0.1, pad=5),
        # dropout of a mini-batch of bf16 rows of an output layer's width (47), pitch 48
        dict(name="dropout-47-bf16", op="dropout", n=8191, d=47, dtype="bf16", p=0.5, pad=1),
        # attention dropout of the 1M-node GAT layer: 17.8M edges (self-loops included) x 4 heads
        dict(name="dropout-gat-edges", op="dropout", n=17825792, d=4, dtype="f32", p=0.6, pad=0),
        # feature dropout over the large graph's hidden rows
        dict(name="dropout-2.4m", op="dropout", n=2449029, d=256, dtype="f32", p=0.5, pad=0),
        # loss only, a small evaluation batch over a few classes
        dict(name="xent-small-eval", op="xent", n=1000, k=64, C=47, labelled=1.0, grad=False),
        # node classification on the large graph: 2.45M nodes, 47 classes, 8% of the nodes labelled
        dict(name="xent-2.4m-47", op="xent", n=2449029, k=256, C=47, labelled=0.08, grad=True),
        # classification over many classes with odd sizes and unlabelled rows
        dict(name="xent-odd", op="xent", n=5003, k=100, C=10007, labelled=0.6, grad=True),
        # every node an answer (link prediction over all nodes of the 131k-node graph), hidden width 256
        dict(name="xent-131k-classes", op="xent", n=16384, k=256, C=131072, labelled=1.0, grad=True),
        # the largest: 16k rows of width 1024 over 131,072 classes
        dict(name="xent-largest", op="xent", n=16384, k=1024, C=131072, labelled=1.0, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "dropout", "xent"])
    if op == "norm":
        # rows of 16 features and more: below, the backward pass is a
        # difference of nearly equal terms and says nothing about either side
        d = _log(rng, 16, 8192)
        n = _log(rng, 1, min(2449029, 2449029 * 256 // d))
        mode = rng.choice(["train", "infer", "bwd"])
        return dict(op=op, mode=mode, n=n, d=d, dtype=rng.choice(["f32", "bf16", "f16"]),
                    act=mode != "train" and rng.random() < 0.7,
                    p=0.0 if mode == "infer" else rng.choice([0.0, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)]),
                    pad=rng.choice([0, 0, 1, 5, 8]))
    if op == "dropout":
        d = _log(rng, 1, 2048)
        n = _log(rng, 1, min(17825792, 2449029 * 256 // d))
        return dict(op=op, n=n, d=d, dtype=rng.choice(["f32", "bf16", "f16"]),
                    p=rng.choice([0.1, 0.5, round(rng.uniform(0.01, 0.95), 3)]), pad=rng.choice([0, 0, 1, 3, 8]))
    k = _log(rng, 8, 1024)
    C = _log(rng, 16, 131072)
    top = 16384 * 1024 * 131072
    n = _log(rng, 1, max(1, min(2449029 if C <= 256 else 131072, top // (k * C), (1 << 31) // C)))
    return dict(op=op, n=n, k=k, C=C, labelled=rng.choice([1.0, 1.0, 0.6, 0.08]), grad=rng.random() < 0.75)


# ----------------------------------------------------------------- inputs --


def _matrix(n, d, pad, dtype, gen, mul=1.0, row_scale=False):
    """n x d values in a buffer of row pitch d + pad."""
    buf = torch.empty(n, d + pad, dtype=dtype, device=DEV)
    x = torch.randn(n, d, device=DEV, generator=gen)
    if row_scale:  # rows of different spread around different centres, as aggregated features are
        x.mul_(0.5 + 1.5 * torch.rand(n, 1, device=DEV, generator=gen))
        x.add_(torch.randn(n, 1, device=DEV, generator=gen))
    buf[:, :d] = x.mul_(mul)
    return buf[:, :d]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case=dict(case), op=case["op"], seed=(seed * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF)
    if case["op"] == "dropout":
        st["x"] = _matrix(case["n"], case["d"], case["pad"], TYPES[case["dtype"]], gen)
        return st
    if case["op"] == "norm":
        n, d, t = case["n"], case["d"], TYPES[case["dtype"]]
        st["x"] = _matrix(n, d, case["pad"], t, gen, row_scale=True)
        st["gamma"] = 1.0 + 0.2 * torch.randn(d, device=DEV, generator=gen)
        st["beta"] = 0.2 * torch.randn(d, device=DEV, generator=gen)
        if case["mode"] != "infer":
            st["dy"] = _matrix(n, d, case["pad"], t, gen, mul=0.25)
        if case["mode"] == "bwd":  # what the forward pass left: statistics, and the ReLU derivative as bits
            x = st["x"].float()
            st["mean"] = x.double().mean(1).float()
            x = x - st["mean"][:, None]
            st["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
            if case["act"]:
                z = x.mul_(st["rstd"][:, None]).mul_(st["gamma"]).add_(st["beta"]) > 0
                words = (d + 31) // 32
                full = torch.zeros(n, words * 32, dtype=torch.bool, device=DEV)
                full[:, :d] = z
                place = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
                bits = torch.empty(n, words, dtype=torch.int32, device=DEV)
                for r in range(0, n, 1 << 18):
                    w = (full[r:r + (1 << 18)].view(-1, words, 32) * place).sum(2)
                    bits[r:r + (1 << 18)] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
                st["relu_bits"] = bits
        return st
    n, k, C = case["n"], case["k"], case["C"]
    k8 = (k + 7) // 8 * 8
    # post-ReLU activations; class rows that give logits a spread of about 2
    st["x"] = torch.zeros(n, k8, dtype=torch.bfloat16, device=DEV)[:, :k]
    st["x"].copy_(torch.randn(n, k, device=DEV, generator=gen).relu_())
    st["w"] = torch.zeros(C, k8, dtype=torch.bfloat16, device=DEV)[:, :k]
    st["w"].copy_(torch.randn(C, k, device=DEV, generator=gen).mul_(2.0 * math.sqrt(2.0 / k)))
    u = torch.rand(n, device=DEV, generator=gen)
    st["labels"] = (u * u * C).long().clamp_(max=C - 1).to(torch.int32)  # frequent and rare classes
    m = max(1, int(round(n * case["labelled"])))
    if m < n:
        st["labels"][torch.randperm(n, device=DEV, generator=gen)[m:]] = -1  # unlabelled nodes
    st["scale"] = 1.0 / m  # the loss is a mean over the labelled nodes
    return st


# ------------------------------------------------------------ plain forms --


def _mix32(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & M32
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def _kept(seed, n, d, p):
    """[noise >= p] of the library's counter hash over (seed, row, column)."""
    s = (seed ^ (seed >> 32)) & M32
    key = _mix32(torch.tensor(s, dtype=torch.int64, device=DEV))
    row = _mix32(torch.arange(n, dtype=torch.int64, device=DEV) ^ key)
    col = (torch.arange(d, dtype=torch.int64, device=DEV) * 0x9E3779B9) & M32
    return (_mix32((row[:, None] + col) & M32) >> 9) >= math.ceil(p * (1 << 23))


def _drop(x, st, p):
    if p == 0.0:
        return x
    return torch.where(_kept(st["seed"], x.shape[0], x.shape[1], p), x * float(1.0 / (1.0 - p)), torch.zeros_like(x))


def _plain_norm_fwd(st, act, p):
    x = st["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None] * st["gamma"] + st["beta"]
    if act:
        y = torch.where(y > 0, y, torch.zeros_like(y))
    return _drop(y, st, p).to(st["x"].dtype), mean, rstd


def _plain_norm_bwd(st, mean, rstd, act, p):
    x, dz = st["x"].float(), _drop(st["dy"].float(), st, p)
    n, d = x.shape
    if act:
        c = torch.arange(d, device=DEV)
        on = (st["relu_bits"][:, c // 32] >> (c % 32).to(torch.int32)) & 1
        dz = torch.where(on > 0, dz, torch.zeros_like(dz))
    xhat = (x - mean[:, None]) * rstd[:, None]
    dgamma = (dz * xhat).sum(0, dtype=torch.float64).float()
    dbeta = dz.sum(0, dtype=torch.float64).float()
    g = dz * st["gamma"]
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - xhat * (g * xhat).mean(1)[:, None])
    return dx.to(st["x"].dtype), dgamma, dbeta


def _plain_xent(st, grad):
    x, w, lab = st["x"].float(), st["w"].float(), st["labels"].long()
    on = (lab >= 0) & (lab < w.shape[0])
    at = torch.where(on, lab, torch.zeros_like(lab))[:, None]
    z = x @ w.t()
    top = z.max(1)[0]
    e = torch.exp(z - top[:, None])
    s = e.sum(1)
    loss = torch.where(on, torch.log(s) + top - z.gather(1, at)[:, 0], torch.zeros_like(s))
    if not grad:
        return {"loss": loss}
    del z
    g = e.div_(s[:, None])
    g.scatter_add_(1, at, torch.full_like(s, -1.0)[:, None])
    g.mul_(torch.where(on, torch.full_like(s, st["scale"]), torch.zeros_like(s))[:, None])
    return {"loss": loss, "dx": (g @ w).to(st["x"].dtype), "dw": (g.t() @ x).to(st["w"].dtype)}


# -------------------------------------------------------------------- run --


def run(st):
    c = st["case"]
    if own:
        import quantized_gnn_message_gb300 as q
        if c["op"] == "dropout":
            return {"y": q.dropout(st["x"], c["p"], st["seed"])}
        if c["op"] == "xent":
            loss, dx, dw = q.linear_xent(st["x"], st["w"], st["labels"], scale=st["scale"], grad=c["grad"])
            return {"loss": loss, "dx": dx, "dw": dw} if c["grad"] else {"loss": loss}
        act = q.ACT_RELU if c["act"] else q.ACT_NONE
        if c["mode"] != "bwd":
            y, mean, rstd = q.layer_norm_fwd(st["x"], st["gamma"], st["beta"], EPS, act=act, p=c["p"],
                                             seed=st["seed"])
            if c["mode"] == "infer":
                return {"y": y, "mean": mean, "rstd": rstd}
            dx, dgamma, dbeta = q.layer_norm_bwd(st["dy"], st["x"], mean, rstd, st["gamma"], act=act, p=c["p"],
                                                 seed=st["seed"])
            return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        dx, dgamma, dbeta = q.layer_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"], act=act,
                                             p=c["p"], seed=st["seed"], relu_bits=st.get("relu_bits"))
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if c["op"] == "dropout":
        return {"y": _drop(st["x"].float(), st, c["p"]).to(st["x"].dtype)}
    if c["op"] == "xent":
        return _plain_xent(st, c["grad"])
    if c["mode"] == "bwd":
        dx, dgamma, dbeta = _plain_norm_bwd(st, st["mean"], st["rstd"], c["act"], c["p"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    y, mean, rstd = _plain_norm_fwd(st, c["act"], c["p"])
    if c["mode"] == "infer":
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = _plain_norm_bwd(st, mean, rstd, c["act"], c["p"])
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def work(case):
    if case["op"] == "xent":
        n, k, C = case["n"], case["k"], case["C"]
        m = max(1, int(round(n * case["labelled"])))
        b = 2 * m * k + 2 * C * k + 4 * n + 4 * n          # labelled rows, class rows, labels, loss
        if case["grad"]:
            b += 2 * n * k + 2 * C * k                     # both gradients
        return {"bytes": b, "flops": (6 if case["grad"] else 2) * m * k * C}
    n, d = case["n"], case["d"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "dropout":
        return {"bytes": 2 * n * d * e, "flops": n * d}
    if case["mode"] == "infer":
        return {"bytes": 2 * n * d * e + 8 * n + 8 * d, "flops": 8 * n * d}
    bwd = 3 * n * d * e + 8 * n + 12 * d + (4 * n * ((d + 31) // 32) if case["act"] else 0)
    if case["mode"] == "bwd":
        return {"bytes": bwd, "flops": 14 * n * d}
    # a step: x and dy read, y and dx written (x is read by both halves, counted once)
    return {"bytes": 4 * n * d * e + 8 * n + 16 * d, "flops": 22 * n * d}


# ------------------------------------------------------------- 64 bits -----


def _hash64(seed, r0, r1, d):
    """The 23-bit noise codes of rows r0..r1, by the definition: 32-bit words, modular products."""
    def fin(v):
        for shift, mul in ((16, 0x85EBCA6B), (13, 0xC2B2AE35)):
            v = torch.bitwise_xor(v, torch.div(v, 1 << shift, rounding_mode="floor"))
            v = torch.remainder(v * (mul & 0xFFFF) + torch.remainder(v * (mul >> 16), 1 << 16) * (1 << 16), 1 << 32)
        return torch.bitwise_xor(v, torch.div(v, 1 << 16, rounding_mode="floor"))
    k = fin(torch.full((1,), (seed % (1 << 32)) ^ (seed // (1 << 32)), dtype=torch.int64, device=DEV))
    rows = fin(torch.bitwise_xor(torch.arange(r0, r1, dtype=torch.int64, device=DEV), k))
    cols = torch.remainder(torch.arange(d, dtype=torch.int64, device=DEV) * 2654435769, 1 << 32)
    return torch.div(fin(torch.remainder(rows.unsqueeze(1) + cols.unsqueeze(0), 1 << 32)), 512, rounding_mode="floor")


def exact(case, seed):
    st = prepare(case, seed)
    f64 = dict(dtype=torch.float64, device=DEV)
    if case["op"] == "xent":
        n, C = case["n"], case["C"]
        w = st["w"].double()
        lab = st["labels"].long()
        loss, dx, dw = torch.zeros(n, **f64), torch.zeros(st["x"].shape, **f64), torch.zeros(w.shape, **f64)
        step = max(256, (1 << 29) // C)
        for r in range(0, n, step):
            x, y = st["x"][r:r + step].double(), lab[r:r + step]
            rows = torch.nonzero((y >= 0) & (y < C))[:, 0]
            if not rows.numel():
                continue
            x, y = x[rows], y[rows]
            z = torch.matmul(x, w.T)
            lse = torch.logsumexp(z, dim=1)
            loss[r + rows] = lse - z[torch.arange(len(rows), device=DEV), y]
            if case["grad"]:
                z = torch.exp(z - lse[:, None])
                z[torch.arange(len(rows), device=DEV), y] -= 1.0
                z *= st["scale"]
                dx[r + rows] = torch.matmul(z, w)
                dw += torch.matmul(z.T, x)
        return {"loss": loss, "dx": dx, "dw": dw} if case["grad"] else {"loss": loss}
    n, d = st["x"].shape
    p = case["p"]
    out = {}
    if case["op"] == "dropout":
        out["y"] = torch.zeros(n, d, **f64)
    else:
        if case["mode"] != "bwd":
            out.update(y=torch.zeros(n, d, **f64), mean=torch.zeros(n, **f64), rstd=torch.zeros(n, **f64))
        if case["mode"] != "infer":
            out.update(dx=torch.zeros(n, d, **f64), dgamma=torch.zeros(d, **f64), dbeta=torch.zeros(d, **f64))
    step = max(1, (1 << 27) // d)
    for r in range(0, n, step):
        e = min(n, r + step)
        x = st["x"][r:e].double()
        factor = 1.0
        if p > 0:
            factor = torch.where(_hash64(st["seed"], r, e, d).double() / (1 << 23) < p, 0.0, 1.0).double() / (1.0 - p)
        if case["op"] == "dropout":
            out["y"][r:e] = x * factor
            continue
        gamma, beta = st["gamma"].double(), st["beta"].double()
        if case["mode"] == "bwd":
            mean, rstd = st["mean"][r:e].double().unsqueeze(1), st["rstd"][r:e].double().unsqueeze(1)
        else:
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            rstd = torch.rsqrt(var + EPS)
        xhat = (x - mean) * rstd
        if case["mode"] != "bwd":
            y = xhat * gamma + beta
            out["y"][r:e] = (y.clamp(min=0.0) if case["act"] else y) * factor
            out["mean"][r:e], out["rstd"][r:e] = mean[:, 0], rstd[:, 0]
        if case["mode"] != "infer":
            dz = st["dy"][r:e].double() * factor
            if case["act"]:
                words = st["relu_bits"][r:e].long() % (1 << 32)
                gate = torch.stack([torch.div(words, 1 << j, rounding_mode="floor") % 2 for j in range(32)], dim=2)
                dz = dz * gate.reshape(e - r, -1)[:, :d]
            out["dgamma"] += (dz * xhat).sum(0)
            out["dbeta"] += dz.sum(0)
            dz = dz * gamma
            dot = (dz * xhat).mean(1, keepdim=True)
            out["dx"][r:e] = rstd * (dz - dz.mean(1, keepdim=True) - dot * xhat)
    return out
