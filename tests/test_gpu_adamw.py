"""AdamW over many tensors against the formulas in 64 bits, and its 8-bit
moments against an integer restatement of their format.  u = 2^-24.

From given p, m, v, one step in fp32 (b, o = beta, 1 - beta rounded to fp32):
  m': u on the coefficient, the product and the sum: 3u (|b1 m| + |o1 g|) =: 3u A
  v': one more for g^2: 4u v'
  quotient lr1 m' / (sqrt(v') rs2 + eps): lr1 and its product 2u, sqrt of v' 2u + u,
      rs2 u, the sum u, the division 2 steps = 4u: 11u of it, with 3u A in m'
  p': coefficient u |p|, the fused sum u |p'|, half a step of the type
A factor 1.1 covers second-order terms.  grad_scale: g is rounded once more (u)."""
import numpy as np
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = [1, 7, 8, 255, 256, 257, 2048, 4095, 4096, 4097, 0, 10007]
LR, B1, B2, EPS, WD = 1e-2, 0.9, 0.999, 1e-8, 0.1


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _inputs(sizes, pt, gt, seed):
    gen = _gen(seed)
    r = lambda n, s: s * torch.randn(n, device="cuda", generator=gen)
    spread = [torch.exp(2 * r(n, 1.0)) for n in sizes]
    return ([r(n, 0.5).to(pt) for n in sizes], [(r(n, 0.1) * s).to(gt) for n, s in zip(sizes, spread)],
            [r(n, 0.05) * s for n, s in zip(sizes, spread)], [r(n, 0.1).square() * s * s for n, s in zip(sizes, spread)])


def _mix(h):
    h = h ^ (h >> np.uint32(16))
    h = (h * np.uint32(0x85EBCA6B)).astype(np.uint32)
    h = h ^ (h >> np.uint32(13))
    h = (h * np.uint32(0xC2B2AE35)).astype(np.uint32)
    return h ^ (h >> np.uint32(16))


def _noise(seed, step, block0, n):
    s = (seed + step * 0x9E3779B97F4A7C15) & (2 ** 64 - 1)
    key = _mix(np.array([(s ^ (s >> 32)) & 0xFFFFFFFF], np.uint32))
    i = np.arange(n)
    row = _mix((block0 + i // 256).astype(np.uint32) ^ key)
    with np.errstate(over="ignore"):
        return _mix((row + (i % 256).astype(np.uint32) * np.uint32(0x9E3779B9)).astype(np.uint32))


def _values(codes, exps, second):
    """The format's definition."""
    c = codes.astype(np.int64)
    bits, top = (4, 8) if second else (3, 7)
    sign = np.where((c >= 128) & (not second), -1.0, 1.0)
    if not second:
        c = c % 128
    x, f = c >> bits, c % (1 << bits)
    y = np.where(x > 0, (1 + f / 2.0 ** bits) * 2.0 ** (x - 7.0), f * 2.0 ** (-6 - bits))
    return sign * y * 2.0 ** (np.repeat(exps.astype(np.float64), 256)[:c.size] - 127 - top)


def _rounded(x, noise, second):
    """(values, exponents) that the moments x are rounded to, by real arithmetic."""
    n = x.size
    bits, top = (4, 8) if second else (3, 7)
    pad = np.zeros(-n % 256)
    rows = np.concatenate([x.astype(np.float64), pad]).reshape(-1, 256)
    big = np.abs(rows).max(1)
    e = np.clip(np.floor(np.log2(np.maximum(big, 2.0 ** -126))) + 127, 16, 254)
    scale = 2.0 ** (top + 127 - e)[:, None]
    y = np.abs(rows) * scale
    step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - bits)
    u = (noise % (1 << 19)) / 2.0 ** 19 if second else (noise >> np.uint32(12)) / 2.0 ** 20
    q = np.floor(y / step + np.concatenate([u, pad]).reshape(-1, 256)) * step
    if second:
        q = np.where(rows > 0, np.clip(q, 2.0 ** -10, 31 * 2.0 ** 4), q)
    return (np.sign(rows) * q / scale).reshape(-1)[:n], e.astype(np.uint8)


def _want(p, g, m, v, t, lr=LR, gs=1.0, extra=0):
    """(p, m, v) and their bounds in 64 bits."""
    p, g, m, v = p.double(), g.double() * gs, m.double(), v.double()
    f = lambda x: float(np.float32(x))
    m2 = B1 * m + (1 - B1) * g
    A = (B1 * m).abs() + ((1 - B1) * g).abs()
    v2 = B2 * v + (1 - B2) * g * g
    den = torch.sqrt(v2 / (1 - B2 ** t)) + EPS
    lr1 = lr / (1 - B1 ** t)
    upd = lr1 * m2 / den
    p2 = p * (1 - lr * WD) - upd
    e = extra
    return (p2, 1.1 * U * (p.abs() + p2.abs() + (11 + e) * upd.abs() + lr1 / den * (3 + e) * A), m2, 1.1 * (3 + e) * U * A,
            v2, 1.1 * (4 + 2 * e) * U * v2)


def _within(got, want, tol, what):
    if got.numel() == 0:
        return
    bad = (got.double() - want).abs() - tol
    assert torch.isfinite(got).all() and bad.max() <= 0, f"{what}: {bad.max().item()} over the bound"


def _half(t, x):
    return torch.finfo(t).eps / 2 * x.abs().clamp(min=torch.finfo(t).tiny) * 1.01


@pytest.mark.parametrize("gt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pt", ["f32", "bf16", "f16"])
def test_step_32bit(pt, gt):
    q = gq()
    p, g, m, v = _inputs(SIZES, TYPES[pt], TYPES[gt], 1)
    m0, v0, p0 = [t.clone() for t in m], [t.clone() for t in v], [t.clone() for t in p]
    opt = q.AdamW(p, LR, (B1, B2), EPS, WD, state=(m, v), step=41)
    opt.step(g)
    for i in range(len(p)):
        P, ptol, M, mtol, V, vtol = _want(p0[i], g[i], m0[i], v0[i], 42)
        _within(m[i], M, mtol, f"m {i}")
        _within(v[i], V, vtol, f"v {i}")
        _within(p[i], P, ptol + (_half(TYPES[pt], P) if pt != "f32" else 0), f"p {i}")


@pytest.mark.parametrize("pt,gt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_steps_8bit(pt, gt):
    """Three steps from nothing: codes, exponents and parameters."""
    q = gq()
    p, _, _, _ = _inputs(SIZES, TYPES[pt], TYPES[gt], 2)
    opt = q.AdamW(p, LR, (B1, B2), EPS, WD, state_bits=8, seed=77)
    for t in range(1, 4):
        _, g, _, _ = _inputs(SIZES, TYPES[pt], TYPES[gt], 10 + t)
        p0 = [x.clone() for x in p]
        m0, v0 = opt.moments()
        opt.step(g)
        m1, v1 = opt.moments()
        block0 = 0
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            P, ptol, _, _, _, _ = _want(p0[i], g[i], m0[i], v0[i], t)
            _within(p[i], P, ptol + (_half(TYPES[pt], P) if pt != "f32" else 0), f"p {i} step {t}")
            # the moments' update is three or four separately rounded fp32 operations
            G = g[i].float().cpu().numpy()
            f = np.float32
            M = m0[i].cpu().numpy() * f(B1) + G * f(1 - B1)
            V = v0[i].cpu().numpy() * f(B2) + (G * G) * f(1 - B2)
            noise = _noise(77, t, block0, n)
            for x, got, codes, exps, second in ((M, m1[i], opt.m[i], opt.m_exp[i], False),
                                                (V, v1[i], opt.v[i], opt.v_exp[i], True)):
                want, e = _rounded(x, noise, second)
                assert np.array_equal(exps.cpu().numpy(), e)
                assert np.array_equal(got.cpu().numpy().astype(np.float64), want), f"moment {i} step {t}"
                assert np.array_equal(_values(codes.cpu().numpy(), e, second), want)
            block0 += (n + 255) // 256


def test_moments_are_separate_roundings():
    """Products and their sum are rounded one by one: where b1 m and (1 - b1) g
    cancel, what is left is exactly 0, and no rounding error of a product."""
    q = gq()
    n = 1 << 16
    gen = _gen(31)
    g = torch.randn(n, device="cuda", generator=gen)
    o = np.float32(1.0 - B1)
    m0 = (-(g.cpu().numpy() * o) / np.float32(B1)).astype(np.float32)
    left = m0 * np.float32(B1) + g.cpu().numpy() * o
    m, v, p = torch.from_numpy(m0).cuda(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    q.AdamW([p], LR, (B1, B2), EPS, WD, state=([m], [v]), step=7).step([g])
    assert (left == 0).sum() > n // 4 and np.array_equal(m.cpu().numpy(), left)


def test_values_of_every_code():
    q = gq()
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(7).cuda()
    exps = torch.tensor([16, 100, 127, 128, 140, 200, 254], dtype=torch.uint8).cuda()
    for second in (False, True):
        want = _values(codes.cpu().numpy(), exps.cpu().numpy(), second)
        got = q.adam_moment(codes, exps, second).cpu().numpy().astype(np.float64)
        with np.errstate(over="ignore"):
            assert np.array_equal(got, want.astype(np.float32).astype(np.float64))
        short = q.adam_moment(codes[3:1000].clone(), exps[:4].clone(), second, torch.bfloat16)  # unaligned in no way
        assert short.dtype == torch.bfloat16 and short.shape == (997,)


def test_rounding_is_right_in_the_mean():
    """A constant moment rounded with 4,096 different seeds: each rounding has
    mean x and a variance of at most (step / 2)^2, so the mean of N is within 6
    step / (2 sqrt(N)) of x but for one chance in 10^8."""
    q = gq()
    n, N = 256, 4096
    p = torch.zeros(n, device="cuda")
    g = torch.linspace(0.001, 1.0, n, device="cuda")
    sums = torch.zeros(2, n, dtype=torch.float64, device="cuda")
    for seed in range(N):
        opt = q.AdamW([p.clone()], state_bits=8, seed=seed * 7919, betas=(0.9, 0.999))
        opt.step([g])
        m, v = opt.moments()
        sums[0] += m[0]
        sums[1] += v[0]
    for s, x, bits, top in ((sums[0], 0.1 * g.double(), 3, 16), (sums[1], 0.001 * g.double() ** 2, 4, 16)):
        step = 2.0 ** (torch.floor(torch.log2(x)) - bits)
        step = torch.maximum(step, 2.0 ** (torch.floor(torch.log2(x.max())) - 13 - bits))
        fine = x >= step  # smaller ones of the second moment are kept from 0
        assert ((s / N - x).abs() <= 6 * step / (2 * N ** 0.5) + 1e-6 * x)[fine].all()


def test_many_tensors_and_pitches():
    """More tensors than one launch takes; rows at a pitch; gradients left out."""
    q = gq()
    gen = _gen(5)
    p, g = [], []
    for i in range(600):
        if i % 5 == 3:
            r, c = 3 + i % 7, 1 + i % 37
            p.append(torch.randn(r, c + 3, device="cuda", generator=gen)[:, :c])
            g.append(torch.randn(r, c + 8 * (i % 2), device="cuda", generator=gen)[:, :c])
        else:
            n = 1 + (i * 37) % 3000
            p.append(torch.randn(n, device="cuda", generator=gen))
            g.append(None if i % 11 == 4 else torch.randn(n, device="cuda", generator=gen))
    whole = [t._base.clone() if t._base is not None else t.clone() for t in p]
    p0 = [t.clone() for t in p]
    opt = q.AdamW(p, LR, (B1, B2), EPS, WD)
    opt.step(g)
    for i, t in enumerate(p):
        if g[i] is None:
            assert torch.equal(t, p0[i])
            continue
        z = torch.zeros_like(p0[i])
        P, ptol, *_ = _want(p0[i], g[i], z, z, 1)
        _within(t, P, ptol, f"p {i}")
        if t._base is not None:
            assert torch.equal(t._base[:, t.shape[1]:], whole[i][:, t.shape[1]:])


def test_8bit_rows_at_a_pitch_equal_dense():
    q = gq()
    gen = _gen(6)
    a = torch.randn(37, 41, device="cuda", generator=gen)
    g = torch.randn(37, 41, device="cuda", generator=gen)
    b = torch.zeros(37, 48, device="cuda")[:, :41]
    b.copy_(a)
    gb = torch.zeros(37, 50, device="cuda")[:, :41]
    gb.copy_(g)
    x, y = q.AdamW([a], state_bits=8, seed=3), q.AdamW([b], state_bits=8, seed=3)
    for _ in range(2):
        x.step([g])
        y.step([gb])
    assert torch.equal(a, b) and torch.equal(x.m[0], y.m[0]) and torch.equal(x.v_exp[0], y.v_exp[0])


def test_mixed_types_share_an_optimizer():
    q = gq()
    gen = _gen(7)
    p = [torch.randn(1000, device="cuda", generator=gen).to(t) for t in (torch.float32, torch.bfloat16, torch.float32)]
    g = [torch.randn(1000, device="cuda", generator=gen).to(t) for t in (torch.float32, torch.bfloat16, torch.bfloat16)]
    p0 = [t.clone() for t in p]
    opt = q.AdamW(p, LR, (B1, B2), EPS, WD, grads=g)
    opt.step()
    for i in range(3):
        z = torch.zeros(1000, device="cuda")
        P, ptol, *_ = _want(p0[i], g[i], z, z, 1)
        _within(p[i], P, ptol + (_half(p[i].dtype, P) if i == 1 else 0), f"p {i}")


@pytest.mark.parametrize("bits", [8, 32])
def test_grad_scale(bits):
    q = gq()
    p, g, _, _ = _inputs([3000], torch.float32, torch.bfloat16, 8)
    p0 = p[0].clone()
    z = torch.zeros_like(p0)
    opt = q.AdamW(p, LR, (B1, B2), EPS, WD, state_bits=bits)
    bad = torch.tensor(float("inf"), device="cuda")
    opt.step(g, grad_scale=bad)
    assert torch.equal(p[0], p0) and not opt.m[0].any()
    opt.steps = 0
    opt.step(g, grad_scale=torch.tensor([0.37], device="cuda"))
    P, ptol, *_ = _want(p0, g[0], z, z, 1, gs=float(np.float32(0.37)), extra=1)
    _within(p[0], P, ptol, "p")


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_count(bits):
    """Three replays equal three eager steps; lr set between replays reaches the next."""
    q = gq()
    p, g, _, _ = _inputs([5000, 33], torch.float32, torch.float32, 9)
    a, b = [t.clone() for t in p], [t.clone() for t in p]
    x = q.AdamW(a, LR, state_bits=bits, seed=5, grads=g, capturable=True)
    y = q.AdamW(b, LR, state_bits=bits, seed=5, grads=g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.step()
    graph.replay()
    x.set_lr(2 * LR)
    graph.replay()
    for lr in (LR, LR, 2 * LR):
        y.set_lr(lr)
        y.step()
    torch.cuda.synchronize()
    assert x.device_steps().item() == 3
    for i in range(2):
        assert torch.equal(x.m[i], y.m[i]) and torch.equal(x.v[i], y.v[i])
        assert (a[i] - b[i]).abs().max() <= 4 * U * b[i].abs().max()
    # a step that is left out does not count
    x.step(grad_scale=torch.tensor(float("nan"), device="cuda"))
    assert x.device_steps().item() == 3


def test_another_stream_and_same_results():
    q = gq()
    outs = []
    for k in range(2):
        p, g, _, _ = _inputs([70000], torch.bfloat16, torch.bfloat16, 11)
        opt = q.AdamW(p, LR, state_bits=8, seed=1)
        s = torch.cuda.Stream() if k else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            opt.step(g)
        torch.cuda.synchronize()
        outs.append((p[0].clone(), opt.m[0].clone(), opt.v[0].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_second_moment_is_never_lost():
    """Gradients 10^6 times smaller than their block's largest keep a divisor."""
    q = gq()
    g = torch.full((512,), 1e-6, device="cuda")
    g[5] = 1.0
    p = torch.zeros(512, device="cuda")
    opt = q.AdamW([p], lr=1e-2, state_bits=8, weight_decay=0.0)
    for _ in range(20):
        opt.step([g])
    assert (opt.v[0] > 0).all() and p.abs().max() <= 20 * 1.2e-2  # |m| / sqrt(v) of 8-bit codes: at most 1 and a step


def test_extreme_values():
    q = gq()
    g = torch.zeros(1024, device="cuda")
    g[:256] = 1e-30
    g[256:512] = 1e18
    g[512:520] = float("nan")
    opt = q.AdamW([torch.ones(1024, device="cuda")], state_bits=8)
    opt.step([g])
    p = opt.params[0]
    assert torch.isfinite(p[:512]).all() and torch.isfinite(p[768:]).all() and torch.isnan(p[512:520]).all()


def test_refusals():
    q = gq()
    p = torch.zeros(10, device="cuda")
    with pytest.raises(q.GQError):
        q.AdamW([p], state_bits=16)
    with pytest.raises(q.GQError):
        q.AdamW([p, p])
    with pytest.raises(q.GQError):
        q.AdamW([p, p[3:]])
    with pytest.raises(q.GQError):
        q.AdamW([p.long()])
    with pytest.raises(q.GQError):
        q.AdamW([p.cpu()])
    with pytest.raises(q.GQError):
        q.AdamW([torch.zeros(4, 4, device="cuda").t()[:, :3]])
    with pytest.raises(q.GQError):
        q.AdamW([p], state=([p.clone()],))
    with pytest.raises(q.GQError):
        q.AdamW([p], state=([p.clone()], [torch.zeros(9, device="cuda")]))
    opt = q.AdamW([p])
    for g in (None, [], [torch.zeros(9, device="cuda")], [torch.zeros(10)], [torch.zeros(10, device="cuda").int()]):
        with pytest.raises(q.GQError):
            opt.step(g)
    with pytest.raises(q.GQError):
        opt.step([p.clone()], grad_scale=torch.ones(2, device="cuda"))
    assert opt.steps == 0 and not p.any()
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=float("nan"))):
        with pytest.raises(q.GQError):
            q.AdamW([p], **kw).step([p.clone()])
