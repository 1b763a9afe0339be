"""AdamW with 8-bit moments where values leave fp32's range."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_a_value_that_is_not_finite_leaves_its_block_alone(bad, off):
    """8-bit moments: the others of its 256 go on as if its gradient had been 0
    (off: unaligned, value by value).  A gradient of 1e30 is finite, its square
    is not: the second moments are left alone, the first ones' block is its own."""
    q = gq()
    n, at = 700, 300
    runs = []
    for value in (0.0, bad):
        buf = torch.zeros(n + 1, device="cuda")
        p = buf[off:n + off].normal_(generator=_gen(1))
        opt = q.AdamW([p], lr=1e-2, betas=(0.9, 0.99), state_bits=8, seed=3)
        steps = []
        for t in range(4):
            g = torch.randn(n, device="cuda", generator=_gen(10 + t))
            g[at] = 0.0
            if t == 1:
                g[at] = value
            opt.step([g])
            m, v = opt.moments()
            steps.append((p.clone(), m[0], v[0], opt.m_exp[0].clone(), opt.v_exp[0].clone()))
        runs.append(steps)
    rest = torch.arange(n, device="cuda") != at
    for t, (a, b) in enumerate(zip(*runs)):
        if t <= 1:  # the step itself
            assert torch.equal(a[2][rest], b[2][rest]) and torch.equal(a[4], b[4]), f"second moments, step {t}"
        if bad == 1e30:
            continue
        if t <= 1:
            assert torch.equal(a[1][rest], b[1][rest]) and torch.equal(a[3], b[3]), f"first moments, step {t}"
        if t <= 2:  # from equal moments
            assert torch.equal(a[0][rest], b[0][rest]), f"parameters, step {t}"
        if t == 2:
            # the lost moment is now one of its block's largest and may hold the exponent up:
            # two roundings of the same value, each within a step of its own
            for k, bits, top in ((1, 3, 134), (2, 4, 135)):
                least = 2.0 ** (torch.maximum(a[k + 2], b[k + 2]).double() - top - 6 - bits).repeat_interleave(256)[:n]
                step = torch.maximum(torch.maximum(a[k].abs(), b[k].abs()).double() * 2.0 ** -bits, least)
                assert ((a[k] - b[k]).abs().double() <= 2 * step)[rest].all(), f"moment {k} in the step after"
        assert torch.isnan(b[0][at]) == (t >= 1) and torch.isfinite(b[0][rest]).all()
        assert torch.isfinite(b[1]).all() and torch.isfinite(b[2]).all()
    # the second moment of the step in which it happened: the greatest code's value
    assert runs[1][1][2][at].double() == 2.0 ** (runs[1][1][4][at // 256].double() - 135) * 31 * 16


def test_a_block_without_a_finite_value():
    q = gq()
    p = torch.ones(512, device="cuda")
    opt = q.AdamW([p], state_bits=8)
    g = torch.full((512,), float("nan"), device="cuda")
    g[256:] = 1.0
    opt.step([g])
    assert torch.isnan(p[:256]).all() and torch.isfinite(p[256:]).all()
    m, v = opt.moments()
    assert torch.isfinite(m[0]).all() and torch.isfinite(v[0]).all() and (opt.m_exp[0][0] == 16) and (opt.v_exp[0][0] == 16)
