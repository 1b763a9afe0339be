"""8-bit moments over some hundred steps against 32-bit ones that see the same
gradients: rounded at random they are right in the mean, where a nearest code
would stand still (b2 = 0.999 moves a second moment by a thousandth of itself a
step, half a code is a thirty-second).

Over N values, each with its own noise, the mean of the differences lies within 6
sigma / sqrt(N) but for one chance in 10^8.  sigma: a rounding to a code of b bits
has a variance of at most (step / 2)^2, step <= 2^-b of the value, or the least step
of its block, and what t steps later is left of it is beta^t of it:
  sigma_T^2 <= 1.5 sum_t beta^(2 (T - t)) ((2^-b x_t)^2 + least^2) / 4
with x_t the 32-bit moment at step t (1.5: the 8-bit one's square, larger by its own
variance, below 0.5 here; its largest, which sets the least step, is within 1.5 of
the 32-bit one's).  fp32's own roundings are 1,000 times smaller.  Left out: a
block's largest second moments, which no code above 31/16 of a power of two rounds
up (its exponent is that of the largest value)."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

N, T, B1, B2 = 1 << 16, 300, 0.9, 0.999


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drift", [0.0, 0.5])
def test_moments_follow_those_of_32_bits(drift, t):
    q = gq()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(10 * drift))
    size = torch.exp(0.7 * torch.randn(N, device="cuda", generator=gen))
    p8, p32 = torch.zeros(N, device="cuda", dtype=t), torch.zeros(N, device="cuda", dtype=t)
    a = q.AdamW([p8], 1e-3, (B1, B2), weight_decay=0.0, state_bits=8, seed=11)
    b = q.AdamW([p32], 1e-3, (B1, B2), weight_decay=0.0)
    var = [torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2)]
    for _ in range(T):
        g = (size * (drift + torch.randn(N, device="cuda", generator=gen))).to(t)
        a.step([g])
        b.step([g])
        for k, (x, beta, bits, top) in enumerate(((b.m[0], B1, 3, 7), (b.v[0], B2, 4, 8))):
            x = x.double()
            # the least step: 2^(-6 - bits) where the block's largest is at least 2^top (half of it, at 1.5 times the largest)
            least = x.abs().view(-1, 256).amax(1, keepdim=True).expand(-1, 256).reshape(-1) * 1.5 * 2.0 ** (-6 - bits - top)
            var[k] = beta ** 2 * var[k] + 1.5 * ((2.0 ** -bits * x) ** 2 + least ** 2) / 4
    (m8,), (v8,) = a.moments()
    m32, v32 = b.m[0].double(), b.v[0].double()
    for k, diff, scale in ((0, (m8.double() - m32) * m32.sign(), m32.abs().mean()), (1, v8.double() / v32 - 1, v32)):
        sd = var[k].sqrt() if k == 0 else var[k].sqrt() / v32
        if k == 1:
            below = v32 < 0.25 * v32.view(-1, 256).amax(1, keepdim=True).expand(-1, 256).reshape(-1)
            diff, sd = diff[below], sd[below]
        bound = 6 * sd.square().mean().sqrt() / diff.numel() ** 0.5
        assert diff.mean().abs() <= bound + 1e-5 * (scale if k == 0 else 1), f"moment {k + 1}"
        assert bound <= (0.02 * scale if k == 0 else 0.02)  # a bound that says something
