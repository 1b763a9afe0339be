"""Products of 8-bit integers whose result is written transposed (fewer rows
than a tile, fewer than columns), with one accumulator, several chunks of columns
and a last warp whose rows end within it.  u = 2^-24; bounds as for other scaled
products: (float)sum u, a product u, a fused product and sum u, half a step."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int8(n, k, seed):
    buf = torch.zeros(n, (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    buf[:, :k] = torch.randint(-128, 128, (n, k), device="cuda", generator=_gen(seed)).to(torch.int8)
    return buf[:, :k]


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(200, 777, 200), (255, 20001, 1024), (160, 1003, 256), (255, 257, 16), (129, 40001, 64),
                                   (97, 4100, 1000), (250, 60003, 130)])
def test_transposed_results_that_end_inside_a_warp(m, n, k, t):
    q = gq()
    a, b = _int8(m, k, 1), _int8(n, k, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sums = a.double() @ b.double().t()
    sa = torch.exp(torch.randn(m, device="cuda", generator=_gen(3))) / 1000
    sb = torch.exp(torch.randn(n, device="cuda", generator=_gen(4))) / 1000
    bias = torch.randn(n, device="cuda", generator=_gen(5))
    buf = torch.full((m + 1, n + 5), 3.0, dtype=t, device="cuda")
    want = sums * sa.double()[:, None] * sb.double()
    for act in (q.ACT_NONE, q.ACT_RELU):
        for _ in range(3):
            q.gemm_i8(a, sa, b, sb, bias, act, out=buf[:m, :n], dev_err=err)
        ref = want + bias.double()
        tol = 2.1 * U * want.abs() + U * ref.abs()
        if t != torch.float32:
            tol = tol + torch.finfo(t).eps / 2 * ref.abs().clamp(min=torch.finfo(t).tiny) * 1.01
        if act == q.ACT_RELU:
            ref = ref.clamp(min=0)
        assert ((buf[:m, :n].double() - ref).abs() <= tol).all()
        assert (buf[m] == 3.0).all() and (buf[:, n:] == 3.0).all()
    one = q.gemm_i8(a, torch.ones(m, device="cuda"), b, torch.ones(n, device="cuda"), dev_err=err)
    assert torch.equal(one, sums.float()) and err.item() == 0
