"""AdamW: which calls count as steps, and which parameters are apart from one another."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("capturable", [False, True])
def test_a_step_that_launches_nothing_does_not_count(capturable):
    q = gq()
    p = [torch.ones(10, device="cuda"), torch.ones(4, device="cuda", dtype=torch.bfloat16)]
    opt = q.AdamW(p, lr=0.1, capturable=capturable)
    opt.step([None, None])
    assert opt.steps == 0 and (p[0] == 1).all()
    opt.set_lr(float("nan"))
    with pytest.raises(q.GQError):
        opt.step([torch.ones_like(t) for t in p])
    assert opt.steps == 0
    opt.set_lr(0.1)
    opt.step([torch.ones_like(p[0]), None])
    assert opt.steps == 1
    if capturable:
        assert opt.device_steps().item() == 1
    # the first step: m / (1 - b1) = g, v / (1 - b2) = g^2, so p falls by lr (and the decay)
    assert torch.allclose(p[0], torch.full_like(p[0], 1 - 0.1 * 0.01 - 0.1), rtol=1e-5)


def test_columns_of_one_buffer_are_parameters_of_their_own():
    """Blocks of columns of one matrix lie between one another's rows and overlap nowhere."""
    q = gq()
    buf = torch.randn(33, 50, device="cuda", generator=_gen(1))
    g = torch.randn(33, 50, device="cuda", generator=_gen(2))
    whole, want = buf.clone(), buf.clone()
    cuts = [(0, 7), (7, 20), (24, 50)]
    opt = q.AdamW([buf[:, a:b] for a, b in cuts] + [torch.ones(3, device="cuda")], lr=0.1)
    opt.step([g[:, a:b] for a, b in cuts] + [None])
    one = q.AdamW([want], lr=0.1)
    one.step([g])
    for a, b in cuts:
        assert torch.equal(buf[:, a:b], want[:, a:b])
    assert torch.equal(buf[:, 20:24], whole[:, 20:24])
    for bad in ([buf[:, :8], buf[:, 7:20]], [buf[:, :7], buf[1:, 6:9]], [buf[:, :7], buf[3:5].reshape(-1)],
                [buf[:, 40:], buf.view(-1)[50 * 5 + 45:50 * 5 + 50]], [buf[:, :7], buf, buf[:, 7:]],
                [buf[:, :7], buf[:, 10:12], buf[:, 3:4]], [buf[:, :7], buf.as_strided((16, 7), (100, 1), 7)]):
        with pytest.raises(q.GQError):
            q.AdamW(bad)
