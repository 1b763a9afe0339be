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
