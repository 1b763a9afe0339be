"""A captured product goes on in its own workspace after a larger call has made the
workspace grow: what is allocated since is not written."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


def test_replays_after_the_workspace_has_grown():
    q = gq()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    a = torch.randint(-9, 9, (64, 8192), device="cuda", generator=gen).to(torch.int8)
    b = torch.randint(-9, 9, (96, 8192), device="cuda", generator=gen).to(torch.int8)
    one, out = torch.ones(96, device="cuda"), torch.zeros(64, 96, device="cuda")
    ws = q.Workspace()
    call = lambda: q.gemm_i8(a, one[:64], b, one, out=out, ws=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    size = ws.buf.numel()
    big = torch.zeros(3000, 8192, dtype=torch.int8, device="cuda")
    q.gemm_i8(big, torch.ones(3000, device="cuda"), b, one, ws=ws)
    assert ws.buf.numel() > size
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.double(), a.double() @ b.double().t())
    assert all((t == 7).all() for t in others)
