"""Group normalization from two host threads at once, on streams and workspaces of
their own: a narrow call does not take shared memory from a wide one."""
import threading

import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide,narrow", [(8192, 64), (512, 8)])
def test_two_threads_of_different_widths(wide, narrow):
    """The wide one needs more than the 48 KB that a kernel has without asking (a
    warp a segment: 8 of them share a block's)."""
    q = gq()
    many = 2000 if wide <= 512 else 1
    work = []
    for d in (wide, narrow):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(d)
        x = torch.randn(4 * many, d, device="cuda", generator=gen)
        ptr = torch.arange(many + 1, device="cuda") * 4
        ws, s = q.Workspace(), torch.cuda.Stream()
        y, mean, rstd = q.group_norm_fwd(x, 2, ptr, max_rows=4, ws=ws)
        dx, dg, db = q.group_norm_bwd(y, x, 2, mean, rstd, ptr, max_rows=4, ws=ws)
        work.append((x, ptr, ws, s, (y, mean, rstd, dx, dg, db)))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def run(x, ptr, ws, s, want):
        try:
            out = [torch.empty_like(t) for t in want]
            with torch.cuda.stream(s):
                start.wait()
                for _ in range(1000):
                    q.group_norm_fwd(x, 2, ptr, max_rows=4, out=out[0], mean=out[1], rstd=out[2], ws=ws)
                    q.group_norm_bwd(out[0], x, 2, out[1], out[2], ptr, max_rows=4, dX=out[3], dgamma=out[4], dbeta=out[5],
                                     ws=ws)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(out, want)):
                failed.append("results differ")
        except Exception as e:  # noqa: BLE001 -- reported by the thread that asserts
            failed.append(repr(e))

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
