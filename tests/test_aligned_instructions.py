"""tcgen05.ld, setmaxnreg and the cluster's barrier are .aligned: every lane of a
warp executes them at once.  What lanes do by themselves before one ends in
__syncwarp().  Read from the source: a warp that comes apart may work, or not."""
import os
import re

import pytest


def _code(name):
    from quantized_gnn_message_gb300 import build
    with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
        return build._code_only(f.read())


def _body(code, head):
    """The function's statements, from its name's definition to its last brace."""
    at = re.search(head + r"\([^;{]*\) \{", code)
    assert at, head
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        i += 1
    return code[at.end():i - 1]


@pytest.mark.parametrize("function", ["put", "put_part"])
def test_the_epilogue_leaves_a_warp_together(function):
    body = _body(_code("gq_i8.cu"), r"__device__ __forceinline__ void " + function)
    ways = [body] + [body[:m.start()] for m in re.finditer(r"\breturn;", body)]
    for way in ways:
        assert way.rstrip().endswith("__syncwarp();"), way[-300:]


@pytest.mark.parametrize("name,kernels", [("gq_i8.cu", 2), ("gq_xent.cu", 1)])
def test_warps_that_gave_up_meet_before_the_clusters_barrier(name, kernels):
    """After a wait that gave up each lane reads the clock until the time is
    over: the lanes leave that loop one by one."""
    code = _code(name)
    loops = re.findall(r"while \(clock64\(\) - t0 < kDrainCycles\) \{\s*\}\s*\}\s*(\w+)\(\);\s*(\w+)\(\);", code)
    assert loops == [("__syncwarp", "cluster_sync")] * kernels
