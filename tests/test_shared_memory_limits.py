"""A kernel's limit on dynamic shared memory belongs to the function and not to a
call: a library call sets it to a constant, the most that any call asks for.
Set to the call's own size, another host thread's narrower call between the
setting and the launch takes it away, and the launch is refused.  Read from the
source; the threads that meet there do so once in very many calls."""
import os
import re

import pytest

CONSTANT = re.compile(r"(k[A-Z]\w*|[A-Z0-9_]+|sizeof|int|float|size_t|bytes|smem_of|Shape)$")


@pytest.mark.parametrize("name,settings", [("gq_gnorm.cu", 1), ("gq_i8.cu", 2), ("gq_xent.cu", 1), ("gq_gemm.cu", 2)])
def test_limits_are_constants(name, settings):
    from quantized_gnn_message_gb300 import build
    with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"\s+", " ", build._code_only(f.read()))
    sizes = re.findall(r"cudaFuncAttributeMaxDynamicSharedMemorySize, (.*?)\)\);", code)
    assert len(sizes) == settings
    for size in sizes:
        # members of a template (Shape<CONV>::smem) are constants of the kernel too
        names = re.findall(r"[A-Za-z_]\w*", re.sub(r"::\w+", "", size))
        assert all(CONSTANT.match(n) for n in names), size
