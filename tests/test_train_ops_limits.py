"""Limits and workspaces of the training operators on the host, without a GPU:
every call below is refused before any CUDA call."""
import ctypes as C

import pytest

INVALID, UNSUPPORTED = 1, 2
FAKE = C.c_void_p(0x1000)


@pytest.fixture(scope="module")
def L():
    import quantized_gnn_message_gb300 as q
    from quantized_gnn_message_gb300 import build
    build.build()
    return q.lib()


@pytest.mark.parametrize("d", [2 ** 31 - 4095, 2 ** 31 - 8, 2 ** 31 - 1])
@pytest.mark.parametrize("ty", [0, 1, 2])
def test_dropout_refuses_columns_that_its_counters_pass_31_bits_on(L, d, ty):
    # a thread's next columns are up to 2,048 further: beyond 2^31 they would be negative
    assert L.gq_dropout(FAKE, ty, 1, d, d, 0.5, 1, FAKE, d, None) == UNSUPPORTED
    assert L.gq_dropout(FAKE, ty, 1, d, d, 1.5, 1, FAKE, d, None) == INVALID
