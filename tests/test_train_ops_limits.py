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


def _up(x, m):
    return (x + m - 1) // m * m


@pytest.mark.parametrize("n,k,C", [(1, 1, 1), (1 << 24, 8, 47), (100_000, 256, 256), (131_072, 8, 131_072),
                                   (5_003, 100, 10_007), (300, 64, 257)])
def test_linear_xent_workspace_of_losses_is_what_the_header_says(L, n, k, C):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    N, t = _up(n, 256), (C + 255) // 256
    want = 2 * N * _up(k, 8) + 16 * N
    if t > 1:
        run = min(16, max(1, N // 256 * t // (4 * sms)))
        want += 4 * N + 16 * N * ((t + run - 1) // run)
    got = L.gq_linear_xent_workspace_bytes(n, k, C, 0)
    # counts of up to 256 blocks, counters and the padding of a dozen buffers to 256 bytes
    assert want <= got <= want + 16 * 256 + 1024
