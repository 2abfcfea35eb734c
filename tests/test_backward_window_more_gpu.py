"""The windowed gradient where its preparation and its items of whole groups could go
wrong: very long documents, offsets that decrease, replays, two streams, lost copies.
Checks and bounds: those of test_backward_window_gpu."""
import pytest
import torch

import exact_attention_11_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def time_us(call, n=5):
    call()
    times = []
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


@pytest.mark.parametrize("sinks", [0, 4])
def test_one_long_document_costs_what_many_short_ones_do(sinks):
    """No part of the call grows with the square of a document's length.  With one
    head and a short window, 2^22 tokens are no more work than as 1024 documents of 4096
    (fewer sequences to search); a loop over the blocks before each block took 1.2 times
    as long."""
    T, d, window = 1 << 22, 64, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (torch.randn(T, 1, d, device=DEV, dtype=BF16, generator=g) for _ in range(4))
    us = []
    for S in (1, 1024):
        cu = torch.arange(S + 1, dtype=torch.int32, device=DEV) * (T // S)
        o, lse = fa.forward_packed_window(q, k, v, cu, window, sinks)
        n = fa.fa_backward_packed_window_workspace_bytes(S, T, 1, 1, d, window, sinks)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        us.append(time_us(lambda: fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks,
                                                            workspace=ws)))
    assert fa.fa_device_status() == 0
    assert us[0] < 1.05 * us[1], us
