"""Failure paths of the packed and paged kernels, without a GPU fault: one CTA's
copies go missing (fa_debug_inject_fault), the bounded wait for them runs out after
about 2 s, the CTA unwinds, the host reads FA_ERR_TIMEOUT once, and the next call
gives the bits of a clean one."""
import time

import pytest
import torch

import exact_attention_11_gb300 as fa
from test_forward_packed_gpu import draw as draw_packed
from test_paged_prefill_gpu import draw as draw_paged

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def check(mode, call, same):
    clean = call()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    fa.fa_debug_inject_fault(mode)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert fa.fa_device_status() == -5 and fa.fa_device_status() == 0
    assert 1.0 < waited < 30.0
    again = call()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for i in same:
        assert torch.equal(clean[i], again[i])


@pytest.mark.parametrize("d", [64, 128])
def test_packed_forward(d):
    q, k, v, cu = draw_packed([300, 7, 900], 8, 2, d, BF16, seed=1)
    check(1, lambda: fa.forward_packed(q, k, v, cu), (0, 1))


def test_paged_prefill():
    x = draw_paged([5, 200, 1], [3000, 900, 5000], 8, 2, seed=2)
    check(1, lambda: (fa.paged_prefill(*x),), (0,))


@pytest.mark.parametrize("d", [64, 128])
def test_packed_backward(d):
    q, k, v, cu = draw_packed([300, 7, 900], 4, 4, d, BF16, seed=3)
    o, lse = fa.forward_packed(q, k, v, cu)
    do = torch.randn_like(o)
    # (dQ is a sum of atomic adds; dK and dV of ungrouped heads repeat exactly)
    check(2, lambda: fa.backward_packed(q, k, v, o, lse, do, cu), (1, 2))
