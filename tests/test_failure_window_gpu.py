"""Failure paths of the windowed and shared-prefix kernels: the checks of
test_failure_packed_gpu."""
import pytest
import torch

import exact_attention_11_gb300 as fa
from test_failure_packed_gpu import check
from test_forward_packed_gpu import draw as draw_packed
from test_paged_prefill_gpu import draw as draw_paged
from test_shared_prefix_gpu import draw as draw_shared

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("d", [64, 128])
def test_packed_forward(d):
    q, k, v, cu = draw_packed([300, 7, 900], 8, 2, d, BF16, seed=1)
    check(1, lambda: fa.forward_packed_window(q, k, v, cu, 200, 4), (0, 1))


def test_paged_prefill():
    x = draw_paged([5, 200, 1], [3000, 900, 5000], 8, 2, seed=2)
    check(1, lambda: (fa.paged_prefill_window(*x, 2000, 4),), (0,))


@pytest.mark.parametrize("S", [30, 150])
def test_shared_prefix(S):
    x = draw_shared([(1500, [(1, 9 + i) for i in range(S)])], 8, 2, seed=3)
    check(1, lambda: (fa.paged_prefill_shared(*x),), (0,))


@pytest.mark.parametrize("d", [64, 128])
def test_packed_backward(d):
    q, k, v, cu = draw_packed([300, 7, 900], 4, 4, d, BF16, seed=3)
    o, lse = fa.forward_packed_window(q, k, v, cu, 200)
    do = torch.randn_like(o)
    check(2, lambda: fa.backward_packed_window(q, k, v, o, lse, do, cu, 200), (1, 2))
