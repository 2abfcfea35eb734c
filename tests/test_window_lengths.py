"""Windows and numbers of first tokens that a C int does not hold, through the Python
calls (no GPU needed: the calls have no sequences)."""
import math

import numpy
import pytest
import torch

import exact_attention_11_gb300 as fa
from exact_attention_11_gb300 import _build
from test_window import BWD, CHUNK, FWD

HUGE = [1 << 31, 1 << 32, (1 << 32) + 5, 1 << 40, (1 << 63) - 1, 1 << 70]
CALLS = [(fa.fa_forward_packed_window, FWD), (fa.fa_forward_packed_window_f16, FWD),
         (fa.fa_backward_packed_window, BWD), (fa.fa_paged_prefill_window, CHUNK)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


@pytest.mark.parametrize("length", HUGE)
def test_lengths_past_an_int_see_everything(length):
    for call, a in CALLS:
        assert call(*{**a, "window": length}.values(), None) == 0
        assert call(*{**a, "sinks": length}.values(), None) == 0
    size = fa.fa_paged_prefill_window_workspace_bytes
    whole = fa.fa_paged_prefill_workspace_bytes(1, 1, 32, 8, 1024)
    assert size(1, 1, 32, 8, 1024, length, 0) == size(1, 1, 32, 8, 1024, 4096, length) == whole > 0
    size = fa.fa_backward_packed_window_workspace_bytes
    assert size(4, 9000, 8, 2, 64, length, 4) == size(4, 9000, 8, 2, 64, 9000, 4) > 0
    assert size(4, 9000, 8, 2, 64, 100, length) == size(4, 9000, 8, 2, 64, 100, 5000) > 0


@pytest.mark.parametrize("length", [-1, -(1 << 32) + 5, -(1 << 40), -(1 << 70)])
def test_negative_lengths_are_refused(length):
    for call, a in CALLS:
        for name in ("window", "sinks"):
            with pytest.raises(fa.FattnError):
                call(*{**a, name: length}.values(), None)
    assert fa.fa_paged_prefill_window_workspace_bytes(1, 1, 32, 8, 1024, length, 0) == 0
    assert fa.fa_backward_packed_window_workspace_bytes(4, 9000, 8, 2, 64, 100, length) == 0


@pytest.mark.parametrize("window,sinks", [(2.5, 0), (4.0, 0), (5, 0.9), (math.inf, 0),
                                          (math.nan, 0), ("5", 0), (5, None)])
def test_lengths_that_are_no_whole_numbers_are_refused(window, sinks):
    q, ints = torch.zeros(4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fa.forward_packed_window(q, q, q, ints, window, sinks),
                 lambda: fa.backward_packed_window(q, q, q, q, q, q, ints, window, sinks),
                 lambda: fa.paged_prefill_window(q, q, q, ints, ints, ints, window, sinks)):
        with pytest.raises(TypeError):
            call()
    for call, a in CALLS:
        with pytest.raises(TypeError):
            call(*{**a, "window": window, "sinks": sinks}.values(), None)


def test_whole_numbers_of_other_types_are_taken():
    for one in (numpy.int64(1), numpy.int32(1), torch.tensor(1)):
        for call, a in CALLS:
            assert call(*{**a, "window": one, "sinks": one}.values(), None) == 0
