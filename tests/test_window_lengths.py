"""Windows and numbers of first tokens that a C int does not hold, through the Python
calls (no GPU needed: the calls have no sequences)."""
import pytest

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
