"""Argument checks of the windowed calls (no GPU needed)."""
import math

import pytest

import exact_attention_11_gb300 as fa
from exact_attention_11_gb300 import _build

NULL, P = None, 4096


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


FWD = dict(q=P, k=P, v=P, o=P, lse=P, cu_seqlens=P, num_seqs=0, total_tokens=10, num_heads=4,
           num_kv_heads=2, d=64, q_stride=256, k_stride=128, v_stride=128, scale=0.125, window=5,
           sinks=1)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=3, total_tokens=0), 0), (dict(lse=NULL, sinks=0), 0),
    (dict(window=(1 << 31) - 1, sinks=(1 << 31) - 1), 0),
    (dict(window=0), -1), (dict(window=-1), -1), (dict(sinks=-1), -1),
    (dict(q=NULL), -1), (dict(o=NULL), -1), (dict(cu_seqlens=NULL), -1),
    (dict(num_seqs=-1), -1), (dict(num_kv_heads=3), -1), (dict(scale=math.nan), -1),
    (dict(d=96), -2), (dict(num_heads=129, num_kv_heads=1, q_stride=129 * 64), -2),
    (dict(k=P + 8), -3), (dict(lse=P + 2), -3), (dict(q_stride=255), -1), (dict(v_stride=132), -3),
])
def test_forward_checks(lib, change, expect):
    a = {**FWD, **change}
    assert lib.fa_forward_packed_window(*a.values(), None) == expect
    assert lib.fa_forward_packed_window_f16(*a.values(), None) == expect


BWD = dict(q=P, k=P, v=P, o=P, dout=P, lse=P, dq=P, dk=P, dv=P, cu_seqlens=P, num_seqs=0,
           total_tokens=10, num_heads=4, num_kv_heads=2, d=64, q_stride=256, k_stride=128,
           v_stride=128, scale=0.125, window=5, sinks=1, workspace=NULL, workspace_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=3, total_tokens=0), 0),
    (dict(window=0), -1), (dict(sinks=-1), -1), (dict(dout=NULL), -1), (dict(lse=NULL), -1),
    (dict(dk=NULL), -1), (dict(num_kv_heads=3), -1), (dict(scale=0.0), -1), (dict(d=256), -2),
    (dict(dv=P + 8), -3), (dict(q_stride=260), -3),
    (dict(num_seqs=1), -1),                                       # needs a workspace
    (dict(num_seqs=1, workspace=P, workspace_bytes=64), -1),
    (dict(num_seqs=1, workspace=P + 4, workspace_bytes=1 << 30), -3),
    (dict(num_seqs=1 << 26), -2),
])
def test_backward_checks(lib, change, expect):
    assert lib.fa_backward_packed_window(*{**BWD, **change}.values(), None) == expect


def test_backward_workspace(lib):
    size = fa.fa_backward_packed_window_workspace_bytes
    whole = fa.fa_backward_packed_workspace_bytes
    for bad in ((0, 5, 4, 2, 64, 9, 0), (1, 0, 4, 2, 64, 9, 0), (1, 1, 4, 3, 64, 9, 0),
                (1, 1, 4, 2, 64, 0, 0), (1, 1, 4, 2, 64, 9, -1)):
        assert size(*bad) == 0
    # the table's second part is all that a window adds
    assert 0 < size(4, 9000, 8, 2, 64, 100, 0) - whole(4, 9000, 8, 2, 64) < 4096
    # first tokens need accumulators of dK and dV where heads are not shared
    assert size(4, 9000, 8, 8, 64, 100, 4) > size(4, 9000, 8, 8, 64, 100, 0) + 2 * 9000 * 8 * 64 * 4
    # no first tokens' far parts under a window over everything, or with very many of them
    assert size(4, 9000, 8, 2, 64, 9000, 4) == size(4, 9000, 8, 2, 64, 9000, 0)
    assert size(4, 9000, 8, 2, 64, 100, 5000) == size(4, 9000, 8, 2, 64, 100, 0)


CHUNK = dict(q=P, k_cache=P, v_cache=P, block_tables=P, context_lens=P, cu_seqlens=P, out=P,
             num_seqs=0, total_tokens=10, num_heads=4, num_kv_heads=2, head_size=128,
             block_size=16, num_blocks=8, max_num_blocks_per_seq=4, q_stride=512, scale=0.1,
             window=5, sinks=1, workspace=NULL, workspace_bytes=0)
LONG = dict(num_seqs=1, total_tokens=1, max_num_blocks_per_seq=4096, window=20000)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=2, total_tokens=0), 0),
    (dict(window=0), -1), (dict(sinks=-2), -1), (dict(k_cache=NULL), -1),
    (dict(block_tables=NULL), -1), (dict(out=NULL), -1), (dict(num_blocks=0), -1),
    (dict(head_size=64), -2), (dict(block_size=32), -2), (dict(q_stride=516), -3),
    (dict(v_cache=P + 8), -3),
    (dict(LONG), -1), (dict(LONG, workspace=P, workspace_bytes=64), -1),
    (dict(LONG, workspace=P + 8, workspace_bytes=1 << 30), -3),
])
def test_chunk_checks(lib, change, expect):
    assert lib.fa_paged_prefill_window(*{**CHUNK, **change}.values(), None) == expect


def test_chunk_workspace(lib):
    size = fa.fa_paged_prefill_window_workspace_bytes
    whole = fa.fa_paged_prefill_workspace_bytes
    for bad in ((0, 5, 4, 2, 100, 9, 0), (1, 0, 4, 2, 100, 9, 0), (1, 1, 4, 3, 100, 9, 0),
                (1, 1, 4, 2, 100, 0, 0), (1, 1, 4, 2, 100, 9, -1)):
        assert size(*bad) == 0
    # a window as long as the table is what the call without one needs; a short one less
    assert size(1, 1, 32, 8, 1024, 1 << 30, 0) == whole(1, 1, 32, 8, 1024)
    assert 0 < size(1, 1, 32, 8, 1024, 4096, 4) < whole(1, 1, 32, 8, 1024)
    assert size(1, 1, 32, 8, 1024, 64, 0) == 0                  # one partition
    assert size(113, 113, 32, 8, 1024, 4096, 4) == 0            # that many are not cut
