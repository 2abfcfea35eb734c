"""Argument checks of the shared-prefix call (no GPU needed)."""
import math

import pytest

import exact_attention_11_gb300 as fa
from exact_attention_11_gb300 import _build

NULL, P = None, 4096


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


CALL = dict(q=P, k_cache=P, v_cache=P, block_tables=P, context_lens=P, cu_seqlens=P, cu_groups=P,
            prefix_lens=P, out=P, num_seqs=0, total_tokens=10, num_groups=1, num_heads=4,
            num_kv_heads=2, head_size=128, block_size=16, num_blocks=8,
            max_num_blocks_per_seq=4, q_stride=512, scale=0.1, workspace=NULL, workspace_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=2, total_tokens=0), 0),
    (dict(num_groups=0, cu_groups=NULL, prefix_lens=NULL), 0),
    (dict(cu_groups=NULL), -1), (dict(prefix_lens=NULL), -1), (dict(num_groups=-1), -1),
    (dict(k_cache=NULL), -1), (dict(context_lens=NULL), -1), (dict(out=NULL), -1),
    (dict(num_blocks=0), -1), (dict(num_kv_heads=3), -1), (dict(scale=math.inf), -1),
    (dict(num_groups=1025), -2), (dict(head_size=64), -2), (dict(block_size=32), -2),
    (dict(num_heads=130, num_kv_heads=1, q_stride=130 * 128), -2),
    (dict(cu_groups=P + 2), -3), (dict(prefix_lens=P + 1), -3), (dict(v_cache=P + 8), -3),
    (dict(q_stride=516), -3),
    (dict(num_seqs=1), -1),                                       # needs a workspace
    (dict(num_seqs=1, workspace=P, workspace_bytes=64), -1),
    (dict(num_seqs=1, workspace=P + 8, workspace_bytes=1 << 30), -3),
])
def test_checks(lib, change, expect):
    assert lib.fa_paged_prefill_shared(*{**CALL, **change}.values(), None) == expect


def test_workspace(lib):
    size = fa.fa_paged_prefill_shared_workspace_bytes
    for bad in ((0, 5, 1, 4, 2, 100), (1, 0, 1, 4, 2, 100), (1, 1, -1, 4, 2, 100),
                (1, 1, 1025, 4, 2, 100), (1, 1, 1, 4, 3, 100), (1, 1, 1, 4, 2, 0)):
        assert size(*bad) == 0
    row = 32 * (128 + 2) * 4
    assert size(1, 1, 0, 32, 8, 4) >= row             # one partial row each, and the plan
    assert size(1, 1, 1, 32, 8, 4) >= 2 * row
    # many rows: one partial row of the context and one of the prefix all the same
    assert size(8, 65536, 1, 32, 8, 4096) >= 65536 * 2 * row
    assert size(256, 256, 1, 32, 8, 4096) < (300 << 20)
