"""Argument checks of the packed and paged-chunk calls (no GPU needed)."""
import math

import pytest
import torch

import exact_attention_11_gb300 as fa
from exact_attention_11_gb300 import _build

NULL, P = None, 4096


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


FWD = dict(q=P, k=P, v=P, o=P, lse=P, cu_seqlens=P, num_seqs=0, total_tokens=10, num_heads=4,
           num_kv_heads=2, d=64, q_stride=256, k_stride=128, v_stride=128, scale=0.125, causal=1)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0),                                     # no sequences: nothing to do
    (dict(num_seqs=3, total_tokens=0), 0),
    (dict(lse=NULL), 0), (dict(d=128, q_stride=512, k_stride=256, v_stride=1024), 0),
    (dict(q=NULL), -1), (dict(o=NULL), -1), (dict(cu_seqlens=NULL), -1),
    (dict(num_seqs=-1), -1), (dict(total_tokens=-1), -1), (dict(num_heads=0), -1),
    (dict(num_kv_heads=0), -1), (dict(num_kv_heads=3), -1), (dict(scale=0.0), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(d=96), -2), (dict(d=256), -2),
    (dict(num_heads=129, num_kv_heads=1, q_stride=129 * 64), -2),      # group over 128
    (dict(total_tokens=1 << 29, num_heads=64, q_stride=4096), -2),     # rows past 32 bits
    (dict(k=P + 8), -3), (dict(lse=P + 2), -3), (dict(cu_seqlens=P + 1), -3),
    (dict(q_stride=255), -1), (dict(q_stride=260), -3), (dict(v_stride=132), -3),
])
def test_forward_checks(lib, change, expect):
    a = {**FWD, **change}
    assert lib.fa_forward_packed(*a.values(), None) == expect
    assert lib.fa_forward_packed_f16(*a.values(), None) == expect


CHUNK = dict(q=P, k_cache=P, v_cache=P, block_tables=P, context_lens=P, cu_seqlens=P, out=P,
             num_seqs=0, total_tokens=10, num_heads=4, num_kv_heads=2, head_size=128,
             block_size=16, num_blocks=8, max_num_blocks_per_seq=4, q_stride=512, scale=0.1,
             workspace=NULL, workspace_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=2, total_tokens=0), 0),
    (dict(k_cache=NULL), -1), (dict(block_tables=NULL), -1), (dict(context_lens=NULL), -1),
    (dict(cu_seqlens=NULL), -1), (dict(out=NULL), -1), (dict(num_blocks=0), -1),
    (dict(max_num_blocks_per_seq=0), -1), (dict(num_kv_heads=3), -1), (dict(scale=-1.0), -1),
    (dict(head_size=64), -2), (dict(block_size=32), -2),
    (dict(num_heads=130, num_kv_heads=1, q_stride=130 * 128), -2),
    (dict(v_cache=P + 8), -3), (dict(context_lens=P + 2), -3), (dict(q_stride=516), -3),
    (dict(q_stride=504), -1),
    (dict(num_seqs=1, total_tokens=1, max_num_blocks_per_seq=4096), -1),   # needs a workspace
    (dict(num_seqs=1, total_tokens=1, max_num_blocks_per_seq=4096, workspace=P,
          workspace_bytes=64), -1),
    (dict(num_seqs=1, total_tokens=1, max_num_blocks_per_seq=4096, workspace=P + 8,
          workspace_bytes=1 << 30), -3),
])
def test_chunk_checks(lib, change, expect):
    assert lib.fa_paged_prefill(*{**CHUNK, **change}.values(), None) == expect


def test_chunk_workspace(lib):
    size = fa.fa_paged_prefill_workspace_bytes
    assert size(0, 5, 4, 2, 100) == 0 and size(1, 0, 4, 2, 100) == 0
    assert size(1, 1, 4, 3, 100) == 0                       # heads that do not divide
    assert size(1, 1, 32, 8, 8) == 0                        # one partition
    assert size(64, 16384, 32, 8, 1024) == 0                # enough rows without a split
    n = size(1, 1, 32, 8, 1024)
    assert n > 0 and n % (32 * 130 * 4) == 0
    assert size(113, 113, 32, 8, 1024) == 0                 # that many sequences are not cut


BWD = dict(q=P, k=P, v=P, o=P, dout=P, lse=P, dq=P, dk=P, dv=P, cu_seqlens=P, num_seqs=0,
           total_tokens=10, num_heads=4, num_kv_heads=2, d=64, q_stride=256, k_stride=128,
           v_stride=128, scale=0.125, causal=1, workspace=NULL, workspace_bytes=0)


@pytest.mark.parametrize("change,expect", [
    (dict(), 0), (dict(num_seqs=2, total_tokens=0), 0),
    (dict(dout=NULL), -1), (dict(lse=NULL), -1), (dict(dv=NULL), -1), (dict(k=NULL), -1),
    (dict(num_kv_heads=3), -1), (dict(scale=0.0), -1), (dict(d=256), -2),
    (dict(dk=P + 8), -3), (dict(dout=P + 2), -3), (dict(k_stride=120), -1),
    (dict(num_seqs=1), -1),                                         # no workspace
    (dict(num_seqs=1, workspace=P, workspace_bytes=100), -1),
    (dict(num_seqs=1, workspace=P + 4, workspace_bytes=1 << 30), -3),
    (dict(num_seqs=1 << 24, num_heads=4), -2),                      # padded rows past 2^30
])
def test_backward_checks(lib, change, expect):
    assert lib.fa_backward_packed(*{**BWD, **change}.values(), None) == expect


def test_backward_workspace(lib):
    size = fa.fa_backward_packed_workspace_bytes
    assert size(0, 10, 4, 2, 64) == 0 and size(1, 10, 4, 3, 64) == 0
    # one padded block: dQ of 4 heads, dK and dV of 2, vectors, table entry
    assert size(1, 10, 4, 2, 64) == 4 * (128 * 64 * (4 + 2 * 2) + 4 * 256 + 4)
    assert size(1, 10, 4, 4, 64) == 4 * (128 * 64 * 4 + 4 * 256 + 4)


def test_helpers_take_every_argument_by_name():
    """The checks are reached (CPU tensors are refused there), whatever the order."""
    q, k = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128)
    pos, freq = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    cu, lse = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(4, 3)
    kc, vc = torch.zeros(5, 2, 16, 16, 8), torch.zeros(5, 2, 128, 16)
    prep = dict(positions=pos, inv_freq=freq, k=k, q=q)
    for name, args in [
            ("qk_norm_rope", prep),
            ("qk_norm_rope_cache", dict(prep, v=k, slots=pos.long(), k_cache=kc, v_cache=vc)),
            ("qk_norm_rope_backward", dict(prep, dk_out=k, dq_out=q)),
            ("forward_packed", dict(cu_seqlens=cu, v=k, k=k, q=q)),
            ("backward_packed", dict(cu_seqlens=cu, v=k, k=k, q=q, o=q, lse=lse, dout=q)),
            ("paged_prefill", dict(q=q.bfloat16(), k_cache=kc, v_cache=vc, cu_seqlens=cu,
                                   block_tables=cu[None], context_lens=cu[1:]))]:
        with pytest.raises(ValueError):
            getattr(fa, name)(**args)
        with pytest.raises(TypeError, match="missing"):
            getattr(fa, name)(**{a: x for a, x in args.items() if a not in ("q", "dq_out")})
