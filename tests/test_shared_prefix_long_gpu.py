"""Chunks of many tokens behind a shared prefix, whose rows are joined token by token over
the whole GPU (from eight tokens a sequence and two rows a warp of 64 an SM on), against
float64.  Tolerances: packed_ref.check_forward."""
import random

import pytest
import torch

import exact_attention_11_gb300 as fa
from test_paged_prefill_gpu import check
from test_shared_prefix_gpu import draw, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def uneven(S, most, seed):
    """(new tokens, tokens behind the prefix): lengths over their logarithm, one of the
    longest, every fifth with more context than its own chunk."""
    r = random.Random(seed)
    lens = [most] + [round(most ** r.random()) for _ in range(S - 1)]
    r.shuffle(lens)
    return [(n, n + (r.randint(0, 300) if i % 5 == 0 else 0)) for i, n in enumerate(lens)]


@pytest.mark.parametrize("H,Hk", [(32, 8), (40, 1), (33, 3), (16, 16)])
def test_uneven_chunks(H, Hk):
    """A number of heads that a warp's share does not divide; sequences without new
    tokens, of no group, too short to share; rows of no sequence."""
    groups = [(1500, uneven(20, 700, 1) + [(0, 30), (5, None)]), (400, uneven(12, 500, 2))]
    x, out = run(groups, H, Hk, seed=H, loose=[(1, 333), (260, 900), (0, 5)], before=7, behind=9)
    T = x[0].shape[0]
    assert T >= 8 * 37 and T * H >= 2 * 64 * 152
    out = torch.full_like(out, 7.0)
    fa.paged_prefill_shared(*x, out=out)
    check(*x[:6], out)
    assert (out[:7] == 7).all() and (out[-9:] == 7).all()


@pytest.mark.parametrize("S", [130, 1024, 1030])
def test_many_sequences_with_long_chunks(S):
    """Numbered by a kernel of its own; up to 1024 sequences the merge searches a copy in
    shared memory, beyond the workspace."""
    r = random.Random(S)
    lens = [r.randint(1, 22) for _ in range(S - 1)] + [9 * S]
    assert sum(lens) >= 8 * S and sum(lens) * 8 >= 2 * 64 * 152
    run([(640, [(n, n) for n in lens])], 8, 4, seed=S)


def test_nothing_shared_and_everything_cut():
    """No rows to join; and a context that is cut without a prefix."""
    run([(10, uneven(8, 900, 3))], 32, 8, seed=1)
    run([(10, [(700, 700)] * 2)], 32, 1, seed=2, loose=[(650, 20000)])


def test_offsets_that_decrease_stay_inside():
    x = list(draw([(1000, uneven(10, 600, 4))], 32, 8, 5))
    T = x[0].shape[0]
    assert T >= 80 and T * 32 >= 2 * 64 * 152
    cu = x[5].clone()
    for bad in (cu.flip(0), torch.roll(cu, 3), (cu * 7919) % (T + 1) - 5, cu * 0 + T, cu * 0):
        fa.paged_prefill_shared(*x[:5], bad.int(), *x[6:])
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
    check(*x[:6], fa.paged_prefill_shared(*x))


def test_replayed_with_other_lengths():
    x = draw([(1000, [(100, 800)] * 10)], 32, 8, 6)
    n = fa.fa_paged_prefill_shared_workspace_bytes(10, 1000, 1, 32, 8, x[3].shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    fa.paged_prefill_shared(*x, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.paged_prefill_shared(*x, workspace=ws)
    for lens, prefix in (([100] * 10, 1000), ([1] * 9 + [700], 1000), ([0] * 10, 1000),
                         ([100] * 10, 0), ([500, 0, 0, 1, 2, 3, 4, 90, 300, 100], 999)):
        x[5].copy_(torch.tensor([0] + lens).cumsum(0).int())
        x[7].fill_(prefix)
        x[0].normal_()
        graph.replay()
        check(*x[:6], out)
        again = fa.paged_prefill_shared(*x, workspace=ws)
        T = sum(lens)
        assert torch.equal(again[:T], out[:T])


def test_sharing_costs_no_more_than_not_sharing():
    """32 chunks up to 300 tokens behind 4096: the longest chunk's rows, joined by its
    sequence's share of the warps, made it 1.2 of the call that shares nothing."""
    x = draw([(4096, uneven(32, 300, 7))], 32, 8, 7)
    n = fa.fa_paged_prefill_shared_workspace_bytes(32, x[0].shape[0], 1, 32, 8, x[3].shape[1])
    n2 = fa.fa_paged_prefill_workspace_bytes(32, x[0].shape[0], 32, 8, x[3].shape[1])
    ws = torch.empty(max(n, n2), dtype=torch.uint8, device=DEV)

    def time_us(call):
        call()
        times = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(5):
                call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 200)
        return min(times)

    shared = time_us(lambda: fa.paged_prefill_shared(*x, workspace=ws))
    alone = time_us(lambda: fa.paged_prefill(*x[:6], workspace=ws))
    assert shared < 1.08 * alone, (shared, alone)
