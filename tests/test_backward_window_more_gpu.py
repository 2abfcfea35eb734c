"""The windowed gradient where its preparation and its items of whole groups could go
wrong: very long documents, offsets that decrease, replays, two streams, lost copies.
Checks and bounds: those of test_backward_window_gpu."""
import pytest
import torch

import exact_attention_11_gb300 as fa
from test_backward_window_gpu import check, inputs
from test_failure_packed_gpu import check as check_lost

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


def draw_grouped(lens, window, sinks, seed, H=32, Hk=8, d=64):
    x = inputs(lens, H, Hk, d, window, sinks, seed)
    T, S = x[0].shape[0], len(lens)
    n = fa.fa_backward_packed_window_workspace_bytes(S, T, H, Hk, d, window, sinks)
    return x, torch.empty(n, dtype=torch.uint8, device=DEV)


def count_grouped(ws, T, S):
    """Key blocks whose items have all query heads of a group, from the workspace: the
    counts lie ahead of one word per padded block, which are the last."""
    blocks = T // 128 + S
    words = ws.view(torch.int32)
    return words[-blocks - 4:-blocks][2].item()


GROUPED = [([2500, 700, 1, 900], 40, 0), ([2500, 700, 129, 0, 900], 200, 4),
           ([64] * 30 + [3300, 900], 33, 130)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,window,sinks", GROUPED)
def test_items_with_all_heads_are_there(lens, window, sinks, d):
    (q, k, v, o, lse, do, cu), ws = draw_grouped(lens, window, sinks, 1, d=d)
    got = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks, workspace=ws)
    assert 0 < count_grouped(ws, q.shape[0], len(lens)) < q.shape[0] // 128 + len(lens)
    check(q, k, v, cu, o, lse, do, got, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_items_with_all_heads_and_decreasing_offsets(d):
    lens = [2500, 700, 1, 900]
    for sinks in (0, 4):
        (q, k, v, o, lse, do, cu), ws = draw_grouped(lens, 40, sinks, 2, d=d)
        for bad in ([4101, 0, 4101, 0, 4101], [3000, 100, 4101, 50, 4000],
                    [1 << 30, -5, 7, 0, 4101], [4101, 3000, 2000, 1000, 0]):
            cu2 = torch.tensor(bad, device=DEV).int()
            fa.backward_packed_window(q, k, v, o, lse, do, cu2, 40, sinks, workspace=ws)
            torch.cuda.synchronize()
            assert fa.fa_device_status() == 0
        got = fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, sinks, workspace=ws)
        assert count_grouped(ws, q.shape[0], len(lens)) > 0
        check(q, k, v, cu, o, lse, do, got, 40, sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_items_with_all_heads_replayed(d):
    """A graph's calls follow the lengths on the device: with most items of whole groups,
    with none, with one document, with no rows."""
    lens = [2500, 700, 1, 900]
    (q, k, v, o, lse, do, cu), ws = draw_grouped(lens, 40, 4, 3, d=d)
    fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 4, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 4, workspace=ws)
    counts = []
    for lens in ([2500, 700, 1, 900], [4101, 0, 0, 0], [5, 9, 100, 70], [0, 0, 0, 0],
                 [0, 2100, 2000, 1]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).int())
        q.normal_()
        fa.forward_packed_window(q, k, v, cu, 40, 4, out=o, lse=lse)
        graph.replay()
        counts.append(count_grouped(ws, 4101, 4))
        fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 4)
        check(q, k, v, cu, o, lse, do, got, 40, 4)
    assert counts[0] > 0 and counts[1] > 0 and counts[2] == counts[3] == 0 and counts[4] > 0


def test_items_with_all_heads_on_two_streams():
    """At the same time, each with its own workspace: both kernels with such items, and
    one whose items all have one head."""
    jobs = []
    shapes = ([2500, 700, 1, 900], 64), ([3000, 1000], 128), ([90, 300], 64)
    for i, (lens, d) in enumerate(shapes):
        x, ws = draw_grouped(lens, 40, 4, 4 + i, d=d)
        jobs.append((x, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for (q, k, v, o, lse, do, cu), ws, stream in jobs:
            with torch.cuda.stream(stream):
                outs.append(fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 4, workspace=ws))
        torch.cuda.synchronize()
        for ((q, k, v, o, lse, do, cu), _, _), got in zip(jobs, outs):
            check(q, k, v, cu, o, lse, do, got, 40, 4)
    assert [count_grouped(ws, x[0].shape[0], x[6].numel() - 1) > 0 for x, ws, _ in jobs] == \
        [True, True, False]


@pytest.mark.parametrize("d", [64, 128])
def test_items_with_all_heads_lose_their_copies(d):
    """The first CTA's first item is one of all heads (there are no first tokens)."""
    (q, k, v, o, lse, do, cu), ws = draw_grouped([2500, 700, 1, 900], 40, 0, 7, d=d)

    def call():
        return fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 0, workspace=ws)

    check_lost(2, call, ())
    got = call()
    assert count_grouped(ws, 4101, 4) > 0
    check(q, k, v, cu, o, lse, do, got, 40, 0)


@pytest.mark.parametrize("window", [400, 690])
@pytest.mark.parametrize("sinks", [0, 5, 400])
def test_a_window_over_every_document_gives_the_causal_bits(window, sinks):
    """dK and dV have one item a key block, as without a window: stored (no first tokens,
    or a window as long as all tokens), or added once to an accumulator of zeros."""
    q, k, v, o, lse, do, cu = inputs([400, 90, 200], 3, 3, 64, window, sinks, seed=3)
    a = fa.backward_packed(q, k, v, o, lse, do, cu)
    b = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
    check(q, k, v, cu, o, lse, do, b, window, sinks)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
