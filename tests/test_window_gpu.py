"""Sliding windows and first tokens that stay visible: packed prompts and chunks over
the paged cache, against float64.  Tolerances: packed_ref.check_forward."""
import pytest
import torch

import exact_attention_11_gb300 as fa
import packed_ref
import window_ref as ref
from test_forward_packed_gpu import draw
from test_paged_prefill_gpu import draw as draw_paged

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


def check(q, k, v, cu, o, lse, window, sinks, scale=None):
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = scale or q.shape[-1] ** -0.5
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        see = ref.near(torch.arange(b - a, device=DEV), b - a, window, sinks)
        r = ref.sequence(q[a:b], k[a:b], v[a:b], scale, see)
        packed_ref.check_forward(o[a:b], None if lse is None else lse[:, a:b], r, scale, q.dtype)


def run(lens, H, Hk, d, dtype, window, sinks, seed, **kw):
    q, k, v, cu = draw(lens, H, Hk, d, dtype, seed, **kw)
    o, lse = fa.forward_packed_window(q, k, v, cu, window, sinks)
    check(q, k, v, cu, o, lse, window, sinks)


WINDOWS = [(1, 0), (1, 1), (7, 0), (64, 4), (127, 128), (128, 1), (129, 127), (130, 129),
           (200, 300), (256, 0), (1000, 4)]


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, d, dtype):
    """Windows and first tokens at the tiles' edges, sequences shorter and longer."""
    run([1, 130, 0, 700, 33, 513, 128], 4, 2, d, dtype, window, sinks, seed=window + sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 2), (6, 2), (7, 1), (10, 2), (16, 1), (40, 1),
                                  (128, 1)])
def test_heads(H, Hk, d):
    for window, sinks in ((33, 0), (100, 5), (300, 200)):
        run([1, 130, 0, 464, 33], H, Hk, d, BF16, window, sinks, seed=H + d)


def test_every_window_and_length():
    """Windows 1 .. 270 with changing first tokens; lengths 1 .. 270 in one call."""
    lens = list(range(1, 271))
    q, k, v, cu = draw(lens, 1, 1, 64, BF16, 5)
    for window in (1, 2, 63, 64, 65, 127, 128, 129, 191, 255, 257):
        o, lse = fa.forward_packed_window(q, k, v, cu, window, window % 7)
        check(q, k, v, cu, o, lse, window, window % 7)
    q, k, v, cu = draw([400], 1, 1, 64, BF16, 6)
    for window in range(1, 271):
        o, lse = fa.forward_packed_window(q, k, v, cu, window, window // 2)
        check(q, k, v, cu, o, lse, window, window // 2)


@pytest.mark.parametrize("H,Hk,d", [(8, 2, 128), (12, 4, 64)])
def test_many_items_per_sm(H, Hk, d):
    run([3100, 1, 257, 2049, 640, 5, 1500, 5000], H, Hk, d, BF16, 500, 4, seed=9)


@pytest.mark.parametrize("S", [112, 113, 1025])
def test_many_sequences(S):
    """Sequences whose numbering fits the kernel's table, and more."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, 300 if S < 200 else 20, (S,), generator=g).tolist()
    run(lens, 2, 1, 64, BF16, 40, 3, seed=S)


@pytest.mark.parametrize("sinks", [0, 5, 1 << 40])
def test_a_window_over_everything_is_the_causal_mask(sinks):
    """Bit for bit: the same tiles in the same order."""
    for d in (64, 128):
        q, k, v, cu = draw([700, 129, 1, 900], 4, 2, d, BF16, seed=d)
        a = fa.forward_packed(q, k, v, cu)
        for window in (900, 901, 1 << 40):
            b = fa.forward_packed_window(q, k, v, cu, window, sinks)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = draw_paged([40, 1, 7, 0, 33], [40, 100, 3000, 50, 34], 8, 2, seed=2)
    assert torch.equal(fa.paged_prefill(*x), fa.paged_prefill_window(*x, 1 << 31, sinks))


def test_first_tokens_over_everything_are_the_causal_mask():
    q, k, v, cu = draw([700, 129, 1, 900], 4, 2, 64, BF16, seed=4)
    o, lse = fa.forward_packed_window(q, k, v, cu, 1, 900)
    check(q, k, v, cu, o, lse, 1 << 20, 0)


def test_rows_of_no_sequence_stay_and_do_not_leak():
    q, k, v, cu = draw([100, 445], 4, 2, 128, BF16, seed=3, before=37, behind=200)
    o = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    lse = torch.full((4, q.shape[0]), 7.0, device=DEV)
    fa.forward_packed_window(q, k, v, cu, 50, 2, out=o, lse=lse)
    check(q, k, v, cu, o, lse, 50, 2)
    for rows in (slice(0, 37), slice(582, None)):
        assert (o[rows] == 7).all() and (lse[:, rows] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_sequences_do_not_mix(bad):
    lens = [200, 3, 129, 40, 257, 1, 385, 64, 5, 130, 66]
    q, k, v, cu = draw(lens, 6, 2, 64, BF16, seed=44)
    o, lse = fa.forward_packed_window(q, k, v, cu, 70, 3)
    ends = cu.tolist()
    for s in range(1, len(lens), 2):
        for x in (q, k, v):
            x[ends[s]:ends[s + 1]] = bad
    o2, lse2 = fa.forward_packed_window(q, k, v, cu, 70, 3)
    for s in range(0, len(lens), 2):
        rows = slice(ends[s], ends[s + 1])
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])


def test_keys_out_of_sight_do_not_count():
    """Huge keys outside every window and not among the first tokens."""
    q, k, v, cu = draw([600], 2, 2, 64, BF16, seed=8)
    o, lse = fa.forward_packed_window(q, k, v, cu, 100, 3)
    k[3:300] *= 1e4
    o2, lse2 = fa.forward_packed_window(q, k, v, cu, 100, 3)
    assert torch.equal(o[399:], o2[399:]) and torch.equal(lse[:, 399:], lse2[:, 399:])


def test_scores_without_a_finite_one():
    """A row whose visible scores are all -inf is NaN, as without a window."""
    q, k, v, cu = draw([300], 1, 1, 64, BF16, seed=8)
    q[:] = 1.0
    k[:] = 0.0
    k[200:210, :, 0] = float("-inf")
    o, lse = fa.forward_packed_window(q, k, v, cu, 4, 0)
    bad = torch.isnan(o).all(-1).flatten()
    assert torch.isnan(o).any(-1).flatten().equal(bad)
    assert bad.nonzero().flatten().tolist() == list(range(203, 210))


# ------------------------------------------------------------------ over the cache
def forget(x, window, sinks, entry):
    """Gives back the blocks that no query of a chunk sees: their table entries hold
    `entry`, their slots NaN."""
    q, kc, vc, bt, ctx, cu = x
    bt = bt.clone()
    for s, (a, b, c) in enumerate(zip(cu.tolist(), cu.tolist()[1:], ctx.tolist())):
        for blk in range((c + 15) // 16):
            if blk * 16 >= sinks and blk * 16 + 15 <= c - (b - a) - window:
                kc[bt[s, blk].item()] = float("nan")
                vc[bt[s, blk].item()] = float("nan")
                bt[s, blk] = bt[s, blk] if entry is None else entry
    return q, kc, vc, bt, ctx, cu


def check_paged(x, out, window, sinks):
    q, kc, vc, bt, ctx, cu = x
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for s, (a, b, c) in enumerate(zip(cu.tolist(), cu.tolist()[1:], ctx.tolist())):
        if a == b:
            continue
        tok = torch.arange(c, device=DEV)
        blk, off = bt[s].long()[tok // 16], tok % 16
        # (entries outside the cache read as zero keys and values)
        there = ((blk >= 0) & (blk < kc.shape[0]))[:, None, None]
        blk = blk.clamp(0, kc.shape[0] - 1)
        k = torch.where(there, kc[blk, :, :, off].flatten(2), 0.0)
        v = torch.where(there, vc[blk, :, :, off], 0.0)
        see = ref.near(c - (b - a) + torch.arange(b - a, device=DEV), c, window, sinks)
        packed_ref.check_forward(out[a:b], None, ref.sequence(q[a:b], k, v, 128 ** -0.5, see),
                                 128 ** -0.5, BF16)


def run_paged(lens, ctx, H, Hk, window, sinks, seed, entry=-1, **kw):
    x = forget(draw_paged(lens, ctx, H, Hk, seed, **kw), window, sinks, entry)
    out = fa.paged_prefill_window(*x, window, sinks)
    check_paged(x, out, window, sinks)
    return x, out


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_paged_windows(window, sinks):
    """Whole prompts, pieces, single tokens, no new tokens; blocks out of sight gone."""
    for entry in (-1, 1 << 30, None):
        run_paged([40, 1, 7, 0, 233, 1, 1], [40, 100, 900, 50, 334, 3000, 513], 8, 2, window,
                  sinks, seed=window, entry=entry)


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (6, 2), (7, 1), (32, 8), (16, 1), (40, 1),
                                  (128, 1)])
def test_paged_heads(H, Hk):
    run_paged([40, 1, 7, 0, 33], [40, 100, 700, 50, 334], H, Hk, 130, 20, seed=H)


@pytest.mark.parametrize("n", [1, 2, 5])
def test_paged_every_position(n):
    """Every place of the window's start in a block and a tile, for few tokens."""
    S = 100
    run_paged([n] * S, [n + 3 * i for i in range(S)], 4, 1, 37, 6, seed=n)
    run_paged([n] * S, [400 + i for i in range(S)], 2, 1, 129, 17, seed=n)


@pytest.mark.parametrize("lens,ctx", [
    ([1, 4, 2], [9000, 5000, 513]),
    ([64, 1], [8192, 8191]),
    ([200], [12345]),
    ([5, 5, 5, 5], [4096, 1, 600, 0]),            # contexts shorter than their chunks too
])
@pytest.mark.parametrize("window,sinks", [(2048, 4), (4000, 600), (700, 0)])
def test_paged_split_contexts(lens, ctx, window, sinks):
    """Partitions of the visible tiles and their merge."""
    S, T = len(lens), sum(lens)
    mb = max((c + 15) // 16 for c in ctx) + 1
    assert fa.fa_paged_prefill_window_workspace_bytes(S, T, 8, 2, mb, window, sinks) > 0
    run_paged(lens, ctx, 8, 2, window, sinks, seed=T)
    run_paged(lens, ctx, 5, 1, window, sinks, seed=T + 1)


@pytest.mark.parametrize("lens,ctx", [
    ([1, 2000], [9000, 9000]),                        # few rows beside many, cut by their own share
    ([64, 1, 65, 3, 0, 2500], [8200, 5, 7777, 8192, 400, 8193]),
    ([700, 1], [700, 4096]),
])
def test_paged_single_tokens_beside_chunks(lens, ctx):
    run_paged(lens, ctx, 8, 2, 4096, 20, seed=8)


@pytest.mark.parametrize("S", [112, 113, 300])
def test_paged_many_sequences(S):
    g = torch.Generator().manual_seed(S)
    ctx = torch.randint(0, 700, (S,), generator=g).tolist()
    run_paged([1] * S, ctx, 4, 2, 200, 4, seed=S)


def test_paged_rows_of_no_sequence_and_zero_rows():
    x = forget(draw_paged([9, 30, 20], [700, 30, 4], 4, 2, seed=7, before=5, behind=50), 64, 3, -1)
    out = torch.full(x[0].shape, 7.0, dtype=BF16, device=DEV)
    fa.paged_prefill_window(*x, 64, 3, out=out)
    check_paged(x, out, 64, 3)
    assert (out[:5] == 7).all() and (out[64:] == 7).all()
    assert (out[44:60] == 0).all() and (out[60:64] != 0).any()


def test_paged_repeats_and_keeps_its_bits():
    """Blocks out of sight change nothing, and calls agree bit for bit."""
    x = draw_paged([1, 30, 4, 1], [3000, 5000, 800, 40], 8, 2, seed=11)
    a = fa.paged_prefill_window(*x, 300, 4)
    y = forget(x, 300, 4, -1)
    for _ in range(3):
        assert torch.equal(a, fa.paged_prefill_window(*y, 300, 4))


def test_captured_with_changing_lengths():
    """One graph over a decode step, replayed as the contexts grow."""
    x = draw_paged([1] * 6, [500, 40, 1, 900, 333, 128], 8, 2, seed=12, poison=False)
    q, kc, vc, bt, ctx, cu = x
    out = torch.empty(q.shape, dtype=BF16, device=DEV)
    ws = torch.empty(fa.fa_paged_prefill_window_workspace_bytes(6, 6, 8, 2, bt.shape[1], 150, 4)
                     or 16, dtype=torch.uint8, device=DEV)
    fa.paged_prefill_window(*x, 150, 4, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_prefill_window(*x, 150, 4, out=out, workspace=ws)
    for step in range(4):
        ctx += torch.tensor([3, 1, 0, -200, 10, 1], dtype=torch.int32, device=DEV)
        graph.replay()
        check_paged(x, out, 150, 4)


def test_refusals():
    q, k, v, cu = draw([10], 2, 1, 64, BF16, seed=1)
    x = draw_paged([1], [40], 2, 1, seed=1)
    for window, sinks in ((0, 0), (-3, 0), (4, -1)):
        with pytest.raises(ValueError):
            fa.forward_packed_window(q, k, v, cu, window, sinks)
        with pytest.raises(ValueError):
            fa.paged_prefill_window(*x, window, sinks)
    with pytest.raises(ValueError):
        fa.forward_packed_window(q.float(), k.float(), v.float(), cu, 4)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_outputs_aligned_to_16_bytes_only(d, dtype):
    q, k, v, cu = draw([300, 41], 4, 2, d, dtype, seed=3)
    a, _ = fa.forward_packed_window(q, k, v, cu, 70, 2)
    room = torch.full((a.numel() + 24,), 7.0, dtype=dtype, device=DEV)
    for off in (8, 16):
        out = room[off:off + a.numel()].view(a.shape)
        fa.forward_packed_window(q, k, v, cu, 70, 2, out=out)
        assert torch.equal(a, out)
        assert (room[:off] == 7).all() and (room[off + a.numel():] == 7).all()
        room.fill_(7.0)


def test_paged_buffers_aligned_to_16_bytes_only():
    x = draw_paged([1, 30, 4, 1], [3000, 5000, 800, 40], 8, 2, seed=11)
    a = fa.paged_prefill_window(*x, 2500, 4)
    n = fa.fa_paged_prefill_window_workspace_bytes(4, 36, 8, 2, x[3].shape[1], 2500, 4)
    assert n > 0
    room = torch.zeros(a.numel() + 8, dtype=BF16, device=DEV)
    ws = torch.empty(n + 16, dtype=torch.uint8, device=DEV)
    out = room[8:].view(a.shape)
    fa.paged_prefill_window(*x, 2500, 4, out=out, workspace=ws[16:])
    assert torch.equal(a, out)
