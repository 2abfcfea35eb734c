"""Chunks of new tokens over a paged cache against float64 on the gathered
keys and values.  Tolerances: packed_ref.check_forward."""
import pytest
import torch

import exact_attention_11_gb300 as fa
import packed_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def draw(lens, ctx, H, Hk, seed, spare=3, before=0, behind=0, poison=True):
    """Chunks, a paged cache with scattered blocks, NaN in every slot past a
    context and in unused blocks, table entries past the context invalid."""
    g = torch.Generator().manual_seed(seed)
    S = len(lens)
    mb = max(1, max((c + 15) // 16 for c in ctx)) + 1
    used = [(c + 15) // 16 for c in ctx]
    nb = sum(used) + spare
    T = before + sum(lens) + behind
    q = torch.randn(T, H + 1, 128, generator=g).to(BF16).to(DEV)[:, :H]
    kc = torch.randn(nb, Hk, 16, 16, 8, generator=g).to(BF16).to(DEV)
    vc = torch.randn(nb, Hk, 128, 16, generator=g).to(BF16).to(DEV)
    perm = torch.randperm(nb, generator=g)
    bt = torch.full((S, mb), -7 if seed % 2 else 1 << 30, dtype=torch.int32)
    at = 0
    free = torch.ones(nb, dtype=torch.bool)
    for s, n in enumerate(used):
        bt[s, :n] = perm[at:at + n].int()
        free[perm[at:at + n]] = False
        if poison and ctx[s] % 16:
            b = bt[s, n - 1].item()
            kc[b, :, :, ctx[s] % 16:] = float("nan")
            vc[b, :, :, ctx[s] % 16:] = float("nan")
        at += n
    if poison:
        kc[free.to(DEV)] = float("nan")
        vc[free.to(DEV)] = float("inf")
    cu = torch.tensor([before] + lens).cumsum(0).int().to(DEV)
    return q, kc, vc, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), cu


def check(q, kc, vc, bt, ctx, cu, out, scale=None):
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = scale or 128 ** -0.5
    for s, (a, b, c) in enumerate(zip(cu.tolist(), cu.tolist()[1:], ctx.tolist())):
        if a == b:
            continue
        tok = torch.arange(c, device=DEV)
        blk, off = bt[s].long()[tok // 16], tok % 16
        k = kc[blk, :, :, off].flatten(2)
        v = vc[blk, :, :, off]
        last = c - (b - a) + torch.arange(b - a, device=DEV)
        ref.check_forward(out[a:b], None, ref.sequence(q[a:b], k, v, scale, last), scale, BF16)


def run(lens, ctx, H, Hk, seed, **kw):
    x = draw(lens, ctx, H, Hk, seed, **kw)
    out = fa.paged_prefill(*x)
    check(*x, out)
    return x, out


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (8, 2), (6, 2), (7, 1), (32, 8), (16, 1),
                                  (40, 1), (128, 1)])
def test_heads(H, Hk):
    """Group sizes that divide 128 and that do not; whole prompts, pieces,
    single tokens, no new tokens."""
    run([40, 1, 7, 0, 33], [40, 100, 300, 50, 34], H, Hk, seed=H)


@pytest.mark.parametrize("n,c", [(1, 1), (1, 16), (1, 17), (2, 128), (3, 129), (16, 16),
                                 (64, 640), (65, 127), (127, 1000), (129, 2049), (300, 300)])
def test_sizes(n, c):
    run([n], [c], 4, 1, seed=n + c)
    run([n, n], [c, max(n, c - 5)], 3, 3, seed=n + c + 1)


def test_every_context_tail():
    """Contexts that end at each slot of a block and each block of a tile."""
    ctx = list(range(5, 5 + 150))
    run([1 + i % 5 for i in range(150)], ctx, 2, 1, seed=3)


@pytest.mark.parametrize("lens,ctx", [
    ([1, 4, 2], [9000, 5000, 513]),               # partitions: all, some, one of a sequence's
    ([64, 1], [8192, 8191]),
    ([200], [12345]),
    ([5, 5, 5, 5], [4096, 1, 600, 0]),            # contexts shorter than their chunks too
])
def test_split_contexts(lens, ctx):
    """Few rows over long contexts: partitions and their merge."""
    S, T = len(lens), sum(lens)
    mb = max((c + 15) // 16 for c in ctx) + 1
    assert fa.fa_paged_prefill_workspace_bytes(S, T, 8, 2, mb) > 0
    run(lens, ctx, 8, 2, seed=T)
    run(lens, ctx, 5, 1, seed=T + 1)


def test_chunks_that_span_split_and_whole_tiles():
    """One call whose query tiles lie on both sides of a partition's length."""
    run([1500, 3], [1500, 7000], 4, 2, seed=4)


def test_context_shorter_than_the_chunk():
    """Queries before the first cached token see nothing: zero rows."""
    x, out = run([20, 8, 5], [4, 0, 5], 4, 2, seed=6)
    assert (out[:16] == 0).all() and (out[20:28] == 0).all() and (out[16] != 0).any()


def test_rows_of_no_sequence_stay():
    x = draw([9, 30], [700, 30], 4, 2, seed=7, before=5, behind=50)
    out = torch.full(x[0].shape, 7.0, dtype=BF16, device=DEV)
    fa.paged_prefill(*x, out=out)
    check(*x, out)
    assert (out[:5] == 7).all() and (out[44:] == 7).all()


def test_bad_block_ids_read_as_zeros():
    """A table entry outside the cache inside a context: zero keys and values,
    nothing out of bounds."""
    q, kc, vc, bt, ctx, cu = draw([3], [64], 2, 1, seed=8, poison=False)
    want = bt.clone()
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        bt[0, 1] = bad
        out = fa.paged_prefill(q, kc, vc, bt, ctx, cu)
        kz = torch.cat([kc, torch.zeros_like(kc[:1])])
        vz = torch.cat([vc, torch.zeros_like(vc[:1])])
        want[0, 1] = kc.shape[0]
        check(q, kz, vz, want, ctx, cu, out)


def test_context_lengths_are_clamped():
    q, kc, vc, bt, ctx, cu = draw([3], [64], 2, 1, seed=10, poison=False)
    bt = bt[:, :4].contiguous()
    want = fa.paged_prefill(q, kc, vc, bt, ctx, cu)
    assert torch.equal(want, fa.paged_prefill(q, kc, vc, bt, ctx + 1000, cu))
    assert (fa.paged_prefill(q, kc, vc, bt, ctx - 1000, cu) == 0).all()


def test_single_tokens_match_the_decode():
    """One new token per sequence is the grouped decode (both to two bf16
    roundings of the same value)."""
    S = 40
    ctx = [1 + 97 * i % 3000 for i in range(S)]
    x = draw([1] * S, ctx, 16, 4, seed=9)
    out = fa.paged_prefill(*x)
    check(*x, out)
    q, kc, vc, bt, c, _ = x
    bt = torch.where((bt < 0) | (bt >= kc.shape[0]), 0, bt)
    dec = fa.paged_decode(q.contiguous(), kc, vc, bt, c)
    assert (dec.float() - out.float()).abs().max() <= 2e-2


def test_chunked_prefill_equals_the_whole_prompt():
    """A prompt written and attended in pieces (norm, rotation and cache in
    one call, then the chunk) against the packed forward of the whole."""
    H, Hk, n, pieces = 8, 2, 333, [100, 1, 64, 168]
    g = torch.Generator().manual_seed(12)
    qkv = torch.randn(n, H + 2 * Hk, 128, generator=g).to(BF16).to(DEV)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    qw, kw = ((1 + 0.1 * torch.randn(128, generator=g)).to(BF16).to(DEV) for _ in range(2))
    freq, _ = fa.rope_frequencies(128, device=DEV)
    pos = torch.arange(n, device=DEV).int()
    bt = torch.randperm(30, generator=g)[:21].int().view(1, 21).to(DEV)
    kc = torch.full((30, Hk, 16, 16, 8), float("nan"), dtype=BF16, device=DEV)
    vc = torch.full((30, Hk, 128, 16), float("nan"), dtype=BF16, device=DEV)
    slots = bt[0].long()[pos.long() // 16] * 16 + pos.long() % 16
    outs, at = [], 0
    for m in pieces:
        r = slice(at, at + m)
        at += m
        qp = fa.qk_norm_rope_cache(q[r], k[r], v[r], pos[r], freq, slots[r], kc, vc, qw, kw)
        outs.append(fa.paged_prefill(qp, kc, vc, bt, torch.tensor([at], device=DEV).int(),
                                     torch.tensor([0, m], device=DEV).int()))
    qr, kr = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    whole, _ = fa.forward_packed(qr, kr, v, torch.tensor([0, n], device=DEV).int())
    got = torch.cat(outs)
    r = ref.sequence(qr, kr, v, 128 ** -0.5, pos.long())
    for o in (got, whole):
        ref.check_forward(o, None, r, 128 ** -0.5, BF16)


def test_repeats_captures_and_streams():
    """Bit-identical repeats; a graph on new inputs; two streams with a
    workspace each."""
    lens, ctx = [6, 1, 130], [5000, 900, 4100]
    q, kc, vc, bt, c, cu = draw(lens, ctx, 8, 2, seed=13, poison=False)
    want = fa.paged_prefill(q, kc, vc, bt, c, cu)
    for _ in range(5):
        assert torch.equal(want, fa.paged_prefill(q, kc, vc, bt, c, cu))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        out = fa.paged_prefill(q, kc, vc, bt, c, cu)
    q.mul_(0.5)
    c.copy_(torch.tensor([4000, 800, 200]))
    graph.replay()
    torch.cuda.synchronize()
    want = fa.paged_prefill(q, kc, vc, bt, c, cu)
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i & 1]):
            outs.append(fa.paged_prefill(q, kc, vc, bt, c, cu))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0 and all(torch.equal(x, want) for x in outs)


def test_helper_refuses():
    q, kc, vc, bt, ctx, cu = draw([3, 4], [20, 30], 4, 2, seed=1)
    bad = [
        lambda: fa.paged_prefill(q.half(), kc, vc, bt, ctx, cu),
        lambda: fa.paged_prefill(q, kc, vc[:1], bt, ctx, cu),
        lambda: fa.paged_prefill(q[:, :3], kc, vc, bt, ctx, cu),
        lambda: fa.paged_prefill(q, kc, vc, bt.long(), ctx, cu),
        lambda: fa.paged_prefill(q, kc, vc, bt, ctx[:1], cu),
        lambda: fa.paged_prefill(q, kc, vc, bt, ctx, cu[:2]),
        lambda: fa.paged_prefill(q, kc, vc, bt.t(), ctx, cu),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    x = draw([1], [9000], 4, 2, seed=2)
    with pytest.raises(fa.FattnError):
        fa.paged_prefill(*x, workspace=small)


@pytest.mark.parametrize("lens,ctx", [([3, 9], [40, 300]), ([1], [9000]), ([3, 2, 140], [9000, 5, 700]),
                                      ([2], [40000])], ids=str)
def test_a_nan_query_gives_a_nan_row(lens, ctx):
    """Whether its context is cut into partitions or not; the other rows keep
    their bits."""
    q, kc, vc, bt, c, cu = draw(lens, ctx, 8, 2, seed=14, poison=False)
    want = fa.paged_prefill(q, kc, vc, bt, c, cu)
    q[0, 3, 5] = q[len(q) - 1, 6, 127] = float("nan")
    out = fa.paged_prefill(q, kc, vc, bt, c, cu)
    for row, head in ((0, 3), (len(q) - 1, 6)):
        assert out[row, head].isnan().all()
        out[row, head] = want[row, head]
    assert torch.equal(out, want)


def test_bounds_written_just_before():
    """cu_seqlens and context_lens that the kernel before the call writes, to other
    values each time: main and merge kernel cut the contexts alike."""
    q, kc, vc, bt, c, cu = draw([6, 1, 130], [9000, 900, 4100], 8, 2, seed=15, poison=False)
    bt = torch.randint(0, len(kc), bt.shape, device=DEV).int()
    bounds = [(c.clone(), cu.clone())]
    for ctx, ends in (((900, 8000, 150), (0, 6, 7, 137)), ((5000, 40, 4096), (0, 1, 130, 137)),
                      ((0, 9000, 9000), (0, 0, 3, 90))):
        bounds.append((torch.tensor(ctx, device=DEV).int(), torch.tensor(ends, device=DEV).int()))
    want = []
    for x, y in bounds:
        torch.cuda.synchronize()
        want.append(fa.paged_prefill(q, kc, vc, bt, x, y, out=torch.zeros(q.shape, dtype=BF16, device=DEV)))
        check(q, kc, vc, bt, x, y, want[-1])
    outs = [torch.zeros_like(want[0]) for _ in range(64)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        c.copy_(bounds[i % 4][0])
        cu.copy_(bounds[i % 4][1])
        fa.paged_prefill(q, kc, vc, bt, c, cu, out=out)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 4])


@pytest.mark.parametrize("lens,ctx", [([3, 9], [40, 300]), ([1], [9000]), ([3, 7, 140], [9000, 5, 700]),
                                      ([2], [40000])], ids=str)
def test_scores_of_minus_infinity(lens, ctx):
    """Over whole and cut contexts NaN, as in the packed forward; zeros only for a
    query that sees no key (the second sequence's first two of [3, 7, 140])."""
    q, kc, vc, bt, c, cu = draw(lens, ctx, 8, 2, seed=16, poison=False)
    kc.abs_()
    want = fa.paged_prefill(q, kc, vc, bt, c, cu)
    rows = [(0, 3), (len(q) - 1, 6)]
    if lens == [3, 7, 140]:
        assert (want[3:5] == 0).all() and (want[5] != 0).any()
        q[3, 1, 9] = float("-inf")
        rows.append((6, 1))
    for row, head in rows:
        q[row, head, 9] = float("-inf")
    out = fa.paged_prefill(q, kc, vc, bt, c, cu)
    for row, head in rows:
        assert out[row, head].isnan().all()
        out[row, head] = want[row, head]
    assert torch.equal(out, want)


@pytest.mark.parametrize("lens,ctx", [([1], [40000]), ([2, 1], [40000, 20001]), ([2], [33000])], ids=str)
@pytest.mark.parametrize("H,Hk", [(8, 1), (8, 2), (3, 3)])
def test_more_partitions_than_lanes(lens, ctx, H, Hk):
    """More than 32 partitions: the merge's later rounds.  Each head has one key that
    its scores favour, the even heads' among the first 32 partitions, the odd heads'
    behind them, so that what is carried over is scaled down as well as kept."""
    mb = max((c + 15) // 16 for c in ctx) + 1
    rows = fa.fa_paged_prefill_workspace_bytes(len(lens), sum(lens), H, Hk, mb) // (130 * 4)
    assert rows // (sum(lens) * H) > 32
    q, kc, vc, bt, c, cu = draw(lens, ctx, H, Hk, seed=17)
    for s, (n, at) in enumerate(zip(ctx, cu.tolist())):
        for h in range(H):
            tok = 100 + 130 * h if h % 2 == 0 else n - 150 - 130 * h
            # |q|^2 / sqrt(d) is about 11: e^11 of some 40000 keys' e^0.5
            kc[bt[s, tok // 16].item(), h * Hk // H, :, tok % 16] = q[at, h].view(16, 8)
    out = fa.paged_prefill(q, kc, vc, bt, c, cu)
    check(q, kc, vc, bt, c, cu, out)


@pytest.mark.parametrize("S", [112, 113])
@pytest.mark.parametrize("long_at", [0, 60])
def test_long_context_among_many_sequences(S, long_at):
    """Contexts are cut up to 112 sequences and whole beyond."""
    ctx = [1 + 37 * i % 500 for i in range(S)]
    ctx[long_at] = 20000
    lens = [1 + i % 2 if c > 1 else 1 for i, c in enumerate(ctx)]
    T, mb = sum(lens), 20000 // 16 + 1
    assert (fa.fa_paged_prefill_workspace_bytes(S, T, 4, 2, mb) > 0) == (S <= 112)
    run(lens, ctx, 4, 2, seed=S)
    run(lens, ctx, 3, 1, seed=S + 1)
