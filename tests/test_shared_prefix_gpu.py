"""Chunks over the paged cache where groups of sequences share a prefix's blocks,
against float64 on the gathered keys and values.  Tolerances:
packed_ref.check_forward."""
import pytest
import torch

import exact_attention_11_gb300 as fa
import packed_ref
from test_paged_prefill_gpu import check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def draw(groups, H, Hk, seed, loose=(), before=0, behind=0, claim=None):
    """groups: (prefix length, [(new tokens, tokens behind the prefix), ..]) each;
    loose: (new tokens, context) of sequences of no group, which come last.  A context
    of None is shorter than the prefix: the sequence has 3 tokens of its own alone.
    Whole blocks of a prefix are the group's, all others each sequence's own; slots
    past a context and unused blocks hold NaN.  claim: prefix lengths passed on."""
    g = torch.Generator().manual_seed(seed)
    lens, ctx, pre = [], [], []
    for p, members in groups:
        for n, c in members:
            lens.append(n)
            ctx.append(3 if c is None else p + c)
            pre.append(0 if c is None else p // 16)
    for n, c in loose:
        lens.append(n)
        ctx.append(c)
        pre.append(0)
    S, T = len(lens), before + sum(lens) + behind
    mb = max((c + 15) // 16 for c in ctx) + 1
    nb = sum(p // 16 for p, _ in groups) + sum((c + 15) // 16 for c in ctx) + 3
    q = torch.randn(T, H + 1, 128, generator=g).to(BF16).to(DEV)[:, :H]
    kc = torch.randn(nb, Hk, 16, 16, 8, generator=g).to(BF16).to(DEV)
    vc = torch.randn(nb, Hk, 128, 16, generator=g).to(BF16).to(DEV)
    perm = torch.randperm(nb, generator=g).int()
    bt = torch.full((S, mb), -7 if seed % 2 else 1 << 30, dtype=torch.int32)
    at = s = 0
    for p, members in groups:
        for _, c in members:
            if c is not None:
                bt[s, :p // 16] = perm[at:at + p // 16]
            s += 1
        at += p // 16
    for s in range(S):
        n = (ctx[s] + 15) // 16 - pre[s]
        bt[s, pre[s]:pre[s] + n] = perm[at:at + n]
        at += n
        if ctx[s] % 16 and n:
            b = bt[s, pre[s] + n - 1].item()
            kc[b, :, :, ctx[s] % 16:] = float("nan")
            vc[b, :, :, ctx[s] % 16:] = float("nan")
    kc[perm[at:].long().to(DEV)] = float("nan")
    vc[perm[at:].long().to(DEV)] = float("inf")
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = torch.tensor([before] + lens).cumsum(0).int().to(DEV)
    cg = torch.tensor([0] + [len(m) for _, m in groups]).cumsum(0).int().to(DEV)
    pl = torch.tensor([p for p, _ in groups] if claim is None else claim, **i32)
    return q, kc, vc, bt.to(DEV), torch.tensor(ctx, **i32), cu, cg, pl


def run(groups, H, Hk, seed, **kw):
    x = draw(groups, H, Hk, seed, **kw)
    out = fa.paged_prefill_shared(*x)
    check(*x[:6], out)
    return x, out


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (8, 2), (6, 2), (7, 1), (32, 8), (16, 1),
                                  (40, 1), (128, 1)])
def test_heads(H, Hk):
    """Group sizes that divide 128 and that do not; single tokens, chunks, no new
    tokens, a member that is too short, sequences of no group."""
    run([(1000, [(1, 40), (1, 1), (7, 30), (0, 50), (33, 40), (1, None)]),
         (300, [(2, 2), (1, 100), (1, 17)])], H, Hk, seed=H, loose=[(1, 333), (20, 50)])


@pytest.mark.parametrize("prefix", [0, 15, 16, 17, 112, 127, 128, 129, 143, 144, 256, 1000, 2047,
                                    2048, 5000, 20000])
@pytest.mark.parametrize("n", [1, 3])
def test_prefixes(prefix, n):
    """Prefixes at the blocks' and tiles' edges, shared by two, by twenty, by ninety."""
    for S in (2, 20, 90):
        run([(prefix, [(n, n + 7 * i % 100) for i in range(S)])], 8, 2, seed=prefix + S)


@pytest.mark.parametrize("c", list(range(1, 34)) + [127, 128, 129, 500, 3000])
def test_own_lengths(c):
    run([(400, [(1, c), (1, max(1, c - 1)), (1, c + 1), (1, 1)] * 3)], 4, 1, seed=c)


def test_groups_of_one_none_and_all():
    run([(500, [(1, 30)]), (400, []), (600, [(1, 5), (2, 9)]), (300, [])], 8, 2, seed=1)
    x, out = run([], 8, 2, seed=2, loose=[(1, 300), (5, 40), (1, 0)])
    assert torch.equal(out, fa.paged_prefill(*x[:6])) and (out[6] == 0).all()


@pytest.mark.parametrize("claim", [[700], [100], [1 << 30], [-5], [(1 << 31) - 1]])
def test_prefix_lengths_that_do_not_fit(claim):
    """A shorter claim shares less; a longer one than the contexts, nothing."""
    x, out = run([(512, [(1, 20 + i) for i in range(30)])], 8, 2, seed=5, claim=claim)
    if claim[0] != 100:
        check(*x[:6], fa.paged_prefill(*x[:6]))


@pytest.mark.parametrize("S", [111, 112, 113, 300, 1100])
def test_many_sequences(S):
    """Up to 112 sequences and groups are numbered by the CTAs, more by a kernel ahead."""
    g = torch.Generator().manual_seed(S)
    own = torch.randint(1, 60, (S,), generator=g).tolist()
    run([(640, [(1, c) for c in own])], 4, 2, seed=S)


def test_many_groups():
    run([(160 + 16 * (i % 5), [(1, 3 + i % 40), (2, 20)][:1 + i % 2]) for i in range(45)], 4, 2,
        seed=5)
    run([(160 + 16 * (i % 5), [(1, 3 + i % 40), (1, 20)]) for i in range(600)], 2, 1, seed=3)
    with pytest.raises(fa.FattnError):
        x = draw([(16, [])] * 1025, 2, 1, 4, loose=[(1, 5)])
        fa.paged_prefill_shared(*x)


@pytest.mark.parametrize("H,Hk", [(8, 1), (32, 8), (3, 3)])
def test_long_chunks_and_partitions(H, Hk):
    """Chunks of more than a block's tokens; long own contexts, cut too."""
    run([(3000, [(100, 200), (200, 200), (1, 9000)]), (1500, [(300, 300), (5, 2000)])], H, Hk,
        seed=8, loose=[(3, 7000)])


def test_rows_of_no_sequence_stay_and_zero_rows():
    x = draw([(600, [(9, 30), (1, 2), (4, 4), (20, None)])], 8, 2, seed=7, before=5, behind=50)
    out = torch.full(x[0].shape, 7.0, dtype=BF16, device=DEV)
    fa.paged_prefill_shared(*x, out=out)
    check(*x[:6], out)
    assert (out[:5] == 7).all() and (out[39:] == 7).all()
    assert (out[19:36] == 0).all() and (out[36:39] != 0).any()


def test_nan_stays_in_its_sequence():
    """A NaN query, and NaN keys behind the prefix, in one sequence of the group."""
    x = draw([(800, [(1, 20), (2, 30), (1, 25)])], 8, 2, seed=9)
    q, kc, vc, bt, ctx, cu = x[:6]
    out = fa.paged_prefill_shared(*x)
    q[2, 3] = float("nan")
    kc[bt[1, 51].item(), :, :, 0] = float("nan")
    out2 = fa.paged_prefill_shared(*x)
    assert torch.equal(out[[0, 3]], out2[[0, 3]])
    assert torch.isnan(out2[1:3]).all()


def test_repeats_streams_and_captures():
    x = draw([(900, [(1, 10 + i) for i in range(40)])], 8, 2, seed=11)
    a = fa.paged_prefill_shared(*x)
    for _ in range(3):
        assert torch.equal(a, fa.paged_prefill_shared(*x))
    many = draw([(900, [(1, 10 + i) for i in range(90)]), (400, [(2, 5 + i) for i in range(90)])],
                8, 2, seed=12)
    want = fa.paged_prefill_shared(*many)
    for _ in range(3):
        assert torch.equal(want, fa.paged_prefill_shared(*many))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s in streams:                       # each call with a workspace of its own
        with torch.cuda.stream(s):
            outs.append([fa.paged_prefill_shared(*x) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for os in outs for o in os)
    q, kc, vc, bt, ctx, cu, cg, pl = x
    out = torch.empty_like(a)
    n = fa.fa_paged_prefill_shared_workspace_bytes(40, 40, 1, 8, 2, bt.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_prefill_shared(*x, out=out, workspace=ws)
    for take in (0, 300, -300, -1000):      # contexts shorter than the prefix at the end
        ctx.copy_((ctx + min(take, 0)).clamp(min=0))
        pl += max(take, 0) - 150
        graph.replay()
        check(*x[:6], out)


def test_offsets_that_decrease_stay_inside():
    x = draw([(400, [(1, 10 + i) for i in range(20)]), (300, [(2, 9)] * 9)], 8, 2, seed=13)
    q, kc, vc, bt, ctx, cu, cg, pl = x
    for bad in ([20, 5, 29], [1 << 30, -4, 3], [29, 29, 0]):
        fa.paged_prefill_shared(*x[:6], torch.tensor(bad, dtype=torch.int32, device=DEV), pl)
    bad = cu.flip(0).contiguous()
    fa.paged_prefill_shared(q, kc, vc, bt, ctx, bad, cg, pl)
    fa.paged_prefill_shared(q, kc, vc, bt, ctx * 0 + (1 << 30), cu, cg, pl)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    check(*x[:6], fa.paged_prefill_shared(*x))


def test_scores_of_minus_infinity():
    """-inf over the whole prefix leaves a row its own keys; over its own too, NaN."""
    x = draw([(512, [(1, 20), (1, 30), (1, 16)])], 2, 1, seed=15)
    q, kc, vc, bt, ctx, cu = x[:6]
    q[:] = 1.0
    first = bt[0, :32].long()
    kc[first] = 0.0
    kc[first, :, 0, :, 0] = float("-inf")
    out = fa.paged_prefill_shared(*x)
    assert torch.isfinite(out).all()
    for s, c in enumerate(ctx.tolist()):
        tok = torch.arange(512, c, device=DEV)
        k = kc[bt[s].long()[tok // 16], :, :, tok % 16].flatten(2)
        v = vc[bt[s].long()[tok // 16], :, :, tok % 16]
        last = torch.full((1,), c - 512, device=DEV)
        ref = packed_ref.sequence(q[s:s + 1], k, v, 128 ** -0.5, last)
        packed_ref.check_forward(out[s:s + 1], None, ref, 128 ** -0.5, BF16)
    own = bt[1, 32:34].long()
    kc[own] = 0.0
    kc[own, :, 0, :, 0] = float("-inf")
    out = fa.paged_prefill_shared(*x)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()


def test_refusals():
    x = draw([(64, [(1, 5), (1, 6)])], 8, 2, seed=17)
    q, kc, vc, bt, ctx, cu, cg, pl = x
    for bad in (dict(cu_groups=cg[:1]), dict(cu_groups=cg.long()), dict(prefix_lens=pl.float()),
                dict(cu_groups=cg.cpu()), dict(q=q.half()), dict(cu_seqlens=cu[:2]),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cpu"))):
        a = dict(q=q, k_cache=kc, v_cache=vc, block_tables=bt, context_lens=ctx, cu_seqlens=cu,
                 cu_groups=cg, prefix_lens=pl)
        a.update(bad)
        with pytest.raises(ValueError):
            fa.paged_prefill_shared(**a)
    with pytest.raises(fa.FattnError):
        fa.paged_prefill_shared(*x, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
