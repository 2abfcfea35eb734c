"""Packed prompts of different lengths with grouped heads against float64.
Tolerances: packed_ref.check_forward."""
import os
import subprocess
import sys

import pytest
import torch

import exact_attention_11_gb300 as fa
import packed_ref as ref
import qk_prep_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


def draw(lens, H, Hk, d, dtype, seed, before=0, behind=0, fill=float("nan")):
    """Views of one fused projection and cu_seqlens; `before` and `behind`
    rows of no sequence hold `fill`."""
    T = before + sum(lens) + behind
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * Hk, d, generator=g)
    qkv[:before] = fill
    qkv[T - behind:] = fill
    qkv = qkv.to(dtype).to(DEV)
    cu = torch.tensor([before] + lens).cumsum(0).int().to(DEV)
    return qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], cu


def check(q, k, v, cu, o, lse, causal, scale=None):
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = scale or q.shape[-1] ** -0.5
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        n = b - a
        last = torch.arange(n, device=DEV) if causal else torch.full((n,), n, device=DEV)
        r = ref.sequence(q[a:b], k[a:b], v[a:b], scale, last)
        ref.check_forward(o[a:b], None if lse is None else lse[:, a:b], r, scale, q.dtype)


def run(lens, H, Hk, d, dtype, causal, seed, **kw):
    q, k, v, cu = draw(lens, H, Hk, d, dtype, seed, **kw)
    o, lse = fa.forward_packed(q, k, v, cu, causal=causal)
    check(q, k, v, cu, o, lse, causal)


HEADS = [(1, 1), (8, 2), (6, 2), (7, 1), (10, 2), (16, 1), (40, 1), (128, 1)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", HEADS)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_heads(H, Hk, d, causal):
    """Group sizes that divide 128 and that do not; lengths at the tiles'
    edges, one token, an empty sequence."""
    run([1, 130, 0, 64, 33], H, Hk, d, BF16, causal, seed=H + d)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens", [[1], [128], [129], [255, 256, 257], [2, 1, 1, 3], [0, 5, 0, 0],
                                  [700, 31, 1100]], ids=str)
def test_lengths(lens, d, dtype, causal):
    run(lens, 4, 2, d, dtype, causal, seed=sum(lens))


def test_every_length_up_to_three_tiles():
    """One sequence of each length 1 .. 270 (one head), causal and not."""
    for causal in (True, False):
        run(list(range(1, 271)), 1, 1, 64, BF16, causal, seed=5)


@pytest.mark.parametrize("S", [31, 32, 33, 1023, 1025, 2100])
def test_many_sequences(S):
    """The 32-way search at one, two and three rounds."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, 9, (S,), generator=g).tolist()
    run(lens, 2, 1, 64, BF16, True, seed=S)


@pytest.mark.parametrize("H,Hk,d", [(8, 2, 128), (12, 4, 64)])
def test_many_items_per_sm(H, Hk, d):
    """Several work items per persistent CTA, light and heavy ones mixed."""
    run([3000, 1, 257, 2049, 640, 5, 1500], H, Hk, d, BF16, True, seed=9)
    run([1200, 77, 900], H, Hk, d, F16, False, seed=10)


def test_rows_of_no_sequence_stay_and_do_not_leak():
    """NaN before the first and behind the last sequence: neither read into a
    sequence nor written."""
    for d in (64, 128):
        q, k, v, cu = draw([100, 45], 4, 2, d, BF16, seed=3, before=37, behind=200)
        o = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
        lse = torch.full((4, q.shape[0]), 7.0, device=DEV)
        fa.forward_packed(q, k, v, cu, out=o, lse=lse)
        check(q, k, v, cu, o, lse, True)
        for rows in (slice(0, 37), slice(182, None)):
            assert (o[rows] == 7).all() and (lse[:, rows] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_mix(bad):
    """A sequence of NaN or Inf leaves its neighbours' bits alone."""
    q, k, v, cu = draw([70, 33, 150], 4, 4, 64, BF16, seed=4)
    o, lse = fa.forward_packed(q, k, v, cu, causal=False)
    for x in (q, k, v):
        x[70:103] = bad
    o2, lse2 = fa.forward_packed(q, k, v, cu, causal=False)
    for rows in (slice(0, 70), slice(103, 253)):
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (8, 2), (6, 2), (40, 1)])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_bad_neighbours_of_every_last_tile(H, Hk, d, dtype, causal):
    """Last key tiles that both query tiles of a block visit, that only the second
    one does, and that end one key in, each followed by a sequence of NaN or Inf."""
    lens = [200, 3, 129, 40, 257, 1, 385, 64, 5, 130, 66]
    q, k, v, cu = draw(lens, H, Hk, d, dtype, seed=44)
    o, lse = fa.forward_packed(q, k, v, cu, causal=causal)
    ends = cu.tolist()
    for bad in (float("nan"), float("-inf")):
        for s in range(1, len(lens), 2):
            for x in (q, k, v):
                x[ends[s]:ends[s + 1]] = bad
        o2, lse2 = fa.forward_packed(q, k, v, cu, causal=causal)
        for s in range(0, len(lens), 2):
            rows = slice(ends[s], ends[s + 1])
            assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])
    check(q[:200], k[:200], v[:200], cu[:2], o[:200], lse[:, :200], causal)


def test_scores_of_large_size():
    """Scores of magnitude 10^3: a running maximum that keeps growing."""
    q, k, v, cu = draw([300, 20], 2, 1, 128, BF16, seed=6)
    q, k = q * 8, k * 8
    k[:300] *= torch.linspace(0.1, 1.0, 300, device=DEV)[:, None, None].to(BF16)
    o, lse = fa.forward_packed(q, k, v, cu, scale=0.5)
    check(q, k, v, cu, o, lse, True, scale=0.5)


def test_matches_the_dense_forward():
    """Sequences of one length: fa_forward's own result (same tiles, other
    rows to a tile), to two roundings."""
    B, H, N, d = 3, 4, 384, 128
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(B, H, N, d, generator=g).to(BF16).to(DEV) for _ in range(3))
    o, lse = fa.forward(q, k, v, causal=True)
    pack = lambda x: x.transpose(1, 2).reshape(B * N, H, d).contiguous()  # noqa: E731
    cu = torch.arange(B + 1, device=DEV).int() * N
    o2, lse2 = fa.forward_packed(pack(q), pack(k), pack(v), cu.int())
    assert (pack(o).float() - o2.float()).abs().max() <= 2e-2
    assert (lse.transpose(0, 1).reshape(H, B * N) - lse2).abs().max() <= 1e-5


def draw_far(H, Hk, d, lens, seed):
    """`lens` behind so many rows of no sequence that q and o have more than
    2^31 values before them."""
    before = (1 << 31) // (H * d) + 5
    T = before + sum(lens)
    qkv = torch.empty(T, H + 2 * Hk, d, dtype=BF16, device=DEV)
    g = torch.Generator().manual_seed(seed)
    qkv[before:] = torch.randn(T - before, H + 2 * Hk, d, generator=g).to(BF16).to(DEV)
    cu = torch.tensor([before] + lens).cumsum(0).int().to(DEV)
    return qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], cu


@pytest.mark.parametrize("d", [64, 128])
def test_far_rows(d):
    q, k, v, cu = draw_far(32, 8, d, [300, 1, 77], seed=41)
    o, lse = fa.forward_packed(q, k, v, cu)
    check(q, k, v, cu, o, lse, True)


def test_without_lse_and_empty():
    q, k, v, cu = draw([40], 2, 1, 64, BF16, seed=1)
    o, lse = fa.forward_packed(q, k, v, cu, want_lse=False)
    check(q, k, v, cu, o, None, True)
    assert lse is None
    empty = torch.zeros(0, 2, 64, dtype=BF16, device=DEV)
    o, lse = fa.forward_packed(empty, empty, empty, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    # no sequence owns any row: nothing is written
    o = torch.full((40, 2, 64), 3.0, dtype=BF16, device=DEV)
    fa.forward_packed(q, k, v, torch.zeros(1, dtype=torch.int32, device=DEV), out=o)
    fa.forward_packed(q, k, v, torch.full((5,), 40, dtype=torch.int32, device=DEV), out=o)
    assert (o == 3).all()


def test_offsets_outside_the_tensor_are_clamped():
    """Offsets past the tensor are taken as its end, negative ones as its start."""
    q, k, v, cu = draw([40, 24], 2, 1, 64, BF16, seed=2)
    want, _ = fa.forward_packed(q, k, v, cu)
    got, _ = fa.forward_packed(q, k, v, torch.tensor([-5, 40, 1 << 30], device=DEV).int())
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0 and torch.equal(want, got)


def test_captured_and_concurrent_calls():
    """A graph replayed on new inputs, and two calls on two streams."""
    q, k, v, cu = draw([300, 41, 7], 8, 2, 128, BF16, seed=11)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        o, lse = fa.forward_packed(q, k, v, cu)
    for seed in (12, 13):
        q2, k2, v2, _ = draw([300, 41, 7], 8, 2, 128, BF16, seed)
        for x, y in ((q, q2), (k, k2), (v, v2)):
            x.copy_(y)
        cu.copy_(torch.tensor([0, 100 + seed, 200, 348]))
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = fa.forward_packed(q, k, v, cu)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i & 1]):
            outs.append(fa.forward_packed(q, k, v, cu)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


@pytest.mark.parametrize("call", ["forward_packed(q, k, v, cu)[0]",
                                  "qk_norm_rope(q, k, pos, freq)[0]"])
def test_first_call_of_a_process_is_captured(call):
    """The library's state is set up inside the capture, and the graph works."""
    code = f"""
import torch, exact_attention_11_gb300 as fa
g = torch.Generator().manual_seed(1)
q = torch.randn(70, 4, 128, generator=g).bfloat16().cuda()
k, v = (torch.randn(70, 2, 128, generator=g).bfloat16().cuda() for _ in range(2))
cu = torch.tensor([0, 30, 70]).int().cuda()
pos, freq = torch.arange(70).int().cuda(), fa.rope_frequencies(128, device="cuda")[0]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    x = fa.{call}
for _ in range(2):
    x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, fa.{call})
assert fa.fa_device_status() == 0
"""
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         timeout=300, cwd=os.path.dirname(os.path.dirname(fa.__file__)))
    assert run.returncode == 0, run.stderr[-2000:]


def test_two_graphs_of_many_launches_at_once():
    """Two graphs of 70 launches each, replayed on two streams at the same time:
    no launch of one shares its work counters with one of the other."""
    n, graphs = 70, []
    for seed in (31, 32):
        q, k, v, cu = draw([900, 300, 1100], 4, 2, 128, BF16, seed)
        want, _ = fa.forward_packed(q, k, v, cu)
        outs = torch.zeros(n, *q.shape, dtype=BF16, device=DEV)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(n):
                fa.forward_packed(q, k, v, cu, out=outs[i], want_lse=False)
        graphs.append((graph, stream, outs, want, (q, k, v, cu)))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, outs, _, _ in graphs:
            with torch.cuda.stream(stream):
                outs.zero_()
                graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for _, _, outs, want, _ in graphs:
        assert (outs == want[None]).all()


def test_helper_refuses():
    q, k, v, cu = draw([40], 4, 2, 64, BF16, seed=1)
    bad = [
        lambda: fa.forward_packed(q.float(), k.float(), v.float(), cu),
        lambda: fa.forward_packed(q, k[:20], v, cu),
        lambda: fa.forward_packed(q, k, v[:, :1], cu),
        lambda: fa.forward_packed(q, k, v.half(), cu),
        lambda: fa.forward_packed(q, k, v, cu.long()),
        lambda: fa.forward_packed(q, k, v, cu.cpu()),
        lambda: fa.forward_packed(q, k, v, cu[:0]),
        lambda: fa.forward_packed(q[:, ::2], k, v, cu),
        lambda: fa.forward_packed(q, k, v, cu, out=torch.empty_like(q)[:20]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for H, Hk, d in ((3, 2, 64), (2, 2, 256), (129, 1, 64)):
        q, k, v, cu = draw([4], H, Hk, d, BF16, seed=1)
        with pytest.raises(fa.FattnError):
            fa.forward_packed(q, k, v, cu)


def test_after_norm_and_rotation():
    """A layer's front half: norm, rotation, packed attention; against the
    same in float64 from the rounded queries and keys of the first step."""
    lens, H, Hk, d = [50, 3, 200], 8, 2, 128
    q, k, v, cu = draw(lens, H, Hk, d, BF16, seed=14)
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(DEV)
    g = torch.Generator().manual_seed(15)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF16).to(DEV) for _ in range(2))
    freq, _ = fa.rope_frequencies(d, device=DEV)
    qr, kr = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    want, size = qk_prep_ref.forward(q.cpu(), qw.cpu(), pos.cpu(), freq.cpu(), 1e-6, False, 1.0)
    assert ((qr.cpu().double() - want).abs() <= qk_prep_ref.bound(want, size, BF16)).all()
    o, lse = fa.forward_packed(qr, kr, v, cu)
    check(qr, kr, v, cu, o, lse, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_scores_of_minus_infinity(d, causal):
    """A query of -inf against positive keys: softmax of scores that are all -inf is
    NaN, as in the dense forward, and not a row of zeros; the other rows keep their bits."""
    q, k, v, cu = draw([1, 300, 40], 4, 2, d, BF16, seed=15)
    k.abs_()
    want, lse0 = fa.forward_packed(q, k, v, cu, causal=causal)
    rows = ((0, 1), (1, 3), (200, 0), (len(q) - 1, 2))
    for row, head in rows:
        q[row, head, 7] = float("-inf")
    o, lse = fa.forward_packed(q, k, v, cu, causal=causal)
    for row, head in rows:
        assert o[row, head].isnan().all() and not lse[head, row].isfinite()
        o[row, head], lse[head, row] = want[row, head], lse0[head, row]
    assert torch.equal(o, want) and torch.equal(lse, lse0)
    x = torch.ones(1, 1, 5, d, dtype=BF16, device=DEV)
    assert fa.forward(x * float("-inf"), x, x, causal=causal)[0].isnan().all()


@pytest.mark.parametrize("H,Hk,dtype", [(8, 1, F16), (2, 2, BF16)], ids=["8on1-fp16", "2-bf16"])
def test_a_prompt_of_16384(H, Hk, dtype):
    """The whole of it, by slices of query rows."""
    n, d = 16384, 128
    q, k, v, cu = draw([n], H, Hk, d, dtype, seed=16)
    o, lse = fa.forward_packed(q, k, v, cu)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for a in range(0, n, 512):
        r = slice(a, a + 512)
        x = ref.sequence(q[r], k[:a + 512], v[:a + 512], d ** -0.5, torch.arange(a, a + 512, device=DEV))
        ref.check_forward(o[r], lse[:, r], x, d ** -0.5, dtype)
