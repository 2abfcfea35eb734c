"""Norm and rotation of queries and keys against float64, the cache form
through the layouts of the paged decode, and the backward against the formulas
and against differences.  Tolerances: qk_prep_ref.bound."""
import numpy as np
import pytest
import torch

import oracle
import exact_attention_11_gb300 as fa
import qk_prep_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def draw(T, H, Hk, d, dtype, seed, extra=0, far=5000):
    """One projection's output [T, H + 2 Hk + extra, d] and views of it."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * Hk + extra, d, generator=g).to(dtype).to(DEV)
    pos = torch.randint(0, far, (T,), generator=g).int().to(DEV)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype).to(DEV) for _ in range(2)]
    return qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:H + 2 * Hk], pos, w[0], w[1]


def check(got, want, size, far=0.0):
    want, size = want.cpu(), size.cpu()
    err = (got.cpu().double() - want).abs()
    assert (err <= ref.bound(want, size, got.dtype, far)).all(), err.max().item()


def check_forward(q, k, pos, freq, qw, kw, eps, pairs, mscale, far=0.0):
    qo, ko = fa.qk_norm_rope(q, k, pos, freq, qw, kw, eps, pairs, mscale)
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        want, size = ref.forward(x.cpu(), None if w is None else w.cpu(), pos.cpu(), freq.cpu(),
                                 eps, pairs, mscale)
        check(o, want, size, far)
    return qo, ko


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256),
                                   (256, 64), (128, 0)])
@pytest.mark.parametrize("pairs", [False, True], ids=["half", "pairs"])
def test_forward(dtype, d, rot, pairs):
    """Strided views of a fused projection; every type, head size and layout."""
    freq, _ = fa.rope_frequencies(rot, device=DEV)
    for T, H, Hk in ((1, 1, 1), (7, 5, 1), (37, 8, 8)):
        q, k, _, pos, qw, kw = draw(T, H, Hk, d, dtype, seed=T + d + rot)
        check_forward(q, k, pos, freq, qw, kw, 1e-6, pairs, 1.0)


@pytest.mark.parametrize("T,H,Hk", [(2, 32, 8), (64, 32, 8), (1221, 3, 1), (2433, 2, 2),
                                    (5000, 1, 1)])
def test_forward_sizes(T, H, Hk):
    """One, two and four tokens a block, whole and ragged last tiles, heads
    spread over several blocks and not; weights on one side only."""
    freq, mscale = fa.rope_frequencies(96, scaling="yarn", factor=8.0, device=DEV)
    q, k, _, pos, qw, kw = draw(T, H, Hk, 128, BF16, seed=T)
    check_forward(q, k, pos, freq, qw, None, 1e-5, False, mscale)
    check_forward(q, k, pos, freq, None, kw, 1e-5, True, mscale)


def test_far_positions():
    """Angles of any int32 position, negative ones too."""
    freq, _ = fa.rope_frequencies(64, device=DEV)
    pos = torch.tensor([0, 1, -1, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31],
                       dtype=torch.int32, device=DEV)
    q, k, _, _, _, _ = draw(8, 2, 1, 64, F32, seed=5)
    for pairs in (False, True):
        check_forward(q, k, pos, freq, None, None, 1e-6, pairs, 1.0, far=2.0 ** 31)


def test_norm_of_small_zero_and_large_rows():
    q, k, _, pos, qw, kw = draw(6, 2, 1, 128, F32, seed=6)
    q, k = q.clone(), k.clone()
    q[0] = 0.0                 # the norm of nothing: eps keeps it finite
    q[1] *= 1e-20
    q[2] *= 1e15
    freq, _ = fa.rope_frequencies(128, device=DEV)
    qo, _ = check_forward(q, k, pos, freq, qw, kw, 1e-6, False, 1.0)
    assert (qo[0] == 0).all()


def test_rows_do_not_mix():
    """NaN and Inf in one row leave every other row's bits alone."""
    freq, _ = fa.rope_frequencies(64, device=DEV)
    q, k, _, pos, qw, kw = draw(9, 4, 2, 64, BF16, seed=7)
    q, k = q.contiguous(), k.contiguous()
    a = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    q2, k2 = q.clone(), k.clone()
    q2[3, 1, 5], k2[8, 0, 63] = float("nan"), float("inf")
    b = fa.qk_norm_rope(q2, k2, pos, freq, qw, kw)
    keep = torch.ones(9, 4, dtype=torch.bool)
    keep[3, 1] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][3, 1]).all()
    keep = torch.ones(9, 2, dtype=torch.bool)
    keep[8, 0] = False
    assert torch.equal(a[1][keep], b[1][keep])


def test_in_place_and_given_outputs():
    freq, _ = fa.rope_frequencies(128, device=DEV)
    q, k, _, pos, qw, kw = draw(33, 6, 3, 128, BF16, seed=8)
    q, k = q.contiguous(), k.contiguous()
    qo, ko = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    fa.qk_norm_rope(q, k, pos, freq, qw, kw, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_no_tokens():
    freq, _ = fa.rope_frequencies(64, device=DEV)
    q, k, v, pos, qw, kw = draw(0, 4, 2, 128, BF16, seed=1)
    qo, ko = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(qo, ko, q, k, pos, freq, qw, kw)
    assert dq.shape == q.shape and (dqw == 0).all() and (dkw == 0).all()


# ------------------------------------------------------------- the cache form
def caches(nb, Hk, seed):
    g = torch.Generator().manual_seed(seed)
    kc = torch.randn(nb, Hk, 16, 16, 8, generator=g).to(BF16).to(DEV)
    vc = torch.randn(nb, Hk, 128, 16, generator=g).to(BF16).to(DEV)
    return kc, vc


def slots_of(kind, T, nb, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "scattered":
        return torch.randperm(nb * 16, generator=g)[:T]
    if kind == "run":                       # a prompt from a block's start
        return 16 + torch.arange(T)
    if kind == "offset_run":                # ... from the middle of a block
        return 16 + 5 + torch.arange(T)
    if kind == "runs":                      # short runs, some backwards, some at odd places
        s = torch.randperm(nb * 4, generator=g)[:(T + 2) // 3] * 4 + 1
        return torch.stack([s, s + 1, s + 2], 1).flatten()[:T]
    s = torch.arange(T).flip(0)             # "padded": reversed, with entries to skip
    s[::5] = -1
    if T > 7:
        s[7] = nb * 16
    if T > 8:
        s[8] = 2 ** 62
    return s


@pytest.mark.parametrize("kind", ["scattered", "run", "offset_run", "runs", "padded"])
@pytest.mark.parametrize("T,H,Hk", [(1, 4, 1), (16, 8, 2), (53, 6, 3), (700, 8, 8), (1300, 2, 1),
                                    (2501, 3, 1), (5003, 1, 1)])
def test_cache_form(kind, T, H, Hk):
    nb = 2 * (T + 15) // 16 + 4
    q, k, v, pos, qw, kw = draw(T, H, Hk, 128, BF16, seed=T + len(kind), extra=1)
    freq, _ = fa.rope_frequencies(64, device=DEV)
    kc, vc = caches(nb, Hk, seed=T)
    slots = slots_of(kind, T, nb, seed=T).long()
    want_k, want_v = kc.cpu().clone(), vc.cpu().clone()
    qd, kd = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    qo = fa.qk_norm_rope_cache(q, k, v, pos, freq, slots.to(DEV), kc, vc, qw, kw)
    torch.cuda.synchronize()
    assert torch.equal(qo, qd)              # the dense form's values, bit for bit
    t = torch.nonzero((slots >= 0) & (slots < nb * 16)).flatten()
    s = slots[t]
    want_k[s // 16, :, :, s % 16] = kd.cpu()[t].view(-1, Hk, 16, 8)
    want_v[s // 16, :, :, s % 16] = v.cpu()[t]
    assert torch.equal(kc.cpu(), want_k)    # and no other slot has changed
    assert torch.equal(vc.cpu(), want_v)


def test_cache_form_feeds_the_decode():
    """Prompts written token by token and in one call, then decoded."""
    H, Hk, lens = 8, 2, [37, 1, 150]
    nb, mb = 32, 10
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(3))[:3 * mb].view(3, mb)
    T = sum(lens)
    q, k, v, _, qw, kw = draw(T, H, Hk, 128, BF16, seed=9)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens))
    pos = torch.cat([torch.arange(n) for n in lens])
    slots = (bt[seq, pos // 16] * 16 + pos % 16).to(DEV)
    pos = pos.int().to(DEV)
    freq, _ = fa.rope_frequencies(128, device=DEV)
    kc, vc = caches(nb, Hk, seed=4)
    kc2, vc2 = kc.clone(), vc.clone()
    qo = fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc, qw, kw)
    for t in range(T):
        fa.qk_norm_rope_cache(q[t:t + 1], k[t:t + 1], v[t:t + 1], pos[t:t + 1], freq,
                              slots[t:t + 1], kc2, vc2, qw, kw)
    torch.cuda.synchronize()
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    last = torch.tensor([sum(lens[:i + 1]) - 1 for i in range(3)], device=DEV)
    bt = bt.int().to(DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = fa.paged_decode(qo[last], kc, vc, bt, ctx)
    torch.cuda.synchronize()
    want, _ = oracle.paged_decode(qo[last], kc, vc, bt, ctx, 128 ** -0.5)
    assert np.abs(out.float().cpu().numpy() - want).max() <= 2e-2


def test_cache_form_in_place():
    T, H, Hk = 37, 6, 2
    q, k, v, pos, qw, kw = draw(T, H, Hk, 128, BF16, seed=51)
    freq, _ = fa.rope_frequencies(128, device=DEV)
    slots = torch.arange(T, device=DEV)
    kc, vc = caches(4, Hk, seed=52)
    want = fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc, qw, kw)
    x = q.contiguous()
    got = fa.qk_norm_rope_cache(x, k, v, pos, freq, slots, kc, vc, qw, kw, q_out=x)
    torch.cuda.synchronize()
    assert got is x and torch.equal(x, want)


def test_cache_form_same_slot_twice():
    """Each stored value is one of the tokens' that name its slot; no other slot
    changes."""
    T, Hk, nb = 40, 2, 8
    q, k, v, pos, qw, kw = draw(T, 3, Hk, 128, BF16, seed=53)
    freq, _ = fa.rope_frequencies(128, device=DEV)
    kc, vc = caches(nb, Hk, seed=54)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.randint(16, 16 + T // 2, (T,), generator=torch.Generator().manual_seed(55))
    slots[20:30] = torch.arange(48, 53).repeat_interleave(2)
    _, kd = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    fa.qk_norm_rope_cache(q, k, v, pos, freq, slots.to(DEV), kc, vc, qw, kw)
    torch.cuda.synchronize()
    for s in range(nb * 16):
        at = torch.nonzero(slots == s).flatten().to(DEV)
        got_k, got_v = kc[s // 16, :, :, s % 16].flatten(1), vc[s // 16, :, :, s % 16]
        if len(at) == 0:
            at_k, at_v = k0[s // 16, :, :, s % 16].flatten(1)[None], v0[s // 16, :, :, s % 16][None]
        else:
            at_k, at_v = kd[at], v[at]
        assert (at_k == got_k[None]).any(0).all() and (at_v == got_v[None]).any(0).all()


def test_cache_form_far_slots():
    """Caches of more than 2^32 values each: the last block, and two around the
    place where a 32-bit index of values would turn over."""
    Hk = 8
    nb = (1 << 32) // (Hk * 16 * 128) + 3
    T = 48
    q, k, v, pos, qw, kw = draw(T, 8, Hk, 128, BF16, seed=56)
    freq, _ = fa.rope_frequencies(128, device=DEV)
    kc = torch.empty(nb, Hk, 16, 16, 8, dtype=BF16, device=DEV)
    vc = torch.empty(nb, Hk, 128, 16, dtype=BF16, device=DEV)
    blocks = torch.tensor([nb - 1, (1 << 31) // (Hk * 16 * 128), (1 << 32) // (Hk * 16 * 128)])
    slots = (blocks[:, None] * 16 + torch.arange(16)).flatten().to(DEV)
    kc[0], vc[0] = 3.0, 3.0
    _, kd = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    qo = fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc, qw, kw)
    torch.cuda.synchronize()
    b = blocks.to(DEV)
    assert torch.equal(kc[b].permute(0, 3, 1, 2, 4).reshape(T, Hk, 128), kd)
    assert torch.equal(vc[b].permute(0, 3, 1, 2).reshape(T, Hk, 128), v)
    assert (kc[0] == 3).all() and (vc[0] == 3).all()
    # ... and the chunk that reads them back equals the one from a small cache
    bt = torch.tensor([[2, 0, 1]], device=DEV)
    ctx, cu = torch.tensor([T], device=DEV).int(), torch.tensor([0, T], device=DEV).int()
    far = fa.paged_prefill(qo, kc, vc, b[bt].int(), ctx, cu)
    near = fa.paged_prefill(qo, kc[b].contiguous(), vc[b].contiguous(), bt.int(), ctx, cu)
    torch.cuda.synchronize()
    assert torch.equal(far, near)


# ----------------------------------------------------------------- backward
def check_backward(T, H, Hk, d, rot, dtype, pairs, norm, seed, mscale=1.0):
    q, k, _, pos, qw, kw = draw(T, H, Hk, d, dtype, seed)
    qw, kw = (qw if norm in ("both", "q") else None), (kw if norm in ("both", "k") else None)
    freq, _ = fa.rope_frequencies(rot, device=DEV)
    g = torch.Generator().manual_seed(seed + 1)
    dqo = torch.randn(T, H, d, generator=g).to(dtype).to(DEV)
    dko = torch.randn(T, Hk, d, generator=g).to(dtype).to(DEV)
    got = fa.qk_norm_rope_backward(dqo, dko, q, k, pos, freq, qw, kw, 1e-6, pairs, mscale)
    for x, dy, w, dx, dw in ((q, dqo, qw, got[0], got[2]), (k, dko, kw, got[1], got[3])):
        want, size, want_w, size_w = ref.backward(dy.cpu(), x.cpu(), None if w is None else w.cpu(),
                                                  pos.cpu(), freq.cpu(), 1e-6, pairs, mscale)
        check(dx, want, size)
        if w is None:
            assert dw is None
            continue
        # fp32 sums: each term to 64 u as in the bound, a thread's rows one
        # after another, then at most 5 + 8 + 19 + 32 more additions.
        rows = 1 + T * x.shape[1] * (d // 16) // 256
        err = (dw.cpu().double() - want_w).abs()
        assert (err <= (128 + min(rows, 4 * x.shape[1])) * 2.0 ** -24 * size_w).all()
    return got


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128), (256, 64), (128, 0)])
@pytest.mark.parametrize("pairs", [False, True], ids=["half", "pairs"])
def test_backward(dtype, d, rot, pairs):
    for T, H, Hk, norm in ((1, 1, 1, "both"), (13, 6, 2, "both"), (5, 4, 1, "q"), (9, 2, 2, "k"),
                           (6, 3, 3, "none")):
        check_backward(T, H, Hk, d, rot, dtype, pairs, norm, seed=T + d, mscale=1.1)


def test_backward_many_tiles_repeats_exactly():
    """More tiles than blocks; the weights' gradients agree bit for bit."""
    a = check_backward(4001, 4, 2, 128, 128, BF16, False, "both", seed=3)
    b = check_backward(4001, 4, 2, 128, 128, BF16, False, "both", seed=3)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -130])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (13, 6, 2), (9, 3, 5)])
def test_backward_without_eps(eps, T, H, Hk):
    """Threads without a row add nothing to the weights' gradients; with an eps
    below fp32's normal range a row of zeros keeps its gradient, r w g."""
    q, k, _, pos, qw, kw = draw(T, H, Hk, 128, F32, seed=T)
    freq, _ = fa.rope_frequencies(64, device=DEV)
    if eps:
        q[T // 2, 0] = 0.0
    g = torch.Generator().manual_seed(T + 1)
    dqo = 1e-3 * torch.randn(T, H, 128, generator=g).to(DEV)
    dko = 1e-3 * torch.randn(T, Hk, 128, generator=g).to(DEV)
    got = fa.qk_norm_rope_backward(dqo, dko, q, k, pos, freq, qw, kw, eps)
    for x, dy, w, dx, dw in ((q, dqo, qw, got[0], got[2]), (k, dko, kw, got[1], got[3])):
        want, size, want_w, size_w = ref.backward(dy.cpu(), x.cpu(), w.cpu(), pos.cpu(),
                                                  freq.cpu(), eps, False, 1.0)
        check(dx, want, size)
        assert ((dw.cpu().double() - want_w).abs() <= 256 * 2.0 ** -24 * size_w).all()


def test_backward_against_differences():
    """The fp32 gradient along a random direction against central differences
    of the float64 forward (error of the differences ~ h^2 = 1e-8)."""
    T, H, Hk, d, rot = 5, 3, 1, 64, 32
    q, k, _, pos, qw, kw = draw(T, H, Hk, d, F32, seed=21)
    freq, _ = fa.rope_frequencies(rot, device=DEV)
    g = torch.Generator().manual_seed(22)
    dqo = torch.randn(T, H, d, generator=g)
    dko = torch.randn(T, Hk, d, generator=g)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(dqo.to(DEV), dko.to(DEV), q, k, pos, freq, qw, kw)
    for x, w, dy, dx, dw in ((q, qw, dqo, dq, dqw), (k, kw, dko, dk, dkw)):
        x, w, dx, dw = (t.cpu().double() for t in (x, w, dx, dw))
        vx, vw = torch.randn(x.shape, generator=g).double(), torch.randn(d, generator=g).double()

        def loss(s):
            y, _ = ref.forward(x + s * vx, w + s * vw, pos.cpu(), freq.cpu(), 1e-6, False, 1.0)
            return (y * dy.double()).sum()
        h = 1e-4
        slope = (loss(h) - loss(-h)) / (2 * h)
        mine = (dx * vx).sum() + (dw * vw).sum()
        scale = (dx * vx).abs().sum() + (dw * vw).abs().sum()
        assert abs(slope - mine) <= 1e-6 * scale


def test_captured_calls_replay():
    """Forward, cache form and backward in one graph, replayed on new inputs."""
    T, H, Hk = 40, 4, 2
    q, k, v, pos, qw, kw = draw(T, H, Hk, 128, BF16, seed=31)
    freq, _ = fa.rope_frequencies(128, device=DEV)
    kc, vc = caches(8, Hk, seed=1)
    slots = (torch.arange(T) + 3).long().to(DEV)
    dq_out, dk_out = torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous())
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qo = fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc, qw, kw)
        grads = fa.qk_norm_rope_backward(dq_out, dk_out, q, k, pos, freq, qw, kw)
    for seed in (32, 33):
        q2 = draw(T, H, Hk, 128, BF16, seed)[0]
        q.copy_(q2)
        graph.replay()
        torch.cuda.synchronize()
        kc2, vc2 = caches(8, Hk, seed=1)
        assert torch.equal(qo, fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc2, vc2, qw, kw))
        for a, b in zip(grads, fa.qk_norm_rope_backward(dq_out, dk_out, q, k, pos, freq, qw, kw)):
            assert torch.equal(a, b)
        sel = torch.arange(3, 3 + T)
        assert torch.equal(kc[sel // 16, :, :, sel % 16], kc2[sel // 16, :, :, sel % 16])


def test_helpers_refuse():
    freq, _ = fa.rope_frequencies(64, device=DEV)
    q, k, v, pos, qw, kw = draw(4, 4, 2, 128, BF16, seed=1)
    kc, vc = caches(2, 2, seed=1)
    slots = torch.arange(4, device=DEV)
    bad = [
        lambda: fa.qk_norm_rope(q, k.half(), pos, freq, qw, kw),
        lambda: fa.qk_norm_rope(q, k[:3], pos, freq, qw, kw),
        lambda: fa.qk_norm_rope(q, k, pos.long(), freq, qw, kw),
        lambda: fa.qk_norm_rope(q, k, pos, freq.float(), qw, kw),
        lambda: fa.qk_norm_rope(q, k, pos, freq, qw[:64], kw),
        lambda: fa.qk_norm_rope(q[:, ::2], k, pos, freq, qw, kw),        # heads not dense
        lambda: fa.qk_norm_rope(q, k, pos.cpu(), freq, qw, kw),
        lambda: fa.qk_norm_rope_cache(q, k, v[:, :1], pos, freq, slots, kc, vc),
        lambda: fa.qk_norm_rope_cache(q, k, v, pos, freq, slots.int(), kc, vc),
        lambda: fa.qk_norm_rope_cache(q, k, v, pos, freq, slots, kc, vc[:1]),
        lambda: fa.qk_norm_rope_cache(q.half(), k.half(), v.half(), pos, freq, slots, kc, vc),
        lambda: fa.qk_norm_rope_backward(q, k.contiguous(), q, k, pos, freq),  # not dense
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fa.FattnError):                                  # rot_dim 40
        fa.qk_norm_rope(q, k, pos, fa.rope_frequencies(40, device=DEV)[0], qw, kw)
