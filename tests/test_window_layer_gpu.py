"""Windowed attention and the shared prefix as a model uses them: with the norm and
rotation before and behind them, in training and in serving."""
import pytest
import torch

import exact_attention_11_gb300 as fa
import packed_ref
import window_ref
from test_backward_window_gpu import gradients
from test_forward_packed_gpu import draw_far
from test_paged_prefill_gpu import draw as draw_paged

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def projection(T, H, Hk, d, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * Hk, d, generator=g).to(BF16).to(DEV)
    w = torch.linspace(0.5, 1.5, d).to(BF16).to(DEV)
    return qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], w


def positions(lens):
    return torch.cat([torch.arange(n) for n in lens]).int().to(DEV)


@pytest.mark.parametrize("d", [64, 128])
def test_training_layer(d):
    """Norm, rotation, windowed attention, and the gradients back through both, each
    step held to the formulas on what the step before gave it."""
    lens, H, Hk, window, sinks = [200, 1, 333], 4, 2, 60, 4
    T = sum(lens)
    q, k, v, w = projection(T, H, Hk, d, 1)
    cu = torch.tensor([0] + lens).cumsum(0).int().to(DEV)
    freq, _ = fa.rope_frequencies(d, device=DEV)
    qr, kr = fa.qk_norm_rope(q, k, positions(lens), freq, w, w)
    o, lse = fa.forward_packed_window(qr, kr, v, cu, window, sinks)
    do = torch.randn(T, H, d, generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    grads = fa.backward_packed_window(qr, kr, v, o, lse, do, cu, window, sinks)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(grads[0], grads[1], q, k, positions(lens), freq,
                                                w, w)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = d ** -0.5
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        see = window_ref.near(torch.arange(b - a, device=DEV), b - a, window, sinks)
        r = window_ref.sequence(qr[a:b], kr[a:b], v[a:b], scale, see)
        packed_ref.check_forward(o[a:b], lse[:, a:b], r, scale, BF16)
        want = gradients(qr[a:b], kr[a:b], v[a:b], o[a:b], lse[:, a:b], do[a:b], scale, see)
        for x, (y, bound) in zip(grads, want):
            assert ((x[a:b].double() - y).abs() <= bound).all()
    for x in (dq, dk, dqw, dkw):
        assert torch.isfinite(x).all()
    assert dq.shape == q.shape and dkw.shape == (d,)


@pytest.mark.parametrize("window,sinks", [(50, 0), (100, 20), (700, 4)])
def test_serving_gives_what_training_gives(window, sinks):
    """Two prompts written into the cache in chunks of changing size, single tokens at
    the end, blocks given back as they leave the window and taken again by the other
    sequence: every token's row is the packed call's, within both calls' bounds."""
    lens, H, Hk, d = [430, 301], 8, 2, 128
    q, k, v, w = projection(sum(lens), H, Hk, d, 3)
    pos = positions(lens)
    cu = torch.tensor([0] + lens).cumsum(0).int().to(DEV)
    freq, _ = fa.rope_frequencies(d, device=DEV)
    qr, kr = fa.qk_norm_rope(q, k, pos, freq, w, w)
    want, _ = fa.forward_packed_window(qr, kr, v, cu, window, sinks)
    got = torch.zeros_like(want)
    nb = 2 * ((max(lens) + 15) // 16) + 2
    kc = torch.full((nb, Hk, 16, 16, 8), float("nan"), dtype=BF16, device=DEV)
    vc = torch.full((nb, Hk, 128, 16), float("nan"), dtype=BF16, device=DEV)
    free = list(range(nb))
    table = torch.full((2, (max(lens) + 15) // 16), -1, dtype=torch.int32)
    done = [0, 0]
    steps = [(100, 33), (1, 50), (129, 1), (7, 100), (190, 115), (1, 1), (1, 1), (1, 0)]
    for step in steps:
        rows, slots = [], []
        for s, n in enumerate(step):
            base = [0, lens[0]][s]
            for t in range(done[s], done[s] + n):
                if table[s, t // 16] < 0:
                    b = free.pop(0)
                    # what others left there is cleared, as an allocator of blocks does
                    kc[b], vc[b] = 0, 0
                    table[s, t // 16] = b
                rows.append(base + t)
                slots.append(table[s, t // 16].item() * 16 + t % 16)
            done[s] += n
        rows = torch.tensor(rows, device=DEV)
        qc = fa.qk_norm_rope_cache(q[rows], k[rows], v[rows], pos[rows].contiguous(), freq,
                                   torch.tensor(slots, device=DEV), kc, vc, w, w)
        out = fa.paged_prefill_window(
            qc, kc, vc, table.to(DEV), torch.tensor(done, dtype=torch.int32, device=DEV),
            torch.tensor([0, step[0], step[0] + step[1]], dtype=torch.int32, device=DEV), window,
            sinks)
        got[rows] = out
        for s in range(2):                  # blocks that no later token sees go back
            for b in range(done[s] // 16):
                if b * 16 >= sinks and b * 16 + 15 <= done[s] - window and table[s, b] >= 0:
                    free.append(table[s, b].item())
                    kc[table[s, b].item()] = float("nan")
                    vc[table[s, b].item()] = float("nan")
                    table[s, b] = -1
    torch.cuda.synchronize()
    assert done == lens and fa.fa_device_status() == 0
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        see = window_ref.near(torch.arange(b - a, device=DEV), b - a, window, sinks)
        r = window_ref.sequence(qr[a:b], kr[a:b], v[a:b], d ** -0.5, see)
        packed_ref.check_forward(got[a:b], None, r, d ** -0.5, BF16)
        packed_ref.check_forward(want[a:b], None, r, d ** -0.5, BF16)


def test_shared_prompt_served():
    """A prompt is prefilled once; twelve continuations share its whole blocks, each with
    a copy of the block it ends in, and grow token by token."""
    H, Hk, d, S, prompt = 8, 2, 128, 12, 650
    q, k, v, w = projection(prompt, H, Hk, d, 5)
    freq, _ = fa.rope_frequencies(d, device=DEV)
    whole, blocks = prompt // 16, (prompt + 15) // 16
    nb = blocks + S * 3
    kc = torch.zeros(nb, Hk, 16, 16, 8, dtype=BF16, device=DEV)
    vc = torch.zeros(nb, Hk, 128, 16, dtype=BF16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    one = torch.arange(blocks, **i32)[None].contiguous()
    at = torch.arange(prompt, device=DEV)
    qc = fa.qk_norm_rope_cache(q, k, v, at.int(), freq, at, kc, vc, w, w)
    fa.paged_prefill(qc, kc, vc, one, torch.tensor([prompt], **i32), torch.tensor([0, prompt], **i32))
    bt = torch.zeros(S, whole + 3, **i32)
    bt[:, :whole] = one[:, :whole]
    for s in range(S):
        mine = blocks + 3 * s
        bt[s, whole:] = torch.arange(mine, mine + 3)
        kc[mine], vc[mine] = kc[whole], vc[whole]
    cu, cg = torch.arange(S + 1, **i32), torch.tensor([0, S], **i32)
    n = 3
    draft = torch.arange(0, n * S + 1, n, **i32)
    for step, (rows, chunks) in enumerate([(S, cu)] * 20 + [(n * S, draft)]):
        q, k, v, w = projection(rows, H, Hk, d, 6 + step)
        new = rows // S
        pos = (prompt + step + torch.arange(new, device=DEV)).repeat(S)
        seq = torch.arange(S, device=DEV).repeat_interleave(new)
        slots = bt[seq, pos // 16].long() * 16 + pos % 16
        qc = fa.qk_norm_rope_cache(q, k, v, pos.int(), freq, slots, kc, vc, w, w)
        ctx = torch.full((S,), prompt + step + new, **i32)
        out = fa.paged_prefill_shared(qc, kc, vc, bt, ctx, chunks, cg,
                                      torch.tensor([prompt], **i32))
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        for s in range(S):
            tok = torch.arange(ctx[s].item(), device=DEV)
            kk = kc[bt[s].long()[tok // 16], :, :, tok % 16].flatten(2)
            vv = vc[bt[s].long()[tok // 16], :, :, tok % 16]
            last = prompt + step + torch.arange(new, device=DEV)
            mine = slice(s * new, (s + 1) * new)
            r = packed_ref.sequence(qc[mine], kk, vv, d ** -0.5, last)
            packed_ref.check_forward(out[mine], None, r, d ** -0.5, BF16)


@pytest.mark.parametrize("d", [64, 128])
def test_far_rows(d):
    """Rows behind more than 2^31 values of q, o and the accumulators."""
    H, Hk, window, sinks = 32, 8, 90, 3
    q, k, v, cu = draw_far(H, Hk, d, [300, 1, 177], seed=42)
    o, lse = fa.forward_packed_window(q, k, v, cu, window, sinks)
    do = torch.empty_like(o)
    a = cu[0].item()
    do[a:] = torch.randn(o[a:].shape, generator=torch.Generator().manual_seed(43)).to(BF16).to(DEV)
    grads = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        see = window_ref.near(torch.arange(b - a, device=DEV), b - a, window, sinks)
        r = window_ref.sequence(q[a:b], k[a:b], v[a:b], d ** -0.5, see)
        packed_ref.check_forward(o[a:b], lse[:, a:b], r, d ** -0.5, BF16)
        want = gradients(q[a:b], k[a:b], v[a:b], o[a:b], lse[:, a:b], do[a:b], d ** -0.5, see)
        for x, (y, bound) in zip(grads, want):
            assert ((x[a:b].double() - y).abs() <= bound).all()


def test_far_blocks_of_the_cache():
    """Blocks behind more than 2^32 bytes of the caches, one of them named twice."""
    H, Hk, S = 8, 4, 12
    nb = (1 << 32) // (Hk * 128 * 16 * 2) + 400
    kc = torch.empty(nb, Hk, 16, 16, 8, dtype=BF16, device=DEV)
    vc = torch.empty(nb, Hk, 128, 16, dtype=BF16, device=DEV)
    g = torch.Generator().manual_seed(8)
    kc[-400:] = torch.randn(400, Hk, 16, 16, 8, generator=g).to(BF16).to(DEV)
    vc[-400:] = torch.randn(400, Hk, 128, 16, generator=g).to(BF16).to(DEV)
    q = torch.randn(S, H, 128, generator=g).to(BF16).to(DEV)
    ids = nb - 400 + torch.randperm(400, generator=g)
    bt = torch.zeros(S, 30, dtype=torch.int64)
    bt[:, :20] = ids[:20]
    bt[:, 20:] = ids[20:20 + 10 * S].view(S, 10)
    bt[3, 25] = bt[3, 22]
    bt = bt.int().to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    ctx, cu = torch.full((S,), 470, **i32), torch.arange(S + 1, **i32)
    near = fa.paged_prefill_window(q, kc, vc, bt, ctx, cu, 200, 5)
    shared = fa.paged_prefill_shared(q, kc, vc, bt, ctx, cu, torch.tensor([0, S], **i32),
                                     torch.tensor([330], **i32))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    tok = torch.arange(470, device=DEV)
    for s in range(S):
        k = kc[bt[s].long()[tok // 16], :, :, tok % 16].flatten(2)
        v = vc[bt[s].long()[tok // 16], :, :, tok % 16]
        last = torch.tensor([469], device=DEV)
        for out, see in ((near, window_ref.near(last, 470, 200, 5)),
                         (shared, window_ref.near(last, 470, 1 << 20, 0))):
            r = window_ref.sequence(q[s:s + 1], k, v, 128 ** -0.5, see)
            packed_ref.check_forward(out[s:s + 1], None, r, 128 ** -0.5, BF16)


def check_gradients(q, k, v, cu, do, o, lse, grads):
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        see = window_ref.near(torch.arange(b - a, device=DEV), b - a, 70, 4)
        want = gradients(q[a:b], k[a:b], v[a:b], o[a:b], lse[:, a:b], do[a:b],
                         q.shape[-1] ** -0.5, see)
        for x, (y, bound) in zip(grads, want):
            assert ((x[a:b].double() - y).abs() <= bound).all()


def test_two_streams_at_once():
    """Calls on two streams, each with tensors and workspaces of its own."""
    calls = []
    for i in range(2):
        x = draw_paged([1, 30, 4], [3000, 5000, 800], 8, 2, seed=20 + i, poison=False)
        q, k, v, _ = projection(900, 4, 2, 64, 30 + i)
        cu = torch.tensor([0, 500, 900], dtype=torch.int32, device=DEV)
        do = torch.randn(900, 4, 64, device=DEV).to(BF16)

        def call(x=x, q=q, k=k, v=v, cu=cu, do=do):
            o, lse = fa.forward_packed_window(q, k, v, cu, 70, 4)
            grads = fa.backward_packed_window(q, k, v, o, lse, do, cu, 70, 4)
            return fa.paged_prefill_window(*x, 2500, 4), o, lse, grads
        calls.append((call, call(), (q, k, v, cu, do)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i][0]())
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for i in range(2):
        want = calls[i][1]
        for out in got[i]:
            for a, b in zip(out[:3], want[:3]):
                assert torch.equal(a, b)
            check_gradients(*calls[i][2], out[1], out[2], out[3])
