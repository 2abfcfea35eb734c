"""Gradients of the windowed forward against the float64 formulas and against
differences of the float64 forward.  Bounds: those of test_backward_packed_gpu,
which hold pair by pair, over the visible pairs."""
import pytest
import torch

import exact_attention_11_gb300 as fa
import window_ref
from test_forward_packed_gpu import draw

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
H8, U = 2.0 ** -8, 2.0 ** -24


def gradients(q, k, v, o, lse, do, scale, see):
    """(value, bound) of dQ, dK, dV of one sequence."""
    n, H, d = q.shape
    Hk = k.shape[1]
    g = H // Hk
    q, o, do = (x.double().transpose(0, 1) for x in (q, o, do))
    k, v = (x.double().transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    s = q @ t(k) * scale
    p = torch.where(see, torch.exp(s - lse.double()[..., None]), 0.0)
    mag = q.abs() @ t(k.abs())
    e = scale * mag * d * U + 2.0 ** -20 + 2.0 ** -22 * (lse.abs()[..., None] + scale * mag)
    dp = do @ t(v)
    dd = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - dd)
    ds_err = (H8 * 1.01 + e) * ds.abs() + \
        p * d * U * (do.abs() @ t(v.abs()) + (do * o).abs().sum(-1, keepdim=True))
    ds_all = ds_err + 2.0 ** -12 * (ds.abs() + p * (dp.abs() + dd.abs()) * U * 8)
    p_all = (H8 * 1.01 + e + 2.0 ** -12) * p
    fold = lambda x: x.unflatten(0, (Hk, g)).sum(1)  # noqa: E731
    dq, dq_e = scale * ds @ k, scale * ds_all @ k.abs()
    dk, dk_e = fold(scale * t(ds) @ q), fold(scale * t(ds_all) @ q.abs())
    dv, dv_e = fold(t(p) @ do), fold(t(p_all) @ do.abs())
    return [(x.transpose(0, 1), (H8 * (x.abs() + b) + b + 1e-30).transpose(0, 1))
            for x, b in ((dq, dq_e), (dk, dk_e), (dv, dv_e))]


def check(q, k, v, cu, o, lse, do, got, window, sinks, scale=None):
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = scale or q.shape[-1] ** -0.5
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        r = slice(a, b)
        see = window_ref.near(torch.arange(b - a, device=DEV), b - a, window, sinks)
        want = gradients(q[r], k[r], v[r], o[r], lse[:, r], do[r], scale, see)
        for name, x, (y, bound) in zip(("dQ", "dK", "dV"), got, want):
            err = (x[r].double() - y).abs()
            assert (err <= bound).all(), \
                f"{name}, rows {a}..{b}: {(err / bound).max().item():.3g} of its bound"


def inputs(lens, H, Hk, d, window, sinks, seed, **kw):
    q, k, v, cu = draw(lens, H, Hk, d, BF16, seed, **kw)
    o, lse = fa.forward_packed_window(q, k, v, cu, window, sinks)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 1)).to(BF16).to(DEV)
    return q, k, v, o, lse, do, cu


def run(lens, H, Hk, d, window, sinks, seed, **kw):
    q, k, v, o, lse, do, cu = inputs(lens, H, Hk, d, window, sinks, seed, **kw)
    got = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
    check(q, k, v, cu, o, lse, do, got, window, sinks)


WINDOWS = [(1, 0), (1, 1), (2, 130), (7, 0), (63, 4), (64, 64), (65, 65), (127, 128), (128, 0),
           (128, 129), (129, 127), (130, 1), (200, 300), (256, 0), (1000, 4), (40, 1025)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, d):
    """Grouped heads (accumulators for all) and one query head a key/value head
    (accumulators for the blocks of first tokens only)."""
    lens = [1, 130, 0, 1700, 33, 513, 128]
    run(lens, 4, 2, d, window, sinks, seed=window + sinks)
    run(lens, 2, 2, d, window, sinks, seed=window + sinks + 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (8, 2), (6, 2), (7, 1), (3, 3)])
def test_heads(H, Hk, d):
    run([1, 130, 0, 64, 33, 400], H, Hk, d, 50, 5, seed=H + d)


@pytest.mark.parametrize("d", [64, 128])
def test_far_queries_of_the_first_tokens(d):
    """Several items per block of first tokens: more steps than an item takes."""
    run([3900, 2000, 20], 2, 1, d, 100, 4, seed=1)
    run([3900, 2000, 20], 1, 1, d, 100, 260, seed=2)
    run([3900, 1100], 1, 1, d, 1200, 1000, seed=3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H,Hk,window,sinks", [
    ([2500, 700, 1, 900], 32, 8, 40, 0),
    ([2500, 700, 129, 0, 900], 32, 8, 200, 4),
    ([1900, 1900, 5, 1900, 1900], 28, 4, 100, 300),
    ([64] * 30 + [3300, 900], 32, 4, 33, 130),
    ([4000], 16, 8, 257, 1),
    ([1111] * 9, 40, 2, 64, 16),
])
def test_items_with_all_heads_of_a_group(lens, H, Hk, window, sinks, d):
    """Enough key blocks that an item takes all query heads of a key/value head and
    stores dK and dV itself, beside others that add them up."""
    run(lens, H, Hk, d, window, sinks, seed=len(lens))


def test_every_length_and_many_windows():
    for d in (64, 128):
        run(list(range(1, 258, 3)), 1, 1, d, 20, 2, seed=5)
        run(list(range(2, 400, 5)), 2, 1, d, 130, 0, seed=6)
    q, k, v, cu = draw([300], 1, 1, 64, BF16, 7)
    do = torch.randn_like(q)
    for window in list(range(1, 140)) + [190, 191, 192, 193, 255, 256, 257, 299, 300]:
        sinks = window % 5
        o, lse = fa.forward_packed_window(q, k, v, cu, window, sinks)
        got = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
        check(q, k, v, cu, o, lse, do, got, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_per_sm(d):
    run([1500, 1, 257, 2049, 640, 5], 8, 2, d, 300, 4, seed=9)
    run([1000, 77, 900], 8, 8, d, 64, 1, seed=10)


@pytest.mark.parametrize("S", [255, 1100, 2048, 2049])
def test_many_sequences(S):
    """Sorted block tables, with far items of the first tokens, and unsorted ones,
    where an item visits them all."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, 9, (S,), generator=g).tolist()
    lens[S // 2] = 1500
    run(lens, 2, 1, 64, 6, 2, seed=2)
    run(lens, 1, 1, 64, 30, 2, seed=3)


def test_a_window_over_everything_is_the_causal_mask():
    """The same items in the same order; dQ, summed by atomics, to rounding."""
    q, k, v, o, lse, do, cu = inputs([400, 90, 200], 3, 3, 64, 400, 5, seed=3)
    a = fa.backward_packed(q, k, v, o, lse, do, cu)
    for sinks in (0, 5, 400):
        b = fa.backward_packed_window(q, k, v, o, lse, do, cu, 400, sinks)
        check(q, k, v, cu, o, lse, do, b, 400, sinks)
    assert torch.equal(a[2], b[2])


def test_decreasing_offsets_stay_inside():
    q, k, v, o, lse, do, cu = inputs([40, 300, 24], 2, 1, 64, 30, 3, seed=5)
    for bad in ([364, 0, 300, 10], [300, 100, 364, 50], [1 << 30, -5, 7, 0]):
        cu2 = torch.tensor(bad, device=DEV).int()
        fa.forward_packed_window(q, k, v, cu2, 30, 3)
        fa.backward_packed_window(q, k, v, o, lse, do, cu2, 30, 3)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
    got = fa.backward_packed_window(q, k, v, o, lse, do, cu, 30, 3)
    check(q, k, v, cu, o, lse, do, got, 30, 3)


def test_rows_of_no_sequence_stay_and_do_not_leak():
    q, k, v, o, lse, do, cu = inputs([100, 245], 4, 2, 128, 60, 2, seed=3, before=37, behind=200)
    for x in (o, do, lse.t()):
        x[:37] = float("nan")
        x[382:] = float("nan")
    T = q.shape[0]
    outs = [torch.full((T, h, 128), 7.0, dtype=BF16, device=DEV) for h in (4, 2, 2)]
    n = fa.fa_backward_packed_window_workspace_bytes(2, T, 4, 2, 128, 60, 2)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    fa.fa_backward_packed_window(
        *(x.data_ptr() for x in (q, k, v, o, do, lse, *outs, cu)), 2, T, 4, 2, 128, q.stride(0),
        k.stride(0), v.stride(0), 128 ** -0.5, 60, 2, ws.data_ptr(), n, 0)
    check(q, k, v, cu, o, lse, do, outs, 60, 2)
    for x in outs:
        assert (x[:37] == 7).all() and (x[382:] == 7).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_mix(bad):
    q, k, v, o, lse, do, cu = inputs([70, 200, 150], 4, 4, 64, 40, 3, seed=4)
    for x in (q, k, v, o, do, lse.t()):
        x[70:270] = bad
    got = fa.backward_packed_window(q, k, v, o, lse, do, cu, 40, 3)
    for a, b in ((0, 70), (270, 420)):
        check(q[a:b], k[a:b], v[a:b], torch.tensor([0, b - a]), o[a:b], lse[:, a:b], do[a:b],
              [x[a:b] for x in got], 40, 3)


def test_against_differences():
    """Directional differences of the float64 forward's sum(o * do), within twice the
    gradients' bounds (once for the kernel against the formula, once for the formula's
    lse, an fp32 value, against the true one) plus what the given o does to D: o has P
    and itself rounded (bf16), so D is off by at most
    dD_i = H8 sum_c |do_ic| (|o_ic| + 1.01 sum_j P_ij |v_jc|), dQ by scale sum_j P dD |K|
    and dK by scale sum_i P dD |Q|."""
    n, H, Hk, d, window, sinks = 150, 2, 1, 64, 20, 3
    scale = d ** -0.5
    q, k, v, o, lse, do, cu = inputs([n], H, Hk, d, window, sinks, seed=21)
    got = fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
    see = window_ref.near(torch.arange(n, device=DEV), n, window, sinks)
    want = gradients(q, k, v, o, lse, do, scale, see)
    base = [x.double() for x in (q, k, v)]
    ro, rl, pv, _, _ = window_ref.sequence(*base, scale, see)
    p = torch.where(see, torch.exp(torch.einsum("nhd,md->hnm", base[0], base[1][:, 0]) * scale
                                   - rl[..., None]), 0.0)
    off = p * (H8 * (do.double().abs() * (o.double().abs() + 1.01 * pv)).sum(-1).t()[..., None])
    extra = (scale * torch.einsum("hnm,md->nhd", off, base[1][:, 0].abs()),
             scale * torch.einsum("hnm,nhd->md", off, base[0].abs())[:, None], 0.0)

    def loss(x):
        return (window_ref.sequence(*x, scale, see)[0] * do.double()).sum()

    for i, (g, (_, bound)) in enumerate(zip(got, want)):
        step = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i)).to(DEV).double()
        h = 1e-5
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + h * step, base[i] - h * step
        diff = (loss(plus) - loss(minus)) / (2 * h)
        slack = ((2 * bound + extra[i]) * step.abs()).sum() + 1e-6 * (1 + abs(diff))
        assert abs((g.double() * step).sum() - diff) <= slack


def test_repeats_and_captures():
    """Replayed with new values, and with an eager call of the same tensors between."""
    q, k, v, o, lse, do, cu = inputs([300, 700], 4, 2, 64, 90, 4, seed=30)
    n = fa.fa_backward_packed_window_workspace_bytes(2, 1000, 4, 2, 64, 90, 4)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    fa.backward_packed_window(q, k, v, o, lse, do, cu, 90, 4, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.backward_packed_window(q, k, v, o, lse, do, cu, 90, 4, workspace=ws)
    for lens in ([300, 700], [1, 999], [0, 20]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).int())
        q.normal_()
        fa.forward_packed_window(q, k, v, cu, 90, 4, out=o, lse=lse)
        graph.replay()
        fa.backward_packed_window(q, k, v, o, lse, do, cu, 90, 4)
        check(q, k, v, cu, o, lse, do, got, 90, 4)


def test_refusals():
    q, k, v, o, lse, do, cu = inputs([30], 2, 1, 64, 9, 0, seed=1)
    for window, sinks in ((0, 0), (4, -1)):
        with pytest.raises(ValueError):
            fa.backward_packed_window(q, k, v, o, lse, do, cu, window, sinks)
    with pytest.raises(ValueError):
        fa.backward_packed_window(q, k, v, o[:, :1], lse, do, cu, 9)
    small = torch.empty(64, dtype=torch.uint8, device=DEV)
    with pytest.raises(fa.FattnError):
        fa.backward_packed_window(q, k, v, o, lse, do, cu, 9, workspace=small)
