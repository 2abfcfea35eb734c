"""Gradients of the packed forward against the float64 formulas and against
differences of the float64 forward.

Bounds.  With P, dP, D, dS in float64 from the bf16 inputs (and from the bf16 o
and fp32 lse that the call is given), u = 2^-24 and h = 2^-8 (a bf16 rounding):
    P    off by e P, e as in packed_ref.check_forward, and once rounded: (h + e) P
    dP   off by d u sum |dO||V|;   D off by d u sum |dO||o|
    dS   = P (dP - D): (h + e) |dS| + P (the two above)
    dV   <= sum_i (h + e) P |dO|;   dQ, dK <= scale sum |dS's error| |K| or |Q|
fp32 accumulation adds at most (rows + 8) u of the sums of sizes (below 2^-12 of
them for the lengths here), and the result is rounded once (h)."""
import pytest
import torch

import exact_attention_11_gb300 as fa
from test_forward_packed_gpu import draw, draw_far

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
H8, U = 2.0 ** -8, 2.0 ** -24


def gradients(q, k, v, o, lse, do, scale, causal):
    """(value, bound) of dQ, dK, dV of one sequence."""
    n, H, d = q.shape
    Hk = k.shape[1]
    g = H // Hk
    q, o, do = (x.double().transpose(0, 1) for x in (q, o, do))
    k, v = (x.double().transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    i = torch.arange(n, device=DEV)
    see = (i[None, :] <= i[:, None]) if causal else torch.ones(n, n, device=DEV) > 0
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


def check(q, k, v, cu, o, lse, do, got, causal, scale=None):
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    scale = scale or q.shape[-1] ** -0.5
    cu = cu.tolist()
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        r = slice(a, b)
        want = gradients(q[r], k[r], v[r], o[r], lse[:, r], do[r], scale, causal)
        for name, x, (y, bound) in zip(("dQ", "dK", "dV"), got, want):
            err = (x[r].double() - y).abs()
            assert (err <= bound).all(), \
                f"{name}, rows {a}..{b}: {(err / bound).max().item():.3g} of its bound"


def run(lens, H, Hk, d, causal, seed, **kw):
    q, k, v, cu = draw(lens, H, Hk, d, BF16, seed, **kw)
    o, lse = fa.forward_packed(q, k, v, cu, causal=causal)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 1)).to(BF16).to(DEV)
    got = fa.backward_packed(q, k, v, o, lse, do, cu, causal=causal)
    check(q, k, v, cu, o, lse, do, got, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (8, 2), (6, 2), (7, 1), (3, 3)])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_heads(H, Hk, d, causal):
    run([1, 130, 0, 64, 33, 200], H, Hk, d, causal, seed=H + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [128], [129], [255, 256, 257],
                                  [2, 1, 1, 3], [0, 5, 0, 0], [700, 31, 1100]], ids=str)
def test_lengths(lens, d, causal):
    run(lens, 4, 2, d, causal, seed=sum(lens))
    run(lens, 2, 2, d, causal, seed=sum(lens) + 1)


def test_every_length_up_to_two_blocks():
    for d in (64, 128):
        run(list(range(1, 258, 3)), 1, 1, d, True, seed=5)
        run(list(range(2, 258, 3)), 2, 1, d, False, seed=6)


@pytest.mark.parametrize("Hk", [8, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_far_rows(d, Hk):
    """Rows behind more than 2^31 values of q, o and the accumulators."""
    H = 32
    q, k, v, cu = draw_far(H, Hk, d, [300, 1, 77], seed=42)
    o, lse = fa.forward_packed(q, k, v, cu)
    do = torch.empty_like(o)
    a = cu[0].item()
    do[a:] = torch.randn(o[a:].shape, generator=torch.Generator().manual_seed(43)).to(BF16).to(DEV)
    got = fa.backward_packed(q, k, v, o, lse, do, cu)
    check(q, k, v, cu, o, lse, do, got, True)


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_per_sm(d):
    """Long and short sequences, several items per persistent CTA."""
    run([1500, 1, 257, 2049, 640, 5], 8, 2, d, True, seed=9)
    run([1000, 77, 900], 8, 8, d, False, seed=10)


@pytest.mark.parametrize("S", [255, 1100, 2048, 2049])
def test_many_sequences(S):
    """Sorted and unsorted block tables."""
    g = torch.Generator().manual_seed(S)
    run(torch.randint(0, 9, (S,), generator=g).tolist(), 2, 1, 64, True, seed=2)


def test_decreasing_offsets_stay_inside():
    """What is computed is not specified; rows outside the tensors are not
    touched, and the library goes on working."""
    q, k, v, cu = draw([40, 300, 24], 2, 1, 64, BF16, seed=5)
    o, lse = fa.forward_packed(q, k, v, cu)
    do = torch.randn_like(o)
    for bad in ([364, 0, 300, 10], [300, 100, 364, 50], [1 << 30, -5, 7, 0]):
        cu2 = torch.tensor(bad, device=DEV).int()
        fa.forward_packed(q, k, v, cu2)
        fa.backward_packed(q, k, v, o, lse, do, cu2)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
    check(q, k, v, cu, o, lse, do, fa.backward_packed(q, k, v, o, lse, do, cu), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk", [4, 2], ids=["own", "shared"])
def test_rows_of_no_sequence(d, Hk):
    """NaN rows before the first and behind the last sequence, in every input:
    not read into a gradient, and the gradients there not written."""
    lens = [100, 45]
    q, k, v, cu = draw(lens, 4, Hk, d, BF16, seed=3, before=37, behind=200)
    o, lse = fa.forward_packed(q, k, v, cu, out=torch.full(q.shape, float("nan"), dtype=BF16,
                                                           device=DEV),
                               lse=torch.full((4, q.shape[0]), float("nan"), device=DEV))
    do = torch.randn(q.shape, device=DEV).to(BF16)
    do[:37] = do[182:] = float("nan")
    T = q.shape[0]
    dq = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    dk, dv = (torch.full((T, Hk, d), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    nbytes = fa.fa_backward_packed_workspace_bytes(2, T, 4, Hk, d)
    ws = torch.full((nbytes // 4,), float("nan"), device=DEV)      # contents do not matter
    fa.fa_backward_packed(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), cu.data_ptr(), 2, T, 4, Hk, d, q.stride(0),
        k.stride(0), v.stride(0), d ** -0.5, True, ws.data_ptr(), nbytes,
        torch.cuda.current_stream().cuda_stream)
    check(q, k, v, cu, o, lse, do, (dq, dk, dv), True)
    for x in (dq, dk, dv):
        assert (x[:37] == 7).all() and (x[182:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_do_not_mix(d):
    """A sequence of NaN or Inf leaves its neighbours' gradients alone (to the
    order of the fp32 sums: dK and dV exactly, with a head of their own)."""
    for bad in (float("nan"), float("inf")):
        q, k, v, cu = draw([70, 33, 150], 2, 2, d, BF16, seed=4)
        do = torch.randn(q.shape, device=DEV).to(BF16)
        o, lse = fa.forward_packed(q, k, v, cu, causal=False)
        a = fa.backward_packed(q, k, v, o, lse, do, cu, causal=False)
        for x in (q, k, v, o, do):
            x[70:103] = bad
        lse[:, 70:103] = bad
        b = fa.backward_packed(q, k, v, o, lse, do, cu, causal=False)
        for rows in (slice(0, 70), slice(103, 253)):
            assert torch.equal(a[1][rows], b[1][rows]) and torch.equal(a[2][rows], b[2][rows])
            assert torch.allclose(a[0][rows].float(), b[0][rows].float(), rtol=2 ** -7, atol=1e-5)


def test_against_differences():
    """Along the returned gradients, central differences of the float64 forward
    (step 1e-4: error of the differences far below the bf16 gradients')."""
    lens, H, Hk, d = [9, 1, 40], 4, 2, 64
    q, k, v, cu = draw(lens, H, Hk, d, BF16, seed=21)
    o, lse = fa.forward_packed(q, k, v, cu)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    grads = fa.backward_packed(q, k, v, o, lse, do, cu)

    def loss(q, k, v):
        total = 0.0
        for a, b in zip(cu.tolist(), cu.tolist()[1:]):
            x, y, z = (t[a:b].transpose(0, 1) for t in (q, k, v))
            y, z = (t.repeat_interleave(H // Hk, 0) for t in (y, z))
            s = (x @ y.transpose(1, 2)) * d ** -0.5
            s = s.masked_fill(torch.ones_like(s).triu(1) > 0, -torch.inf)
            total += ((s.softmax(-1) @ z).transpose(0, 1) * do[a:b].double()).sum()
        return total
    x = [t.double() for t in (q, k, v)]
    for i, g in enumerate(grads):
        g = g.double()
        h = 1e-4
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * g, x[i] - h * g
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # three roundings to bf16 (P or dS, D's o, the result) of 2^-8 each
        # bound the gradient to 2^-6 of its size in the 2-norm
        assert abs(slope - g.square().sum()) <= 2.0 ** -6 * g.square().sum()


def test_repeats_captures_and_streams():
    """dK, dV of ungrouped heads repeat bit for bit; a graph on new inputs; two
    streams with a workspace each."""
    q, k, v, cu = draw([300, 41, 7], 4, 4, 128, BF16, seed=11)
    do = torch.randn(q.shape, device=DEV).to(BF16)
    o, lse = fa.forward_packed(q, k, v, cu)
    want = fa.backward_packed(q, k, v, o, lse, do, cu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(12):
        with torch.cuda.stream(streams[i & 1]):
            outs.append(fa.backward_packed(q, k, v, o, lse, do, cu))
    torch.cuda.synchronize()
    for x in outs:
        assert torch.equal(x[1], want[1]) and torch.equal(x[2], want[2])
        check(q, k, v, cu, o, lse, do, x, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        o, lse = fa.forward_packed(q, k, v, cu)
        got = fa.backward_packed(q, k, v, o, lse, do, cu)
    q.copy_(torch.randn(q.shape, device=DEV))
    cu.copy_(torch.tensor([0, 130, 200, 348]))
    graph.replay()
    check(q, k, v, cu, o, lse, do, got, True)


def test_a_training_step():
    """Norm, rotation, packed attention and all their gradients, end to end in
    one chain, against float64 autograd from the same bf16 inputs."""
    lens, H, Hk, d = [30, 75], 4, 2, 64
    q, k, v, cu = draw(lens, H, Hk, d, BF16, seed=31)
    g = torch.Generator().manual_seed(32)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF16).to(DEV) for _ in range(2))
    pos = torch.cat([torch.arange(n) for n in lens]).int().to(DEV)
    freq, _ = fa.rope_frequencies(d, device=DEV)
    do = torch.randn(q.shape, generator=g).to(BF16).to(DEV)
    qr, kr = fa.qk_norm_rope(q, k, pos, freq, qw, kw)
    o, lse = fa.forward_packed(qr, kr, v, cu)
    dqr, dkr, dv = fa.backward_packed(qr, kr, v, o, lse, do, cu)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(dqr, dkr, q, k, pos, freq, qw, kw)
    x = [t.double().detach().clone().requires_grad_() for t in (q, k, v, qw, kw)]
    ang = pos.double()[:, None] * freq
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def prep(y, w):
        y = y * (y.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    yq, yk = prep(x[0], x[3]), prep(x[1], x[4])
    total = 0.0
    for a, b in zip(cu.tolist(), cu.tolist()[1:]):
        sc = torch.einsum("nhd,mhd->hnm", yq[a:b], yk[a:b].repeat_interleave(H // Hk, 1)) * d ** -0.5
        sc = sc.masked_fill(torch.ones_like(sc).triu(1) > 0, -torch.inf)
        y = torch.einsum("hnm,mhd->nhd", sc.softmax(-1), x[2][a:b].repeat_interleave(H // Hk, 1))
        total = total + (y * do[a:b].double()).sum()
    total.backward()
    # Relative 2-norm: bf16 roundings of qr / kr, P, o, dS, dqr, the result (2^-8
    # at most each, 2^-8 / sqrt(3) rms) add up to less than six of them.
    for got, want in zip((dq, dk, dv, dqw, dkw), (t.grad for t in x)):
        rel = (got.double() - want).norm() / want.norm()
        assert rel <= 6 * H8, rel.item()


def test_helper_refuses():
    q, k, v, cu = draw([40], 4, 2, 64, BF16, seed=1)
    o, lse = fa.forward_packed(q, k, v, cu)
    do = torch.randn_like(o)
    bad = [
        lambda: fa.backward_packed(q, k, v, o[:20], lse, do, cu),
        lambda: fa.backward_packed(q, k, v, o, lse.t(), do, cu),
        lambda: fa.backward_packed(q, k, v, o, lse, do.transpose(0, 1), cu),
        lambda: fa.backward_packed(q, k, v, o, lse[:1], do, cu),
        lambda: fa.backward_packed(q.half(), k.half(), v.half(), o.half(), lse, do.half(), cu),
        lambda: fa.backward_packed(q, k, v, o, lse, do, cu.long()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fa.FattnError):
        fa.backward_packed(q, k, v, o, lse, do, cu,
                           workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
