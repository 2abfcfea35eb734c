"""Attention of one sequence with grouped heads in float64 (plain torch on the
tensors' device), and the bounds its results are held to."""
import math

import torch


def sequence(q, k, v, scale, last):
    """q [n,H,d], k, v [m,Hk,d]; query i sees keys 0 .. last[i].  Returns O
    [n,H,d], LSE [H,n], sum_j p_j |v_j| and sum_j |v_j| over visible keys
    ([n,H,d]), and sum_c |q_c k_c| maximised over visible keys ([H,n])."""
    n, H, d = q.shape
    g = H // k.shape[1]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    see = torch.arange(k.shape[1], device=q.device)[None, :] <= last[:, None]
    s = (q @ k.transpose(1, 2)) * scale
    s = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[1] else torch.full((H, n), -math.inf, device=q.device)
    p = torch.where(see, torch.exp(s - lse[..., None].nan_to_num(neginf=0.0)), 0.0)
    mag = torch.where(see, q.abs() @ k.abs().transpose(1, 2), 0.0)
    mag = mag.amax(-1) if k.shape[1] else torch.zeros_like(lse)
    # (v of keys that nothing sees may be anything: weights are zero there)
    v = torch.where(see.any(0)[None, :, None], v, 0.0)
    return ((p @ v).transpose(0, 1), lse, (p @ v.abs()).transpose(0, 1),
            (see.double() @ v.abs()).transpose(0, 1), mag)


def check_forward(o, lse, ref, scale, dtype):
    """Holds O (and LSE, unless None) to the reference.

    A score is an fp32 sum of d exact products: off by at most d 2^-24 of
    sum |q_c k_c|, times scale; the running sum and the exponential (2 ulp)
    and the exponent's argument (two roundings of up to |s| log2 e) add
    2^-20 + 2^-22 |s|.  A relative change e of every weight moves O by at
    most 2 e sum p |v|.  P and O are each rounded once to the type (eps / 2);
    fp16 weights below 2^-14 are off by 2^-25 at most, against a row sum of
    at least 1."""
    ro, rl, pv, sv, mag = ref
    d = o.shape[-1]
    half = torch.finfo(dtype).eps / 2
    size = torch.where(torch.isfinite(rl), rl.abs(), 0.0)
    e = scale * mag * d * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * (size + scale * mag)
    tiny = 2.0 ** -25 * sv if dtype == torch.float16 else 0.0
    err = (half * 1.01 + 2 * e.transpose(0, 1)[..., None]) * pv + tiny
    diff = (o.double() - ro).abs()
    assert (diff <= half * (ro.abs() + err) + err).all(), \
        f"O: {(diff - err - half * ro.abs()).max().item():.3g} over its bound"
    if lse is None:
        return
    none = ~torch.isfinite(rl)
    assert (lse[none] == -math.inf).all()
    diff = (lse.double() - rl).abs()[~none]
    assert (diff <= (e + 2.0 ** -22 * size)[~none]).all(), f"LSE: {diff.max().item():.3g}"
