"""Attention of one sequence under any mask in float64 (plain torch on the tensors'
device), in the form that packed_ref.check_forward holds results to."""
import math

import torch


def near(pos, n_keys, window, sinks):
    """[n, m]: whether the query at position pos[i] sees key j."""
    j = torch.arange(n_keys, device=pos.device)
    p = pos[:, None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def sequence(q, k, v, scale, see):
    """q [n,H,d], k, v [m,Hk,d], see [n,m].  As packed_ref.sequence: O [n,H,d], LSE
    [H,n], sum_j p_j |v_j|, sum_j |v_j| over visible keys, and sum_c |q_c k_c|
    maximised over visible keys."""
    n, H, d = q.shape
    g = H // k.shape[1]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    # (keys and values that nothing sees may be anything)
    used = see.any(0)[None, :, None]
    k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    s = torch.where(see, (q @ k.transpose(1, 2)) * scale, -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[1] else torch.full((H, n), -math.inf, device=q.device)
    p = torch.where(see, torch.exp(s - lse[..., None].nan_to_num(neginf=0.0)), 0.0)
    mag = torch.where(see, q.abs() @ k.abs().transpose(1, 2), 0.0)
    mag = mag.amax(-1) if k.shape[1] else torch.zeros_like(lse)
    return ((p @ v).transpose(0, 1), lse, (p @ v.abs()).transpose(0, 1),
            (see.double() @ v.abs()).transpose(0, 1), mag)
