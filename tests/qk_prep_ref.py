"""Norm and rotation of queries and keys in float64 (plain torch on the CPU),
with the bounds that the fp32 kernels' results are held to."""
import torch


def angles(positions, inv_freq):
    return positions.double()[:, None] * inv_freq.double()[None, :]


def rotate(y, ang, interleaved, mscale):
    """y [T,H,d] rotated by ang [T,rot/2]; and, per value, the size of the
    pair it comes from (|y1| + |y2|, or |y| where not rotated)."""
    n = ang.shape[1]
    out, size = y.clone(), y.abs()
    if n == 0:
        return out, size
    c, s = (mscale * f(ang)[:, None, :] for f in (torch.cos, torch.sin))
    i = torch.arange(n)
    p1, p2 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = y[..., p1], y[..., p2]
    out[..., p1], out[..., p2] = a * c - b * s, b * c + a * s
    both = (a.abs() + b.abs()) * abs(mscale)
    size[..., p1], size[..., p2] = both, both
    return out, size


def forward(x, w, positions, inv_freq, eps, interleaved, mscale):
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    return rotate(x, angles(positions, inv_freq), interleaved, mscale)


def backward(dy, x, w, positions, inv_freq, eps, interleaved, mscale):
    """dx, its size (the sum of its terms' sizes), dw, and the sum of the
    sizes of dw's terms."""
    g, size = rotate(dy.double(), -angles(positions, inv_freq), interleaved, mscale)
    if w is None:
        return g, size, None, None
    x, w = x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    wgx = (w * g * x).mean(-1, keepdim=True)
    dx = r * (w * g - x * r * r * wgx)
    dsize = r * (w.abs() * size + x.abs() * r * r * (w * size * x).abs().mean(-1, keepdim=True))
    return dx, dsize, (g * x * r).sum((0, 1)), (size * x * r).abs().sum((0, 1))


def bound(ref, size, dtype, far=0.0):
    """Largest allowed |result - ref|.

    One rounding to the output type: eps/2 of the value (fp16 below 2^-14:
    2^-25).  The fp32 arithmetic before it, u = 2^-24: the norm factor (a sum
    of up to 256 squares in at most 16 + 4 sequential roundings, halved by the
    root, a root of 2 ulp = 4 u, two products: < 20 u), the angle (rounded to
    2^-25 turns = 2 pi u / 2 < 4 u, sine and cosine to 2 ulp = 4 u, mscale u)
    and two products and a sum (3 u), < 32 u of the pair's size; a
    gradient's mean adds another such sum, its final difference 4 u: < 64 u
    of its terms' sizes.  ``far``: the largest angle in radians, whose
    frequency is known to 2^-53, multiplied once in 64 bits by each side:
    4 * 2^-53 * far."""
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = size * (64 * 2.0 ** -24 + 4 * far * 2.0 ** -53)
    return half * (ref.abs() + err) + err + tiny
