"""What a prompt goes through, written out plainly in 64 bits: attention, rotation, append."""

import math

import numpy as np
import torch


def attention(q, k, v, cu, scale, window=0, sinks=0):
    """(out, spread) [rows, Hq, D]; NaN in rows of no prompt.  spread = sum_j p_j |v_j - out|: the factor by which a relative error of the
    weights reaches the output."""
    rows, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.full((rows, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    spread = out.clone()
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        i = torch.arange(hi - lo, device=q.device)
        sees = i[None, :] <= i[:, None]
        if window:
            sees &= (i[None, :] > i[:, None] - window) | (i[None, :] < sinks)
        for h in range(Hq):
            kk, vv = k[lo:hi, h // G].double(), v[lo:hi, h // G].double()
            s = (q[lo:hi, h].double() @ kk.T * scale).masked_fill(~sees, -math.inf)
            p = torch.softmax(s, dim=1)
            o = p @ vv
            out[lo:hi, h] = o
            for r0 in range(0, hi - lo, 256):   # rows x keys x columns at a time
                r = slice(r0, r0 + 256)
                spread[lo:hi, h][r] = torch.einsum("ij,ijd->id", p[r], (vv[None] - o[r, None]).abs())
    return out, spread


def attention_tolerance(q, k, scale, longest, out, spread):
    """With u = 2^-24 and r = 2^-8 (bf16's rounding to nearest moves a value by at most that): a score to base 2 is a float32 dot product
    of D terms and a multiplication, off by at most e = (D + 4) u log2(e) scale |q| |k|; a weight by ln 2 e + 4 u (exp2, rescalings), and r where it is
    rounded to bf16; a relative error d of the weights moves the output by at most 2 d spread; the values' sums add (keys + 8) u, the
    output's rounding r of it in bf16."""
    u, r = 2.0 ** -24, 2.0 ** -8
    bf16 = q.dtype == torch.bfloat16
    e = (q.shape[2] + 4) * u * 1.4427 * abs(scale) * q.double().norm(dim=2).max().item() * k.double().norm(dim=2).max().item()
    d = 0.6932 * e + 4 * u * (1 + longest / 64) + (r if bf16 else 0.0)
    return 2 * d * spread + (longest + 8) * u * (spread + out.abs()) + (r if bf16 else u) * out.abs() + 1e-30


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=4096, slow=1.0, fast=32.0):
    j = np.arange(dim // 2, dtype=np.float64)
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = base ** (-2 * j / dim)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        g = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        return f * g + f / factor * (1 - g)
    return f


def rotate(x, positions, f, magnitude=1.0, interleaved=False):
    """(turned, tolerance) of float32/bf16 rows [rows, heads, D] at positions [rows].

    Tolerance: sine and cosine come from an angle known to p f 2^-51 (a frequency's power and its division by 2 pi are off by 2^-52 each) and
    rounded to 2^-25 of an eighth of a turn, through a function good to 2 units in the last place (4 u); the magnitude, the two products and their
    sum round once each: (|a| + |b|) m (8 u + p f 2^-50), and the output's own rounding."""
    n = len(f)
    f = torch.as_tensor(np.asarray(f), device=x.device)
    angle = positions.double()[:, None] * f
    c, s = torch.cos(angle)[:, None] * magnitude, torch.sin(angle)[:, None] * magnitude
    y = x.double().clone()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    tol = torch.zeros_like(y)
    tol[..., a] = tol[..., b] = (xa.abs() + xb.abs()) * abs(magnitude) * (8 * 2.0 ** -24 + angle.abs()[:, None] * 2.0 ** -50)
    turned = torch.zeros(x.shape[-1], dtype=torch.bool, device=x.device)
    turned[:2 * n] = True
    return y, tol + torch.where(turned, y.abs() * (2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24), 0.0)


def positions_of(cu, length):
    """Position of every row; -1 behind the last stream's."""
    return [int(length[b]) + i for b in range(len(cu) - 1) for i in range(cu[b + 1] - cu[b])]
