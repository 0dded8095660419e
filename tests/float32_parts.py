"""Inputs, bounds and a model of float32 attention by three bf16 parts a number, for tests that have to notice a part, a
product of parts or a rounded sum that is missing.

u = 2^-24.  x = x0 + x1 + x2, each the rounding of what the ones before leave, so |x1| <= 2^-8 |x|, |x2| <= 2^-16 |x| and the
rest is at most u |x|.  A product takes six terms (x0 y0, x0 y1, x1 y0, x1 y1, x0 y2, x2 y0); those left out, x1 y2, x2 y1 and x2 y2, are
below 3 u |x y| together, and six sums that may be cut off instead of rounded add 2 u |x y| each:
  a score is within 15 u |s|,
  a weight within its scores' error, 4 u of the exponential and u of its own parts,
  two weighted values' sum within 12 u of six cut sums, 4 u of roundings, and the weight's.
So with two visible keys, values 0 and v, and p the second one's share, the output p v is within
  v (p (1 - p) (30 |s| + 8) u + 21 u p).
A lost term is worth up to 2^-16 = 256 u of its product."""

import numpy as np

U = 2.0 ** -24
TERMS = ((2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0))   # (part of x, part of y), the smallest first


def two_key_inputs(kind, n, seed):
    """(q0, k0, q1, k1, v) [n] float32: the query's and the first key's number in one column, the query's and the second key's
    in another, and the second key's value (the first one's is 0)."""
    rng = np.random.default_rng(seed)
    f = np.float32
    if kind == "scores":    # large and close together: the scores' last bits are what counts
        q0, q1 = rng.uniform(8, 16, n).astype(f), rng.uniform(8, 16, n).astype(f)
        k0 = (rng.uniform(8, 16, n) * rng.choice([-1, 1], n)).astype(f)
        k1 = (q0 * k0 * (1 + rng.uniform(-0.01, 0.01, n)) / q1).astype(f)
        v = np.ones(n, f)
    else:                    # small: the weights' and the values' last bits are
        q0, q1, k0, k1 = rng.uniform(1, 2, n).astype(f), rng.uniform(1, 2, n).astype(f), np.zeros(n, f), rng.uniform(-1, 1, n).astype(f)
        v = rng.uniform(1, 2, n).astype(f)
    return q0, k0, q1, k1, v


def two_key_output(q0, k0, q1, k1, v):
    """(output, bound) in float64."""
    q0, k0, q1, k1, v = (x.astype(np.float64) for x in (q0, k0, q1, k1, v))
    p = 1 / (1 + np.exp(q0 * k0 - q1 * k1))
    top = np.maximum(np.abs(q0 * k0), np.abs(q1 * k1))
    return p * v, v * (p * (1 - p) * (30 * top + 8) * U + 21 * U * p)


def bf16(x):
    """float32 rounded to the nearest bf16, ties to even."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)


def parts(x):
    x0 = bf16(x)
    x1 = bf16(x - x0)
    return x0, x1, bf16(x - x0 - x1)


def cut(x):
    """float64 cut off to float32."""
    f = x.astype(np.float32)
    return np.where(np.abs(f) > np.abs(x), np.nextafter(f, np.float32(0)), f).astype(np.float32)


def product(x, y, without=None, n_parts=3):
    """x y by its terms, sums cut off; ``without`` is left out, and parts from n_parts on are lost."""
    px, py = parts(x), parts(y)
    s = np.zeros_like(px[0])
    for i, j in TERMS:
        if (i, j) != without and i < n_parts and j < n_parts:
            s = cut(s.astype(np.float64) + px[i].astype(np.float64) * py[j])
    return s


def two_key_model(q0, k0, q1, k1, v, without_scores=None, without_values=None, n_parts=3):
    s0, s1 = product(q0, k0, without_scores, n_parts), product(q1, k1, without_scores, n_parts)
    m = np.maximum(s0, s1)
    e0, e1 = np.exp((s0 - m).astype(np.float32)), np.exp((s1 - m).astype(np.float32))
    return product(e1, v, without_values, n_parts) / (e0 + e1)


def mean_shift(tiles_per_sum, rows, positions, seed):
    """Mean relative shift of sums of positive weighted values over `positions`, cut off after each of six terms of 16 positions
    at a time; a sum runs over `tiles_per_sum` tiles of 64 before it is added to the total (rounded)."""
    rng = np.random.default_rng(seed)
    e = rng.uniform(0, 1, (positions, rows)).astype(np.float32)
    v = rng.uniform(1, 2, (positions, rows)).astype(np.float32)
    pe, pv = parts(e), parts(v)
    total = np.zeros(rows, np.float32)
    for t in range(0, positions, 64 * tiles_per_sum):
        s = np.zeros(rows, np.float32)
        for u in range(t, min(t + 64 * tiles_per_sum, positions), 64):
            for i, j in TERMS:
                for c in range(u, min(u + 64, positions), 16):
                    s = cut(s.astype(np.float64) + (pe[i][c:c + 16].astype(np.float64) * pv[j][c:c + 16]).sum(axis=0))
        total = (total + s).astype(np.float32)
    exact = (e.astype(np.float64) * v).sum(axis=0)
    return float(((total - exact) / exact).mean())


# 24 cuts of a tile's sum, each below 2 u and all of them downwards, and the roundings of 79 tiles' sums of weights and of
# values, which go either way: three standard deviations of 79 roundings of u / sqrt(3)
SHIFT = 24 * 2 * U + 3 * (79 ** 0.5) * U / 3 ** 0.5
