"""The error bound of kvq_prefix_decode, weighted by the softmax.

One row (sequence, query head) over its n positions, in the cache's basis.  A
score z_t that moves by e_t gives p'_t = p_t e^(e_t) / sum_s p_s e^(e_s), so
with |e^(e_t) - 1| <= u_t
    |o' - o| = |sum_t p_t (e^(e_t) - 1) (v_t - o)| / |1 + sum_s p_s (e^(e_s) - 1)|
            <= sum_t p_t u_t |v_t - o| / (1 - sum_s p_s u_s):
a position counts by its own weight and its own reach r_t = sum_c |q_c k_tc| /
sqrt(d), not by the largest reach of the row.  The parts:
  e_t   2^-11 r_t for each rounding to f16 of what makes a score (per-channel K
        times its scale, a rotated query; per-token K codes and BF16 queries have
        none), 2 d 2^-24 r_t for the FP32 sum of d products, and 2^-12 for the
        row's reference (|m| up to 2^10 in log2 units: half a
        step is 2^-14, in the exponent and in the stored m)
  p, V' one rounding to f16 each: (1 + 2^-11)^2 - 1 of A = sum_t p_t |v_t|, and
        the f16 subnormals' 2^-28 max |v| per token
  sums  FP32, 16 positions at a time, and at most 64 partials: (n / 16 + 64) 2^-23 A
  out   one rounding to BF16: 2^-8 of what is left
"""
import numpy as np


def row_bound(q, k, v, roundings=1):
    """q [d], k and v [n, d] in float64: (o [d], error of o before the output's
    rounding [d])."""
    n, d = k.shape
    z = k @ q / np.sqrt(d)
    p = np.exp(z - z.max())
    p /= p.sum()
    o = p @ v
    reach = np.abs(k) @ np.abs(q) / np.sqrt(d)
    u = np.expm1((2.0 ** -11 * roundings + 2 * d * 2.0 ** -24) * reach + 2.0 ** -12)
    moved = float(p @ u)
    a = p @ np.abs(v)
    err = (p * u) @ np.abs(v - o) / (1 - moved) if moved < 0.5 else np.full(d, np.inf)
    err = err + a * ((1 + 2.0 ** -11) ** 2 - 1 + (n / 16 + 64) * 2.0 ** -23) + 2.0 ** -28 * n * np.abs(v).max()
    return o, err


def rounded(o, err):
    """The bound after the output's rounding to BF16."""
    return err + 2.0 ** -8 * (np.abs(o) + err)
