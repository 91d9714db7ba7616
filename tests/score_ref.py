"""Attention with modified scores in 64 bits for one (token, KV head) at a time, with bounds on how far a kernel may be off.

Beside the roundings that attn_ref counts (products, sums, exp2, P, O, LSE):
  cap      tanh has slope 1 at most, so an error of its argument does not grow; the argument's own rounding is one more
           step of the score; tanh itself is off by 2^-22 of 1 at most, times cap.
  slopes   the distance, its product and the sum are rounded once each: 3 2^-24 slope dist, and 2^-23 |x| for the sums.
  int8     the power of two is exact on scores and P; K and V are bf16 values, P is rounded to bf16.
  range    p_j relative to the row's maximum is an fp32 number: a weight below 2^-126 (an exponent below -126) is taken as
           zero, so n keys may lack n 2^-126 max|v|.  (Values of dims whose heavy keys hold zeros are that small: with a
           weight of 2^-190 the formula gives 6e-59 there, and fp32, whose least number is 1.4e-45, gives 0.)
"""
import numpy as np


def rows(q, k, v, pos, seen, scale, softcap, slopes, f16_p):
    """q [G, D], k, v [n, D], seen [n], slopes [G] or None -> o [G, D], lse [G], tol_o, tol_lse."""
    g, d = q.shape
    j = np.nonzero(seen)[0]
    if len(j) == 0:
        z = np.zeros((g, v.shape[1]))
        return z, np.full(g, -np.inf), z, np.zeros(g)
    k, v = k[j], v[j]
    with np.errstate(invalid="ignore", over="ignore"):
        x = (q @ k.T) * scale
        B = (np.abs(q) @ np.abs(np.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)).T).max(1) * scale
        more = np.zeros(g)
        if softcap:
            x = softcap * np.tanh(x / softcap)
            more += softcap * 2.0 ** -21
        if slopes is not None:
            dist = np.abs(pos - j)
            near = x - slopes[:, None] * dist
            # Only keys whose weight is not below 2^-60 of the largest one's count.
            heavy = near > near.max(1, keepdims=True) - 42
            more += (heavy * (np.abs(slopes)[:, None] * dist * 3 * 2.0 ** -24 + 2.0 ** -22 * np.abs(near))).max(1)
            x = near
        m = x.max(1)
        e = np.exp(x - m[:, None])
        l = e.sum(1)
        p = e / l[:, None]
        o = p @ v
    A = p @ np.abs(np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0))
    lse = m + np.log(l)
    ds = np.nan_to_num((d + 8) * 2.0 ** -24 * B + 2.0 ** -15 + more)
    up = 2.0 ** -11 if f16_p else 2.0 ** -8
    tol_o = (up + 2 * ds[:, None] + len(j) * 2.0 ** -24) * A + 2.0 ** -8 * np.abs(o)
    tol_o = tol_o + len(j) * 2.0 ** -126 * np.abs(np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)).max()
    if f16_p:
        tol_o = tol_o + len(j) * 2.0 ** -25 * np.abs(np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)).max()
    return o, lse, tol_o, ds + 2.0 ** -23 * np.abs(lse)


def sees(pos, ctx, prefix, first, window):
    j = np.arange(ctx)
    ok = (j >= first) & (j <= pos)
    if window:
        ok &= j > pos - window
    return ok | (j < prefix)
