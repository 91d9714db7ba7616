"""A plain attention in 64 bits for the tests of the tree and the block-selected attention, with bounds on how far a
kernel may be off.

The bounds count roundings.  u = half a step: 2^-8 for bf16, 2^-11 for f16, 2^-24 for fp32.
  scores   products of 8-bit significands are exact in fp32; a sum of D of them in any order is off by at most
           D 2^-24 B, B = scale * sum_d |q_d k_d|; scaling, maximum and exp2 add a few steps of 2^-22 of an exponent
           below 2^7: ds = (D + 8) 2^-24 B + 2^-15.
  O        P is rounded once (u_p: bf16 for bf16 pools, f16 for FP8 pools), so every term p_j v_j is off by at most
           (u_p + 2 ds) |p_j v_j|, and O, rounded to bf16, by (u_p + 2 ds) A + 2^-8 |O| with A = sum_j p_j |v_j|.  f16
           has no steps below 2^-24: n keys add n 2^-25 max|v| at most.  The sums of up to n terms in fp32 add
           n 2^-24 A at most.
  LSE      off by ds plus one rounding of the result.
"""
import numpy as np
import torch


def softmax_rows(q, k, v, seen, scale, f16_p, n_for_sum=None):
    """q [rows, D], k, v [keys, D] (float64), seen [rows, keys] bool.
    Returns o, lse, tol_o, tol_lse; rows without a key: 0 and -inf."""
    D = q.shape[1]
    s = (q @ k.T) * scale
    B = (np.abs(q) @ np.abs(np.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)).T) * scale
    s = np.where(seen, s, -np.inf)
    B = np.where(seen, B, 0.0)
    n = s.shape[1]
    if n == 0:
        z = np.zeros((q.shape[0], v.shape[1]))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    m = s.max(1)
    some = m != -np.inf
    e = np.exp(s - np.where(some, m, 0.0)[:, None])
    l = e.sum(1)
    p = e / np.where(some, l, 1.0)[:, None]
    vz = np.where(seen.any(0)[:, None], v, 0.0)
    o = np.zeros((q.shape[0], v.shape[1]))
    for i in range(q.shape[0]):                 # a key that the row does not see takes no part, whatever it holds
        j = seen[i]
        o[i] = p[i, j] @ vz[j]
    va = np.abs(np.nan_to_num(vz, nan=0.0, posinf=0.0, neginf=0.0))
    A = p @ va
    lse = np.where(some, m + np.log(np.where(some, l, 1.0)), -np.inf)
    ds = (D + 8) * 2.0 ** -24 * B.max(1) + 2.0 ** -15
    up = 2.0 ** -11 if f16_p else 2.0 ** -8
    ds = np.nan_to_num(ds)
    tol_o = (up + 2 * ds[:, None] + n * 2.0 ** -24) * A + 2.0 ** -8 * np.abs(o)
    if f16_p:
        tol_o = tol_o + n * 2.0 ** -25 * (va.max() if va.size else 0.0)
    tol_lse = ds + 2.0 ** -24 * np.abs(np.where(some, lse, 0.0))
    return o, lse, tol_o, tol_lse


def pool_values(pool, which):
    """The pool's K or V as float64 [blocks, heads, 16, D] (FP8 codes times their scale)."""
    x = getattr(pool, which).cpu()
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).float().double().numpy() * getattr(pool, which + "_scale")
    return x.float().double().numpy()


def gather(vals, row, ctx, g):
    """Keys [0, ctx) of KV head g through a block-table row; a bad id's keys come back as None in the second value."""
    nb = (ctx + 15) // 16
    ids = row[:nb]
    good = (ids >= 0) & (ids < vals.shape[0])
    x = vals[np.where(good, ids, 0), g].reshape(nb * 16, vals.shape[-1])[:ctx]
    return x, np.repeat(good, 16)[:ctx]


def assert_close(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - want)[bad]):.3e} against {tol[bad].max():.3e}")


def random_pool(pool, seed):
    """Fills the pool with N(0, 1) values (FP8: codes of such values) and returns it."""
    gen = torch.Generator(device=pool.k.device).manual_seed(seed)
    for which in ("k", "v"):
        x = getattr(pool, which)
        v = torch.randn(x.shape, generator=gen, device=x.device)
        if x.dtype == torch.uint8:
            x.copy_((v / getattr(pool, which + "_scale")).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            x.copy_(v.to(torch.bfloat16))
    return pool


def tables(rng, ctxs, num_blocks, width=None, spare=0):
    """Scattered, disjoint block-table rows (numpy int32, -1 beyond a request's blocks)."""
    need = [(c + 15) // 16 + spare for c in ctxs]
    width = max(max(need), 1) if width is None else width
    perm = rng.permutation(num_blocks)
    bt = np.full((len(ctxs), width), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()
