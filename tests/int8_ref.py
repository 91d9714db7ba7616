"""The 8-bit cache with an exponent for each (block, KV head), by its definition, in 64 bits on the CPU."""
import numpy as np

TOP = 127.0 * 2.0 ** 121


def least_exponent(amax):
    """The smallest e in [-126, 121] with amax <= 127 * 2^e, by trial."""
    e = -126
    while e < 121 and amax > np.ldexp(127.0, e):
        e += 1
    return e


class Cache:
    """codes [blocks, heads, 16, D], exps [blocks, heads] of K (or of V)."""

    def __init__(self, codes, exps):
        self.codes, self.exps = codes.astype(np.int64).copy(), exps.astype(np.int64).copy()

    def append(self, bt, cu, pos, held, x):
        """x [T, heads, D] float64.  Returns the slots whose contents are defined: those written or held."""
        x = np.where(np.isnan(x), 0.0, np.clip(x, -TOP, TOP))
        kept = np.zeros(self.codes.shape[:1] + (16,), bool)
        for r in range(len(cu) - 1):
            blocks = {}
            for t in range(cu[r], cu[r + 1]):
                blocks.setdefault(int(pos[t]) // 16, {})[int(pos[t]) % 16] = t
            for b, rows in blocks.items():
                pb = bt[r][b]
                holds = [s for s in range(16) if b * 16 + s < held[r]]
                for g in range(x.shape[1]):
                    e_old = int(self.exps[pb, g])
                    e = least_exponent(max(np.abs(x[t, g]).max() for t in rows.values()))
                    if holds:
                        e = max(e, e_old)
                        down = np.rint(np.ldexp(self.codes[pb, g, holds].astype(np.float64), e_old - e))
                        self.codes[pb, g, holds] = down.astype(np.int64)
                    for s, t in rows.items():
                        self.codes[pb, g, s] = np.rint(np.ldexp(x[t, g], -e)).astype(np.int64)
                    self.exps[pb, g] = e
                kept[pb, list(rows) + holds] = True
        return kept

    def values(self):
        return np.ldexp(self.codes.astype(np.float64), np.clip(self.exps, -126, 121)[:, :, None, None])
