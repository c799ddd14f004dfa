"""Plain references of the paged 8-bit K/V cache and of attention over it, for the tests.

The cache's decisions are single IEEE fp32 operations, so ``append`` repeats them in numpy float32
and is compared bit for bit; ``attention`` is in 64 bits.
"""
import numpy as np

F = np.float32


class Cache:
    """Codes [pages, heads, page, dim], steps [pages, heads, page / block], K first, then V."""

    def __init__(self, pages, heads, dim, page, block, rng):
        self.page, self.block = page, block
        # what earlier owners left in the pages: codes of any value and large steps
        self.codes = [rng.integers(-128, 128, (pages, heads, page, dim)).astype(np.int8)
                      for _ in range(2)]
        self.steps = [rng.uniform(5, 9, (pages, heads, page // block)).astype(F)
                      for _ in range(2)]

    def copy(self):
        other = object.__new__(Cache)
        other.page, other.block = self.page, self.block
        other.codes = [c.copy() for c in self.codes]
        other.steps = [s.copy() for s in self.steps]
        return other

    def append(self, states, q_start, kv_len, table):
        """states: (K, V) as float32 [tokens, heads, dim]."""
        for codes, steps, x in zip(self.codes, self.steps, states):
            for s, length in enumerate(kv_len):
                rows = x[q_start[s]:q_start[s + 1]].astype(F)
                first = length - len(rows)
                for lo in range(first // self.block * self.block, length, self.block):
                    new = rows[max(lo - first, 0):lo + self.block - first]
                    if not len(new):
                        continue
                    page, at = table[s][lo // self.page], lo % self.page
                    had = max(first - lo, 0)
                    mx = np.maximum(np.abs(new).max((0, 2)), F(1e-5))
                    old = steps[page, :, at // self.block]
                    g_old = F(127) * old if had else np.zeros_like(old)
                    grown = mx > g_old
                    g = np.where(grown, mx, g_old).astype(F)
                    inv = F(127) / g
                    factor = old * inv
                    for h in np.flatnonzero(grown):
                        c = codes[page, h, at:at + had]
                        codes[page, h, at:at + had] = np.clip(
                            np.rint(c.astype(F) * factor[h]), -127, 127)
                    steps[page, :, at // self.block] = np.where(grown, g / F(127), old)
                    c = np.clip(np.rint(new * inv[None, :, None]), -127, 127)
                    codes[page, :, at + had:at + had + len(new)] = c.transpose(1, 0, 2)

    def states(self, which, s, length, table):
        """(codes [heads, length, dim], steps [heads, length]) of one sequence, in 64 bits."""
        pages = np.asarray(table[s][:-(-length // self.page)], int)
        heads, dim = self.codes[0].shape[1], self.codes[0].shape[3]
        c = self.codes[which][pages].transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :length]
        d = self.steps[which][pages].transpose(1, 0, 2).reshape(heads, -1)
        return c.astype(np.float64), np.repeat(d.astype(np.float64), self.block, 1)[:, :length]


def attention(cache, q, q_start, kv_len, table, scale, causal):
    """q float64 [tokens, q_heads, dim].  Returns y, lse and, for each output, how far a kernel may
    be from it (before the output's own rounding):

    * a score is a sum of dim exact products in fp32, taken in any order and possibly truncated at
      each step: off by dim * 2^-22 * sum |q c| d scale at most; with exp2's argument and result in
      fp32, another 2^-21 * (1 + |s|);
    * a weight is rounded to 11 bits (2^-11 of it), or to a fixed point 2^-25 below the row's
      largest weight * step (doubled here: the maximum may be up to a power of two older);
    * numerator and denominator carry these errors: twice the relative one;
    * sums of n terms in fp32 add n * 2^-24.
    """
    tokens, q_heads, dim = q.shape
    y = np.zeros((tokens, q_heads, dim))
    lse = np.full((tokens, q_heads), -np.inf)
    tol_y, tol_lse = np.zeros_like(y), np.zeros_like(lse)
    heads = cache.codes[0].shape[1]
    group = q_heads // heads
    for s, length in enumerate(kv_len):
        if length == 0:
            continue
        (ck, dk), (cv, dv) = (cache.states(w, s, length, table) for w in (0, 1))
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            seen = min(length, length - n + i + 1) if causal else length
            if seen <= 0:
                continue
            for h in range(q_heads):
                kh, row = h // group, q[q_start[s] + i, h]
                k, v = ck[kh, :seen], cv[kh, :seen]
                score = (k @ row) * dk[kh, :seen] * scale
                size = (np.abs(k) @ np.abs(row)) * dk[kh, :seen] * scale
                m = score.max()
                p = np.exp(score - m)
                total = p.sum()
                w = p * dv[kh, :seen] / total
                y[q_start[s] + i, h] = w @ v
                lse[q_start[s] + i, h] = m + np.log(total)
                e = (dim * 2.0**-22 * size.max() + 2.0**-21 * (1 + np.abs(score).max())
                     + seen * 2.0**-24)
                tol_y[q_start[s] + i, h] = ((2 * e + 2.0**-11) * (w @ np.abs(v))
                                            + 2.0**-24 * w.max() * np.abs(v).sum(0))
                tol_lse[q_start[s] + i, h] = e + 2.0**-23 * (1 + abs(lse[q_start[s] + i, h]))
    return y, lse, tol_y, tol_lse
