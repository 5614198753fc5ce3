"""Float64 definitions of the operators around the FFN block (numpy, CPU).

Written from the formulas alone and sharing no code with the CUDA path.  Each
function that has a rounded counterpart on the GPU also says how far a binary32
evaluation of it may be off (`*_bound`), from the number of roundings that the
formula's terms pass through; u is binary32's unit roundoff.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -150}   # half the smallest subnormal
BLOCK = 16
MIN_EXP = -64


# ---- E4M3 and the cache -----------------------------------------------------------

def e4m3_table() -> np.ndarray:
    """The value of each of the 256 bit patterns: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 0x7f == 0x7f else v
        if c & 0x80:
            out[c] = -out[c]
    return out


def e4m3_round(x) -> np.ndarray:
    """Nearest E4M3 value, ties to the even code; +-inf and beyond go to +-448, NaN stays."""
    t = e4m3_table()[:127]                                  # 0 .. 448, ascending
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(t, np.where(np.isnan(a), 0.0, a))  # t[hi-1] < a <= t[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = t[hi] - a, a - t[lo]
    pick = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.where(np.isnan(x), np.nan, np.copysign(t[pick], x))


def block_scale(x) -> float:
    """Smallest power of two s >= 2^MIN_EXP with every finite |x| <= 448 s."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    amax = x.max() if x.size else 0.0
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class CacheOracle:
    """A paged cache as values: codes' values [pages, heads, page, dim] and scales [pages, heads, page / BLOCK]."""

    def __init__(self, codes_k, scales_k, codes_v, scales_v):
        t = e4m3_table()
        self.value = [t[np.asarray(c)] for c in (codes_k, codes_v)]
        self.scale = [np.asarray(s, dtype=np.float64).copy() for s in (scales_k, scales_v)]
        self.page = self.value[0].shape[2]

    def write(self, k, v, table, cu, start):
        """k, v float64 [tokens, heads, dim]; tokens of one block at a time."""
        for which, x in enumerate((k, v)):
            value, scale = self.value[which], self.scale[which]
            for s in range(len(start)):
                pos, end = int(start[s]), int(start[s]) + int(cu[s + 1] - cu[s])
                while pos < end:
                    stop = min(end, (pos // BLOCK + 1) * BLOCK)
                    rows = x[cu[s] + pos - start[s]:cu[s] + stop - start[s]]
                    pg, off = table[s][pos // self.page], pos % self.page
                    b = off // BLOCK
                    for h in range(x.shape[1]):
                        new = block_scale(rows[:, h])
                        if off % BLOCK:
                            old = scale[pg, h, b]
                            new = max(new, old)
                            kept = value[pg, h, b * BLOCK:off]
                            value[pg, h, b * BLOCK:off] = e4m3_round(kept * (old / new))
                        value[pg, h, off:off + stop - pos] = e4m3_round(rows[:, h] / new)
                        scale[pg, h, b] = new
                    pos = stop

    def rows(self, which, table_row, first, last):
        """Values [last - first, heads, dim] of positions first .. last - 1 of one sequence."""
        out = []
        for pos in range(first, last):
            pg, off = table_row[pos // self.page], pos % self.page
            out.append(self.value[which][pg, :, off] * self.scale[which][pg, :, off // BLOCK, None])
        return np.array(out).reshape(last - first, *self.value[which].shape[1::2])


# ---- attention ----------------------------------------------------------------------

def attention(q, k, v, first, scale, causal=True):
    """One head's rows: q [n, dim] at positions first .. first + n - 1 over k, v
    [keys, dim].  Returns out, lse and a bound on each one's binary32 error with
    weights kept in fp16."""
    n, dim = q.shape
    out, lse = np.zeros((n, dim)), np.full(n, -np.inf)
    tol_o, tol_l = np.zeros((n, dim)), np.zeros(n)
    for i in range(n):
        m = min(len(k), first + i + 1) if causal else len(k)
        if m <= 0:
            continue
        s = scale * (k[:m] @ q[i])
        if np.isnan(s).any() or np.isposinf(s).any():
            out[i], lse[i] = np.nan, np.nan
            continue
        top = s.max()
        if np.isneginf(top):
            continue
        p = np.exp(s - top)
        total = p.sum()
        p /= total
        out[i] = p @ v[:m]
        lse[i] = top + np.log(total)
        mass = p @ np.abs(v[:m])
        # an exponent: the dot product's sum (tensor-core sums keep at least 2^-23 a term), its scaling, its
        # subtraction and 2^x (2^-22); a weight: that, twice (numerator and sum), and fp16's rounding
        size = abs(scale) * (np.abs(k[:m]) @ np.abs(q[i])).max()
        d = (dim + 8) * 2.0 ** -23 * size + 6 * U32 * (size + abs(top)) + 2.0 ** -22
        tol_o[i] = mass * (UNIT["float16"] * 1.01 + 2 * d + (m / 16 + 64) * 2 * U32)
        tol_l[i] = d + (m / 16 + 64) * U32 + 4 * U32 * abs(lse[i])
    return out, lse, tol_o, tol_l


# ---- layer norm -----------------------------------------------------------------------

def layer_norm(x, w, b, eps):
    """Rows x [n, d]: y, mean, rstd and the bounds of each in binary32 with sums of
    at most 16 terms in a row and a tree above them."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    h = c * rstd[:, None]
    y = h * w + b
    d_mean = 40 * U32 * np.abs(x).mean(1)
    # the mean's error shifts every c alike, which adds its square to the variance
    d_rstd = rstd * (40 * U32 + d_mean ** 2 * rstd ** 2)
    d_h = (d_mean * rstd)[:, None] + np.abs(h) * (d_rstd / rstd + 4 * U32)[:, None]
    return y, mean, rstd, np.abs(w) * d_h + 4 * U32 * (np.abs(h * w) + np.abs(b)), d_mean, d_rstd


def layer_norm_backward(dy, x, w, mean, rstd, d_sum=None, chain=None):
    """dx, dw, db from given mean and rstd, and their bounds; chain: terms that a
    column's sum adds one after another (default: all rows)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    h = (x - np.asarray(mean, np.float64)[:, None]) * r
    g = dy * w
    m1, m2 = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    dx = r * (g - m1 - h * m2)
    tol = 64 * U32 * r * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(h) * np.abs(g * h).mean(1, keepdims=True))
    if d_sum is not None:
        dx = dx + d_sum
        tol = tol + 2 * U32 * (np.abs(dx) + np.abs(d_sum))
    n = (dy.shape[0] if chain is None else chain) + 8
    return (dx, (dy * h).sum(0), dy.sum(0), tol, n * U32 * np.abs(dy * h).sum(0), n * U32 * np.abs(dy).sum(0))


# ---- log-probabilities ----------------------------------------------------------------

def token_logprobs(x, targets, top_k):
    """x [rows, vocab]: logprob, entropy, lse, top_index, top_logprob and a bound
    that holds for all of them in binary32."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    logp, ent, lse = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    idx, val, tol = np.zeros((rows, top_k), int), np.zeros((rows, top_k)), np.zeros(rows)
    for r in range(rows):
        m = x[r].max()                                       # NaN if any
        rank = np.where(np.isnan(x[r]), np.inf, x[r])
        nan_first = (~np.isnan(x[r])).astype(int)
        order = np.lexsort((np.arange(vocab), -rank, nan_first))
        idx[r] = order[:top_k]
        if not np.isfinite(m):
            lse[r] = -np.inf if np.isneginf(m) else np.nan
            ent[r], val[r] = np.nan, np.nan
            logp[r] = 0.0 if targets is not None and targets[r] < 0 else np.nan
            continue
        z = x[r] - m
        e = np.exp(z)
        p = e / e.sum()
        lse[r] = m + np.log(e.sum())
        live = e > 0
        spread = -(p[live] * z[live]).sum()
        ent[r] = np.log(e.sum()) + spread
        val[r] = x[r][idx[r]] - lse[r]
        if targets is not None:
            t = targets[r]
            logp[r] = 0.0 if t < 0 else np.nan if t >= vocab else x[r, t] - lse[r]
        # 2^x (2^-22), z's scaling, sums of up to vocab / 128 terms in a row, and the last difference
        step = 2.0 ** -21 + (vocab / 128 + 128) * U32
        far = max(abs(lse[r]), abs(logp[r]) if np.isfinite(logp[r]) else 0.0,
                  np.abs(val[r][np.isfinite(val[r])]).max(initial=0.0))
        tol[r] = (1 + 2 * spread) * step + 4 * U32 * (far + abs(m))
    return logp, ent, lse, idx, val, tol


def score_bounds(x, logp, ent, lse):
    """Bounds on binary32's entropy, lse and logprob, each with its own terms (one
    [rows] array each).  The entropy depends on differences of logits alone, so it
    has no term in their size; lse is one sum m + ln Z, logprob one difference
    more."""
    x = np.asarray(x, dtype=np.float64)
    step = 2.0 ** -21 + (x.shape[1] / 128 + 128) * U32
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):                      # rows without a distribution: NaN bounds, not used
        z = x - m
        p = np.exp(z)
        total = p.sum(1)
        spread = -np.where(p > 0, p * np.where(p > 0, z, 0.0), 0.0).sum(1) / total
        log_z = np.log(total)
        t_ent = (1 + 2 * spread) * step + 4 * U32 * (np.abs(log_z) + spread + np.abs(ent))
        t_lse = step + 4 * U32 * log_z + 2 * U32 * np.abs(lse)
        t_logp = t_lse + 2 * U32 * np.abs(logp)
    return t_ent, t_lse, t_logp
