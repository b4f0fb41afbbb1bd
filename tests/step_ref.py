"""The operators around the 8-bit cache in plain Python / numpy in 64 bits, as the
header states them (test oracle, CPU only): norm and rotation, attention under a
window or a tree, log probabilities."""
import numpy as np

from tests import serving_ref as R

TREE = 64


def window_sees(lens, cu, window, sinks):
    """sees(s, i, pos): which positions the i-th new token of sequence s sees."""
    def sees(s, i, pos):
        p = lens[s] - (cu[s + 1] - cu[s]) + i
        return (pos <= p) & ((pos > p - window) | (pos < sinks))
    return sees


def tree_sees(lens, cu, parent):
    def sees(s, i, pos):
        n = cu[s + 1] - cu[s]
        start, b = lens[s] - n, max(0, n - TREE)
        if i < b:
            return pos <= start + i
        line, at = {i}, i
        while b <= parent[cu[s] + at] < at:
            at = parent[cu[s] + at]
            line.add(at)
        return (pos < start + b) & (start + i >= pos) | np.isin(pos, [start + j for j in line])
    return sees


class Masked(R.Cache):
    """A cache whose attention takes its visible positions from `sees`."""

    @classmethod
    def of(cls, ref, sees):
        c = cls(ref.k, ref.v, ref.ks, ref.vs)
        c.sees = sees
        return c

    def attention(self, q, table, lens, cu, scale):
        T, Hq, D = q.shape
        G = Hq // self.H
        out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
        lse, smag = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
        for s in range(len(lens)):
            pages = [j for j in range(-(-lens[s] // self.B)) if 0 <= table[s][j] < self.P]
            if not pages:
                continue
            pos = np.concatenate([np.arange(j * self.B, (j + 1) * self.B) for j in pages])
            for h in range(self.H):
                kv = [self.values(table[s][j], h) for j in pages]
                k, v = np.concatenate([a for a, _ in kv]), np.concatenate([b for _, b in kv])
                for i in range(cu[s + 1] - cu[s]):
                    t = cu[s] + i
                    see = self.sees(s, i, pos) & (pos < lens[s])
                    if not see.any():
                        continue
                    for g in range(h * G, h * G + G):
                        x = scale * (k[see] @ q[t, g].astype(np.float64))
                        m = x.max()
                        p = np.exp(x - m)
                        lse[t, g] = m + np.log(p.sum())
                        out[t, g] = p @ v[see] / p.sum()
                        mag[t, g] = p @ np.abs(v[see]) / p.sum()
                        smag[t, g] = abs(scale) * (np.abs(k[see]) @ np.abs(q[t, g].astype(np.float64))).max()
        return out, lse, mag, smag


def rotate(x, pos, freq, weight=None, eps=0.0, interleaved=False):
    """(y, |a| + |b| of each element's pair after the norm); x [T, H, D] float64."""
    x = x.astype(np.float64)
    if weight is not None:
        with np.errstate(all="ignore"):
            x = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * weight.astype(np.float64)
    half = len(freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    t = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    # (the product of 31 and 24 bits is one of 55: its low part is put in at the end)
    hi = pos.astype(np.float64) // 4096 * 4096
    low = (hi[:, None] * freq.astype(np.float64)[None] - t) + (pos - hi)[:, None] * freq.astype(np.float64)[None]
    c, s = np.cos(t) - low * np.sin(t), np.sin(t) + low * np.cos(t)
    y, mag = x.copy(), np.abs(x)
    xa, xb = x[..., a], x[..., b]
    y[..., a], y[..., b] = xa * c[:, None] - xb * s[:, None], xb * c[:, None] + xa * s[:, None]
    mag[..., a] = mag[..., b] = np.abs(xa) + np.abs(xb)
    return y, mag


def logprobs(x, tokens, top):
    """(logprob, entropy, ids, top logprobs, sum of p |x - max|) of float64 rows."""
    M, V = x.shape
    lp, h, ids, tl, mag = np.zeros(M), np.zeros(M), np.zeros((M, top), int), np.zeros((M, top)), np.zeros(M)
    for r in range(M):
        if not (x[r] < np.inf).all():   # a NaN or +inf
            lp[r] = h[r] = np.nan
            ids[r], tl[r] = -1, np.nan
            continue
        order = np.argsort(-x[r], kind="stable")[:top]
        ids[r] = order
        m = x[r].max()
        if m == -np.inf:
            lp[r], tl[r] = -np.inf, -np.inf
            continue
        z = np.exp(x[r] - m)
        ls = np.log(z.sum())
        p = z / z.sum()
        d = np.where(p > 0, x[r] - m, 0.0)
        lp[r] = x[r, tokens[r]] - m - ls if 0 <= tokens[r] < V else -np.inf
        h[r] = ls - p @ d
        mag[r] = p @ -d
        tl[r] = x[r, order] - m - ls
    return lp, h, ids, tl, mag
