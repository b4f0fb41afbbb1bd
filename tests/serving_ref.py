"""The 8-bit serving operators in plain Python / numpy, sums in 64 bits, one
step after the other as the header states them (test oracle, CPU only).

Codes and scales are fp32 by definition (scale = fl32(amax / 127), code =
rint(fl32(v / scale))), so the quantizer here is numpy float32, whose division
is correctly rounded; everything that is summed is float64 or Python ints."""
import numpy as np

F = np.float32
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}    # half an ulp, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the spacing of subnormals


def scale_of(v):
    v = np.asarray(v, F)
    if not v.size:
        return F(0)
    if not np.all(np.isfinite(v)):
        return F(np.nan)
    return F(np.abs(v).max() / F(127))


def codes_of(v, s):
    v = np.asarray(v, F)
    if not s > 0:
        return np.zeros(v.shape, np.int8)
    return np.clip(np.rint(v / F(s)), -127, 127).astype(np.int8)


def i8_quantize(x):
    s = np.array([scale_of(r) for r in x], F)
    return np.stack([codes_of(r, t) for r, t in zip(x, s)]), s


def i8_t(xq, sx, wq, sw, bias=None):
    """(y, magnitude of the terms that fp32 rounds) in float64."""
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    y = sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None] * acc
    mag = np.abs(y)
    if bias is not None:
        y = y + bias[None]
        mag = mag + np.abs(bias)[None]
    return y, mag


class Cache:
    def __init__(self, k, v, ks, vs):   # k [P,H,B,D], v [P,H,D,B] int8
        self.k, self.v, self.ks, self.vs = k.copy(), v.copy(), ks.copy(), vs.copy()
        self.P, self.H, self.B, self.D = k.shape

    def append(self, kx, vx, table, lens, cu):
        """kx, vx [T, H, D] float32."""
        B = self.B
        for s in range(len(lens)):
            n = cu[s + 1] - cu[s]
            begin = lens[s] - n
            for j in range(begin // B, -(-lens[s] // B)):
                p = table[s][j]
                if n == 0 or not 0 <= p < self.P:
                    continue
                o0, o1 = max(begin - j * B, 0), min(lens[s] - j * B, B)
                rows = slice(cu[s] + j * B + o0 - begin, cu[s] + j * B + o1 - begin)
                for h in range(self.H):
                    for x, sc, page in ((kx, self.ks, self.k[p, h]), (vx, self.vs, self.v[p, h].T)):
                        new, old = scale_of(x[rows, h]), sc[p, h]
                        now = new
                        if o0 > 0:
                            now = F(np.nan) if np.isnan(old) or np.isnan(new) else max(old, new)
                        page[:o0] = codes_of(page[:o0].astype(F) * old, now)
                        page[o0:o1] = codes_of(x[rows, h], now)
                        page[o1:] = 0
                        sc[p, h] = now

    def values(self, p, h):
        """k, v [B, D] in float64."""
        return (self.k[p, h] * np.float64(self.ks[p, h]), self.v[p, h].T * np.float64(self.vs[p, h]))

    def attention(self, q, table, lens, cu, scale):
        """(out, lse, weighted magnitude of the values, magnitude of the scores'
        terms) in float64; q [T, Hq, D]."""
        T, Hq, D = q.shape
        G = Hq // self.H
        out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
        lse, smag = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
        for s in range(len(lens)):
            n = cu[s + 1] - cu[s]
            pages = [j for j in range(-(-lens[s] // self.B)) if 0 <= table[s][j] < self.P]
            if not pages:
                continue
            pos = np.concatenate([np.arange(j * self.B, (j + 1) * self.B) for j in pages])
            for h in range(self.H):
                kv = [self.values(table[s][j], h) for j in pages]
                k, v = np.concatenate([a for a, _ in kv]), np.concatenate([b for _, b in kv])
                for i in range(n):
                    t, see = cu[s] + i, pos <= lens[s] - n + i
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


def update(ref, table, lens, parent, new_lens, B):
    """Page bookkeeping with Python lists; returns (ref, table, shortage,
    [(from, to)])."""
    P, S, W = len(ref), len(lens), len(table[0])
    ok = lambda p: 0 <= p < P  # noqa: E731
    clip = lambda n: min(max(n, 0), W * B)  # noqa: E731
    free = iter([p for p in range(P) if ref[p] == 0])
    out, new = list(ref), [[-1] * W for _ in range(S)]
    keep = [min(clip(lens[p]), clip(n)) if 0 <= p < S else 0 for p, n in zip(parent, new_lens)]
    shares = [set() for _ in range(P)]
    for s in range(S):
        for j in range(-(-clip(lens[s]) // B)):
            if ok(table[s][j]):
                out[table[s][j]] -= 1
    for s in range(S):
        for j in range(keep[s] // B):
            p = table[parent[s]][j]
            if ok(p):
                new[s][j] = p
                out[p] += 1
                shares[p].add(s)
    short, copies = 0, []
    for s in range(S):
        j = keep[s] // B
        last = table[parent[s]][j] if keep[s] % B else -1
        want = -(-clip(new_lens[s]) // B)
        if keep[s] % B:
            if ok(last) and parent[s] == s and ref[last] == 1 and not shares[last] - {s}:
                new[s][j] = last
                out[last] += 1
            elif ok(last):
                p = next(free, -1)
                new[s][j] = p
                short += p < 0
                if p >= 0:
                    out[p] = 1
                    copies.append((last, p))
            j += 1
        for j in range(j, want):
            p = next(free, -1)
            new[s][j] = p
            short += p < 0
            if p >= 0:
                out[p] = 1
    return out, new, short, copies


def compact(ref, table):
    P = len(ref)
    used = [p for p in range(P) if ref[p] > 0]
    n = len(used)
    movers, holes = [p for p in used if p >= n], [p for p in range(n) if ref[p] <= 0]
    assert len(movers) == len(holes)
    remap = [p if ref[p] > 0 else -1 for p in range(P)]
    for a, b in zip(movers, holes):
        remap[a] = b
    out = [0] * P
    for p in used:
        out[remap[p]] = ref[p]
    return out, [[remap[p] if 0 <= p < P else -1 for p in row] for row in table], remap, n, list(zip(movers, holes))
