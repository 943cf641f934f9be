"""Plain fp64 forms of the training-step operators, in numpy, on the CPU.

Rounding errors of an fp32 evaluation are bounded from the magnitudes that
these forms return beside the values: with u = 2^-24, an fp32 result off by
less than C u times its magnitude is within what C roundings can make.
"""
import numpy as np

from oracle import pyoracle as po

U = 2.0 ** -24


def dithers(n, seed, rnd, worker, site, first=0):
    """The 16-bit dithers of elements first .. first + n - 1 (first a multiple
    of 8)."""
    u = np.uint64
    b = np.arange(first // 8, (first + n + 7) // 8, dtype=u)
    x = [b & u(0xFFFFFFFF), (b >> u(32)) | u(worker << 16), np.full_like(b, rnd), np.full_like(b, (1 << 31) | site)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(q >> u(32)) ^ x[1] ^ u(k[0]), q & u(0xFFFFFFFF), (p >> u(32)) ^ x[3] ^ u(k[1]), p & u(0xFFFFFFFF)]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    w = np.stack(x, 1).astype(np.uint32)
    return np.stack((w & 0xFFFF, w >> 16), 2).reshape(-1)[:n].astype(np.int64)


def dithers_by_oracle(block, seed, rnd, worker, site):
    """The eight dithers of one block from the C oracle's Philox."""
    w = po.philox4x32([block & 0xFFFFFFFF, (block >> 32) | (worker << 16), rnd, (1 << 31) | site],
                      [seed & 0xFFFFFFFF, seed >> 32])
    return [int(h) for x in w for h in (int(x) & 0xFFFF, int(x) >> 16)]


def threshold(p):
    return int(np.floor(65536.0 * p + 0.5))


def choose(l, k):
    """Order of choice of one row: falling, equal logits (-0 = +0) by index, NaN
    first, -inf never; -1 fills up."""
    order = sorted((j for j in range(len(l)) if not l[j] == -np.inf),
                   key=lambda j: (0 if np.isnan(l[j]) else 1, 0.0 if np.isnan(l[j]) else -l[j], j))[:k]
    return order + [-1] * (k - len(order))


class Routed:
    """Forward pass of one worker's logits [T, E]."""

    def __init__(self, logits, k, renorm=True, mask=None):
        self.l = l = np.asarray(logits, np.float64)
        T, E = l.shape
        self.k, self.renorm = k, renorm
        keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
        self.ok = keep & ~np.all(l == -np.inf, axis=1)
        self.p = np.zeros((T, E))
        self.ids = np.full((T, k), -1, np.int64)
        self.gates = np.zeros((T, k))
        for t in np.flatnonzero(self.ok):
            with np.errstate(invalid="ignore"):
                e = np.exp(l[t] - np.max(l[t]))
                self.p[t] = e / e.sum()
            self.ids[t] = choose(l[t], k)
            open_ = self.ids[t] >= 0
            g = self.p[t][self.ids[t][open_]]
            self.gates[t][open_] = g / g.sum() if renorm else g
        self.counts = np.bincount(self.ids[self.ids >= 0], minlength=E)
        self.psum = self.p.sum(0)
        self.tokens = int(self.ok.sum())
        finite = np.where(np.isfinite(l) & self.ok[:, None], l, np.nan)
        with np.errstate(invalid="ignore"):
            span = np.nanmax(finite) - np.nanmin(finite) if np.isfinite(finite).any() else 0.0
        # relative roundings of one p or gate: its exponent (l - m and its product
        # with log2 e are rounded: 3 span u), exp and its range reduction (4), the
        # sum of E terms (at most E / lanes + log2 lanes <= 40 deep), its
        # reciprocal or quotient and the product (4); the same for the denominator
        self.roundings = 2 * (3 * span + 48)


def balance(routed):
    """(loss, coef, counts, N) of several workers' forward passes."""
    E, k = routed[0].l.shape[1], routed[0].k
    counts = sum(r.counts for r in routed)
    psum = sum(r.psum for r in routed)
    N = sum(r.tokens for r in routed)
    coef = E * counts / (k * N * N) if N else np.zeros(E)
    return float((coef * psum).sum()), coef, counts, N


def backward(r, dgates, coef, dloss):
    """(gradient by the logits, its magnitude for rounding errors) of a Routed."""
    T, E = r.l.shape
    a = np.zeros(E) if coef is None else dloss * np.asarray(coef, np.float64)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in np.flatnonzero(r.ok):
        p = r.p[t]
        out[t] = p * (a - (p * a).sum())
        mag[t] = p * (np.abs(a) + (p * np.abs(a)).sum())
        if dgates is None:
            continue
        open_ = r.ids[t] >= 0
        at, dg = r.ids[t][open_], np.asarray(dgates[t], np.float64)[open_]
        g = r.gates[t][open_]
        if r.renorm:
            out[t][at] += g * (dg - (g * dg).sum())
            mag[t][at] += g * (np.abs(dg) + (g * np.abs(dg)).sum())
        else:
            out[t] -= p * (g * dg).sum()
            mag[t] += p * (g * np.abs(dg)).sum()
            out[t][at] += g * dg
            mag[t][at] += g * np.abs(dg)
    return out, mag
