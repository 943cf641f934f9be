"""Plain fp64 forms of the experts' operators, in numpy, on the CPU, with the
magnitudes from which rounding errors are bounded (U = 2^-24 a rounding of fp32
by half a step)."""
import numpy as np

from oracle import pyoracle as po

U = 2.0 ** -24


class Rows:
    """Every expert's slots in the order of the tokens, those without one last."""

    def __init__(self, ids, experts):
        ids = np.asarray(ids)
        self.tokens, self.k = ids.shape
        self.experts = experts
        flat = ids.reshape(-1)
        lists = [[s for s in range(flat.size) if flat[s] == e] for e in range(experts)]
        none = [s for s in range(flat.size) if not 0 <= flat[s] < experts]
        self.offsets = np.cumsum([0] + [len(l) for l in lists])
        self.source = np.array(sum(lists, []) + none, np.int64)
        self.n = int(self.offsets[-1])
        self.row = np.full(flat.size, -1, np.int64)
        self.row[self.source[:self.n]] = np.arange(self.n)
        self.row = self.row.reshape(ids.shape)
        self.token = self.source // self.k

    def of(self, e):
        return slice(int(self.offsets[e]), int(self.offsets[e + 1]))


def matmul(x, w, rows, gather=False):
    """(y, sum of |x| |w|) for the rows of experts."""
    x = x[rows.token] if gather else x
    y, mag = (np.zeros((rows.n, w.shape[2])) for _ in range(2))
    for e in range(rows.experts):
        r = rows.of(e)
        y[r], mag[r] = x[r] @ w[e], np.abs(x[r]) @ np.abs(w[e])
    return y, mag


def matmul_grad(x, dy, rows, gather=None):
    x = x[rows.token] if gather == "x" else x
    dy = dy[rows.token] if gather == "dout" else dy
    dw, mag = (np.zeros((rows.experts, x.shape[1], dy.shape[1])) for _ in range(2))
    for e in range(rows.experts):
        r = rows.of(e)
        dw[e], mag[e] = x[r].T @ dy[r], np.abs(x[r]).T @ np.abs(dy[r])
    return dw, mag


def back(y, rows, residual=None):
    """(sums per token, their magnitude)."""
    out = np.zeros((rows.tokens, y.shape[1])) if residual is None else residual.copy()
    mag = np.abs(out)
    for t in range(rows.tokens):
        for r in rows.row[t]:
            if r >= 0:
                out[t] += y[r]
                mag[t] += np.abs(y[r])
    return out, mag


def sigmoid(x):
    return 1 / (1 + np.exp(-x))


def act(u, gate, kind):
    """a of rows u with gates [n]."""
    if kind == "relu":
        return gate[:, None] * np.maximum(u, 0)
    g, v = np.split(u, 2, 1)
    return gate[:, None] * g * sigmoid(g) * v


# Roundings in the sigmoid, relative: exp2 and the reciprocal one unit (2 U) each, the
# compensated exponent and the sum half a unit each, the constants' last bits one.
SIGMOID = 8


def act_backward(u, da, gate, kind):
    """(du, dgate, a) and bounds of what fp32 makes of them."""
    a = act(u, gate, kind)
    if kind == "relu":
        h = np.maximum(u, 0)
        du = gate[:, None] * da * (u > 0)
        e_du, e_a, e_h = U * np.abs(du), U * np.abs(a), np.zeros_like(h)
    else:
        g, v = np.split(u, 2, 1)
        s, t = sigmoid(g), gate[:, None] * da
        h = g * s * v
        slope = 1 + g * (1 - s)
        du = np.concatenate((t * v * s * slope, t * g * s), 1)
        # 1 - s is off by the sigmoid's error and a rounding, then a product and a sum
        e_slope = U * (np.abs(g) * (SIGMOID * s + 2 * (1 - s)) + np.abs(slope))
        e_du = np.concatenate((np.abs(t * v * s) * (e_slope + (SIGMOID + 5) * U * np.abs(slope)),
                               (SIGMOID + 4) * U * np.abs(du[:, g.shape[1]:])), 1)
        e_h, e_a = (SIGMOID + 3) * U * np.abs(h), (SIGMOID + 4) * U * np.abs(a)
    n = h.shape[1]
    e_gate = (np.abs(da) * (e_h + (n + 2) * U * np.abs(h))).sum(1)
    return (du, (da * h).sum(1), a), (e_du, e_gate, e_a)


def dithers(n, seed=1, rnd=0, worker=0, site=0):
    """The 16-bit dithers of elements 0 .. n - 1 of a keep call, by the oracle's
    Philox."""
    out = []
    for b in range((n + 7) // 8):
        w = po.philox4x32([b & 0xFFFFFFFF, (b >> 32) | 0x8000 | worker << 16, rnd, (1 << 31) | site],
                          [seed & 0xFFFFFFFF, seed >> 32])
        out += [h for x in w for h in (int(x) & 0xFFFF, int(x) >> 16)]
    return np.array(out[:n], np.int64)


def keep(x, d):
    """(codes, exponent bytes, values) of a matrix with its elements' dithers."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.int64)
    exps = np.zeros((rows, (cols + 31) // 32), np.int64)
    values = np.zeros((rows, cols))
    d = np.broadcast_to(np.asarray(d).reshape(-1, cols) if np.ndim(d) else d, (rows, cols))
    for r in range(rows):
        for b in range(exps.shape[1]):
            at = slice(32 * b, min(cols, 32 * b + 32))
            v = x[r, at]
            if not (np.abs(v) <= 127 * 2.0 ** 121).all():
                exps[r, b] = 255
                values[r, at] = np.nan
                continue
            s = -110
            while np.abs(v).max() > 127 * 2.0 ** s:
                s += 1
            q = np.floor((np.floor(np.abs(v) * 2.0 ** (16 - s)) + d[r, at]) / 65536)
            codes[r, at] = np.sign(v) * q
            exps[r, b] = s + 127
            values[r, at] = codes[r, at] * 2.0 ** s
    return codes, exps, values
