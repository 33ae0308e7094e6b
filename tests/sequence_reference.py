"""The sequence operators from their definitions in float64 (numpy, step by
step), each with a bound of the error that float32 arithmetic may make.

Bounds are running error bounds: next to every value runs the largest
deviation that its roundings can have caused, each operation off by a few
unit roundoffs u = 2^-24 of its operands' absolute values. They hold for any
order of association of the scan, because a decay or a product of n decays
carries at most n times the error charged per step here."""
import math

import numpy as np

U = 2.0 ** -24
# half a unit in the last place of a stored value, and half the smallest subnormal
STORE = {"fp32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}


def stored(dtype, v):
    rel, tiny = STORE[dtype]
    return rel * np.abs(v) + tiny


def terms(decay, drive, dtype, x, g):
    """(a, 1-a, da/dg, u, ua): the decay, the drive, and the relative error of a, 1-a and da/dg in units of U."""
    if decay == "sigmoid":
        a = 1.0 / (1.0 + np.exp(-g))
        rest = 1.0 / (1.0 + np.exp(g))
        slope = a * rest
    elif decay == "exp":
        a, rest = np.exp(g), -np.expm1(g)
        slope = a
    else:
        a, rest, slope = g, 1.0 - g, np.ones_like(g)
    # exponential, sum, reciprocal and product: an ulp (2 U) each; where the
    # exponent's argument is rounded before exp2, |g| U log2(e) ln 2 more, twice
    ua = 10.0 + 2.0 * np.abs(g)
    return a, rest, slope, (rest * x if drive == "complement" else x), ua


class Recurrence:
    """One sequence [T][C]: h, last, and with dh the gradients, each with its bound."""

    def __init__(self, x, g, h0, decay, drive, dtype, dh=None, dlast=None):
        T, C = x.shape
        a, rest, slope, u, ua = terms(decay, drive, dtype, x, g)
        aa, au = np.abs(a), np.abs(u)
        if drive == "complement" and decay == "value":
            au = (1.0 + aa) * np.abs(x)  # 1 - a rounds against 1 and a
        h, e, size = h0.astype(np.float64), np.zeros(C), np.abs(h0)
        self.h, self.eh = np.zeros((T, C)), np.zeros((T, C))
        before, ebefore, sbefore = np.zeros((T, C)), np.zeros((T, C)), np.zeros((T, C))
        for t in range(T):
            before[t], ebefore[t], sbefore[t] = h, e, size
            h = a[t] * h + u[t]
            e = aa[t] * e + U * ((ua[t] + 3.0) * aa[t] * size + (ua[t] + 2.0) * au[t])
            size = aa[t] * size + au[t]
            e = e + U * size
            self.h[t], self.eh[t] = h, e
        self.last, self.elast = h, e + U * np.abs(h)
        self.eh = self.eh * 1.01 + stored(dtype, self.h)
        if dh is None:
            return
        back = np.zeros(C) if dlast is None else dlast.astype(np.float64)
        e, size = np.zeros(C), np.abs(back)
        self.dx, self.edx, self.dg, self.edg = (np.zeros((T, C)) for _ in range(4))
        for t in range(T - 1, -1, -1):
            r, er, sr = dh[t] + back, e + U * (np.abs(dh[t]) + size), np.abs(dh[t]) + size
            if drive == "complement":
                self.dx[t], self.edx[t] = r * rest[t], er * np.abs(rest[t]) + U * (ua[t] + 2.0) * sr * np.abs(rest[t])
                if decay == "value":
                    self.edx[t] += U * sr * (1.0 + aa[t])
                w, ew = before[t] - x[t], ebefore[t] + 2.0 * U * (sbefore[t] + np.abs(x[t]))
            else:
                self.dx[t], self.edx[t] = r, er
                w, ew = before[t], ebefore[t] + U * sbefore[t]
            sl = np.abs(slope[t])
            self.dg[t] = r * w * slope[t]
            self.edg[t] = er * np.abs(w) * sl + sr * ew * sl + U * (ua[t] + 5.0) * sr * (np.abs(w) + ew) * sl
            back = a[t] * r
            e = aa[t] * er + U * (ua[t] + 3.0) * aa[t] * sr
            size = aa[t] * sr
        self.dh0, self.edh0 = back, e * 1.01 + 2.0 * U * size
        self.edx = self.edx * 1.01 + stored(dtype, self.dx)
        self.edg = self.edg * 1.01 + stored(dtype, self.dg)


def _act(activation, z):
    """act, act', and a bound of |act''|."""
    if activation == "silu":
        p = 1.0 / (1.0 + np.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p)), 0.5
    if activation == "gelu":
        p = np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2.0)))(z) if z.size else z
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi), 0.8
    return z, np.ones_like(z), 0.0


# Roundings in sequence that a sum of a few million terms may take: every
# kernel sums at most some tens of terms one after the other before it joins
# partial sums in a tree.
DEPTH = 100.0


class GroupNorm:
    """One sample [S][C] (its held rows only): y, stats, and with dy the gradients, each with its bound."""

    def __init__(self, x, groups, w, b, eps, activation, dtype, dy=None):
        S, C = x.shape
        D = C // groups
        v = x.reshape(S, groups, D)
        n = S * D
        self.mean, var = v.mean((0, 2)), v.var((0, 2))
        self.rstd = 1.0 / np.sqrt(var + eps)
        self.emean = U * (DEPTH * np.abs(v).mean((0, 2)))
        off = np.abs(v - self.mean[:, None]).mean((0, 2))
        # the variance: its own sum's roundings, the rounded differences, the shifted mean
        evar = U * DEPTH * var + 2.0 * off * U * (np.abs(v).max((0, 2)) if S else 0.0) + self.emean ** 2
        rel = 0.5 * evar / (var + eps) + 4.0 * U
        self.erstd = rel * self.rstd

        def wide(s):
            return np.broadcast_to(s[None, :, None], (S, groups, D)).reshape(S, C)

        mean, rstd = wide(self.mean), wide(self.rstd)
        xhat = (x - mean) * rstd
        exhat = rstd * (wide(self.emean) + U * (np.abs(x) + np.abs(mean))) + np.abs(xhat) * (wide(rel) + 3.0 * U)
        z = xhat * w + b
        ez = exhat * np.abs(w) + 3.0 * U * (np.abs(xhat * w) + np.abs(b))
        f, slope, curve = _act(activation, z)
        steep = 1.13  # both activations' slopes stay under this
        # exponential of an argument rounded to |z| U: relative 2 |z| U, and some ulps
        ef = steep * ez + U * (20.0 + 2.0 * np.abs(z)) * np.abs(f) + U * 2.0 * np.abs(z)
        eslope = curve * ez + U * (30.0 + 4.0 * np.abs(z)) * (1.0 + np.abs(z)) * (0.0 if activation is None else 1.0)
        self.y, self.ey = f, ef + stored(dtype, f)
        if dy is None:
            return
        dz, edz = dy * slope, np.abs(dy) * (eslope + 2.0 * U * np.abs(slope))
        self.db, self.edb = dz.sum(0), edz.sum(0) + U * DEPTH * np.abs(dz).sum(0)
        self.dw = (dz * xhat).sum(0)
        self.edw = (edz * np.abs(xhat) + np.abs(dz) * exhat).sum(0) + U * DEPTH * np.abs(dz * xhat).sum(0)
        t, et = dz * w, edz * np.abs(w) + U * np.abs(dz * w)

        def mean_of(q):
            return wide(q.reshape(S, groups, D).sum((0, 2)) / n)

        m1, em1 = mean_of(t), mean_of(et + U * DEPTH * np.abs(t))
        m2 = mean_of(t * xhat)
        em2 = mean_of(et * np.abs(xhat) + np.abs(t) * exhat + U * DEPTH * np.abs(t * xhat))
        inner = t - m1 - xhat * m2
        size = np.abs(t) + np.abs(m1) + np.abs(xhat * m2)
        einner = et + em1 + exhat * np.abs(m2) + np.abs(xhat) * em2 + 4.0 * U * size
        self.dx = rstd * inner
        self.edx = rstd * einner + np.abs(self.dx) * (wide(rel) + 2.0 * U) + stored(dtype, self.dx)
