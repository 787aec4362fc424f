"""The selective scan in 64 bits with a running bound of its FP32 rounding errors.

A ``V`` carries values and, in half-steps of FP32 (2^-24), how far FP32 may be off each: a product or a sum
adds a half-step of its result to what its operands' errors make of it, to first order.  Unlike a count of
roundings times the terms' magnitudes, the bound forgets with the state what happened many tokens ago.
"""
import torch

from tests import _layers_ref as R

F64 = torch.float64


class V:
    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def __mul__(self, o):
        p = self.v * o.v
        return V(p, self.v.abs() * o.e + o.v.abs() * self.e + p.abs())

    def __add__(self, o):
        s = self.v + o.v
        return V(s, self.e + o.e + s.abs())

    def __getitem__(self, i):
        return V(self.v[i], self.e[i])

    def sum(self, dim, depth):
        """A sum whose terms go through at most `depth` additions."""
        return V(self.v.sum(dim), self.e.sum(dim) + depth * self.v.abs().sum(dim))

    def f(self, fn):
        """Shapes only."""
        return V(fn(self.v), fn(self.e))


def _stack(vs):
    return V(torch.stack([x.v for x in vs]), torch.stack([x.e for x in vs]))


def _own(x):
    """Half-steps of the activations themselves: 12 + 1.23 |x| below zero, 12 above."""
    return 12 + 1.23 * x.clamp(max=0).abs()


def sigmoid(x):
    s = torch.sigmoid(x.v)
    return V(s, _own(x.v) * s + s * (1 - s) * x.e)


def silu(x):
    s = R.silu(x.v)
    return V(s, _own(x.v) * s.abs() + R.dsilu(x.v).abs() * x.e)


def softplus(x):
    s = torch.logaddexp(x.v, torch.zeros((), dtype=F64))
    return V(s, _own(x.v) * s + torch.sigmoid(x.v) * x.e)


def ssm(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, bounds, dout, dh_T, span):
    """V of (out, h_T) and of (du, ddt, dA, dB, dC, dDskip, dz, ddt_bias, dh0); every optional input given.

    `span`: the most rows of a span.  A decay factor's exponent is delta times A log2(e): the latter's rounding
    and the product's are 3 half-steps of it with log2(e)'s own, and where a span's factors are taken as one, their
    deltas' sum adds a half-step a row.  The exponential is off by 4, the products of factors add 1 each.
    """
    rows, D = u.shape
    G, N = Bm.shape[1:]
    wide = lambda t: V(t.repeat_interleave(D // G, 1))  # noqa: E731
    u, A, skip, z, dout = V(u), V(A), V(Dskip), V(z), V(dout)
    raw = V(dt) + V(dt_bias.expand_as(dt))
    delta = softplus(raw)
    gate = silu(z)
    Bw, Cw = wide(Bm), wide(Cm)
    decay = torch.exp(delta.v[..., None] * A.v)
    alpha = (delta.v[..., None] * A.v).abs()
    a = V(decay, decay * (5 + alpha * (3 + span) + A.v.abs() * delta.e[..., None]))
    x = delta * u
    last = lambda t: t.f(lambda v: v[..., None])  # noqa: E731
    inp = last(x) * Bw
    h, hp, ends, starts = [], [], [], []
    for s, (lo, hi) in enumerate(bounds):
        v = V(h0[s])
        for t in range(lo, hi):
            hp.append(v)
            v = a[t] * v + inp[t]
            h.append(v)
        ends.append(v)
    h, hp, h_T = _stack(h), _stack(hp), _stack(ends)
    y = (h * Cw).sum(-1, N) + skip * u
    out = y * gate
    dy = dout * gate
    g = last(dy) * Cw
    e = [None] * rows
    for s, (lo, hi) in enumerate(bounds):
        v = V(dh_T[s])
        for t in range(hi - 1, lo - 1, -1):
            e[t] = v + g[t]
            v = a[t] * e[t]
        starts.append(v)
    e, dh0 = _stack(e), _stack(starts)
    kept = a * e * hp
    sb = (e * Bw).sum(-1, N)
    # kept goes with A log2(e), and the sum with ln 2: two constants' and three products' roundings
    sq = (kept * V(A.v.expand_as(kept.v), 4 * A.v.abs().expand_as(kept.v))).sum(-1, N)
    sq = V(sq.v, sq.e + 2 * sq.v.abs())
    dd = sq + u * sb
    ddt = dd * sigmoid(raw)
    du = skip * dy + delta * sb
    depth = span + 8 + rows // span // 8 + 1 + len(bounds)   # a span's rows, then eight shares of the spans
    fold = lambda t: t.f(lambda v: v.reshape(rows, G, D // G, N)).sum(2, D // G)  # noqa: E731
    one = V(torch.ones_like(z.v))
    sg = sigmoid(z)
    dsilu = sg * (one + z * (one + V(-sg.v, sg.e)))
    grads = (du, ddt, (kept * last(delta)).sum(0, depth), fold(e * last(x)), fold(h * last(dy)),
             (dy * u).sum(0, depth), dout * y * dsilu, ddt.sum(0, depth), dh0)
    return (out, h_T), grads


def check(name, got, want):
    """Within the bound (1 % for what is beyond first order) and half a step of the output's type."""
    g = R.d(got).reshape(want.v.shape)
    half = torch.finfo(got.dtype).eps / 2
    tol = half * want.v.abs() + 1.01 * R.U * want.e + 1e-37
    worst = float(((g - want.v).abs() / tol).max())
    assert worst <= 1, f"{name}: {worst:.3g} x the bound"
    return worst
