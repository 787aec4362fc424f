"""Plain 64-bit forms of the operators around a recurrent mixer, and how far FP32 may be off them.

Every function takes ``mag``: False computes the operator; True computes, with every term of
every sum replaced by its absolute value, what the FP32 rounding errors are relative to.
Rows are flat ([rows, D]); ``bounds`` lists the sequences' (first, last + 1) rows.
"""
import torch

F64 = torch.float64
U = 2.0 ** -24   # half a step of FP32, relative


def d(t):
    return None if t is None else t.detach().to("cpu", F64)


def _a(t, mag):
    return None if t is None else t.abs() if mag else t


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x, mag=False):
    """silu' = p + p x (1 - p); its two terms cancel at x = -1.278, so its rounding is relative to their sum."""
    p = torch.sigmoid(x)
    return p * (1 + (x.abs() if mag else x) * (1 - p))


# ------------------------------------------------------------------ short convolution
def conv_pre(x, w, bias, state0, bounds, mag=False):
    """Pre-activations [rows, D] and last states [S, K-1, D]."""
    K, D = w.shape[1], x.shape[1]
    pre, ends = torch.zeros_like(x), []
    for s, (lo, hi) in enumerate(bounds):
        head = torch.zeros(K - 1, D, dtype=F64) if state0 is None else state0[s]
        ext = torch.cat([head, x[lo:hi]])
        for t in range(hi - lo):
            v = torch.zeros(D, dtype=F64) if bias is None else _a(bias, mag).clone()
            for j in range(K):
                v = v + _a(w[:, j], mag) * _a(ext[t + j], mag)
            pre[lo + t] = v
        ends.append(ext[hi - lo:])
    return pre, torch.stack(ends) if ends else torch.zeros(0, K - 1, D, dtype=F64)


def conv_fwd(x, w, bias, state0, bounds, act=True):
    pre, state_T = conv_pre(x, w, bias, state0, bounds)
    return (silu(pre) if act else pre), state_T


def conv_bwd(x, w, bias, state0, dy, dstate_T, bounds, act=True, mag=False):
    """(dx, dw, dbias, dstate0) by the formulas."""
    K, D = w.shape[1], x.shape[1]
    pre, _ = conv_pre(x, w, bias, state0, bounds)
    dpre = dy * dsilu(pre) if act else dy
    if mag:   # the error of pre enters through |silu''| <= 1/2, beside dpre's own
        far, _ = conv_pre(x, w, bias, state0, bounds, mag=True)
        dpre = dy.abs() * (1.1 + 0.5 * far) if act else dy.abs()
    wa = _a(w, mag)
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(D, dtype=F64)
    ds = torch.zeros(len(bounds), K - 1, D, dtype=F64)
    for s, (lo, hi) in enumerate(bounds):
        head = torch.zeros(K - 1, D, dtype=F64) if state0 is None else state0[s]
        ext = _a(torch.cat([head, x[lo:hi]]), mag)
        dext = torch.zeros_like(ext)
        if dstate_T is not None:
            dext[hi - lo:] += _a(dstate_T[s], mag)
        for t in range(hi - lo):
            for j in range(K):
                dext[t + j] += wa[:, j] * dpre[lo + t]
                dw[:, j] += ext[t + j] * dpre[lo + t]
            db += dpre[lo + t]
        ds[s], dx[lo:hi] = dext[:K - 1], dext[K - 1:]
    return dx, dw, db, ds


# ------------------------------------------------------------------ selective scan
def ssm(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, bounds, dout=None, dh_T=None, softplus=True, mag=False):
    """(out, h_T), or with dout the gradients (du, ddt, dA, dB, dC, dDskip, dz, ddt_bias, dh0)."""
    rows, D = u.shape
    G, N = Bm.shape[1:]
    raw = dt + (0 if dt_bias is None else dt_bias)
    delta = torch.logaddexp(raw, torch.zeros((), dtype=F64)) if softplus else raw
    a = torch.exp(delta[..., None] * A)
    gate = torch.ones_like(u) if z is None else silu(z)
    if mag:
        u, Bm, Cm, Dskip, gate, h0, dout, dh_T = (_a(v, True) for v in (u, Bm, Cm, Dskip, gate, h0, dout, dh_T))
        delta = delta.abs()
    Bw, Cw = (v.repeat_interleave(D // G, 1) for v in (Bm, Cm))
    skip = torch.zeros(D, dtype=F64) if Dskip is None else Dskip
    h, hp = torch.zeros(rows, D, N, dtype=F64), torch.zeros(rows, D, N, dtype=F64)   # h_t, h_{t-1}
    ends = []
    for s, (lo, hi) in enumerate(bounds):
        v = torch.zeros(D, N, dtype=F64) if h0 is None else h0[s]
        for t in range(lo, hi):
            hp[t] = v
            v = a[t] * v + (delta[t] * u[t])[:, None] * Bw[t]
            h[t] = v
        ends.append(v)
    y = (h * Cw).sum(-1) + skip * u
    if dout is None:
        return y * gate, torch.stack(ends) if ends else torch.zeros(0, D, N, dtype=F64)
    dy = dout * gate
    e = torch.zeros_like(h)
    dh0 = torch.zeros(len(bounds), D, N, dtype=F64)
    for s, (lo, hi) in enumerate(bounds):
        v = torch.zeros(D, N, dtype=F64) if dh_T is None else dh_T[s]
        for t in range(hi - 1, lo - 1, -1):
            e[t] = v + dy[t][:, None] * Cw[t]
            v = a[t] * e[t]
        dh0[s] = v
    kept = e * a * hp
    sb = (e * Bw).sum(-1)
    An = A.abs() if mag else A
    dd = (kept * An).sum(-1) + u * sb
    du = skip * dy + delta * sb
    sg = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    ddt = dd * sg
    dA = (kept * delta[..., None]).sum(0)
    fold = lambda v: v.reshape(rows, G, D // G, N).sum(2)  # noqa: E731
    dB, dC = fold(e * (delta * u)[..., None]), fold(h * dy[..., None])
    dz = None if z is None else dout * y * dsilu(z, mag)
    return du, ddt, dA, dB, dC, (dy * u).sum(0), dz, ddt.sum(0), dh0


# ------------------------------------------------------------------ block norm
def rms(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def norm_fwd(residual, block, gate, scale, w_post, w_pre, eps):
    one = torch.ones((), dtype=F64)
    s, wp, wx = (one if v is None else v for v in (scale, w_post, w_pre))
    out = residual
    if block is not None:
        out = residual + s * (one if gate is None else torch.sigmoid(gate)) * rms(block, eps) * wp
    return out, rms(out, eps) * wx


def norm_bwd(r, block, gate, scale, w_post, w_pre, dres, dx, eps, mag=False):
    one = torch.ones((), dtype=F64)
    s, wp, wx = (one if v is None else _a(v, mag) for v in (scale, w_post, w_pre))
    zero = torch.zeros_like(r)
    sub = 1 if mag else -1
    ir = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    m = _a(r * ir, mag)
    dx0 = zero if dx is None else _a(dx, mag)
    dm = dx0 * wx
    dr = zero if dx is None else ir * (dm + sub * m * (dm * m).mean(-1, keepdim=True))
    if dres is not None:
        dr = dr + _a(dres, mag)
    dwx = (dx0 * m).sum(0)
    if block is None:
        return dr, None, None, None, None, dwx
    p = one if gate is None else torch.sigmoid(gate)
    ib = 1 / torch.sqrt((block * block).mean(-1, keepdim=True) + eps)
    n = _a(block * ib, mag)
    dn = dr * s * p * wp
    db = ib * (dn + sub * n * (dn * n).mean(-1, keepdim=True))
    dg = None if gate is None else dr * s * n * wp * p * (1 - p)
    return dr, db, dg, (dr * p * n * wp).sum(0), (dr * p * n * s).sum(0), dwx


# ------------------------------------------------------------------ comparison
def check(name, got, ref, far, n):
    """|got - ref| <= half a step of got's type at ref, and n FP32 half-steps of `far`, the sum of
    the terms' magnitudes: a sum or recursion of n operations is off by at most n U far."""
    if ref is None:
        assert got is None, name
        return
    g = d(got)
    assert g.shape == ref.shape, (name, tuple(g.shape), tuple(ref.shape))
    assert torch.isfinite(g).all(), f"{name}: not finite"
    half = torch.finfo(got.dtype).eps / 2
    tol = half * ref.abs() + n * U * (1 + half) * far + 1e-37   # + FP32's smallest normal number
    bad = (g - ref).abs() > tol
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((g - ref).abs() / tol).max()):.3g} x the tolerance")
