"""The 64-bit forms that the GPU tests compare with: their gradients against autograd and differences."""
import pytest
import torch

from tests import _layers_err as E
from tests import _layers_ref as R

F64 = torch.float64


def _t(g, *shape):
    return torch.randn(*shape, generator=g, dtype=F64)


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv_formulas(K, act, state):
    g = torch.Generator().manual_seed(K)
    bounds = [(0, 1), (1, 1), (1, 8), (9, 11)]
    D, rows, S = 3, 12, 4
    x, w, b = _t(g, rows, D), _t(g, D, K), _t(g, D)
    s0 = _t(g, S, K - 1, D) if state else None
    dy, dsT = _t(g, rows, D), _t(g, S, K - 1, D)
    inside = torch.zeros(rows, 1, dtype=F64)
    for lo, hi in bounds:
        inside[lo:hi] = 1
    leaves = [v.requires_grad_() for v in (x, w, b) + ((s0,) if state else ())]

    def loss():
        y, sT = R.conv_fwd(x, w, b, s0, bounds, act)
        return (y * dy * inside).sum() + (sT * dsT).sum()

    auto = torch.autograd.grad(loss(), leaves)
    with torch.no_grad():
        mine = R.conv_bwd(x, w, b, s0, dy, dsT, bounds, act)
        for a, m in zip(auto, mine):
            assert torch.allclose(a, m, rtol=1e-11, atol=1e-11)
        far = R.conv_bwd(x, w, b, s0, dy, dsT, bounds, act, mag=True)
        for m, f in zip(mine, far):
            assert (m.abs() <= f * (1 + 1e-12) + 1e-12).all()
        v = [_t(g, *p.shape) for p in leaves]
        h = 1e-6   # central difference: error h^2 from the third derivative, 1e-16 / h from rounding
        for p, q in zip(leaves, v):
            p += h * q
        up = loss()
        for p, q in zip(leaves, v):
            p -= 2 * h * q
        down = loss()
        want = sum((a * q).sum() for a, q in zip(auto, v))
        assert abs((up - down) / (2 * h) - want) <= 1e-7 * (1 + abs(want))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("G", [1, 2])
def test_ssm_formulas(G, softplus, gated):
    g = torch.Generator().manual_seed(G)
    bounds = [(0, 5), (5, 5), (5, 6), (6, 11)]
    rows, D, N, S = 11, 4, 3, 4
    u, z, dt = _t(g, rows, D), _t(g, rows, D), _t(g, rows, D)
    if not softplus:
        dt = dt.abs() * 0.3
    A, Bm, Cm = -_t(g, D, N).abs(), _t(g, rows, G, N), _t(g, rows, G, N)
    Ds, bias, h0 = _t(g, D), _t(g, D) * 0.1, _t(g, S, D, N)
    dout, dhT = _t(g, rows, D), _t(g, S, D, N)
    if not gated:
        z = None
    leaves = [u, dt, A, Bm, Cm, Ds] + ([z] if gated else []) + [bias, h0]
    for v in leaves:
        v.requires_grad_()

    def loss():
        # the recursion again, without in-place writes, for autograd
        raw = dt + bias
        delta = torch.nn.functional.softplus(raw, threshold=100) if softplus else raw
        total = 0.0
        for s, (lo, hi) in enumerate(bounds):
            h = h0[s]
            for t in range(lo, hi):
                Bt, Ct = (v[t].repeat_interleave(D // G, 0) for v in (Bm, Cm))
                h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * u[t])[:, None] * Bt
                y = (h * Ct).sum(-1) + Ds * u[t]
                total = total + (dout[t] * (y * R.silu(z[t]) if gated else y)).sum()
            total = total + (dhT[s] * h).sum()
        return total

    auto = torch.autograd.grad(loss(), leaves)
    with torch.no_grad():
        args = (u, dt, A, Bm, Cm, Ds, z, bias, h0, bounds, dout, dhT, softplus)
        mine = [v for v in R.ssm(*args) if v is not None]
        far = [v for v in R.ssm(*args, mag=True) if v is not None]
        for a, m, f in zip(auto, mine, far):
            assert torch.allclose(a, m, rtol=1e-10, atol=1e-10)
            assert (m.abs() <= f * (1 + 1e-12) + 1e-12).all()
        v = [_t(g, *p.shape) for p in leaves]
        h = 1e-6
        for p, q in zip(leaves, v):
            p += h * q
        up = loss()
        for p, q in zip(leaves, v):
            p -= 2 * h * q
        down = loss()
        want = sum((a * q).sum() for a, q in zip(auto, v))
        assert abs((up - down) / (2 * h) - want) <= 1e-6 * (1 + abs(want))


@pytest.mark.parametrize("gated", [False, True])
def test_norm_formulas(gated):
    g = torch.Generator().manual_seed(0)
    rows, D, eps = 4, 6, 1e-5
    r, b, gate = _t(g, rows, D), _t(g, rows, D), _t(g, rows, D) if gated else None
    s, wp, wx = _t(g, D), _t(g, D), _t(g, D)
    dres, dx = _t(g, rows, D), _t(g, rows, D)
    leaves = [v.requires_grad_() for v in [r, b] + ([gate] if gated else []) + [s, wp, wx]]
    out, x = R.norm_fwd(r, b, gate, s, wp, wx, eps)
    auto = torch.autograd.grad((out * dres).sum() + (x * dx).sum(), leaves)
    with torch.no_grad():
        args = (out.detach(), b, gate, s, wp, wx, dres, dx, eps)
        mine = [v for v in R.norm_bwd(*args) if v is not None]
        far = [v for v in R.norm_bwd(*args, mag=True) if v is not None]
        for a, m, f in zip(auto, mine, far):
            assert torch.allclose(a, m, rtol=1e-10, atol=1e-10)
            assert (m.abs() <= f * (1 + 1e-12) + 1e-12).all()


@pytest.mark.parametrize("G", [1, 2])
def test_ssm_running_error_bound(G):
    """Its values are the plain form's, and FP32 of the plain recursion stays within its bound, by less than 100 times."""
    g = torch.Generator().manual_seed(G)
    bounds, rows, D, N = [(0, 150), (150, 151), (151, 151), (151, 300)], 300, 4, 8
    u, z, dt = _t(g, rows, D), _t(g, rows, D), _t(g, rows, D)
    A, Bm, Cm = -_t(g, D, N).abs() - 0.1, _t(g, rows, G, N), _t(g, rows, G, N)
    Ds, bias, h0 = _t(g, D), _t(g, D) - 3, _t(g, 4, D, N)
    dout, dhT = _t(g, rows, D), _t(g, 4, D, N)
    single = [v.float() for v in (u, dt, A, Bm, Cm, Ds, z, bias, h0, dout, dhT)]
    u, dt, A, Bm, Cm, Ds, z, bias, h0, dout, dhT = (v.double() for v in single)
    args = (u, dt, A, Bm, Cm, Ds, z, bias, h0, bounds)
    fwd, bwd = E.ssm(*args, dout, dhT, 64)
    worst = 0.0
    u, dt, A, Bm, Cm, Ds, z, bias, h0, dout, dhT = single
    # the plain recursion token by token in FP32
    out, ends = [], []
    for s, (lo, hi) in enumerate(bounds):
        h = h0[s]
        for t in range(lo, hi):
            delta = torch.log1p(torch.exp(dt[t] + bias))[:, None]
            h = torch.exp(delta * A) * h + delta * u[t][:, None] * Bm[t].repeat_interleave(D // G, 0)
            out.append(((h * Cm[t].repeat_interleave(D // G, 0)).sum(-1) + Ds * u[t]) * R.silu(z[t]))
        ends.append(h)
    for name, o, w, r in zip(("out", "h_T"), (torch.stack(out), torch.stack(ends)), fwd, R.ssm(*args)):
        assert torch.allclose(w.v, r, rtol=1e-12, atol=1e-12)
        worst = max(worst, E.check(name, o, w))
    assert worst > 0.01
    for w, r in zip(bwd, R.ssm(*args, dout.double(), dhT.double())):
        assert torch.allclose(w.v, r, rtol=1e-11, atol=1e-11)
