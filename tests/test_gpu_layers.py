"""Short convolution, selective scan and block norm on the GPU against their plain 64-bit forms.

Tolerances are counted, not fitted (``_layers_ref.check``): half a step of the output's type at the
value, and n half-steps of FP32 relative to the sum of the terms' magnitudes.  n counts roundings on
the longest path into a value: the additions of its sum, and about 48 for the activations (the
hardware's exponential and reciprocal are off by 2 half-steps or so each, and an exponential of an
argument x also by 1.5 |x| half-steps for the argument's own rounding, |x| < 20 here).  For the
recursion each token adds the same again, at most 24: its decay factor's, delta's, the products'.
"""
import threading

import pytest
import torch

from tests import _layers_err as E
from tests import _layers_ref as R

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.bfloat16]
NAN = float("nan")


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_73_b200 import build
    build.build()
    import gated_delta_rule_73_b200 as K
    return K


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _n(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def _u(g, lo, hi, *shape, dtype=torch.float32):
    return (torch.rand(*shape, generator=g) * (hi - lo) + lo).to(dtype).cuda()


def _wide(t, extra, fill=NAN):
    """The same values as a column range of a wider tensor whose other columns hold NaN."""
    w = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), fill, dtype=t.dtype, device=t.device)
    w[..., :t.shape[-1]] = t
    return w[..., :t.shape[-1]]


def _dense(B, T):
    return (B, T), None, [(i * T, (i + 1) * T) for i in range(B)]


def _packed(cuts, rows):
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    return (rows,), cu, list(zip(cuts[:-1], cuts[1:]))


def _flat(t, tail=1):
    return None if t is None else R.d(t).reshape(-1, *t.shape[t.dim() - tail:])


# ------------------------------------------------------------------ short convolution
CONV = [
    # layout, D, K, state, bias, act, wide
    (_dense(1, 1), 8, 4, False, True, True, 0),
    (_dense(3, 2), 16, 4, True, True, True, 0),
    (_dense(2, 37), 64, 4, True, True, True, 8),
    (_dense(2, 130), 24, 3, False, False, True, 0),
    (_dense(1, 65), 7, 2, True, True, False, 0),
    (_dense(2, 33), 20, 4, True, True, True, 5),
    (_packed([0, 5, 5, 6, 40, 41], 41), 32, 4, True, True, True, 0),
    (_packed([3, 10, 12, 12, 77], 90), 9, 3, True, True, True, 0),
    (_packed([0, 0, 300], 300), 264, 4, False, True, True, 8),
    (_packed([0], 5), 8, 4, False, True, True, 0),
] if torch.cuda.is_available() else []


def _conv_inputs(lay, D, k, state, bias, dtype, wide, seed=0):
    lead, cu, bounds = lay
    g = _gen(seed)
    x = _n(g, *lead, D, dtype=dtype)
    if wide:
        x = _wide(x, wide)
    S = len(bounds)
    return (x, _u(g, -0.7, 0.7, D, k, dtype=dtype), _n(g, D, dtype=dtype, std=0.3) if bias else None,
            _n(g, S, k - 1, D, dtype=dtype) if state else None, cu, bounds, g)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", range(len(CONV)))
def test_short_conv_forward_and_backward(K, case, dtype):
    lay, D, k, state, bias, act, wide = CONV[case]
    x, w, b, s0, cu, bounds, g = _conv_inputs(lay, D, k, state, bias, dtype, wide)
    S, rows = len(bounds), x.numel() // D
    y, sT = K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu, silu=act)
    ref = [_flat(x), R.d(w), R.d(b), R.d(s0)]
    pre, rsT = R.conv_pre(*ref, bounds)
    far, _ = R.conv_pre(*ref, bounds, mag=True)
    ry = R.silu(pre) if act else pre
    R.check("y", y.reshape(-1, D), ry, 1.1 * far + ry.abs(), k + 48)   # |silu'| <= 1.1
    assert torch.equal(R.d(sT), rsT)                                   # copies

    dy = _n(g, *x.shape, dtype=dtype)
    if wide:
        dy = _wide(dy, wide)
    dsT = _n(g, S, k - 1, D) if state else None
    got = K.short_conv_bwd(x, w, b, s0, dy, dsT, cu_seqlens=cu, silu=act)
    args = (*ref, _flat(dy), R.d(dsT), bounds, act)
    want, mag = R.conv_bwd(*args), R.conv_bwd(*args, mag=True)
    if not bias:
        want, mag = want[:2] + (None,) + want[3:], mag
    if not state:
        want = want[:3] + (None,)
    for name, o, r, f, n in zip(("dx", "dw", "dbias", "dstate0"), got, want, mag,
                                (k + 48, rows + 48, rows + 48, k + 48)):
        R.check(name, o.reshape(-1, D) if name == "dx" else o, r, f, n)


@pytest.mark.parametrize("dtype", DT)
def test_short_conv_leaves_rows_of_no_sequence(K, dtype):
    lay = _packed([3, 10, 12, 12, 77], 90)
    for D in (16, 5):
        x, w, b, s0, cu, bounds, g = _conv_inputs(lay, D, 4, True, True, dtype, 0)
        x[:3] = NAN
        x[77:] = NAN
        y = torch.full_like(x, 7.0)
        K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu, y=y)
        assert (y[:3] == 7).all() and (y[77:] == 7).all() and torch.isfinite(y[3:77]).all()
        y2, sT = K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu)
        assert (y2[:3] == 0).all() and (y2[77:] == 0).all() and torch.equal(y2[3:77], y[3:77])
        assert torch.isfinite(sT).all() and torch.equal(sT[2], s0[2])
        dy = torch.full_like(x, NAN)
        dy[3:77] = _n(g, 74, D, dtype=dtype)
        for o in K.short_conv_bwd(x, w, b, s0, dy, _n(g, 4, 3, D), cu_seqlens=cu):
            assert torch.isfinite(o).all()
        # a table beyond the rows is cut off at them
        cu2 = torch.tensor([3, 10, 12, 12, 4000], dtype=torch.int32, device="cuda")
        x[77:] = 0
        y3, _ = K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu2)
        assert torch.equal(y3[3:77], y[3:77])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,k", [(8, 4), (33, 3), (1024, 2)])
def test_short_conv_step_continues_the_sequence(K, D, k, dtype):
    B, T = 3, 7
    x, w, b, s0, _, _, _ = _conv_inputs(_dense(B, T), D, k, True, True, dtype, 0)
    y, sT = K.short_conv_fwd(x, w, b, s0)
    _, st = K.short_conv_fwd(x[:, :4].contiguous(), w, b, s0)
    before = st.clone()
    out = torch.empty_like(st)
    K.short_conv_step(x[:, 4], w, b, st, state_out=out)
    assert torch.equal(st, before)
    for t in range(4, T):
        o = K.short_conv_step(x[:, t], w, b, st)   # in place, strided rows
        assert torch.equal(o, y[:, t])             # the same sums in the same order
        if t == 4:
            assert torch.equal(st, out)
    assert torch.equal(st, sT)


# ------------------------------------------------------------------ selective scan
SSM = [
    # layout, D, N, G, state, softplus, gated, skip, wide
    (_dense(1, 1), 8, 16, 1, False, True, True, True, 0),
    (_dense(2, 15), 64, 16, 1, True, True, True, True, 0),
    (_dense(1, 16), 96, 8, 1, True, True, False, True, 8),
    (_dense(2, 65), 40, 32, 2, True, True, True, False, 8),
    (_dense(1, 130), 7, 64, 1, False, True, True, True, 0),
    (_dense(3, 200), 66, 16, 3, True, False, True, True, 0),
    (_dense(1, 333), 130, 8, 2, True, True, True, True, 3),
    (_dense(40, 20), 64, 64, 1, True, True, True, True, 0),
    (_packed([0, 5, 5, 69, 200, 201], 201), 72, 16, 1, True, True, True, True, 0),
    (_packed([2, 3, 130, 130, 150], 170), 33, 32, 1, True, True, True, True, 0),
    (_packed([0, 64, 128], 128), 16, 64, 4, False, True, False, True, 8),
    (_packed([0, 0, 0], 3), 16, 16, 1, True, True, True, True, 0),
    (_packed([0], 3), 16, 16, 1, False, True, True, True, 0),
    # by size: spans of time (few channels, long), four states a lane, a lane a channel
    (_dense(1, 1500), 8, 8, 1, True, True, True, True, 0),
    (_packed([0, 700, 701, 1600], 1600), 6, 16, 2, True, True, True, True, 0),
    (_dense(1, 100), 301, 16, 1, True, True, False, False, 1),
    (_dense(130, 3), 256, 8, 1, True, True, True, True, 0),
    (_dense(250, 2), 384, 16, 1, True, True, True, True, 0),
    (_dense(250, 2), 93, 64, 1, False, True, True, True, 0),
    (_dense(300, 3), 162, 32, 3, True, False, False, True, 0),
    (_dense(12, 126), 4096, 16, 1, True, True, True, True, 0),   # enough blocks for the longest spans of the backward
    (_packed(sorted([0] + [(i * 7919) % 601 for i in range(260)] + [601]), 601), 380, 16, 1, True, True, True, True, 4),
] if torch.cuda.is_available() else []


def _ssm_inputs(lay, D, N, G, state, softplus, gated, skip, wide, dtype, seed=0):
    lead, cu, bounds = lay
    g = _gen(seed)
    S = len(bounds)
    row = lambda t: _wide(t, wide) if wide else t  # noqa: E731
    u, z = row(_n(g, *lead, D, dtype=dtype)), row(_n(g, *lead, D, dtype=dtype)) if gated else None
    dt = _n(g, *lead, D, dtype=dtype) if softplus else _u(g, 0.0, 0.3, *lead, D, dtype=dtype)
    bc = _n(g, *lead, 2 * G * N + wide, dtype=dtype)
    Bm, Cm = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:2 * G * N].unflatten(-1, (G, N))
    if wide % 8:
        Bm, Cm = Bm.contiguous(), Cm.contiguous()
    A = -_u(g, 0.05, 1.0, D, N) * torch.arange(1, N + 1, device="cuda")
    bias = _u(g, -5.0, -1.0, D) if softplus else None
    return (u, dt, A.contiguous(), Bm, Cm, _n(g, D) if skip else None, z, bias, _n(g, S, D, N) if state else None), cu, bounds, g


def _ssm_ref(args, bounds, *more, **kw):
    u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
    return R.ssm(_flat(u), _flat(dt), R.d(A), _flat(Bm, 2), _flat(Cm, 2), R.d(Ds), _flat(z), R.d(bias), R.d(h0), bounds,
                 *more, **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", range(len(SSM)))
def test_ssm_scan_forward_and_backward(K, case, dtype):
    lay, D, N, G, state, softplus, gated, skip, wide = SSM[case]
    args, cu, bounds, g = _ssm_inputs(lay, D, N, G, state, softplus, gated, skip, wide, dtype)
    S, T = len(bounds), max([0] + [hi - lo for lo, hi in bounds])
    u = args[0]
    rows = u.numel() // D
    kw = dict(softplus=softplus)
    out, hT = K.ssm_scan_fwd(*args, cu_seqlens=cu, dt_softplus=softplus)
    (ro, rh), (fo, fh) = _ssm_ref(args, bounds, **kw), _ssm_ref(args, bounds, mag=True, **kw)
    for lo, hi in bounds:   # rows of no sequence: see the zero test below
        R.check("out", out.reshape(-1, D)[lo:hi], ro[lo:hi], fo[lo:hi], 24 * T + N + 64)
    R.check("h_T", hT, rh, fh, 24 * T + 64)

    dout = _n(g, *u.shape, dtype=dtype)
    if wide:
        dout = _wide(dout, wide)
    dhT = _n(g, S, D, N) if state else None
    got = K.ssm_scan_bwd(*args, dout, dhT, cu_seqlens=cu, dt_softplus=softplus)
    inside = torch.zeros(rows, 1, dtype=R.F64)
    for lo, hi in bounds:
        inside[lo:hi] = 1
    more = (_flat(dout) * inside, R.d(dhT))
    ref, far = _ssm_ref(args, bounds, *more, **kw), _ssm_ref(args, bounds, *more, mag=True, **kw)
    names = ("du", "ddt", "dA", "dB", "dC", "dDskip", "dz", "ddt_bias", "dh0")
    have = (1, 1, 1, 1, 1, skip, gated, softplus, state)
    for name, o, r, f, h in zip(names, got, ref, far, have):
        if not h:
            assert o is None
            continue
        n = 48 * T + N + D + 128 + (rows if name in ("dA", "dDskip", "ddt_bias") else 0)
        R.check(name, o.reshape(r.shape), r, f, n)


@pytest.mark.parametrize("lay,D,N,G", [(_dense(1, 1500), 8, 8, 1),                    # spans of time
                                       (_dense(1, 500), 24, 16, 1),                   # four states a lane
                                       (_packed([0, 700, 701, 701, 1600], 1600), 6, 16, 2),
                                       (_packed([0, 900, 1000], 1000), 12, 32, 1)]
                         if torch.cuda.is_available() else [])
def test_ssm_error_of_long_sequences(K, lay, D, N, G):
    """FP32 over long sequences within a running bound of the roundings, which decays as the states do: 60 to 2,000
    times below a count of all tokens' roundings."""
    args, cu, bounds, g = _ssm_inputs(lay, D, N, G, True, True, True, True, 0, torch.float32)
    S = len(bounds)
    dout, dhT = _n(g, *args[0].shape), _n(g, S, D, N)
    u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
    (out, hT), grads = E.ssm(_flat(u), _flat(dt), R.d(A), _flat(Bm, 2), _flat(Cm, 2), R.d(Ds), _flat(z), R.d(bias), R.d(h0),
                             bounds, _flat(dout), R.d(dhT), 64)
    got, ghT = K.ssm_scan_fwd(*args, cu_seqlens=cu)
    E.check("out", got, out)
    E.check("h_T", ghT, hT)
    for name, o, w in zip(("du", "ddt", "dA", "dB", "dC", "dDskip", "dz", "ddt_bias", "dh0"),
                          K.ssm_scan_bwd(*args, dout, dhT, cu_seqlens=cu), grads):
        E.check(name, o, w)


@pytest.mark.parametrize("dtype", DT)
def test_ssm_scan_leaves_rows_of_no_sequence(K, dtype):
    for D, N in ((64, 16), (33, 64)):
        args, cu, bounds, g = _ssm_inputs(_packed([2, 3, 130, 130, 150], 170), D, N, 1, True, True, True, True, 0, dtype)
        for t in args[:2] + args[3:5] + (args[6],):
            t[:2] = NAN
            t[150:] = NAN
        out = torch.full_like(args[0], 7.0)
        K.ssm_scan_fwd(*args, cu_seqlens=cu, out=out)
        assert (out[:2] == 7).all() and (out[150:] == 7).all() and torch.isfinite(out[2:150]).all()
        o2, hT = K.ssm_scan_fwd(*args, cu_seqlens=cu)
        assert (o2[:2] == 0).all() and (o2[150:] == 0).all() and torch.equal(o2[2:150], out[2:150])
        assert torch.isfinite(hT).all() and torch.equal(hT[2], args[8][2])
        dout = torch.full_like(args[0], NAN)
        dout[2:150] = _n(g, 148, D, dtype=dtype)
        dhT = _n(g, 4, D, N)
        got = K.ssm_scan_bwd(*args, dout, dhT, cu_seqlens=cu)
        for o in got:
            assert torch.isfinite(o).all()
        for o in (got[0], got[1], got[3], got[4], got[6]):
            assert (o[:2] == 0).all() and (o[150:] == 0).all()
        assert torch.equal(got[8][2], dhT[2])   # no token: the gradient passes


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,D,N,G", [(3, 64, 16, 1), (3, 33, 8, 3), (3, 20, 64, 2), (3, 130, 32, 1),
                                     # lanes walk several sequences: 9 in one part, parts of 3, 7 and 8, the last one shorter
                                     (9, 75776, 16, 1), (11, 3 * 12600, 8, 3), (13, 9472, 64, 1), (22, 12000, 32, 2)])
def test_ssm_step_continues_the_sequence(K, B, D, N, G, dtype):
    T = 6 if B == 3 else 2
    args, _, bounds, _ = _ssm_inputs(_dense(B, T), D, N, G, True, True, True, True, 0, dtype)
    u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
    (ro, rh), (fo, fh) = _ssm_ref(args, bounds), _ssm_ref(args, bounds, mag=True)
    h = h0.clone()
    outs = []
    for t in range(T):
        if t == 0:   # out of place first: the old state stays
            h1 = torch.empty_like(h)
            o1 = K.ssm_step(u[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0], Ds, z[:, 0], bias, h, h_out=h1)
            assert torch.equal(h, h0)
        outs.append(K.ssm_step(u[:, t], dt[:, t], A, Bm[:, t], Cm[:, t], Ds, z[:, t], bias, h))
        if t == 0:
            assert torch.equal(outs[0], o1) and torch.equal(h, h1)
    R.check("out", torch.stack(outs, 1).reshape(-1, D), ro, fo, 24 * T + N + 64)
    R.check("h", h, rh, fh, 24 * T + 64)


@pytest.mark.parametrize("dtype", DT)
def test_empty_calls(K, dtype):
    """No tokens: states go through; no sequences or no channels: sums of nothing."""
    e = lambda *s, t=dtype: torch.randn(*s, device="cuda").to(t)  # noqa: E731
    for B, T, D in ((3, 0, 16), (0, 5, 16), (2, 4, 0), (0, 0, 0)):
        x, w, b, s0 = e(B, T, D), e(D, 4), e(D), e(B, 3, D)
        y, sT = K.short_conv_fwd(x, w, b, s0)
        assert y.shape == x.shape and sT.shape == s0.shape
        g = e(B, 3, D, t=torch.float32)
        dx, dw, db, ds = K.short_conv_bwd(x, w, b, s0, e(B, T, D), g)
        A, Bm, Cm = -torch.rand(D, 8, device="cuda"), e(B, T, 1, 8), e(B, T, 1, 8)
        Ds, bias, h0 = e(D, t=torch.float32), e(D, t=torch.float32), e(B, D, 8, t=torch.float32)
        out, hT = K.ssm_scan_fwd(x, x.clone(), A, Bm, Cm, Ds, x.clone(), bias, h0)
        gh = torch.randn_like(h0)
        got = K.ssm_scan_bwd(x, x.clone(), A, Bm, Cm, Ds, x.clone(), bias, h0, e(B, T, D), gh)
        if T == 0:
            assert torch.equal(sT, s0) and torch.equal(ds, g) and torch.equal(hT, h0) and torch.equal(got[8], gh)
        if B == 0 or T == 0:
            assert (dw == 0).all() and (db == 0).all() and all((got[i] == 0).all() for i in (2, 5, 7))
        if D > 0:
            _, n = K.block_norm_fwd(x)
            assert n.shape == x.shape


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_ssm_state_behind_a_cut_tile(K, N):
    """An infinite decay rate forgets everything at every token, and only there: the last state is the
    last token's input whatever the sequence's length is to the tiles, forward and from gradients."""
    g = _gen(N)
    for T in (1, 5, 17, 33, 70):
        u, dt = _n(g, 1, T, 40), _n(g, 1, T, 40)
        Bm, Cm = _n(g, 1, T, 1, N), _n(g, 1, T, 1, N)
        for A in (torch.full((40, N), -float("inf"), device="cuda"), torch.full((40, N), -3.4e38, device="cuda")):
            h0 = _n(g, 1, 40, N)
            out, hT = K.ssm_scan_fwd(u, dt, A, Bm, Cm, h0=h0)
            d = torch.nn.functional.softplus(R.d(dt), threshold=100)
            ref = (d * R.d(u))[..., None] * R.d(Bm)
            R.check("h_T", hT, ref[:, -1], ref[:, -1].abs(), 48)
            h = torch.empty_like(h0)
            K.ssm_step(u[:, -1], dt[:, -1], A, Bm[:, -1], Cm[:, -1], None, None, None, h0, h_out=h)
            R.check("step", h, ref[:, -1], ref[:, -1].abs(), 48)
            dout = _n(g, 1, T, 40)
            got = K.ssm_scan_bwd(u, dt, A, Bm, Cm, None, None, None, h0, dout, torch.zeros_like(h0))
            dC = (R.d(dout)[..., None] * ref).sum(2, keepdim=True).squeeze(2)[:, :, None]
            far = (R.d(dout)[..., None] * ref).abs().sum(2)[:, :, None]
            R.check("dC", got[4], dC, far, 48 + 40)
            assert (got[8] == 0).all()


def test_ssm_extreme_steps(K):
    """delta of 0 keeps the state, a large delta forgets it; gates far out shut or pass."""
    B, T, D, N = 1, 70, 32, 16
    args, _, _, _ = _ssm_inputs(_dense(B, T), D, N, 1, True, True, True, True, 0, torch.float32)
    u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
    out, hT = K.ssm_scan_fwd(u, torch.full_like(dt, -1e30), A, Bm, Cm, Ds, z, bias, h0)
    assert torch.equal(hT, h0)
    out, hT = K.ssm_scan_fwd(u, torch.full_like(dt, 1e4), A, Bm, Cm, None, None, None, h0)
    last = (1e4 * R.d(u)[:, -1])[..., None] * R.d(Bm)[:, -1]
    R.check("h_T", hT, last, last.abs(), 8)
    out, _ = K.ssm_scan_fwd(u, dt, A, Bm, Cm, Ds, torch.full_like(z, -1e30), bias, h0)
    assert (out == 0).all()
    got = K.ssm_scan_bwd(u, torch.full_like(dt, -1e30), A, Bm, Cm, Ds, torch.full_like(z, -1e30), bias, h0,
                         torch.ones_like(u), torch.ones_like(h0))
    assert all(torch.isfinite(o).all() for o in got) and torch.equal(got[8], torch.ones_like(h0))


def test_activations_far_out(K):
    """SiLU and softplus in FP32, each by itself (a tap of 1; no decay, inputs of 1), relative to the value.

    12 + 1.23 |x| half-steps: log2(e) x is rounded (1) with log2(e) itself (0.22), which e^x sees |x| times; the
    hardware's exponential is off by at most 2^-22 (4) and its reciprocal by 2^-23 (2); a sum, a product, and for
    softplus the polynomial (2^-27 and 2 roundings), the quotient's product and the last sum make 12 in all.
    """
    D, n = 1024, 1 << 20
    x = torch.linspace(-87, 87, n, dtype=R.F64).float()
    X = R.d(x)
    tol = (12 + 1.23 * X.clamp(max=0).abs()) * R.U
    w = torch.tensor([[0.0, 1.0]]).repeat(D, 1).cuda()
    y, _ = K.short_conv_fwd(x.view(1, -1, D).cuda(), w)
    assert ((R.d(y).view(-1) - R.silu(X)).abs() <= tol * R.silu(X).abs()).all()
    one, B = torch.ones(n // D, 1, D, device="cuda"), torch.ones(n // D, 1, 1, 8, device="cuda")
    _, h = K.ssm_scan_fwd(one, x.view(-1, 1, D).cuda(), torch.zeros(D, 8, device="cuda"), B, B)
    ref = torch.log1p(torch.exp(-X.abs())) + X.clamp(min=0)
    assert ((R.d(h) - ref.view(-1, D, 1)).abs() <= (tol * ref).view(-1, D, 1)).all()


# ------------------------------------------------------------------ block norm
NORM = [
    # rows, D, block, gate, weights, wide
    ((1,), 1, True, True, True, 0),
    ((5,), 64, True, True, True, 0),
    ((2, 3), 1000, True, False, True, 8),
    ((7,), 37, True, True, False, 0),
    ((3,), 2051, True, True, True, 0),
    ((3,), 4100, True, True, True, 4),
    ((2,), 8192, True, False, True, 0),
    ((2,), 8200, True, True, True, 0),
    ((2,), 16384, True, True, True, 0),
    ((2,), 16383, True, True, True, 0),
    ((700,), 72, True, True, True, 0),
    ((150,), 1000, True, True, True, 0),
    ((150,), 1500, True, False, True, 4),
    ((149,), 2056, True, True, False, 0),
    ((149,), 3001, True, True, True, 0),
    ((149,), 8184, True, True, True, 0),
    ((149,), 8001, False, False, True, 0),
    ((1300,), 1032, True, True, True, 0),
    ((4000,), 40, True, True, True, 0),
    ((4,), 256, False, False, True, 0),
    ((200,), 1002, True, True, True, 0),
    ((200,), 4100, True, True, True, 0),
    ((160,), 5001, True, True, True, 0),
    ((160,), 6002, True, False, False, 0),
    ((160,), 8200, False, False, True, 0),
    ((301,), 11002, True, True, True, 0),
    ((0,), 256, True, True, True, 0),
] if torch.cuda.is_available() else []


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", range(len(NORM)))
def test_block_norm_forward_and_backward(K, case, dtype):
    lead, D, has_block, has_gate, weights, wide = NORM[case]
    g = _gen(case)
    row = lambda t: _wide(t, wide) if wide else t  # noqa: E731
    r = row(_n(g, *lead, D, dtype=dtype, std=3.0))
    b = row(_n(g, *lead, D, dtype=dtype, std=0.5)) if has_block else None
    gate = row(_n(g, *lead, D, dtype=dtype)) if has_gate else None
    s, wp, wx = (_u(g, 0.3, 1.5, D) if weights else None for _ in range(3))
    if not has_block:
        s = wp = None
    eps = 1e-5
    res, x = K.block_norm_fwd(r, b, gate, s, wp, wx, eps=eps)
    ref = [_flat(r), _flat(b), _flat(gate), R.d(s), R.d(wp), R.d(wx)]
    rr, rx = R.norm_fwd(*ref, eps)
    far = ref[0].abs() + (rr - ref[0]).abs()
    n = 16 + 10 + 48   # a thread's values, the levels of the block's sum, the activations
    if has_block:
        R.check("res_out", res.reshape(-1, D), rr, far, n)
    else:
        assert res is None
    scale = (rx / rr).abs().nan_to_num()
    R.check("x", x.reshape(-1, D), rx, far * scale + rx.abs(), n)
    if has_block:   # either output alone, and in place
        only, none = K.block_norm_fwd(r, b, gate, s, wp, wx, eps=eps, want_x=False)
        assert none is None and torch.equal(only, res)
        own = r.clone(memory_format=torch.contiguous_format)
        x2 = torch.empty_like(x)
        K.kda_block_norm_fwd(own, b, gate, s, wp, wx, own, x2, eps=eps)
        assert torch.equal(own, res) and torch.equal(x2, x)

    stored = row(res) if has_block else r
    for use in ((1, 1), (1, 0), (0, 1)):
        dres = _n(g, *lead, D, dtype=dtype) if use[0] else None
        dx = _n(g, *lead, D, dtype=dtype) if use[1] else None
        got = K.block_norm_bwd(stored, b, gate, s, wp, wx, dres, dx, eps=eps)
        args = (_flat(stored), *ref[1:], _flat(dres), _flat(dx), eps)
        want, mag = R.norm_bwd(*args), R.norm_bwd(*args, mag=True)
        rows = max(1, ref[0].shape[0])
        for name, o, w, f, p in zip(("dresidual", "dblock", "dgate", "dscale", "dw_post", "dw_pre"), got, want, mag,
                                    (True, has_block, has_gate, s is not None, wp is not None, wx is not None)):
            if not p:
                assert o is None
                continue
            R.check(name, o.reshape(w.shape), w, f, 2 * n + (rows if o.dim() == 1 else 0))
    if has_block:   # dres may be the buffer of dresidual
        own = _n(g, *lead, D, dtype=dtype)
        dx = _n(g, *lead, D, dtype=dtype)
        want = K.block_norm_bwd(stored, b, gate, s, wp, wx, own, dx, eps=eps)
        e = lambda t: None if t is None else torch.empty(t.shape, dtype=dtype, device="cuda")  # noqa: E731
        ws = torch.empty(max(16, K.kda_block_norm_bwd_workspace_bytes(stored)), dtype=torch.uint8, device="cuda")
        db, dg = e(b), e(gate)
        K.kda_block_norm_bwd(stored, b, gate, s, wp, wx, own, dx, own, db, dg, None, None, None, ws, eps=eps)
        assert torch.equal(own, want[0]) and torch.equal(db, want[1])


def test_block_norm_of_zero_rows(K):
    """A row of zeros: eps alone stands under the root; with eps = 0 the row of the formula is NaN and no other."""
    r = torch.zeros(3, 64, device="cuda")
    r[1] = 1.0
    _, x = K.block_norm_fwd(r, eps=1e-5)
    assert (x[0] == 0).all() and (x[2] == 0).all() and torch.isfinite(x).all()
    _, x = K.block_norm_fwd(r, eps=0.0)
    assert x[0].isnan().all() and torch.isfinite(x[1]).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_ssm_order_of_sequences(K, N, dtype):
    """Long sequences start first; each has the values that it has alone, equal lengths and empty ones too."""
    D = 40
    for lens in ([300, 0, 700, 128, 300, 1], [10] + 31 * [140], [0, 0, 900]):
        cuts = [7]
        for n in lens:
            cuts.append(cuts[-1] + n)
        args, cu, bounds, _ = _ssm_inputs(_packed(cuts, cuts[-1] + 4), D, N, 2, True, True, True, True, 0, dtype)
        u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
        out, hT = K.ssm_scan_fwd(*args, cu_seqlens=cu)
        assert (out[:7] == 0).all() and (out[-4:] == 0).all()
        ro, rh = _ssm_ref(args, bounds)
        fo, fh = _ssm_ref(args, bounds, mag=True)
        R.check("out", out[7:-4], ro[7:-4], fo[7:-4], 24 * max(lens) + N + 64)
        R.check("h_T", hT, rh, fh, 24 * max(lens) + 64)


def test_bounds_outside_the_rows_are_cut_off(K):
    for D, T in ((24, 100), (8, 1500)):   # whole sequences, spans of time
        at = _packed([0, 3, 70, T], T)
        x, w, b, s0, cu, _, g = _conv_inputs(at, D, 4, True, True, torch.float32, 0)
        a, _, _, _ = _ssm_inputs(at, D, 8, 1, True, True, True, True, 0, torch.float32)
        dy, dsT, dh = _n(g, T, D), _n(g, 3, 3, D), _n(g, 3, D, 8)
        run = lambda cu: (*K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu),  # noqa: E731
                          *K.short_conv_bwd(x, w, b, s0, dy, dsT, cu_seqlens=cu),
                          *K.ssm_scan_fwd(*a, cu_seqlens=cu), *K.ssm_scan_bwd(*a, dy, dh, cu_seqlens=cu))
        far = torch.tensor([-5, 3, 70, T + 1000], dtype=torch.int32, device="cuda")
        assert all(torch.equal(p, q) for p, q in zip(run(far), run(cu)))


# ------------------------------------------------------------------ rows at any element
def _off(t, tail=1):
    """The same rows one element into rows that are an odd number of elements longer."""
    row = t.shape[-tail:].numel()
    w = torch.full(t.shape[:-tail] + (row + 3,), NAN, dtype=t.dtype, device=t.device)
    v = w[..., 1:1 + row].unflatten(-1, t.shape[-tail:])
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T", [1, 150])
def test_ssm_rows_at_any_element(K, N, T, dtype):
    """Widths of whole vectors in rows that start at none: each tensor alone, and all; the same bits as aligned rows."""
    D, G = 256, 2
    args, _, _, g = _ssm_inputs(_dense(2, T), D, N, G, True, True, True, True, 0, dtype)
    u, dt, A, Bm, Cm, Ds, z, bias, h0 = args
    dout, dhT = _n(g, 2, T, D, dtype=dtype), _n(g, 2, D, N)
    rows = dict(u=(u, 1), dt=(dt, 1), Bm=(Bm, 2), Cm=(Cm, 2), z=(z, 1), dout=(dout, 1))

    def run(off):
        r = {k: _off(t, n) if k in off else t.contiguous() for k, (t, n) in rows.items()}
        a = (r["u"], r["dt"], A, r["Bm"], r["Cm"], Ds, r["z"], bias)
        step = tuple(t[:, 0] if t is not None and t.dim() > 2 else t for t in a)
        h = h0.clone()
        o = _off(u) if "u" in off else torch.empty_like(u)
        out, hT = K.ssm_scan_fwd(*a, h0, out=o)
        return (out, hT, *K.ssm_scan_bwd(*a, h0, r["dout"], dhT), K.ssm_step(*step, h), h)

    want = run(())
    for off in [(k,) for k in rows] + [("Bm", "Cm"), tuple(rows)]:
        for i, (a, b) in enumerate(zip(run(off), want)):
            assert torch.equal(a, b), (off, i)


@pytest.mark.parametrize("dtype", DT)
def test_conv_rows_at_any_element(K, dtype):
    x, w, b, s0, _, _, g = _conv_inputs(_dense(2, 70), 64, 4, True, True, dtype, 0)
    dy, dsT = _n(g, *x.shape, dtype=dtype), _n(g, 2, 3, 64)

    def run(x, dy, y):
        st = s0.clone()
        y, sT = K.short_conv_fwd(x, w, b, s0, y=y)
        return (y, sT, *K.short_conv_bwd(x, w, b, s0, dy, dsT), K.short_conv_step(x[:, 0], w, b, st), st)

    want = run(x, dy, torch.empty_like(x))
    for a, b_, y in ((_off(x), dy, torch.empty_like(x)), (x, _off(dy), torch.empty_like(x)), (x, dy, _off(x)),
                     (_off(x), _off(dy), _off(x))):
        for i, (o, r) in enumerate(zip(run(a, b_, y), want)):
            assert torch.equal(o, r), i


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 2048, 4096])
def test_norm_rows_at_any_element(K, D, dtype):
    """Each row tensor alone, and all: against the 64-bit form (the order of a row's sum depends on the vectors)."""
    g = _gen(D)
    r, b, gate, dres, dx = (_n(g, 5, D, dtype=dtype) for _ in range(5))
    s, wp, wx = (_u(g, 0.3, 1.5, D) for _ in range(3))
    n, eps = 16 + 10 + 48, 1e-5
    ref = (R.d(r), R.d(b), R.d(gate), R.d(s), R.d(wp), R.d(wx))
    rr, rx = R.norm_fwd(*ref, eps)
    far = ref[0].abs() + (rr - ref[0]).abs()
    args = (*ref, R.d(dres), R.d(dx), eps)   # r stands for the stored sum here
    want, mag = R.norm_bwd(*args), R.norm_bwd(*args, mag=True)
    for off in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        t = [_off(v) if o else v for v, o in zip((r, b, gate), off)]
        res, x = K.block_norm_fwd(*t, s, wp, wx, eps=eps)
        R.check("res_out", res, rr, far, n)
        R.check("x", x, rx, far * (rx / rr).abs().nan_to_num() + rx.abs(), n)
        for name, o, w, f in zip(("dresidual", "dblock", "dgate", "dscale", "dw_post", "dw_pre"),
                                 K.block_norm_bwd(*t, s, wp, wx, dres, dx, eps=eps), want, mag):
            R.check(name, o, w, f, 2 * n + (5 if o.dim() == 1 else 0))


# ------------------------------------------------------------------ how they are called
def _calls(K, seed=0, dtype=torch.bfloat16):
    """One call of each operator, as (name, function of nothing, outputs)."""
    lay = _packed([0, 100, 100, 350], 350)
    x, w, b, s0, cu, _, g = _conv_inputs(lay, 72, 4, True, True, dtype, 0, seed)
    dy = _n(g, 350, 72, dtype=dtype)
    a, _, _, _ = _ssm_inputs(lay, 72, 16, 1, True, True, True, True, 0, dtype, seed)
    dh = _n(g, 3, 72, 16)
    r, blk, gate = (_n(g, 350, 72, dtype=dtype) for _ in range(3))
    ws = [_u(g, 0.3, 1.5, 72) for _ in range(3)]
    st, so = _n(g, 350, 3, 72, dtype=dtype), torch.empty(350, 3, 72, dtype=dtype, device="cuda")
    h, ho = _n(g, 350, 72, 16), torch.empty(350, 72, 16, device="cuda")
    return [
        lambda kw: K.short_conv_fwd(x, w, b, s0, cu_seqlens=cu, **kw),
        lambda kw: K.short_conv_bwd(x, w, b, s0, dy, None, cu_seqlens=cu, **kw),
        lambda kw: (K.short_conv_step(x, w, b, st, state_out=so, **kw), so),
        lambda kw: K.ssm_scan_fwd(*a, cu_seqlens=cu, **kw),
        lambda kw: K.ssm_scan_bwd(*a, dy, dh, cu_seqlens=cu, **kw),
        lambda kw: (K.ssm_step(*a[:8], h, h_out=ho, **kw), ho),
        lambda kw: K.block_norm_fwd(r, blk, gate, *ws, **kw),
        lambda kw: K.block_norm_bwd(r, blk, gate, *ws, dy, dy, **kw),
    ]


def test_same_bits_every_time_and_on_another_stream(K):
    for call in _calls(K):
        one = [t.clone() for t in call({}) if t is not None]
        two = [t.clone() for t in call({}) if t is not None]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        three = call({"stream": side})
        side.synchronize()
        for p, q, r in zip(one, two, [t for t in three if t is not None]):
            assert torch.equal(p, q) and torch.equal(p, r)


def test_two_streams_at_once(K):
    """Calls on two streams share nothing: each has its workspace."""
    a, b = _calls(K, 1), _calls(K, 2)
    want = [[t.clone() for t in c({}) if t is not None] for c in a + b]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for p, q in zip(a, b):
        got.append((p({"stream": s1}), q({"stream": s2})))
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(got):
        for o, w in ((p, want[i]), (q, want[len(a) + i])):
            assert all(torch.equal(x, y) for x, y in zip([t for t in o if t is not None], w))


def test_captured_and_replayed(K):
    for call in _calls(K, 3):
        want = [t.clone() for t in call({}) if t is not None]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call({})
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [t for t in call({}) if t is not None]
        for t in out:
            t.fill_(0)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_offsets_beyond_31_bits(K):
    """Rows 70,000 values apart: the last of 40,000 lie behind 2^31 values."""
    rows, D, N = 40000, 8, 16
    wide = torch.empty(1, rows, 70000, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    wide[..., 69000:69000 + 4 * D] = n(1, rows, 4 * D)
    wide[..., 69500:69500 + 2 * N] = n(1, rows, 2 * N)
    x = wide[..., 69000:69000 + D]
    w, b = n(D, 4), n(D)
    y, sT = K.short_conv_fwd(x, w, b)
    y2, sT2 = K.short_conv_fwd(x.contiguous(), w, b)
    assert torch.equal(y, y2) and torch.equal(sT, sT2)
    u, dt, z = (wide[..., 69000 + i * D:69000 + (i + 1) * D] for i in range(3))
    Bm, Cm = (wide[..., 69500 + i * N:69500 + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    A = -torch.rand(D, N, generator=g, device="cuda") - 0.1
    o, h = K.ssm_scan_fwd(u, dt, A, Bm, Cm, None, z)
    o2, h2 = K.ssm_scan_fwd(*(t.contiguous() for t in (u, dt)), A, Bm.contiguous(), Cm.contiguous(), None, z.contiguous())
    assert torch.equal(o, o2) and torch.equal(h, h2)
    r, p = K.block_norm_fwd(x, u, z)
    r2, p2 = K.block_norm_fwd(x.contiguous(), u.contiguous(), z.contiguous())
    assert torch.equal(r, r2) and torch.equal(p, p2)


@pytest.mark.parametrize("dtype", DT)
def test_norm_backward_from_two_threads(K, dtype, monkeypatch):
    """Two widths of one kernel, from two host threads through the C interface, which the interpreter's lock does
    not order: neither thread may change what the other's launch was given."""
    runs, jobs = 30000, []
    for D in (8200, 16384):
        g = _gen(D)
        r, b, gate, dres, dx = (_n(g, 4, D, dtype=dtype) for _ in range(5))
        s, wp, wx = (_u(g, 0.3, 1.5, D) for _ in range(3))
        outs = [torch.empty_like(r) for _ in range(3)] + [torch.empty_like(s) for _ in range(3)]
        ws = torch.empty(K.kda_block_norm_bwd_workspace_bytes(r), dtype=torch.uint8, device="cuda")
        tensors = (r, b, gate, s, wp, wx, dres, dx, *outs, ws)
        want = K.block_norm_bwd(*tensors[:8])
        made = []
        with monkeypatch.context() as m:
            m.setattr(K.layers, "_launch", lambda fn, call, args, dims, opts, stream: made.append((fn, args, dims, opts)))
            K.kda_block_norm_bwd(*tensors)
        jobs.append((made[0], outs, want, torch.cuda.Stream(), tensors))
    torch.cuda.synchronize()
    ready, statuses = threading.Barrier(2), []

    def work(call, stream):
        fn, args, dims, opts = call
        handle = stream.cuda_stream
        ready.wait()
        statuses.append({fn(*args, dims, opts, handle) for _ in range(runs)})

    threads = [threading.Thread(target=work, args=(j[0], j[3])) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{0}, {0}]
    for _, outs, want, _, _ in jobs:
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_offsets_beyond_31_bits_backward_and_steps(K):
    """The same layout for the gradients and the single tokens, outputs with row strides among them; equal bits."""
    rows, D, N = 40000, 8, 16
    wide = torch.empty(1, rows, 70000, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    wide[..., 69000:69000 + 6 * D] = n(1, rows, 6 * D)
    wide[..., 69500:69500 + 2 * N] = n(1, rows, 2 * N)
    u, dt, z, dout, out, out2 = (wide[..., 69000 + i * D:69000 + (i + 1) * D] for i in range(6))
    Bm, Cm = (wide[..., 69500 + i * N:69500 + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    c = lambda *t: [v.contiguous() for v in t]  # noqa: E731
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)  # noqa: E731
    w, b = n(D, 4), n(D)
    dw, db = torch.empty(D, 4, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(K.kda_short_conv_bwd_workspace_bytes(u, w), dtype=torch.uint8, device="cuda")
    K.kda_short_conv_bwd(u, w, b, None, dout, None, out, dw, db, None, ws)
    assert same((out, dw, db), K.short_conv_bwd(*c(u), w, b, None, *c(dout)))
    K.kda_short_conv_fwd(u, w, b, None, out2, None)
    assert torch.equal(out2, K.short_conv_fwd(*c(u), w, b)[0])
    A = -torch.rand(D, N, generator=g, device="cuda") - 0.1
    K.ssm_scan_fwd(u, dt, A, Bm, Cm, None, z, out=out)
    assert torch.equal(out, K.ssm_scan_fwd(*c(u, dt), A, *c(Bm, Cm), None, *c(z))[0])
    assert same(K.ssm_scan_bwd(u, dt, A, Bm, Cm, None, z, None, None, dout),
                K.ssm_scan_bwd(*c(u, dt), A, *c(Bm, Cm), None, *c(z), None, None, *c(dout)))
    dres, dx = n(1, rows, D), n(1, rows, D)
    assert same(K.block_norm_bwd(u, dt, z, None, None, None, dres, dx),
                K.block_norm_bwd(*c(u, dt, z), None, None, None, dres, dx))
    # every row a sequence
    st = n(rows, 3, D)
    st2 = st.clone()
    K.short_conv_step(u[0], w, b, st, y=out[0])
    assert torch.equal(K.short_conv_step(u[0].contiguous(), w, b, st2), out[0]) and torch.equal(st, st2)
    h = n(rows, D, N, dtype=torch.float32)
    h2 = h.clone()
    K.ssm_step(u[0], dt[0], A, Bm[0], Cm[0], None, z[0], None, h, out=out[0])
    assert torch.equal(K.ssm_step(*c(u[0], dt[0]), A, *c(Bm[0], Cm[0]), None, *c(z[0]), None, h2), out[0])
    assert torch.equal(h, h2)


@pytest.fixture
def memory_back():
    """Leaves the device's memory to others again."""
    yield
    torch.cuda.empty_cache()


def test_tensors_of_more_than_31_bits(K, memory_back):
    """Contiguous tensors of more than 2^31 values, with the workspaces that they need: a short sequence behind a
    long one, and the last rows of the norm, against their 64-bit forms."""
    D, N, long, T = 2048, 32, (1 << 20) + 7, 70
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("about 70 GB of device memory")
    rows = long + T
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    cu = torch.tensor([0, long, rows], dtype=torch.int32, device="cuda")
    last, bounds = slice(long, rows), [(0, T)]
    u, dout = n(rows, D), n(rows, D)
    # the norm: its rows are independent
    s, wp, wx = (torch.rand(D, generator=g, device="cuda") + 0.3 for _ in range(3))
    res, x = K.block_norm_fwd(u, dout, None, s, wp, wx)
    ref = (R.d(u[last]), R.d(dout[last]), None, R.d(s), R.d(wp), R.d(wx))
    rr, rx = R.norm_fwd(*ref, 1e-5)
    far = ref[0].abs() + (rr - ref[0]).abs()
    R.check("res_out", res[last], rr, far, 74)
    R.check("x", x[last], rx, far * (rx / rr).abs().nan_to_num() + rx.abs(), 74)
    got = K.block_norm_bwd(res, dout, None, s, wp, wx, x, None)
    args = (R.d(res[last]), ref[1], None, *ref[3:], R.d(x[last]), None, 1e-5)
    for name, o, r, f in zip(("dresidual", "dblock"), got, R.norm_bwd(*args), R.norm_bwd(*args, mag=True)):
        R.check(name, o[last], r, f, 2 * 74)
    del res, x, got
    # the convolution
    w, b, s0 = n(D, 4), n(D), n(2, 3, D)
    y, sT = K.short_conv_fwd(u, w, b, s0, cu_seqlens=cu)
    ref = (R.d(u[last]), R.d(w), R.d(b), R.d(s0[1:]))
    pre, rsT = R.conv_pre(*ref, bounds)
    far, _ = R.conv_pre(*ref, bounds, mag=True)
    R.check("y", y[last], R.silu(pre), 1.1 * far + R.silu(pre).abs(), 4 + 48)
    assert torch.equal(R.d(sT[1:]), rsT)
    del y
    dsT = n(2, 3, D, dtype=torch.float32)
    got = K.short_conv_bwd(u, w, b, s0, dout, dsT, cu_seqlens=cu)
    args = (*ref, R.d(dout[last]), R.d(dsT[1:]), bounds)
    want, mag = R.conv_bwd(*args), R.conv_bwd(*args, mag=True)
    R.check("dx", got[0][last], want[0], mag[0], 4 + 48)
    R.check("dstate0", got[3][1:], want[3], mag[3], 4 + 48)
    del got
    # the scan
    dt, z = n(rows, D), n(rows, D)
    Bm, Cm = n(rows, 1, N), n(rows, 1, N)
    A = -(torch.rand(D, N, generator=g, device="cuda") + 0.05)
    Ds, bias = n(D, dtype=torch.float32), torch.rand(D, generator=g, device="cuda") * 4 - 5
    h0, dhT = n(2, D, N, dtype=torch.float32), n(2, D, N, dtype=torch.float32)
    out, hT = K.ssm_scan_fwd(u, dt, A, Bm, Cm, Ds, z, bias, h0, cu_seqlens=cu)
    cut = (u[last], dt[last], A, Bm[last], Cm[last], Ds, z[last], bias, h0[1:])
    (ro, rh), (fo, fh) = _ssm_ref(cut, bounds), _ssm_ref(cut, bounds, mag=True)
    R.check("out", out[last], ro, fo, 24 * T + N + 64)
    R.check("h_T", hT[1:], rh, fh, 24 * T + 64)
    del out
    got = K.ssm_scan_bwd(u, dt, A, Bm, Cm, Ds, z, bias, h0, dout, dhT, cu_seqlens=cu)
    more = (R.d(dout[last]), R.d(dhT[1:]))
    ref, far = _ssm_ref(cut, bounds, *more), _ssm_ref(cut, bounds, *more, mag=True)
    for i, name in ((0, "du"), (1, "ddt"), (3, "dB"), (4, "dC"), (6, "dz")):
        R.check(name, got[i][last], ref[i], far[i], 48 * T + N + D + 128)
    R.check("dh0", got[8][1:], ref[8], far[8], 48 * T + N + D + 128)


# ------------------------------------------------------------------ a run of them together
def _layer_weights(g, dm, D, N, Rk):
    s = lambda *shape: torch.randn(*shape, generator=g, dtype=R.F64) / shape[0] ** 0.5  # noqa: E731
    f = lambda t: t.float().cuda()  # noqa: E731
    W = {"in": s(dm, 2 * D), "x": s(D, Rk + 2 * N), "dt": s(Rk, D), "out": s(D, dm)}
    W = {k: f(v) for k, v in W.items()}
    W["conv"], W["cb"] = f(torch.rand(D, 4, generator=g) - 0.5), f(torch.randn(D, generator=g) * 0.1)
    W["A"] = f(-(torch.rand(D, N, generator=g) + 0.5) * torch.arange(1, N + 1))
    W["D"], W["bias"] = f(torch.rand(D, generator=g) + 0.5), f(torch.rand(D, generator=g) * 3 - 5)
    W["scale"], W["post"], W["pre"] = (f(torch.rand(dm, generator=g) + 0.5) for _ in range(3))
    return W


def _layer(K, W, res, x, N, Rk, conv_state, h):
    """One layer on a prompt: (residual, next input, what the backward needs, states)."""
    D = W["D"].shape[0]
    uz = x @ W["in"]
    u0, z = uz[..., :D], uz[..., D:]
    u, conv_state = K.short_conv_fwd(u0, W["conv"], W["cb"], conv_state)
    p = u @ W["x"]
    dt = p[..., :Rk] @ W["dt"]
    Bm, Cm = (p[..., Rk + i * N:Rk + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    y, h = K.ssm_scan_fwd(u, dt, W["A"], Bm, Cm, W["D"], z, W["bias"], h)
    blk = y @ W["out"]
    res, nxt = K.block_norm_fwd(res, blk, None, W["scale"], W["post"], W["pre"])
    return res, nxt, (uz, u, p, dt, y, blk), conv_state, h


def test_layer_prompt_then_tokens(K):
    """A prompt in one call, and the same rows as a prompt and single tokens, give one result."""
    g = _gen(5)
    B, T, dm, D, N, Rk = 2, 40, 32, 64, 16, 8
    W = _layer_weights(g, dm, D, N, Rk)
    xs = torch.randn(B, T, dm, generator=g).cuda()
    _, x0 = K.block_norm_fwd(xs)
    res, nxt, _, cs, h = _layer(K, W, xs, x0, N, Rk, None, None)
    T0 = 33
    _, _, _, cs1, h1 = _layer(K, W, xs[:, :T0].contiguous(), x0[:, :T0].contiguous(), N, Rk, None, None)
    for t in range(T0, T):
        uz = x0[:, t] @ W["in"]
        u = K.short_conv_step(uz[:, :D], W["conv"], W["cb"], cs1)
        p = u @ W["x"]
        y = K.ssm_step(u, p[:, :Rk] @ W["dt"], W["A"], p[:, Rk:Rk + N].unflatten(-1, (1, N)),
                       p[:, Rk + N:].unflatten(-1, (1, N)), W["D"], uz[:, D:], W["bias"], h1)
        r, n = K.block_norm_fwd(xs[:, t], y @ W["out"], None, W["scale"], W["post"], W["pre"])
        # FP32 throughout; the matrix products' sums are ordered otherwise for one row: 200 terms
        # of products on the path, 2^-24 of values of order 10 each
        assert (r - res[:, t]).abs().max() <= 200 * 2 ** -24 * 10
        assert (n - nxt[:, t]).abs().max() <= 200 * 2 ** -24 * 10
    assert (h1 - h).abs().max() <= 200 * 2 ** -24 * 10 and torch.allclose(cs1, cs, rtol=1e-5, atol=1e-5)


def test_layer_gradients(K):
    """Forward and backward of a layer out of these operators against autograd of the plain layer in 64 bits."""
    g = _gen(6)
    B, T, dm, D, N, Rk = 2, 21, 16, 32, 8, 4
    W = _layer_weights(g, dm, D, N, Rk)
    xs = torch.randn(B, T, dm, generator=g).cuda()
    dres, dnxt = (torch.randn(B, T, dm, generator=g).cuda() for _ in range(2))
    _, x0 = K.block_norm_fwd(xs)
    res, nxt, (uz, u, p, dt, y, blk), _, _ = _layer(K, W, xs, x0, N, Rk, None, None)
    grad = {}
    dr, dblk, _, grad["scale"], grad["post"], grad["pre"] = K.block_norm_bwd(res, blk, None, W["scale"], W["post"],
                                                                             W["pre"], dres, dnxt)
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    grad["out"] = flat(y).T @ flat(dblk)
    Bm, Cm = (p[..., Rk + i * N:Rk + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    du, ddt, grad["A"], dB, dC, grad["D"], dz, grad["bias"], _ = K.ssm_scan_bwd(
        u, dt, W["A"], Bm, Cm, W["D"], uz[..., D:], W["bias"], None, dblk @ W["out"].T)
    grad["dt"] = flat(p[..., :Rk]).T @ flat(ddt)
    dp = torch.cat([ddt @ W["dt"].T, dB.flatten(-2), dC.flatten(-2)], -1)
    grad["x"] = flat(u).T @ flat(dp)
    du0, grad["conv"], grad["cb"], _ = K.short_conv_bwd(uz[..., :D], W["conv"], W["cb"], None, du + dp @ W["x"].T)
    duz = torch.cat([du0, dz], -1)
    grad["in"] = flat(x0).T @ flat(duz)
    dx = K.block_norm_bwd(xs, None, None, None, None, None, dr, duz @ W["in"].T)[0]

    L = {k: R.d(v).requires_grad_() for k, v in W.items()}
    X = R.d(xs).requires_grad_()
    bounds = _dense(B, T)[2]
    n0 = R.rms(X, 1e-5)
    UZ = (n0 @ L["in"]).reshape(-1, 2 * D)
    zero = torch.zeros(3, D, dtype=R.F64)
    pre = torch.cat([sum(torch.cat([zero, UZ[lo:hi, :D]])[j:j + hi - lo] * L["conv"][:, j] for j in range(4)) for lo, hi in bounds])
    Uc = R.silu(pre + L["cb"])
    P = Uc @ L["x"]
    delta = torch.nn.functional.softplus(P[:, :Rk] @ L["dt"] + L["bias"], threshold=100)
    ys = []
    for lo, hi in bounds:
        h = torch.zeros(D, N, dtype=R.F64)
        for t in range(lo, hi):
            h = torch.exp(delta[t][:, None] * L["A"]) * h + (delta[t] * Uc[t])[:, None] * P[t, Rk:Rk + N]
            ys.append((h * P[t, Rk + N:]).sum(-1) + L["D"] * Uc[t])
    Y = torch.stack(ys) * R.silu(UZ[:, D:])
    out, fin = R.norm_fwd(X.reshape(-1, dm), Y @ L["out"], None, L["scale"], L["post"], L["pre"], 1e-5)
    ((out * flat(R.d(dres))).sum() + (fin * flat(R.d(dnxt))).sum()).backward()
    # FP32 values through about ten operators, sums of up to 100 terms each: some 10^3 half-steps of
    # the largest value
    for name, got, want in [("dx", dx, X.grad)] + [(k, grad[k], L[k].grad) for k in grad]:
        err = (R.d(got).reshape(want.shape) - want).abs().max()
        assert err <= 1000 * R.U * max(1.0, float(want.abs().max())), (name, float(err), float(want.abs().max()))


def test_delta_rule_layer_gradients(K):
    """The convolutions ahead of the delta rule and the norm behind it, forward and backward in FP32 (the rule's
    gradients are FP32: FP32 calls take them as they are), against autograd of the plain layer in 64 bits."""
    g = torch.Generator().manual_seed(7)
    B, T, H, d = 2, 33, 2, 64
    D = H * d
    s = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    X = [s(B, T, D) for _ in range(3)]                                # inputs of the three branches
    W = [torch.rand(D, 4, generator=g) - 0.5 for _ in range(3)]
    bias = [s(D) * 0.1 for _ in range(3)]
    decay, beta = -5 * torch.sigmoid(s(B, T, H, d)), torch.sigmoid(s(B, T, H))
    res, scale, post, pre = s(B, T, D), *(torch.rand(D, generator=g) + 0.5 for _ in range(3))
    dres, dnxt = s(B, T, D), s(B, T, D)
    c = lambda v: v.cuda()  # noqa: E731
    heads = lambda v: v.reshape(B, T, H, d)  # noqa: E731

    qkv = [K.short_conv_fwd(c(x), c(w), c(b))[0] for x, w, b in zip(X, W, bias)]
    o, _ = K.chunk_fwd(*(heads(v) for v in qkv), c(decay), c(beta))
    blk = o.reshape(B, T, D)
    out, nxt = K.block_norm_fwd(c(res), blk, None, c(scale), c(post), c(pre))
    dr, dblk, *_ = K.block_norm_bwd(out, blk, None, c(scale), c(post), c(pre), c(dres), c(dnxt))
    dqkv = K.chunk_bwd(*(heads(v) for v in qkv), c(decay), c(beta), None, heads(dblk), want_dS0=False)[:3]
    got = [K.short_conv_bwd(c(x), c(w), c(b), None, v.reshape(B, T, D)) for x, w, b, v in zip(X, W, bias, dqkv)]

    L = [[R.d(v).requires_grad_() for v in group] for group in (X, W, bias)]
    zero = torch.zeros(B, 3, D, dtype=R.F64)
    conv = lambda x, w, b: R.silu(sum(torch.cat([zero, x], 1)[:, j:j + T] * w[:, j] for j in range(4)) + b)  # noqa: E731
    acts = [conv(x, w, b) for x, w, b in zip(*L)]
    for a in acts:
        a.retain_grad()
    unit = lambda v: v / torch.sqrt((v * v).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    q, k, v = (heads(a) for a in acts)
    q, k = unit(q), unit(k)
    S, os = torch.zeros(B, H, d, d, dtype=R.F64), []
    for t in range(T):
        S = torch.exp(R.d(decay[:, t]))[..., None] * S
        err = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)
        S = S + R.d(beta[:, t])[..., None, None] * k[:, t, :, :, None] * err[:, :, None]
        os.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    r0 = R.d(res).requires_grad_()
    fo, fx = R.norm_fwd(r0, torch.stack(os, 1).reshape(B, T, D), None, R.d(scale), R.d(post), R.d(pre), 1e-5)
    ((fo * R.d(dres)).sum() + (fx * R.d(dnxt)).sum()).backward()
    assert (R.d(nxt) - fx.detach()).abs().max() <= 1e-4 * fx.detach().abs().max() * 4   # x / rms(x): |r'| <= 4 rms
    assert (R.d(dr) - r0.grad).abs().max() <= 1e-4 * 4 * r0.grad.abs().max()
    # The delta rule and its gradients are tested to 1e-4 of the largest value; the gradients of its inputs see
    # the forward's and the norm's as well (twice that, with the norm's mean three times), and the convolution
    # passes them on through |silu'| <= 1.1 and four taps of at most 0.5, or sums them over B T rows of inputs
    for i in range(3):
        top = acts[i].grad.abs().max()
        near = 3e-4 * top
        assert (R.d(dqkv[i]).reshape(B, T, D) - acts[i].grad).abs().max() <= near
        assert (R.d(got[i][0]) - L[0][i].grad).abs().max() <= near * 1.1 * 2
        rows = 1.1 * B * T
        assert (R.d(got[i][1]) - L[1][i].grad).abs().max() <= near * rows * X[i].abs().max()
        assert (R.d(got[i][2]) - L[2][i].grad).abs().max() <= near * rows
