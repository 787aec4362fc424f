"""The measured cases of the short convolution, the selective state space scan and the block norm.

A case is one pass through one operator: ``prepare`` makes what a caller has in hand, ``run`` computes the
operator in elementary torch operations, or through the library where ``own`` is true.

Notation (rows are tokens, packed sequence after sequence; s runs over sequences, c over channels):

    short convolution  pre[t] = bias + sum_j w[j] x[t-K+1+j],  y = pre * sigmoid(pre)
    selective scan     d = softplus(dt + dt_bias),  h_t = exp(d A) h_{t-1} + d u B_t,
                       y = sum_n C_t[n] h_t[n] + D u,  out = y z sigmoid(z)
    block norm         r' = r + scale sigmoid(gate) rms(block) w_post,  x' = rms(r') w_pre
"""
import math
import random

import torch

own = False

_EPS = 1e-5


def listed():
    return [
        # the three branches of one prompt at the length sweep's 96 heads x 128 channels
        {"name": "conv_fwd_prompt", "op": "conv_fwd", "seqs": 1, "rows": 8192, "D": 12288, "K": 4, "dtype": "bf16", "packed": False, "state": False},
        # packed prompts that go on from a carried state, an odd channel count, fp32
        {"name": "conv_fwd_packed_f32", "op": "conv_fwd", "seqs": 9, "rows": 3001, "D": 1001, "K": 3, "dtype": "f32", "packed": True, "state": True},
        # a training batch: 16 heads x 128 channels
        {"name": "conv_bwd_train", "op": "conv_bwd", "seqs": 4, "rows": 16384, "D": 2048, "K": 4, "dtype": "bf16", "packed": False, "state": False},
        # a decode batch of 256 sequences at 96 x 128 channels
        {"name": "conv_step_decode", "op": "conv_step", "seqs": 256, "rows": 256, "D": 12288, "K": 4, "dtype": "bf16", "packed": False, "state": True},
        # one long prompt
        {"name": "scan_fwd_prompt", "op": "scan_fwd", "seqs": 1, "rows": 8192, "D": 4096, "N": 16, "G": 1, "dtype": "bf16", "packed": False, "state": False},
        # packed prompts of uneven lengths going on from a state, odd channel count, two groups, fp32
        {"name": "scan_fwd_packed_f32", "op": "scan_fwd", "seqs": 7, "rows": 3001, "D": 1002, "N": 32, "G": 2, "dtype": "f32", "packed": True, "state": True},
        # a training batch
        {"name": "scan_bwd_train", "op": "scan_bwd", "seqs": 2, "rows": 4096, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "packed": False, "state": False},
        # a decode batch: bound by the state's bytes
        {"name": "scan_step_decode", "op": "scan_step", "seqs": 256, "rows": 256, "D": 12288, "N": 16, "G": 1, "dtype": "bf16", "packed": False, "state": True},
        # one user's decode: latency alone
        {"name": "scan_step_single", "op": "scan_step", "seqs": 1, "rows": 1, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "packed": False, "state": True},
        # between two layers of a long prompt or a training batch
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 16384, "D": 2048, "gated": True, "dtype": "bf16"},
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "D": 2048, "gated": True, "dtype": "bf16"},
        # between two layers of a small decode batch, fp32, odd width, no gate
        {"name": "norm_fwd_decode_f32", "op": "norm_fwd", "rows": 8, "D": 4099, "gated": False, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = _log(rng, 64, 12288)
    if rng.random() < 0.6:
        D = -(-D // 8) * 8
    if op.startswith("norm"):
        return {"op": op, "rows": min(_log(rng, 1, 16384), (1 << 25) // D), "D": D, "gated": rng.random() < 0.6, "dtype": dtype}
    c = {"op": op, "seqs": 1, "rows": 1, "D": D, "dtype": dtype, "packed": False, "state": rng.random() < 0.5}
    if op.startswith("conv"):
        c["K"] = rng.choice([2, 3, 4, 4])
    else:
        c["N"] = rng.choice([8, 16, 16, 32, 64])
        c["G"] = rng.choice([g for g in (1, 1, 2, 4) if D % g == 0])
    if op.endswith("step"):
        c["seqs"] = c["rows"] = max(1, min(_log(rng, 1, 256), (1 << 26) // (D * c.get("N", 4))))
        c["state"] = True
        return c
    most = (1 << 25) // D if "K" in c else (1 << (28 if op == "scan_fwd" else 26)) // (D * c["N"])
    rows = max(1, min(_log(rng, 1, 16384), most))
    c["packed"] = rng.random() < 0.5
    seqs = min(rows, _log(rng, 1, 16))
    c["seqs"], c["rows"] = seqs, rows if c["packed"] else rows // seqs * seqs
    return c


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, D, rows = _type(case), case["D"], case["rows"]

    def normal(*shape, dtype=t, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    op = case["op"]
    f = torch.float32
    s = {"op": op}
    if op.startswith("norm"):
        s["residual"], s["block"] = normal(rows, D, std=4.0), normal(rows, D)
        s["gate"] = normal(rows, D) if case["gated"] else None
        s["scale"], s["w_post"], s["w_pre"] = uniform(0.1, 1.0, D), uniform(0.5, 1.5, D), uniform(0.5, 1.5, D)
        if op == "norm_bwd":
            s["dres"], s["dx"] = normal(rows, D), normal(rows, D)
        return s

    S = case["seqs"]
    lead = (rows,) if case["packed"] or op.endswith("step") else (S, rows // S)
    if case["packed"]:  # cuts from the seed; two at one place leave a sequence without tokens
        r = random.Random(seed)
        cuts = [0] + sorted(r.randint(0, rows) for _ in range(S - 1)) + [rows]
        s["cu_seqlens"] = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    else:
        s["cu_seqlens"] = None
    if "K" in case:
        K = case["K"]
        s["x"] = normal(*lead, D)
        s["w"] = uniform(-0.5, 0.5, D, K).to(t)
        s["bias"] = normal(D, std=0.1)
        s["state0"] = normal(S, K - 1, D) if case["state"] else None
        if op == "conv_step":
            s["state_out"] = torch.empty_like(s["state0"])
        if op == "conv_bwd":
            s["dy"] = normal(*lead, D)
            s["dstate_T"] = normal(S, K - 1, D, dtype=f) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    # u and z are halves of one projection, B and C lie side by side in another, as a layer has them
    pad = -(-D // 8) * 8
    uz = normal(*lead, 2 * pad)
    s["u"], s["z"] = uz[..., :D], uz[..., pad:pad + D]
    bc = normal(*lead, 2 * G * N)
    s["Bm"] = bc[..., :G * N].unflatten(-1, (G, N))
    s["Cm"] = bc[..., G * N:].unflatten(-1, (G, N))
    s["dt"] = normal(*lead, D)
    # steps between 0.001 and 0.1 at dt = 0, decay rates around 1 .. N
    step = torch.exp(uniform(math.log(1e-3), math.log(0.1), D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=f) * uniform(0.8, 1.25, D, N))
    s["Dskip"] = uniform(0.5, 1.5, D)
    s["h0"] = normal(S, D, N, dtype=f, std=0.5) if case["state"] else None
    if op == "scan_step":
        s["h_out"] = torch.empty_like(s["h0"])
    if op == "scan_bwd":
        s["dout"] = normal(*lead, D)
        s["dh_T"] = normal(S, D, N, dtype=f) if case["state"] else None
    return s


# ---------------------------------------------------------------- the library
def _run_own(s):
    import gated_delta_rule_73_b200 as K
    op = s["op"]
    if op == "conv_fwd":
        return K.short_conv_fwd(s["x"], s["w"], s["bias"], s["state0"], cu_seqlens=s["cu_seqlens"])
    if op == "conv_bwd":
        return K.short_conv_bwd(s["x"], s["w"], s["bias"], s["state0"], s["dy"], s["dstate_T"], cu_seqlens=s["cu_seqlens"])
    if op == "conv_step":
        return K.short_conv_step(s["x"], s["w"], s["bias"], s["state0"], state_out=s["state_out"]), s["state_out"]
    if op == "scan_fwd":
        return K.ssm_scan_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["z"], s["dt_bias"], s["h0"], cu_seqlens=s["cu_seqlens"])
    if op == "scan_bwd":
        return K.ssm_scan_bwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["z"], s["dt_bias"], s["h0"], s["dout"], s["dh_T"],
                              cu_seqlens=s["cu_seqlens"])
    if op == "scan_step":
        return K.ssm_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["z"], s["dt_bias"], s["h0"], h_out=s["h_out"]), s["h_out"]
    if op == "norm_fwd":
        return K.block_norm_fwd(s["residual"], s["block"], s["gate"], s["scale"], s["w_post"], s["w_pre"], eps=_EPS)
    return K.block_norm_bwd(s["residual"], s["block"], s["gate"], s["scale"], s["w_post"], s["w_pre"], s["dres"], s["dx"], eps=_EPS)


# ------------------------------------------------------------- the plain forms
def _places(s, lead):
    """Of every row: its sequence, its place in it, the sequence's end; and the sequences' bounds."""
    rows = math.prod(lead)
    cu = s["cu_seqlens"]
    if cu is None:
        S, T = (lead[0], lead[1]) if len(lead) == 2 else (lead[0], 1)
        cu = torch.arange(S + 1, device="cuda") * T
    else:
        cu = cu.long()
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, row - cu[seq], cu[seq + 1] - row, cu[:-1], cu[1:]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    p = 1 / (1 + torch.exp(-x))
    return p * (1 + x * (1 - p))


def _down(x, n):
    """Rows moved n places later, zeros ahead of them."""
    out = torch.zeros_like(x)
    out[n:] = x[:x.shape[0] - n]
    return out


def _up(x, n):
    out = torch.zeros_like(x)
    out[:x.shape[0] - n] = x[n:]
    return out


def _taps(x, state0, seq, place, K):
    """The K inputs that each row's output sees, oldest first."""
    got = []
    for n in range(K - 1, -1, -1):
        v = _down(x, n) if n < x.shape[0] else torch.zeros_like(x)
        before = (place < n)[:, None]
        old = state0[seq, (place - n + K - 1).clamp(0, K - 2)] if state0 is not None else 0.0
        got.append(torch.where(before, old, v) if n else v)
    return got


def _conv_state(x, state0, starts, ends, K):
    """The last K-1 inputs of each sequence, the carried ones where it is shorter."""
    place = (ends - starts)[:, None] - (K - 1) + torch.arange(K - 1, device="cuda")
    new = x[(starts[:, None] + place).clamp(0, x.shape[0] - 1)]
    if state0 is None:
        return torch.where((place >= 0)[..., None], new, 0.0)
    carried = state0.gather(1, (place + K - 1).clamp(0, K - 2)[..., None].expand_as(new))
    return torch.where((place >= 0)[..., None], new, carried)


def _conv(s):
    x0, t = s["x"], s["x"].dtype
    lead, D = x0.shape[:-1], x0.shape[-1]
    w, bias, K = s["w"].float(), s["bias"].float(), s["w"].shape[1]
    state0 = None if s["state0"] is None else s["state0"].float()
    x = x0.float().reshape(-1, D)
    seq, place, left, starts, ends = _places(s, lead)
    taps = _taps(x, state0, seq, place, K)
    pre = bias + sum(w[:, j] * taps[j] for j in range(K))
    if s["op"] != "conv_bwd":
        return _silu(pre).to(t).reshape(x0.shape), _conv_state(x, state0, starts, ends, K).to(t)
    dpre = s["dy"].float().reshape(-1, D) * _dsilu(pre)
    dw = torch.stack([(dpre * taps[j]).sum(0) for j in range(K)], 1)
    dx = w[:, K - 1] * dpre
    for n in range(1, min(K, dpre.shape[0])):
        dx = dx + w[:, K - 1 - n] * torch.where((left > n)[:, None], _up(dpre, n), 0.0)
    if s["dstate_T"] is not None:  # the last K-1 inputs are the state that goes on
        at = (K - 1 - left).clamp(0, K - 2)
        dx = dx + torch.where((left <= K - 1)[:, None], s["dstate_T"][seq, at], 0.0)
    dstate0 = None
    if state0 is not None:
        length = (ends - starts)[:, None]
        r = torch.arange(K - 1, device="cuda")
        dstate0 = torch.zeros_like(state0)
        for j in range(K - 1):
            p = (r - j)[None].expand(length.shape[0], -1)  # the row whose output saw state row r through tap j
            seen = (p >= 0) & (p < length)
            dstate0 = dstate0 + torch.where(seen[..., None], w[:, j] * dpre[(starts[:, None] + p).clamp(0, dpre.shape[0] - 1)], 0.0)
        back = r[None] - length  # a state row that is still there at the end
        there = s["dstate_T"].gather(1, back.clamp(0, K - 2)[..., None].expand_as(dstate0))
        dstate0 = dstate0 + torch.where((back >= 0)[..., None], there, 0.0)
    return dx.to(t).reshape(x0.shape), dw, dpre.sum(0), dstate0


def _scan(a, b, shift):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... over the rows, by doubling."""
    n, rows = 1, a.shape[0]
    while n < rows:
        b = b + a * shift(b, n)
        n *= 2
        if n < rows:
            a = a * shift(a, n // 2)
    return b


def _ssm(s):
    u0, t = s["u"], s["u"].dtype
    lead, D = u0.shape[:-1], u0.shape[-1]
    G, N = s["Bm"].shape[-2:]
    flat = lambda v: v.float().reshape(-1, D)  # noqa: E731
    wide = lambda v: v.float().reshape(-1, G, N).repeat_interleave(D // G, 1)  # noqa: E731
    u, z = flat(u0), flat(s["z"])
    raw = flat(s["dt"]) + s["dt_bias"]
    d = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A, h0 = s["A"], s["h0"]
    seq, place, left, starts, ends = _places(s, lead)
    first, last = (place == 0)[:, None, None], (left == 1)[:, None, None]
    a = torch.exp(d[..., None] * A)
    Bw, Cw = wide(s["Bm"]), wide(s["Cm"])
    b = (d * u)[..., None] * Bw
    if h0 is not None:
        b = b + torch.where(first, a * h0[seq], 0.0)
    gone = torch.where(first, 0.0, a)
    h = _scan(gone, b, _down)
    y = (h * Cw).sum(-1) + s["Dskip"] * u
    if s["op"] != "scan_bwd":
        empty = (ends == starts)[:, None, None]
        h_T = torch.where(empty, 0.0 if h0 is None else h0, h[(ends - 1).clamp(min=0)])
        return (y * _silu(z)).to(t).reshape(u0.shape), h_T
    dout = flat(s["dout"])
    dz, dy = dout * y * _dsilu(z), dout * _silu(z)
    dC = (dy[..., None] * h).reshape(-1, G, D // G, N).sum(2)
    g = dy[..., None] * Cw
    if s["dh_T"] is not None:
        g = g + torch.where(last, s["dh_T"][seq], 0.0)
    dh = _scan(_up(gone, 1), g, _up)
    kept = a * (torch.where(first, 0.0 if h0 is None else h0[seq], _down(h, 1)))  # exp(d A) h_{t-1}
    dB = (dh * (d * u)[..., None]).reshape(-1, G, D // G, N).sum(2)
    dd = (dh * (kept * A + u[..., None] * Bw)).sum(-1)
    du = s["Dskip"] * dy + d * (dh * Bw).sum(-1)
    ddt = dd / (1 + torch.exp(-raw))
    dA = (dh * kept * d[..., None]).sum(0)
    dh0 = None
    if h0 is not None:
        at = starts.clamp(max=a.shape[0] - 1)
        dh0 = torch.where((ends == starts)[:, None, None], s["dh_T"], a[at] * dh[at])
    like = lambda v, w: v.to(t).reshape(w.shape)  # noqa: E731
    return (like(du, u0), like(ddt, s["dt"]), dA, like(dB, s["Bm"]), like(dC, s["Cm"]), (dy * u).sum(0), like(dz, u0), ddt.sum(0), dh0)


def _rms(x):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)


def _norm(s):
    t = s["residual"].dtype
    r, b = s["residual"].float(), s["block"].float()
    p = 1 / (1 + torch.exp(-s["gate"].float())) if s["gate"] is not None else torch.ones_like(b)
    scale, w_post, w_pre = s["scale"], s["w_post"], s["w_pre"]
    rb = _rms(b)
    n = b * rb
    if s["op"] == "norm_fwd":
        r2 = r + scale * p * n * w_post
        return r2.to(t), (r2 * _rms(r2) * w_pre).to(t)
    # here `residual` is what the forward left: the backward reads that and the block
    rr = _rms(r)
    m, dx = r * rr, s["dx"].float()
    dm = dx * w_pre
    dr = s["dres"].float() + rr * (dm - m * (dm * m).mean(-1, keepdim=True))
    dn = dr * scale * p * w_post
    db = rb * (dn - n * (dn * n).mean(-1, keepdim=True))
    dgate = (dr * scale * n * w_post * p * (1 - p)).to(t) if s["gate"] is not None else None
    return dr.to(t), db.to(t), dgate, (dr * p * n * w_post).sum(0), (dr * scale * p * n).sum(0), (dx * m).sum(0)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op.startswith("conv"):
        if op == "conv_step":
            state = {**state, "cu_seqlens": None}
        return _conv(state)
    return _ssm(state) if op.startswith("scan") else _norm(state)


# ------------------------------------------------------------ in 64 bits, token by token
def _bounds(s, lead):
    if s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].tolist()
    else:
        T = lead[1] if len(lead) == 2 else 1
        cu = [i * T for i in range(lead[0] + 1)]
    return list(zip(cu[:-1], cu[1:]))


def _exact_conv(s):
    op, x0 = s["op"], s["x"]
    D, K = x0.shape[-1], s["w"].shape[1]
    need = op == "conv_bwd"
    leaf = lambda v: v.double().detach().clone().requires_grad_(need)  # noqa: E731
    x, w, bias = leaf(x0.reshape(-1, D)), leaf(s["w"]), leaf(s["bias"])
    bounds = _bounds(s, x0.shape[:-1])
    state0 = leaf(s["state0"]) if s["state0"] is not None else None
    none = torch.zeros(K - 1, D, dtype=torch.float64, device="cuda")
    ys, ends = [], []
    for i, (lo, hi) in enumerate(bounds):
        ext = torch.cat([none if state0 is None else state0[i], x[lo:hi]])
        if hi > lo:
            pre = (ext.unfold(0, K, 1) * w).sum(-1) + bias
            ys.append(pre * torch.sigmoid(pre))
        ends.append(ext[hi - lo:])
    y, state_T = torch.cat(ys), torch.stack(ends)
    if not need:
        return y.reshape(x0.shape), state_T
    loss = (y * s["dy"].double().reshape(-1, D)).sum()
    if s["dstate_T"] is not None:
        loss = loss + (state_T * s["dstate_T"].double()).sum()
    loss.backward()
    return x.grad.reshape(x0.shape), w.grad, bias.grad, None if state0 is None else state0.grad


def _exact_ssm(s):
    u0 = s["u"]
    lead, D = u0.shape[:-1], u0.shape[-1]
    G, N = s["Bm"].shape[-2:]
    bounds = _bounds(s, lead)
    S, T = len(bounds), max(hi - lo for lo, hi in bounds)
    rows = u0.numel() // D
    # sequences side by side, short ones filled up; `real` says which tokens are there
    lo = torch.tensor([b[0] for b in bounds], device="cuda")[:, None]
    n = torch.tensor([b[1] - b[0] for b in bounds], device="cuda")[:, None]
    step = torch.arange(T, device="cuda")[None]
    at, real = (lo + step).clamp(max=rows - 1), step < n
    need = s["op"] == "scan_bwd"
    leaf = lambda v: v.double().detach().clone().requires_grad_(need)  # noqa: E731
    u, dt, z = (leaf(s[k].reshape(-1, D)) for k in ("u", "dt", "z"))
    Bm, Cm = (leaf(s[k].reshape(-1, G, N)) for k in ("Bm", "Cm"))
    A, Ds, bias = leaf(s["A"]), leaf(s["Dskip"]), leaf(s["dt_bias"])
    h0 = leaf(s["h0"]) if s["h0"] is not None else None
    h = torch.zeros(S, D, N, dtype=torch.float64, device="cuda") if h0 is None else h0
    delta = torch.logaddexp(dt + bias, torch.zeros((), dtype=torch.float64, device="cuda"))
    ut, dl, Bt, Ct = u[at].transpose(0, 1), delta[at].transpose(0, 1), Bm[at].transpose(0, 1), Cm[at].transpose(0, 1)
    every = bool(real.all())
    ys = []
    uu, dd, BB, CC = ut.unbind(0), dl.unbind(0), Bt.unbind(0), Ct.unbind(0)
    A4 = A.reshape(G, D // G, N)
    for k in range(T):
        d4 = dd[k].reshape(S, G, D // G, 1)
        new = torch.exp(d4 * A4) * h.reshape(S, G, D // G, N) + d4 * uu[k].reshape(S, G, D // G, 1) * BB[k][:, :, None]
        ys.append(torch.matmul(new, CC[k][..., None]).reshape(S, D))
        h = new.reshape(S, D, N) if every else torch.where(real[:, k, None, None], new.reshape(S, D, N), h)
    y = torch.stack(ys, 1)[real]  # packed again, in order
    y = (y + Ds * u) * (z * torch.sigmoid(z))
    if not need:
        return y.reshape(u0.shape), h
    loss = (y * s["dout"].double().reshape(-1, D)).sum()
    if s["dh_T"] is not None:
        loss = loss + (h * s["dh_T"].double()).sum()
    loss.backward()
    return (u.grad.reshape(u0.shape), dt.grad.reshape(u0.shape), A.grad, Bm.grad.reshape(s["Bm"].shape), Cm.grad.reshape(s["Cm"].shape), Ds.grad,
            z.grad.reshape(u0.shape), bias.grad, None if h0 is None else h0.grad)


def _exact_norm(s):
    D = s["block"].shape[-1]
    need = s["op"] == "norm_bwd"
    leaf = lambda v: None if v is None else v.double().detach().clone().requires_grad_(need)  # noqa: E731
    r, b, gate, scale, w_post, w_pre = (leaf(s[k]) for k in ("residual", "block", "gate", "scale", "w_post", "w_pre"))
    unit = lambda v: v * (v.square().sum(-1, keepdim=True) / D + _EPS).rsqrt()  # noqa: E731
    branch = unit(b) * w_post * scale
    if gate is not None:
        branch = branch * torch.sigmoid(gate)
    if not need:
        out = r + branch
        return out, unit(out) * w_pre
    x = unit(r) * w_pre
    dx, dres = s["dx"].double(), s["dres"].double()
    down = torch.autograd.grad((x * dx).sum(), (r, w_pre))
    dr = dres + down[0]
    leaves = [v for v in (b, gate, scale, w_post) if v is not None]
    got = list(torch.autograd.grad((branch * dr).sum(), leaves))
    if gate is None:
        got.insert(1, None)
    return dr, got[0], got[1], got[2], got[3], down[1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("scan") and case["op"] != "scan_bwd":
        with torch.no_grad():
            return _exact_ssm({"cu_seqlens": None, **s})
    if case["op"].startswith("scan"):
        if case["rows"] // case["seqs"] > 1 << 14:
            return None
        return _exact_ssm(s)
    if case["op"].startswith("conv"):
        return _exact_conv({"cu_seqlens": None, **s})
    return _exact_norm(s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows, D, op = case["rows"], case["D"], case["op"]
    one = rows * D * e
    if op.startswith("norm"):
        gate = 1 if case["gated"] else 0
        if op == "norm_fwd":
            return {"bytes": (4 + gate) * one + 12 * D, "flops": (10 + 4 * gate) * rows * D}
        return {"bytes": (6 + 2 * gate) * one + 24 * D, "flops": (26 + 8 * gate) * rows * D}
    S = case["seqs"]
    carried = 1 if case["state"] else 0
    if "K" in case:
        K = case["K"]
        row = S * (K - 1) * D
        if op == "conv_bwd":
            return {"bytes": 3 * one + D * (K + 1) * (e + 4) + carried * row * (e + 8), "flops": rows * D * (6 * K + 10)}
        return {"bytes": 2 * one + D * (K + 1) * e + (1 + carried) * row * e, "flops": rows * D * (2 * K + 4)}
    N, G = case["N"], case["G"]
    state, bc = S * D * N * 4, 2 * rows * G * N * e
    if op == "scan_bwd":
        return {"bytes": 7 * one + 2 * bc + D * (2 * N + 4) * 4 + 3 * carried * state, "flops": rows * D * (24 * N + 40)}
    return {"bytes": 4 * one + bc + D * (N + 2) * 4 + (1 + carried) * state, "flops": rows * D * (7 * N + 16)}
