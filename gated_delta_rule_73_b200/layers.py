"""Binding of the operators of ``include/kda_layers.h``: short convolution, selective scan, block norm.

As ``kda.py``: argument checks and marshalling only, no arithmetic and no fallback.  The ``kda_*``
functions take every output; the functions without the prefix allocate outputs and workspaces
with torch and return them.  Sequences are dense (``x [B, T, D]``) or packed (``x [rows, D]`` and
``cu_seqlens`` int32 ``[B + 1]`` on the device); a row tensor may be a column range of a wider one
(its last dimension contiguous, its rows evenly spaced).  Outputs that these functions allocate
for packed sequences hold zeros in rows of no sequence; outputs that are passed in keep theirs.

All tensors of a call live on one device; work goes to ``stream`` or to that device's current one,
whichever device is current in the calling thread.  What the functions without the prefix allocate
belongs to that stream: use it there, or order other streams behind it and tell the allocator
(``Tensor.record_stream``).
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import kda as _kda
from .kda import KDA_F32, KdaError, kda_opts

_lib = _kda._lib
# what torch.cuda.current_stream(i).cuda_stream and current_device() return, without their objects
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_ip, _ll, _vp, _sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t


class kda_conv_dims(ctypes.Structure):
    _fields_ = [("B", _ip), ("T", _ip), ("D", _ip), ("K", _ip), ("silu", _ip), ("cu_seqlens", _vp),
                ("zero_rest", _ip), ("ld_x", _ll), ("ld_y", _ll), ("ld_dx", _ll)]


class kda_ssm_dims(ctypes.Structure):
    _fields_ = [("B", _ip), ("T", _ip), ("D", _ip), ("N", _ip), ("G", _ip), ("dt_softplus", _ip),
                ("cu_seqlens", _vp), ("zero_rest", _ip), ("ld_u", _ll), ("ld_dt", _ll), ("ld_z", _ll),
                ("ld_B", _ll), ("ld_C", _ll), ("ld_out", _ll)]


class kda_norm_dims(ctypes.Structure):
    _fields_ = [("rows", _ip), ("D", _ip), ("eps", ctypes.c_float), ("ld_res", _ll), ("ld_block", _ll),
                ("ld_gate", _ll)]


def _declare():
    op = ctypes.POINTER(kda_opts)
    cd, sd, nd = (ctypes.POINTER(s) for s in (kda_conv_dims, kda_ssm_dims, kda_norm_dims))
    for name, pointers, dims in (("kda_short_conv_fwd", 6, cd), ("kda_short_conv_bwd", 10, cd),
                                 ("kda_short_conv_step", 6, cd), ("kda_ssm_scan_fwd", 11, sd),
                                 ("kda_ssm_scan_bwd", 20, sd), ("kda_ssm_step", 11, sd),
                                 ("kda_block_norm_fwd", 8, nd), ("kda_block_norm_bwd", 14, nd)):
        f = getattr(_lib, name)
        f.argtypes = [_vp] * pointers + [dims, op, _vp]
        f.restype = _ip
    for name, dims in (("kda_short_conv_bwd_workspace_bytes", cd), ("kda_ssm_scan_fwd_workspace_bytes", sd),
                       ("kda_ssm_scan_bwd_workspace_bytes", sd), ("kda_block_norm_bwd_workspace_bytes", nd)):
        f = getattr(_lib, name)
        f.argtypes = [dims, op]
        f.restype = _sz


_declare()
_F32 = torch.float32


# ------------------------------------------------------------------ argument checks
# A decode step runs for a few microseconds on the device, so a tensor's checks are one chain of
# cheap comparisons; what is wrong is found out only when something is.
class _Call:
    """Checks the tensors of one call: type, shape, device, layout; gives their addresses."""
    __slots__ = ("dtype", "device", "lead")

    def __init__(self, x, name, lead):
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        self.dtype, self.device, self.lead = x.dtype, x.get_device(), tuple(lead)

    def flat(self, t, name, shape, dtype=None):
        """Address of a contiguous tensor of this shape; None stays None."""
        if t is None:
            return None
        if dtype is None:
            dtype = self.dtype
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == self.device
                and t.is_contiguous()):
            return t.data_ptr()
        self._refuse(t, name, shape, dtype)
        raise ValueError(f"{name} must be contiguous")

    def rows(self, t, name, tail):
        """(address, row stride) of a row tensor [*lead, *tail]; (None, 0) for None."""
        if t is None:
            return None, 0
        if not (isinstance(t, torch.Tensor) and t.dtype is self.dtype and t.shape == self.lead + tail
                and t.get_device() == self.device):
            self._refuse(t, name, self.lead + tail, self.dtype)
        return t.data_ptr(), 0 if t.is_contiguous() else self._row_stride(t.stride(), name, tail)

    def _refuse(self, t, name, shape, dtype):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{self.device}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")

    def _row_stride(self, st, name, tail):
        lead = len(self.lead)
        # the row itself is contiguous
        want = 1
        for n, s in zip(reversed(tail), reversed(st[lead:])):
            if n != 1 and s != want:
                raise ValueError(f"{name}: the values of a row must be contiguous (strides {st})")
            want *= n
        # rows evenly spaced: dimensions of one element say nothing about it
        ld, span = None, 1
        for n, s in zip(reversed(self.lead), reversed(st[:lead])):
            if n != 1:
                if ld is None:
                    if s % span:
                        raise ValueError(f"{name}: rows must be evenly spaced (strides {st})")
                    ld = s // span
                elif s != ld * span:
                    raise ValueError(f"{name}: rows must be evenly spaced (strides {st})")
            span *= n
        if ld is None:
            ld = want
        if ld < want:
            raise ValueError(f"{name}: rows overlap (strides {st})")
        return ld


def _opts(dtype, workspace=None, device=None):
    o = kda_opts()
    if dtype is _F32:
        o.dtype = KDA_F32
    elif dtype is not torch.bfloat16:   # KDA_BF16 is 0
        raise TypeError(f"unsupported activation dtype {dtype}; use bfloat16 or float32")
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if workspace.get_device() != device:
            raise ValueError(f"workspace is on {workspace.device}, expected cuda:{device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    return o


def _launch(fn, call, args, dims, opts, stream):
    """Runs the C call on the tensors' device, whichever is current."""
    dev = call.device
    if stream is None:
        handle = _raw_stream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError(f"stream is on {stream.device}, expected cuda:{dev}")
        handle = stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, dims, opts, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, dims, opts, handle)
    if st != 0:
        raise KdaError(fn.__name__, st)


def _on_stream(f):
    """What f allocates comes from the memory of the stream that it is given."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, stream=stream, **kw)
    return call


def _workspace(nbytes, device):
    """Scratch for one call."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _rows_like(x):
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _sequences(x, cu_seqlens):
    """(lead, B, T) of a row tensor; checks cu_seqlens."""
    lead = tuple(x.shape[:-1])
    if cu_seqlens is None:
        if len(lead) != 2:
            raise ValueError(f"expected [B, T, ...] without cu_seqlens, got shape {tuple(x.shape)}")
        return lead, lead[0], lead[1]
    if len(lead) != 1:
        raise ValueError(f"expected [rows, ...] with cu_seqlens, got shape {tuple(x.shape)}")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 \
            or cu_seqlens.shape[0] < 1:
        raise TypeError("cu_seqlens must be an int32 tensor of B + 1 values")
    return lead, cu_seqlens.shape[0] - 1, lead[0]


_INT = 0x7fffffff   # the C structures hold sizes as int


def _cu(call, cu_seqlens):
    return None if cu_seqlens is None else call.flat(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32)


# ------------------------------------------------------------------ short convolution
def _conv_call(x, w, cu_seqlens, silu, zero_rest, step=False):
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise TypeError("x and w must be torch.Tensors")
    if w.dim() != 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected [D, K]")
    shape = x.shape
    if step:
        if len(shape) != 2:
            raise ValueError(f"x has shape {tuple(shape)}, expected [B, D]")
        B, T = shape[0], 1
        lead = (B,)
    else:
        lead, B, T = _sequences(x, cu_seqlens)
    call = _Call(x, "x", lead)
    D, K = shape[-1], w.shape[1]
    if B | T | D | K > _INT:
        raise ValueError(f"sizes {(B, T, D, K)} do not fit an int")
    d = kda_conv_dims(B=B, T=T, D=D, K=K, silu=1 if silu else 0, cu_seqlens=_cu(call, cu_seqlens), zero_rest=1 if zero_rest else 0)
    return call, d, (B, K - 1, D), (D, K)


def kda_short_conv_fwd(x, w, bias, state0, y, state_T, *, cu_seqlens=None, silu=True, zero_rest=False,
                       stream=None) -> None:
    """Call ``kda_short_conv_fwd``; x, y [B,T,D] or packed [rows,D], w [D,K], bias [D], states [B,K-1,D]."""
    call, d, state, taps = _conv_call(x, w, cu_seqlens, silu, zero_rest)
    px, d.ld_x = call.rows(x, "x", (d.D,))
    py, d.ld_y = call.rows(y, "y", (d.D,))
    args = (px, call.flat(w, "w", taps), call.flat(bias, "bias", (d.D,)), call.flat(state0, "state0", state), py,
            call.flat(state_T, "state_T", state))
    _launch(_lib.kda_short_conv_fwd, call, args, d, _opts(x.dtype), stream)


def kda_short_conv_bwd_workspace_bytes(x, w, *, cu_seqlens=None) -> int:
    """Workspace bytes ``kda_short_conv_bwd`` needs for these tensors."""
    _, d, _, _ = _conv_call(x, w, cu_seqlens, True, False)
    return int(_lib.kda_short_conv_bwd_workspace_bytes(d, _opts(x.dtype)))


def kda_short_conv_bwd(x, w, bias, state0, dy, dstate_T, dx, dw, dbias, dstate0, workspace, *, cu_seqlens=None,
                       silu=True, zero_rest=False, stream=None) -> None:
    """Call ``kda_short_conv_bwd``: gradients of <dy, y> + <dstate_T, state_T> of ``kda_short_conv_fwd``."""
    call, d, state, taps = _conv_call(x, w, cu_seqlens, silu, zero_rest)
    px, d.ld_x = call.rows(x, "x", (d.D,))
    py, d.ld_y = call.rows(dy, "dy", (d.D,))
    pdx, d.ld_dx = call.rows(dx, "dx", (d.D,))
    args = (px, call.flat(w, "w", taps), call.flat(bias, "bias", (d.D,)), call.flat(state0, "state0", state), py,
            call.flat(dstate_T, "dstate_T", state, _F32), pdx, call.flat(dw, "dw", taps, _F32),
            call.flat(dbias, "dbias", (d.D,), _F32), call.flat(dstate0, "dstate0", state, _F32))
    _launch(_lib.kda_short_conv_bwd, call, args, d, _opts(x.dtype, workspace, call.device), stream)


def kda_short_conv_step(x, w, bias, state, state_out, y, *, silu=True, stream=None) -> None:
    """Call ``kda_short_conv_step``; x, y [B,D], state, state_out [B,K-1,D] (state_out may be state)."""
    call, d, shape, taps = _conv_call(x, w, None, silu, False, step=True)
    row = taps[:1]
    px, d.ld_x = call.rows(x, "x", row)
    py, d.ld_y = call.rows(y, "y", row)
    args = (px, call.flat(w, "w", taps), call.flat(bias, "bias", row), call.flat(state, "state", shape),
            call.flat(state_out, "state_out", shape), py)
    _launch(_lib.kda_short_conv_step, call, args, d, _opts(x.dtype), stream)


@_on_stream
def short_conv_fwd(x, w, bias=None, state0=None, *, cu_seqlens=None, silu=True, y=None, stream=None):
    """Causal depthwise convolution with SiLU; returns (y, state_T)."""
    zero = y is None and cu_seqlens is not None
    if y is None:
        y = _rows_like(x)
    B = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
    state_T = x.new_empty((B, w.shape[1] - 1, x.shape[-1]))
    kda_short_conv_fwd(x, w, bias, state0, y, state_T, cu_seqlens=cu_seqlens, silu=silu, zero_rest=zero, stream=stream)
    return y, state_T


@_on_stream
def short_conv_bwd(x, w, bias, state0, dy, dstate_T=None, *, cu_seqlens=None, silu=True, workspace=None,
                   stream=None):
    """Gradients of ``short_conv_fwd``; returns (dx, dw, dbias, dstate0), None for what was not passed."""
    if workspace is None:
        workspace = _workspace(kda_short_conv_bwd_workspace_bytes(x, w, cu_seqlens=cu_seqlens), x.device)
    e = lambda t, dtype=_F32: None if t is None else torch.empty(t.shape, dtype=dtype, device=x.device)  # noqa: E731
    dx, dw, dbias, dstate0 = e(x, x.dtype), e(w), e(bias), e(state0)
    kda_short_conv_bwd(x, w, bias, state0, dy, dstate_T, dx, dw, dbias, dstate0, workspace, cu_seqlens=cu_seqlens,
                       silu=silu, zero_rest=cu_seqlens is not None, stream=stream)
    return dx, dw, dbias, dstate0


@_on_stream
def short_conv_step(x, w, bias, state, *, state_out=None, silu=True, y=None, stream=None):
    """One row a sequence; state is updated in place unless state_out is given.  Returns y."""
    if y is None:
        y = _rows_like(x)
    kda_short_conv_step(x, w, bias, state, state if state_out is None else state_out, y, silu=silu, stream=stream)
    return y


# ------------------------------------------------------------------ selective scan
def _ssm_call(u, A, Bm, cu_seqlens, dt_softplus, zero_rest, step=False):
    if not (isinstance(u, torch.Tensor) and isinstance(A, torch.Tensor) and isinstance(Bm, torch.Tensor)):
        raise TypeError("u, A and Bm must be torch.Tensors")
    if A.dim() != 2:
        raise ValueError(f"A has shape {tuple(A.shape)}, expected [D, N]")
    shape, groups = u.shape, Bm.shape
    if step:
        if len(shape) != 2:
            raise ValueError(f"u has shape {tuple(shape)}, expected [B, D]")
        B, T = shape[0], 1
        lead = (B,)
    else:
        lead, B, T = _sequences(u, cu_seqlens)
    if len(groups) != len(lead) + 2:
        raise ValueError(f"Bm has shape {tuple(groups)}, expected {tuple(lead)} + [G, N]")
    call = _Call(u, "u", lead)
    D, N, G = shape[-1], A.shape[1], groups[-2]
    if B | T | D | N | G > _INT:
        raise ValueError(f"sizes {(B, T, D, N, G)} do not fit an int")
    d = kda_ssm_dims(B=B, T=T, D=D, N=N, G=G, dt_softplus=1 if dt_softplus else 0, cu_seqlens=_cu(call, cu_seqlens),
                     zero_rest=1 if zero_rest else 0)
    return call, d, (B, D, N)


def _ssm_inputs(call, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, state):
    rates = state[1:]                     # (D, N)
    row, bc = rates[:1], (d.G, rates[1])
    rows, flat = call.rows, call.flat
    pu, d.ld_u = rows(u, "u", row)
    pdt, d.ld_dt = rows(dt, "dt", row)
    pz, d.ld_z = rows(z, "z", row)
    pB, d.ld_B = rows(Bm, "Bm", bc)
    pC, d.ld_C = rows(Cm, "Cm", bc)
    return (pu, pdt, flat(A, "A", rates, _F32), pB, pC, flat(Dskip, "Dskip", row, _F32), pz,
            flat(dt_bias, "dt_bias", row, _F32), flat(h0, "h0", state, _F32))


def kda_ssm_scan_fwd_workspace_bytes(u, A, Bm, *, cu_seqlens=None) -> int:
    """Workspace bytes ``kda_ssm_scan_fwd`` needs for these tensors."""
    _, d, _ = _ssm_call(u, A, Bm, cu_seqlens, True, False)
    return int(_lib.kda_ssm_scan_fwd_workspace_bytes(d, _opts(u.dtype)))


def kda_ssm_scan_fwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, out, h_T, workspace, *, cu_seqlens=None,
                     dt_softplus=True, zero_rest=False, stream=None) -> None:
    """Call ``kda_ssm_scan_fwd``; u, dt, z, out [B,T,D] or packed [rows,D], A [D,N], Bm, Cm [...,G,N]."""
    call, d, state = _ssm_call(u, A, Bm, cu_seqlens, dt_softplus, zero_rest)
    args = _ssm_inputs(call, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, state)
    po, d.ld_out = call.rows(out, "out", (d.D,))
    _launch(_lib.kda_ssm_scan_fwd, call, args + (po, call.flat(h_T, "h_T", state, _F32)), d,
            _opts(u.dtype, workspace, call.device), stream)


def kda_ssm_scan_bwd_workspace_bytes(u, A, Bm, *, cu_seqlens=None) -> int:
    """Workspace bytes ``kda_ssm_scan_bwd`` needs for these tensors."""
    _, d, _ = _ssm_call(u, A, Bm, cu_seqlens, True, False)
    return int(_lib.kda_ssm_scan_bwd_workspace_bytes(d, _opts(u.dtype)))


def kda_ssm_scan_bwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, dout, dh_T, du, ddt, dA, dB, dC, dDskip, dz, ddt_bias,
                     dh0, workspace, *, cu_seqlens=None, dt_softplus=True, zero_rest=False, stream=None) -> None:
    """Call ``kda_ssm_scan_bwd``: gradients of <dout, out> + <dh_T, h_T> of ``kda_ssm_scan_fwd``."""
    call, d, state = _ssm_call(u, A, Bm, cu_seqlens, dt_softplus, zero_rest)
    args = _ssm_inputs(call, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, state)
    po, d.ld_out = call.rows(dout, "dout", (d.D,))
    row, bc = call.lead + (d.D,), call.lead + (d.G, d.N)
    args += (po, call.flat(dh_T, "dh_T", state, _F32), call.flat(du, "du", row), call.flat(ddt, "ddt", row),
             call.flat(dA, "dA", (d.D, d.N), _F32), call.flat(dB, "dB", bc), call.flat(dC, "dC", bc),
             call.flat(dDskip, "dDskip", (d.D,), _F32), call.flat(dz, "dz", row),
             call.flat(ddt_bias, "ddt_bias", (d.D,), _F32), call.flat(dh0, "dh0", state, _F32))
    _launch(_lib.kda_ssm_scan_bwd, call, args, d, _opts(u.dtype, workspace, call.device), stream)


def kda_ssm_step(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h, h_out, out, *, dt_softplus=True, stream=None) -> None:
    """Call ``kda_ssm_step``; u, dt, z, out [B,D], Bm, Cm [B,G,N], h, h_out [B,D,N] (h_out may be h)."""
    call, d, state = _ssm_call(u, A, Bm, None, dt_softplus, False, step=True)
    args = _ssm_inputs(call, d, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h, state)
    po, d.ld_out = call.rows(out, "out", (d.D,))
    _launch(_lib.kda_ssm_step, call, args + (call.flat(h_out, "h_out", state, _F32), po), d, _opts(u.dtype), stream)


@_on_stream
def ssm_scan_fwd(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, h0=None, *, cu_seqlens=None, dt_softplus=True,
                 out=None, workspace=None, stream=None):
    """Selective scan over sequences; returns (out, h_T)."""
    if workspace is None:
        workspace = _workspace(kda_ssm_scan_fwd_workspace_bytes(u, A, Bm, cu_seqlens=cu_seqlens), u.device)
    zero = out is None and cu_seqlens is not None
    if out is None:
        out = _rows_like(u)
    B = u.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
    h_T = torch.empty((B,) + A.shape, dtype=_F32, device=u.device)
    kda_ssm_scan_fwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, out, h_T, workspace, cu_seqlens=cu_seqlens,
                     dt_softplus=dt_softplus, zero_rest=zero, stream=stream)
    return out, h_T


@_on_stream
def ssm_scan_bwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, dout, dh_T=None, *, cu_seqlens=None, dt_softplus=True,
                 workspace=None, stream=None):
    """Gradients of ``ssm_scan_fwd``; returns (du, ddt, dA, dB, dC, dDskip, dz, ddt_bias, dh0), None for
    what was not passed."""
    if workspace is None:
        workspace = _workspace(kda_ssm_scan_bwd_workspace_bytes(u, A, Bm, cu_seqlens=cu_seqlens), u.device)
    e = lambda t, dtype: None if t is None else torch.empty(t.shape, dtype=dtype, device=u.device)  # noqa: E731
    g = (e(u, u.dtype), e(u, u.dtype), e(A, _F32), e(Bm, u.dtype), e(Bm, u.dtype), e(Dskip, _F32), e(z, u.dtype),
         e(dt_bias, _F32), e(h0, _F32))
    kda_ssm_scan_bwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, dout, dh_T, *g, workspace, cu_seqlens=cu_seqlens,
                     dt_softplus=dt_softplus, zero_rest=cu_seqlens is not None, stream=stream)
    return g


@_on_stream
def ssm_step(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h, *, h_out=None, dt_softplus=True, out=None, stream=None):
    """One token a sequence; h is updated in place unless h_out is given.  Returns out."""
    if out is None:
        out = _rows_like(u)
    kda_ssm_step(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h, h if h_out is None else h_out, out,
                 dt_softplus=dt_softplus, stream=stream)
    return out


# ------------------------------------------------------------------ block norm
def _norm_call(residual, name, eps):
    if not isinstance(residual, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if residual.dim() < 1:
        raise ValueError(f"{name} must be [..., D]")
    lead, D = residual.shape[:-1], residual.shape[-1]
    rows = math.prod(lead)
    if rows | D > _INT:
        raise ValueError(f"sizes {(rows, D)} do not fit an int")
    return _Call(residual, name, lead), kda_norm_dims(rows=rows, D=D, eps=eps)


def kda_block_norm_fwd(residual, block, gate, scale, w_post, w_pre, res_out, x, *, eps=1e-5, stream=None) -> None:
    """Call ``kda_block_norm_fwd``; residual, block, gate, res_out, x [..., D]; scale, w_post, w_pre [D]."""
    call, d = _norm_call(residual, "residual", eps)
    w, row = (d.D,), residual.shape
    pr, d.ld_res = call.rows(residual, "residual", w)
    pb, d.ld_block = call.rows(block, "block", w)
    pg, d.ld_gate = call.rows(gate, "gate", w)
    args = (pr, pb, pg, call.flat(scale, "scale", w, _F32), call.flat(w_post, "w_post", w, _F32),
            call.flat(w_pre, "w_pre", w, _F32), call.flat(res_out, "res_out", row), call.flat(x, "x", row))
    _launch(_lib.kda_block_norm_fwd, call, args, d, _opts(residual.dtype), stream)


def kda_block_norm_bwd_workspace_bytes(res_out) -> int:
    """Workspace bytes ``kda_block_norm_bwd`` needs for these rows."""
    _, d = _norm_call(res_out, "res_out", 0.0)
    return int(_lib.kda_block_norm_bwd_workspace_bytes(d, _opts(res_out.dtype)))


def kda_block_norm_bwd(res_out, block, gate, scale, w_post, w_pre, dres, dx, dresidual, dblock, dgate, dscale,
                       dw_post, dw_pre, workspace, *, eps=1e-5, stream=None) -> None:
    """Call ``kda_block_norm_bwd``: gradients of <dres, res_out> + <dx, x> of ``kda_block_norm_fwd``."""
    call, d = _norm_call(res_out, "res_out", eps)
    w, row = (d.D,), res_out.shape
    pr, d.ld_res = call.rows(res_out, "res_out", w)
    pb, d.ld_block = call.rows(block, "block", w)
    pg, d.ld_gate = call.rows(gate, "gate", w)
    args = (pr, pb, pg, call.flat(scale, "scale", w, _F32), call.flat(w_post, "w_post", w, _F32),
            call.flat(w_pre, "w_pre", w, _F32), call.flat(dres, "dres", row), call.flat(dx, "dx", row),
            call.flat(dresidual, "dresidual", row), call.flat(dblock, "dblock", row), call.flat(dgate, "dgate", row),
            call.flat(dscale, "dscale", w, _F32), call.flat(dw_post, "dw_post", w, _F32),
            call.flat(dw_pre, "dw_pre", w, _F32))
    _launch(_lib.kda_block_norm_bwd, call, args, d, _opts(res_out.dtype, workspace, call.device), stream)


@_on_stream
def block_norm_fwd(residual, block=None, gate=None, scale=None, w_post=None, w_pre=None, *, eps=1e-5,
                   want_x=True, stream=None):
    """Norms behind a block and ahead of the next; returns (res_out, x), None for what is not computed."""
    res_out = _rows_like(residual) if block is not None else None
    x = _rows_like(residual) if want_x else None
    kda_block_norm_fwd(residual, block, gate, scale, w_post, w_pre, res_out, x, eps=eps, stream=stream)
    return res_out, x


@_on_stream
def block_norm_bwd(res_out, block, gate, scale, w_post, w_pre, dres, dx, *, eps=1e-5, workspace=None, stream=None):
    """Gradients of ``block_norm_fwd``; returns (dresidual, dblock, dgate, dscale, dw_post, dw_pre), None for
    what was not passed."""
    if workspace is None:
        workspace = _workspace(kda_block_norm_bwd_workspace_bytes(res_out), res_out.device)
    e = lambda t, dtype: None if t is None else torch.empty(t.shape, dtype=dtype, device=res_out.device)  # noqa: E731
    g = (e(res_out, res_out.dtype), e(block, res_out.dtype), e(gate, res_out.dtype), e(scale, _F32), e(w_post, _F32),
         e(w_pre, _F32))
    kda_block_norm_bwd(res_out, block, gate, scale, w_post, w_pre, dres, dx, *g, workspace, eps=eps, stream=stream)
    return g
