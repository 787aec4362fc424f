// kda_layers_abi.cu -- the C ABI of kda_layers.h: argument checks, workspace sizes, launches.
//
// Every check runs on the host before the first CUDA call, so a rejected call touches no device
// state.  No exception crosses the ABI.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/kda_layers.h"
#include "kda_checks.h"
#include "kda_layers_internal.h"

using namespace kda;

namespace {

constexpr long long kMaxElems = 1LL << 40;   // refuse sizes whose byte offsets could overflow
constexpr long long kMaxRows = 0x7fffff00LL;  // a few rows more still fit an int
constexpr long long kMaxStride = 1LL << 27;  // a few rows' offsets fit 32 bits of bytes

kda_opts resolve(const kda_opts *o) {
    kda_opts r;
    memset(&r, 0, sizeof(r));
    r.dtype = KDA_BF16;
    r.flags = KDA_QK_L2NORM;
    r.scale = 1.0f;
    if (o) r = *o;
    return r;
}

int check_layer_opts(const kda_opts &o) {
    const int s = check_opts(o);
    if (s != KDA_OK) return s;
    return (o.flags & ~(unsigned)KDA_QK_L2NORM) ? KDA_ERR_ARG : KDA_OK;
}

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p & 15u) return false;
    return true;
}
// row tensors: at a whole element
bool rows_aligned(bool bf16, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p & (bf16 ? 1u : 3u)) return false;
    return true;
}
// A tensor's memory: rows of `width` bytes, `ld` apart.  A NULL pointer or no bytes: none.
struct Mem {
    const char *p;
    long long rows, ld, width;
};
Mem flat(const void *p, long long bytes) { return {(const char *)p, 1, bytes, bytes}; }
Mem rows_of(const void *p, long long rows, long long ld, long long width, bool bf16) {
    const long long e = bf16 ? 2 : 4;
    return {(const char *)p, rows, ld * e, width * e};
}
bool overlap(const Mem &a, const Mem &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    if (pb >= pa + (a.rows - 1) * a.ld + a.width || pa >= pb + (b.rows - 1) * b.ld + b.width) return false;
    if (a.ld != b.ld) return true;
    // column ranges of rows equally far apart
    const long long d = (long long)((pb >= pa ? pb - pa : (uintptr_t)a.ld - (pa - pb) % a.ld) % a.ld);
    return !(d >= a.width && d + b.width <= a.ld);
}
// outputs against the inputs and against each other
bool distinct(std::initializer_list<Mem> outs, std::initializer_list<Mem> ins) {
    for (const Mem *o = outs.begin(); o != outs.end(); ++o) {
        for (const Mem &i : ins)
            if (overlap(*o, i)) return false;
        for (const Mem *p = outs.begin(); p != o; ++p)
            if (overlap(*o, *p)) return false;
    }
    return true;
}
// all of `p`, or nothing of it, is `q`: in place
bool same_or_apart(const Mem &p, const Mem &q) {
    return (p.p == q.p && p.rows == q.rows && p.ld == q.ld && p.width == q.width) || !overlap(p, q);
}

// A row stride: 0 stands for the row's own length.
int stride(long long &ld, long long length) {
    if (ld == 0) ld = length;
    if (ld < 0) return KDA_ERR_ARG;
    return ld < length || ld > kMaxStride ? KDA_ERR_SHAPE : KDA_OK;
}
int check_rows(int B, int T, bool packed, long long widest, long long *rows) {
    if (B < 0 || T < 0) return KDA_ERR_ARG;
    *rows = packed ? T : (long long)B * T;
    if (*rows > kMaxRows) return KDA_ERR_SHAPE;
    if (*rows > 0 && widest > kMaxElems / *rows) return KDA_ERR_SHAPE;
    return KDA_OK;
}
int status(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return KDA_ERR_UNSUPPORTED;
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Sizes of the short convolution; fills in strides and a's layout.
int conv_dims(const kda_conv_dims *d, const kda_opts &o, bool step, ConvArgs &a) {
    memset(&a, 0, sizeof(a));
    if (!d) return KDA_ERR_ARG;
    if (d->B < 0 || (!step && d->T < 0) || d->D < 0) return KDA_ERR_ARG;
    if ((d->silu | 1) != 1 || (d->zero_rest | 1) != 1) return KDA_ERR_ARG;
    if (d->K < 2 || d->K > 4) return KDA_ERR_UNSUPPORTED;
    a.cu = step ? nullptr : d->cu_seqlens;
    if ((uintptr_t)a.cu & 3u) return KDA_ERR_ALIGN;
    a.S = d->B; a.D = d->D; a.K = d->K; a.silu = d->silu;
    a.T = step ? 1 : d->T;
    a.ld_x = d->ld_x; a.ld_y = d->ld_y; a.ld_dx = d->ld_dx;
    int s = stride(a.ld_x, a.D);
    if (s == KDA_OK) s = stride(a.ld_y, a.D);
    if (s == KDA_OK) s = stride(a.ld_dx, a.D);
    if (s != KDA_OK) return s;
    long long w = a.ld_x > a.ld_y ? a.ld_x : a.ld_y;
    if (a.ld_dx > w) w = a.ld_dx;
    if ((s = check_rows(d->B, (int)a.T, a.cu != nullptr, w, &a.rows)) != KDA_OK) return s;
    if ((long long)a.S * 4 * a.D > kMaxElems || (long long)a.D * 5 > 0x7fffffffLL) return KDA_ERR_SHAPE;
    a.bf16 = o.dtype == KDA_BF16;
    return KDA_OK;
}

int ssm_dims(const kda_ssm_dims *d, const kda_opts &o, bool step, SsmArgs &a) {
    memset(&a, 0, sizeof(a));
    if (!d) return KDA_ERR_ARG;
    if (d->B < 0 || (!step && d->T < 0) || d->D < 0 || d->G <= 0) return KDA_ERR_ARG;
    if ((d->dt_softplus | 1) != 1 || (d->zero_rest | 1) != 1) return KDA_ERR_ARG;
    if (d->N != 8 && d->N != 16 && d->N != 32 && d->N != 64) return KDA_ERR_UNSUPPORTED;
    if (d->D % d->G) return KDA_ERR_SHAPE;
    a.cu = step ? nullptr : d->cu_seqlens;
    if ((uintptr_t)a.cu & 3u) return KDA_ERR_ALIGN;
    a.S = d->B; a.D = d->D; a.N = d->N; a.G = d->G; a.softplus = d->dt_softplus;
    a.T = step ? 1 : d->T;
    a.ld_u = d->ld_u; a.ld_dt = d->ld_dt; a.ld_z = d->ld_z; a.ld_B = d->ld_B; a.ld_C = d->ld_C; a.ld_out = d->ld_out;
    const long long bc = (long long)a.G * a.N;
    long long *const ld[] = {&a.ld_u, &a.ld_dt, &a.ld_z, &a.ld_out, &a.ld_B, &a.ld_C};
    long long w = 0;
    for (int i = 0; i < 6; ++i) {
        const int s = stride(*ld[i], i < 4 ? a.D : bc);
        if (s != KDA_OK) return s;
        if (*ld[i] > w) w = *ld[i];
    }
    const int s = check_rows(d->B, (int)a.T, a.cu != nullptr, w, &a.rows);
    if (s != KDA_OK) return s;
    // states of all sequences, and the seams' states: at most one a sequence and shortest span
    if (a.D > 0 && (long long)a.N * (a.S + a.rows / kShortestSpan + 1) > kMaxElems / a.D) return KDA_ERR_SHAPE;
    a.bf16 = o.dtype == KDA_BF16;
    return KDA_OK;
}

int norm_dims(const kda_norm_dims *d, const kda_opts &o, NormArgs &a) {
    memset(&a, 0, sizeof(a));
    if (!d) return KDA_ERR_ARG;
    if (d->rows < 0 || d->D < 0 || !isfinite(d->eps) || d->eps < 0.f) return KDA_ERR_ARG;
    if (d->D < 1 || d->D > 16384) return KDA_ERR_UNSUPPORTED;
    a.rows = d->rows; a.D = d->D; a.eps = d->eps;
    a.ld_res = d->ld_res; a.ld_block = d->ld_block; a.ld_gate = d->ld_gate;
    long long *const ld[] = {&a.ld_res, &a.ld_block, &a.ld_gate};
    for (int i = 0; i < 3; ++i) {
        const int s = stride(*ld[i], a.D);
        if (s != KDA_OK) return s;
        if (a.rows > 0 && *ld[i] > kMaxElems / a.rows) return KDA_ERR_SHAPE;
    }
    a.bf16 = o.dtype == KDA_BF16;
    return KDA_OK;
}

// Zeroes n FP32 values; NULL is nobody's.
cudaError_t zero_f32(float *p, size_t n, cudaStream_t st) {
    return p && n ? cudaMemsetAsync(p, 0, n * sizeof(float), st) : cudaSuccess;
}

LaunchMarks marks_of(const kda_opts &o) { return LaunchMarks{o.events, o.n_events, 0}; }

}  // namespace

extern "C" {

size_t kda_short_conv_bwd_workspace_bytes(const kda_conv_dims *dims, const kda_opts *opts) {
    const kda_opts o = resolve(opts);
    ConvArgs a;
    if (check_layer_opts(o) != KDA_OK || conv_dims(dims, o, false, a) != KDA_OK) return 0;
    return short_conv_bwd_workspace_bytes(a.rows, a.D, a.K);
}

int kda_short_conv_fwd(const void *x, const void *w, const void *bias, const void *state0, void *y, void *state_T,
                       const kda_conv_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    ConvArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = conv_dims(dims, o, false, a)) != KDA_OK) return s;
    if (a.D == 0) return KDA_OK;
    if (!w || (a.rows > 0 && (!x || !y))) return KDA_ERR_ARG;
    if (!all_aligned({w, bias, state0, state_T}) || !rows_aligned(a.bf16, {x, y}))
        return KDA_ERR_ALIGN;
    const long long es = a.bf16 ? 2 : 4, ns = (long long)a.S * (a.K - 1) * a.D, D = a.D;
    if (!distinct({rows_of(y, a.rows, a.ld_y, D, a.bf16), flat(state_T, ns * es)},
                  {rows_of(x, a.rows, a.ld_x, D, a.bf16), flat(w, D * a.K * es), flat(bias, D * es), flat(state0, ns * es),
                   flat(a.cu, a.cu ? 4 * (a.S + 1LL) : 0)}))
        return KDA_ERR_ARG;
    a.x = x; a.w = w; a.bias = bias; a.state0 = state0; a.y = y; a.state_T = state_T;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    cudaError_t e = a.S > 0 ? launch_short_conv_fwd(a, stream) : cudaSuccess;
    if (e == cudaSuccess && a.cu && dims->zero_rest && a.rows > 0) {
        const ZeroRest z = {{y}, {a.D * es}, {a.ld_y * es}, 1};
        m.mark(stream);
        e = launch_zero_rest(z, a.cu, a.S, a.T, stream);
    }
    m.end(stream);
    return status(e);
}

int kda_short_conv_bwd(const void *x, const void *w, const void *bias, const void *state0, const void *dy,
                       const float *dstate_T, void *dx, float *dw, float *dbias, float *dstate0,
                       const kda_conv_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    ConvArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = conv_dims(dims, o, false, a)) != KDA_OK) return s;
    if (a.D == 0) return KDA_OK;
    if (!w || !dw || (a.rows > 0 && (!x || !dy || !dx))) return KDA_ERR_ARG;
    if (!all_aligned({w, bias, state0, dstate_T, dw, dbias, dstate0, o.workspace}) ||
        !rows_aligned(a.bf16, {x, dy, dx}))
        return KDA_ERR_ALIGN;
    const size_t need = short_conv_bwd_workspace_bytes(a.rows, a.D, a.K);
    const long long es = a.bf16 ? 2 : 4, ns = (long long)a.S * (a.K - 1) * a.D, D = a.D;
    if (!distinct({rows_of(dx, a.rows, a.ld_dx, D, a.bf16), flat(dw, D * a.K * 4), flat(dbias, D * 4), flat(dstate0, ns * 4),
                   flat(o.workspace, (long long)need)},
                  {rows_of(x, a.rows, a.ld_x, D, a.bf16), flat(w, D * a.K * es), flat(bias, D * es), flat(state0, ns * es),
                   rows_of(dy, a.rows, a.ld_y, D, a.bf16), flat(dstate_T, ns * 4), flat(a.cu, a.cu ? 4 * (a.S + 1LL) : 0)}))
        return KDA_ERR_ARG;
    if (need > 0 && (!o.workspace || o.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    a.x = x; a.w = w; a.bias = bias; a.state0 = state0; a.dy = dy; a.dstate_T = dstate_T;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.dstate0 = dstate0;
    a.workspace = o.workspace;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    cudaError_t e;
    if (a.S > 0) {
        e = launch_short_conv_bwd(a, stream);
    } else {   // no sequence: sums of nothing
        e = zero_f32(dw, (size_t)a.D * a.K, stream);
        if (e == cudaSuccess) e = zero_f32(dbias, a.D, stream);
    }
    if (e == cudaSuccess && a.cu && dims->zero_rest && a.rows > 0) {
        const ZeroRest z = {{dx}, {a.D * es}, {a.ld_dx * es}, 1};
        m.mark(stream);
        e = launch_zero_rest(z, a.cu, a.S, a.T, stream);
    }
    m.end(stream);
    return status(e);
}

int kda_short_conv_step(const void *x, const void *w, const void *bias, const void *state, void *state_out, void *y,
                        const kda_conv_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    ConvArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = conv_dims(dims, o, true, a)) != KDA_OK) return s;
    if (a.S == 0 || a.D == 0) return KDA_OK;
    if (!x || !w || !state || !state_out || !y) return KDA_ERR_ARG;
    if (!all_aligned({w, bias, state, state_out}) || !rows_aligned(a.bf16, {x, y}))
        return KDA_ERR_ALIGN;
    const long long es = a.bf16 ? 2 : 4, ns = (long long)a.S * (a.K - 1) * a.D, D = a.D;
    const Mem my = rows_of(y, a.rows, a.ld_y, D, a.bf16), so = flat(state_out, ns * es), si = flat(state, ns * es);
    if (!distinct({my, so}, {rows_of(x, a.rows, a.ld_x, D, a.bf16), flat(w, D * a.K * es), flat(bias, D * es)}) ||
        overlap(my, si) || !same_or_apart(so, si))
        return KDA_ERR_ARG;
    a.x = x; a.w = w; a.bias = bias; a.state0 = state; a.state_T = state_out; a.y = y;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    const cudaError_t e = launch_short_conv_step(a, stream);
    m.end(stream);
    return status(e);
}

size_t kda_ssm_scan_fwd_workspace_bytes(const kda_ssm_dims *dims, const kda_opts *opts) {
    const kda_opts o = resolve(opts);
    SsmArgs a;
    if (check_layer_opts(o) != KDA_OK || ssm_dims(dims, o, false, a) != KDA_OK || a.S == 0 || a.D == 0) return 0;
    return ssm_scan_fwd_workspace_bytes(a);
}
size_t kda_ssm_scan_bwd_workspace_bytes(const kda_ssm_dims *dims, const kda_opts *opts) {
    const kda_opts o = resolve(opts);
    SsmArgs a;
    if (check_layer_opts(o) != KDA_OK || ssm_dims(dims, o, false, a) != KDA_OK || a.D == 0) return 0;
    return ssm_scan_bwd_workspace_bytes(a);
}

int kda_ssm_scan_fwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                     const float *Dskip, const void *z, const float *dt_bias, const float *h0, void *out, float *h_T,
                     const kda_ssm_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    SsmArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = ssm_dims(dims, o, false, a)) != KDA_OK) return s;
    if (a.D == 0) return KDA_OK;
    if (!A || (a.rows > 0 && (!u || !dt || !Bm || !Cm || !out))) return KDA_ERR_ARG;
    if (!all_aligned({A, Dskip, dt_bias, h0, h_T, o.workspace}) ||
        !rows_aligned(a.bf16, {u, dt, Bm, Cm, z, out}))
        return KDA_ERR_ALIGN;
    const size_t need = a.S > 0 ? ssm_scan_fwd_workspace_bytes(a) : 0;
    const long long es = a.bf16 ? 2 : 4, D = a.D, bc = (long long)a.G * a.N, ns = (long long)a.S * D * a.N * 4;
    if (!distinct({rows_of(out, a.rows, a.ld_out, D, a.bf16), flat(h_T, ns), flat(o.workspace, (long long)need)},
                  {rows_of(u, a.rows, a.ld_u, D, a.bf16), rows_of(dt, a.rows, a.ld_dt, D, a.bf16), rows_of(z, a.rows, a.ld_z, D, a.bf16),
                   rows_of(Bm, a.rows, a.ld_B, bc, a.bf16), rows_of(Cm, a.rows, a.ld_C, bc, a.bf16), flat(A, D * a.N * 4),
                   flat(Dskip, D * 4), flat(dt_bias, D * 4), flat(h0, ns), flat(a.cu, a.cu ? 4 * (a.S + 1LL) : 0)}))
        return KDA_ERR_ARG;
    if (need > 0 && (!o.workspace || o.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias;
    a.h0 = h0; a.out = out; a.h_T = h_T; a.workspace = o.workspace;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    cudaError_t e = a.S > 0 ? launch_ssm_scan_fwd(a, stream) : cudaSuccess;
    if (e == cudaSuccess && a.cu && dims->zero_rest && a.rows > 0) {
        const ZeroRest zr = {{out}, {a.D * es}, {a.ld_out * es}, 1};
        m.mark(stream);
        e = launch_zero_rest(zr, a.cu, a.S, a.T, stream);
    }
    m.end(stream);
    return status(e);
}

int kda_ssm_scan_bwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                     const float *Dskip, const void *z, const float *dt_bias, const float *h0, const void *dout,
                     const float *dh_T, void *du, void *ddt, float *dA, void *dB, void *dC, float *dDskip, void *dz,
                     float *ddt_bias, float *dh0, const kda_ssm_dims *dims, const kda_opts *opts,
                     cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    SsmArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = ssm_dims(dims, o, false, a)) != KDA_OK) return s;
    if (a.D == 0) return KDA_OK;
    if (!A || !dA || (z == nullptr) != (dz == nullptr)) return KDA_ERR_ARG;
    if (a.rows > 0 && (!u || !dt || !Bm || !Cm || !dout || !du || !ddt || !dB || !dC)) return KDA_ERR_ARG;
    if (!all_aligned({A, Dskip, dt_bias, h0, dh_T, du, ddt, dA, dB, dC, dDskip, dz, ddt_bias, dh0, o.workspace}) ||
        !rows_aligned(a.bf16, {u, dt, Bm, Cm, z, dout}))
        return KDA_ERR_ALIGN;
    const size_t need = ssm_scan_bwd_workspace_bytes(a);
    const long long es = a.bf16 ? 2 : 4, D = a.D, bc = (long long)a.G * a.N, ns = (long long)a.S * D * a.N * 4;
    const long long nd = a.rows * D * es, nbc = a.rows * bc * es;
    if (!distinct({flat(du, nd), flat(ddt, nd), flat(dz, nd), flat(dB, nbc), flat(dC, nbc), flat(dA, D * a.N * 4),
                   flat(dDskip, D * 4), flat(ddt_bias, D * 4), flat(dh0, ns), flat(o.workspace, (long long)need)},
                  {rows_of(u, a.rows, a.ld_u, D, a.bf16), rows_of(dt, a.rows, a.ld_dt, D, a.bf16), rows_of(z, a.rows, a.ld_z, D, a.bf16),
                   rows_of(Bm, a.rows, a.ld_B, bc, a.bf16), rows_of(Cm, a.rows, a.ld_C, bc, a.bf16), flat(A, D * a.N * 4),
                   flat(Dskip, D * 4), flat(dt_bias, D * 4), flat(h0, ns),
                   rows_of(dout, a.rows, a.ld_out, D, a.bf16), flat(dh_T, ns), flat(a.cu, a.cu ? 4 * (a.S + 1LL) : 0)}))
        return KDA_ERR_ARG;
    if (need > 0 && (!o.workspace || o.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias;
    a.h0 = h0; a.dout = dout; a.dh_T = dh_T; a.du = du; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC;
    a.dDskip = dDskip; a.dz = dz; a.ddt_bias = ddt_bias; a.dh0 = dh0; a.workspace = o.workspace;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    cudaError_t e;
    if (a.S > 0) {
        e = launch_ssm_scan_bwd(a, stream);
    } else {
        e = zero_f32(dA, (size_t)a.D * a.N, stream);
        if (e == cudaSuccess) e = zero_f32(dDskip, dDskip ? a.D : 0, stream);
        if (e == cudaSuccess) e = zero_f32(ddt_bias, ddt_bias ? a.D : 0, stream);
    }
    if (e == cudaSuccess && a.cu && dims->zero_rest && a.rows > 0) {
        const long long row = a.D * es, bc = (long long)a.G * a.N * es;
        ZeroRest zr = {{du, ddt, dB, dC, dz}, {row, row, bc, bc, row}, {row, row, bc, bc, row}, dz ? 5 : 4};
        m.mark(stream);
        e = launch_zero_rest(zr, a.cu, a.S, a.T, stream);
    }
    m.end(stream);
    return status(e);
}

int kda_ssm_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *Dskip,
                 const void *z, const float *dt_bias, const float *h, float *h_out, void *out,
                 const kda_ssm_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    SsmArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = ssm_dims(dims, o, true, a)) != KDA_OK) return s;
    if (a.S == 0 || a.D == 0) return KDA_OK;
    if (!u || !dt || !A || !Bm || !Cm || !h || !h_out || !out) return KDA_ERR_ARG;
    if (!all_aligned({A, Dskip, dt_bias, h, h_out}) ||
        !rows_aligned(a.bf16, {u, dt, Bm, Cm, z, out}))
        return KDA_ERR_ALIGN;
    const long long D = a.D, bc = (long long)a.G * a.N, ns = (long long)a.S * D * a.N * 4;
    const Mem mo = rows_of(out, a.rows, a.ld_out, D, a.bf16), ho = flat(h_out, ns), hi = flat(h, ns);
    if (!distinct({mo, ho}, {rows_of(u, a.rows, a.ld_u, D, a.bf16), rows_of(dt, a.rows, a.ld_dt, D, a.bf16), rows_of(z, a.rows, a.ld_z, D, a.bf16),
                   rows_of(Bm, a.rows, a.ld_B, bc, a.bf16), rows_of(Cm, a.rows, a.ld_C, bc, a.bf16), flat(A, D * a.N * 4),
                   flat(Dskip, D * 4), flat(dt_bias, D * 4)}) ||
        overlap(mo, hi) || !same_or_apart(ho, hi))
        return KDA_ERR_ARG;
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias;
    a.h0 = h; a.h_T = h_out; a.out = out;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    const cudaError_t e = launch_ssm_step(a, stream);
    m.end(stream);
    return status(e);
}

int kda_block_norm_fwd(const void *residual, const void *block, const void *gate, const float *scale,
                       const float *w_post, const float *w_pre, void *res_out, void *x, const kda_norm_dims *dims,
                       const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    NormArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = norm_dims(dims, o, a)) != KDA_OK) return s;
    if (a.rows == 0) return KDA_OK;
    if (!residual || (!res_out && !x)) return KDA_ERR_ARG;
    if (block ? !res_out : (res_out || gate || scale || w_post)) return KDA_ERR_ARG;
    if (!all_aligned({scale, w_post, w_pre, res_out, x}) ||
        !rows_aligned(a.bf16, {residual, block, gate}))
        return KDA_ERR_ALIGN;
    const long long D = a.D;
    const Mem mr = rows_of(residual, a.rows, a.ld_res, D, a.bf16), mo = rows_of(res_out, a.rows, D, D, a.bf16),
              mx = rows_of(x, a.rows, D, D, a.bf16);
    if (!distinct({mx, mo}, {rows_of(block, a.rows, a.ld_block, D, a.bf16), rows_of(gate, a.rows, a.ld_gate, D, a.bf16),
                             flat(scale, D * 4), flat(w_post, D * 4), flat(w_pre, D * 4)}) ||
        overlap(mx, mr) || !same_or_apart(mo, mr))
        return KDA_ERR_ARG;
    a.residual = residual; a.block = block; a.gate = gate; a.scale = scale; a.w_post = w_post; a.w_pre = w_pre;
    a.res_out = res_out; a.x = x;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    const cudaError_t e = launch_block_norm_fwd(a, stream);
    m.end(stream);
    return status(e);
}

size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_dims *dims, const kda_opts *opts) {
    const kda_opts o = resolve(opts);
    NormArgs a;
    if (check_layer_opts(o) != KDA_OK || norm_dims(dims, o, a) != KDA_OK) return 0;
    return block_norm_bwd_workspace_bytes(a.rows, a.D);
}

int kda_block_norm_bwd(const void *res_out, const void *block, const void *gate, const float *scale,
                       const float *w_post, const float *w_pre, const void *dres, const void *dx, void *dresidual,
                       void *dblock, void *dgate, float *dscale, float *dw_post, float *dw_pre,
                       const kda_norm_dims *dims, const kda_opts *opts, cudaStream_t stream) {
    const kda_opts o = resolve(opts);
    NormArgs a;
    int s = check_layer_opts(o);
    if (s != KDA_OK || (s = norm_dims(dims, o, a)) != KDA_OK) return s;
    if (a.rows > 0) {
        if ((!dres && !dx) || !dresidual || (dx && !res_out)) return KDA_ERR_ARG;
        if ((block == nullptr) != (dblock == nullptr) || (gate == nullptr) != (dgate == nullptr)) return KDA_ERR_ARG;
        if (!block && (gate || scale || w_post || dscale || dw_post)) return KDA_ERR_ARG;
    }
    if (!all_aligned({scale, w_post, w_pre, dres, dx, dresidual, dblock, dgate, dscale, dw_post, dw_pre, o.workspace}) ||
        !rows_aligned(a.bf16, {res_out, block, gate}))
        return KDA_ERR_ALIGN;
    const size_t need = block_norm_bwd_workspace_bytes(a.rows, a.D);
    const long long D = a.D, nd = (long long)a.rows * D * (a.bf16 ? 2 : 4);
    const Mem md = flat(dresidual, nd), mi = flat(dres, nd), mb = flat(dblock, nd), mg = flat(dgate, nd),
              mw = flat(o.workspace, (long long)need);
    if (!distinct({md, mb, mg, flat(dscale, D * 4), flat(dw_post, D * 4), flat(dw_pre, D * 4), mw},
                  {rows_of(res_out, a.rows, a.ld_res, D, a.bf16), rows_of(block, a.rows, a.ld_block, D, a.bf16),
                   rows_of(gate, a.rows, a.ld_gate, D, a.bf16), flat(scale, D * 4), flat(w_post, D * 4), flat(w_pre, D * 4),
                   flat(dx, nd)}))
        return KDA_ERR_ARG;
    if (!same_or_apart(md, mi) || overlap(mb, mi) || overlap(mg, mi) || overlap(mw, mi) || overlap(flat(dscale, D * 4), mi) ||
        overlap(flat(dw_post, D * 4), mi) || overlap(flat(dw_pre, D * 4), mi))
        return KDA_ERR_ARG;
    if (need > 0 && (!o.workspace || o.workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    a.residual = res_out; a.block = block; a.gate = gate; a.scale = scale; a.w_post = w_post; a.w_pre = w_pre;
    a.dres = dres; a.dx = dx; a.dresidual = dresidual; a.dblock = dblock; a.dgate = dgate;
    a.dscale = dscale; a.dw_post = dw_post; a.dw_pre = dw_pre;
    a.workspace = o.workspace;
    LaunchMarks m = marks_of(o);
    a.marks = &m;
    const cudaError_t e = launch_block_norm_bwd(a, stream);
    m.end(stream);
    return status(e);
}

}  // extern "C"
