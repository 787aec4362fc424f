// kda_ssm_scan.cu -- selective state space scan: forward over sequences, one-token step.
//
//   delta = softplus(dt + dt_bias),  h_t = exp(delta A) h_{t-1} + delta u B_t,
//   out = (C_t . h_t + Dskip u) z sigmoid(z)
//
// A channel's recurrence is sequential in time, its N states and all channels are independent.
// The states stay in registers, four a lane; a tile of 16 tokens is loaded by all threads while
// the one before it is computed, delta and delta u are worked out once a (token, channel) and
// read from shared memory by the channel's lanes.  One exponential a state and token: the
// special-function unit takes 16 a clock and SM, which bounds the kernel before HBM does.
//
// Where sequences and channels alone leave the device idle, time is cut into spans.  A span's
// effect on the state is h -> exp(A sum delta) h + (its end from zero), so one sweep finds the
// ends of all spans, a small pass chains them, and the spans then run side by side; that doubles
// the exponentials.
#include "kda_ssm.cuh"

namespace kda {
namespace {

template <typename T, int N, bool SWEEP>
__global__ void __launch_bounds__(kSsmThreads) ssm_fwd_kernel(const SsmP a) {
    using S = SsmShape<N>;
    constexpr int NQ = S::NQ, CH = S::CH, EPT = S::EPT, ROW = S::ROW;
    __shared__ __align__(16) float2 sX[kTile * CH];   // delta, delta u
    __shared__ __align__(16) float sB[kTile * N], sC[kTile * N];
    __shared__ float sY[kTile * ROW];
    const SsmBlock b = ssm_block(a, CH);
    if (b.sp.seq < 0 || (SWEEP && b.sp.k == b.sp.count - 1)) return;
    const int tid = threadIdx.x;
    // the recurrence's lanes
    const int ch = tid / NQ, q = tid % NQ;
    const bool live = b.cin + ch < a.Dg;
    const long long c = (long long)b.g * a.Dg + b.cin + ch;
    float A2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        load_f32<float, 4>(a.A + c * N + 4 * q, A2);
#pragma unroll
        for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
        if (!SWEEP) {
            const float *src = b.sp.k ? a.hst + (b.slot * a.D + c) * N
                               : a.h0 ? a.h0 + ((long long)b.sp.seq * a.D + c) * N
                                      : nullptr;
            if (src) load_f32<float, 4>(src + 4 * q, h);
        }
    }
    // the tile's loads
    const int lt = tid >> 4, lc = (tid & 15) * EPT;
    const int lleft = a.Dg - b.cin - lc;               // channels of the group from this thread's on
    const int gc = b.g * a.Dg + b.cin + lc;
    float bias[EPT], skip[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        bias[i] = a.dt_bias && i < lleft ? a.dt_bias[gc + i] : 0.f;
        skip[i] = a.Dskip && i < lleft ? a.Dskip[gc + i] : 0.f;
    }
    Raw<T, EPT> nu, ndt, nz;
    BcTile<T, N> bc;
    auto fetch = [&](int t0) {
        const int n = b.sp.n - t0;
        const long long row = b.sp.r0 + t0 + lt;
        const bool ok = lt < n;
        nu = load_tile<T, EPT>(a.u, row, a.ld_u, gc, lleft, ok, a.vec);
        ndt = load_tile<T, EPT>(a.dt, row, a.ld_dt, gc, lleft, ok, a.vec);
        if (!SWEEP && a.z) nz = load_tile<T, EPT>(a.z, row, a.ld_z, gc, lleft, ok, a.vec);
        bc.fetch(a, b.sp.r0 + t0, n, b.g, !SWEEP);
    };
    float dsum = 0.f;
    fetch(0);
    for (int t0 = 0; t0 < b.sp.n; t0 += kTile) {
        const bool ok = t0 + lt < b.sp.n;
        const Raw<T, EPT> zr = nz;
        float u[EPT], d[EPT];
        widen<T, EPT>(nu, u);
        widen<T, EPT>(ndt, d);
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            d[i] += bias[i];
            if (a.softplus) d[i] = softplus_f32(d[i]);
            if (!ok || i >= lleft) d[i] = 0.f;   // a row behind the span leaves the state as it is
            sX[lt * CH + lc + i] = make_float2(d[i], d[i] * u[i]);
        }
        bc.put(sB, SWEEP ? nullptr : sC);
        if (t0 + kTile < b.sp.n) fetch(t0 + kTile);
        __syncthreads();
#pragma unroll
        for (int tg = 0; tg < kTile; tg += NQ) {
            float y[NQ];
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                const float2 x = sX[(tg + j) * CH + ch];
                const float4 bv = *reinterpret_cast<const float4 *>(sB + (tg + j) * N + 4 * q);
                const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = fmaf(ex2(x.x * A2[i]), h[i], x.y * bb[i]);
                if (SWEEP) {
                    dsum += x.x;
                } else {
                    const float4 cv = *reinterpret_cast<const float4 *>(sC + (tg + j) * N + 4 * q);
                    y[j] = fmaf(cv.x, h[0], cv.y * h[1]) + fmaf(cv.z, h[2], cv.w * h[3]);
                }
            }
            if (!SWEEP) sY[(tg + q) * ROW + ch] = reduce_states<NQ>(y, q);
        }
        __syncthreads();
        if (!SWEEP && ok) {
            float y[EPT], z[EPT];
            if (a.z) widen<T, EPT>(zr, z);
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                y[i] = fmaf(skip[i], u[i], sY[lt * ROW + lc + i]);
                if (a.z) y[i] *= silu_f32(z[i]);
            }
            T *o = (T *)a.out + (b.sp.r0 + t0 + lt) * a.ld_out + gc;
            if (a.vec && lleft >= EPT) store_f32<T, EPT>(o, y);
            else store_part<T, EPT>(o, y, lleft);
        }
    }
    if (!live) return;
    if (SWEEP) {
        store_f32<float, 4>(a.hst + (b.slot * a.D + c) * N + 4 * q, h);
        if (q == 0) a.sdel[b.slot * a.D + c] = dsum;
    } else if (a.h_T && b.sp.k == b.sp.count - 1) {
        store_f32<float, 4>(a.h_T + ((long long)b.sp.seq * a.D + c) * N + 4 * q, h);
    }
}

// One thread per sequence and four states walks the spans: forward, hst[slot] goes from the
// slot's own end to its start state; with gst, backward, gst[slot] goes from the gradient at the
// span's start that its own outputs make to the gradient at its end that later spans make.
__global__ void __launch_bounds__(128) ssm_seams_kernel(const SsmP a, int N) {
    const long long per = (long long)a.D * N / 4;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    if (id >= per * a.q.S) return;
    const int s = (int)(id / per);
    const long long e = id % per * 4, c = e / N;   // state within [D][N]
    const long long len = a.q.hi(s) - a.q.lo(s);
    const int count = len > 0 ? (int)((len + a.L - 1) / a.L) : 1;
    const long long slot0 = first_slot(a.q, s, a.L), all = (long long)a.D * N;
    float A2[4];
    load_f32<float, 4>(a.A + e, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
    if (blockIdx.y == 0) {
        float h[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.h0) load_f32<float, 4>(a.h0 + s * all + e, h);
        for (int k = 0; k < count - 1; ++k) {
            float *p = a.hst + (slot0 + k) * all + e, end[4];
            load_f32<float, 4>(p, end);
            const float d = a.sdel[(slot0 + k) * a.D + c];
            store_f32<float, 4>(p, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fmaf(ex2(A2[i] * d), h[i], end[i]);
        }
        store_f32<float, 4>(a.hst + (slot0 + count - 1) * all + e, h);
    } else {
        float g[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.dh_T) load_f32<float, 4>(a.dh_T + s * all + e, g);
        for (int k = count - 1; k >= 0; --k) {
            float *p = a.gst + (slot0 + k) * all + e, own[4] = {0.f, 0.f, 0.f, 0.f};
            const bool on = len > 0 && (k > 0 || a.dh0);   // the others are not read, nor were they written
            float d = 0.f;
            if (on) {
                load_f32<float, 4>(p, own);
                d = a.sdel[(slot0 + k) * a.D + c];
            }
            store_f32<float, 4>(p, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = fmaf(ex2(A2[i] * d), g[i], own[i]);
        }
        if (a.dh0) store_f32<float, 4>(a.dh0 + s * all + e, g);
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(128) ssm_step_kernel(const SsmP a) {
    constexpr int NQ = N / 4;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long unit = id / NQ;
    const int q = (int)(id % NQ);
    const bool live = unit < (long long)a.q.S * a.D;
    const long long s = live ? unit / a.D : 0;
    const int c = live ? (int)(unit % a.D) : 0;
    const long long at = (s * a.D + c) * N + 4 * q;
    float h[4], A[4], B[4], C[4];
    load_f32<float, 4>(a.h0 + at, h);
    load_f32<float, 4>(a.A + (long long)c * N + 4 * q, A);
    const int g = c / a.Dg;
    const T *pb = (const T *)a.Bm + s * a.ld_B + g * N + 4 * q, *pc = (const T *)a.Cm + s * a.ld_C + g * N + 4 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        B[i] = to_f32(pb[i]);
        C[i] = to_f32(pc[i]);
    }
    const float u = to_f32(((const T *)a.u)[s * a.ld_u + c]);
    float d = to_f32(((const T *)a.dt)[s * a.ld_dt + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
    if (a.softplus) d = softplus_f32(d);
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(ex2(d * (A[i] * kLog2e)), h[i], d * u * B[i]);
        y = fmaf(C[i], h[i], y);
    }
#pragma unroll
    for (int o = NQ / 2; o >= 1; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!live) return;
    store_f32<float, 4>(a.h_T + at, h);
    if (q == 0) {
        if (a.Dskip) y = fmaf(a.Dskip[c], u, y);
        if (a.z) y *= silu_f32(to_f32(((const T *)a.z)[s * a.ld_z + c]));
        ((T *)a.out)[s * a.ld_out + c] = from_f32<T>(y);
    }
}

// Rows a span of the forward takes: whole sequences where their blocks give each SM one,
// otherwise spans for three blocks a SM.  Packed sequences' lengths are not known here: a span
// holds twice the mean, so that even ones stay whole and a long one among short ones is cut.
int fwd_span(const SsmArgs &a) {
    const int CH = 4 * kSsmThreads / a.N, Dg = a.D / a.G;
    const long long per_span = (long long)a.G * ((Dg + CH - 1) / CH);
    const long long want = 444 / per_span;   // spans in all
    const long long longest = a.T > 0 ? a.T : 1;
    long long L;
    if (a.cu) {
        const long long n = want > a.S ? want : a.S;
        L = n > 1 ? (2 * a.rows + n - 1) / n : longest;
    } else {
        if (want <= 1 || per_span * a.S >= 148) return (int)longest;
        L = (a.rows + want - 1) / want;
    }
    L = (L + kTile - 1) / kTile * kTile;
    if (L < 64) L = 64;
    return (int)(L < longest ? L : longest);
}

template <typename T, int N>
cudaError_t run_fwd(const SsmArgs &a, cudaStream_t st) {
    SsmP p = ssm_params<N>(a, fwd_span(a));
    const long long blocks = p.slots * p.nblk;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.L < a.T) {
        p.hst = (float *)a.workspace;
        p.sdel = p.hst + p.slots * a.D * N;
        a.marks->mark(st);
        ssm_fwd_kernel<T, N, true><<<(unsigned)blocks, kSsmThreads, 0, st>>>(p);
        a.marks->mark(st);
        const cudaError_t e = launch_ssm_seams(p, N, st);
        if (e != cudaSuccess) return e;
    }
    a.marks->mark(st);
    ssm_fwd_kernel<T, N, false><<<(unsigned)blocks, kSsmThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, int N>
cudaError_t run_step(const SsmArgs &a, cudaStream_t st) {
    const SsmP p = ssm_params<N>(a, 1);
    const long long blocks = ((long long)a.S * a.D * (N / 4) + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    a.marks->mark(st);
    ssm_step_kernel<T, N><<<(unsigned)blocks, 128, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T>
cudaError_t dispatch(const SsmArgs &a, bool step, cudaStream_t st) {
    switch (a.N) {
        case 8: return step ? run_step<T, 8>(a, st) : run_fwd<T, 8>(a, st);
        case 16: return step ? run_step<T, 16>(a, st) : run_fwd<T, 16>(a, st);
        case 32: return step ? run_step<T, 32>(a, st) : run_fwd<T, 32>(a, st);
        default: return step ? run_step<T, 64>(a, st) : run_fwd<T, 64>(a, st);
    }
}

}  // namespace

cudaError_t launch_ssm_seams(const SsmP &p, int N, cudaStream_t st) {
    const long long blocks = ((long long)p.D * N / 4 * p.q.S + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    ssm_seams_kernel<<<dim3((unsigned)blocks, p.gst ? 2 : 1), 128, 0, st>>>(p, N);
    return cudaGetLastError();
}

size_t ssm_scan_fwd_workspace_bytes(const SsmArgs &a) {
    const int L = fwd_span(a);
    if (L >= a.T) return 0;
    return (size_t)span_slots(a.cu != nullptr, a.S, a.T, L) * a.D * (a.N + 1) * sizeof(float);
}
cudaError_t launch_ssm_scan_fwd(const SsmArgs &a, cudaStream_t st) {
    return a.bf16 ? dispatch<__nv_bfloat16>(a, false, st) : dispatch<float>(a, false, st);
}
cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st) {
    return a.bf16 ? dispatch<__nv_bfloat16>(a, true, st) : dispatch<float>(a, true, st);
}

}  // namespace kda
