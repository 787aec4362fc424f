// kda_block_norm.cu -- the norms behind one block and ahead of the next, with the block's gate,
// its residual scale and the residual sum between them.
//
//   n = b / sqrt(mean b^2 + eps),  r' = r + scale p n w_post  (p = sigmoid(gate)),
//   m = r' / sqrt(mean r'^2 + eps),  x = m w_pre
// backward, from r' as stored, b and the gate:
//   dr = dr' + rr (dm - m mean(dm m))        dm = dx w_pre, rr = 1 / sqrt(mean r'^2 + eps)
//   db = rb (dn - n mean(dn n))              dn = dr scale p w_post
//   dgate = dr scale n w_post p (1 - p)
//   dw_pre = sum dx m,  dscale = w_post sum dr p n,  dw_post = scale sum dr p n   (over rows)
//
// Bound by HBM: 5 values a place forward (b, r, gate in; r', x out), 8 backward.  A block holds a
// row in registers, so every value is read once; the sums of a row go through warp shuffles and one
// exchange in shared memory.  Blocks walk the rows, the next row's loads under way while one is
// computed, with the weights of their columns in registers.  16384 x 2048 in bf16 with a
// gate: forward 59 us (5.7 TB/s), backward 119 us (4.5 TB/s, 112 with 1 - p as a
// difference, which loses dgate's precision where the gate is open; issue slots 65 % taken).
#include "kda_layers_internal.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

struct NormP {
    const void *residual, *block, *gate;
    const float *scale, *w_post, *w_pre;
    void *res_out, *x;
    const void *dres, *dx;
    void *dresidual, *dblock, *dgate;
    float *part;          // [grid][2][D]: sums of dr p n and of dx m
    int rows, D;
    float eps, inv_d;
    long long ld_res, ld_block, ld_gate;
};

// Sums over the block; buf: K x 32 floats that no other thread still reads.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (*buf)[32]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < warps ? buf[k][lane] : 0.f);
}

// w[c ..] * v[c ..], NULL = ones
template <int V>
__device__ __forceinline__ void load_weights(const float *w, const float *v, int c, float *out) {
    float f[V];
    if (w) load_f32<float, V>(w + c, out);
    if (v) load_f32<float, V>(v + c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (w ? out[i] : 1.f) * (v ? f[i] : 1.f);
}

// 1 / sqrt: the hardware's estimate and one Newton step, for fp32 rows
__device__ __forceinline__ float inv_sqrt(float x) {
    const float y = rsqrtf(x);
    return isinf(y) || y == 0.f ? y : y * fmaf(-0.5f * x * y, y, 1.5f);
}

// p = sigmoid(x) and 1 - p, which for x > 0 is e^-x p: the difference would keep the absolute error of p only
__device__ __forceinline__ void gate_of(float x, float &p, float &rest) {
    const float e = ex2(-kLog2e * x);
    p = rcp(1.f + e);
    rest = x > 0.f ? e * p : 1.f - p;
}

// A thread's columns: vectors threadIdx.x, + blockDim.x, ... of V.
template <int V>
__device__ __forceinline__ int column(int e) { return (e * (int)blockDim.x + (int)threadIdx.x) * V; }

template <typename T, int V, int E>
__device__ __forceinline__ void load_cols(Raw<T, V> (&r)[E], const void *p, long long row, long long ld, int D) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = column<V>(e);
        if (p && c < D) {
            r[e] = load_raw<T, V>((const T *)p + row * ld + c);
        } else {
#pragma unroll
            for (int i = 0; i < Raw<T, V>::kWords; ++i) r[e].w[i] = 0u;
        }
    }
}

template <typename T, int V, int E, int NT>
__global__ void __launch_bounds__(NT) block_norm_fwd_kernel(const NormP a) {
    __shared__ float buf[2][1][32];
    const int D = a.D;
    float ws[E][V], wx[E][V];
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (column<V>(e) < D) {
            load_weights<V>(a.w_post, a.scale, column<V>(e), ws[e]);
            load_weights<V>(a.w_pre, nullptr, column<V>(e), wx[e]);
        }
    Raw<T, V> nr[E], nb[E], ng[E];
    auto fetch = [&](long long row) {
        load_cols<T, V, E>(nb, a.block, row, a.ld_block, D);
        load_cols<T, V, E>(nr, a.residual, row, a.ld_res, D);
        load_cols<T, V, E>(ng, a.gate, row, a.ld_gate, D);
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float v[E][V], r[E][V], g[E][V];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            widen<T, V>(nr[e], r[e]);
            widen<T, V>(nb[e], v[e]);
            widen<T, V>(ng[e], g[e]);
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float ss[1] = {0.f};
        if (a.block) {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i) ss[0] = fmaf(v[e][i], v[e][i], ss[0]);
            block_sum<1>(ss, buf[0]);
            const float inv = inv_sqrt(fmaf(ss[0], a.inv_d, a.eps));
            ss[0] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float p = a.gate ? sigmoid_f32(g[e][i]) : 1.f;
                        r[e][i] = fmaf(v[e][i] * inv, ws[e][i] * p, r[e][i]);
                        ss[0] = fmaf(r[e][i], r[e][i], ss[0]);
                    }
                    store_f32<T, V>((T *)a.res_out + row * D + column<V>(e), r[e]);
                }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i) ss[0] = fmaf(r[e][i], r[e][i], ss[0]);
        }
        if (a.x) {
            block_sum<1>(ss, buf[1]);
            const float inv = inv_sqrt(fmaf(ss[0], a.inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
#pragma unroll
                    for (int i = 0; i < V; ++i) r[e][i] *= inv * wx[e][i];
                    store_f32<T, V>((T *)a.x + row * D + column<V>(e), r[e]);
                }
        }
        // with one sum a row, its exchange buffer is written again one row on
        if (!(a.block && a.x)) __syncthreads();
    }
}

// The columns' sums over a block's rows stay with the thread that owns the columns and leave once, to
// the block's place in the workspace.
template <typename T, int V, int E, int NT>
__global__ void __launch_bounds__(NT) block_norm_bwd_kernel(const NormP a) {
    __shared__ float buf[3][32], buf_n[1][32];
    const int D = a.D;
    float ws[E][V], wx[E][V], accq[E][V], accm[E][V];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (column<V>(e) < D) {
            load_weights<V>(a.w_post, a.scale, column<V>(e), ws[e]);
            load_weights<V>(a.w_pre, nullptr, column<V>(e), wx[e]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) accq[e][i] = accm[e][i] = 0.f;
    }
    Raw<T, V> nr[E], nb[E], ng[E], ndr[E], ndx[E];
    auto fetch = [&](long long row) {
        load_cols<T, V, E>(nr, a.dx ? a.residual : nullptr, row, a.ld_res, D);
        load_cols<T, V, E>(ndx, a.dx, row, D, D);
        load_cols<T, V, E>(nb, a.block, row, a.ld_block, D);
        load_cols<T, V, E>(ng, a.gate, row, a.ld_gate, D);
        load_cols<T, V, E>(ndr, a.dres, row, D, D);
    };
    if (blockIdx.x < a.rows) fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Raw<T, V> qr[E], qb[E], qg[E], qdr[E], qdx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qr[e] = nr[e];
            qb[e] = nb[e];
            qg[e] = ng[e];
            qdr[e] = ndr[e];
            qdx[e] = ndx[e];
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float s[3] = {0.f, 0.f, 0.f};   // sums of r'^2, of dx w_pre r', of b^2
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (column<V>(e) < D) {
                float r[V], d[V], b[V];
                widen<T, V>(qr[e], r);
                widen<T, V>(qdx[e], d);
                widen<T, V>(qb[e], b);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[0] = fmaf(r[i], r[i], s[0]);
                    s[1] = fmaf(d[i] * wx[e][i], r[i], s[1]);
                    s[2] = fmaf(b[i], b[i], s[2]);
                }
            }
        block_sum<3>(s, buf);
        const float inv_r = a.dx ? inv_sqrt(fmaf(s[0], a.inv_d, a.eps)) : 0.f;
        const float mean_m = s[1] * inv_r * a.inv_d;   // mean of dm m
        const float inv_b = inv_sqrt(fmaf(s[2], a.inv_d, a.eps));
        float dn[E][V], sn[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (column<V>(e) < D) {
                float r[V], d[V], b[V], g[V], dr[V];
                widen<T, V>(qr[e], r);
                widen<T, V>(qdx[e], d);
                widen<T, V>(qdr[e], dr);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float mi = r[i] * inv_r;
                    accm[e][i] = fmaf(d[i], mi, accm[e][i]);
                    dr[i] = fmaf(inv_r, fmaf(-mi, mean_m, d[i] * wx[e][i]), dr[i]);
                }
                store_f32<T, V>((T *)a.dresidual + row * D + column<V>(e), dr);
                if (a.block) {
                    widen<T, V>(qb[e], b);
                    widen<T, V>(qg[e], g);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float p = 1.f, rest = 0.f;
                        if (a.gate) gate_of(g[i], p, rest);
                        const float n = b[i] * inv_b, q = dr[i] * p * n;
                        dn[e][i] = dr[i] * p * ws[e][i];
                        sn[0] = fmaf(dn[e][i], n, sn[0]);
                        g[i] = q * ws[e][i] * rest;   // dgate
                        accq[e][i] += q;
                    }
                    if (a.gate) store_f32<T, V>((T *)a.dgate + row * D + column<V>(e), g);
                }
            }
        block_sum<1>(sn, buf_n);   // also between this row's reads of buf and the next one's writes
        if (a.block) {
            const float mean_n = sn[0] * a.inv_d;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
                    float b[V];
                    widen<T, V>(qb[e], b);
#pragma unroll
                    for (int i = 0; i < V; ++i) b[i] = inv_b * fmaf(-(b[i] * inv_b), mean_n, dn[e][i]);
                    store_f32<T, V>((T *)a.dblock + row * D + column<V>(e), b);
                }
        }
    }
    float *part = a.part + (long long)blockIdx.x * 2 * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (column<V>(e) < D)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[column<V>(e) + i] = accq[e][i];
                part[D + column<V>(e) + i] = accm[e][i];
            }
}

// ---------------------------------------------------------------- wide rows
// More columns than a thread's registers hold with the next row's and the weights: a row is read again
// for each of its passes, from L1 or L2, and only what a later pass cannot read stays (r' forward, dn
// backward); the columns' sums lie in shared memory, place i of thread t at [i][t].  3000 x 11184 in
// FP32: forward 174 us (3.9 TB/s), backward 307 (3.5); with the row held, and spilled, 510 and 664.
template <typename T, int V>
__device__ __forceinline__ void load_at(const void *p, long long row, long long ld, int c, float *x) {
    if (p) {
        load_f32<T, V>((const T *)p + row * ld + c, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.f;
    }
}

template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) block_norm_fwd_wide_kernel(const NormP a) {
    __shared__ float buf[2][1][32];
    const int D = a.D;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float r[E][V], ss[1] = {0.f}, inv = 0.f;
        if (a.block) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
                    float v[V];
                    load_at<T, V>(a.block, row, a.ld_block, column<V>(e), v);
#pragma unroll
                    for (int i = 0; i < V; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
                }
            block_sum<1>(ss, buf[0]);
            inv = inv_sqrt(fmaf(ss[0], a.inv_d, a.eps));
            ss[0] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<V>(e);
            if (c < D) {
                load_at<T, V>(a.residual, row, a.ld_res, c, r[e]);
                if (a.block) {
                    float v[V], g[V], w[V];
                    load_at<T, V>(a.block, row, a.ld_block, c, v);
                    load_at<T, V>(a.gate, row, a.ld_gate, c, g);
                    load_weights<V>(a.w_post, a.scale, c, w);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        r[e][i] = fmaf(v[i] * inv, w[i] * (a.gate ? sigmoid_f32(g[i]) : 1.f), r[e][i]);
                    store_f32<T, V>((T *)a.res_out + row * D + c, r[e]);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) ss[0] = fmaf(r[e][i], r[e][i], ss[0]);
            }
        }
        if (a.x) {
            block_sum<1>(ss, buf[1]);
            inv = inv_sqrt(fmaf(ss[0], a.inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
                    float w[V];
                    load_weights<V>(a.w_pre, nullptr, column<V>(e), w);
#pragma unroll
                    for (int i = 0; i < V; ++i) r[e][i] *= inv * w[i];
                    store_f32<T, V>((T *)a.x + row * D + column<V>(e), r[e]);
                }
        }
        // with one sum a row, its exchange buffer is written again one row on
        if (!(a.block && a.x)) __syncthreads();
    }
}

template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) block_norm_bwd_wide_kernel(const NormP a) {
    __shared__ float buf[3][32], buf_n[1][32];
    extern __shared__ __align__(16) float acc[];   // [2][E V][blockDim.x]
    constexpr int EV = E * V;
    const int D = a.D, nt = blockDim.x, tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2 * EV; ++i) acc[i * nt + tid] = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float s[3] = {0.f, 0.f, 0.f};   // sums of r'^2, of dx w_pre r', of b^2
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<V>(e);
            if (c < D) {
                float r[V], d[V], b[V], w[V];
                load_at<T, V>(a.dx ? a.residual : nullptr, row, a.ld_res, c, r);
                load_at<T, V>(a.dx, row, D, c, d);
                load_at<T, V>(a.block, row, a.ld_block, c, b);
                load_weights<V>(a.w_pre, nullptr, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[0] = fmaf(r[i], r[i], s[0]);
                    s[1] = fmaf(d[i] * w[i], r[i], s[1]);
                    s[2] = fmaf(b[i], b[i], s[2]);
                }
            }
        }
        block_sum<3>(s, buf);
        const float inv_r = a.dx ? inv_sqrt(fmaf(s[0], a.inv_d, a.eps)) : 0.f;
        const float mean_m = s[1] * inv_r * a.inv_d;   // mean of dm m
        const float inv_b = inv_sqrt(fmaf(s[2], a.inv_d, a.eps));
        float dn[E][V], sn[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<V>(e);
            if (c < D) {
                float r[V], d[V], w[V], dr[V];
                load_at<T, V>(a.dx ? a.residual : nullptr, row, a.ld_res, c, r);
                load_at<T, V>(a.dx, row, D, c, d);
                load_at<T, V>(a.dres, row, D, c, dr);
                load_weights<V>(a.w_pre, nullptr, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float mi = r[i] * inv_r;
                    acc[(EV + e * V + i) * nt + tid] += d[i] * mi;
                    dr[i] = fmaf(inv_r, fmaf(-mi, mean_m, d[i] * w[i]), dr[i]);
                }
                store_f32<T, V>((T *)a.dresidual + row * D + c, dr);
                if (a.block) {
                    float b[V], g[V];
                    load_at<T, V>(a.block, row, a.ld_block, c, b);
                    load_at<T, V>(a.gate, row, a.ld_gate, c, g);
                    load_weights<V>(a.w_post, a.scale, c, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float p = 1.f, rest = 0.f;
                        if (a.gate) gate_of(g[i], p, rest);
                        const float n = b[i] * inv_b, q = dr[i] * p * n;
                        dn[e][i] = dr[i] * p * w[i];
                        sn[0] = fmaf(dn[e][i], n, sn[0]);
                        g[i] = q * w[i] * rest;   // dgate
                        acc[(e * V + i) * nt + tid] += q;
                    }
                    if (a.gate) store_f32<T, V>((T *)a.dgate + row * D + c, g);
                }
            }
        }
        block_sum<1>(sn, buf_n);   // also between this row's reads of buf and the next one's writes
        if (a.block) {
            const float mean_n = sn[0] * a.inv_d;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (column<V>(e) < D) {
                    float b[V];
                    load_at<T, V>(a.block, row, a.ld_block, column<V>(e), b);
#pragma unroll
                    for (int i = 0; i < V; ++i) b[i] = inv_b * fmaf(-(b[i] * inv_b), mean_n, dn[e][i]);
                    store_f32<T, V>((T *)a.dblock + row * D + column<V>(e), b);
                }
        }
    }
    float *part = a.part + (long long)blockIdx.x * 2 * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (column<V>(e) < D)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[column<V>(e) + i] = acc[(e * V + i) * nt + tid];
                part[D + column<V>(e) + i] = acc[(EV + e * V + i) * nt + tid];
            }
}

// The blocks' sums, 32 columns of [2][D] a block, in a fixed order.
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const float *__restrict__ part, int count, int D,
                                                              const float *scale, const float *w_post, float *dscale,
                                                              float *dw_post, float *dw_pre) {
    __shared__ float s[32][33];
    const int i = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (i < 2 * D)
        for (int k = threadIdx.y; k < count; k += 32) v += part[(long long)k * 2 * D + i];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(s[threadIdx.x][threadIdx.y]);
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < 2 * D) {
        if (o >= D) {
            if (dw_pre) dw_pre[o - D] = v;
        } else {
            if (dscale) dscale[o] = w_post ? v * w_post[o] : v;
            if (dw_post) dw_post[o] = scale ? v * scale[o] : v;
        }
    }
}

NormP params(const NormArgs &a) {
    NormP p;
    p.residual = a.residual; p.block = a.block; p.gate = a.gate;
    p.scale = a.scale; p.w_post = a.w_post; p.w_pre = a.w_pre;
    p.res_out = a.res_out; p.x = a.x; p.dres = a.dres; p.dx = a.dx;
    p.dresidual = a.dresidual; p.dblock = a.dblock; p.dgate = a.dgate;
    p.part = (float *)a.workspace;
    p.rows = a.rows; p.D = a.D; p.eps = a.eps; p.inv_d = 1.f / (float)a.D;
    p.ld_res = a.ld_res; p.ld_block = a.ld_block; p.ld_gate = a.ld_gate;
    return p;
}

int threads(int D, int per) { return ((D + per - 1) / per + 31) / 32 * 32; }

// Blocks: enough for `want` threads on each of 148 SMs, and no more than rows.
int grid(int rows, int nt, int want) {
    const int k = want / nt;
    const long long n = 148LL * (k < 1 ? 1 : k > 24 ? 24 : k);
    return rows < n ? rows : (int)n;
}
// 16384 x 2048 in bf16, at 512, 768, 1024 and 1536: forward 68, 59, 72 and 60 us, backward 119, 134, 126 and
// 133.  2^25 values of other widths, forward at 768: 1024 columns 57 (67 at 512, 70 at 1024), 2048 in FP32 115 (104
// at 512), 2560 66 and 4096 76 (59 each at 1024: `want / nt` rounded down leaves an SM 640 and 512 threads at
// 768); backward at 512: 1024 columns 118 (131 at 768), 2560 156 (161), 1028 in FP32 257 (206), 1002 in bf16 190 (172).
constexpr int kFwdWant = 768, kBwdWant = 512;

template <typename T, int V, int E, int NT, bool WIDE = false>
cudaError_t launch(const NormArgs &a, bool bwd, cudaStream_t st) {
    // the most registers: forward with the next row's loads under way, backward with the columns' sums too
    constexpr bool FWD = (V * E <= 8 && !WIDE) || (NT <= 512 && V * E * (int)sizeof(T) <= 32), BWD = V * E <= 8 && NT <= 512;
    const int nt = threads(a.D, V * E);
    const NormP p = params(a);
    a.marks->mark(st);
    if (!bwd) {
        const int n = grid(a.rows, nt, kFwdWant);
        if (n > 0) {
            if constexpr (FWD) block_norm_fwd_kernel<T, V, E, NT><<<n, nt, 0, st>>>(p);
            else block_norm_fwd_wide_kernel<T, V, E><<<n, nt, 0, st>>>(p);
        }
        return cudaGetLastError();
    }
    const int n = grid(a.rows, nt, kBwdWant);
    if constexpr (BWD) {
        if (n > 0) block_norm_bwd_kernel<T, V, E, NT><<<n, nt, 0, st>>>(p);
    } else {
        const int smem = 2 * V * E * nt * (int)sizeof(float);
        // The limit is kept per kernel for all host threads: every call sets the same one, that of 1024
        // threads, and a call of fewer cannot take it away from another's launch.
        constexpr int most = 2 * V * E * 1024 * (int)sizeof(float);
        const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_wide_kernel<T, V, E>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        if (n > 0) block_norm_bwd_wide_kernel<T, V, E><<<n, nt, smem, st>>>(p);
    }
    a.marks->mark(st);
    if (a.dscale || a.dw_post || a.dw_pre)
        block_norm_sum_kernel<<<(2 * a.D + 31) / 32, dim3(32, 32), 0, st>>>(p.part, n, a.D, a.scale, a.w_post,
                                                                            a.dscale, a.dw_post, a.dw_pre);
    return cudaGetLastError();
}

// E: vectors a thread; NT: the most threads that may make of a block, which sets the registers a
// thread has.  A row of few has an SM to itself: all the threads that the registers allow.
// Forward / backward in us, 2^25 values with a gate, and what the neighbouring choice takes:
//   one vector a thread, up to 256 of them    FP32, 512 columns: 107 / 183, 8 values 116 / 217; bf16 on vectors
//                                             of 4, 516: 100 / 201, where 8 values take 85 / 189
//   4 values on vectors of 1 or 2, to 1024    bf16, 1001: 140 / 282, 8 values 171 / 287
//   8 values, registers of 256 threads, 2048  FP32, 2048: 115 / 198, of 512 threads 119 / 204
//   8 values, of 512 threads, 4096            FP32, 4096: 106 / 203, of 1024 threads 127 / 359
//   16 values of 512, bf16 forward, 8192      8192: 59, 8 values of 1024 threads 64, wide 119
//   8 values, wide, 8192                      FP32, 8192, backward 255, 16 values 347; forward 146, where the row
//                                             held in registers takes 124 (bf16 on vectors of 4, 4100: 234 and 93)
//   16 values, wide, all that is left         FP32, 16384: 139 / 250
// Up to 148 rows a call is short either way: 148 x 2048 in FP32 4.6 / 10.3 with all threads, 5.0 / 10.6 with
// those of many rows; 148 x 3001 8.3 / 16.5, and 6.2 / 12.7 with those.
template <typename T, int V>
cudaError_t launch_v(const NormArgs &a, bool bwd, cudaStream_t st) {
    constexpr int E = 8 / V;
    const int D = a.D;
    const bool few = a.rows <= 148;
    if (D <= 256 * V && E > 1 && !(few && D > 1024)) return launch<T, V, 1, 256>(a, bwd, st);
    if constexpr (V <= 2)
        if (D <= 1024) return launch<T, V, 4 / V, 256>(a, bwd, st);
    if (few && D > 1024 && D <= 1024 * V) return launch<T, V, 1, 1024>(a, bwd, st);
    if (few && D > 2048 && D <= 8192) return launch<T, V, E, 1024>(a, bwd, st);
    if (D <= 2048) return launch<T, V, E, 256>(a, bwd, st);
    if (D <= 4096) return launch<T, V, E, 512>(a, bwd, st);
    if constexpr (V == 8)
        if (!bwd && D <= 8192) return launch<T, V, 2 * E, 512>(a, bwd, st);
    if (D <= 8192) return launch<T, V, E, 1024, true>(a, bwd, st);
    return launch<T, V, 2 * E, 1024>(a, bwd, st);
}

// V: the widest vectors, up to 16 bytes, that the width, the row strides and the addresses allow: 8184 x
// 4100 in bf16 takes 235 us forward and 320 backward on vectors of 4, 526 and 1515 on single values.
cudaError_t dispatch(const NormArgs &a, bool bwd, cudaStream_t st) {
    using B = __nv_bfloat16;
    const long long all = a.D | a.ld_res | a.ld_block | a.ld_gate | elements(a.residual, a.bf16) |
                          elements(a.block, a.bf16) | elements(a.gate, a.bf16);
    if (a.bf16) {
        if (all % 8 == 0) return launch_v<B, 8>(a, bwd, st);
        if (all % 4 == 0) return launch_v<B, 4>(a, bwd, st);
        if (all % 2 == 0) return launch_v<B, 2>(a, bwd, st);
        return launch_v<B, 1>(a, bwd, st);
    }
    if (all % 4 == 0) return launch_v<float, 4>(a, bwd, st);
    if (all % 2 == 0) return launch_v<float, 2>(a, bwd, st);
    return launch_v<float, 1>(a, bwd, st);
}

}  // namespace

// Whichever of the variants runs (a block has at least D / 16 threads, of 32): not the addresses,
// which the workspace's size cannot depend on.
size_t block_norm_bwd_workspace_bytes(int rows, int D) {
    return (size_t)grid(rows, threads(D, 16), kBwdWant) * 2 * D * sizeof(float);
}
cudaError_t launch_block_norm_fwd(const NormArgs &a, cudaStream_t st) { return dispatch(a, false, st); }
cudaError_t launch_block_norm_bwd(const NormArgs &a, cudaStream_t st) { return dispatch(a, true, st); }

}  // namespace kda
