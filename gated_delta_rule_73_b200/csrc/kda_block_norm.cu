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
// gate: forward 59 us (5.7 TB/s), backward 112 us (4.8 TB/s; issue slots 67 % taken).
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

// The columns' sums over a block's rows stay with the thread that owns the columns, in registers
// (REG) or in shared memory (place i of thread t at [i][t]), and leave once, to the block's place in
// the workspace.
template <typename T, int V, int E, int NT, bool REG>
__global__ void __launch_bounds__(NT) block_norm_bwd_kernel(const NormP a) {
    __shared__ float buf[3][32], buf_n[1][32];
    extern __shared__ __align__(16) float acc[];   // without REG: [2][E V][blockDim.x]
    constexpr int EV = E * V;
    const int D = a.D, nt = blockDim.x, tid = threadIdx.x;
    float ws[REG ? E : 1][V], wx[REG ? E : 1][V], accq[REG ? EV : 1], accm[REG ? EV : 1];
    auto weights = [&](int e, float *s, float *x) {
        load_weights<V>(a.w_post, a.scale, column<V>(e), s);
        load_weights<V>(a.w_pre, nullptr, column<V>(e), x);
    };
    if (REG) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (column<V>(e) < D) weights(e, ws[REG ? e : 0], wx[REG ? e : 0]);
    }
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        if (REG) accq[REG ? i : 0] = accm[REG ? i : 0] = 0.f;
        else acc[i * nt + tid] = acc[(EV + i) * nt + tid] = 0.f;
    }
    auto add = [&](int i, float q, float m) {
        if (REG) {
            accq[REG ? i : 0] += q;
            accm[REG ? i : 0] += m;
        } else {
            acc[i * nt + tid] += q;
            acc[(EV + i) * nt + tid] += m;
        }
    };
    Raw<T, V> nr[E], nb[E], ng[E], ndr[E], ndx[E];
    auto fetch = [&](long long row) {
        load_cols<T, V, E>(nr, a.dx ? a.residual : nullptr, row, a.ld_res, D);
        load_cols<T, V, E>(ndx, a.dx, row, D, D);
        load_cols<T, V, E>(nb, a.block, row, a.ld_block, D);
        load_cols<T, V, E>(ng, a.gate, row, a.ld_gate, D);
        load_cols<T, V, E>(ndr, a.dres, row, D, D);
    };
    if (REG && blockIdx.x < a.rows) fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!REG) fetch(row);
        Raw<T, V> qr[E], qb[E], qg[E], qdr[E], qdx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qr[e] = nr[e];
            qb[e] = nb[e];
            qg[e] = ng[e];
            qdr[e] = ndr[e];
            qdx[e] = ndx[e];
        }
        if (REG && row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float s[3] = {0.f, 0.f, 0.f};   // sums of r'^2, of dx w_pre r', of b^2
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (column<V>(e) < D) {
                float r[V], d[V], b[V], w[V], v[V];
                widen<T, V>(qr[e], r);
                widen<T, V>(qdx[e], d);
                widen<T, V>(qb[e], b);
                if (!REG) weights(e, v, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[0] = fmaf(r[i], r[i], s[0]);
                    s[1] = fmaf(d[i] * (REG ? wx[REG ? e : 0][i] : w[i]), r[i], s[1]);
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
                float r[V], d[V], b[V], g[V], w[V], v[V], dr[V], q[V], m[V];
                widen<T, V>(qr[e], r);
                widen<T, V>(qdx[e], d);
                widen<T, V>(qdr[e], dr);
                if (!REG) weights(e, v, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float wi = REG ? wx[REG ? e : 0][i] : w[i], mi = r[i] * inv_r;
                    m[i] = d[i] * mi;
                    q[i] = 0.f;
                    dr[i] = fmaf(inv_r, fmaf(-mi, mean_m, d[i] * wi), dr[i]);
                }
                store_f32<T, V>((T *)a.dresidual + row * D + column<V>(e), dr);
                if (a.block) {
                    widen<T, V>(qb[e], b);
                    widen<T, V>(qg[e], g);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float n = b[i] * inv_b, wi = REG ? ws[REG ? e : 0][i] : v[i];
                        const float p = a.gate ? sigmoid_f32(g[i]) : 1.f;
                        q[i] = dr[i] * p * n;
                        dn[e][i] = dr[i] * p * wi;
                        sn[0] = fmaf(dn[e][i], n, sn[0]);
                        g[i] = q[i] * wi * (1.f - p);   // dgate
                    }
                    if (a.gate) store_f32<T, V>((T *)a.dgate + row * D + column<V>(e), g);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) add(e * V + i, q[i], m[i]);
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
                const int k = e * V + i, c = column<V>(e) + i;
                part[c] = REG ? accq[REG ? k : 0] : acc[k * nt + tid];
                part[D + c] = REG ? accm[REG ? k : 0] : acc[(EV + k) * nt + tid];
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
// 16384 x 2048 in bf16: forward 58 us at 768, 71 at 1024, 59 at 1536; backward 108 at 512, 118 at 768
constexpr int kFwdWant = 768, kBwdWant = 512;

template <typename T, int V, int E, int NT>
cudaError_t launch(const NormArgs &a, bool bwd, cudaStream_t st) {
    constexpr bool REG = V * E <= 8 && NT <= 512;
    const int nt = threads(a.D, V * E);
    const NormP p = params(a);
    a.marks->mark(st);
    if (!bwd) {
        if (a.rows > 0) block_norm_fwd_kernel<T, V, E, NT><<<grid(a.rows, nt, kFwdWant), nt, 0, st>>>(p);
        return cudaGetLastError();
    }
    const size_t smem = REG ? 0 : (size_t)2 * V * E * nt * sizeof(float);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_kernel<T, V, E, NT, REG>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int n = grid(a.rows, nt, kBwdWant);
    if (n > 0) block_norm_bwd_kernel<T, V, E, NT, REG><<<n, nt, smem, st>>>(p);
    a.marks->mark(st);
    if (a.dscale || a.dw_post || a.dw_pre)
        block_norm_sum_kernel<<<(2 * a.D + 31) / 32, dim3(32, 32), 0, st>>>(p.part, n, a.D, a.scale, a.w_post,
                                                                            a.dscale, a.dw_post, a.dw_pre);
    return cudaGetLastError();
}

// V: 16 bytes where the width, the row strides and the addresses allow them.  E: vectors a thread;
// NT: the most threads that may make of a block, which sets the registers a thread has.
cudaError_t dispatch(const NormArgs &a, bool bwd, cudaStream_t st) {
    using B = __nv_bfloat16;
    const long long all = a.D | a.ld_res | a.ld_block | a.ld_gate | elements(a.residual, a.bf16) |
                          elements(a.block, a.bf16) | elements(a.gate, a.bf16);
    const int D = a.D;
    const bool few = a.rows <= 148;   // a row has an SM to itself: all the threads that the registers allow
    if (a.bf16 && all % 8 == 0) {
        if (few && D > 2048 && D <= 8192) return launch<B, 8, 1, 1024>(a, bwd, st);
        if (D <= 2048) return launch<B, 8, 1, 256>(a, bwd, st);
        if (D <= 4096) return launch<B, 8, 1, 512>(a, bwd, st);
        if (D <= 8192) return launch<B, 8, 2, 512>(a, bwd, st);
        return launch<B, 8, 2, 1024>(a, bwd, st);
    }
    if (!a.bf16 && all % 4 == 0) {
        if (few && D > 1024 && D <= 4096) return launch<float, 4, 1, 1024>(a, bwd, st);
        if (D <= 1024) return launch<float, 4, 1, 256>(a, bwd, st);
        if (D <= 2048) return launch<float, 4, 2, 256>(a, bwd, st);
        if (D <= 4096) return launch<float, 4, 2, 512>(a, bwd, st);
        if (D <= 8192) return launch<float, 4, 4, 512>(a, bwd, st);
        return launch<float, 4, 4, 1024>(a, bwd, st);
    }
    if (a.bf16) {
        if (few && D > 1024 && D <= 8192) return launch<B, 1, 8, 1024>(a, bwd, st);
        if (D <= 256) return launch<B, 1, 1, 256>(a, bwd, st);
        if (D <= 1024) return launch<B, 1, 4, 256>(a, bwd, st);
        if (D <= 4096) return launch<B, 1, 8, 512>(a, bwd, st);
        if (D <= 8192) return launch<B, 1, 16, 512>(a, bwd, st);
        return launch<B, 1, 16, 1024>(a, bwd, st);
    }
    if (few && D > 1024 && D <= 8192) return launch<float, 1, 8, 1024>(a, bwd, st);
    if (D <= 256) return launch<float, 1, 1, 256>(a, bwd, st);
    if (D <= 1024) return launch<float, 1, 4, 256>(a, bwd, st);
    if (D <= 4096) return launch<float, 1, 8, 512>(a, bwd, st);
    if (D <= 8192) return launch<float, 1, 16, 512>(a, bwd, st);
    return launch<float, 1, 16, 1024>(a, bwd, st);
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
