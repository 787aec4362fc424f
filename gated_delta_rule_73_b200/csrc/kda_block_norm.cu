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
// Bound by HBM: 5 values a place forward (b, r, gate in; r', x out), 8 backward.  A block of
// threads holds a row in registers, so every value is read once; the sums of a row go through
// warp shuffles and one exchange in shared memory.
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

// Sum over the block; buf: 32 floats that no other thread still reads.
__device__ __forceinline__ float block_sum(float v, float *buf) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? buf[threadIdx.x & 31] : 0.f;
    return warp_sum(v);
}

template <int V>
__device__ __forceinline__ void load_weights(const float *w, int c, float *out) {
    if (w) {
        load_f32<float, V>(w + c, out);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 1.f;
    }
}

// 1 / sqrt: the hardware's estimate and one Newton step, for fp32 rows
__device__ __forceinline__ float inv_sqrt(float x) {
    const float y = rsqrtf(x);
    return isinf(y) || y == 0.f ? y : y * fmaf(-0.5f * x * y, y, 1.5f);
}

template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) block_norm_fwd_kernel(const NormP a) {
    __shared__ float buf[2][32];
    const long long row = blockIdx.x;
    const int nt = blockDim.x, D = a.D;
    const T *pr = (const T *)a.residual + row * a.ld_res;
    Raw<T, V> rr[E], rb[E], rg[E];
    float v[E][V];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * nt + threadIdx.x) * V;
        if (c < D) {
            rr[e] = load_raw<T, V>(pr + c);
            if (a.block) rb[e] = load_raw<T, V>((const T *)a.block + row * a.ld_block + c);
            if (a.gate) rg[e] = load_raw<T, V>((const T *)a.gate + row * a.ld_gate + c);
        } else {
            rr[e] = rb[e] = rg[e] = load_part<T, V>(pr, 0);
        }
    }
    if (a.block) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            widen<T, V>(rb[e], v[e]);
            if ((e * nt + threadIdx.x) * V < D)
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[e][i], v[e][i], ss);
        }
        const float inv = inv_sqrt(fmaf(block_sum(ss, buf[0]), a.inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * nt + threadIdx.x) * V;
            if (c < D) {
                float w[V], s[V], r[V], g[V];
                load_weights<V>(a.w_post, c, w);
                load_weights<V>(a.scale, c, s);
                widen<T, V>(rr[e], r);
                if (a.gate) {
                    widen<T, V>(rg[e], g);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] = sigmoid_f32(g[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] = 1.f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) v[e][i] = fmaf(v[e][i] * inv * w[i], s[i] * g[i], r[i]);
                if (a.res_out) store_f32<T, V>((T *)a.res_out + row * D + c, v[e]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) widen<T, V>(rr[e], v[e]);
    }
    if (!a.x) return;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if ((e * nt + threadIdx.x) * V < D)
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(v[e][i], v[e][i], ss);
    const float inv = inv_sqrt(fmaf(block_sum(ss, buf[1]), a.inv_d, a.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * nt + threadIdx.x) * V;
        if (c < D) {
            float w[V];
            load_weights<V>(a.w_pre, c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[e][i] *= inv * w[i];
            store_f32<T, V>((T *)a.x + row * D + c, v[e]);
        }
    }
}

// Rows blockIdx.x, + gridDim.x, ...: the columns' sums over them stay with the thread that owns
// the columns, in shared memory (two FP32 read-modify-writes a place against 16 bytes of HBM),
// and leave once, to the block's place in the workspace.
template <typename T, int V, int E>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(const NormP a) {
    __shared__ float buf[4][32];
    extern __shared__ __align__(16) float acc[];   // [2][D]
    const int nt = blockDim.x, D = a.D;
    float *accq = acc, *accm = acc + D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * nt + threadIdx.x) * V;
        if (c < D)
#pragma unroll
            for (int i = 0; i < V; ++i) accq[c + i] = accm[c + i] = 0.f;
    }
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Raw<T, V> q_r[E], q_b[E], q_g[E], q_dr[E], q_dx[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * nt + threadIdx.x) * V;
            q_r[e] = q_b[e] = q_g[e] = q_dr[e] = q_dx[e] = load_part<T, V>((const T *)a.residual, 0);
            if (c < D) {
                if (a.dx) {
                    q_r[e] = load_raw<T, V>((const T *)a.residual + row * a.ld_res + c);
                    q_dx[e] = load_raw<T, V>((const T *)a.dx + row * D + c);
                }
                if (a.block) q_b[e] = load_raw<T, V>((const T *)a.block + row * a.ld_block + c);
                if (a.gate) q_g[e] = load_raw<T, V>((const T *)a.gate + row * a.ld_gate + c);
                if (a.dres) q_dr[e] = load_raw<T, V>((const T *)a.dres + row * D + c);
            }
        }
        float s_r = 0.f, s_m = 0.f, s_b = 0.f;   // sums of r'^2, of dx w_pre r', of b^2
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * nt + threadIdx.x) * V;
            if (c < D) {
                float r[V], d[V], b[V], w[V];
                widen<T, V>(q_r[e], r);
                widen<T, V>(q_dx[e], d);
                widen<T, V>(q_b[e], b);
                load_weights<V>(a.w_pre, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s_r = fmaf(r[i], r[i], s_r);
                    s_m = fmaf(d[i] * w[i], r[i], s_m);
                    s_b = fmaf(b[i], b[i], s_b);
                }
            }
        }
        // three sums, one exchange
        s_r = warp_sum(s_r);
        s_m = warp_sum(s_m);
        s_b = warp_sum(s_b);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = nt >> 5;
        if (warps > 1) {
            if (lane == 0) {
                buf[0][warp] = s_r;
                buf[1][warp] = s_m;
                buf[2][warp] = s_b;
            }
            __syncthreads();
            s_r = warp_sum(lane < warps ? buf[0][lane] : 0.f);
            s_m = warp_sum(lane < warps ? buf[1][lane] : 0.f);
            s_b = warp_sum(lane < warps ? buf[2][lane] : 0.f);
        }
        const float inv_r = a.dx ? inv_sqrt(fmaf(s_r, a.inv_d, a.eps)) : 0.f;
        const float mean_m = s_m * inv_r * a.inv_d;   // mean of dm m
        const float inv_b = inv_sqrt(fmaf(s_b, a.inv_d, a.eps));
        float dn[E][V], s_n = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e * nt + threadIdx.x) * V;
            if (c < D) {
                float r[V], d[V], b[V], w[V], dr[V];
                widen<T, V>(q_r[e], r);
                widen<T, V>(q_dx[e], d);
                widen<T, V>(q_dr[e], dr);
                load_weights<V>(a.w_pre, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float m = r[i] * inv_r;
                    accm[c + i] += d[i] * m;
                    dr[i] = fmaf(inv_r, fmaf(-m, mean_m, d[i] * w[i]), dr[i]);
                }
                store_f32<T, V>((T *)a.dresidual + row * D + c, dr);
                if (a.block) {
                    float p[V], s[V], wp[V];
                    load_weights<V>(a.w_post, c, wp);
                    load_weights<V>(a.scale, c, s);
                    widen<T, V>(q_b[e], b);
                    if (a.gate) {
                        float dg[V];
                        widen<T, V>(q_g[e], p);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            p[i] = sigmoid_f32(p[i]);
                            dg[i] = dr[i] * s[i] * wp[i] * (b[i] * inv_b) * (p[i] * (1.f - p[i]));
                        }
                        store_f32<T, V>((T *)a.dgate + row * D + c, dg);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) p[i] = 1.f;
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float n = b[i] * inv_b, q = dr[i] * p[i];
                        accq[c + i] += q * n;
                        dn[e][i] = q * s[i] * wp[i];
                        s_n = fmaf(dn[e][i], n, s_n);
                    }
                }
            }
        }
        s_n = block_sum(s_n, buf[3]);   // also between this row's reads of buf[0..2] and the next one's writes
        if (a.block) {
            const float mean_n = s_n * a.inv_d;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = (e * nt + threadIdx.x) * V;
                if (c < D) {
                    float b[V];
                    widen<T, V>(q_b[e], b);
#pragma unroll
                    for (int i = 0; i < V; ++i) b[i] = inv_b * fmaf(-(b[i] * inv_b), mean_n, dn[e][i]);
                    store_f32<T, V>((T *)a.dblock + row * D + c, b);
                }
            }
        }
    }
    float *part = a.part + (long long)blockIdx.x * 2 * D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = (e * nt + threadIdx.x) * V;
        if (c < D)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                part[c + i] = accq[c + i];
                part[D + c + i] = accm[c + i];
            }
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

constexpr int kMaxBlocks = 592;   // blocks of the backward: 4 a SM, where their threads fit

template <typename T, int V, int E>
cudaError_t launch(const NormArgs &a, bool bwd, cudaStream_t st) {
    const int nt = ((a.D + V * E - 1) / (V * E) + 31) / 32 * 32;
    const NormP p = params(a);
    a.marks->mark(st);
    if (!bwd) {
        if (a.rows > 0) block_norm_fwd_kernel<T, V, E><<<a.rows, nt, 0, st>>>(p);
        return cudaGetLastError();
    }
    const size_t smem = (size_t)2 * a.D * sizeof(float);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_kernel<T, V, E>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int grid = a.rows < kMaxBlocks ? a.rows : kMaxBlocks;
    if (grid > 0) block_norm_bwd_kernel<T, V, E><<<grid, nt, smem, st>>>(p);
    a.marks->mark(st);
    if (a.dscale || a.dw_post || a.dw_pre)
        block_norm_sum_kernel<<<(2 * a.D + 31) / 32, dim3(32, 32), 0, st>>>(p.part, grid, a.D, a.scale, a.w_post,
                                                                            a.dscale, a.dw_post, a.dw_pre);
    return cudaGetLastError();
}

// V: 16 bytes where the width, the row strides and the addresses allow them.  E: vectors a thread, the fewest
// that 1024 threads need.
cudaError_t dispatch(const NormArgs &a, bool bwd, cudaStream_t st) {
    const long long all = a.D | a.ld_res | a.ld_block | a.ld_gate | elements(a.residual, a.bf16) |
                          elements(a.block, a.bf16) | elements(a.gate, a.bf16);
    if (a.bf16 && all % 8 == 0)
        return a.D <= 8192 ? launch<__nv_bfloat16, 8, 1>(a, bwd, st) : launch<__nv_bfloat16, 8, 2>(a, bwd, st);
    if (!a.bf16 && all % 4 == 0)
        return a.D <= 4096   ? launch<float, 4, 1>(a, bwd, st)
               : a.D <= 8192 ? launch<float, 4, 2>(a, bwd, st)
                             : launch<float, 4, 4>(a, bwd, st);
    if (a.bf16)
        return a.D <= 1024   ? launch<__nv_bfloat16, 1, 1>(a, bwd, st)
               : a.D <= 4096 ? launch<__nv_bfloat16, 1, 4>(a, bwd, st)
               : a.D <= 8192 ? launch<__nv_bfloat16, 1, 8>(a, bwd, st)
                             : launch<__nv_bfloat16, 1, 16>(a, bwd, st);
    return a.D <= 1024   ? launch<float, 1, 1>(a, bwd, st)
           : a.D <= 4096 ? launch<float, 1, 4>(a, bwd, st)
           : a.D <= 8192 ? launch<float, 1, 8>(a, bwd, st)
                         : launch<float, 1, 16>(a, bwd, st);
}

}  // namespace

size_t block_norm_bwd_workspace_bytes(int rows, int D) {
    return (size_t)(rows < kMaxBlocks ? rows : kMaxBlocks) * 2 * D * sizeof(float);
}
cudaError_t launch_block_norm_fwd(const NormArgs &a, cudaStream_t st) { return dispatch(a, false, st); }
cudaError_t launch_block_norm_bwd(const NormArgs &a, cudaStream_t st) { return dispatch(a, true, st); }

}  // namespace kda
