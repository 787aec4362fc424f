// kda_short_conv.cu -- causal depthwise convolution over time with bias and SiLU: forward,
// backward, one-row step.
//
//   pre[t] = bias + sum_j w[j] x[t-K+1+j],   y = pre sigmoid(pre)
//   dpre = dy silu'(pre),  dx[t] = sum_j w[j] dpre[t+K-1-j],  dw[j] = sum_t dpre[t] x[t-K+1+j]
//
// K = 2 .. 4 taps on bytes that pass once: bound by HBM.  A thread holds V neighbouring
// channels and walks kRows rows with the K-1 rows before them in registers, so a row is read
// once by its own thread and K-1 times more, from L2, at the seams of the walks.  Neighbouring
// threads hold neighbouring channels: rows are read in whole sectors.
#include "kda_layers_internal.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

struct ConvP {
    const void *x, *w, *bias, *state0;
    void *y, *state_T;
    const void *dy;
    const float *dstate_T;
    void *dx;
    float *part, *dstate0;
    Seqs q;
    int D, silu, groups;                 // groups: ceil(D / V)
    long long ld_x, ld_y, ld_dx, walks;  // walks: ceil(rows / L)
    int L;
};

// V taps sets of K, channel after channel
template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const T *w, float (&out)[V][K]) {
    if constexpr (V * K * sizeof(T) % 16 == 0) {
        constexpr int P = 16 / sizeof(T);
        float flat[V * K];
#pragma unroll
        for (int i = 0; i < V * K; i += P) load_f32<T, P>(w + i, flat + i);
#pragma unroll
        for (int i = 0; i < V * K; ++i) out[i / K][i % K] = flat[i];
    } else {
#pragma unroll
        for (int i = 0; i < V * K; ++i) out[i / K][i % K] = to_f32(w[i]);
    }
}

// Input row p of a sequence that starts at row lo: from x, from the carried state, or zero.
template <typename T, int V, int K>
__device__ __forceinline__ void load_row(const ConvP &a, int s, long long lo, long long p, int c, float *out) {
    if (p >= lo) {
        load_f32<T, V>((const T *)a.x + p * a.ld_x + c, out);
    } else if (a.state0) {
        const long long k = p - lo + (K - 1);   // 0 .. K-2
        load_f32<T, V>((const T *)a.state0 + ((long long)s * (K - 1) + k) * a.D + c, out);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.f;
    }
}

template <int V, int K>
__device__ __forceinline__ void preact(const float (&w)[V][K], const float *bias, const float (&win)[K - 1][V],
                                       const float *x, float *pre) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = fmaf(w[i][K - 1], x[i], bias[i]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) p = fmaf(w[i][j], win[j][i], p);
        pre[i] = p;
    }
}
template <int V, int K>
__device__ __forceinline__ void push(float (&win)[K - 1][V], const float *x) {
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) win[K - 2][i] = x[i];
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) short_conv_fwd_kernel(const ConvP a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long walk = id / a.groups;
    const int c = (int)(id % a.groups) * V;
    const T *x = (const T *)a.x;
    if (walk >= a.walks) {   // one thread per sequence and channel group: the state that goes on
        const long long s = walk - a.walks;
        if (s >= a.q.S || !a.state_T) return;
        const long long lo = a.q.lo((int)s), hi = a.q.hi((int)s);
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            float v[V];
            load_row<T, V, K>(a, (int)s, lo, hi - (K - 1) + r, c, v);
            store_f32<T, V>((T *)a.state_T + (s * (K - 1) + r) * a.D + c, v);
        }
        return;
    }
    float w[V][K], bias[V];
    load_taps<T, V, K>((const T *)a.w + (long long)c * K, w);
    if (a.bias) {
        load_f32<T, V>((const T *)a.bias + c, bias);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = 0.f;
    }
    long long r = walk * a.L;
    const long long rows = a.q.rows(), r1 = r + a.L < rows ? r + a.L : rows;
    int s = a.q.at(r);
    while (r < r1) {
        long long lo = a.q.lo(s), hi = a.q.hi(s);
        if (r >= hi) {   // on to the next sequence, past empty ones
            if (++s >= a.q.S) break;
            continue;
        }
        if (r < lo) {    // rows of no sequence
            r = lo;
            continue;
        }
        float win[K - 1][V];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) load_row<T, V, K>(a, s, lo, r - (K - 1) + j, c, win[j]);
        const long long e = hi < r1 ? hi : r1;
        const T *px = x + r * a.ld_x + c;
        T *py = (T *)a.y + r * a.ld_y + c;
        constexpr int U = 8;   // rows in flight
        for (; r + U <= e; r += U) {
            Raw<T, V> raw[U];
#pragma unroll
            for (int i = 0; i < U; ++i) raw[i] = load_raw<T, V>(px + i * a.ld_x);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float v[V], p[V];
                widen<T, V>(raw[i], v);
                preact<V, K>(w, bias, win, v, p);
                push<V, K>(win, v);
                if (a.silu) {
#pragma unroll
                    for (int m = 0; m < V; ++m) p[m] = silu_f32(p[m]);
                }
                store_f32<T, V>(py + i * a.ld_y, p);
            }
            px += U * a.ld_x;
            py += U * a.ld_y;
        }
        for (; r < e; ++r) {
            float v[V], p[V];
            load_f32<T, V>(px, v);
            preact<V, K>(w, bias, win, v, p);
            push<V, K>(win, v);
            if (a.silu) {
#pragma unroll
                for (int m = 0; m < V; ++m) p[m] = silu_f32(p[m]);
            }
            store_f32<T, V>(py, p);
            px += a.ld_x;
            py += a.ld_y;
        }
    }
}

__device__ __forceinline__ float dsilu(float x) {
    const float p = sigmoid_f32(x);
    return p * fmaf(x, 1.f - p, 1.f);
}

// dpre of row p of the sequence [lo, hi), whose input row is v; zero behind the sequence
template <typename T, int V, int K>
__device__ __forceinline__ void dpre_of(const ConvP &a, const float (&w)[V][K], const float *bias,
                                        const float (&win)[K - 1][V], const float *v, const float *g, float *d) {
    float p[V];
    preact<V, K>(w, bias, win, v, p);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = a.silu ? g[i] * dsilu(p[i]) : g[i];
}

// A walk owns the rows r0 .. r1-1: it writes their dx, for which it needs dpre up to K-1 rows
// on, and sums dpre and dpre x over its own rows into its partial sums [walk][K + 1][D].
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) short_conv_bwd_kernel(const ConvP a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long walk = id / a.groups;
    const int c = (int)(id % a.groups) * V;
    const T *x = (const T *)a.x, *dy = (const T *)a.dy;
    if (walk >= a.walks && (walk - a.walks >= a.q.S || !a.dstate0)) return;
    float w[V][K], bias[V];
    load_taps<T, V, K>((const T *)a.w + (long long)c * K, w);
    if (a.bias) {
        load_f32<T, V>((const T *)a.bias + c, bias);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = 0.f;
    }
    if (walk >= a.walks) {   // gradient of the carried state: its rows act on the first K-1 outputs
        const int s = (int)(walk - a.walks);
        const long long lo = a.q.lo(s), hi = a.q.hi(s);
        float win[K - 1][V], out[K - 1][V];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            load_row<T, V, K>(a, s, lo, lo - (K - 1) + j, c, win[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) out[j][i] = 0.f;
            const long long back = j - (hi - lo);   // still in the last state, at this row of it
            if (back >= 0 && a.dstate_T)
                load_f32<float, V>(a.dstate_T + ((long long)s * (K - 1) + back) * a.D + c, out[j]);
        }
#pragma unroll
        for (int t = 0; t < K - 1; ++t) {
            if (lo + t < hi) {
                float v[V], g[V], d[V];
                load_f32<T, V>(x + (lo + t) * a.ld_x + c, v);
                load_f32<T, V>(dy + (lo + t) * a.ld_y + c, g);
                dpre_of<T, V, K>(a, w, bias, win, v, g, d);
                push<V, K>(win, v);
#pragma unroll
                for (int j = 0; j < K - 1 - t; ++j)   // tap j of row t sees state row t + j
#pragma unroll
                    for (int i = 0; i < V; ++i) out[t + j][i] = fmaf(w[i][j], d[i], out[t + j][i]);
            }
        }
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
            store_f32<float, V>(a.dstate0 + ((long long)s * (K - 1) + r) * a.D + c, out[r]);
        return;
    }
    float dw[K][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = 0.f;
    }
    long long r = walk * a.L;
    const long long rows = a.q.rows(), r1 = r + a.L < rows ? r + a.L : rows;
    int s = a.q.at(r);
    while (r < r1) {
        const long long lo = a.q.lo(s), hi = a.q.hi(s);
        if (r >= hi) {
            if (++s >= a.q.S) break;
            continue;
        }
        if (r < lo) {
            r = lo;
            continue;
        }
        const long long e = hi < r1 ? hi : r1;
        float win[K - 1][V], ring[K - 1][V];   // inputs before row p; dpre of the rows before it
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            load_row<T, V, K>(a, s, lo, r - (K - 1) + j, c, win[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) ring[j][i] = 0.f;
        }
        // row p: dpre[p], then dx[p - K + 1], whose last term it is
        auto step = [&](long long p, const Raw<T, V> &rx, const Raw<T, V> &rg) {
            float d[V];
            if (p < hi) {
                float v[V], g[V];
                widen<T, V>(rx, v);
                widen<T, V>(rg, g);
                dpre_of<T, V, K>(a, w, bias, win, v, g, d);
                if (p < e) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        db[i] += d[i];
                        dw[K - 1][i] = fmaf(d[i], v[i], dw[K - 1][i]);
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) dw[j][i] = fmaf(d[i], win[j][i], dw[j][i]);
                    }
                }
                push<V, K>(win, v);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] = 0.f;
            }
            const long long t = p - (K - 1);
            if (t >= r) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[i] = w[i][0] * d[i];
#pragma unroll
                    for (int j = 1; j < K; ++j) o[i] = fmaf(w[i][j], ring[K - 1 - j][i], o[i]);
                }
                const long long back = t - hi + (K - 1);   // >= 0: a row of the last state
                if (a.dstate_T && back >= 0) {
                    float g[V];
                    load_f32<float, V>(a.dstate_T + ((long long)s * (K - 1) + back) * a.D + c, g);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] += g[i];
                }
                store_f32<T, V>((T *)a.dx + t * a.ld_dx + c, o);
            }
            push<V, K>(ring, d);
        };
        long long p = r;
        const long long pe = e + K - 1;
        constexpr int U = 4;
        for (; p + U <= hi && p + U <= pe; p += U) {
            Raw<T, V> rx[U], rg[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                rx[i] = load_raw<T, V>(x + (p + i) * a.ld_x + c);
                rg[i] = load_raw<T, V>(dy + (p + i) * a.ld_y + c);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) step(p + i, rx[i], rg[i]);
        }
        for (; p < pe; ++p) {
            Raw<T, V> rx, rg;
            if (p < hi) {
                rx = load_raw<T, V>(x + p * a.ld_x + c);
                rg = load_raw<T, V>(dy + p * a.ld_y + c);
            } else {
                rx = rg = load_part<T, V>(x, 0);
            }
            step(p, rx, rg);
        }
        r = e;
    }
    float *part = a.part + walk * (K + 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < K; ++j) store_f32<float, V>(part + (long long)j * a.D, dw[j]);
    store_f32<float, V>(part + (long long)K * a.D, db);
}

// dw[c, j] and dbias[c] from the walks' partial sums: a block sums 32 columns of [K + 1][D],
// 32 lanes of walks each, then the lanes in order.
__global__ void __launch_bounds__(1024) short_conv_sum_kernel(const float *__restrict__ part, float *dw, float *dbias,
                                                              long long walks, int D, int K) {
    __shared__ float s[32][33];
    const int n = (K + 1) * D;
    const int i = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (i < n)
        for (long long k = threadIdx.y; k < walks; k += 32) v += part[k * n + i];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(s[threadIdx.x][threadIdx.y]);
    if (threadIdx.x == 0) {
        const int o = blockIdx.x * 32 + threadIdx.y;
        if (o < n) {
            const int j = o / D, c = o % D;
            if (j < K) dw[(long long)c * K + j] = v;
            else if (dbias) dbias[c] = v;
        }
    }
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const ConvP a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long s = id / a.groups;
    if (s >= a.q.S) return;
    const int c = (int)(id % a.groups) * V;
    float w[V][K], bias[V], win[K - 1][V], v[V], p[V];
    const T *st = (const T *)a.state0 + s * (K - 1) * a.D + c;
    T *so = (T *)a.state_T + s * (K - 1) * a.D + c;
    load_f32<T, V>((const T *)a.x + s * a.ld_x + c, v);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_f32<T, V>(st + (long long)j * a.D, win[j]);
    load_taps<T, V, K>((const T *)a.w + (long long)c * K, w);
    if (a.bias) {
        load_f32<T, V>((const T *)a.bias + c, bias);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = 0.f;
    }
    preact<V, K>(w, bias, win, v, p);
    push<V, K>(win, v);
    if (a.silu) {
#pragma unroll
        for (int m = 0; m < V; ++m) p[m] = silu_f32(p[m]);
    }
    store_f32<T, V>((T *)a.y + s * a.ld_y + c, p);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_f32<T, V>(so + (long long)j * a.D, win[j]);
}

enum class Run { FWD, BWD, STEP };

ConvP params(const ConvArgs &a, int V) {
    ConvP p;
    p.x = a.x; p.w = a.w; p.bias = a.bias; p.state0 = a.state0;
    p.y = a.y; p.state_T = a.state_T; p.dy = a.dy; p.dstate_T = a.dstate_T; p.dx = a.dx;
    p.part = (float *)a.workspace; p.dstate0 = a.dstate0;
    p.q.cu = a.cu; p.q.S = a.S; p.q.T = a.T;
    p.D = a.D; p.silu = a.silu; p.groups = (a.D + V - 1) / V;
    p.ld_x = a.ld_x; p.ld_y = a.ld_y; p.ld_dx = a.ld_dx;
    p.walks = 0; p.L = 0;
    return p;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Rows a forward walk takes: 32 where that leaves 2^18 threads (the device holds 303,104),
// down to 8 below.
int fwd_rows(long long rows, int groups) {
    int L = 32;
    while (L > 8 && ceil_div(rows, L) * groups < (1 << 18)) L /= 2;
    return L;
}
// Rows a backward walk takes; at least 16, so that the partial sums of (K + 1) FP32 values a
// channel and walk stay small against the rows' bytes.
int bwd_rows(long long rows, int D) {
    int L = 128;
    while (L > 16 && ceil_div(rows, L) * (D / 4) < (1 << 17)) L /= 2;
    return L;
}

template <typename T, int V, int K>
cudaError_t launch(const ConvArgs &a, Run run, cudaStream_t st) {
    ConvP p = params(a, V);
    long long threads;
    if (run == Run::STEP) {
        threads = (long long)p.groups * a.S;
    } else {
        p.L = run == Run::FWD ? fwd_rows(a.rows, p.groups) : bwd_rows(a.rows, a.D);
        p.walks = ceil_div(a.rows, p.L);
        const bool states = run == Run::FWD ? a.state_T != nullptr : a.dstate0 != nullptr;
        threads = (long long)p.groups * (p.walks + (states ? a.S : 0));
    }
    const long long blocks = ceil_div(threads, kThreads);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    a.marks->mark(st);
    if (blocks > 0) {
        if (run == Run::FWD) short_conv_fwd_kernel<T, V, K><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        if (run == Run::BWD) short_conv_bwd_kernel<T, V, K><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        if (run == Run::STEP) short_conv_step_kernel<T, V, K><<<(unsigned)blocks, kThreads, 0, st>>>(p);
    }
    if (run == Run::BWD) {
        a.marks->mark(st);
        short_conv_sum_kernel<<<(unsigned)ceil_div((long long)(K + 1) * a.D, 32), dim3(32, 32), 0, st>>>(
            p.part, a.dw, a.dbias, p.walks, a.D, K);
    }
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_k(const ConvArgs &a, Run run, cudaStream_t st) {
    switch (a.K) {
        case 2: return launch<T, V, 2>(a, run, st);
        case 3: return launch<T, V, 3>(a, run, st);
        default: return launch<T, V, 4>(a, run, st);
    }
}

// 16-byte accesses where channels, row strides and addresses allow them; single values otherwise.  The
// backward takes 8 bytes of bf16: its sums for 8 channels would not stay in registers.
cudaError_t dispatch(const ConvArgs &a, Run run, cudaStream_t st) {
    long long all = a.D | a.ld_x | a.ld_y | elements(a.x, a.bf16);
    if (run == Run::BWD) all |= a.ld_dx | elements(a.dy, a.bf16) | elements(a.dx, a.bf16);
    else all |= elements(a.y, a.bf16);
    if (a.bf16) {
        if (run != Run::BWD && all % 8 == 0) return launch_k<__nv_bfloat16, 8>(a, run, st);
        if (run == Run::BWD && all % 4 == 0) return launch_k<__nv_bfloat16, 4>(a, run, st);
        return launch_k<__nv_bfloat16, 1>(a, run, st);
    }
    if (all % 4 == 0) return launch_k<float, 4>(a, run, st);
    return launch_k<float, 1>(a, run, st);
}

}  // namespace

size_t short_conv_bwd_workspace_bytes(long long rows, int D, int K) {
    return (size_t)ceil_div(rows, bwd_rows(rows, D)) * (K + 1) * D * sizeof(float);
}
cudaError_t launch_short_conv_fwd(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::FWD, st); }
cudaError_t launch_short_conv_bwd(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::BWD, st); }
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::STEP, st); }

}  // namespace kda
