// kda_short_conv.cu -- causal depthwise convolution over time with bias and SiLU: forward,
// backward, one-row step.
//
//   pre[t] = bias + sum_j w[j] x[t-K+1+j],   y = pre sigmoid(pre)
//   dpre = dy silu'(pre),  dx[t] = sum_j w[j] dpre[t+K-1-j],  dw[j] = sum_t dpre[t] x[t-K+1+j]
//
// K = 2 .. 4 taps on bytes that pass once: bound by HBM, with the two special functions of an output
// (16 results a clock and SM) close behind in bf16.  A thread holds P pairs of neighbouring channels
// and walks L rows with the K-1 rows before them in registers, so a row is read once by its own walk
// and K-1 times more, from L2, at the seams.  Neighbouring threads hold neighbouring channels: rows
// are read in whole sectors.  Pairs go through packed FP32 instructions, which halves the issue slots.
// K = 4: forward 8192 x 12288 in bf16 74 us (5.4 TB/s), in FP32 160 (5.0); backward 16384 x 2048 in
// bf16 70 (2.9 TB/s; 69 instructions a pair of channels and row), in FP32 88 (4.6); step 256 x 12288
// in bf16 8.2 (6.2 TB/s).
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
    int D, silu, groups;                 // groups: ceil(D / (2 P))
    long long ld_x, ld_y, ld_dx, walks;  // walks: ceil(rows / L)
    int L;
};

// 2 P channels from c on.  V: all of them exist and addresses are aligned; otherwise `have` exist.
template <typename T, int P, bool V>
struct Row {
    Raw<T, 2 * P> r;
    __device__ __forceinline__ void load(const T *p, int have) {
        r = V ? load_raw<T, 2 * P>(p) : load_part<T, 2 * P>(p, have);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < Raw<T, 2 * P>::kWords; ++i) r.w[i] = 0u;
    }
    __device__ __forceinline__ void get(float2 (&v)[P]) const {
        float f[2 * P];
        widen<T, 2 * P>(r, f);
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
};
template <typename T, int P, bool V>
__device__ __forceinline__ void store_row(T *p, const float2 (&v)[P], int have) {
    float f[2 * P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        f[2 * i] = v[i].x;
        f[2 * i + 1] = v[i].y;
    }
    if (V) store_f32<T, 2 * P>(p, f);
    else store_part<T, 2 * P>(p, f, have);
}

template <typename T, int P, int K, bool V>
struct Taps {
    float2 w[K][P], bias[P];
    __device__ __forceinline__ void load(const ConvP &a, int c, int have) {
        const T *p = (const T *)a.w + (long long)c * K;
        float f[2 * P * K];
        if constexpr (V && 2 * P * K * sizeof(T) % 16 == 0) {
            load_f32<T, 2 * P * K>(p, f);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * P * K; ++i) f[i] = i < have * K ? to_f32(p[i]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][i] = make_float2(f[2 * i * K + j], f[(2 * i + 1) * K + j]);
            bias[i] = make_float2(0.f, 0.f);
        }
        if (a.bias) {
            Row<T, P, V> r;
            r.load((const T *)a.bias + c, have);
            r.get(bias);
        }
    }
    // pre-activation of row x behind the rows in win, oldest first
    __device__ __forceinline__ void pre(const float2 (&win)[K - 1][P], const float2 (&x)[P], float2 (&out)[P]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 v = __ffma2_rn(w[K - 1][i], x[i], bias[i]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v = __ffma2_rn(w[j][i], win[j][i], v);
            out[i] = v;
        }
    }
};

// Input row p of a sequence that starts at row lo: from x, from the carried state, or zero.
template <typename T, int P, int K, bool V>
__device__ __forceinline__ void load_row(const ConvP &a, int s, long long lo, long long p, int c, int have,
                                         float2 (&out)[P]) {
    Row<T, P, V> r;
    if (p >= lo) r.load((const T *)a.x + p * a.ld_x + c, have);
    else if (a.state0) r.load((const T *)a.state0 + ((long long)s * (K - 1) + (p - lo + K - 1)) * a.D + c, have);
    else r.zero();
    r.get(out);
}
template <int N, int P>
__device__ __forceinline__ void push(float2 (&win)[N][P], const float2 (&x)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < N; ++j) win[j][i] = win[j + 1][i];
        win[N - 1][i] = x[i];
    }
}

__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 t = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
    const float2 e = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(e.x), rcp(e.y));
}

template <typename T, int P, int K, bool V>
__global__ void __launch_bounds__(kThreads, 5) short_conv_fwd_kernel(const ConvP a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long walk = id / a.groups;
    const int c = (int)(id % a.groups) * 2 * P, have = a.D - c < 2 * P ? a.D - c : 2 * P;
    if (walk >= a.walks) {   // one thread per sequence and channel group: the state that goes on
        const long long s = walk - a.walks;
        if (s >= a.q.S || !a.state_T) return;
        const long long lo = a.q.lo((int)s), hi = a.q.hi((int)s);
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            float2 v[P];
            load_row<T, P, K, V>(a, (int)s, lo, hi - (K - 1) + r, c, have, v);
            store_row<T, P, V>((T *)a.state_T + (s * (K - 1) + r) * a.D + c, v, have);
        }
        return;
    }
    Taps<T, P, K, V> taps;
    taps.load(a, c, have);
    int r = (int)(walk * a.L);
    const int r1 = (int)(a.q.rows() - r < a.L ? a.q.rows() : r + a.L);
    int s = a.q.at(r);
    while (r < r1) {
        const int lo = (int)a.q.lo(s), hi = (int)a.q.hi(s);
        if (r >= hi) {   // on to the next sequence, past empty ones
            if (++s >= a.q.S) break;
            continue;
        }
        if (r < lo) {    // rows of no sequence
            r = lo;
            continue;
        }
        float2 win[K - 1][P];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) load_row<T, P, K, V>(a, s, lo, r - (K - 1) + j, c, have, win[j]);
        const int e = hi < r1 ? hi : r1;
        const T *px = (const T *)a.x + (long long)r * a.ld_x + c;
        T *py = (T *)a.y + (long long)r * a.ld_y + c;
        auto row = [&](const Row<T, P, V> &raw, T *o) {
            float2 v[P], p[P];
            raw.get(v);
            taps.pre(win, v, p);
            push(win, v);
            if (a.silu) {
#pragma unroll
                for (int m = 0; m < P; ++m) p[m] = __fmul2_rn(p[m], sigmoid2(p[m]));
            }
            store_row<T, P, V>(o, p, have);
        };
        constexpr int U = V ? 8 : 4;  // rows a batch; the next one is loaded while one is computed
        Row<T, P, V> cur[U], next[U];
        if (r + U <= e)
#pragma unroll
            for (int i = 0; i < U; ++i) cur[i].load(px + i * a.ld_x, have);
        for (; r + U <= e; r += U) {
            px += U * a.ld_x;
            if (r + 2 * U <= e)
#pragma unroll
                for (int i = 0; i < U; ++i) next[i].load(px + i * a.ld_x, have);
#pragma unroll
            for (int i = 0; i < U; ++i) row(cur[i], py + i * a.ld_y);
            py += U * a.ld_y;
#pragma unroll
            for (int i = 0; i < U; ++i) cur[i] = next[i];
        }
        for (; r < e; ++r) {
            Row<T, P, V> raw;
            raw.load(px, have);
            row(raw, py);
            px += a.ld_x;
            py += a.ld_y;
        }
    }
}

// gradient of the pre-activations p where the outputs' gradient is g
template <int P>
__device__ __forceinline__ void dpre_of(const float2 (&p)[P], float2 (&g)[P], bool silu) {
    if (!silu) return;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 s = sigmoid2(p[i]), one = make_float2(1.f, 1.f);
        const float2 t = __ffma2_rn(p[i], __ffma2_rn(s, make_float2(-1.f, -1.f), one), one);   // 1 + p (1 - s)
        g[i] = __fmul2_rn(g[i], __fmul2_rn(s, t));
    }
}

// A walk owns the rows r0 .. r1-1: it writes their dx, for which it needs dpre up to K-1 rows
// on, and sums dpre and dpre x over its own rows into its partial sums [walk][K + 1][D].  One pair
// of channels a thread: its 2 K + 2 sums, taps and rows take 60 registers, and the 20 warps an
// SM that fit hide most of HBM's latency: 64 us for 16384 x 2048 in bf16, 72 with 16 warps, 110 with
// two pairs a thread.
template <typename T, int K, bool V>
__global__ void __launch_bounds__(kThreads, 5) short_conv_bwd_kernel(const ConvP a) {
    constexpr int P = 1;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long walk = id / a.groups;
    const int c = (int)(id % a.groups) * 2 * P, have = a.D - c < 2 * P ? a.D - c : 2 * P;
    const T *x = (const T *)a.x + c, *dy = (const T *)a.dy + c;
    if (walk >= a.walks && (walk - a.walks >= a.q.S || !a.dstate0)) return;
    Taps<T, P, K, V> taps;
    taps.load(a, c, have);
    if (walk >= a.walks) {   // gradient of the carried state: its rows act on the first K-1 outputs
        const int s = (int)(walk - a.walks);
        const long long lo = a.q.lo(s), hi = a.q.hi(s);
        float2 win[K - 1][P], out[K - 1][P];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            load_row<T, P, K, V>(a, s, lo, lo - (K - 1) + j, c, have, win[j]);
            const long long back = j - (hi - lo);   // still in the last state, at this row of it
            Row<float, P, V> r;
            if (back >= 0 && a.dstate_T) r.load(a.dstate_T + ((long long)s * (K - 1) + back) * a.D + c, have);
            else r.zero();
            r.get(out[j]);
        }
#pragma unroll
        for (int t = 0; t < K - 1; ++t) {
            if (lo + t < hi) {
                Row<T, P, V> rx, rg;
                float2 v[P], p[P], d[P];
                rx.load(x + (lo + t) * a.ld_x, have);
                rg.load(dy + (lo + t) * a.ld_y, have);
                rx.get(v);
                rg.get(d);
                taps.pre(win, v, p);
                dpre_of<P>(p, d, a.silu);
                push(win, v);
#pragma unroll
                for (int j = 0; j < K - 1 - t; ++j)   // tap j of row t sees state row t + j
#pragma unroll
                    for (int i = 0; i < P; ++i) out[t + j][i] = __ffma2_rn(taps.w[j][i], d[i], out[t + j][i]);
            }
        }
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
            store_row<float, P, V>(a.dstate0 + ((long long)s * (K - 1) + r) * a.D + c, out[r], have);
        return;
    }
    float2 dw[K + 1][P];   // the last: dbias
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) dw[j][i] = make_float2(0.f, 0.f);
    int r = (int)(walk * a.L);
    const int r1 = (int)(a.q.rows() - r < a.L ? a.q.rows() : r + a.L);
    int s = a.q.at(r);
    while (r < r1) {
        const int lo = (int)a.q.lo(s), hi = (int)a.q.hi(s);
        if (r >= hi) {
            if (++s >= a.q.S) break;
            continue;
        }
        if (r < lo) {
            r = lo;
            continue;
        }
        const int e = hi < r1 ? hi : r1;
        float2 win[K - 1][P], ring[K - 1][P];   // inputs before row p; dpre of the rows before it
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            load_row<T, P, K, V>(a, s, lo, r - (K - 1) + j, c, have, win[j]);
#pragma unroll
            for (int i = 0; i < P; ++i) ring[j][i] = make_float2(0.f, 0.f);
        }
        const T *px = x + (long long)r * a.ld_x, *pg = dy + (long long)r * a.ld_y;
        T *po = (T *)a.dx + c + (long long)(r - (K - 1)) * a.ld_dx;
        // A row's dpre d, and dx of the row K-1 before it, whose last term it is.
        auto gather = [&](const float2 (&d)[P], float2 (&o)[P]) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                o[i] = __fmul2_rn(taps.w[0][i], d[i]);
#pragma unroll
                for (int j = 1; j < K; ++j) o[i] = __ffma2_rn(taps.w[j][i], ring[K - 1 - j][i], o[i]);
            }
            push(ring, d);
        };
        auto own = [&](const Row<T, P, V> &rx, const Row<T, P, V> &rg, float2 (&d)[P]) {   // a row of the walk
            float2 v[P], p[P];
            rx.get(v);
            rg.get(d);
            taps.pre(win, v, p);
            dpre_of<P>(p, d, a.silu);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dw[K][i] = __fadd2_rn(dw[K][i], d[i]);
                dw[K - 1][i] = __ffma2_rn(d[i], v[i], dw[K - 1][i]);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) dw[j][i] = __ffma2_rn(d[i], win[j][i], dw[j][i]);
            }
            push(win, v);
        };
        auto put = [&](int t, T *o, float2 (&v)[P]) {   // dx of row t, with what the last state adds
            const int back = t - hi + (K - 1);
            if (a.dstate_T && back >= 0) {
                Row<float, P, V> g;
                float2 f[P];
                g.load(a.dstate_T + ((long long)s * (K - 1) + back) * a.D + c, have);
                g.get(f);
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = __fadd2_rn(v[i], f[i]);
            }
            store_row<T, P, V>(o, v, have);
        };
        int p = r;
        // Whole batches inside the walk.  (With the next batch loaded while one is computed the registers
        // leave fewer warps: 77 to 87 us for 16384 x 2048 in bf16.)
        constexpr int U = 8;
        for (; p + U <= e; p += U) {
            Row<T, P, V> rx[U], rg[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                rx[i].load(px + i * a.ld_x, have);
                rg[i].load(pg + i * a.ld_y, have);
            }
            const bool plain = p - (K - 1) >= r && (!a.dstate_T || p + U <= hi - (K - 1));
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float2 d[P], o[P];
                own(rx[i], rg[i], d);
                gather(d, o);
                if (plain) store_row<T, P, V>(po + i * a.ld_dx, o, have);
                else if (p + i - (K - 1) >= r) put(p + i - (K - 1), po + i * a.ld_dx, o);
            }
            px += U * a.ld_x;
            pg += U * a.ld_y;
            po += U * a.ld_dx;
        }
        // the rest of the walk, and the K-1 rows behind it (zero behind the sequence)
        for (; p < e + K - 1; ++p) {
            float2 d[P], o[P];
            if (p < hi) {
                Row<T, P, V> rx, rg;
                rx.load(px, have);
                rg.load(pg, have);
                if (p < e) {
                    own(rx, rg, d);
                } else {
                    float2 v[P], q[P];
                    rx.get(v);
                    rg.get(d);
                    taps.pre(win, v, q);
                    dpre_of<P>(q, d, a.silu);
                    push(win, v);
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) d[i] = make_float2(0.f, 0.f);
            }
            gather(d, o);
            if (p - (K - 1) >= r) put(p - (K - 1), po, o);
            px += a.ld_x;
            pg += a.ld_y;
            po += a.ld_dx;
        }
        r = e;
    }
    float *part = a.part + walk * (K + 1) * a.D + c;
#pragma unroll
    for (int j = 0; j <= K; ++j) store_row<float, P, V>(part + (long long)j * a.D, dw[j], have);
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

template <typename T, int P, int K, bool V>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const ConvP a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long s = id / a.groups;
    if (s >= a.q.S) return;
    const int c = (int)(id % a.groups) * 2 * P, have = a.D - c < 2 * P ? a.D - c : 2 * P;
    const T *st = (const T *)a.state0 + s * (K - 1) * a.D + c;
    T *so = (T *)a.state_T + s * (K - 1) * a.D + c;
    Row<T, P, V> rx, rs[K - 1];
    rx.load((const T *)a.x + s * a.ld_x + c, have);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) rs[j].load(st + (long long)j * a.D, have);
    Taps<T, P, K, V> taps;
    taps.load(a, c, have);
    float2 win[K - 1][P], v[P], p[P];
    rx.get(v);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) rs[j].get(win[j]);
    taps.pre(win, v, p);
    push(win, v);
    if (a.silu) {
#pragma unroll
        for (int m = 0; m < P; ++m) p[m] = __fmul2_rn(p[m], sigmoid2(p[m]));
    }
    store_row<T, P, V>((T *)a.y + s * a.ld_y + c, p, have);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_row<T, P, V>(so + (long long)j * a.D, win[j], have);
}

enum class Run { FWD, BWD, STEP };

ConvP params(const ConvArgs &a, int width) {
    ConvP p;
    p.x = a.x; p.w = a.w; p.bias = a.bias; p.state0 = a.state0;
    p.y = a.y; p.state_T = a.state_T; p.dy = a.dy; p.dstate_T = a.dstate_T; p.dx = a.dx;
    p.part = (float *)a.workspace; p.dstate0 = a.dstate0;
    p.q.cu = a.cu; p.q.S = a.S; p.q.T = a.T;
    p.D = a.D; p.silu = a.silu; p.groups = (a.D + width - 1) / width;
    p.ld_x = a.ld_x; p.ld_y = a.ld_y; p.ld_dx = a.ld_dx;
    p.walks = 0; p.L = 0;
    return p;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Rows a forward walk takes: 64 where that leaves 2^18 threads (the device holds 303,104),
// down to 8 below.  In bf16, in us: 8192 x 12288 74 (64 rows; 76 with 32, 78 with 128), 16384 x 2048 31 (32; 35
// with 16, 31 with 64), 1024 x 2048 6.2 (8; 6.2 with 16 and 32, 9.4 with 64), 3001 x 1001 9.8 (8; 8.3 with 16).
int fwd_rows(long long rows, int groups) {
    int L = 64;
    while (L > 8 && ceil_div(rows, L) * groups < (1 << 18)) L /= 2;
    return L;
}
// Rows a backward walk takes; at least 16, so that the partial sums of (K + 1) FP32 values a
// channel and walk stay small against the rows' bytes.  In bf16, in us: 8192 x 12288 191 (64 rows; 215 with 32,
// 193 with 128), 16384 x 2048 70 (64; 86 and 77), 4096 x 2048 29 (16; 25 with 32 and 64), 1024 x 2048 14.5 (16; 17
// with 8, 16.4 with 32), 3001 x 1001 18.5 (16; 17.5 with 32).
int bwd_rows(long long rows, int D) {
    int L = 64;
    while (L > 16 && ceil_div(rows, L) * (D / 2) < (1 << 18)) L /= 2;
    return L;
}

template <typename T, int P, int K, bool V>
cudaError_t launch(const ConvArgs &a, Run run, cudaStream_t st) {
    constexpr int BP = 1;   // pairs a thread of the backward
    ConvP p = params(a, run == Run::BWD ? 2 * BP : 2 * P);
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
        if (run == Run::FWD) short_conv_fwd_kernel<T, P, K, V><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        if (run == Run::BWD) short_conv_bwd_kernel<T, K, V><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        if (run == Run::STEP) short_conv_step_kernel<T, P, K, V><<<(unsigned)blocks, kThreads, 0, st>>>(p);
    }
    if (run == Run::BWD) {
        a.marks->mark(st);
        short_conv_sum_kernel<<<(unsigned)ceil_div((long long)(K + 1) * a.D, 32), dim3(32, 32), 0, st>>>(
            p.part, a.dw, a.dbias, p.walks, a.D, K);
    }
    return cudaGetLastError();
}

template <typename T, int P, bool V>
cudaError_t launch_k(const ConvArgs &a, Run run, cudaStream_t st) {
    switch (a.K) {
        case 2: return launch<T, P, 2, V>(a, run, st);
        case 3: return launch<T, P, 3, V>(a, run, st);
        default: return launch<T, P, 4, V>(a, run, st);
    }
}

// Whole vectors where channels, row strides and addresses allow them; single values otherwise.
cudaError_t dispatch(const ConvArgs &a, Run run, cudaStream_t st) {
    long long all = a.D | a.ld_x | a.ld_y | elements(a.x, a.bf16);
    if (run == Run::BWD) all |= a.ld_dx | elements(a.dy, a.bf16) | elements(a.dx, a.bf16);
    else all |= elements(a.y, a.bf16);
    if (a.bf16) {
        if (all % (4) == 0) return launch_k<__nv_bfloat16, 2, true>(a, run, st);
        return launch_k<__nv_bfloat16, 1, false>(a, run, st);
    }
    if (all % 4 == 0) return launch_k<float, 2, true>(a, run, st);
    return launch_k<float, 1, false>(a, run, st);
}

}  // namespace

size_t short_conv_bwd_workspace_bytes(long long rows, int D, int K) {
    return (size_t)ceil_div(rows, bwd_rows(rows, D)) * (K + 1) * D * sizeof(float);
}
cudaError_t launch_short_conv_fwd(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::FWD, st); }
cudaError_t launch_short_conv_bwd(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::BWD, st); }
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st) { return dispatch(a, Run::STEP, st); }

}  // namespace kda
