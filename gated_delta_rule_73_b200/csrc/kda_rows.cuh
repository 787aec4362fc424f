// kda_rows.cuh -- what the short convolution, the selective scan and the block norm share:
// vector access to rows, activations in full FP32 accuracy, sequence bounds and spans.
#pragma once
#include "kda_common.cuh"

namespace kda {

// ---------------------------------------------------------------- V consecutive values
// V * sizeof(T) is 2, 4, 8, 16 or 32 bytes; the address is a multiple of min(that, 16).
template <typename T, int V>
struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Raw {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, V> *>(p);
}
// The first n values (n <= 0: none) one by one; the others are zero.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_part(const T *p, int n) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = i < n ? p[i] : from_f32<T>(0.f);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V> &r, float *x) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(r.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void load_f32(const T *p, float *x) {
    widen<T, V>(load_raw<T, V>(p), x);
}
template <typename T, int V>
__device__ __forceinline__ void store_f32(T *p, const float *x) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f32<T>(x[i]);
    *reinterpret_cast<Raw<T, V> *>(p) = r;
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, const float *x, int n) {
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n) p[i] = from_f32<T>(x[i]);
}

// ---------------------------------------------------------------- activations
// Relative error of a few 2^-23: fp32 outputs keep their precision.  The limits are exact:
// sigmoid(-inf) = 0 (the quotient's denominator is inf), sigmoid(inf) = 1.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float silu_f32(float x) { return x * sigmoid_f32(x); }

// log(1 + e^x) = max(x, 0) + 2 atanh(e / (2 + e)) with e = exp(-|x|) in (0, 1]: the series of
// atanh in s = e / (2 + e) <= 1/3 keeps the relative precision of small values, which
// log2(1 + e) loses.  The first term left out, s^14 / 15, is below 2^-25 of the sum.
__device__ __forceinline__ float softplus_f32(float x) {
    const float e = ex2(-kLog2e * fabsf(x));
    const float s = e * rcp(2.f + e);
    const float q = s * s;
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(q, p, 1.f / 9.f);
    p = fmaf(q, p, 1.f / 7.f);
    p = fmaf(q, p, 1.f / 5.f);
    p = fmaf(q, p, 1.f / 3.f);
    p = fmaf(q, p, 1.f);
    return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

// ---------------------------------------------------------------- sequences
// Without cu: S sequences of T rows.  With cu: S sequences packed in T rows, bounds clamped
// to 0 .. T so that no table can send an access out of range.
struct Seqs {
    const int *cu;
    int S;
    long long T;
    __device__ __forceinline__ long long rows() const { return cu ? T : T * S; }
    __device__ __forceinline__ long long lo(int s) const {
        if (!cu) return T * s;
        const long long v = cu[s];
        return v < 0 ? 0 : v > T ? T : v;
    }
    __device__ __forceinline__ long long hi(int s) const {
        if (!cu) return T * (s + 1);
        const long long a = lo(s), b = lo(s + 1);
        return b < a ? a : b;
    }
    // the last sequence that starts at or before row r (0 if none does)
    __device__ __forceinline__ int at(long long r) const {
        if (!cu) return T > 0 ? (int)(r / T) : 0;
        int a = 0, b = S;   // lo(a) <= r (or a == 0), lo(b) > r (or b == S)
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (lo(m) <= r) a = m; else b = m;
        }
        return a;
    }
};

// A sequence's rows are cut into spans of L.  Slots number the spans of all sequences without
// a table of counts: dense, ceil(T / L) a sequence (one for an empty one); packed, sequence s
// starts at slot lo(s) / L + s, which leaves room for ceil(len / L) spans, one at least, and
// T / L + S slots in all.  A slot without a span has seq = -1.
struct Span {
    int seq, k, count;      // sequence, number in it, spans of it
    long long r0;           // first row
    int n;                  // rows
    long long first_slot;
};
__host__ __device__ __forceinline__ long long span_slots(bool packed, int S, long long T, long long L) {
    if (packed) return T / L + S;
    const long long per = (T + L - 1) / L;
    return (per > 0 ? per : 1) * S;
}
__device__ __forceinline__ long long first_slot(const Seqs &q, int s, long long L) {
    if (q.cu) return q.lo(s) / L + s;
    const long long per = (q.T + L - 1) / L;
    return (per > 0 ? per : 1) * s;
}
__device__ __forceinline__ Span span_at(const Seqs &q, long long slot, long long L) {
    Span x;
    int s;
    if (!q.cu) {
        const long long per = (q.T + L - 1) / L;
        s = (int)(slot / (per > 0 ? per : 1));
    } else {
        int a = 0, b = q.S;
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (q.lo(m) / L + m <= slot) a = m; else b = m;
        }
        s = a;
    }
    const long long lo = q.lo(s), len = q.hi(s) - lo;
    x.first_slot = first_slot(q, s, L);
    const long long k = slot - x.first_slot;
    x.count = len > 0 ? (int)((len + L - 1) / L) : 1;
    x.seq = (k >= 0 && k < x.count) ? s : -1;
    x.k = (int)k;
    x.r0 = lo + k * L;
    const long long left = len - k * L;
    x.n = (int)(left < L ? (left > 0 ? left : 0) : L);
    return x;
}

}  // namespace kda
