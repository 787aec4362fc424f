// kda_rows.cuh -- what the short convolution, the selective scan and the block norm share:
// vector access to rows, activations in full FP32 accuracy, sequence bounds and spans.
#pragma once
#include "kda_common.cuh"

namespace kda {

// ---------------------------------------------------------------- V consecutive values
// V * sizeof(T) is 2, 4, 8, 16, 32 or 64 bytes; a whole access wants the address to be a multiple
// of min(that, 16).  Values stay in the words that were loaded until widen(): a value taken out of
// its word earlier, where two ways of loading meet, would make the thread wait for the load there.
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p) {
    using R = Raw<T, V>;
    R r;
    if constexpr (R::kBytes == 2) {
        r.w[0] = *reinterpret_cast<const unsigned short *>(p);
    } else if constexpr (R::kBytes == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (R::kBytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < R::kWords; i += 4) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i / 4];
            r.w[i] = v.x;
            r.w[i + 1] = v.y;
            r.w[i + 2] = v.z;
            r.w[i + 3] = v.w;
        }
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, V> &r) {
    using R = Raw<T, V>;
    if constexpr (R::kBytes == 2) {
        *reinterpret_cast<unsigned short *>(p) = (unsigned short)r.w[0];
    } else if constexpr (R::kBytes == 4) {
        *reinterpret_cast<uint32_t *>(p) = r.w[0];
    } else if constexpr (R::kBytes == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < R::kWords; i += 4)
            reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V> &r, float *x) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __uint_as_float(r.w[i]);
    } else {   // bf16 is the upper half of FP32
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> narrow(const float *x) {
    Raw<T, V> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(x[i]);
    } else if constexpr (V == 1) {
        r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[i], x[i + 1]);
            r.w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return r;
}
// The first n values (n <= 0: none) one by one; the others are zero.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_part(const T *p, int n) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kWords; ++i) r.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n) {
            if constexpr (sizeof(T) == 4) r.w[i] = reinterpret_cast<const uint32_t *>(p)[i];
            else r.w[i / 2] |= (uint32_t)reinterpret_cast<const unsigned short *>(p)[i] << (i & 1 ? 16 : 0);
        }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void load_f32(const T *p, float *x) {
    widen<T, V>(load_raw<T, V>(p), x);
}
template <typename T, int V>
__device__ __forceinline__ void store_f32(T *p, const float *x) {
    store_raw<T, V>(p, narrow<T, V>(x));
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, const float *x, int n) {
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n) p[i] = from_f32<T>(x[i]);
}

// ---------------------------------------------------------------- activations
// Relative error of at most 12 + 1.23 |x| half-steps of FP32 (2^-24) where x < 0 and 12 where x > 0
// (measured up to |x| = 87: 4 + 1.23 |x| and 4).  1.23 |x| is what the rounding of log2(e) x makes, with
// log2(e)'s own (0.22 of a half-step): 6 half-steps at x = -5, where sigmoid is 0.7 %, 74 at -60, where it
// is 10^-26.  Below 2^-126, from x = -87.3 on, sigmoid and softplus are 0.  The limits are exact:
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

// log(1 + e^x) = max(x, 0) + 2 atanh(e / (2 + e)) with e = exp(-|x|) in (0, 1]: atanh in
// s = e / (2 + e) <= 1/3 keeps the relative precision of small values, which log2(1 + e) loses.
// atanh(s) / s is a polynomial of degree 4 in s^2 through the Chebyshev points of [0, 1/9]
// (relative error 2^-27).
__device__ __forceinline__ float softplus_f32(float x) {
    const float e = ex2(-kLog2e * fabsf(x));
    const float s = e * rcp(2.f + e);
    const float q = s * s;
    float p = fmaf(q, 0.14078889f, 0.13982579f);
    p = fmaf(q, p, 0.20012298f);
    p = fmaf(q, p, 0.33333161f);
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
    __host__ __device__ __forceinline__ long long rows() const { return cu ? T : T * S; }
    __host__ __device__ __forceinline__ long long lo(int s) const {
        if (!cu) return T * s;
        const long long v = cu[s];
        return v < 0 ? 0 : v > T ? T : v;
    }
    __host__ __device__ __forceinline__ long long hi(int s) const {
        if (!cu) return T * (s + 1);
        const long long a = lo(s), b = lo(s + 1);
        return b < a ? a : b;
    }
    // the last sequence that starts at or before row r (0 if none does)
    __host__ __device__ __forceinline__ int at(long long r) const {
        if (!cu) return T > 0 ? (int)(r / T) : 0;
        int a = 0, b = S;   // lo(a) <= r (or a == 0), lo(b) > r (or b == S)
        while (b - a > 1) {
            const int m = a + ((b - a) >> 1);   // a + b may not fit an int
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
__host__ __device__ __forceinline__ long long first_slot(const Seqs &q, int s, long long L) {
    if (q.cu) return q.lo(s) / L + s;
    const long long per = (q.T + L - 1) / L;
    return (per > 0 ? per : 1) * s;
}
__host__ __device__ __forceinline__ Span span_at(const Seqs &q, long long slot, long long L) {
    Span x;
    int s;
    if (!q.cu) {
        const long long per = (q.T + L - 1) / L;
        s = (int)(slot / (per > 0 ? per : 1));
    } else {
        int a = 0, b = q.S;
        while (b - a > 1) {
            const int m = a + ((b - a) >> 1);   // a + b may not fit an int
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
