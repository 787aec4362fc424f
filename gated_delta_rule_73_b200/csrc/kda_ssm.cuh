// kda_ssm.cuh -- what the selective scan's kernels share: arguments and the lanes' layouts, decay
// rates, exponentials, the loads of a tile of B and C, the sums between lanes.
#pragma once
#include "kda_layers_internal.h"
#include "kda_rows.cuh"

#include <initializer_list>

namespace kda {

struct SsmP {
    const void *u, *dt, *Bm, *Cm, *z, *dout;
    const float *A, *Dskip, *dt_bias, *h0, *dh_T;
    void *out, *du, *ddt, *dz;
    float *h_T, *dh0;
    Seqs q;
    int D, G, Dg, cpg, nblk;   // channels, groups, channels a group, channel blocks a group, in all
    bool vec, vecb;            // whole vectors: channels of u, dt, z, out, dout; values of B and C
    bool vec_grad, vecb_sweep; // backward: channels of du, ddt, dz; B and C in the sweep
    int softplus;
    int L;                     // rows a span
    long long ld_u, ld_dt, ld_z, ld_B, ld_C, ld_out, slots;
    // workspace: states and their gradients at the spans' seams [slots][D][N], the spans' sums of
    // delta [slots][D], partial sums (backward)
    float *hst, *gst, *sdel, *part, *part_BC;   // part: [slots][part_ld], of dA, dDskip, ddt_bias
    long long part_ld;                          // D N + 2 D up to the next multiple of 4: rows of float4
};

constexpr int kTile = 16;       // tokens a tile of B and C

// ---------------------------------------------------------------- a lane a channel
constexpr int kFwdThreads = 128;
constexpr int kBatch = 4;       // tokens whose u, dt and z a channel's lanes hold at a time

// A channel's N states lie on NQ neighbouring lanes, SPT (at most 16) a lane.
template <int N>
struct FwdShape {
    static constexpr int SPT = N < 16 ? N : 16;
    static constexpr int NQ = N / SPT;
    static constexpr int CH = kFwdThreads / NQ;          // channels a block
    static constexpr int BATCH = NQ > kBatch ? NQ : kBatch;   // tokens whose u, dt and z a channel's lanes hold
    static constexpr int OWN = BATCH / NQ;               // of them, a lane's: q, q + NQ, ...
    static constexpr int BC = N / 4;                     // values of B and C a thread loads: 8 threads a token
};

// A log2(e), the exponent a unit of delta.  Finite where A is or is -inf: a token behind a span has
// delta = 0 and has to leave the state as it is.
__device__ __forceinline__ float rate(float a) {
    const float r = a * kLog2e;
    return r < -3.4028234e38f ? -3.4028234e38f : r;
}

// Sum of v[i] over the NQ lanes of a channel; lane q gets the sum of v[q].
template <int NQ>
__device__ __forceinline__ float reduce_states(float (&v)[NQ], int q) {
#pragma unroll
    for (int o = NQ / 2; o >= 1; o >>= 1) {
        const bool up = q & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// Where chunk c of a row of lanes' parts lies: eight threads that read chunks 2, 4 or 8 apart find
// them in different banks.  Chunks c to c + 7 of a thread that starts at a multiple c of 8 lie at
// spread(c) ^ 0 .. spread(c) ^ 7.
__device__ __forceinline__ int spread(int c) { return c ^ ((c >> 3) & 7); }

// The raw values of one tensor that a thread loads for its token and EPT channels.
template <typename T, int EPT>
__device__ __forceinline__ Raw<T, EPT> load_tile(const void *p, long long row, long long ld, int c, int left,
                                                 bool ok, bool vec) {
    const T *a = (const T *)p + row * ld + c;
    if (ok && vec && left >= EPT) return load_raw<T, EPT>(a);
    return load_part<T, EPT>(a, ok ? left : 0);
}

// A block's span and channels.
struct SsmBlock {
    Span sp;
    long long slot;
    int blk, g, cin;   // block of channels, its group, first channel within the group
};
__device__ __forceinline__ SsmBlock ssm_block(const SsmP &a, int CH) {
    SsmBlock b;
    b.slot = blockIdx.x / a.nblk;
    b.blk = blockIdx.x % a.nblk;
    b.g = b.blk / a.cpg;
    b.cin = (b.blk % a.cpg) * CH;
    b.sp = span_at(a.q, b.slot, a.L);
    return b;
}

// 2^x of two values on the FMA pipe, which has room while the special-function unit (16 results a
// clock and SM) is what the scans wait for.  x = n + f with f in [-1/2, 1/2]; 2^f = 1 + f p(f), p the
// polynomial of degree 5 through (2^f - 1) / f at its Chebyshev points: with the coefficients as they
// stand its relative error is 2^-26.7 anywhere (2^-23.7 with the roundings of its evaluation), and that of
// 2^f - 1 near 0 is 2^-28, which counts where factors close to 1 are multiplied thousands of times.  2^n is put together from n's bits.  Clamped to 2^-127 = 0 and 2^128 = inf;
// NaN stays NaN.
__device__ __forceinline__ float clamp_exponent(float x) {
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x));   // -127
    asm("min.NaN.f32 %0, %0, 0f43000000;" : "+f"(x));   // 128
    return x;
}
__device__ __forceinline__ float2 ex2_poly(float2 x) {
    constexpr float kRound = 12582912.f;   // 1.5 * 2^23: the sum's low bits are n
    x = make_float2(clamp_exponent(x.x), clamp_exponent(x.y));
    const float2 t = __fadd2_rn(x, make_float2(kRound, kRound));
    const float2 n = __fadd2_rn(t, make_float2(-kRound, -kRound));
    const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
    float2 p = make_float2(1.5453163e-4f, 1.5453163e-4f);
    p = __ffma2_rn(p, f, make_float2(1.3390863e-3f, 1.3390863e-3f));
    p = __ffma2_rn(p, f, make_float2(9.6180830e-3f, 9.6180830e-3f));
    p = __ffma2_rn(p, f, make_float2(5.5503570e-2f, 5.5503570e-2f));
    p = __ffma2_rn(p, f, make_float2(2.4022651e-1f, 2.4022651e-1f));
    p = __ffma2_rn(p, f, make_float2(6.9314718e-1f, 6.9314718e-1f));
    p = __ffma2_rn(p, f, make_float2(1.f, 1.f));
    const float2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                 __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
    return __fmul2_rn(p, s);
}

// Fills in sizes and layout for blocks of CH channels, of which a thread takes EPT neighbouring ones
// at a time, and BE values of B or C.  The kernels' own pointers are the launchers' to set.
template <int CH, int EPT, int BE>
SsmP ssm_params(const SsmArgs &a, int L) {
    SsmP p = {};
    p.u = a.u; p.dt = a.dt; p.Bm = a.Bm; p.Cm = a.Cm; p.z = a.z; p.dout = a.dout;
    p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias; p.h0 = a.h0; p.dh_T = a.dh_T;
    p.out = a.out; p.du = a.du; p.ddt = a.ddt; p.dz = a.dz; p.h_T = a.h_T; p.dh0 = a.dh0;
    p.q.cu = a.cu; p.q.S = a.S; p.q.T = a.T;
    p.D = a.D; p.G = a.G; p.Dg = a.D / a.G;
    p.cpg = (p.Dg + CH - 1) / CH;
    p.nblk = p.cpg * a.G;
    p.softplus = a.softplus;
    long long ld = a.ld_u | a.ld_dt | (a.z ? a.ld_z : 0) | a.ld_out;
    for (const void *r : {a.u, a.dt, a.z, (const void *)a.out, a.dout}) ld |= elements(r, a.bf16);
    // a whole vector of EPT channels is in the group, or none of it, and is aligned to 16 bytes or its size
    const int per16 = a.bf16 ? 8 : 4;
    p.vec = ld % (EPT < per16 ? EPT : per16) == 0 && p.Dg % EPT == 0;
    p.vecb = (a.ld_B | a.ld_C | elements(a.Bm, a.bf16) | elements(a.Cm, a.bf16)) % (BE < per16 ? BE : per16) == 0;
    p.L = L;
    p.ld_u = a.ld_u; p.ld_dt = a.ld_dt; p.ld_z = a.ld_z; p.ld_B = a.ld_B; p.ld_C = a.ld_C; p.ld_out = a.ld_out;
    p.slots = span_slots(a.cu != nullptr, a.S, a.T, L);
    return p;
}

// One token: the sequences in `count` parts of `per`, for 2368 blocks with `blocks` of channels.
struct StepParts {
    int per, count;
};
inline StepParts step_parts(int S, int blocks) {
    const int parts = 2368 / blocks > 1 ? 2368 / blocks : 1;
    StepParts x;
    x.per = (int)(((long long)S + parts - 1) / parts);
    x.count = (int)(((long long)S + x.per - 1) / x.per);
    return x;
}

// Start states of the spans (hst) from the spans' own ends, and, where gst is set, the
// gradients at the spans' ends from the spans' own gradients at their starts.
cudaError_t launch_ssm_seams(const SsmP &p, int N, cudaStream_t st);

}  // namespace kda
