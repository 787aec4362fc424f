// kda_ssm_scan.cu -- selective state space scan: forward over sequences, one-token step.
//
//   delta = softplus(dt + dt_bias),  h_t = exp(delta A) h_{t-1} + delta u B_t,
//   out = (C_t . h_t + Dskip u) z sigmoid(z)
//
// A channel's recurrence is sequential in time, its N states and all channels are independent;
// the states stay in registers.  One exponential a state and token: the special-function unit takes
// 16 a clock and SM (4.5e12 a second on the device), which bounds the scan before HBM does (8192
// tokens x 4096 channels x 16 states: 119 us of exponentials, 41 us of bytes).  Three ways, chosen by
// plan() from measured costs:
//
//  * whole sequences, a lane a channel (ssm_fwd_kernel): the fewest instructions an update (7.3),
//    for calls whose channels and sequences fill the device: 200 us for 64 x 128 x 4096 x 16, 75 % of
//    the special-function unit's rate.
//  * whole sequences, four states a lane (ssm_seq_kernel): four times the lanes, and warps of their
//    own for what surrounds the recurrence, so that a few thousand channels fill the device without
//    a second pass over the exponentials: 306 us for 8192 x 4096 x 16, where the first takes 1780.
//  * spans of time side by side (ssm_fwd_kernel twice): a span's effect on the state is
//    h -> exp(A sum delta) h + (its end from zero), so one sweep finds the ends of all spans, a small
//    pass chains them, and the spans then run side by side, for twice the exponentials: 82 us for
//    8192 x 256 x 16, where whole sequences take 301 at best.
#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace {

// ---------------------------------------------------------------- a lane a channel
template <typename T, int N, bool SWEEP>
__global__ void __launch_bounds__(kFwdThreads, 4) ssm_fwd_kernel(const SsmP a) {
    using S = FwdShape<N>;
    constexpr int SPT = S::SPT, NQ = S::NQ, CH = S::CH, BATCH = S::BATCH, OWN = S::OWN, BC = S::BC, P = SPT / 2;
    __shared__ __align__(16) float sBC[2][kTile][2 * N];
    const SsmBlock b = ssm_block(a, CH);
    if (b.sp.seq < 0 || (SWEEP && b.sp.k == b.sp.count - 1)) return;
    const int tid = threadIdx.x, ch = tid / NQ, q = tid % NQ, n = b.sp.n;
    const bool live = b.cin + ch < a.Dg;
    // lanes behind the last channel compute the first one's values again and store nothing
    const int c = b.g * a.Dg + b.cin + (live ? ch : 0);
    float2 A2[P], h[P];
    {
        const float *src = SWEEP      ? nullptr
                           : b.sp.k   ? a.hst + (b.slot * a.D + c) * N
                           : a.h0     ? a.h0 + ((long long)b.sp.seq * a.D + c) * N
                                      : nullptr;
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 v = *reinterpret_cast<const float4 *>(a.A + (long long)c * N + q * SPT + 2 * i);
            A2[i] = make_float2(rate(v.x), rate(v.y));
            A2[i + 1] = make_float2(rate(v.z), rate(v.w));
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (src) s = *reinterpret_cast<const float4 *>(src + q * SPT + 2 * i);
            h[i] = make_float2(s.x, s.y);
            h[i + 1] = make_float2(s.z, s.w);
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.Dskip ? a.Dskip[c] : 0.f;
    // B and C of the next tile, a token to eight threads
    const int bt = tid >> 3, bk = (tid & 7) * BC;
    const T *pbc = bk < N ? (const T *)a.Bm + (b.sp.r0 + bt) * a.ld_B + b.g * N + bk
                          : (const T *)a.Cm + (b.sp.r0 + bt) * a.ld_C + b.g * N + bk - N;
    const long long ldbc = bk < N ? a.ld_B : a.ld_C;
    auto fetch_bc = [&](int t0) {
        const bool ok = t0 + bt < n;
        const T *p = pbc + t0 * ldbc;
        return ok && a.vecb ? load_raw<T, BC>(p) : load_part<T, BC>(p, ok ? BC : 0);
    };
    auto put_bc = [&](const Raw<T, BC> &r, int buf) {
        float v[BC];
        widen<T, BC>(r, v);
#pragma unroll
        for (int i = 0; i < BC; ++i) sBC[buf][bt][bk + i] = v[i];
    };
    // The lane's own tokens of a batch.  A lane's offset is 32 bits wide and fixed, the rows' base is
    // the same for all lanes.
    const unsigned ou = (unsigned)(q * a.ld_u + c), od = (unsigned)(q * a.ld_dt + c), oz = (unsigned)(q * a.ld_z + c),
                   oo = (unsigned)(q * a.ld_out + c);
    const T *pu = (const T *)a.u + b.sp.r0 * a.ld_u, *pd = (const T *)a.dt + b.sp.r0 * a.ld_dt;
    const T *pz = (const T *)a.z + b.sp.r0 * a.ld_z;
    T *po = (T *)a.out + b.sp.r0 * a.ld_out;
    const bool gate = !SWEEP && a.z;
    T nu[OWN], nd[OWN], nz[OWN];
    auto fetch = [&](int left) {   // the batch at pu, pd, pz, of which `left` tokens are the span's
        if (left >= BATCH) {
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                nu[l] = (pu + l * NQ * a.ld_u)[ou];
                nd[l] = (pd + l * NQ * a.ld_dt)[od];
                if (gate) nz[l] = (pz + l * NQ * a.ld_z)[oz];
            }
        } else {
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                nu[l] = nd[l] = nz[l] = from_f32<T>(0.f);
                if (l * NQ + q < left) {
                    nu[l] = (pu + l * NQ * a.ld_u)[ou];
                    nd[l] = (pd + l * NQ * a.ld_dt)[od];
                    if (gate) nz[l] = (pz + l * NQ * a.ld_z)[oz];
                }
            }
        }
    };
    float dsum = 0.f;
    put_bc(fetch_bc(0), 0);
    fetch(n);
    for (int t0 = 0, buf = 0; t0 < n; t0 += kTile, buf ^= 1) {
        __syncthreads();   // this tile's B and C are there; the other buffer is read no more
        Raw<T, BC> rbc;
        if (t0 + kTile < n) rbc = fetch_bc(t0 + kTile);
#pragma unroll 1
        for (int b0 = 0; b0 < kTile; b0 += BATCH) {
            const int left = n - t0 - b0;
            if (left <= 0) break;
            float u[OWN], d[OWN], z[OWN], y[BATCH];
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                u[l] = to_f32(nu[l]);
                if (gate) z[l] = to_f32(nz[l]);
                d[l] = to_f32(nd[l]) + bias;
                if (a.softplus) d[l] = softplus_f32(d[l]);
            }
            if (left < BATCH)   // a token behind the span leaves the state as it is
#pragma unroll
                for (int l = 0; l < OWN; ++l)
                    if (l * NQ + q >= left) d[l] = 0.f;
            pu += BATCH * a.ld_u;
            pd += BATCH * a.ld_dt;
            pz += BATCH * a.ld_z;
            fetch(left - BATCH);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                float dl = d[i / NQ], x = dl * u[i / NQ];
                if (NQ > 1) {
                    dl = __shfl_sync(0xffffffffu, dl, i % NQ, NQ);
                    x = __shfl_sync(0xffffffffu, x, i % NQ, NQ);
                }
                const float *B = sBC[buf][b0 + i] + q * SPT, *C = B + N;
                const float2 d2 = make_float2(dl, dl), x2 = make_float2(x, x);
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                if (SWEEP) dsum += dl;
#pragma unroll
                for (int k = 0; k < P; k += 2) {
                    const float4 bv = *reinterpret_cast<const float4 *>(B + 2 * k);
                    float2 e0 = __fmul2_rn(d2, A2[k]), e1 = __fmul2_rn(d2, A2[k + 1]);
                    // two of 16 exponentials go to the FMA pipe: 2 % faster than none, and than four
                    e0 = k == 0 ? ex2_poly(e0) : make_float2(ex2(e0.x), ex2(e0.y));
                    e1 = make_float2(ex2(e1.x), ex2(e1.y));
                    h[k] = __ffma2_rn(e0, h[k], __fmul2_rn(x2, make_float2(bv.x, bv.y)));
                    h[k + 1] = __ffma2_rn(e1, h[k + 1], __fmul2_rn(x2, make_float2(bv.z, bv.w)));
                    if (!SWEEP) {
                        const float4 cv = *reinterpret_cast<const float4 *>(C + 2 * k);
                        s0 = __ffma2_rn(make_float2(cv.x, cv.y), h[k], s0);
                        s1 = __ffma2_rn(make_float2(cv.z, cv.w), h[k + 1], s1);
                    }
                }
                s0 = __fadd2_rn(s0, s1);
                y[i] = s0.x + s0.y;
            }
            if (!SWEEP) {
#pragma unroll
                for (int l = 0; l < OWN; ++l) {
                    float v[NQ];
#pragma unroll
                    for (int j = 0; j < NQ; ++j) v[j] = y[l * NQ + j];
                    float o = fmaf(skip, u[l], reduce_states<NQ>(v, q));
                    if (gate) o *= silu_f32(z[l]);
                    if (live && l * NQ + q < left) (po + l * NQ * a.ld_out)[oo] = from_f32<T>(o);
                }
                po += BATCH * a.ld_out;
            }
        }
        if (t0 + kTile < n) put_bc(rbc, buf ^ 1);
    }
    if (!live) return;
    float *dst = SWEEP ? a.hst + (b.slot * a.D + c) * N
                 : a.h_T && b.sp.k == b.sp.count - 1 ? a.h_T + ((long long)b.sp.seq * a.D + c) * N : nullptr;
    if (dst)
#pragma unroll
        for (int i = 0; i < P; i += 2)
            *reinterpret_cast<float4 *>(dst + q * SPT + 2 * i) = make_float4(h[i].x, h[i].y, h[i + 1].x, h[i + 1].y);
    if (SWEEP && q == 0) a.sdel[b.slot * a.D + c] = dsum;
}

// ---------------------------------------------------------------- lanes for states
// Warps 0-3 run the recurrence, one each a scheduler: N / 4 lanes a channel, four states a lane.  The
// other eight load the next tile, work out delta and delta u, and turn the last-but-one tile's parts
// of C . h into outputs; three tiles are on the way.  Nothing but two barriers a tile ties the two
// kinds together, so that the recurrence's dependent steps run while the others wait for memory.
// Two blocks fit an SM: one alone takes 38 ns a token (32 channels x 16 states), two 65.

// bar.sync / bar.arrive of all of a block's threads
template <int THREADS>
__device__ __forceinline__ void wait_at(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory"); }
template <int THREADS>
__device__ __forceinline__ void arrive_at(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory"); }

template <typename T, int N>
struct SeqShape {
    static constexpr int SPT = 4;                      // states a lane
    static constexpr int SCAN = 128, HELP = 256, THREADS = SCAN + HELP;   // threads of either kind
    static constexpr int NL = N / SPT;                 // lanes a channel
    static constexpr int CH = SCAN / NL;               // channels a block
    static constexpr int TT = CH >= 64 ? 16 : 32;      // tokens a tile
    static constexpr int E = TT * CH / HELP > 0 ? TT * CH / HELP : 1;   // (token, channel) places a helper thread has in a tile
    static constexpr int EV = E < 4 ? E : 4;           // neighbouring channels of them
    static constexpr int PASS = E / EV;
    static constexpr int TPR = CH / EV;                // threads a token
    static constexpr int TSTEP = HELP / TPR;           // tokens between a thread's places
    static constexpr int VB = TT * 2 * N / HELP;       // values of B and C a helper thread loads
    static constexpr int BPT = 2 * N / VB;             // threads a token
    static constexpr int STAGES = 3;
    struct Stage {
        float2 x[TT][CH];              // delta, delta u
        float bc[TT][2 * N];
        float y[TT][SCAN];             // the lanes' parts of C . h
        T u[TT][CH], z[TT][CH];
    };
};

// The sequence that is the rank-th longest of up to 32, whole: blocks start in the order of their
// numbers, and a long sequence that starts last is what all others then wait for.  8192 x 1024 x 16 in
// 20 random sequences: 81 us against 107 in the order given; 3001 x 1002 x 32 in 7: 54 to 62 against 64
// to 74.  Not where a sequence's blocks alone would share SMs by twos while others run (8100 x 4096 x
// 16, all but 100 rows one sequence: 515 us where it comes first, 303 where it comes last), nor for
// short ones, which the ranking would hold up (64 x 2048 x 16 in 32: 51 against 39).
__device__ __forceinline__ Span longest_first(const Seqs &q, int rank) {
    const int lane = threadIdx.x & 31;
    const int len = lane < q.S ? (int)(q.hi(lane) - q.lo(lane)) : -1;
    int before = 0;
    for (int j = 0; j < q.S; ++j) {
        const int other = __shfl_sync(0xffffffffu, len, j);
        before += other > len || (other == len && j < lane);
    }
    Span x = {};
    x.seq = __reduce_max_sync(0xffffffffu, lane < q.S && before == rank ? lane : -1);
    x.count = 1;
    if (x.seq >= 0) {
        x.r0 = q.lo(x.seq);
        x.n = (int)(q.hi(x.seq) - x.r0);
    }
    return x;
}

template <typename T, int N, bool RANKED>
__global__ void __launch_bounds__(SeqShape<T, N>::THREADS, 2) ssm_seq_kernel(const SsmP a) {
    using S = SeqShape<T, N>;
    constexpr int SPT = S::SPT, NL = S::NL, CH = S::CH, TT = S::TT, EV = S::EV, PASS = S::PASS, TPR = S::TPR, TSTEP = S::TSTEP, VB = S::VB,
                  BPT = S::BPT, ST = S::STAGES, ALL = S::THREADS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename S::Stage *stage = reinterpret_cast<typename S::Stage *>(smem_raw);
    SsmBlock b = ssm_block(a, CH);
    if (RANKED) b.sp = longest_first(a.q, (int)b.slot);
    if (b.sp.seq < 0) return;
    // rows are fewer than 2^31; out of the ranking they take registers of every thread, of which none are left
    using Row = typename std::conditional<RANKED, int, long long>::type;
    const Row r0 = (Row)b.sp.r0;
    const int seq = b.sp.seq;
    const int n = b.sp.n, tiles = (n + TT - 1) / TT;
    const int FULL = 1, DONE = 1 + ST;
    if (threadIdx.x < S::SCAN) {
        const int tid = threadIdx.x, ch = tid / NL, q = tid % NL;
        const bool live = b.cin + ch < a.Dg;
        const long long c = (long long)b.g * a.Dg + b.cin + (live ? ch : 0);
        const int at_y = spread(tid >> 2) * 4 + (tid & 3);
        float A2[SPT], h[SPT];
        load_f32<float, SPT>(a.A + c * N + q * SPT, A2);
        const float *src = a.h0 ? a.h0 + ((long long)seq * a.D + c) * N : nullptr;
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
            A2[i] = rate(A2[i]);
            h[i] = 0.f;
        }
        if (src) load_f32<float, SPT>(src + q * SPT, h);
        for (int i = 0; i < tiles; ++i) {
            typename S::Stage &s = stage[i % ST];
            wait_at<ALL>(FULL + i % ST);
            // Four tokens at a time: their decay factors and inputs are worked out while the four
            // before them go through the recurrence, so that its dependent steps and the exponentials'
            // latency overlap.
            float e[4][SPT], in[4][SPT];
            auto ahead = [&](int j, int t) {
                const float2 x = s.x[t][ch];
                float bv[SPT];
                load_f32<float, SPT>(&s.bc[t][q * SPT], bv);
#pragma unroll
                for (int k = 0; k < SPT; k += 2) {
                    const float2 m = __fmul2_rn(make_float2(x.x, x.x), make_float2(A2[k], A2[k + 1]));
                    const float2 r = __fmul2_rn(make_float2(x.y, x.y), make_float2(bv[k], bv[k + 1]));
                    e[j][k] = ex2(m.x);
                    e[j][k + 1] = ex2(m.y);
                    in[j][k] = r.x;
                    in[j][k + 1] = r.y;
                }
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) ahead(j, j);
#pragma unroll
            for (int t = 0; t < TT; t += 4) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float cv[SPT];
                    load_f32<float, SPT>(&s.bc[t + j][N + q * SPT], cv);
                    float2 sum;
#pragma unroll
                    for (int k = 0; k < SPT; k += 2) {
                        const float2 hk = __ffma2_rn(make_float2(e[j][k], e[j][k + 1]), make_float2(h[k], h[k + 1]),
                                                     make_float2(in[j][k], in[j][k + 1]));
                        h[k] = hk.x;
                        h[k + 1] = hk.y;
                        sum = k ? __ffma2_rn(make_float2(cv[k], cv[k + 1]), hk, sum) : __fmul2_rn(make_float2(cv[0], cv[1]), hk);
                    }
                    y[j] = sum.x + sum.y;
                    if (t + 4 < TT) ahead(j, t + 4 + j);
                }
                // behind the loads ahead, which could not pass them
#pragma unroll
                for (int j = 0; j < 4; ++j) s.y[t + j][at_y] = y[j];
            }
            arrive_at<ALL>(DONE + i % ST);
        }
        if (!live) return;
        if (a.h_T) store_f32<float, SPT>(a.h_T + ((long long)seq * a.D + c) * N + q * SPT, h);
        return;
    }
    // helpers
    const int tid = threadIdx.x - S::SCAN;
    const int lt = tid / TPR, lc = tid % TPR * EV;
    const int left = a.Dg - b.cin - lc;                       // channels of the group from the thread's first on
    const int c = b.g * a.Dg + b.cin + lc;
    const bool gate = a.z != nullptr;
    float bias[EV], skip[EV];
#pragma unroll
    for (int k = 0; k < EV; ++k) {
        bias[k] = a.dt_bias && k < left ? a.dt_bias[c + k] : 0.f;
        skip[k] = a.Dskip && k < left ? a.Dskip[c + k] : 0.f;
    }
    const int bt = tid / BPT, bk = tid % BPT * VB;
    const bool is_b = bk < N;
    const T *pbc = is_b ? (const T *)a.Bm + (long long)(r0 + bt) * a.ld_B + b.g * N + bk
                        : (const T *)a.Cm + (long long)(r0 + bt) * a.ld_C + b.g * N + bk - N;
    const long long ldbc = is_b ? a.ld_B : a.ld_C;
    constexpr int DEPTH = 2;   // a tile's loads are two tiles on the way: a tile takes a microsecond, HBM's latency is more
    struct Next {
        Raw<T, EV> u[PASS], d[PASS], z[PASS];
        Raw<T, VB> bc;
    } next[DEPTH];
    auto fetch = [&](Next &x, int t0) {
#pragma unroll
        for (int p = 0; p < PASS; ++p) {
            const int t = t0 + p * TSTEP + lt;
            const bool ok = t < n && p * TSTEP + lt < TT;
            x.u[p] = load_tile<T, EV>(a.u, r0 + t, a.ld_u, c, left, ok, a.vec);
            x.d[p] = load_tile<T, EV>(a.dt, r0 + t, a.ld_dt, c, left, ok, a.vec);
            if (gate) x.z[p] = load_tile<T, EV>(a.z, r0 + t, a.ld_z, c, left, ok, a.vec);
        }
        const bool ok = t0 + bt < n;
        x.bc = ok && a.vecb ? load_raw<T, VB>(pbc + t0 * ldbc) : load_part<T, VB>(pbc + t0 * ldbc, ok ? VB : 0);
    };
    auto tile = [&](int i, Next &cur) {
        if (i < tiles) {
            typename S::Stage &s = stage[i % ST];
            const int t0 = i * TT;
#pragma unroll
            for (int p = 0; p < PASS; ++p) {
                const int t = p * TSTEP + lt;
                if (t >= TT) break;
                float u[EV], d[EV], x[2 * EV];
                widen<T, EV>(cur.u[p], u);
                widen<T, EV>(cur.d[p], d);
#pragma unroll
                for (int k = 0; k < EV; ++k) {
                    d[k] += bias[k];
                    if (a.softplus) d[k] = softplus_f32(d[k]);
                    if (t0 + t >= n || k >= left) d[k] = 0.f;   // a token behind the span leaves the state as it is
                    x[2 * k] = d[k];
                    x[2 * k + 1] = d[k] * u[k];
                }
                store_f32<float, 2 * EV>(&s.x[t][lc].x, x);
                store_raw<T, EV>(&s.u[t][lc], cur.u[p]);
                if (gate) store_raw<T, EV>(&s.z[t][lc], cur.z[p]);
            }
            float v[VB];
            widen<T, VB>(cur.bc, v);
            store_f32<float, VB>(&s.bc[bt][bk], v);
            if (i + DEPTH < tiles) fetch(cur, t0 + DEPTH * TT);
            arrive_at<ALL>(FULL + i % ST);
        }
        if (i >= 2) {
            typename S::Stage &s = stage[(i - 2) % ST];
            const int t0 = (i - 2) * TT;
            wait_at<ALL>(DONE + (i - 2) % ST);
#pragma unroll
            for (int p = 0; p < PASS; ++p) {
                const int t = p * TSTEP + lt;
                if (t >= TT || t0 + t >= n) break;
                float u[EV], z[EV], y[EV];
                load_f32<T, EV>(&s.u[t][lc], u);
                if (gate) load_f32<T, EV>(&s.z[t][lc], z);
                float part[EV * NL];
#pragma unroll
                for (int m = 0; m < EV * NL; m += 4)
                    load_f32<float, 4>(&s.y[t][spread((lc * NL + m) >> 2) * 4], part + m);
#pragma unroll
                for (int k = 0; k < EV; ++k) {
#pragma unroll
                    for (int o = NL / 2; o >= 1; o /= 2)
#pragma unroll
                        for (int m = 0; m < o; ++m) part[k * NL + m] += part[k * NL + m + o];
                    y[k] = fmaf(skip[k], u[k], part[k * NL]);
                    if (gate) y[k] *= silu_f32(z[k]);
                }
                T *o = (T *)a.out + (long long)(r0 + t0 + t) * a.ld_out + c;
                if (a.vec && left >= EV) store_f32<T, EV>(o, y);
                else store_part<T, EV>(o, y, left);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) fetch(next[j], j * TT);
    for (int i = 0; i < tiles + 2; i += DEPTH)
#pragma unroll
        for (int j = 0; j < DEPTH; ++j)
            if (i + j < tiles + 2) tile(i + j, next[j]);
}

// One thread per sequence and four states walks the spans: forward, hst[slot] goes from the
// slot's own end to its start state; with gst, backward, gst[slot] goes from the gradient at the
// span's start that its own outputs make to the gradient at its end that later spans make.  Eight
// spans' values are loaded ahead of the chain through them.
__global__ void __launch_bounds__(128) ssm_seams_kernel(const SsmP a, int N) {
    constexpr int U = 8;
    const long long per = (long long)a.D * N / 4;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    if (id >= per * a.q.S) return;
    const int s = (int)(id / per);
    const long long e = id % per * 4, c = e / N;   // state within [D][N]
    const long long len = a.q.hi(s) - a.q.lo(s);
    const int count = len > 0 ? (int)((len + a.L - 1) / a.L) : 1;
    const long long slot0 = first_slot(a.q, s, a.L), all = (long long)a.D * N;
    const bool back = blockIdx.y != 0;
    float A2[4], v[4] = {0.f, 0.f, 0.f, 0.f};
    load_f32<float, 4>(a.A + e, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = rate(A2[i]);
    const float *from = back ? a.dh_T : a.h0;
    if (from) load_f32<float, 4>(from + s * all + e, v);
    float *seam = back ? a.gst : a.hst;
    // the values that no span wrote, or that nothing needs: the last span's end, the first one's
    // gradient where the start state has none
    const int unread = back ? (a.dh0 ? -1 : 0) : count - 1;
    for (int k0 = 0; k0 < count; k0 += U) {
        float own[U][4], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = back ? count - 1 - k0 - j : k0 + j;
            d[j] = own[j][0] = own[j][1] = own[j][2] = own[j][3] = 0.f;
            if (k >= 0 && k < count && k != unread && len > 0) {
                load_f32<float, 4>(seam + (slot0 + k) * all + e, own[j]);
                d[j] = a.sdel[(slot0 + k) * a.D + c];
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = back ? count - 1 - k0 - j : k0 + j;
            if (k >= 0 && k < count) {
                store_f32<float, 4>(seam + (slot0 + k) * all + e, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(ex2(A2[i] * d[j]), v[i], own[j][i]);
            }
        }
    }
    if (back && a.dh0) store_f32<float, 4>(a.dh0 + s * all + e, v);
}

// One token: bound by the states' bytes, read and written once.  A lane holds four states of a channel,
// its parameters with them, and walks sequences, R at a time, the next R's loads under way.  What a
// sequence and channel has once (delta, the gate) is worked out by one lane (of each R) and handed round.
template <typename T, int N, int R>
__global__ void __launch_bounds__(128) ssm_step_kernel(const SsmP a, int per) {
    constexpr int NQ = N / 4;
    static_assert(R <= NQ, "a lane for each sequence");
    const int unit = blockIdx.x * (128 / NQ) + threadIdx.x / NQ, q = threadIdx.x % NQ, own = q % R;
    const bool live = unit < a.D;                        // lanes of a channel agree
    const int c = live ? unit : 0, g = c / a.Dg;
    const int s1 = (blockIdx.y + 1) * per < a.q.S ? (blockIdx.y + 1) * per : a.q.S;
    float nh[R][4];
    Raw<T, 4> nB[R], nC[R];
    T nu, ndt, nz;
    const T *pB = (const T *)a.Bm + g * N + 4 * q, *pC = (const T *)a.Cm + g * N + 4 * q;
    const float *ph = a.h0 + (long long)c * N + 4 * q;
    const long long hs = (long long)a.D * N;             // states of a sequence
    auto fetch = [&](int s) {                            // past the last: the last again, not stored
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long t = s + r < s1 ? s + r : s1 - 1;
            load_f32<float, 4>(ph + t * hs, nh[r]);
            nB[r] = a.vecb ? load_raw<T, 4>(pB + t * a.ld_B) : load_part<T, 4>(pB + t * a.ld_B, 4);
            nC[r] = a.vecb ? load_raw<T, 4>(pC + t * a.ld_C) : load_part<T, 4>(pC + t * a.ld_C, 4);
        }
        const long long t = s + own < s1 ? s + own : s1 - 1;
        nu = ((const T *)a.u)[t * a.ld_u + c];
        ndt = ((const T *)a.dt)[t * a.ld_dt + c];
        if (a.z) nz = ((const T *)a.z)[t * a.ld_z + c];
    };
    int s = blockIdx.y * per;
    if (s >= s1) return;
    fetch(s);
    float A[4];
    load_f32<float, 4>(a.A + (long long)c * N + 4 * q, A);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.Dskip ? a.Dskip[c] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) A[i] = rate(A[i]);
    for (; s < s1; s += R) {
        float h[R][4], y[R];
        Raw<T, 4> B[R], C[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            B[r] = nB[r];
            C[r] = nC[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[r][i] = nh[r][i];
        }
        const float u = to_f32(nu), z = a.z ? to_f32(nz) : 0.f;
        float d = to_f32(ndt) + bias;
        if (s + R < s1) fetch(s + R);
        if (a.softplus) d = softplus_f32(d);
        const float x = d * u;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float bv[4], cv[4];
            widen<T, 4>(B[r], bv);
            widen<T, 4>(C[r], cv);
            const float dr = R > 1 ? __shfl_sync(0xffffffffu, d, r, NQ) : d;
            const float xr = R > 1 ? __shfl_sync(0xffffffffu, x, r, NQ) : x;
            y[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(ex2(dr * A[i]), h[r][i], xr * bv[i]);
                y[r] = fmaf(cv[i], h[r][i], y[r]);
            }
#pragma unroll
            for (int o = NQ / 2; o >= R; o >>= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
            if (live && s + r < s1) store_f32<float, 4>(a.h_T + (s + r) * hs + (long long)c * N + 4 * q, h[r]);
        }
        float o = fmaf(skip, u, reduce_states<R>(y, own));
        if (a.z) o *= silu_f32(z);
        if (live && q < R && s + own < s1) ((T *)a.out)[(long long)(s + own) * a.ld_out + c] = from_f32<T>(o);
    }
}

// Which kernel, and the rows a span takes (L >= T: whole sequences).  Estimated nanoseconds, from
// measurements on a B200 between 256 and 12288 channels, 128 and 8192 tokens, 8 and 64 states:
//   four states a lane   a token 38 with one block a SM, 65 with two, and so on in pairs
//   a lane a channel     a token 100 + 105 k, k warps a scheduler (at least one), from four on 68 + 113 k
//   spans                0.00076 an update and 0.0024 a channel and token, and 20 us for its passes
// Packed sequences' lengths are not known here.  The longest counts as 1.5 times the mean for four states
// a lane, whose blocks queue and share the SMs evenly, and as twice the mean for a lane a channel,
// whose blocks run at once and wait for the longest (8192 x 4096 x 16 in 20 random sequences: 257
// to 277 us against 306 to 499; 64 x 2048 x 16 in 32 sequences: 39 against 8).  A span holds twice
// the mean of as many rows as spans are wanted, so that even sequences stay whole.
struct FwdPlan {
    bool lanes;   // four states a lane
    int L;
};
FwdPlan plan(const SsmArgs &a) {
    const int Dg = a.D / a.G, ch_seq = 512 / a.N, ch = kFwdThreads / (a.N <= 16 ? 1 : a.N / 16);
    const long long rows = a.rows, whole = a.T > 0 ? a.T : 1;
    const long long blocks_seq = (long long)a.S * a.G * ((Dg + ch_seq - 1) / ch_seq), per_span = (long long)a.G * ((Dg + ch - 1) / ch);
    const double k = (double)per_span * a.S / 148.0;   // warps a scheduler: blocks of four warps
    double t_seq, t_whole;
    if (a.cu && a.S > 1) {
        const double mean = (double)rows / a.S, some = 100.0 + 105.0 * (k > 4.0 ? 4.0 : k > 1.0 ? k : 1.0);
        t_seq = fmax(1.5 * mean * (blocks_seq > 148 ? 65.0 : 38.0), blocks_seq / 148.0 * (mean * 36.0 + 3000.0));
        t_whole = fmax(2.0 * mean * some, mean * (68.0 + 113.0 * k));
    } else {
        const long long n = (blocks_seq + 147) / 148;
        t_seq = a.T * (n / 2 * 65.0 + n % 2 * 38.0);
        t_whole = a.T * (k <= 4.0 ? 100.0 + 105.0 * (k > 1.0 ? k : 1.0) : 68.0 + 113.0 * k);
    }
    const double t_span = (double)rows * a.D * (0.00076 * a.N + 0.0024) + 20000.0;
    if (t_span < t_seq && t_span < t_whole) {
        const long long want = 592 / per_span > 1 ? 592 / per_span : 1;   // spans in all: one wave of 4 blocks a SM
        const long long m = want > a.S ? want : a.S;
        long long L = a.cu ? (2 * rows + m - 1) / m : (rows + want - 1) / want;
        L = (L + kTile - 1) / kTile * kTile;
        if (L < 64) L = 64;
        if (L < whole) return {false, (int)L};
    }
    return {t_seq < t_whole, (int)whole};
}

template <typename T, int N>
cudaError_t run_seq(const SsmArgs &a, cudaStream_t st) {
    using S = SeqShape<T, N>;
    const SsmP p = ssm_params<S::CH, S::EV, S::VB>(a, a.T > 0 ? (int)a.T : 1);
    const long long blocks = p.slots * p.nblk;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    constexpr int smem = sizeof(typename S::Stage) * S::STAGES;
    // see longest_first
    const bool ranked = a.cu && a.S <= 32 && a.T >= 128LL * a.S && p.nblk <= 74;
    const auto kernel = ranked ? ssm_seq_kernel<T, N, true> : ssm_seq_kernel<T, N, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    a.marks->mark(st);
    kernel<<<(unsigned)blocks, S::THREADS, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int N>
cudaError_t run_fwd(const SsmArgs &a, cudaStream_t st) {
    const FwdPlan f = plan(a);
    if (f.lanes) return run_seq<T, N>(a, st);
    using F = FwdShape<N>;
    SsmP p = ssm_params<F::CH, 1, F::BC>(a, f.L);
    const long long blocks = p.slots * p.nblk;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.L < a.T) {
        p.hst = (float *)a.workspace;
        p.sdel = p.hst + p.slots * a.D * N;
        a.marks->mark(st);
        ssm_fwd_kernel<T, N, true><<<(unsigned)blocks, kFwdThreads, 0, st>>>(p);
        a.marks->mark(st);
        const cudaError_t e = launch_ssm_seams(p, N, st);
        if (e != cudaSuccess) return e;
    }
    a.marks->mark(st);
    ssm_fwd_kernel<T, N, false><<<(unsigned)blocks, kFwdThreads, 0, st>>>(p);
    return cudaGetLastError();
}
// Blocks of 128 / (N / 4) channels, and as many parts of the sequences as make 2368 blocks; four
// sequences at a time where a part has them.  256 x 12288 x 16 in bf16: 80 us (83 with twice the
// blocks); with every lane working out delta and the gate 85; a lane for each sequence, no walk, 115.
template <typename T, int N>
cudaError_t run_step(const SsmArgs &a, cudaStream_t st) {
    const SsmP p = ssm_params<1, 1, 4>(a, 1);
    constexpr int R = N == 8 ? 2 : 4;
    const int blocks = (a.D + 512 / N - 1) / (512 / N);
    const StepParts x = step_parts(a.S, blocks);
    if (x.count > 65535) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)x.count);
    a.marks->mark(st);
    if (x.per >= R) ssm_step_kernel<T, N, R><<<grid, 128, 0, st>>>(p, x.per);
    else ssm_step_kernel<T, N, 1><<<grid, 128, 0, st>>>(p, x.per);
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
    const int L = plan(a).L;
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
