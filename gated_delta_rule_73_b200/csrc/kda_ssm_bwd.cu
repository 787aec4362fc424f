// kda_ssm_bwd.cu -- backward of the selective state space scan.
//
// With a_t = exp(delta_t A), dy = dout silu(z), e_t the gradient of h_t:
//   e_t = C_t dy_t + a_{t+1} e_{t+1}   (behind the last token: dh_T)
//   dC_t = sum_d dy_t h_t,   dB_t = sum_d e_t delta_t u_t,   dA = sum_t e_t delta_t a_t h_{t-1}
//   ddelta_t = sum_n e_t a_t h_{t-1} A + u_t sum_n e_t B_t,   du_t = Dskip dy_t + delta_t sum_n e_t B_t
//   dz_t = dout_t y_t silu'(z_t),   ddt = ddelta sigmoid(dt + dt_bias),   dh0 = a_1 e_1
//
// Time is cut into spans of up to 64 tokens that run side by side.  One sweep finds for every span its
// end state from zero and, with the running product P of the a, the gradient at its start that
// its own outputs make, sum_t P_t C_t dy_t: both go forward, on the same exponentials.  A small
// pass chains the spans.  The main kernel then walks its span forward once, keeping the state
// every 8 tokens in shared memory, and goes back over windows of 4 tokens whose states and decay
// factors stay in registers (the first four tokens of 8 are walked again for the second four):
// 3.4 exponentials a state and token in all, no state in HBM but at the spans' seams.  It is bound
// by issue slots and latencies (31.5 instructions a state and token, 43 % of the slots, 11 warps an
// SM): the products of the formulas above, on packed pairs, and the sums between lanes.  4096 tokens
// x 2048 channels x 16 states in bf16: sweep 67 us, chain 8, main kernel 273, last sums 8.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kSpan = 64;      // tokens a span, at most

// Both sweeps of a span: end state from zero (hst), gradient at the start (gst), sum of delta.
// Lanes and loads as in the forward's ssm_fwd_kernel: a lane a channel, 16 states.
template <typename T, int N>
__global__ void __launch_bounds__(kFwdThreads, 3) ssm_bwd_sweep_kernel(const SsmP a) {
    using S = FwdShape<N>;
    constexpr int SPT = S::SPT, NQ = S::NQ, CH = S::CH, BATCH = S::BATCH, OWN = S::OWN, BC = S::BC, P = SPT / 2;
    __shared__ __align__(16) float sBC[2][kTile][2 * N];
    SsmP f = a;                                    // this kernel's blocks of channels
    f.cpg = (a.Dg + CH - 1) / CH;
    f.nblk = f.cpg * a.G;
    const SsmBlock b = ssm_block(f, CH);
    if (b.sp.seq < 0 || (b.sp.count == 1 && !a.dh0)) return;
    const int tid = threadIdx.x, ch = tid / NQ, q = tid % NQ, n = b.sp.n;
    const bool live = b.cin + ch < a.Dg;
    const int c = b.g * a.Dg + b.cin + (live ? ch : 0);
    float2 A2[P], h[P], G[P], W[P];                // W: the running product of the decay factors
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(a.A + (long long)c * N + q * SPT + 2 * i);
        A2[i] = make_float2(rate(v.x), rate(v.y));
        A2[i + 1] = make_float2(rate(v.z), rate(v.w));
        h[i] = h[i + 1] = G[i] = G[i + 1] = make_float2(0.f, 0.f);
        W[i] = W[i + 1] = make_float2(1.f, 1.f);
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const int bt = tid >> 3, bk = (tid & 7) * BC;
    const T *pbc = bk < N ? (const T *)a.Bm + (b.sp.r0 + bt) * a.ld_B + b.g * N + bk
                          : (const T *)a.Cm + (b.sp.r0 + bt) * a.ld_C + b.g * N + bk - N;
    const long long ldbc = bk < N ? a.ld_B : a.ld_C;
    auto fetch_bc = [&](int t0) {
        const bool ok = t0 + bt < n;
        const T *p = pbc + t0 * ldbc;
        return ok && a.vecb_sweep ? load_raw<T, BC>(p) : load_part<T, BC>(p, ok ? BC : 0);
    };
    auto put_bc = [&](const Raw<T, BC> &r, int buf) {
        float v[BC];
        widen<T, BC>(r, v);
#pragma unroll
        for (int i = 0; i < BC; ++i) sBC[buf][bt][bk + i] = v[i];
    };
    const unsigned ou = (unsigned)(q * a.ld_u + c), od = (unsigned)(q * a.ld_dt + c), oz = (unsigned)(q * a.ld_z + c),
                   og = (unsigned)(q * a.ld_out + c);
    const T *pu = (const T *)a.u + b.sp.r0 * a.ld_u, *pd = (const T *)a.dt + b.sp.r0 * a.ld_dt;
    const T *pz = (const T *)a.z + b.sp.r0 * a.ld_z, *pg = (const T *)a.dout + b.sp.r0 * a.ld_out;
    const bool gate = a.z != nullptr;
    T nu[OWN], nd[OWN], nz[OWN], ng[OWN];
    auto fetch = [&](int left) {
        if (left >= BATCH) {
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                nu[l] = (pu + l * NQ * a.ld_u)[ou];
                nd[l] = (pd + l * NQ * a.ld_dt)[od];
                ng[l] = (pg + l * NQ * a.ld_out)[og];
                if (gate) nz[l] = (pz + l * NQ * a.ld_z)[oz];
            }
        } else {
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                nu[l] = nd[l] = nz[l] = ng[l] = from_f32<T>(0.f);
                if (l * NQ + q < left) {
                    nu[l] = (pu + l * NQ * a.ld_u)[ou];
                    nd[l] = (pd + l * NQ * a.ld_dt)[od];
                    ng[l] = (pg + l * NQ * a.ld_out)[og];
                    if (gate) nz[l] = (pz + l * NQ * a.ld_z)[oz];
                }
            }
        }
    };
    float dsum = 0.f;
    put_bc(fetch_bc(0), 0);
    fetch(n);
    for (int t0 = 0, buf = 0; t0 < n; t0 += kTile, buf ^= 1) {
        __syncthreads();
        Raw<T, BC> rbc;
        if (t0 + kTile < n) rbc = fetch_bc(t0 + kTile);
#pragma unroll 1
        for (int b0 = 0; b0 < kTile; b0 += BATCH) {
            const int left = n - t0 - b0;
            if (left <= 0) break;
            float x[OWN], d[OWN], dy[OWN];
#pragma unroll
            for (int l = 0; l < OWN; ++l) {
                d[l] = to_f32(nd[l]) + bias;
                if (a.softplus) d[l] = softplus_f32(d[l]);
                if (l * NQ + q >= left) d[l] = 0.f;   // behind the span; dy is zero there as loaded
                x[l] = d[l] * to_f32(nu[l]);
                dy[l] = to_f32(ng[l]);
                if (gate) dy[l] *= silu_f32(to_f32(nz[l]));
            }
            pu += BATCH * a.ld_u;
            pd += BATCH * a.ld_dt;
            pz += BATCH * a.ld_z;
            pg += BATCH * a.ld_out;
            fetch(left - BATCH);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                float dl = d[i / NQ], xl = x[i / NQ], gl = dy[i / NQ];
                if (NQ > 1) {
                    dl = __shfl_sync(0xffffffffu, dl, i % NQ, NQ);
                    xl = __shfl_sync(0xffffffffu, xl, i % NQ, NQ);
                    gl = __shfl_sync(0xffffffffu, gl, i % NQ, NQ);
                }
                const float *B = sBC[buf][b0 + i] + q * SPT, *C = B + N;
                const float2 d2 = make_float2(dl, dl), x2 = make_float2(xl, xl), g2 = make_float2(gl, gl);
                dsum += dl;
#pragma unroll
                for (int k = 0; k < P; k += 2) {
                    const float4 bv = *reinterpret_cast<const float4 *>(B + 2 * k);
                    const float4 cv = *reinterpret_cast<const float4 *>(C + 2 * k);
                    float2 e0 = __fmul2_rn(d2, A2[k]), e1 = __fmul2_rn(d2, A2[k + 1]);
                    e0 = make_float2(ex2(e0.x), ex2(e0.y));
                    e1 = make_float2(ex2(e1.x), ex2(e1.y));
                    h[k] = __ffma2_rn(e0, h[k], __fmul2_rn(x2, make_float2(bv.x, bv.y)));
                    h[k + 1] = __ffma2_rn(e1, h[k + 1], __fmul2_rn(x2, make_float2(bv.z, bv.w)));
                    W[k] = __fmul2_rn(W[k], e0);
                    W[k + 1] = __fmul2_rn(W[k + 1], e1);
                    G[k] = __ffma2_rn(W[k], __fmul2_rn(g2, make_float2(cv.x, cv.y)), G[k]);
                    G[k + 1] = __ffma2_rn(W[k + 1], __fmul2_rn(g2, make_float2(cv.z, cv.w)), G[k + 1]);
                }
            }
        }
        if (t0 + kTile < n) put_bc(rbc, buf ^ 1);
    }
    if (!live) return;
    const long long at = (b.slot * a.D + c) * N + q * SPT;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        *reinterpret_cast<float4 *>(a.hst + at + 2 * i) = make_float4(h[i].x, h[i].y, h[i + 1].x, h[i + 1].y);
        *reinterpret_cast<float4 *>(a.gst + at + 2 * i) = make_float4(G[i].x, G[i].y, G[i + 1].x, G[i + 1].y);
    }
    if (q == 0) a.sdel[b.slot * a.D + c] = dsum;
}

// ---------------------------------------------------------------- the main kernel
// A lane holds four states of two neighbouring channels, so a channel's states lie on NQ = N / 4
// lanes and a warp covers CL = 32 / NQ pairs.  dB and dC sum over channels: over the lane's two in
// its products, over the warp's pairs by exchanges that halve the values.  For those the lane's
// register i holds state i ^ (two bits of the lane's pair), so that what a lane sends is always its
// upper half and nothing is selected; B and C lie in shared memory in all four orders.
constexpr int kBwdThreads = 128;
constexpr int kStep = 8;        // tokens a tile: states kept at its start, loaded together
constexpr int kWin = 4;         // tokens a window

template <typename T, int N>
struct BwdShape {
    static constexpr int NQ = N / 4, CL = 32 / NQ;
    static constexpr int CH = 8 * CL;              // channels a block: four warps of CL pairs
    static constexpr int EPT = CH / 16;            // for the loads 16 threads share a token
    static constexpr int BE = N >= 16 ? N / 16 : 1;
    static constexpr int ROW = CH + 16;            // a row of sums: two rows' pairs fill the banks
    struct Smem {
        // first and second channels of the pairs apart: a warp's reads are one run of memory
        float4 x[kStep][2][CH / 2];                // delta, delta, delta u, delta u
        float2 g[kStep][2][CH / 2];                // dy, dy
        float4 h[kSpan / kStep][2][kBwdThreads];   // states at the tiles' starts
        float B[kStep][4][N], C[kStep][4][N];      // in the four orders
        float y[kStep][ROW], e[kStep][ROW], q[kStep][ROW];   // sums over states: C h, e B, e a h A
        float r[kStep][4][2 * N];                  // dB, dC of each warp
    };
};

// The values of four states in the order i ^ p, and back.
__device__ __forceinline__ float4 order(float4 v, int p) {
    if (p & 1) v = make_float4(v.y, v.x, v.w, v.z);
    if (p & 2) v = make_float4(v.z, v.w, v.x, v.y);
    return v;
}

// v[i] = dB, w[i] = dC of state i ^ p, summed over the warp's pairs.  A lane ends with KEEP states
// of both, or, where enough pairs are left, with one of one: first of dB, second of dC.
template <int NQ>
struct PairSum {
    static constexpr int KEEP = NQ == 16 ? 2 : 1;        // states a lane ends with
    static constexpr bool ONE = NQ <= 4;                 // only dB or only dC
    static __device__ __forceinline__ int perm(int lane) { return NQ == 16 ? (lane >> 4) * 2 : lane >> 3; }
    static __device__ __forceinline__ bool second(int lane) { return ONE && (lane & 4); }
    static __device__ __forceinline__ bool writes(int lane) { return NQ != 2 || !(lane & 2); }
    static __device__ __forceinline__ void sum(float (&v)[4], float (&w)[4], int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] += __shfl_xor_sync(0xffffffffu, v[i + 2], 16);
            w[i] += __shfl_xor_sync(0xffffffffu, w[i + 2], 16);
        }
        if (NQ <= 8) {
            v[0] += __shfl_xor_sync(0xffffffffu, v[1], 8);
            w[0] += __shfl_xor_sync(0xffffffffu, w[1], 8);
        }
        if (NQ <= 4) {
            const bool up = lane & 4;
            const float send = up ? v[0] : w[0], keep = up ? w[0] : v[0];
            v[0] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
        }
        if (NQ == 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    }
};

template <typename T, int N>
__global__ void __launch_bounds__(kBwdThreads, 3) ssm_bwd_kernel(const SsmP a) {
    using S = BwdShape<T, N>;
    using Sum = PairSum<S::NQ>;
    constexpr int NQ = S::NQ, CH = S::CH, EPT = S::EPT, BE = S::BE;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename S::Smem &s = *reinterpret_cast<typename S::Smem *>(smem_raw);
    const SsmBlock b = ssm_block(a, CH);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = b.sp.seq >= 0 ? b.sp.n : 0;
    const int q = lane % NQ, pr = warp * S::CL + lane / NQ, cl = 2 * pr;   // the pair, its first channel in the block
    const int p = Sum::perm(lane);
    // the loads: a thread's token of a tile and its channels
    const int lt = tid >> 4, lc = (tid & 15) * EPT;
    const int lleft = a.Dg - b.cin - lc;
    const int gc = b.g * a.Dg + b.cin + lc;
    float2 dA[2][2];
    float dD[EPT], dbias[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) dD[i] = dbias[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) dA[j][0] = dA[j][1] = make_float2(0.f, 0.f);
    const long long at = b.slot * a.D + (long long)b.g * a.Dg + b.cin + cl;   // the pair at this seam

    if (n > 0) {
        float2 A2[2][2], h[2][2], carry[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float4 va = make_float4(0.f, 0.f, 0.f, 0.f), vh = va, vg = va;
            if (b.cin + cl + j < a.Dg) {
                va = order(*reinterpret_cast<const float4 *>(a.A + ((long long)b.g * a.Dg + b.cin + cl + j) * N + 4 * q), p);
                vh = order(*reinterpret_cast<const float4 *>(a.hst + (at + j) * N + 4 * q), p);
                vg = order(*reinterpret_cast<const float4 *>(a.gst + (at + j) * N + 4 * q), p);
            }
            A2[j][0] = make_float2(rate(va.x), rate(va.y));
            A2[j][1] = make_float2(rate(va.z), rate(va.w));
            h[j][0] = make_float2(vh.x, vh.y);
            h[j][1] = make_float2(vh.z, vh.w);
            carry[j][0] = make_float2(vg.x, vg.y);
            carry[j][1] = make_float2(vg.z, vg.w);
        }
        float bias[EPT], skip[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            bias[i] = a.dt_bias && i < lleft ? a.dt_bias[gc + i] : 0.f;
            skip[i] = a.Dskip && i < lleft ? a.Dskip[gc + i] : 0.f;
        }
        // B and C of a tile: BE values a thread, in all orders
        const int bt = tid / (N / BE), bk = tid % (N / BE) * BE;
        Raw<T, BE> rb, rc;
        auto fetch_bc = [&](int t0, bool with_c) {
            const bool ok = bt < kStep && t0 + bt < n;
            const T *pb = (const T *)a.Bm + (b.sp.r0 + t0 + bt) * a.ld_B + b.g * N + bk;
            rb = ok && a.vecb ? load_raw<T, BE>(pb) : load_part<T, BE>(pb, ok ? BE : 0);
            if (with_c) {
                const T *pc = (const T *)a.Cm + (b.sp.r0 + t0 + bt) * a.ld_C + b.g * N + bk;
                rc = ok && a.vecb ? load_raw<T, BE>(pc) : load_part<T, BE>(pc, ok ? BE : 0);
            }
        };
        auto put_bc = [&](bool with_c) {
            if (bt < kStep) {
                float v[BE], w[BE];
                widen<T, BE>(rb, v);
                if (with_c) widen<T, BE>(rc, w);
#pragma unroll
                for (int i = 0; i < BE; ++i)
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        s.B[bt][o][(bk + i) ^ o] = v[i];
                        if (with_c) s.C[bt][o][(bk + i) ^ o] = w[i];
                    }
            }
        };
        Raw<T, EPT> ru, rd, rz, rg;
        auto fetch = [&](int t0, bool all) {
            const bool ok = t0 + lt < n;
            const long long row = b.sp.r0 + t0 + lt;
            ru = load_tile<T, EPT>(a.u, row, a.ld_u, gc, lleft, ok, a.vec);
            rd = load_tile<T, EPT>(a.dt, row, a.ld_dt, gc, lleft, ok, a.vec);
            if (all) {
                rg = load_tile<T, EPT>(a.dout, row, a.ld_out, gc, lleft, ok, a.vec);
                if (a.z) rz = load_tile<T, EPT>(a.z, row, a.ld_z, gc, lleft, ok, a.vec);
            }
        };
        // one token of the recurrence for the lane's pair: decay factors e, states h
        auto advance = [&](int t, float2 (&e)[2][2], float2 (&st)[2][2]) {
            const float4 bv = *reinterpret_cast<const float4 *>(&s.B[t][p][4 * q]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 x = s.x[t][j][pr];
                const float2 d2 = make_float2(x.x, x.y), x2 = make_float2(x.z, x.w);
                const float2 m0 = __fmul2_rn(d2, A2[j][0]), m1 = __fmul2_rn(d2, A2[j][1]);
                e[j][0] = make_float2(ex2(m0.x), ex2(m0.y));
                e[j][1] = make_float2(ex2(m1.x), ex2(m1.y));
                st[j][0] = __ffma2_rn(e[j][0], st[j][0], __fmul2_rn(x2, make_float2(bv.x, bv.y)));
                st[j][1] = __ffma2_rn(e[j][1], st[j][1], __fmul2_rn(x2, make_float2(bv.z, bv.w)));
            }
        };
        // forward: the states at the tiles' starts
        const int tiles = (n + kStep - 1) / kStep;
        fetch(0, false);
        fetch_bc(0, false);
        for (int i = 0; i + 1 < tiles; ++i) {   // the last tile's end is not needed
            float u[EPT], d[EPT];
            widen<T, EPT>(ru, u);
            widen<T, EPT>(rd, d);
#pragma unroll
            for (int k = 0; k < EPT; ++k) {     // all tiles but the last are full
                d[k] += bias[k];
                if (a.softplus) d[k] = softplus_f32(d[k]);
                if (k >= lleft) d[k] = 0.f;
                s.x[lt][(lc + k) & 1][(lc + k) >> 1] = make_float4(d[k], d[k], d[k] * u[k], d[k] * u[k]);
            }
            put_bc(false);
            fetch((i + 1) * kStep, false);
            fetch_bc((i + 1) * kStep, false);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j) s.h[i][j][tid] = make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
#pragma unroll
            for (int t = 0; t < kStep; ++t) {
                float2 e[2][2];
                advance(t, e, h);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) s.h[tiles - 1][j][tid] = make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y);
        // backward over the tiles
        fetch((tiles - 1) * kStep, true);
        fetch_bc((tiles - 1) * kStep, true);
        for (int i = tiles - 1; i >= 0; --i) {
            const int t0 = i * kStep;
            const bool ok = t0 + lt < n;
            const Raw<T, EPT> cu = ru, cd = rd, cz = rz, cg = rg;
            {
                float u[EPT], d[EPT], z[EPT], g[EPT];
                widen<T, EPT>(cu, u);
                widen<T, EPT>(cd, d);
                widen<T, EPT>(cg, g);
                if (a.z) widen<T, EPT>(cz, z);
#pragma unroll
                for (int k = 0; k < EPT; ++k) {
                    d[k] += bias[k];
                    if (a.softplus) d[k] = softplus_f32(d[k]);
                    if (!ok || k >= lleft) d[k] = 0.f;   // a token behind the span: no decay, no input, no gradient
                    if (a.z) g[k] *= silu_f32(z[k]);
                    s.x[lt][(lc + k) & 1][(lc + k) >> 1] = make_float4(d[k], d[k], d[k] * u[k], d[k] * u[k]);
                    s.g[lt][(lc + k) & 1][(lc + k) >> 1] = make_float2(g[k], g[k]);
                }
            }
            put_bc(true);
            if (i > 0) {
                fetch(t0 - kStep, true);
                fetch_bc(t0 - kStep, true);
            }
            __syncthreads();
#pragma unroll 1   // unrolled, the windows' registers would be held at once
            for (int w = kStep / kWin - 1; w >= 0; --w) {
                float2 E[kWin][2][2], H[kWin][2][2], hs[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 v = s.h[i][j][tid];
                    hs[j][0] = make_float2(v.x, v.y);
                    hs[j][1] = make_float2(v.z, v.w);
                }
                if (w > 0)
#pragma unroll
                    for (int t = 0; t < kWin; ++t) {
                        float2 e[2][2];
                        advance(t, e, hs);
                    }
                float y[2][kWin], sb[2][kWin], sq[2][kWin];
#pragma unroll
                for (int m = 0; m < kWin; ++m) {
                    const int t = w * kWin + m;
                    const float4 cv = *reinterpret_cast<const float4 *>(&s.C[t][p][4 * q]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        H[m][j][0] = m ? H[m ? m - 1 : 0][j][0] : hs[j][0];
                        H[m][j][1] = m ? H[m ? m - 1 : 0][j][1] : hs[j][1];
                    }
                    advance(t, E[m], H[m]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 v = __ffma2_rn(make_float2(cv.z, cv.w), H[m][j][1],
                                                    __fmul2_rn(make_float2(cv.x, cv.y), H[m][j][0]));
                        y[j][m] = v.x + v.y;
                    }
                }
#pragma unroll
                for (int m = kWin - 1; m >= 0; --m) {
                    const int t = w * kWin + m;
                    const float4 bv = *reinterpret_cast<const float4 *>(&s.B[t][p][4 * q]);
                    const float4 cv = *reinterpret_cast<const float4 *>(&s.C[t][p][4 * q]);
                    const float2 bb[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
                    const float2 cc[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)};
                    float2 vB[2], vC[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 x = s.x[t][j][pr];
                        const float2 d2 = make_float2(x.x, x.y), x2 = make_float2(x.z, x.w), g2 = s.g[t][j][pr];
                        float2 pb, pq;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 e = __ffma2_rn(cc[k], g2, carry[j][k]);
                            carry[j][k] = __fmul2_rn(E[m][j][k], e);
                            const float2 kept = __fmul2_rn(carry[j][k], m ? H[m ? m - 1 : 0][j][k] : hs[j][k]);   // e a h_{t-1}
                            dA[j][k] = __ffma2_rn(kept, d2, dA[j][k]);
                            pb = k ? __ffma2_rn(e, bb[k], pb) : __fmul2_rn(e, bb[k]);
                            pq = k ? __ffma2_rn(kept, A2[j][k], pq) : __fmul2_rn(kept, A2[j][k]);
                            vB[k] = j ? __ffma2_rn(e, x2, vB[k]) : __fmul2_rn(e, x2);
                            vC[k] = j ? __ffma2_rn(g2, H[m][j][k], vC[k]) : __fmul2_rn(g2, H[m][j][k]);
                        }
                        sb[j][m] = pb.x + pb.y;
                        sq[j][m] = pq.x + pq.y;
                    }
                    float v[4] = {vB[0].x, vB[0].y, vB[1].x, vB[1].y}, u[4] = {vC[0].x, vC[0].y, vC[1].x, vC[1].y};
                    Sum::sum(v, u, lane);
                    if (Sum::writes(lane)) {
                        float *r = s.r[t][warp];
#pragma unroll
                        for (int k = 0; k < Sum::KEEP; ++k) {
                            const int state = 4 * q + (k ^ p);
                            r[Sum::second(lane) ? N + state : state] = v[k];
                            if (!Sum::ONE) r[N + state] = u[k];
                        }
                    }
                }
                // sums over states
                if constexpr (NQ <= kWin) {
#pragma unroll
                    for (int o = 0; o < kWin; o += NQ) {
                        float2 ry, re, rq;
                        float v[NQ];
                        auto both = [&](float (&f)[2][kWin]) {
#pragma unroll
                            for (int m = 0; m < NQ; ++m) v[m] = f[0][o + m];
                            const float r0 = reduce_states<NQ>(v, q);
#pragma unroll
                            for (int m = 0; m < NQ; ++m) v[m] = f[1][o + m];
                            return make_float2(r0, reduce_states<NQ>(v, q));
                        };
                        ry = both(y);
                        re = both(sb);
                        rq = both(sq);
                        const int t = w * kWin + o + q;
                        *reinterpret_cast<float2 *>(&s.y[t][cl]) = ry;
                        *reinterpret_cast<float2 *>(&s.e[t][cl]) = re;
                        *reinterpret_cast<float2 *>(&s.q[t][cl]) = rq;
                    }
                } else {   // lane q & 7: token q & 3 of channel (q >> 2) & 1
                    const int t = w * kWin + (q & 3), c = cl + ((q >> 2) & 1);
                    auto eight = [&](float (&f)[2][kWin], bool halved) {
                        float v[8];
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            v[m] = f[m >> 2][m & 3];
                            if (halved) v[m] += __shfl_xor_sync(0xffffffffu, v[m], 8);
                        }
                        return reduce_states<8>(v, q & 7);
                    };
                    const float rq = eight(sq, NQ == 16);
                    if constexpr (NQ == 8) {
                        const float ry = eight(y, false), re = eight(sb, false);
                        s.y[t][c] = ry;
                        s.e[t][c] = re;
                        s.q[t][c] = rq;
                    } else {   // 16 lanes: y for the lower eight, the sum of e B for the upper
                        float v[16];
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            v[m] = y[m >> 2][m & 3];
                            v[8 + m] = sb[m >> 2][m & 3];
                        }
                        const float r = reduce_states<16>(v, q);
                        (q < 8 ? s.y : s.e)[t][c] = r;
                        if (q < 8) s.q[t][c] = rq;
                    }
                }
            }
            __syncthreads();
            // the block's part of dB, dC: the warps' sums in order
#pragma unroll
            for (int k = tid; k < kStep * 2 * N; k += kBwdThreads) {
                const int t = k / (2 * N), m = k % (2 * N);
                if (t0 + t < n)
                    a.part_BC[((long long)b.blk * a.q.rows() + b.sp.r0 + t0 + t) * (2 * N) + m] =
                        (s.r[t][0][m] + s.r[t][1][m]) + (s.r[t][2][m] + s.r[t][3][m]);
            }
            if (ok) {
                float u[EPT], raw[EPT], z[EPT], go[EPT], du[EPT], dd[EPT], dz[EPT];
                widen<T, EPT>(cu, u);
                widen<T, EPT>(cd, raw);
                widen<T, EPT>(cg, go);
                if (a.z) widen<T, EPT>(cz, z);
#pragma unroll
                for (int k = 0; k < EPT; ++k) {
                    raw[k] += bias[k];
                    const int j = (lc + k) & 1, r = (lc + k) >> 1;
                    const float delta = s.x[lt][j][r].x, dy = s.g[lt][j][r].x, se = s.e[lt][lc + k];
                    du[k] = fmaf(delta, se, skip[k] * dy);
                    dd[k] = fmaf(s.q[lt][lc + k], kLn2, u[k] * se);
                    if (a.softplus) dd[k] *= sigmoid_f32(raw[k]);
                    if (a.z) {
                        const float sg = sigmoid_f32(z[k]);
                        dz[k] = go[k] * fmaf(skip[k], u[k], s.y[lt][lc + k]) * sg * fmaf(z[k], 1.f - sg, 1.f);
                    }
                    if (k < lleft) {
                        dD[k] = fmaf(dy, u[k], dD[k]);
                        dbias[k] += dd[k];
                    }
                }
                const long long o = (b.sp.r0 + t0 + lt) * a.D + gc;
                if (a.vec_grad && lleft >= EPT) {
                    store_f32<T, EPT>((T *)a.du + o, du);
                    store_f32<T, EPT>((T *)a.ddt + o, dd);
                    if (a.z) store_f32<T, EPT>((T *)a.dz + o, dz);
                } else {
                    store_part<T, EPT>((T *)a.du + o, du, lleft);
                    store_part<T, EPT>((T *)a.ddt + o, dd, lleft);
                    if (a.z) store_part<T, EPT>((T *)a.dz + o, dz, lleft);
                }
            }
            __syncthreads();   // before the next tile is put in place
        }
    }
    // the span's part of dA, dDskip, ddt_bias; a slot without rows adds zeros
    float *part = a.part + b.slot * a.part_ld;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (b.cin + cl + j < a.Dg)
            *reinterpret_cast<float4 *>(part + ((long long)b.g * a.Dg + b.cin + cl + j) * N + 4 * q) =
                order(make_float4(dA[j][0].x, dA[j][0].y, dA[j][1].x, dA[j][1].y), p);
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        s.y[lt][lc + i] = dD[i];
        s.e[lt][lc + i] = dbias[i];
    }
    __syncthreads();
    if (tid < CH && b.cin + tid < a.Dg) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int t = 0; t < kStep; ++t) {
            x += s.y[t][tid];
            y += s.e[t][tid];
        }
        const long long c = (long long)b.g * a.Dg + b.cin + tid;
        part[(long long)a.D * N + c] = x;
        part[(long long)a.D * (N + 1) + c] = y;
    }
}

// The last sums, in a fixed order: dB and dC over a group's channel blocks, 128 values a block of
// threads; dA, dDskip and ddt_bias over the spans, 32 columns.  Eight warps share the terms.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_sum_kernel(const SsmP a, T *dB, T *dC, float *dA, float *dDskip,
                                                          float *ddt_bias, int N, unsigned bc_blocks) {
    __shared__ float4 sums[8][32];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    if (blockIdx.x < bc_blocks) {
        const long long rows = a.q.rows(), all = rows * 2 * N;   // values of a channel block
        const long long i = ((long long)blockIdx.x * 32 + lane) * 4;
        const int g = (int)(i / all);
        const long long in = i % all, row = in / (2 * N);        // a quad lies in one row, in B or in C
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g < a.G) {
            const float *p = a.part_BC + (long long)g * a.cpg * all + in;
#pragma unroll 4
            for (int m = y; m < a.cpg; m += 8) {
                const float4 w = *reinterpret_cast<const float4 *>(p + m * all);
                v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
            }
        }
        sums[y][lane] = v;
        __syncthreads();
        if (y > 0 || g >= a.G) return;
        if (a.q.cu && (row < a.q.lo(0) || row >= a.q.lo(a.q.S))) return;   // of no sequence: not written
#pragma unroll
        for (int m = 1; m < 8; ++m) {
            const float4 w = sums[m][lane];
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        const int k = (int)(in % (2 * N));
        const float f[4] = {v.x, v.y, v.z, v.w};
        store_f32<T, 4>((k < N ? dB + k : dC + k - N) + (row * a.G + g) * N, f);
        return;
    }
    const long long n = (long long)a.D * (N + 2), all = (long long)a.D * N;
    const long long i = (long long)(blockIdx.x - bc_blocks) * 32 + lane;
    float v = 0.f;
    if (i < n)
#pragma unroll 8
        for (long long k = y; k < a.slots; k += 8) v += a.part[k * a.part_ld + i];
    sums[y][lane].x = v;
    __syncthreads();
    if (y == 0 && i < n) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += sums[k][lane].x;
        if (i < all) dA[i] = v;
        else if (i < all + a.D) {
            if (dDskip) dDskip[i - all] = v;
        } else if (ddt_bias) {
            ddt_bias[i - all - a.D] = v;
        }
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

long long part_ld(const SsmArgs &a) { return ((long long)a.D * (a.N + 2) + 3) / 4 * 4; }

// Rows a span takes: the main kernel's time goes by the waves of 444 blocks (three an SM) and by a
// span's rows in each, with 24 rows' worth for a block's start and end; the chain through a
// sequence's spans takes a quarter of a row's time for each.  Few blocks take short spans, many
// stay at 64: 4 x 256 x 512 x 8 takes 43 us with 16 rows a span and 94 with 64, 512 x 1024 x 16 46 with 32 rows
// and 62 with 64, 2 x 900 x 900 x 8 106 with 40 and 131 with 64.  Larger calls keep 64: 8192 x 1024 x 32 takes 567 us
// with 64 and 577 with 56.
int span_rows(const SsmArgs &a) {
    const int CH = 1024 / a.N, Dg = a.D / a.G;
    const long long nblk = (long long)a.G * ((Dg + CH - 1) / CH);
    int best = kSpan;
    double least = 0.0;
    for (int L = kSpan; L >= kShortestSpan; L -= kStep) {
        const long long waves = (span_slots(a.cu != nullptr, a.S, a.T, L) * nblk + 443) / 444;
        const double cost = (double)waves * (L + 24) + 0.25 * (double)(a.T / L);
        if (L == kSpan || cost < least) {
            least = cost;
            best = L;
        }
    }
    return best;
}

// Parts of the workspace: hst, gst, sdel, part, part_BC; off[5] is the whole.
void bwd_parts(const SsmArgs &a, size_t (&off)[6]) {
    const int CH = 1024 / a.N, Dg = a.D / a.G;
    const size_t nblk = (size_t)a.G * ((Dg + CH - 1) / CH);
    const size_t slots = (size_t)span_slots(a.cu != nullptr, a.S, a.T, span_rows(a));
    const size_t sd = slots * a.D * sizeof(float);
    off[0] = 0;
    off[1] = off[0] + up256(sd * a.N);
    off[2] = off[1] + up256(sd * a.N);
    off[3] = off[2] + up256(sd);
    off[4] = off[3] + up256(slots * part_ld(a) * sizeof(float));
    off[5] = off[4] + up256(nblk * (size_t)a.rows * 2 * a.N * sizeof(float));
}

template <typename T, int N>
cudaError_t run(const SsmArgs &a, cudaStream_t st) {
    using S = BwdShape<T, N>;
    using F = FwdShape<N>;
    static_assert(S::CH == 1024 / N, "bwd_parts");
    const int L = span_rows(a);
    SsmP p = ssm_params<S::CH, S::EPT, S::BE>(a, L);
    p.vec_grad = p.Dg % S::EPT == 0;   // contiguous rows at 16 bytes
    p.vecb_sweep = ssm_params<S::CH, S::EPT, F::BC>(a, L).vecb;
    size_t off[6];
    bwd_parts(a, off);
    char *ws = (char *)a.workspace;
    p.hst = (float *)(ws + off[0]);
    p.gst = (float *)(ws + off[1]);
    p.sdel = (float *)(ws + off[2]);
    p.part = (float *)(ws + off[3]);
    p.part_BC = (float *)(ws + off[4]);
    p.part_ld = part_ld(a);
    const long long blocks = p.slots * p.nblk;
    const long long sweep_blocks = p.slots * a.G * ((p.Dg + F::CH - 1) / F::CH);
    const long long bc_blocks = (a.rows * a.G * 2 * N + 127) / 128, sum_blocks = ((long long)a.D * (N + 2) + 31) / 32;
    if (blocks > 0x7fffffffLL || sweep_blocks > 0x7fffffffLL || bc_blocks + sum_blocks > 0x7fffffffLL)
        return cudaErrorInvalidValue;
    constexpr int smem = sizeof(typename S::Smem);
    cudaError_t e = cudaFuncSetAttribute(ssm_bwd_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    a.marks->mark(st);
    ssm_bwd_sweep_kernel<T, N><<<(unsigned)sweep_blocks, kFwdThreads, 0, st>>>(p);
    a.marks->mark(st);
    if ((e = launch_ssm_seams(p, N, st)) != cudaSuccess) return e;
    a.marks->mark(st);
    ssm_bwd_kernel<T, N><<<(unsigned)blocks, kBwdThreads, smem, st>>>(p);
    a.marks->mark(st);
    ssm_bwd_sum_kernel<T><<<(unsigned)(bc_blocks + sum_blocks), 256, 0, st>>>(
        p, (T *)a.dB, (T *)a.dC, a.dA, a.dDskip, a.ddt_bias, N, (unsigned)bc_blocks);
    return cudaGetLastError();
}
template <typename T>
cudaError_t dispatch(const SsmArgs &a, cudaStream_t st) {
    switch (a.N) {
        case 8: return run<T, 8>(a, st);
        case 16: return run<T, 16>(a, st);
        case 32: return run<T, 32>(a, st);
        default: return run<T, 64>(a, st);
    }
}

}  // namespace

size_t ssm_scan_bwd_workspace_bytes(const SsmArgs &a) {
    size_t off[6];
    bwd_parts(a, off);
    return off[5];
}
cudaError_t launch_ssm_scan_bwd(const SsmArgs &a, cudaStream_t st) {
    return a.bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace kda
