// kda_ssm_bwd.cu -- backward of the selective state space scan.
//
// With a_t = exp(delta_t A), dy = dout silu(z), e_t the gradient of h_t:
//   e_t = C_t dy_t + a_{t+1} e_{t+1}   (behind the last token: dh_T)
//   dC_t = sum_d dy_t h_t,   dB_t = sum_d e_t delta_t u_t,   dA = sum_t e_t delta_t a_t h_{t-1}
//   ddelta_t = sum_n e_t a_t h_{t-1} A + u_t sum_n e_t B_t,   du_t = Dskip dy_t + delta_t sum_n e_t B_t
//   dz_t = dout_t y_t silu'(z_t),   ddt = ddelta sigmoid(dt + dt_bias),   dh0 = a_1 e_1
//
// Time is cut into spans of 64 tokens that run side by side.  One sweep finds for every span its
// end state from zero and, with the running product P of the a, the gradient at its start that
// its own outputs make, sum_t P_t C_t dy_t: both go forward, on the same exponentials.  A small
// pass chains the spans.  The main kernel then walks its span forward once, keeping the state
// every 8 tokens in shared memory, and goes back over windows of 8 tokens whose states and decay
// factors stay in registers: three exponentials a state and token, no state in HBM but at the
// spans' seams.  dB and dC sum over channels: over a warp's lanes by exchanges that halve the
// values (one a value, not five), over the block in shared memory, over blocks in a last pass.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kSpan = 64;      // tokens a span
constexpr int kWin = 8;        // tokens a window

// Both sweeps of a span: end state from zero (hst), gradient at the start (gst), sum of delta.
template <typename T, int N>
__global__ void __launch_bounds__(kSsmThreads) ssm_bwd_sweep_kernel(const SsmP a) {
    using S = SsmShape<N>;
    constexpr int NQ = S::NQ, CH = S::CH, EPT = S::EPT;
    __shared__ __align__(16) float4 sX[kTile * CH];   // delta, delta u, dy
    __shared__ __align__(16) float sB[kTile * N], sC[kTile * N];
    const SsmBlock b = ssm_block(a, CH);
    if (b.sp.seq < 0 || (b.sp.count == 1 && !a.dh0)) return;
    const int tid = threadIdx.x;
    const int ch = tid / NQ, q = tid % NQ;
    const bool live = b.cin + ch < a.Dg;
    const long long c = (long long)b.g * a.Dg + b.cin + ch;
    float A2[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) load_f32<float, 4>(a.A + c * N + 4 * q, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
    const int lt = tid >> 4, lc = (tid & 15) * EPT;
    const int lleft = a.Dg - b.cin - lc;
    const int gc = b.g * a.Dg + b.cin + lc;
    float bias[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) bias[i] = a.dt_bias && i < lleft ? a.dt_bias[gc + i] : 0.f;
    Raw<T, EPT> nu, ndt, nz, ng;
    BcTile<T, N> bc;
    auto fetch = [&](int t0) {
        const int n = b.sp.n - t0;
        const long long row = b.sp.r0 + t0 + lt;
        const bool ok = lt < n;
        nu = load_tile<T, EPT>(a.u, row, a.ld_u, gc, lleft, ok, a.vec);
        ndt = load_tile<T, EPT>(a.dt, row, a.ld_dt, gc, lleft, ok, a.vec);
        ng = load_tile<T, EPT>(a.dout, row, a.ld_out, gc, lleft, ok, a.vec);
        if (a.z) nz = load_tile<T, EPT>(a.z, row, a.ld_z, gc, lleft, ok, a.vec);
        bc.fetch(a, b.sp.r0 + t0, n, b.g, true);
    };
    float h[4] = {0.f, 0.f, 0.f, 0.f}, g[4] = {0.f, 0.f, 0.f, 0.f}, P[4] = {1.f, 1.f, 1.f, 1.f}, dsum = 0.f;
    fetch(0);
    for (int t0 = 0; t0 < b.sp.n; t0 += kTile) {
        const bool ok = t0 + lt < b.sp.n;
        float u[EPT], d[EPT], z[EPT], dy[EPT];
        widen<T, EPT>(nu, u);
        widen<T, EPT>(ndt, d);
        widen<T, EPT>(ng, dy);
        if (a.z) widen<T, EPT>(nz, z);
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            d[i] += bias[i];
            if (a.softplus) d[i] = softplus_f32(d[i]);
            if (!ok || i >= lleft) d[i] = 0.f;
            if (a.z) dy[i] *= silu_f32(z[i]);
            sX[lt * CH + lc + i] = make_float4(d[i], d[i] * u[i], dy[i], 0.f);
        }
        bc.put(sB, sC);
        if (t0 + kTile < b.sp.n) fetch(t0 + kTile);
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < kTile; ++t) {
            const float4 x = sX[t * CH + ch];
            const float4 bv = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
            const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
            const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
            dsum += x.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = ex2(x.x * A2[i]);
                h[i] = fmaf(e, h[i], x.y * bb[i]);
                P[i] *= e;
                g[i] = fmaf(P[i], cc[i] * x.z, g[i]);
            }
        }
        __syncthreads();
    }
    if (!live) return;
    const long long at = b.slot * a.D + c;
    store_f32<float, 4>(a.hst + at * N + 4 * q, h);
    store_f32<float, 4>(a.gst + at * N + 4 * q, g);
    if (q == 0) a.sdel[at] = dsum;
}

// v[0..3] (dB) and v[4..7] (dC) of a lane's four states, summed over the warp's channels; every
// lane ends with KEEP of the eight sums, its own first one numbered `first`.
template <int NQ>
struct ChannelSum {
    static constexpr int KEEP = NQ >= 4 ? 8 * NQ / 32 : 1;
    static __device__ __forceinline__ int first(int lane) {
        return NQ == 2 ? lane >> 2 : lane / NQ * KEEP;
    }
    static __device__ __forceinline__ bool writes(int lane) { return NQ != 2 || !(lane & 2); }
    static __device__ __forceinline__ void sum(float (&v)[8], int lane) {
        int n = 8;
#pragma unroll
        for (int o = 16; o >= NQ; o >>= 1) {
            if (n > 1) {
                n /= 2;
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n) {
                        const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
            }
        }
    }
};

template <int N>
constexpr size_t bwd_smem() {
    using S = SsmShape<N>;
    return sizeof(float) * (kTile * S::CH * 4 + 2 * kTile * N + 3 * kTile * S::ROW + kTile * 8 * 2 * N +
                            (kSpan / kWin) * kSsmThreads * 4);
}

template <typename T, int N>
__global__ void __launch_bounds__(kSsmThreads, 2) ssm_bwd_kernel(const SsmP a) {
    using S = SsmShape<N>;
    using Sum = ChannelSum<S::NQ>;
    constexpr int NQ = S::NQ, CH = S::CH, EPT = S::EPT, ROW = S::ROW;
    extern __shared__ __align__(16) float4 smem[];
    float4 *sX = smem;                                    // [kTile][CH]: delta, delta u, dy
    float4 *sH = sX + kTile * CH;                         // [kSpan / kWin][threads]: states
    float *sB = (float *)(sH + (kSpan / kWin) * kSsmThreads), *sC = sB + kTile * N;
    float *sR = sC + kTile * N;                           // [kTile][8 warps][2 N]: dB, dC
    float *sY = sR + kTile * 8 * 2 * N;                   // [kTile][ROW] each: y, sum e B,
    float *sE = sY + kTile * ROW, *sQ = sE + kTile * ROW; //   sum e a h A
    const SsmBlock b = ssm_block(a, CH);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ch = tid / NQ, q = tid % NQ;
    const bool live = b.cin + ch < a.Dg;
    const long long c = (long long)b.g * a.Dg + b.cin + ch, at = b.slot * a.D + c;
    const int lt = tid >> 4, lc = (tid & 15) * EPT;
    const int lleft = a.Dg - b.cin - lc;
    const int gc = b.g * a.Dg + b.cin + lc;
    float dA[4] = {0.f, 0.f, 0.f, 0.f}, dD[EPT], dbias[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) dD[i] = dbias[i] = 0.f;

    if (b.sp.seq >= 0 && b.sp.n > 0) {
        float A2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f}, carry[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
            load_f32<float, 4>(a.A + c * N + 4 * q, A2);
            load_f32<float, 4>(a.hst + at * N + 4 * q, h);
            load_f32<float, 4>(a.gst + at * N + 4 * q, carry);
#pragma unroll
            for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
        }
        float bias[EPT], skip[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            bias[i] = a.dt_bias && i < lleft ? a.dt_bias[gc + i] : 0.f;
            skip[i] = a.Dskip && i < lleft ? a.Dskip[gc + i] : 0.f;
        }
        // forward: the states at the windows' starts
        for (int t0 = 0; t0 < b.sp.n; t0 += kTile) {
            const bool ok = t0 + lt < b.sp.n;
            const long long row = b.sp.r0 + t0 + lt;
            BcTile<T, N> bc;
            bc.fetch(a, b.sp.r0 + t0, b.sp.n - t0, b.g, false);
            float u[EPT], d[EPT];
            widen<T, EPT>(load_tile<T, EPT>(a.u, row, a.ld_u, gc, lleft, ok, a.vec), u);
            widen<T, EPT>(load_tile<T, EPT>(a.dt, row, a.ld_dt, gc, lleft, ok, a.vec), d);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                d[i] += bias[i];
                if (a.softplus) d[i] = softplus_f32(d[i]);
                if (!ok || i >= lleft) d[i] = 0.f;
                sX[lt * CH + lc + i] = make_float4(d[i], d[i] * u[i], 0.f, 0.f);
            }
            bc.put(sB, nullptr);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kTile / kWin; ++w) {
                sH[(t0 / kWin + w) * kSsmThreads + tid] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
                for (int j = 0; j < kWin; ++j) {
                    const float4 x = sX[(w * kWin + j) * CH + ch];
                    const float4 bv = *reinterpret_cast<const float4 *>(sB + (w * kWin + j) * N + 4 * q);
                    const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = fmaf(ex2(x.x * A2[i]), h[i], x.y * bb[i]);
                }
            }
        }
        // backward over the tiles
        for (int t0 = (b.sp.n - 1) / kTile * kTile; t0 >= 0; t0 -= kTile) {
            const bool ok = t0 + lt < b.sp.n;
            const long long row = b.sp.r0 + t0 + lt;
            BcTile<T, N> bc;
            bc.fetch(a, b.sp.r0 + t0, b.sp.n - t0, b.g, true);
            float u[EPT], raw[EPT], d[EPT], z[EPT], go[EPT], dy[EPT];
            widen<T, EPT>(load_tile<T, EPT>(a.u, row, a.ld_u, gc, lleft, ok, a.vec), u);
            widen<T, EPT>(load_tile<T, EPT>(a.dt, row, a.ld_dt, gc, lleft, ok, a.vec), raw);
            widen<T, EPT>(load_tile<T, EPT>(a.dout, row, a.ld_out, gc, lleft, ok, a.vec), go);
            if (a.z) widen<T, EPT>(load_tile<T, EPT>(a.z, row, a.ld_z, gc, lleft, ok, a.vec), z);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                raw[i] += bias[i];
                d[i] = a.softplus ? softplus_f32(raw[i]) : raw[i];
                if (!ok || i >= lleft) d[i] = 0.f;
                dy[i] = a.z ? go[i] * silu_f32(z[i]) : go[i];
                sX[lt * CH + lc + i] = make_float4(d[i], d[i] * u[i], dy[i], 0.f);
            }
            bc.put(sB, sC);
            __syncthreads();
            for (int w = kTile / kWin - 1; w >= 0; --w) {
                float H[kWin][4], E[kWin][4], y[kWin];
                const float4 h0 = sH[(t0 / kWin + w) * kSsmThreads + tid];
                const float hs[4] = {h0.x, h0.y, h0.z, h0.w};
#pragma unroll
                for (int j = 0; j < kWin; ++j) {
                    const int t = w * kWin + j;
                    const float4 x = sX[t * CH + ch];
                    const float4 bv = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
                    const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
                    const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        E[j][i] = ex2(x.x * A2[i]);
                        H[j][i] = fmaf(E[j][i], j ? H[j - 1][i] : hs[i], x.y * bb[i]);
                    }
                    y[j] = fmaf(cv.x, H[j][0], cv.y * H[j][1]) + fmaf(cv.z, H[j][2], cv.w * H[j][3]);
                }
                float sb[kWin], sq[kWin];
#pragma unroll
                for (int j = kWin - 1; j >= 0; --j) {
                    const int t = w * kWin + j;
                    const float4 x = sX[t * CH + ch];
                    const float4 bv = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
                    const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
                    const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
                    float v[8];
                    sb[j] = sq[j] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = fmaf(cc[i], x.z, carry[i]);
                        carry[i] = E[j][i] * e;
                        const float k = carry[i] * (j ? H[j - 1][i] : hs[i]);   // e a h_{t-1}
                        sb[j] = fmaf(e, bb[i], sb[j]);
                        sq[j] = fmaf(k, A2[i], sq[j]);
                        dA[i] = fmaf(k, x.x, dA[i]);
                        v[i] = e * x.y;
                        v[4 + i] = x.z * H[j][i];
                    }
                    Sum::sum(v, lane);
                    if (Sum::writes(lane)) {
#pragma unroll
                        for (int k = 0; k < Sum::KEEP; ++k) {
                            const int id = Sum::first(lane) + k;
                            sR[(t * 8 + warp) * 2 * N + (id >> 2) * N + 4 * q + (id & 3)] = v[k];
                        }
                    }
                }
                if constexpr (NQ <= kWin) {
#pragma unroll
                    for (int o = 0; o < kWin; o += NQ) {
                        float r0[NQ], r1[NQ], r2[NQ];
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            r0[j] = y[o + j];
                            r1[j] = sb[o + j];
                            r2[j] = sq[o + j];
                        }
                        const int p = (w * kWin + o + q) * ROW + ch;
                        sY[p] = reduce_states<NQ>(r0, q);
                        sE[p] = reduce_states<NQ>(r1, q);
                        sQ[p] = reduce_states<NQ>(r2, q);
                    }
                } else {   // 16 lanes, 8 tokens: y and the sum of e B share one exchange
                    float r0[NQ], r2[kWin];
#pragma unroll
                    for (int j = 0; j < kWin; ++j) {
                        r0[j] = y[j];
                        r0[kWin + j] = sb[j];
                        r2[j] = sq[j] + __shfl_xor_sync(0xffffffffu, sq[j], 8);
                    }
                    const float v = reduce_states<NQ>(r0, q);
                    const int p = (w * kWin + (q & 7)) * ROW + ch;
                    (q < 8 ? sY : sE)[p] = v;
                    const float k = reduce_states<kWin>(r2, q & 7);
                    if (q < 8) sQ[p] = k;
                }
            }
            __syncthreads();
            // the block's part of dB, dC: the warps' sums in order
            for (int i = tid; i < kTile * 2 * N; i += kSsmThreads) {
                const int t = i / (2 * N), k = i % (2 * N);
                if (t0 + t < b.sp.n) {
                    float v = 0.f;
#pragma unroll
                    for (int m = 0; m < 8; ++m) v += sR[(t * 8 + m) * 2 * N + k];
                    a.part_BC[((long long)b.blk * a.q.rows() + b.sp.r0 + t0 + t) * (2 * N) + k] = v;
                }
            }
            if (ok) {
                float du[EPT], dd[EPT], dz[EPT];
#pragma unroll
                for (int i = 0; i < EPT; ++i) {
                    const int p = lt * ROW + lc + i;
                    const float se = sE[p];
                    du[i] = fmaf(d[i], se, skip[i] * dy[i]);
                    dd[i] = fmaf(sQ[p], kLn2, u[i] * se);
                    if (a.softplus) dd[i] *= sigmoid_f32(raw[i]);
                    if (a.z) {
                        const float sg = sigmoid_f32(z[i]);
                        dz[i] = go[i] * fmaf(skip[i], u[i], sY[p]) * sg * fmaf(z[i], 1.f - sg, 1.f);
                    }
                    if (i < lleft) {
                        dD[i] = fmaf(dy[i], u[i], dD[i]);
                        dbias[i] += dd[i];
                    }
                }
                const long long o = row * a.D + gc;
                if (a.vec && lleft >= EPT) {
                    store_f32<T, EPT>((T *)a.du + o, du);
                    store_f32<T, EPT>((T *)a.ddt + o, dd);
                    if (a.z) store_f32<T, EPT>((T *)a.dz + o, dz);
                } else {
                    store_part<T, EPT>((T *)a.du + o, du, lleft);
                    store_part<T, EPT>((T *)a.ddt + o, dd, lleft);
                    if (a.z) store_part<T, EPT>((T *)a.dz + o, dz, lleft);
                }
            }
        }
    }
    // the span's part of dA, dDskip, ddt_bias; a slot without rows adds zeros
    if (live) store_f32<float, 4>(a.part_A + at * N + 4 * q, dA);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        sY[lt * ROW + lc + i] = dD[i];
        sE[lt * ROW + lc + i] = dbias[i];
    }
    __syncthreads();
    if (tid < CH && b.cin + tid < a.Dg) {
        float x = 0.f, y = 0.f;
        for (int t = 0; t < kTile; ++t) {
            x += sY[t * ROW + tid];
            y += sE[t * ROW + tid];
        }
        const long long o = b.slot * a.D + (long long)b.g * a.Dg + b.cin + tid;
        a.part_D[o] = x;
        a.part_bias[o] = y;
    }
}

// dB, dC of a row: the sums of its group's channel blocks, in order.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_bc_kernel(const SsmP a, T *dB, T *dC, int N) {
    const long long per = (long long)a.G * 2 * N, rows = a.q.rows();
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = id / per;
    if (row >= rows) return;
    if (a.q.cu && (row < a.q.lo(0) || row >= a.q.lo(a.q.S))) return;   // of no sequence: not written
    const int k = (int)(id % per), g = k / (2 * N), i = k % (2 * N);
    const float *p = a.part_BC + ((long long)g * a.cpg * rows + row) * (2 * N) + i;
    float v = 0.f;
#pragma unroll 4
    for (int m = 0; m < a.cpg; ++m) v += p[(long long)m * rows * (2 * N)];
    const long long o = (row * a.G + g) * N;
    if (i < N) dB[o + i] = from_f32<T>(v);
    else dC[o + i - N] = from_f32<T>(v);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Parts of the workspace: seams, sums of delta, partial sums; off[6] is the whole.
void bwd_parts(const SsmArgs &a, size_t (&off)[7]) {
    const int CH = 4 * kSsmThreads / a.N, Dg = a.D / a.G;
    const size_t nblk = (size_t)a.G * ((Dg + CH - 1) / CH);
    const size_t slots = (size_t)span_slots(a.cu != nullptr, a.S, a.T, kSpan);
    const size_t sd = up256(slots * a.D * sizeof(float)), sdn = up256(slots * a.D * a.N * sizeof(float));
    off[0] = 0;                 // hst
    off[1] = off[0] + sdn;      // gst
    off[2] = off[1] + sdn;      // sdel, then part_D, part_bias
    off[3] = off[2] + 3 * sd;   // part_A
    off[4] = off[3] + sdn;      // part_BC
    off[5] = off[4] + up256(nblk * (size_t)a.rows * 2 * a.N * sizeof(float));
    off[6] = off[5];
}

template <typename T, int N>
cudaError_t run(const SsmArgs &a, cudaStream_t st) {
    SsmP p = ssm_params<N>(a, kSpan);
    // the gradients' rows are contiguous: whole vectors also need D to be a multiple of EPT
    p.vec = p.vec && a.D % SsmShape<N>::EPT == 0;
    size_t off[7];
    bwd_parts(a, off);
    char *ws = (char *)a.workspace;
    const size_t sd = up256((size_t)p.slots * a.D * sizeof(float));
    p.hst = (float *)(ws + off[0]);
    p.gst = (float *)(ws + off[1]);
    p.sdel = (float *)(ws + off[2]);
    p.part_D = (float *)(ws + off[2] + sd);
    p.part_bias = (float *)(ws + off[2] + 2 * sd);
    p.part_A = (float *)(ws + off[3]);
    p.part_BC = (float *)(ws + off[4]);
    const long long blocks = p.slots * p.nblk;
    const long long bc_blocks = (a.rows * a.G * 2 * N + 255) / 256;
    if (blocks > 0x7fffffffLL || bc_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(ssm_bwd_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)bwd_smem<N>());
    if (e != cudaSuccess) return e;
    a.marks->mark(st);
    ssm_bwd_sweep_kernel<T, N><<<(unsigned)blocks, kSsmThreads, 0, st>>>(p);
    a.marks->mark(st);
    if ((e = launch_ssm_seams(p, N, st)) != cudaSuccess) return e;
    a.marks->mark(st);
    ssm_bwd_kernel<T, N><<<(unsigned)blocks, kSsmThreads, bwd_smem<N>(), st>>>(p);
    a.marks->mark(st);
    if (bc_blocks > 0) ssm_bwd_bc_kernel<T><<<(unsigned)bc_blocks, 256, 0, st>>>(p, (T *)a.dB, (T *)a.dC, N);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    a.marks->mark(st);
    e = launch_sum_rows(p.part_A, a.dA, (long long)a.D * N, p.slots, (long long)a.D * N, st);
    if (e == cudaSuccess && a.dDskip) e = launch_sum_rows(p.part_D, a.dDskip, a.D, p.slots, a.D, st);
    if (e == cudaSuccess && a.ddt_bias) e = launch_sum_rows(p.part_bias, a.ddt_bias, a.D, p.slots, a.D, st);
    return e;
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
    size_t off[7];
    bwd_parts(a, off);
    return off[6];
}
cudaError_t launch_ssm_scan_bwd(const SsmArgs &a, cudaStream_t st) {
    return a.bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace kda
