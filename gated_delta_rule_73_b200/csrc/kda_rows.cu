// kda_rows.cu -- small passes that several operators of kda_layers.h share.
#include "kda_layers_internal.h"
#include "kda_rows.cuh"

namespace kda {
namespace {

// Rows before cu[0] and from cu[S] on, of up to five outputs.  Where there are none, which is
// the usual case, every block ends after two loads.
__global__ void __launch_bounds__(256) zero_rest_kernel(const ZeroRest z, const int *cu, int S, long long T) {
    Seqs q{cu, S, T};
    const long long head = q.lo(0), tail = q.lo(S) > head ? q.lo(S) : head;
    for (int i = 0; i < z.count; ++i) {
        unsigned char *p = (unsigned char *)z.p[i];
        for (long long k = blockIdx.x; k < head + (T - tail); k += gridDim.x) {
            const long long r = k < head ? k : tail + (k - head);
            unsigned char *row = p + r * z.pitch[i];
            // element types are 2 or 4 bytes and rows start at one of them
            for (long long b = 2 * threadIdx.x; b < z.bytes[i]; b += 512)
                *reinterpret_cast<unsigned short *>(row + b) = 0;
        }
    }
}

__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *__restrict__ in, float *out, long long n,
                                                        long long count, long long stride) {
    __shared__ float s[32][33];
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (i < n)
        for (long long k = threadIdx.y; k < count; k += 32) v += in[k * stride + i];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(s[threadIdx.x][threadIdx.y]);
    const long long o = (long long)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < n) out[o] = v;
}

}  // namespace

cudaError_t launch_zero_rest(const ZeroRest &z, const int *cu, int S, long long T, cudaStream_t st) {
    zero_rest_kernel<<<T < 296 ? (T > 0 ? (unsigned)T : 1u) : 296u, 256, 0, st>>>(z, cu, S, T);
    return cudaGetLastError();
}

cudaError_t launch_sum_rows(const float *in, float *out, long long n, long long count, long long stride,
                            cudaStream_t st) {
    if (n <= 0) return cudaSuccess;
    sum_rows_kernel<<<(unsigned)((n + 31) / 32), dim3(32, 32), 0, st>>>(in, out, n, count, stride);
    return cudaGetLastError();
}

}  // namespace kda
