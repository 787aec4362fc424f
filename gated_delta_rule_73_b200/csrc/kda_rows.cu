// kda_rows.cu -- the pass that zeroes the rows of no sequence in packed calls.  2.7 us of a 3001-row
// call, where its one launch and the bounds' loads are all it does.
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

}  // namespace

cudaError_t launch_zero_rest(const ZeroRest &z, const int *cu, int S, long long T, cudaStream_t st) {
    zero_rest_kernel<<<T < 296 ? (T > 0 ? (unsigned)T : 1u) : 296u, 256, 0, st>>>(z, cu, S, T);
    return cudaGetLastError();
}

}  // namespace kda
