// zero_rest.cu -- zeros into the rows of a packed buffer that belong to no sequence: those before the first offset and from
// the last one on.
//
// Bound: memory where there are such rows, a launch where there are none (no row is read or written then, and the host needs
// not know).

#include "internal.h"

namespace triattn {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) zero_rest_kernel(uint4* x, long long vecs, const int32_t* cu, int num_seqs, int total) {
    const long long lo = min(max(cu[0], 0), total), hi = min(max((long long)cu[num_seqs], lo), (long long)total);
    const long long n = (lo + total - hi) * vecs;  // vectors: of the rows [0, lo), then of [hi, total)
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < n; e += (long long)gridDim.x * kThreads)
        x[e < lo * vecs ? e : e + (hi - lo) * vecs] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

cudaError_t launch_zero_rest(void* x, long long row_bytes, const int32_t* cu, int num_seqs, int total, cudaStream_t stream) {
    const long long blocks = ((long long)total * (row_bytes / 16) + kThreads - 1) / kThreads;
    zero_rest_kernel<<<(unsigned)(blocks < 304 ? blocks : 304), kThreads, 0, stream>>>(static_cast<uint4*>(x), row_bytes / 16, cu, num_seqs, total);
    return cudaGetLastError();
}

}  // namespace triattn
