// host_cache.cu -- the C entry points of rotary positions and of the paged cache:
// argument checks and launches (include/triattn.h).

#include <cuda_runtime.h>

#include "host_checks.h"

using namespace triattn;

namespace {

// The row stride of a packed (total, H, D) buffer: 0 = H * D, at least H * D, whole 16-byte
// vectors.
ta_status row_stride(long long& rs, int H, int D, int esz) {
    const long long hd = (long long)H * D;
    if (rs == 0) rs = hd;
    if (rs < hd) return TA_ERR_INVALID_ARG;
    if ((rs * esz) % 16 != 0 || rs * esz >= (1LL << 40)) return TA_ERR_UNSUPPORTED;
    return TA_OK;
}

}  // namespace

TA_EXPORT ta_status tri_attn_rotary(const void* q, const void* k, ta_dtype dtype, const int32_t* positions,
                                    const uint64_t* turns, int rotary_dim, int interleaved, float mscale,
                                    int inverse, int total, int Hq, int Hk, int D, long long q_row_stride,
                                    long long k_row_stride, long long q_out_row_stride,
                                    long long k_out_row_stride, void* q_out, void* k_out, void* stream) {
    if (!q || !q_out || !positions || !turns) return TA_ERR_INVALID_ARG;
    if (total < 0 || Hq <= 0 || Hk < 0 || D <= 0) return TA_ERR_INVALID_ARG;
    if (Hk > 0 ? (!k || !k_out) : (k || k_out)) return TA_ERR_INVALID_ARG;
    if (!valid_dtype(dtype)) return TA_ERR_INVALID_ARG;
    if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) return TA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) ||
        !aligned(turns, 8))
        return TA_ERR_INVALID_ARG;
    if (!supported_d(dtype, D)) return TA_ERR_UNSUPPORTED;
    const int esz = dtype_bytes(dtype);
    ta_status st;
    if ((st = row_stride(q_row_stride, Hq, D, esz)) != TA_OK) return st;
    if ((st = row_stride(q_out_row_stride, Hq, D, esz)) != TA_OK) return st;
    if (Hk > 0) {
        if ((st = row_stride(k_row_stride, Hk, D, esz)) != TA_OK) return st;
        if ((st = row_stride(k_out_row_stride, Hk, D, esz)) != TA_OK) return st;
    }
    if ((q == q_out && q_row_stride != q_out_row_stride) || (k && k == k_out && k_row_stride != k_out_row_stride))
        return TA_ERR_INVALID_ARG;
    if (total == 0) return TA_OK;
    RotaryParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.positions = positions;
    p.turns = reinterpret_cast<const unsigned long long*>(turns);
    p.dtype = dtype;
    p.dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    p.mscale = mscale;
    p.total = total;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.q_rs = q_row_stride;
    p.k_rs = k_row_stride;
    p.qo_rs = q_out_row_stride;
    p.ko_rs = k_out_row_stride;
    return launch_rotary(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}
