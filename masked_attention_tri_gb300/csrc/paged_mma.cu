// paged_mma.cu -- host side of the tensor-core kernel over a paged cache: tensor maps
// of the pages and the choice of the variant.

#include "paged_mma.cuh"

namespace triattn {
namespace tc {
bool encode_map_4d(CUtensorMap* m, CUtensorMapDataType dt, const void* ptr, const uint64_t (&dims)[4],
                   const uint64_t (&strides)[3], const uint32_t (&box)[4], CUtensorMapSwizzle sw);
}
namespace paged {

TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_EXTERN, 0)
TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_EXTERN, 1)
TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_EXTERN, 2)

namespace {

template <int TYPE>
cudaError_t launch_type(const MmaParams& P, cudaStream_t stream) {
    const int nt = P.p.RT / 8;
    if (P.p.D <= 64)
        return nt == 1   ? launch_mma_variant<TYPE, 1, 1>(P, stream)
               : nt == 2 ? launch_mma_variant<TYPE, 1, 2>(P, stream)
                         : launch_mma_variant<TYPE, 1, 4>(P, stream);
    if (P.p.D <= 128)
        return nt == 1 ? launch_mma_variant<TYPE, 2, 1>(P, stream) : launch_mma_variant<TYPE, 2, 2>(P, stream);
    return nt == 1 ? launch_mma_variant<TYPE, 4, 1>(P, stream) : launch_mma_variant<TYPE, 4, 2>(P, stream);
}

}  // namespace

cudaError_t launch_mma(const PagedParams& p, cudaStream_t stream) {
    MmaParams P;
    P.p = p;
    const bool codes = p.cache_dtype == TA_E4M3;
    const uint64_t esz = codes ? 1 : 2;
    // (codes move as pairs: only their bytes count)
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    // (D, slot, head, page); boxes of 128 bytes x the slots of a page that fall in one tile
    const uint64_t dims[4] = {(uint64_t)p.D * esz / 2, (uint64_t)p.page, (uint64_t)p.Hk, (uint64_t)p.num_pages};
    const uint32_t box[4] = {64u, (uint32_t)(p.page < p.tile ? p.page : p.tile), 1, 1};
    const uint64_t ks[3] = {p.ks[2] * esz, p.ks[1] * esz, p.ks[0] * esz};
    const uint64_t vs[3] = {p.vs[2] * esz, p.vs[1] * esz, p.vs[0] * esz};
    if (!tc::encode_map_4d(&P.tm_k, dt, p.k_cache, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tc::encode_map_4d(&P.tm_v, dt, p.v_cache, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (codes) return launch_type<2>(P, stream);
    return p.cache_dtype == TA_BF16 ? launch_type<1>(P, stream) : launch_type<0>(P, stream);
}

}  // namespace paged
}  // namespace triattn
