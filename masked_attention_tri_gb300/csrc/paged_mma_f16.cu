// paged_mma_f16.cu -- instantiates the paged attention kernel's fp16 cache variants.
#include "paged_mma.cuh"

namespace triattn {
namespace paged {

TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_INSTANTIATE, 0)

}  // namespace paged
}  // namespace triattn
