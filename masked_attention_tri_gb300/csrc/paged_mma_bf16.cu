// paged_mma_bf16.cu -- instantiates the paged attention kernel's bf16 cache variants.
#include "paged_mma.cuh"

namespace triattn {
namespace paged {

TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_INSTANTIATE, 1)

}  // namespace paged
}  // namespace triattn
