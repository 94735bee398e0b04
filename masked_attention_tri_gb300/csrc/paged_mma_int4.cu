// paged_mma_int4.cu -- instantiates the paged attention kernel's 4-bit cache variants.
#include "paged_mma.cuh"

namespace triattn {
namespace paged {

TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_INSTANTIATE, 3)

}  // namespace paged
}  // namespace triattn
