// paged_mma_e4m3.cu -- instantiates the paged attention kernel's 8-bit cache variants.
#include "paged_mma.cuh"

namespace triattn {
namespace paged {

TRIATTN_PAGED_VARIANTS(TRIATTN_PAGED_INSTANTIATE, 2)

}  // namespace paged
}  // namespace triattn
