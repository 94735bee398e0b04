// tc_inst_varlen_sink.cu -- instantiates the packed-sequence variants of the two-tile tcgen05 forward
// kernel under a sink window.
#include "tc_kernel.cuh"

namespace triattn {
namespace tc {

TRIATTN_TC_INSTANTIATE(2, true, true, false, false, true)
TRIATTN_TC_INSTANTIATE(2, true, true, false, true, true)
TRIATTN_TC_INSTANTIATE(2, true, false, false, false, true)
TRIATTN_TC_INSTANTIATE(2, true, false, false, true, true)

}  // namespace tc
}  // namespace triattn
