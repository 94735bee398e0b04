// tc_inst_split_sink.cu -- instantiates the key-split kernel's packed-sequence
// variants under a sink window, without a bias.
#include "tc_split.cuh"

namespace triattn {
namespace tc {

TRIATTN_SPLIT_VARLEN_VARIANTS(TRIATTN_SPLIT_INSTANTIATE, true)

}  // namespace tc
}  // namespace triattn
