// tc_inst_split_sink_vbias.cu -- instantiates the key-split kernel's packed-sequence
// variants under a sink window, with a post-scale bias.
#include "tc_split.cuh"

namespace triattn {
namespace tc {

TRIATTN_SPLIT_VARLEN_BIAS_VARIANTS(TRIATTN_SPLIT_INSTANTIATE, true)

}  // namespace tc
}  // namespace triattn
