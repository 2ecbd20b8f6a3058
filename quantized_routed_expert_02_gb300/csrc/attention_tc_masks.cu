// The tensor-core attention kernel for trees of drafted tokens and for sinks
// (moe_attention_cache over 16-bit values).
#include "attention_tc.cuh"

namespace moeq4k {
namespace attn {

cudaError_t init_tc_masks() { return tc5::init_form<tc5::kMasked>(); }

cudaError_t launch_tc_masks(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s) {
    return tc5::launch_form<tc5::kMasked>(a, p, num_sms, s);
}

}  // namespace attn
}  // namespace moeq4k
