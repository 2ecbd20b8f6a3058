// The tensor-core attention kernel over 8-bit codes (moe_attention_cache with scales).
#include "attention_tc.cuh"

namespace moeq4k {
namespace attn {

cudaError_t init_tc_codes() { return tc5::init_form<tc5::kCodes>(); }

cudaError_t launch_tc_codes(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s) {
    return tc5::launch_form<tc5::kCodes>(a, p, num_sms, s);
}

}  // namespace attn
}  // namespace moeq4k
