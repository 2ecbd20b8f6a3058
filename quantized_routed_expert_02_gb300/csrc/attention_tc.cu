// The tensor-core attention kernel for chains in a window (moe_attention_paged).
#include "attention_tc.cuh"

namespace moeq4k {
namespace attn {

size_t tc_part_bytes(int D) { return size_t(2) * tc5::kMaxGrid * part_floats(2 * tc5::kHalf, D) * 4; }

cudaError_t init_tc() { return tc5::init_form<tc5::kPaged>(); }

cudaError_t launch_tc(const AttnArgs &a, const Params &p, int num_sms, cudaStream_t s) {
    return tc5::launch_form<tc5::kPaged>(a, p, num_sms, s);
}

}  // namespace attn
}  // namespace moeq4k
