// Attention with a block table and a length for each request, and the workspace of both kinds.
#include "attn_kernel.cuh"

namespace moe {

size_t attn_workspace_bytes(int B, int q_heads, int heads, int head_dim, size_t* done_off, size_t* group_off, size_t* parts_off) {
    // the group counters and the parts come first: their place does not depend on B, so that the
    // counters after them stay zero whatever the calls' batch sizes are
    const int group = q_heads / heads, dp = dp_of(head_dim);
    const size_t floats = (size_t)rows_of(group, dp, false) * (dp + 2);
    *group_off = 512;
    *parts_off = 512 + 2 * kAttnMaxCtas * sizeof(uint32_t);
    *done_off = *parts_off + 2 * kAttnMaxCtas * floats * sizeof(float);
    const size_t total = *done_off + (size_t)B * heads * ((group + 7) / 8) * sizeof(uint32_t);
    return (total + 255) / 256 * 256;   // moe_workspace_init clears whole 16-byte words
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t s) { return launch_any<false>(a, s); }

}  // namespace moe
