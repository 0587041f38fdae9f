// Attention with a table of pages and a length for each key-value head of a request: a.B counts those, and
// table, table_ld and seq_lens are theirs.
#include "attn_kernel.cuh"

namespace moe {

cudaError_t launch_attn_pages(const AttnArgs& a, cudaStream_t s) { return launch_any<true>(a, s); }

}  // namespace moe
