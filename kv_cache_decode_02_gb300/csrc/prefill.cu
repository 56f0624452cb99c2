// Causal attention of packed prompts and of chunks over a cache, every token over all cells in front
// of it: the plain form of prefill_kernel.cuh.
#include "prefill_kernel.cuh"

namespace kvattn {

cudaError_t launch_prefill(const PrefillParams& p, int kv_type, int head_dim, int n_ctas, cudaStream_t stream, bool pdl) {
    return run_prefill<kPlain>(p, kv_type, head_dim, n_ctas, stream, pdl);
}

}  // namespace kvattn
