// kvd_paged_attn64.cu -- paged_attention's kernels at head_dim 64.

#include "kvd_paged_attn.cuh"

namespace kvd {

cudaError_t launch_paged_attention_64(const PaArgs &a, bool bf16, bool cap, cudaStream_t st) {
    return launch_paged<64>(a, bf16, cap, st);
}

}  // namespace kvd
