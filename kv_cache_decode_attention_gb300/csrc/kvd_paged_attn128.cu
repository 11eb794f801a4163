// kvd_paged_attn128.cu -- paged_attention's kernels at head_dim 128.

#include "kvd_paged_attn.cuh"

namespace kvd {

cudaError_t launch_paged_attention_128(const PaArgs &a, bool bf16, bool cap, cudaStream_t st) {
    return launch_paged<128>(a, bf16, cap, st);
}

}  // namespace kvd
