// gdn_linear_bf16.cu -- linear attention with a fixed decay for each head, bf16 states (gdn_linear.cuh).
#include "gdn_linear.cuh"

namespace gdn {

cudaError_t launch_linear_bf16state(const LinearParams& p, bool qkv_bf16, cudaStream_t s) {
    return launch_linear<__nv_bfloat16>(p, qkv_bf16, s);
}

}  // namespace gdn
