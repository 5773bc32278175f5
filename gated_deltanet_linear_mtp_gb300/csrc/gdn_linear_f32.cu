// gdn_linear_f32.cu -- linear attention with a fixed decay for each head, fp32 states (gdn_linear.cuh).
#include "gdn_linear.cuh"

namespace gdn {

cudaError_t launch_linear_f32state(const LinearParams& p, bool qkv_bf16, cudaStream_t s) {
    return launch_linear<float>(p, qkv_bf16, s);
}

}  // namespace gdn
