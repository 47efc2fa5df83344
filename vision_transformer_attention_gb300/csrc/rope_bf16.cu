// rope_bf16.cu -- the rotary kernels of rope_kernel.cuh for bf16 elements.
#include "rope_kernel.cuh"

namespace vta {

cudaError_t launch_rope_bf16(const RopeArgs &a, cudaStream_t stream) {
    return rope_launch<__nv_bfloat16>(a, stream);
}

}  // namespace vta
