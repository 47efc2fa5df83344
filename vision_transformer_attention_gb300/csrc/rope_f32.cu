// rope_f32.cu -- the rotary kernels of rope_kernel.cuh for f32 elements.
#include "rope_kernel.cuh"

namespace vta {

cudaError_t launch_rope_f32(const RopeArgs &a, cudaStream_t stream) {
    return rope_launch<float>(a, stream);
}

}  // namespace vta
