// rope_f16.cu -- the rotary kernels of rope_kernel.cuh for f16 elements.
#include "rope_kernel.cuh"

namespace vta {

cudaError_t launch_rope_f16(const RopeArgs &a, cudaStream_t stream) {
    return rope_launch<__half>(a, stream);
}

}  // namespace vta
