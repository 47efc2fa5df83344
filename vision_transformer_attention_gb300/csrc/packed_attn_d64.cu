// packed_attn_d64.cu -- the packed attention kernels for head sizes up to 64.
#include "packed_attn.cuh"

namespace vta {

cudaError_t launch_packed_attn_d64(const PackedAttnMaps &m, const PackedAttnArgs &a, bool bf16,
                                   int kind, int ctas, cudaStream_t stream) {
    return bf16 ? pa_launch<__nv_bfloat16, 64>(m, a, kind, ctas, stream)
                : pa_launch<__half, 64>(m, a, kind, ctas, stream);
}

}  // namespace vta
