// rope.cu -- rotary positions: the phase tables (rope_build_phases) and the
// entry points rope_fwd and qk_norm_rope_fwd of rpe_attn.h (argument checks
// and the launch; the kernels are in rope_kernel.cuh).
#include "rpe_attn.h"
#include "vta_internal.h"

#include <cmath>
#include <cstdint>

namespace vta {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// One thread per pair of one axis. f is formed in 64 bits; f / 2 pi mod 1, a
// fraction of a turn per position, is kept as a 64-bit fixed-point number. The
// attention of a position p then sees an angle p f within p 2^-52 f of the
// exact one (5e-7 rad at p = 2^31, f = 1).
__global__ void build_phases_kernel(int per_axis, int axes, int scaling, double base, double factor,
                                    double context, double low, double high, uint64_t *phases) {
    const int i = threadIdx.x, half = per_axis / 2;
    if (i >= half) return;
    if (scaling == RPE_ROPE_NTK)
        base *= pow(factor, static_cast<double>(per_axis) / (per_axis - 2));
    double f = pow(base, -2.0 * i / per_axis);
    if (scaling == RPE_ROPE_LINEAR) {
        f /= factor;
    } else if (scaling == RPE_ROPE_BANDS) {
        // the pair's turns over the context: few -> stretched, many -> kept
        const double s = fmin(fmax((context * f / kTwoPi - low) / (high - low), 0.0), 1.0);
        f *= (1.0 - s) / factor + s;
    } else if (scaling == RPE_ROPE_YARN) {
        // pair indices (over the whole head) that turn `high` and `low` times
        const double unit = per_axis / (2.0 * log(base));
        const double first = fmax(floor(unit * log(context / (high * kTwoPi))), 0.0);
        const double last = fmin(ceil(unit * log(context / (low * kTwoPi))), per_axis - 1.0);
        const double ramp = fmin(fmax((i - first) / fmax(last - first, 0.001), 0.0), 1.0);
        f = f / factor * ramp + f * (1.0 - ramp);
    }
    const double turns = f / kTwoPi;
    const double frac = turns - floor(turns);  // < 1, exact
    const uint64_t phase = static_cast<uint64_t>(frac * 0x1p64);
    for (int a = 0; a < axes; ++a) phases[a * half + i] = phase;
}

bool element_aligned(const void *p, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % size == 0;
}

// Takes a caller's view; strides of axes with one entry are dropped so that
// they do not narrow the vectors.
bool take_view(const rpe_view *v, bool out, int64_t batch, int64_t tokens, int heads, size_t size,
               RopeView *r) {
    if (v == nullptr || v->data == nullptr || !element_aligned(v->data, size)) return false;
    if (v->batch_stride < 0 || v->token_stride < 0 || v->head_stride < 0) return false;
    r->data = v->data;
    r->batch_stride = batch > 1 ? v->batch_stride : 0;
    r->token_stride = tokens > 1 ? v->token_stride : 0;
    r->head_stride = heads > 1 ? v->head_stride : 0;
    // an output whose entries share memory has no defined value
    return !out || ((batch <= 1 || r->batch_stride > 0) && (tokens <= 1 || r->token_stride > 0) &&
                    (heads <= 1 || r->head_stride > 0));
}

int rope_call(const rpe_view *q, const rpe_view *k, const rpe_view *q_out, const rpe_view *k_out,
              const int32_t *positions, int axes, const uint64_t *phases, int rotary_dim,
              float magnitude, unsigned flags, int64_t batch, int64_t tokens, int heads_q,
              int heads_k, int d, int dtype, RopeArgs &a, void *stream) {
    if (batch < 0 || tokens < 0 || heads_q < 1 || heads_k < 0 || d < 1 || rotary_dim < 0 ||
        rotary_dim > d || (axes != 1 && axes != 2) || rotary_dim % (2 * axes) != 0)
        return RPE_ERR_INVALID_ARG;
    if ((flags & ~static_cast<unsigned>(RPE_ROPE_INTERLEAVED | RPE_ROPE_INVERSE |
                                        RPE_ROPE_BATCH_POSITIONS)) != 0 ||
        !std::isfinite(magnitude))
        return RPE_ERR_INVALID_ARG;
    if (dtype != RPE_DTYPE_BF16 && dtype != RPE_DTYPE_F32 && dtype != RPE_DTYPE_F16)
        return RPE_ERR_INVALID_ARG;
    if (d > 256 || heads_q > 65536 || heads_k > 65536) return RPE_ERR_UNSUPPORTED;
    if (batch > INT32_MAX || tokens > INT32_MAX || batch * tokens > INT32_MAX)
        return RPE_ERR_UNSUPPORTED;
    a.units = batch * tokens;
    if (a.units == 0) return RPE_OK;  // nothing to turn
    const size_t size = dtype == RPE_DTYPE_F32 ? 4 : 2;
    if (!take_view(q, false, batch, tokens, heads_q, size, &a.src[0]) ||
        !take_view(q_out, true, batch, tokens, heads_q, size, &a.dst[0]))
        return RPE_ERR_INVALID_ARG;
    if (heads_k > 0 && (!take_view(k, false, batch, tokens, heads_k, size, &a.src[1]) ||
                        !take_view(k_out, true, batch, tokens, heads_k, size, &a.dst[1])))
        return RPE_ERR_INVALID_ARG;
    if (rotary_dim > 0 && (positions == nullptr || phases == nullptr ||
                           !element_aligned(positions, 4) || !element_aligned(phases, 8)))
        return RPE_ERR_INVALID_ARG;
    a.heads[0] = heads_q;
    a.heads[1] = heads_k;
    a.tokens = tokens;
    a.d = d;
    a.rotary = rotary_dim;
    a.axes = axes;
    a.axis_pairs = rotary_dim / 2 / axes;
    a.positions = positions;
    a.pos_batch = (flags & RPE_ROPE_BATCH_POSITIONS) ? tokens : 0;
    a.phases = phases;
    a.magnitude = magnitude;
    a.inverse = (flags & RPE_ROPE_INVERSE) ? 1 : 0;
    a.interleaved = (flags & RPE_ROPE_INTERLEAVED) ? 1 : 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == RPE_DTYPE_BF16  ? launch_rope_bf16(a, st)
                            : dtype == RPE_DTYPE_F16 ? launch_rope_f16(a, st)
                                                     : launch_rope_f32(a, st);
    if (err == cudaErrorNotSupported) return RPE_ERR_UNSUPPORTED;
    return err == cudaSuccess ? RPE_OK : RPE_ERR_CUDA;
}

}  // namespace
}  // namespace vta

using namespace vta;

extern "C" {

int rope_build_phases(int rotary_dim, int axes, int scaling, double base, double factor,
                      double context, double low, double high, uint64_t *phases, float *magnitude,
                      void *stream) {
    if (phases == nullptr || magnitude == nullptr || !element_aligned(phases, 8) ||
        (axes != 1 && axes != 2) || rotary_dim < 2 || rotary_dim % (2 * axes) != 0 ||
        scaling < RPE_ROPE_NONE || scaling > RPE_ROPE_YARN)
        return RPE_ERR_INVALID_ARG;
    if (rotary_dim > 256) return RPE_ERR_UNSUPPORTED;
    if (!std::isfinite(base) || base <= 1.0) return RPE_ERR_INVALID_ARG;
    if (scaling != RPE_ROPE_NONE && (!std::isfinite(factor) || factor < 1.0))
        return RPE_ERR_INVALID_ARG;
    if (scaling == RPE_ROPE_NTK && rotary_dim / axes < 4) return RPE_ERR_INVALID_ARG;
    if ((scaling == RPE_ROPE_BANDS || scaling == RPE_ROPE_YARN) &&
        (!std::isfinite(context) || context <= 0.0 || !std::isfinite(low) || low <= 0.0 ||
         !std::isfinite(high) || high <= low))
        return RPE_ERR_INVALID_ARG;
    *magnitude = scaling == RPE_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    build_phases_kernel<<<1, 128, 0, static_cast<cudaStream_t>(stream)>>>(
        rotary_dim / axes, axes, scaling, base, factor, context, low, high, phases);
    return cudaGetLastError() == cudaSuccess ? RPE_OK : RPE_ERR_CUDA;
}

int rope_fwd(const rpe_view *q, const rpe_view *k, const rpe_view *q_out, const rpe_view *k_out,
             const int32_t *positions, int axes, const uint64_t *phases, int rotary_dim,
             float magnitude, unsigned flags, int64_t batch, int64_t tokens, int heads_q,
             int heads_k, int d, int dtype, void *stream) {
    if (rotary_dim < 2) return RPE_ERR_INVALID_ARG;
    RopeArgs a{};
    return rope_call(q, k, q_out, k_out, positions, axes, phases, rotary_dim, magnitude, flags,
                     batch, tokens, heads_q, heads_k, d, dtype, a, stream);
}

int qk_norm_rope_fwd(const rpe_view *q, const rpe_view *k, const rpe_view *q_out,
                     const rpe_view *k_out, int norm, float eps, const void *gain_q,
                     const void *gain_k, int gain_dtype, const int32_t *positions, int axes,
                     const uint64_t *phases, int rotary_dim, float magnitude, unsigned flags,
                     int64_t batch, int64_t tokens, int heads_q, int heads_k, int d, int dtype,
                     void *stream) {
    if ((norm != RPE_NORM_RMS && norm != RPE_NORM_LAYER) || !std::isfinite(eps) || eps < 0.f ||
        (gain_dtype != dtype && gain_dtype != RPE_DTYPE_F32) || (flags & RPE_ROPE_INVERSE) != 0)
        return RPE_ERR_INVALID_ARG;
    const size_t size = gain_dtype == RPE_DTYPE_F32 ? 4 : 2;
    if ((gain_q != nullptr && !element_aligned(gain_q, size)) ||
        (gain_k != nullptr && !element_aligned(gain_k, size)))
        return RPE_ERR_INVALID_ARG;
    RopeArgs a{};
    a.norm = 1;
    a.layer = norm == RPE_NORM_LAYER ? 1 : 0;
    a.eps = eps;
    a.gain[0] = gain_q;
    a.gain[1] = gain_k;
    a.gain_f32 = gain_dtype == RPE_DTYPE_F32 ? 1 : 0;
    return rope_call(q, k, q_out, k_out, positions, axes, phases, rotary_dim, magnitude, flags,
                     batch, tokens, heads_q, heads_k, d, dtype, a, stream);
}

}  // extern "C"
