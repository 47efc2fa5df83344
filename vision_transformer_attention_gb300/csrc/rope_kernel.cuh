// rope_kernel.cuh -- rotary positions on queries and keys, alone or after a
// norm of each head, in one pass over the data: the kernel template and its
// launcher, instantiated per element type by rope_bf16.cu, rope_f16.cu and
// rope_f32.cu.
//
// Pair p of a head turns by the angle pos * f_p:
//   (x1, x2) -> m (x1 cos - x2 sin, x2 cos + x1 sin),
// with (x1, x2) = (x[p], x[p + rd/2]) (half layout) or (x[2p], x[2p + 1])
// (interleaved); elements from rd on pass. With a norm the head is scaled
// first, y = x g / sqrt(mean x^2 + eps), or (x - mean) g / sqrt(var + eps),
// in 32 bits, and rounded once after the rotation.
//
// Angles: phases[p] is f_p / 2 pi in units of 2^-64 turns, so the low 64 bits
// of pos * phases[p] are the angle's fraction of a turn with no rounding at
// any position, three integer multiplies instead of a 64-bit floating product
// and a range reduction. Its top 32 bits, as a signed fraction of a half turn,
// go to sincospif.
//
// Bound: every element is read and written once (memory). A lane holds the
// same 8 (16-bit types) or 4 (32-bit) pairs of each head it visits, so the
// angles of a token are formed once per warp and used for all of its heads;
// L lanes cover one head, 32 / L heads are in flight per warp, and a head's
// norm is a butterfly over its L lanes. Loads are V elements wide, the widest
// width that the pair layout, the strides and the pointers allow. A token's
// heads are dealt over `wpt` warps where there are too few tokens to fill the
// GPU.
#pragma once
#include "vta_internal.h"
#include "sm103_ptx.cuh"

namespace vta {
namespace {

constexpr int kRopeWarps = 4;  // warps per CTA

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float &y) { y = x; }
__device__ __forceinline__ void from_f32(float x, __half &y) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&x)[V]) {
    const RopeVec<T, V> v = *reinterpret_cast<const RopeVec<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(v.e[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[V]) {
    RopeVec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(x[i], v.e[i]);
    *reinterpret_cast<RopeVec<T, V> *>(p) = v;
}

// Sum over the L consecutive lanes (a power of two) that share a head.
__device__ __forceinline__ float lanes_sum(float x, int L) {
    for (int o = L >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

template <typename T, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeArgs A) {
    constexpr int K = (sizeof(T) == 2 ? 8 : 4) / V;  // slots (pairs of vectors) per lane
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int64_t unit = w / A.wpt;
    if (unit >= A.units) return;
    const int first = static_cast<int>(w - unit * A.wpt);
    const int64_t b = unit / A.tokens, t = unit - b * A.tokens;
    const int L = A.lanes, HP = 32 / L;
    const int group = lane / L, sl = lane & (L - 1);
    const int heads = A.heads[0] + A.heads[1];

    // This lane's slots: element offsets of the two vectors of each, and
    // whether they exist. Slots below srot turn; the others hold two
    // neighbouring vectors of the part that passes.
    const int srot = A.rotary / (2 * V);
    int o1[K], o2[K];
    bool has1[K], has2[K], rot[K];
    float c[K][V], s[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int slot = sl + k * L;
        rot[k] = slot < srot;
        if (rot[k] && !INTER) {
            o1[k] = slot * V;
            o2[k] = A.rotary / 2 + slot * V;
        } else {
            o1[k] = rot[k] ? 2 * slot * V : A.rotary + 2 * (slot - srot) * V;
            o2[k] = o1[k] + V;
        }
        has1[k] = o1[k] < A.d;
        has2[k] = o2[k] < A.d;
    }
    if (A.rotary > 0) {
        const int32_t *pos = A.positions + (b * A.pos_batch + t) * A.axes;
        const int p0 = pos[0], p1 = A.axes == 2 ? pos[1] : 0;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (rot[k]) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int pair = (sl + k * L) * V + i;
                    const int64_t at = pair < A.axis_pairs ? p0 : p1;
                    const uint64_t turn = static_cast<uint64_t>(at) * A.phases[pair];
                    const float half_turns =
                        static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
                    float sn, cs;
                    sincospif(half_turns, &sn, &cs);
                    c[k][i] = cs * A.magnitude;
                    s[k][i] = sn * (A.inverse ? -A.magnitude : A.magnitude);
                }
            }
    }

    float g1[NORM ? K : 1][V], g2[NORM ? K : 1][V];  // gains of the current role
    int gains_of = -1;
    const float inv_d = 1.f / static_cast<float>(A.d);
    for (int it = first; it * HP < heads; it += A.wpt) {
        const int hh = it * HP + group;
        const bool live = hh < heads;
        const int role = hh >= A.heads[0] ? 1 : 0;
        const int64_t h = hh - (role ? A.heads[0] : 0);
        float x[K][V], y[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = y[k][i] = 0.f;
        if (live) {
            const T *src = static_cast<const T *>(A.src[role].data) + b * A.src[role].batch_stride +
                           t * A.src[role].token_stride + h * A.src[role].head_stride;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (has1[k]) load_vec<T, V>(src + o1[k], x[k]);
                if (has2[k]) load_vec<T, V>(src + o2[k], y[k]);
            }
        }
        if constexpr (NORM) {
            if (live && role != gains_of) {
                gains_of = role;
                const void *g = A.gain[role];
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int i = 0; i < V; ++i) g1[k][i] = g2[k][i] = 1.f;
                    if (g == nullptr) continue;
                    if (A.gain_f32) {
                        if (has1[k]) load_vec<float, V>(static_cast<const float *>(g) + o1[k], g1[k]);
                        if (has2[k]) load_vec<float, V>(static_cast<const float *>(g) + o2[k], g2[k]);
                    } else {
                        if (has1[k]) load_vec<T, V>(static_cast<const T *>(g) + o1[k], g1[k]);
                        if (has2[k]) load_vec<T, V>(static_cast<const T *>(g) + o2[k], g2[k]);
                    }
                }
            }
            if (A.layer) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += x[k][i] + y[k][i];
                const float mean = lanes_sum(sum, L) * inv_d;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        x[k][i] = has1[k] ? x[k][i] - mean : 0.f;
                        y[k][i] = has2[k] ? y[k][i] - mean : 0.f;
                    }
            }
            float sq = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) sq += x[k][i] * x[k][i] + y[k][i] * y[k][i];
            const float r = rsqrtf(lanes_sum(sq, L) * inv_d + A.eps);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[k][i] *= r * g1[k][i];
                    y[k][i] *= r * g2[k][i];
                }
        }
        if (!live) continue;
        T *dst = static_cast<T *>(A.dst[role].data) + b * A.dst[role].batch_stride +
                 t * A.dst[role].token_stride + h * A.dst[role].head_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (rot[k]) {
                if constexpr (INTER && V > 1) {
                    // pairs are neighbours inside each vector
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float a = x[k][2 * i], bb = x[k][2 * i + 1];
                        x[k][2 * i] = a * c[k][i] - bb * s[k][i];
                        x[k][2 * i + 1] = bb * c[k][i] + a * s[k][i];
                        const float e = y[k][2 * i], f = y[k][2 * i + 1];
                        y[k][2 * i] = e * c[k][V / 2 + i] - f * s[k][V / 2 + i];
                        y[k][2 * i + 1] = f * c[k][V / 2 + i] + e * s[k][V / 2 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float a = x[k][i], bb = y[k][i];
                        x[k][i] = a * c[k][i] - bb * s[k][i];
                        y[k][i] = bb * c[k][i] + a * s[k][i];
                    }
                }
            }
            if (has1[k]) store_vec<T, V>(dst + o1[k], x[k]);
            if (has2[k]) store_vec<T, V>(dst + o2[k], y[k]);
        }
    }
}

template <typename T, int V>
cudaError_t rope_launch_v(RopeArgs A, cudaStream_t stream) {
    constexpr int K = (sizeof(T) == 2 ? 8 : 4) / V;
    const int slots = A.rotary / (2 * V) + (A.d - A.rotary + 2 * V - 1) / (2 * V);
    A.lanes = 1;
    while (A.lanes * K < slots) A.lanes *= 2;
    const int heads = A.heads[0] + A.heads[1];
    const int iters = (heads * A.lanes + 31) / 32;
    // warps per token: one, unless that leaves fewer than 16 warps per SM
    const int64_t want = 16ll * sm_count();
    int64_t wpt = (want + A.units - 1) / A.units;
    A.wpt = static_cast<int>(wpt < iters ? wpt : iters);
    const int64_t ctas = (A.units * A.wpt + kRopeWarps - 1) / kRopeWarps;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    const dim3 grid(static_cast<unsigned>(ctas));
    const bool norm = A.norm != 0;
    void (*kernel)(const RopeArgs) =
        A.interleaved ? (norm ? rope_kernel<T, V, true, true> : rope_kernel<T, V, true, false>)
                      : (norm ? rope_kernel<T, V, false, true> : rope_kernel<T, V, false, false>);
    return launch_pdl(kernel, grid, dim3(32 * kRopeWarps), 0, stream, A);
}

// The widest vectors that the pair layout, the strides and the pointers allow.
template <typename T>
cudaError_t rope_launch(const RopeArgs &A, cudaStream_t stream) {
    int64_t bits = A.rotary / 2;  // a slot turns whole: 2 V divides the rotated part
    bits |= A.d - A.rotary;
    for (int r = 0; r < 2; ++r) {
        if (A.heads[r] == 0) continue;
        for (const RopeView *v : {&A.src[r], &A.dst[r]})
            bits |= v->batch_stride | v->token_stride | v->head_stride |
                    static_cast<int64_t>(reinterpret_cast<uintptr_t>(v->data) / sizeof(T));
        if (A.norm && A.gain[r] != nullptr)
            bits |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(A.gain[r]) /
                                         (A.gain_f32 ? sizeof(float) : sizeof(T)));
    }
    if constexpr (sizeof(T) == 2)
        if (bits % 8 == 0) return rope_launch_v<T, 8>(A, stream);
    if (bits % 4 == 0) return rope_launch_v<T, 4>(A, stream);
    if (bits % 2 == 0) return rope_launch_v<T, 2>(A, stream);
    return rope_launch_v<T, 1>(A, stream);
}

}  // namespace
}  // namespace vta
