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
// Bound: every element is read and written once (memory). Two kernels:
//
//   Where everything can move in 16-byte vectors, persistent warps: L lanes take
//   a head, each lane two vectors, 32 / L heads at a time (a pass). The vectors
//   of the next kRopeStages - 1 passes are on their way into a shared-memory
//   ring (cp.async, each lane reads back only what it asked for, so no barrier);
//   with loads into registers a warp had one pass in flight and reached 2.4 to
//   4.2 TB/s. Cosines and sines are formed once per token, by the lanes
//   together. A head's norm is a butterfly over its L lanes, and the arithmetic
//   runs on pairs of floats (one instruction for two).
//     rope_token_kernel: a warp takes a token's passes, angles and gains in
//     registers, addresses by additions.
//     rope_run_kernel, for few heads: a warp takes a run of (token, head) rows
//     whatever tokens they belong to, so that no lanes idle and a token's start
//     is not paid per pass; angles and gains in shared memory.
//
//   rope_any_kernel, for every other stride, alignment and pair count: the
//   same split, element by element, V at a time, no ring.
//
// Where there are too few tokens to fill the GPU a token's passes are dealt
// over `wpt` warps.
#pragma once
#include "vta_internal.h"
#include "sm103_ptx.cuh"

namespace vta {
namespace {

constexpr int kRopeWarps = 4;  // per CTA
constexpr int kRopeStages = 4;     // passes of a warp in shared memory or on their way
// CTAs per SM of the persistent kernel (its registers allow no more)
constexpr int rope_ctas_per_sm(bool norm) { return norm ? 5 : 6; }

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

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

// A 16-byte vector as pairs of floats (E elements, E / 2 pairs) and back.
template <typename T>
struct Wide;
template <>
struct Wide<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void get(uint4 v, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 put(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y),
                          __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    }
};
template <>
struct Wide<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void get(uint4 v, float2 (&x)[4]) {
        x[0] = two(v.x), x[1] = two(v.y), x[2] = two(v.z), x[3] = two(v.w);
    }
    static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
        return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                          pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
    }
};
template <>
struct Wide<__half> {
    static constexpr int E = 8;
    static __device__ __forceinline__ float2 two(uint32_t w) {
        return __half22float2(*reinterpret_cast<__half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float2 x) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ void get(uint4 v, float2 (&x)[4]) {
        x[0] = two(v.x), x[1] = two(v.y), x[2] = two(v.z), x[3] = two(v.w);
    }
    static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
        return make_uint4(pack(x[0]), pack(x[1]), pack(x[2]), pack(x[3]));
    }
};

template <typename T, bool INTER, bool NORM>
__global__ void __launch_bounds__(32 * kRopeWarps, rope_ctas_per_sm(NORM))
rope_token_kernel(const __grid_constant__ RopeArgs A) {
    using W = Wide<T>;
    constexpr int E = W::E;  // elements per vector: a lane holds 2 E, E pairs
    extern __shared__ __align__(128) float rope_smem[];
    const int pairs = A.rotary / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // shared memory: the ring [stage][vector][thread] of 16 bytes, each warp's
    // cosines and sines, the gains of both roles in fp32
    float *cos_s = rope_smem + kRopeStages * 2 * 32 * kRopeWarps * 4 + warp * 2 * pairs;
    float *sin_s = cos_s + pairs;
    float *gain_s = rope_smem + kRopeStages * 2 * 32 * kRopeWarps * 4 + kRopeWarps * 2 * pairs;
    const uint32_t ring = smem_u32(rope_smem) + threadIdx.x * 16;
    constexpr uint32_t kVec = 32 * kRopeWarps * 16, kStage = 2 * kVec;

    const int L = A.lanes, HP = 32 / L;
    const int group = lane / L, sl = lane & (L - 1);
    // This lane's slot: the element offsets of its two vectors. Slots below
    // srot turn; the others hold two neighbouring vectors of the part that
    // passes (the last of them may have one).
    const int srot = A.rotary / (2 * E);
    const bool rot = sl < srot;
    const int o1 = rot && !INTER ? sl * E : (rot ? 2 * sl * E : A.rotary + 2 * (sl - srot) * E);
    const int o2 = rot && !INTER ? pairs + sl * E : o1 + E;
    const bool has1 = o1 < A.d, has2 = o2 < A.d;

    const int pq = (A.heads[0] + HP - 1) / HP, passes = pq + (A.heads[1] + HP - 1) / HP;
    const uint32_t items = static_cast<uint32_t>(A.units) * static_cast<uint32_t>(A.wpt);
    const uint32_t warps = gridDim.x * kRopeWarps;
    const uint32_t item0 = blockIdx.x * kRopeWarps + warp;

    // A walk over this warp's passes (the queries', then the keys', of each
    // item). Inside a role a pass costs two additions; jump() does the rest.
    struct Walk {
        uint32_t item, unit;
        int pass, end;  // end: of the role's passes
        int h, heads;   // this lane's head, the role's heads
        T *p;           // its first channel
        int64_t step;
    };
    const int hs = A.wpt * HP;
    const auto jump = [&](Walk &c, const RopeView *views) {
        if (c.pass >= passes) {
            c.item += warps;
            if (c.item >= items) return;
            c.unit = A.wpt == 1 ? c.item : c.item / A.wpt;
            c.pass = static_cast<int>(c.item - c.unit * A.wpt);
        }
        const uint32_t tokens = static_cast<uint32_t>(A.tokens);
        const uint32_t b = A.units == A.tokens ? 0 : c.unit / tokens, t = c.unit - b * tokens;
        const bool key = c.pass >= pq;
        const RopeView &v = views[key ? 1 : 0];
        c.end = key ? passes : pq;
        c.heads = key ? A.heads[1] : A.heads[0];
        c.h = (c.pass - (key ? pq : 0)) * HP + group;
        c.p = static_cast<T *>(v.data) + b * v.batch_stride + t * v.token_stride +
              c.h * v.head_stride;
        c.step = hs * v.head_stride;
    };
    const auto next = [&](Walk &c, const RopeView *views) {
        c.pass += A.wpt;
        c.h += hs;
        c.p += c.step;
        if (c.pass >= c.end) jump(c, views);
    };
    const auto start = [&](Walk &c, const RopeView *views) {
        c.item = item0 - warps;  // jump() moves on to item0
        c.pass = passes;
        jump(c, views);
    };

    griddep_wait();
    Walk in, out;
    start(in, A.src);
    start(out, A.dst);
    const auto ask = [&](int stage) {  // the next pass's vectors into the ring
        if (in.item < items) {
            if (in.h < in.heads && has1) {
                cp_async16(ring + stage * kStage, in.p + o1);
                if (has2) cp_async16(ring + stage * kStage + kVec, in.p + o2);
            }
            next(in, A.src);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kRopeStages - 1; ++s) ask(s);
    // the gains behind the first passes, so that the two reads' latencies overlap
    if constexpr (NORM) {
        for (int i = threadIdx.x; i < 2 * A.d; i += 32 * kRopeWarps) {
            const int role = i >= A.d ? 1 : 0, e = i - role * A.d;
            const void *g = A.gain[role];
            // channels past d would be read by lanes without a second vector
            gain_s[role * (A.d + E) + e] =
                g == nullptr ? 1.f
                             : (A.gain_f32 ? static_cast<const float *>(g)[e]
                                           : to_f32(static_cast<const T *>(g)[e]));
        }
        if (threadIdx.x < 2 * E)
            gain_s[(threadIdx.x >= E ? A.d + E : 0) + A.d + threadIdx.x % E] = 0.f;
        __syncthreads();
    }
    if (item0 >= items) return;

    // (c, s, n = -s) of this lane's pairs, two pairs to a float2
    const auto turn = [&](float2 v1, float2 v2, float2 c, float2 s, float2 n, float2 &y1,
                          float2 &y2) {
        y1 = ffma2(v2, n, fmul2(v1, c));
        y2 = ffma2(v1, s, fmul2(v2, c));
    };
    float2 c[E / 2], s[E / 2], n[E / 2];
    float2 g1[NORM ? E / 2 : 1], g2[NORM ? E / 2 : 1];
    const float inv_d = 1.f / static_cast<float>(A.d);
    uint32_t turned = ~0u;  // the token whose angles c, s and n hold
    int gains_of = -1;      // the end of the role whose gains g1 and g2 hold
    int stage = 0;
    while (out.item < items) {
        if (pairs > 0 && out.unit != turned) {
            turned = out.unit;
            const uint32_t tokens = static_cast<uint32_t>(A.tokens), b = out.unit / tokens;
            const int32_t *pos =
                A.positions + (b * A.pos_batch + (out.unit - b * tokens)) * A.axes;
            __syncwarp();
            for (int p = lane; p < pairs; p += 32) {
                const int64_t at = pos[p < A.axis_pairs ? 0 : 1];
                const uint64_t angle = static_cast<uint64_t>(at) * A.phases[p];
                float sn, cs;
                sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &sn, &cs);
                cos_s[p] = cs * A.magnitude;
                sin_s[p] = sn * (A.inverse ? -A.magnitude : A.magnitude);
            }
            __syncwarp();
            if (rot) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    c[i] = *reinterpret_cast<const float2 *>(cos_s + sl * E + 2 * i);
                    s[i] = *reinterpret_cast<const float2 *>(sin_s + sl * E + 2 * i);
                    n[i] = make_float2(-s[i].x, -s[i].y);
                }
            }
        }
        if constexpr (NORM) {
            if (out.end != gains_of) {
                gains_of = out.end;
                const float *g = gain_s + (out.pass >= pq ? A.d + E : 0);
                if (has1) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        g1[i] = *reinterpret_cast<const float2 *>(g + o1 + 2 * i);
                        g2[i] = *reinterpret_cast<const float2 *>(g + o2 + 2 * i);
                    }
                }
            }
        }
        const bool live = out.h < out.heads && has1;
        float2 x[E / 2], y[E / 2];
        cp_async_wait<kRopeStages - 2>();
        {
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (live) a = ld_shared_v4(ring + stage * kStage);
            if (live && has2) b = ld_shared_v4(ring + stage * kStage + kVec);
            W::get(a, x);
            W::get(b, y);
        }
        if constexpr (NORM) {
            if (A.layer) {
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < E / 2; ++i) sum = fadd2(sum, fadd2(x[i], y[i]));
                const float mean = lanes_sum(sum.x + sum.y, L) * inv_d;
                const float2 m1 = has1 ? make_float2(-mean, -mean) : make_float2(0.f, 0.f);
                const float2 m2 = has2 ? m1 : make_float2(0.f, 0.f);  // no channel, no mean
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    x[i] = fadd2(x[i], m1);
                    y[i] = fadd2(y[i], m2);
                }
            }
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) sq = ffma2(x[i], x[i], ffma2(y[i], y[i], sq));
            const float rs = rsqrtf(lanes_sum(sq.x + sq.y, L) * inv_d + A.eps);
            const float2 rr = make_float2(rs, rs);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                x[i] = fmul2(x[i], fmul2(rr, g1[i]));
                y[i] = fmul2(y[i], fmul2(rr, g2[i]));
            }
        }
        if (rot) {
            if constexpr (INTER) {
                // pairs are neighbours: gather (x1, x1'), (x2, x2') and spread again
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    float2 u, v;
                    turn(make_float2(x[2 * i].x, x[2 * i + 1].x),
                         make_float2(x[2 * i].y, x[2 * i + 1].y), c[i], s[i], n[i], u, v);
                    x[2 * i] = make_float2(u.x, v.x), x[2 * i + 1] = make_float2(u.y, v.y);
                    turn(make_float2(y[2 * i].x, y[2 * i + 1].x),
                         make_float2(y[2 * i].y, y[2 * i + 1].y), c[E / 4 + i], s[E / 4 + i],
                         n[E / 4 + i], u, v);
                    y[2 * i] = make_float2(u.x, v.x), y[2 * i + 1] = make_float2(u.y, v.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    float2 u, v;
                    turn(x[i], y[i], c[i], s[i], n[i], u, v);
                    x[i] = u, y[i] = v;
                }
            }
        }
        if (live) {
            *reinterpret_cast<uint4 *>(out.p + o1) = W::put(x);
            if (has2) *reinterpret_cast<uint4 *>(out.p + o2) = W::put(y);
        }
        // the slot that this pass's predecessor was read from is free
        ask(stage == 0 ? kRopeStages - 1 : stage - 1);
        stage = stage + 1 == kRopeStages ? 0 : stage + 1;
        next(out, A.dst);
    }
}

template <typename T>
cudaError_t rope_launch_token(RopeArgs A, cudaStream_t stream) {
    constexpr int E = Wide<T>::E;
    const int slots = A.rotary / (2 * E) + (A.d - A.rotary + 2 * E - 1) / (2 * E);
    A.lanes = 1;
    while (A.lanes < slots) A.lanes *= 2;
    const int HP = 32 / A.lanes;
    const int64_t passes = (A.heads[0] + HP - 1) / HP + (A.heads[1] + HP - 1) / HP;
    const bool norm = A.norm != 0;
    const int64_t most = static_cast<int64_t>(rope_ctas_per_sm(norm)) * sm_count();
    // warps per token: one, unless that leaves fewer than two items per warp
    const int64_t want = (2 * most * kRopeWarps + A.units - 1) / A.units;
    A.wpt = static_cast<int>(want < passes ? want : passes);
    const int64_t ctas = (A.units * A.wpt + kRopeWarps - 1) / kRopeWarps;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    const size_t smem = kRopeStages * 2 * 32 * kRopeWarps * 16 +
                        static_cast<size_t>(kRopeWarps) * A.rotary * sizeof(float) +
                        (norm ? 2 * (A.d + E) * sizeof(float) : 0);
    void (*kernel)(const RopeArgs) =
        A.interleaved ? (norm ? rope_token_kernel<T, true, true> : rope_token_kernel<T, true, false>)
                      : (norm ? rope_token_kernel<T, false, true> : rope_token_kernel<T, false, false>);
    return launch_pdl(kernel, grid, dim3(32 * kRopeWarps), smem, stream, A);
}

template <typename T, bool INTER, bool NORM>
__global__ void __launch_bounds__(32 * kRopeWarps, rope_ctas_per_sm(NORM))
rope_run_kernel(const __grid_constant__ RopeArgs A) {
    using W = Wide<T>;
    constexpr int E = W::E;  // elements per vector: a lane holds 2 E, E pairs
    extern __shared__ __align__(128) float rope_smem[];
    const int pairs = A.rotary / 2, heads = A.heads[0] + A.heads[1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // shared memory: the ring [stage][vector][thread] of 16 bytes, the gains of
    // both roles in fp32, each warp's cosines and sines [token][pair]
    constexpr int kRingFloats = kRopeStages * 2 * 32 * kRopeWarps * 4;
    float *gain_s = rope_smem + kRingFloats;
    const int gain_row = A.d + E;  // E zeros behind each, for lanes without a second vector
    float *cos_s = gain_s + (NORM ? 2 * gain_row : 0) + warp * 2 * A.run_tokens * pairs;
    float *sin_s = cos_s + A.run_tokens * pairs;
    const uint32_t ring = smem_u32(rope_smem) + threadIdx.x * 16;
    constexpr uint32_t kVec = 32 * kRopeWarps * 16, kStage = 2 * kVec;

    const int L = A.lanes, HP = 32 / L;
    const int group = lane / L, sl = lane & (L - 1);
    // This lane's slot: the element offsets of its two vectors. Slots below
    // srot turn; the others hold two neighbouring vectors of the part that
    // passes (the last of them may have one).
    const int srot = A.rotary / (2 * E);
    const bool rot = sl < srot;
    const int o1 = rot && !INTER ? sl * E : (rot ? 2 * sl * E : A.rotary + 2 * (sl - srot) * E);
    const int o2 = rot && !INTER ? pairs + sl * E : o1 + E;
    const bool has1 = o1 < A.d, has2 = o2 < A.d;

    const int64_t rows = A.units * heads, runs = (rows + A.run_rows - 1) / A.run_rows;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRopeWarps;
    const int64_t run0 = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
    const float inv_heads = 1.f / static_cast<float>(heads), inv_d = 1.f / static_cast<float>(A.d);

    // A run: its first token and that token's batch and position, the rows of
    // the token that lie before it, its length.
    struct Run {
        int64_t id, unit;
        uint32_t b, t;
        int skip, rows;
    };
    const auto enter = [&](Run &r, int64_t id) {
        r.id = id;
        if (id >= runs) return;
        const int64_t row = id * A.run_rows;
        r.unit = row / heads;
        r.skip = static_cast<int>(row - r.unit * heads);
        r.rows = static_cast<int>(rows - row < A.run_rows ? rows - row : A.run_rows);
        r.b = A.units == A.tokens ? 0 : static_cast<uint32_t>(r.unit / A.tokens);
        r.t = static_cast<uint32_t>(r.unit - r.b * A.tokens);
    };
    // Row i of the run: its token within the run, its role and its first channel.
    // (The products of small numbers below cannot reach the next integer.)
    const auto locate = [&](const Run &r, int i, const RopeView *views, int &tok, int &role) -> T * {
        const int at = r.skip + i;
        tok = static_cast<int>((static_cast<float>(at) + 0.5f) * inv_heads);
        int h = at - tok * heads;
        role = h >= A.heads[0] ? 1 : 0;
        h -= role ? A.heads[0] : 0;
        uint32_t b = r.b, t = r.t + tok;
        while (t >= static_cast<uint32_t>(A.tokens)) {
            t -= static_cast<uint32_t>(A.tokens);
            ++b;
        }
        const RopeView &v = views[role];
        return static_cast<T *>(v.data) + b * v.batch_stride + t * v.token_stride + h * v.head_stride;
    };

    griddep_wait();
    Run in, out;
    enter(in, run0);
    int in_row = group;  // of the run `in`, the next to be asked for
    const auto ask = [&](int stage) {  // the next pass's vectors into the ring
        if (in.id < runs) {
            if (in_row < in.rows && has1) {
                int tok, role;
                const T *src = locate(in, in_row, A.src, tok, role);
                cp_async16(ring + stage * kStage, src + o1);
                if (has2) cp_async16(ring + stage * kStage + kVec, src + o2);
            }
            in_row += HP;
            if (in_row - group >= in.rows) {
                enter(in, in.id + stride);
                in_row = group;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kRopeStages - 1; ++s) ask(s);
    if constexpr (NORM) {
        for (int i = threadIdx.x; i < 2 * gain_row; i += 32 * kRopeWarps) {
            const int role = i >= gain_row ? 1 : 0, e = i - role * gain_row;
            const void *g = A.gain[role];
            gain_s[i] = e >= A.d       ? 0.f
                        : g == nullptr ? 1.f
                                       : (A.gain_f32 ? static_cast<const float *>(g)[e]
                                                     : to_f32(static_cast<const T *>(g)[e]));
        }
        __syncthreads();
    }
    if (run0 >= runs) return;

    const auto turn = [&](float2 v1, float2 v2, float2 c, float2 s, float2 &y1, float2 &y2) {
        y1 = ffma2(v2, make_float2(-s.x, -s.y), fmul2(v1, c));
        y2 = ffma2(v1, s, fmul2(v2, c));
    };
    int stage = 0;
    for (int64_t id = run0; id < runs; id += stride) {
        enter(out, id);
        if (pairs > 0) {  // the angles of the run's tokens
            const int tokens = static_cast<int>((static_cast<float>(out.skip + out.rows - 1) + 0.5f) * inv_heads) + 1;
            __syncwarp();
            for (int i = lane; i < tokens * pairs; i += 32) {
                const int tok = i / pairs, p = i - tok * pairs;
                uint32_t b = out.b, t = out.t + tok;
                while (t >= static_cast<uint32_t>(A.tokens)) {
                    t -= static_cast<uint32_t>(A.tokens);
                    ++b;
                }
                const int64_t pos =
                    A.positions[(b * A.pos_batch + t) * A.axes + (p < A.axis_pairs ? 0 : 1)];
                const uint64_t angle = static_cast<uint64_t>(pos) * A.phases[p];
                float sn, cs;
                sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &sn, &cs);
                cos_s[i] = cs * A.magnitude;
                sin_s[i] = sn * (A.inverse ? -A.magnitude : A.magnitude);
            }
            __syncwarp();
        }
        for (int first = 0; first < out.rows; first += HP) {
            const int i = first + group;
            const bool live = i < out.rows && has1;
            int tok = 0, role = 0;
            T *dst = locate(out, live ? i : first, A.dst, tok, role);
            float2 x[E / 2], y[E / 2];
            cp_async_wait<kRopeStages - 2>();
            {
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (live) a = ld_shared_v4(ring + stage * kStage);
                if (live && has2) b = ld_shared_v4(ring + stage * kStage + kVec);
                W::get(a, x);
                W::get(b, y);
            }
            if constexpr (NORM) {
                if (A.layer) {
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) sum = fadd2(sum, fadd2(x[e], y[e]));
                    const float mean = lanes_sum(sum.x + sum.y, L) * inv_d;
                    const float2 m1 = has1 ? make_float2(-mean, -mean) : make_float2(0.f, 0.f);
                    const float2 m2 = has2 ? m1 : make_float2(0.f, 0.f);  // no channel, no mean
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        x[e] = fadd2(x[e], m1);
                        y[e] = fadd2(y[e], m2);
                    }
                }
                float2 sq = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) sq = ffma2(x[e], x[e], ffma2(y[e], y[e], sq));
                const float rs = rsqrtf(lanes_sum(sq.x + sq.y, L) * inv_d + A.eps);
                const float2 rr = make_float2(rs, rs);
                if (has1) {
                    const float *g = gain_s + role * gain_row;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        x[e] = fmul2(x[e], fmul2(rr, *reinterpret_cast<const float2 *>(g + o1 + 2 * e)));
                        y[e] = fmul2(y[e], fmul2(rr, *reinterpret_cast<const float2 *>(g + o2 + 2 * e)));
                    }
                }
            }
            if (rot) {
                const float *cp = cos_s + tok * pairs + sl * E, *sp = sin_s + tok * pairs + sl * E;
                float2 c[E / 2], s[E / 2];
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    c[e] = *reinterpret_cast<const float2 *>(cp + 2 * e);
                    s[e] = *reinterpret_cast<const float2 *>(sp + 2 * e);
                }
                if constexpr (INTER) {
                    // pairs are neighbours: gather (x1, x1'), (x2, x2') and spread again
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        float2 u, v;
                        turn(make_float2(x[2 * e].x, x[2 * e + 1].x),
                             make_float2(x[2 * e].y, x[2 * e + 1].y), c[e], s[e], u, v);
                        x[2 * e] = make_float2(u.x, v.x), x[2 * e + 1] = make_float2(u.y, v.y);
                        turn(make_float2(y[2 * e].x, y[2 * e + 1].x),
                             make_float2(y[2 * e].y, y[2 * e + 1].y), c[E / 4 + e], s[E / 4 + e], u, v);
                        y[2 * e] = make_float2(u.x, v.x), y[2 * e + 1] = make_float2(u.y, v.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        float2 u, v;
                        turn(x[e], y[e], c[e], s[e], u, v);
                        x[e] = u, y[e] = v;
                    }
                }
            }
            if (live) {
                *reinterpret_cast<uint4 *>(dst + o1) = W::put(x);
                if (has2) *reinterpret_cast<uint4 *>(dst + o2) = W::put(y);
            }
            // the slot that this pass's predecessor was read from is free
            ask(stage == 0 ? kRopeStages - 1 : stage - 1);
            stage = stage + 1 == kRopeStages ? 0 : stage + 1;
        }
    }
}

template <typename T>
cudaError_t rope_launch_run(RopeArgs A, cudaStream_t stream) {
    constexpr int E = Wide<T>::E;
    const int slots = A.rotary / (2 * E) + (A.d - A.rotary + 2 * E - 1) / (2 * E);
    A.lanes = 1;
    while (A.lanes < slots) A.lanes *= 2;
    const bool norm = A.norm != 0;
    const int HP = 32 / A.lanes, heads = A.heads[0] + A.heads[1], pairs = A.rotary / 2;
    const int64_t rows = A.units * heads;
    const int64_t most = static_cast<int64_t>(rope_ctas_per_sm(norm)) * sm_count();
    // Runs of as many passes as make one run per warp with norms, three without
    // (12 heads of 64: 22.1 us with one, 23.4 with three; without norms, fp32, 20.3
    // and 18.6), of 16 passes at most, and of no more tokens than 1024 pairs of
    // angles (8 KB per warp) serve.
    const int64_t round = (norm ? 1 : 3) * most * kRopeWarps * HP;
    int64_t passes = (rows + round - 1) / round;
    passes = passes > 16 ? 16 : passes;
    const auto tokens_of = [&](int64_t p) { return static_cast<int>((p * HP + heads - 2) / heads + 1); };
    while (passes > 1 && tokens_of(passes) * pairs > 1024) --passes;
    A.run_rows = static_cast<int>(passes * HP);
    A.run_tokens = tokens_of(passes);
    const int64_t runs = (rows + A.run_rows - 1) / A.run_rows;
    const int64_t ctas = (runs + kRopeWarps - 1) / kRopeWarps;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    const size_t smem = kRopeStages * 2 * 32 * kRopeWarps * 16 +
                        (norm ? 2 * (A.d + E) * sizeof(float) : 0) +
                        static_cast<size_t>(kRopeWarps) * 2 * A.run_tokens * pairs * sizeof(float);
    void (*kernel)(const RopeArgs) =
        A.interleaved ? (norm ? rope_run_kernel<T, true, true> : rope_run_kernel<T, true, false>)
                      : (norm ? rope_run_kernel<T, false, true> : rope_run_kernel<T, false, false>);
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(kernel, grid, dim3(32 * kRopeWarps), smem, stream, A);
}

// 16-byte vectors throughout: by token where its heads fill four passes or more
// (40 heads of 128: 56 us by token, 70 in runs), else in runs (12 heads of 64: 32
// and 22 us).
template <typename T>
cudaError_t rope_launch_wide(const RopeArgs &A, cudaStream_t stream) {
    constexpr int E = Wide<T>::E;
    const int slots = A.rotary / (2 * E) + (A.d - A.rotary + 2 * E - 1) / (2 * E);
    return (A.heads[0] + A.heads[1]) * slots >= 4 * 32 ? rope_launch_token<T>(A, stream)
                                                       : rope_launch_run<T>(A, stream);
}

template <typename T, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_any_kernel(const RopeArgs A) {
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
cudaError_t rope_launch_any(RopeArgs A, cudaStream_t stream) {
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
        A.interleaved ? (norm ? rope_any_kernel<T, V, true, true> : rope_any_kernel<T, V, true, false>)
                      : (norm ? rope_any_kernel<T, V, false, true> : rope_any_kernel<T, V, false, false>);
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
    if (bits % Wide<T>::E == 0) return rope_launch_wide<T>(A, stream);
    if constexpr (sizeof(T) == 2)
        if (bits % 4 == 0) return rope_launch_any<T, 4>(A, stream);
    if (bits % 2 == 0) return rope_launch_any<T, 2>(A, stream);
    return rope_launch_any<T, 1>(A, stream);
}

}  // namespace
}  // namespace vta
