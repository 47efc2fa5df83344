// packed_attn.cuh -- softmax attention over packed sequences of different
// lengths on sm_103a, causal or not, with grouped heads: the kernel template,
// instantiated for 16-bit types and head sizes by packed_attn_*.cu.
//
//   out_i = sum_j softmax_j(scale q_i . k_j) v_j   over the keys j that
//   query i of its sequence sees (all nk; causal: j <= i + nk - nq).
//
// Tiles. The g query heads that share a key/value head sit side by side in
// memory, so a tile of 128 rows holds TQ = 128 / g tokens x g heads (one TMA
// box), and every key tile is read once for all of them. A CTA works
// on two such tiles at a time, each with its own softmax warpgroup, one thread
// per row, and its own issuing thread for the tensor-core products, so that one
// tile's softmax and waits run under the other's products (with one issuing
// thread for both the tensor pipe stood still during its waits: 501 us on long
// causal prompts, 487 with two, when the rest was as slow as then).
//
// Measured (device time): causal prompts of 500 to 8192 tokens, 32 over 8 heads
// of 128, 385 us, 1520 TFLOP/s, 1700 once items are long, where the tensor pipe
// waits for little but the softmax's exponentials; images of 196 to 3136
// patches, 6 heads of 64, 191 us, 870 TFLOP/s (half the product per
// exponential); a token each against 32 caches of 110 to 7927 keys, 52 us,
// 4.9 TB/s (6.4 with 7680 keys each: 17 us of start, end and join).
//
// Three kinds of work:
//   whole (kWhole): two neighbouring tiles of one sequence and key/value head,
//     sharing every key tile, all keys;
//   shared (kShared; too few items to fill the GPU): the same against a run of
//     the key tiles;
//   twins (kTwins; sequences of one or two tiles on average): as whole, but a
//     last item of one tile and one key tile takes two heads, a tile each, whose
//     chains (load, S, softmax, P V, rows out: 3.9 us) then run side by side.
//     (Sequences of 40 tokens, 12 over 4 heads of 80: 41 us, 65 as whole. In one
//     kernel with the long ones it cost those: images 215 us, 191 without.)
//   alternate (kAlternate; rows for one tile at most): one tile against a run
//     of key tiles, the warpgroups taking every other key tile of it.
// In shared and alternate a CTA's runs are its equal share of all key tiles (and of
// what starting an item costs), the unnormalised outputs go to the caller's
// workspace in fp32, and packed_combine_kernel joins them.
//
// Per key tile (128 keys, or 96 for D = 64) and tile: S = Q K^T into tensor
// memory (fp32), the row's scores into registers, p = 2^(scale log2e (s - m))
// in fp32, summed in fp32 and rounded to the 16-bit type over the scores, where
// the product P V reads its A operand, at most half a step off (2^-8 for bf16,
// 2^-11 for fp16 of itself), the precision that the values have. The reference
// m is the row's maximum over its first key tile; later tiles form no maximum
// (it took 300 of the 1150 cycles between S and P): a tile whose sum passes 2^8
// moves the reference by log2 of it, which is within 2^7 of its maximum, for
// the next tile, O being rescaled then; only where the sum says that a p may
// have left the type's range (2^15 for fp16; 2^60 for bf16) the tile is done
// again with its own maximum. O stays in tensor memory.
//
// Tensor memory (512 columns). D = 128: S of the tiles at 0 and 128 (P over S),
// O at 256 and 384; the next S waits for P V. D = 64: O at 0 and 64 and two
// slots of S per tile, for which key tiles have 96 keys: S of the tile after
// next is formed behind P V, and a softmax finds its S ready. (128 keys in one
// slot with P beside it took 2400 cycles per 128 keys and pair of tiles.)
//
// Keys past a sequence's end and, in the tile on the diagonal, past a row's
// last key are masked in registers whatever their scores are; V rows past the
// end are zeroed in shared memory before the product, so that nothing behind a
// sequence (NaN included) reaches an output.
#pragma once
#include "vta_internal.h"
#include "sm103_ptx.cuh"

#include <type_traits>

namespace vta {
namespace {

constexpr int kPaThreads = 384;  // two softmax warpgroups, then loads, products (2), schedule
constexpr int kPaRegsControl = 80, kPaRegsSoftmax = 208, kPaRegsLaunch = 168;
static_assert(128 * kPaRegsControl + 256 * kPaRegsSoftmax <= kPaThreads * kPaRegsLaunch, "register split");
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpSched = 11;  // kWarpMma + tile
enum { kWhole = 0, kShared = 1, kAlternate = 2, kTwins = 3 };
constexpr int kWorkSlots = 3;
// What starting an item costs beside its key tiles, in key tiles.
// Single tokens against 32 caches of 110 to 7927 keys: 66 us with nothing for
// it, 55 with one, 56 with two or three; a prompt's piece 92, 92 (two), 93 (six).
template <int KIND>
constexpr int kPaStart = KIND == kAlternate ? 1 : 2;
constexpr float kPaMove = 256.f;  // a tile's sum that moves the reference
// ... and one that has the tile done again: every p is below its tile's sum, so
// p stays finite in the type, and its products and sums in fp32
template <typename T>
constexpr float kPaRedo = std::is_same<T, __half>::value ? 0x1p15f : 0x1p60f;
constexpr int kSlab = 128 * 128;  // 128 rows x 64 16-bit channels

template <int D>
struct PaGeo {
    static constexpr int KEYS = D == 64 ? 96 : 128;  // per key tile
    static constexpr int SLABS = D / 64;
    static constexpr int Q_TILE = SLABS * kSlab;
    static constexpr int KV_SLAB = KEYS * 128, TILE = SLABS * KV_SLAB;  // one K or V tile
    static constexpr int STAGES = D == 128 ? 5 : 15;  // K and V tiles in flight
    static constexpr int SMEM = 2 * Q_TILE + STAGES * TILE;
    static constexpr int SLOTS = D == 64 ? 2 : 1;  // S of a tile in tensor memory
    static constexpr uint32_t O_COL = D == 64 ? 0 : 256, S_COL = D == 64 ? 128 : 0;
};

// The waits of the warps that load, issue and schedule. Out of line (but for the
// first try) for D = 128, where some twenty loops in line make the code of a tile
// outgrow the instruction cache (long causal prompts 396 us, 385 out of line); in
// line for D = 64, whose waits are more and mostly not over at the first try
// (images 188 us, 196 out of line).
struct PaWait {
    unsigned *status;
    volatile int *abort;
};
__device__ __noinline__ bool pa_wait_on(uint64_t *bar, uint32_t parity, unsigned code, unsigned *status,
                                        volatile int *abort) {
    return mbar_wait(bar, parity, WaitCtl{status, kDefaultWaitNs}, code, abort, false);
}
template <int D>
__device__ __forceinline__ bool pa_wait(uint64_t *bar, uint32_t parity, unsigned code, const PaWait &w) {
    if constexpr (D == 64) return mbar_wait(bar, parity, WaitCtl{w.status, kDefaultWaitNs}, code, w.abort, false);
    return mbar_try_wait(bar, parity) || pa_wait_on(bar, parity, code, w.status, w.abort);
}

// In line altogether: for the softmax warps, which hold too much for a call.
__device__ __forceinline__ bool pa_wait_in(uint64_t *bar, uint32_t parity, unsigned code, const PaWait &w) {
    return mbar_wait(bar, parity, WaitCtl{w.status, kDefaultWaitNs}, code, w.abort, false);
}

// One unit of work, as the schedule warp hands it to the others.
struct PaWork {
    int q_tok;  // first token of the first tile (of all tokens)
    int toks;   // tokens from there to the end of the sequence
    int head;   // key/value head; -1: no more work
    int k_row, nk;  // the sequence's keys
    int lim0;   // keys that the first token sees (causal; may be <= 0)
    int lo, n;  // key tiles lo .. lo + n - 1
    int n0, n1; // of them, how many the two tiles need (alternate: not used)
    int twin;   // twins: 1: tile x is the same tokens of head + x, its key tile the ring's x-th
    int slot;   // shared, alternate: where the unnormalised output goes
};

struct PaBars {
    uint64_t q_full[2], q_empty[2];  // of a tile; alternate: of every other item
    uint64_t kv_full[15], kv_empty[15];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // tile, slot
    uint64_t o_empty[2];
    uint64_t w_full[kWorkSlots], w_empty[kWorkSlots];
    uint64_t turn[2], fin[2];
};

struct PaSeq {
    int q0, nq, k0, nk;
};

// Sequence b's rows, clamped into the tensors; *bad if they were not.
__device__ __forceinline__ PaSeq pa_seq(const PackedAttnArgs &P, int b, bool *bad) {
    PaSeq s;
    const int q0 = P.cu_q[b], q1 = P.cu_q[b + 1], k0 = P.cu_k[b], k1 = P.cu_k[b + 1];
    s.q0 = min(max(q0, 0), P.total_q);
    s.nq = min(max(q1, s.q0), P.total_q) - s.q0;
    s.k0 = min(max(k0, 0), P.total_k);
    s.nk = min(max(k1, s.k0), P.total_k) - s.k0;
    *bad = *bad || q0 != s.q0 || q1 != s.q0 + s.nq || k0 != s.k0 || k1 != s.k0 + s.nk;
    if (P.k_lens != nullptr) {
        const int n = P.k_lens[b];
        *bad = *bad || n < 0 || n > s.nk;
        s.nk = min(max(n, 0), s.nk);
    }
    return s;
}

// Key tiles that the tokens up to `last` of a sequence need (at least one, so
// that rows without keys are written too).
template <int KEYS>
__device__ __forceinline__ int pa_tiles(const PackedAttnArgs &P, const PaSeq &s, int last) {
    const int vis = P.causal ? min(s.nk, last + 1 + s.nk - s.nq) : s.nk;
    return vis <= KEYS ? 1 : (vis + KEYS - 1) / KEYS;
}

__device__ __forceinline__ int warp_sum(int v) {
    return __reduce_add_sync(~0u, v);
}
__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
template <typename V>
__device__ __forceinline__ V warp_scan(V v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

template <typename T>
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pa_pack<__nv_bfloat16>(float lo, float hi) {
    return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pa_pack<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One lane of a converged warp, always the same. Products issued under it keep
// their descriptors in uniform registers; issued by a lane of its own branch they
// take several times the instructions, and the softmax warps beside them leave
// few slots for those: 1660 instead of 1100 cycles for the 16 products of a key
// tile (1024 at full rate), measured with two softmax warps per scheduler.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// The products with descriptors as (low, high) words: only the low one, which
// holds the address, changes.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: fp32 D, A and B both bf16 or both fp16.
template <typename T>
__device__ __forceinline__ uint32_t pa_idesc(int N, bool b_mn_major) {
    const uint32_t f = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Writes 64 bytes of each of a warp's rows, held one row per thread in v. Four
// neighbouring threads exchange their 16-byte units first, so that an
// instruction writes 64 bytes of each of 8 rows and not 16 of each of 32 (which
// took 62 cycles of the SM's store path each, 4000 for a tile of 128 x 128).
// rows: the four threads' rows; at: the byte offset of the 64; bit i of rows_ok:
// row i is to be written; unit_ok: this thread's unit (lane & 3) is.
__device__ __forceinline__ void store_rows(uint32_t (&v)[16], char *const (&rows)[4], int at,
                                           unsigned rows_ok, bool unit_ok, int lane) {
    const int j = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // 4 x 4 transpose in two rounds
        const int d = r == 0 ? 1 : 2;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int lo = r == 0 ? 2 * p : p, up = lo + d;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = v[4 * lo + k], b = v[4 * up + k];
                const uint32_t got = __shfl_xor_sync(~0u, (j & d) ? a : b, d);
                if (j & d)
                    v[4 * lo + k] = got;
                else
                    v[4 * up + k] = got;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (unit_ok && ((rows_ok >> i) & 1u))
            *reinterpret_cast<uint4 *>(rows[i] + at + 16 * j) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// ------------------------------------------------------------- schedule

// Hands PaWork entries to the other roles through a ring in shared memory.
template <int D>
struct PaRing {
    PaWork *slots;
    uint64_t *full, *empty;
    PaWait wc;
    int n = 0;
    // Called by the whole warp with the same values; false: give up.
    __device__ __forceinline__ bool put(const PaWork &w, int lane) {
        const int s = n % kWorkSlots, use = n / kWorkSlots;
        ++n;
        if (!__all_sync(~0u, pa_wait<D>(&empty[s], (use & 1) ^ 1, kStatusTimeoutSync, wc)))
            return false;
        if (lane == 0) {
            slots[s] = w;
            mbar_arrive(&full[s]);
        }
        __syncwarp();
        return true;
    }
};

// Whole items, the costliest first (by key tiles, in at most 64 levels), dealt
// to the CTAs round by round, every other round backwards.
template <int KEYS, int D, bool TWINS>
__device__ __forceinline__ void pa_schedule_items(const PackedAttnArgs &P, PaRing<D> ring, int lane,
                                                  int most_tiles) {
    const int TT = 2 * P.tile_tokens;
    int shift = 0;
    while (((most_tiles - 1) >> shift) >= 64) ++shift;
    long long base = 0;  // items before this level and chunk
    int round = 0;
    const auto target = [&]() {
        const int c = (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        return static_cast<long long>(round) * gridDim.x + c;
    };
    long long want = target();
    // items of s with at most (q + 1) << shift key tiles
    const auto upto = [&](const PaSeq &s, int q) -> int {
        if (q < 0) return 0;
        const int nb = (s.nq + TT - 1) / TT;
        const long long keys = (static_cast<long long>(q + 1) << shift) * KEYS;
        if (s.nk <= keys) return nb;
        if (!P.causal) return 0;
        const long long t = (keys - (s.nk - s.nq)) / TT;
        return static_cast<int>(t < 0 ? 0 : t > nb ? nb : t);
    };
    bool bad = false;
    PaSeq s{0, 0, 0, 0};
    bool alive = true;
    for (int q = (most_tiles - 1) >> shift; alive && q >= 0; --q) {
        for (int b0 = 0; alive && b0 < P.batch; b0 += 32) {
            if (P.batch > 32 || q == (most_tiles - 1) >> shift) {
                s = PaSeq{0, 0, 0, 0};
                if (b0 + lane < P.batch) s = pa_seq(P, b0 + lane, &bad);
            }
            const int high = upto(s, q), mine = high - upto(s, q - 1);
            // a last item of one tile and one key tile takes its heads by twos
            const bool single = TWINS && mine > 0 && s.nk <= KEYS &&
                                s.nq - (s.nq - 1) / TT * TT <= P.tile_tokens;
            const long long count = static_cast<long long>(mine) * P.heads_kv - (single ? P.heads_kv / 2 : 0);
            const long long sum = warp_scan(count, lane);
            const long long all = __shfl_sync(~0u, sum, 31);
            while (alive && want < base + all) {
                const uint32_t after = __ballot_sync(~0u, base + sum > want);
                const int src = __ffs(after) - 1;
                const long long first = base + sum - count;
                int r = static_cast<int>(want - __shfl_sync(~0u, first, src));
                const bool by_twos = __shfl_sync(~0u, single ? 1 : 0, src) != 0;
                int twin = 0;
                if (by_twos) {
                    if (2 * r < P.heads_kv) {
                        r *= 2;
                        twin = r + 1 < P.heads_kv ? 1 : 0;
                    } else {
                        r += P.heads_kv / 2;  // as if the last item had come head by head
                    }
                }
                PaSeq q_seq{__shfl_sync(~0u, s.q0, src), __shfl_sync(~0u, s.nq, src),
                            __shfl_sync(~0u, s.k0, src), __shfl_sync(~0u, s.nk, src)};
                const int t = __shfl_sync(~0u, high, src) - 1 - r / P.heads_kv;
                const int tok = t * TT;
                PaWork w;
                w.q_tok = q_seq.q0 + tok;
                w.toks = q_seq.nq - tok;
                w.head = r % P.heads_kv;
                w.k_row = q_seq.k0;
                w.nk = q_seq.nk;
                w.lim0 = tok + 1 + q_seq.nk - q_seq.nq;
                w.lo = 0;
                w.n0 = pa_tiles<KEYS>(P, q_seq, min(q_seq.nq, tok + P.tile_tokens) - 1);
                w.n1 = w.toks > P.tile_tokens ? pa_tiles<KEYS>(P, q_seq, min(q_seq.nq, tok + TT) - 1) : 0;
                w.n = max(w.n0, w.n1);
                w.slot = 0;
                if (TWINS) {
                    w.twin = twin;
                    if (twin) w.n = 2, w.n1 = 1;
                }
                alive = ring.put(w, lane);
                ++round;
                want = target();
            }
            base += all;
        }
    }
    if (alive) {
        PaWork w{};
        w.head = -1;
        ring.put(w, lane);
    }
}

// The CTAs' shares of `all` units: the first `more` CTAs have size + 1 units, the
// others size. No more CTAs than units, so that an item's pieces lie on
// neighbouring ones. Divisions in 32 bits where the numbers allow it (a division
// in 64 bits takes some 500 cycles here, in front of everything else).
struct PaShares {
    int ctas, more;
    long long size;
    __device__ __forceinline__ PaShares(long long all, int grid) {
        ctas = static_cast<int>(all < grid ? all : grid);
        size = divide(all, ctas > 0 ? ctas : 1);
        more = static_cast<int>(all - size * ctas);
    }
    static __device__ __forceinline__ long long divide(long long a, long long b) {
        if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
        return a / b;
    }
    __device__ __forceinline__ long long begin(int cta) const { return size * cta + min(cta, more); }
    __device__ __forceinline__ int cta_of(long long unit) const {
        const long long split = (size + 1) * more;
        return static_cast<int>(unit < split ? divide(unit, size + 1) : more + divide(unit - split, size));
    }
};

// Units (key tiles of one item, and kPaStart before them) and items of a
// sequence; an item is TT tokens of one key/value head.
template <int KEYS, int START>
__device__ __forceinline__ void pa_units(const PackedAttnArgs &P, const PaSeq &s, int TT,
                                         long long *units, int *items) {
    long long u = 0;
    const int nt = (s.nq + TT - 1) / TT;
    if (!P.causal || nt <= 1)
        u = static_cast<long long>(nt) * (nt ? pa_tiles<KEYS>(P, s, s.nq - 1) + START : 0);
    else
        for (int t = 0; t < nt; ++t) u += pa_tiles<KEYS>(P, s, min(s.nq, (t + 1) * TT) - 1) + START;
    *units = u * P.heads_kv;
    *items = nt * P.heads_kv;
}

// Shared and alternate: this CTA's share [u0, u1) of all units, in (sequence,
// tokens, head, key tile) order. per: sequences per warp of the count before.
template <int KEYS, int D, int START>
__device__ __forceinline__ void pa_schedule_pieces(const PackedAttnArgs &P, PaRing<D> ring, int lane,
                                                   int TT, const long long *warp_units,
                                                   const int *warp_tiles, int per) {
    long long all = 0;
    int tiles_all = 0;
    for (int i = 0; i < kPaThreads / 32; ++i) {
        all += warp_units[i];
        tiles_all += warp_tiles[i];
    }
    PaWork none{};
    none.head = -1;
    int *header = static_cast<int *>(P.workspace);
    if (blockIdx.x == 0 && lane == 0)
        header[0] = tiles_all <= P.max_items ? tiles_all : 0;
    if (tiles_all > P.max_items) {  // overlapping sequences: the workspace is too small
        if (lane == 0) atomicOr(P.status, kStatusBadSequence);
        ring.put(none, lane);
        return;
    }
    const PaShares shares(all, gridDim.x);
    const bool mine = blockIdx.x < shares.ctas;
    const long long u0 = mine ? shares.begin(blockIdx.x) : 0, u1 = mine ? shares.begin(blockIdx.x + 1) : 0;
    // the sequence that holds unit u0
    long long base = 0;
    int item = 0, i = 0;
    while (i < kPaThreads / 32 - 1 && base + warp_units[i] <= u0) {
        base += warp_units[i];
        item += warp_tiles[i];
        ++i;
    }
    bool bad = false;
    int b = i * per;
    PaSeq s{0, 0, 0, 0};
    if (u0 < u1) {
        for (;; b += 32) {
            long long u = 0;
            int n = 0;
            s = PaSeq{0, 0, 0, 0};
            if (b + lane < P.batch) {
                s = pa_seq(P, b + lane, &bad);
                pa_units<KEYS, START>(P, s, TT, &u, &n);
            }
            const long long us = warp_scan(u, lane);
            const int ns = warp_scan(n, lane);
            const uint32_t after = __ballot_sync(~0u, base + us > u0);
            if (after != 0u) {
                const int src = __ffs(after) - 1;
                base += __shfl_sync(~0u, us - u, src);
                item += __shfl_sync(~0u, ns - n, src);
                b += src;
                s = PaSeq{__shfl_sync(~0u, s.q0, src), __shfl_sync(~0u, s.nq, src),
                          __shfl_sync(~0u, s.k0, src), __shfl_sync(~0u, s.nk, src)};
                break;
            }
            base += __shfl_sync(~0u, us, 31);
            item += __shfl_sync(~0u, ns, 31);
            if (b >= P.batch) {  // cannot happen: u0 < all
                ring.put(none, lane);
                return;
            }
        }
    }
    long long u = u0;
    int4 *meta = reinterpret_cast<int4 *>(header + 16);
    for (int t = 0; u < u1;) {
        const int last = min(s.nq, (t + 1) * TT) - 1;
        const int kt = pa_tiles<KEYS>(P, s, last);
        const long long span = static_cast<long long>(kt + START) * P.heads_kv;
        if (t * TT >= s.nq) {  // next sequence
            ++b;
            t = 0;
            if (b >= P.batch) break;
            s = pa_seq(P, b, &bad);
            continue;
        }
        if (base + span <= u) {
            base += span;
            item += P.heads_kv;
            ++t;
            continue;
        }
        const int h = static_cast<int>(PaShares::divide(u - base, kt + START));
        // the unit of the item's first key tile; the key tiles of this share
        const long long first = base + static_cast<long long>(h) * (kt + START) + START;
        const int lo = static_cast<int>(u > first ? u - first : 0);
        const int n = static_cast<int>(u1 - first < kt ? u1 - first : kt) - lo;
        if (n <= 0) break;  // the share ends before it
        const int tok = t * TT;
        PaWork w;
        w.q_tok = s.q0 + tok;
        w.toks = min(s.nq - tok, TT);
        w.head = h;
        w.k_row = s.k0;
        w.nk = s.nk;
        w.lim0 = tok + 1 + s.nk - s.nq;
        w.lo = lo;
        w.n = n;
        const int kt0 = pa_tiles<KEYS>(P, s, min(s.nq, tok + P.tile_tokens) - 1);
        w.n0 = min(max(kt0 - lo, 0), n);
        w.n1 = w.toks > P.tile_tokens ? n : 0;
        w.slot = item + h + blockIdx.x;
        if (lo == 0) {  // for the kernel that joins the pieces: the item, and its tokens' item
            if (lane == 0) {
                const int ctas = n == kt ? 1 : shares.cta_of(first + kt - 1) - static_cast<int>(blockIdx.x) + 1;
                meta[item + h] = make_int4(blockIdx.x, ctas | h << 16, w.q_tok, w.toks);
            }
            if (h == 0)
                for (int i = lane; i < w.toks; i += 32) P.ws_item[w.q_tok + i] = item;
        }
        if (!ring.put(w, lane)) return;
        u = first + lo + n;
    }
    ring.put(none, lane);
}

// ------------------------------------------------------------- the kernel

template <typename T, int D, int KIND>
__global__ void __launch_bounds__(kPaThreads, 1)
packed_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PackedAttnArgs P) {
    using G = PaGeo<D>;
    constexpr bool ALT = KIND == kAlternate, PIECES = KIND == kShared || KIND == kAlternate;
    constexpr bool TWINS = KIND == kTwins;
    constexpr int KEYS = G::KEYS, SLOTS = ALT ? 1 : G::SLOTS;
    extern __shared__ __align__(1024) uint8_t pa_smem[];
    __shared__ PaBars bars;
    __shared__ PaWork work[kWorkSlots];
    __shared__ long long warp_units[kPaThreads / 32];
    __shared__ int warp_tiles[kPaThreads / 32];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(~0u, tid >> 5, 0);  // the same in all lanes
    const PaWait wc{P.status, &abort_flag}, drain{P.status, nullptr};
    uint8_t *sQ = pa_smem, *sKV = pa_smem + 2 * G::Q_TILE;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], ALT ? 2 : 1);  // one arrival per warp that reads it
        }
        for (int i = 0; i < G::STAGES; ++i) {
            mbar_init(&bars.kv_full[i], 1);
            mbar_init(&bars.kv_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int s = 0; s < 2; ++s) {
                mbar_init(&bars.s_full[i][s], 1);
                mbar_init(&bars.p_full[i][s], 4);
                mbar_init(&bars.pv_done[i][s], 1);
            }
            mbar_init(&bars.o_empty[i], 4);
        }
        for (int i = 0; i < kWorkSlots; ++i) {
            mbar_init(&bars.w_full[i], 1);
            mbar_init(&bars.w_empty[i], 11);
        }
        mbar_init(&bars.turn[0], 1);
        mbar_init(&bars.turn[1], 1);
        mbar_init(&bars.fin[0], 1);
        mbar_init(&bars.fin[1], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base_s, 512);
    griddep_wait();
    griddep_launch_dependents();
    // Count before the roles part: units and tiles (pieces) or the most key
    // tiles of a sequence (whole items), each warp over its run of sequences.
    const int per = (P.batch + kPaThreads - 1) / kPaThreads * 32;
    const int TT = (ALT ? 1 : 2) * P.tile_tokens;
    {
        bool bad = false;
        long long units = 0;
        int tiles = 0;
        for (int i = 0; i < per; i += 32) {
            const int b = warp * per + i + lane;
            if (b >= P.batch) continue;
            const PaSeq s = pa_seq(P, b, &bad);
            if constexpr (PIECES) {
                long long u;
                int n;
                pa_units<KEYS, kPaStart<KIND>>(P, s, TT, &u, &n);
                units += u;
                tiles += n;
            } else {
                tiles = max(tiles, pa_tiles<KEYS>(P, s, s.nq - 1));
            }
        }
        if (bad) atomicOr(P.status, kStatusBadSequence);
        if constexpr (PIECES) {
            units = warp_sum64(units);
            tiles = warp_sum(tiles);
        } else {
            tiles = __reduce_max_sync(~0u, tiles);
        }
        if (lane == 0) {
            warp_units[warp] = units;
            warp_tiles[warp] = tiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;

    // The next entry of the schedule; every role walks the same list.
    int wn = 0;
    const auto next_work = [&](PaWork &w) -> bool {  // by the whole warp
        const int s = wn % kWorkSlots, use = wn / kWorkSlots;
        ++wn;
        if (!__all_sync(~0u, pa_wait_in(&bars.w_full[s], use & 1, kStatusTimeoutSync, wc)))
            return false;
        w = work[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.w_empty[s]);
        return w.head >= 0;
    };

    if (warp >= 8) {
        regs_dealloc<kPaRegsControl>();
        if (warp == kWarpSched) {
            PaRing<D> ring{work, bars.w_full, bars.w_empty, wc};
            if constexpr (PIECES) {
                pa_schedule_pieces<KEYS, D, kPaStart<KIND>>(P, ring, lane, TT, warp_units, warp_tiles, per);
            } else {
                int most = 1;
                for (int i = 0; i < kPaThreads / 32; ++i) most = max(most, warp_tiles[i]);
                pa_schedule_items<KEYS, D, TWINS>(P, ring, lane, most);
            }
        } else if (warp == kWarpLoad) {
            if (lane == 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_v);
            }
            int g = 0, q_loads[2] = {0, 0};  // K and V tiles, Q tiles
            bool ok = true;
            const uint32_t q_bytes = 128u * P.group * P.tile_tokens * G::SLABS;
            PaWork w;
            const auto load_q = [&](int i, int tok, int head) {  // into buffer i
                ok = __all_sync(~0u, pa_wait<D>(&bars.q_empty[i], (q_loads[i] & 1) ^ 1, kStatusTimeoutSync, wc));
                if (!ok) return;
                ++q_loads[i];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars.q_full[i], q_bytes);
                    for (int sl = 0; sl < G::SLABS; ++sl)
                        tma_load_3d(sQ + i * G::Q_TILE + sl * kSlab, &tm_q, &bars.q_full[i], sl * 64,
                                    head * P.group, w.q_tok + tok);
                }
            };
            int it = 0;
            while (ok && next_work(w)) {
                const int twin = TWINS ? w.twin : 0;
                const int tiles_q = ALT ? 1 : (w.n0 > 0 ? 1 : 0) + (w.n1 > 0 ? 2 : 0);  // bits
                // Q is read once and comes from far: on its way to L2 before its
                // place is free
                if (lane < 2 * G::SLABS && ((tiles_q >> (lane & 1)) & 1))
                    tma_prefetch_3d(&tm_q, (lane >> 1) * 64, (w.head + (lane & twin)) * P.group,
                                    w.q_tok + (lane & 1 & ~twin) * P.tile_tokens);
                __syncwarp();
                // in the order of use: K0 V0 K1 V1 ..., with two slots of S
                // K0 K1 V0 K2 V1 ...; Q behind the first two, whose places are free
                // before Q's is
                for (int j = 0; ok && j < 2 * w.n; ++j) {
                    const bool is_k = SLOTS == 1 ? (j & 1) == 0 : j == 0 || ((j & 1) != 0 && j < 2 * w.n - 1);
                    const int kt = SLOTS == 1 ? j / 2
                                   : is_k     ? (j + 1) / 2
                                              : (j == 2 * w.n - 1 ? w.n - 1 : j / 2 - 1);
                    const int st = g % G::STAGES, use = g / G::STAGES;
                    ok = __all_sync(~0u, pa_wait<D>(&bars.kv_empty[st], (use & 1) ^ 1, kStatusTimeoutSync, wc));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars.kv_full[st], G::TILE);
                        for (int sl = 0; sl < G::SLABS; ++sl)
                            tma_load_3d(sKV + st * G::TILE + sl * G::KV_SLAB, is_k ? &tm_k : &tm_v,
                                        &bars.kv_full[st], sl * 64, twin ? w.head + kt : w.head,
                                        w.k_row + (twin ? 0 : w.lo + kt) * KEYS);
                    }
                    ++g;
                    if (j == 1) {
                        if (ALT) {
                            load_q(it++ & 1, 0, w.head);
                        } else {
                            if (tiles_q & 1) load_q(0, 0, w.head);
                            if (ok && (tiles_q & 2)) load_q(1, twin ? 0 : P.tile_tokens, w.head + twin);
                        }
                    }
                }
            }
            // drain: the most recent load on every barrier has landed
            if (lane == 0) {
                for (int i = 0; i < 2; ++i)
                    if (q_loads[i] > 0)
                        pa_wait<D>(&bars.q_full[i], (q_loads[i] - 1) & 1, kStatusTimeoutDrain, drain);
                for (int st = 0; st < G::STAGES; ++st) {
                    const int uses = (g - st + G::STAGES - 1) / G::STAGES;  // loads into this stage
                    if (uses > 0)
                        pa_wait<D>(&bars.kv_full[st], (uses - 1) & 1, kStatusTimeoutDrain, drain);
                }
            }
            __syncwarp();
        } else {
            // -------------------------------------------- products of tile x
            // The whole warp walks; one lane issues.
            const int x = warp - kWarpMma;
            const uint32_t hi = static_cast<uint32_t>(smem_desc(0, 0, 1024, kSwizzle128B) >> 32);
            constexpr uint32_t kLboK = (16u >> 4) << 16, kLboV = static_cast<uint32_t>(G::KV_SLAB >> 4) << 16;
            uint32_t aQ = ((smem_u32(sQ) + (ALT ? 0 : x) * G::Q_TILE) >> 4) | kLboK;
            const uint32_t aKV = smem_u32(sKV) >> 4;
            const uint32_t t0 = __shfl_sync(~0u, tmem, 0);
            const uint32_t tS0 = t0 + G::S_COL + x * KEYS * G::SLOTS, tO = t0 + G::O_COL + x * D;
            const int q_steps = (P.d + 15) / 16;
            const uint32_t id_s = pa_idesc<T>(KEYS, false), id_o = pa_idesc<T>(q_steps * 16, true);
            int st = 0, ph = 0;  // stage and parity of the next K or V tile
            int it = 0, ns = 0, np = 0, no = 0;  // items, S and P tiles, outputs of this tile
            const auto slot = [&](int i) { return tS0 + (SLOTS == 2 && (i & 1) ? KEYS : 0); };
            int turns = 0;
            bool ok = true;

            const auto wait = [&](uint64_t *bar, uint32_t parity, unsigned code) {
                ok = ok && __all_sync(~0u, pa_wait<D>(bar, parity, code, wc));
                return ok;
            };
            const auto kv_wait = [&]() { return wait(&bars.kv_full[st], ph, kStatusTimeoutLoad); };
            // the stage after this one, which is waited for again later
            const auto kv_peek = [&]() {
                const int s2 = st + 1 == G::STAGES ? 0 : st + 1;
                wait(&bars.kv_full[s2], s2 == 0 ? ph ^ 1 : ph, kStatusTimeoutLoad);
            };
            // The two warps issue their P V and Q K^T in turn, so that the tiles
            // stay half a period apart: without it they fall into step, both
            // softmaxes beside an idle tensor pipe and then both products.
            const auto take_turn = [&]() {
                wait(&bars.turn[x], (turns & 1) ^ (x ^ 1), kStatusTimeoutSync);
                ++turns;
            };
            const auto pass_turn = [&]() {
                if (elect_one()) mbar_arrive(&bars.turn[x ^ 1]);
            };
            // done with the stage: after the products issued so far, or at once
            const auto kv_done = [&](bool used) {
                if (elect_one()) {
                    if (used)
                        mma_commit(&bars.kv_empty[st]);
                    else
                        mbar_arrive(&bars.kv_empty[st]);
                }
                if (++st == G::STAGES) {
                    st = 0;
                    ph ^= 1;
                }
            };
            // S = Q K^T; pass: hand the turn over while the last products are issued
            const auto qk = [&](bool pass) {
                uint64_t *full = &bars.s_full[x][SLOTS == 2 ? ns & 1 : 0];
                const uint32_t tS = slot(ns++);
                const uint32_t b = (aKV + st * (G::TILE >> 4)) | kLboK;
                if (q_steps == D / 16) {
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t in = (kk & 3) * (32 >> 4), sl = kk >> 2;
                            mma_ss(tS, aQ + sl * (kSlab >> 4) + in, b + sl * (G::KV_SLAB >> 4) + in, hi, id_s,
                                   kk > 0 ? 1u : 0u);
                            if (kk == D / 16 - 2 && pass) mbar_arrive(&bars.turn[x ^ 1]);
                        }
                        mma_commit(full);
                    }
                } else if (elect_one()) {  // channels past d are zero in shared memory: left out
#pragma unroll 1
                    for (int kk = 0; kk < q_steps; ++kk) {
                        const uint32_t in = (kk & 3) * (32 >> 4), sl = kk >> 2;
                        mma_ss(tS, aQ + sl * (kSlab >> 4) + in, b + sl * (G::KV_SLAB >> 4) + in, hi, id_s,
                               kk > 0 ? 1u : 0u);
                    }
                    if (pass) mbar_arrive(&bars.turn[x ^ 1]);
                    mma_commit(full);
                }
            };
            // O (+)= P V; left: keys of the tile; turn: the two warps' P V in turn
            const auto pv = [&](int left, bool first, bool turn) {
                const uint32_t b = (aKV + st * (G::TILE >> 4)) | kLboV;
                const uint32_t acc = first ? 0u : 1u;
                if (turn) take_turn();
                if (first) wait(&bars.o_empty[x], (no & 1) ^ 1, kStatusTimeoutSync);
                if (!wait(&bars.p_full[x][SLOTS == 2 ? np & 1 : 0], (SLOTS == 2 ? np >> 1 : np) & 1,
                          kStatusTimeoutSync))
                    return;
                uint64_t *done = &bars.pv_done[x][SLOTS == 2 ? np & 1 : 0];
                const uint32_t tP = slot(np++);
                tc_fence_after();
                if (left >= KEYS) {
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < KEYS / 16; ++kk)
                            mma_ts(tO, tP + kk * 8, b + kk * (2048 >> 4), hi, id_o, kk > 0 ? 1u : acc);
                        mma_commit(done);
                    }
                } else {  // only the 16-key steps that hold keys (one at least)
                    const int steps = max((left + 15) / 16, 1);
                    if (elect_one()) {
#pragma unroll 1
                        for (int kk = 0; kk < steps; ++kk)
                            mma_ts(tO, tP + kk * 8, b + kk * (2048 >> 4), hi, id_o, kk > 0 ? 1u : acc);
                        mma_commit(done);
                    }
                }
            };
            const auto q_done = [&]() {
                if (elect_one()) mma_commit(&bars.q_empty[ALT ? (it - 1) & 1 : x]);
            };
            PaWork w;
            while (ok && next_work(w)) {
                const int n = __shfl_sync(~0u, w.n, 0);
                const int nx = ALT ? (n + 1 - x) / 2 : __shfl_sync(~0u, x ? w.n1 : w.n0, 0);
                const int keys = __shfl_sync(~0u, w.nk - w.lo * KEYS, 0);
                if (ALT) {  // every other item's Q in the other buffer
                    if (!wait(&bars.q_full[it & 1], (it >> 1) & 1, kStatusTimeoutLoad)) break;
                    aQ = ((smem_u32(sQ) + (it & 1) * G::Q_TILE) >> 4) | kLboK;
                    if (nx == 0 && elect_one()) mbar_arrive(&bars.q_empty[it & 1]);
                    ++it;
                } else if (nx > 0) {
                    if (!wait(&bars.q_full[x], it & 1, kStatusTimeoutLoad)) break;
                    ++it;
                }
                if constexpr (!ALT) {
                    // the first S; then per key tile: P V, and S in the slot it frees.
                    // Twins share no key tile and wait for nothing of each other.
                    const bool twin = TWINS && __shfl_sync(~0u, w.twin, 0) != 0;
                    const int end = twin ? x : nx - 1;  // this tile's last
                    const auto uses = [&](int j) { return twin ? j == x : j < nx; };
                    for (int j = 0; j < SLOTS && j < n; ++j) {
                        if (!kv_wait()) break;
                        tc_fence_after();
                        if (uses(j)) qk(false);
                        kv_done(uses(j));
                    }
                    if (!ok) break;
                    if (nx > 0 && end < SLOTS) q_done();
                    for (int j = 0; j < n; ++j) {
                        const bool more = j + SLOTS < n, mine = more && uses(j + SLOTS);
                        if (!kv_wait()) break;
                        if (more) kv_peek();
                        if (uses(j))
                            pv(twin ? keys : keys - j * KEYS, twin || j == 0, !twin);
                        else if (!twin)
                            take_turn();
                        if (!ok) break;
                        kv_done(uses(j));
                        if (mine)
                            qk(!twin);
                        else if (!twin)
                            pass_turn();
                        if (more) kv_done(mine);
                        if (mine && j + SLOTS == end) q_done();
                        if (uses(j) && j == end) ++no;
                    }
                } else {
                    // this warp's key tiles are x, x + 2, ...; it lets go of the
                    // others as they land
                    for (int j = 0; j < n; ++j) {
                        const bool mine = (j & 1) == x;
                        if (!kv_wait()) break;
                        tc_fence_after();
                        if (mine) qk(false);
                        kv_done(mine);
                        if (mine && j + 2 >= n) q_done();
                        if (!kv_wait()) break;
                        if (mine) pv(keys - j * KEYS, j < 2, false);
                        if (!ok) break;
                        kv_done(mine);
                        if (mine && j + 2 >= n) ++no;
                    }
                }
            }
            // drain: a last commit completes after every product issued here
            __syncwarp();
            if (elect_one()) {
                mma_commit(&bars.fin[x]);
                pa_wait<D>(&bars.fin[x], 0, kStatusTimeoutDrain, drain);
            }
        }
        __syncwarp();
    } else {
        regs_alloc<kPaRegsSoftmax>();
        const int x = warp >> 2;                     // which tile
        const int row = tid & 127;                   // of the tile
        const int tok = row / P.group, hd = row - tok * P.group;
        const int tok_first = (row & ~31) / P.group; // token of the warp's first row
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane field: 32 * warp
        const uint32_t tS0 = tmem + lanes + G::S_COL + x * KEYS * G::SLOTS, tO = tmem + lanes + G::O_COL + x * D;
        int ns = 0, g = 0;  // S tiles of this tile, K and V tiles
        const float c = P.scale_log2;
        const float2 c2 = make_float2(c, c);
        // The P V before S tile ns is complete. (Of the barrier of its slot, the
        // P V two before it is complete, since S tile ns - 1 came behind it, and
        // none after it can be: the phase is unambiguous.)
        const auto pv_over = [&]() {
            const int k = ns - 1;
            return __all_sync(~0u, pa_wait_in(&bars.pv_done[x][SLOTS == 2 ? k & 1 : 0],
                                              (SLOTS == 2 ? k >> 1 : k) & 1, kStatusTimeoutMma, wc));
        };
        // What is to be written of the item before: its rows are written once the
        // last P V is complete, which the next item's first S comes behind; O is
        // free for the next P V once it is in registers.
        struct Due {
            bool live, valid;
            float m, l;
            int token, head, slot;
        } due{};
        bool is_due = false;
        PaWork w{};
        bool ok = true, more = true;
        while (more) {
            more = next_work(w);
            if (is_due) {
                is_due = false;
                if (!(ok = pv_over())) break;
                tc_fence_after();
                const float l = due.l, inv = l == 0.f ? 0.f : 1.f / l;
                const int64_t at = (static_cast<int64_t>(due.slot) * 2 + x) * P.ws_rows + row;
                const int64_t token = due.token, head = static_cast<int64_t>(due.head) * P.group + hd;
                if constexpr (ALT) {
                    // few rows: 128 bytes of each per thread and step, no exchange
                    float *dst = P.ws_o + at * D;
#pragma unroll 1
                    for (int q = 0; q < D; q += 32) {
                        uint32_t o[32];
                        if (due.live) {
                            tmem_ld32(tO + q, o);
                            tmem_ld_wait(o);
                        }
                        if (due.valid)
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<uint4 *>(dst + q + e) =
                                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.o_empty[x]);
                } else {
                    char *mine = PIECES ? reinterpret_cast<char *>(P.ws_o + at * D)
                                        : reinterpret_cast<char *>(static_cast<T *>(P.out) +
                                                                   token * P.out_token + head * P.out_head);
                    char *rows[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rows[i] = reinterpret_cast<char *>(
                            __shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine), (lane & ~3) + i));
                    const unsigned rows_ok = __ballot_sync(~0u, due.valid) >> (lane & ~3);
                    constexpr int COLS = PIECES ? 16 : 32;  // 64 bytes
#pragma unroll 1
                    for (int q = 0; q < P.d; q += COLS) {
                        uint32_t v[16];
                        if (due.live) {
                            if constexpr (PIECES) {
                                tmem_ld16(tO + q, v);
                                tmem_ld_wait(v);
                            } else {
                                uint32_t o[32];
                                tmem_ld32(tO + q, o);
                                tmem_ld_wait(o);
                                // a row that sees no key (or only scores of -inf) gives zeros
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    v[e] = l == 0.f ? 0u
                                                    : pa_pack<T>(__uint_as_float(o[2 * e]) * inv,
                                                                 __uint_as_float(o[2 * e + 1]) * inv);
                            }
                        }
                        if (q + COLS >= P.d) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars.o_empty[x]);
                        }
                        if (due.live)
                            store_rows(v, rows, q * (PIECES ? 4 : 2), rows_ok,
                                       q + (lane & 3) * (COLS / 4) < P.d, lane);
                    }
                }
                if (due.valid) {
                    if constexpr (PIECES) {
                        P.ws_ml[at] = make_float2(due.m, l);
                    } else if (P.lse != nullptr) {
                        P.lse[token * P.group * P.heads_kv + head] =
                            l == 0.f ? -INFINITY : (due.m + __log2f(l)) * 0.69314718055994531f;
                    }
                }
            }
            if (!more) break;
            const int n = ALT ? (w.n + 1 - x) / 2 : (x ? w.n1 : w.n0);
            const int twin = TWINS ? w.twin : 0;
            const int shift_tok = ALT || twin ? 0 : x * P.tile_tokens;
            const int toks = min(w.toks - shift_tok, P.tile_tokens);  // of this tile
            const bool valid = tok < toks;
            const int lim = P.causal ? min(w.nk, w.lim0 + shift_tok + tok) : w.nk;
            // masking is tested per warp against its first row, which sees least
            const int lim_first = P.causal ? min(w.nk, w.lim0 + shift_tok + tok_first) : w.nk;
            const bool warp_live = tok_first < toks && tok_first < P.tile_tokens;
            // the reference, the one that the next tile takes, the sum (rows that
            // do not exist keep a reference that asks for nothing)
            float m = valid ? -INFINITY : 0.f, m_next = m, l = 0.f;
            for (int i = 0; i < n; ++i, ++ns) {
                const int j = ALT ? 2 * i + x : i, kt = w.lo + j;
                const int sl = SLOTS == 2 ? ns & 1 : 0;
                ok = __all_sync(~0u, pa_wait_in(&bars.s_full[x][sl], (SLOTS == 2 ? ns >> 1 : ns) & 1,
                                                kStatusTimeoutMma, wc));
                if (!ok) break;
                if (w.nk < (kt + 1) * KEYS) {
                    // A part tile (the item's last): V's rows behind the sequence in
                    // the last 16-key step that the product reads become zero. (Of
                    // this stage's fills the one before has been used, K behind it
                    // having given S, and the one after waits for this P V, so the
                    // parity is unambiguous. Both tiles may do this: they write the
                    // same.)
                    const int idx = g + (twin ? (SLOTS == 1 ? 2 * x + 1 : 2 + x) : 2 * w.n - 1);
                    const int st = idx % G::STAGES, use = idx / G::STAGES;
                    ok = __all_sync(~0u, pa_wait_in(&bars.kv_full[st], use & 1, kStatusTimeoutLoad, wc));
                    if (!ok) break;
                    const int keys = max(w.nk - kt * KEYS, 0), end = max((keys + 15) / 16, 1) * 16;
                    const uint32_t dst = smem_u32(sKV) + st * G::TILE;
                    for (int k = 0; k < G::SLABS; ++k)
                        for (int e = keys * 8 + row; e < end * 8; e += 128)
                            st_shared_v4(dst + k * G::KV_SLAB + e * 16, 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                if (warp_live) {
                    tc_fence_after();
                    constexpr int NC = KEYS / 32;  // 32 scores at a time
                    const uint32_t tS = tS0 + sl * KEYS;
                    uint32_t s[NC][32];
#pragma unroll
                    for (int q = 0; q < NC; ++q) tmem_ld32(tS + q * 32, s[q]);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < NC; ++q) tmem_ready(s[q]);
                    const int seen = lim - kt * KEYS;  // columns that this row sees
                    if (lim_first < (kt + 1) * KEYS) {
#pragma unroll
                        for (int q = 0; q < NC; ++q)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (q * 32 + e >= seen) s[q][e] = 0xFF800000u;  // -inf
                    }
                    bool own = m == -INFINITY;  // no reference yet: the tile's maximum
                    float part;
                    while (true) {
                        if (__any_sync(~0u, own || m_next > m)) {
                            if (__any_sync(~0u, own)) {
                                float mx[NC];
#pragma unroll
                                for (int q = 0; q < NC; ++q) {
                                    mx[q] = -INFINITY;
#pragma unroll
                                    for (int e = 0; e < 32; e += 2)
                                        mx[q] = fmax3(mx[q], __uint_as_float(s[q][e]),
                                                      __uint_as_float(s[q][e + 1]));
                                }
                                float top = fmax3(mx[0], mx[1], mx[2]);
                                if constexpr (NC == 4) top = fmaxf(top, mx[3]);
                                if (own) m_next = fmaxf(m, top * c);
                            }
                            const float alpha = m_next > m ? (m == -INFINITY ? 0.f : ex2_approx(m - m_next)) : 1.f;
                            m = m_next;
                            l *= alpha;
                            if (i > 0) {
                                // once this tile's earlier products are complete (one
                                // slot: they are, the commit behind these scores covers
                                // them; two: all but the last)
                                if (SLOTS == 2) {
                                    ok = pv_over();
                                    if (!ok) break;
                                    tc_fence_after();
                                }
#pragma unroll 1
                                for (int r = 0; r < D / 16; ++r) {
                                    uint32_t o[16];
                                    tmem_ld16(tO + r * 16, o);
                                    tmem_ld_wait(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tmem_st16(tO + r * 16, o);
                                }
                            }
                        }
                        const float mm = m == -INFINITY ? 0.f : m;
                        const float2 nm = make_float2(-mm, -mm);
                        float2 sum[NC];
#pragma unroll
                        for (int q = 0; q < NC; ++q) {
                            uint32_t pk[16];
                            sum[q] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 y = ffma2(make_float2(__uint_as_float(s[q][2 * e]),
                                                                   __uint_as_float(s[q][2 * e + 1])),
                                                       c2, nm);
                                const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                                sum[q] = fadd2(sum[q], p);
                                pk[e] = pa_pack<T>(p.x, p.y);
                            }
                            tmem_st16(tS + q * 16, pk);
                        }
                        float2 t = fadd2(fadd2(sum[0], sum[1]), sum[2]);
                        if constexpr (NC == 4) t = fadd2(t, sum[3]);
                        part = t.x + t.y;
                        own = valid && part > kPaRedo<T>;
                        if (!__any_sync(~0u, own)) break;
                    }
                    if (!ok) break;
                    l += part;
                    if (valid && part > kPaMove) m_next = m + __log2f(part);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[x][sl]);
            }
            if (!ok) break;
            g += 2 * w.n;
            if (n > 0) {
                due.live = warp_live;
                due.valid = valid && (!PIECES || row < P.ws_rows);
                due.m = m;
                due.l = l;
                due.token = w.q_tok + shift_tok + tok;
                due.head = w.head + (twin ? x : 0);
                due.slot = w.slot;
                is_due = true;
            } else if (PIECES && valid && row < P.ws_rows) {
                P.ws_ml[(static_cast<int64_t>(w.slot) * 2 + x) * P.ws_rows + row] =
                    make_float2(-INFINITY, 0.f);
            }
        }
    }
    tc_fence_before();
    asm volatile("barrier.sync 0;" ::: "memory");
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of the rows: out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p.
// Its time is that of its chain of reads (the row's item, the item's pieces,
// then (m, l) and O together), so nothing is divided between them, the first O
// vectors are under way before their factors are known, and half a warp takes a
// row where rows are many. WIDE: a CTA per row, its warps taking every 16th
// piece (few rows, many pieces). Rows of no sequence are left alone: their entry
// of ws_item is whatever the workspace held, which is believed only if the item
// it names says that it holds the row.
constexpr int join_warps(bool wide) { return wide ? 16 : 4; }

template <int N>
__device__ __forceinline__ float join_max(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

template <int N>
__device__ __forceinline__ float join_sum(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <typename T, int D, bool ALT, bool WIDE>
__global__ void __launch_bounds__(32 * join_warps(WIDE))
packed_combine_kernel(const __grid_constant__ PackedAttnArgs P, int ctas) {
    constexpr int LANES = WIDE ? 32 : 16;             // of a row
    constexpr int W = D / LANES < 4 ? D / LANES : 4;  // floats of a vector
    constexpr int N = D / LANES / W;                  // vectors of a lane, LANES * W apart
    constexpr int WARPS = join_warps(WIDE), STEP = WIDE ? WARPS : 1, U = WIDE ? 2 : 4;
    __shared__ float part[WIDE ? WARPS : 1][WIDE ? D : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & (LANES - 1);
    const int heads = P.group * P.heads_kv, rows = P.total_q * heads;  // below 2^31
    const int want = WIDE ? blockIdx.x : blockIdx.x * (2 * WARPS) + threadIdx.x / LANES;
    const int out_row = min(want, rows - 1);
    const int token = out_row / heads;
    const int out_head = out_row - token * heads, kv_head = out_head / P.group;
    griddep_wait();
    const int *header = static_cast<const int *>(P.workspace);
    const int count = header[0], item = P.ws_item[token] + kv_head;
    bool valid = want < rows && item >= kv_head && item < count;
    const int4 a = valid ? reinterpret_cast<const int4 *>(header + 16)[item] : make_int4(0, 0, 0, 0);
    const int tok = token - a.z, x = tok >= P.tile_tokens ? 1 : 0;
    valid = valid && tok >= 0 && tok < a.w && static_cast<int>(static_cast<uint32_t>(a.y) >> 16) == kv_head;
    const int row = (tok - x * P.tile_tokens) * P.group + (out_head - kv_head * P.group);
    // (in range whatever the entry holds: after a wait that ran out it may be stale)
    valid = valid && row >= 0 && row < P.ws_rows && a.x >= 0 && a.x + (a.y & 0xFFFF) <= ctas;
    const int pieces = valid ? (ALT ? 2 : 1) * (a.y & 0xFFFF) : 0;
    const int64_t at0 = (static_cast<int64_t>(item + a.x) * 2 + (ALT ? 0 : x)) * P.ws_rows + row;
    const int64_t hop = static_cast<int64_t>(ALT ? 1 : 2) * P.ws_rows;
    const int most = WIDE ? pieces : max(pieces, __shfl_xor_sync(~0u, pieces, 16));

    float M = -INFINITY, L = 0.f, acc[N][W], v[U][N][W];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < W; ++e) acc[n][e] = 0.f;
    const auto fetch = [&](int p) {  // O of pieces p, p + STEP, ...
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p + u * STEP < pieces)
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const float *src = P.ws_o + (at0 + (p + u * STEP) * hop) * D + (n * LANES + lane) * W;
                    if constexpr (W == 4)
                        *reinterpret_cast<float4 *>(v[u][n]) = *reinterpret_cast<const float4 *>(src);
                    else
                        *reinterpret_cast<float2 *>(v[u][n]) = *reinterpret_cast<const float2 *>(src);
                }
    };
    for (int p0 = 0; p0 < most; p0 += LANES) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (p0 + lane < pieces) ml = P.ws_ml[at0 + (p0 + lane) * hop];
        int q = WIDE ? warp : 0;
        fetch(p0 + q);
        const float top = fmaxf(M, join_max<LANES>(ml.y == 0.f ? -INFINITY : ml.x));
        const float base = top == -INFINITY ? 0.f : top;
        const float keep = M == -INFINITY ? 0.f : ex2_approx(M - base);
        // no key seen: nothing was written
        const float f = ml.y == 0.f ? 0.f : ex2_approx(ml.x - base);
        L = L * keep + join_sum<LANES>(f * ml.y);
        M = top;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < W; ++e) acc[n][e] *= keep;
        for (; q < LANES && p0 + q < most; q += U * STEP) {
            if (q >= U * STEP) fetch(p0 + q);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float fu = __shfl_sync(~0u, f, (q + u * STEP) & (LANES - 1), LANES);
                if (fu != 0.f && p0 + q + u * STEP < pieces && q + u * STEP < LANES)
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int e = 0; e < W; ++e) acc[n][e] += fu * v[u][n][e];
            }
        }
    }
    if constexpr (WIDE) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < W; ++e) part[warp][(n * LANES + lane) * W + e] = acc[n][e];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < WARPS; ++i) s += part[i][(n * LANES + lane) * W + e];
                acc[n][e] = s;
            }
    }
    if (!valid) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (lane == 0 && P.lse != nullptr)
        P.lse[out_row] =
            L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
    T *dst = static_cast<T *>(P.out) + token * P.out_token + out_head * P.out_head;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int col = (n * LANES + lane) * W;
        if (col >= P.d) continue;
        float *o = acc[n];
#pragma unroll
        for (int e = 0; e < W; ++e) o[e] = L == 0.f ? 0.f : o[e] * inv;
        if constexpr (W == 4)
            *reinterpret_cast<uint2 *>(dst + col) = make_uint2(pa_pack<T>(o[0], o[1]), pa_pack<T>(o[2], o[3]));
        else
            *reinterpret_cast<uint32_t *>(dst + col) = pa_pack<T>(o[0], o[1]);
    }
}

template <typename T, int D, int KIND>
cudaError_t pa_launch_kind(const PackedAttnMaps &m, const PackedAttnArgs &a, int ctas,
                           cudaStream_t stream) {
    auto kernel = packed_attn_kernel<T, D, KIND>;
    cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           PaGeo<D>::SMEM);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kernel, dim3(ctas), dim3(kPaThreads), PaGeo<D>::SMEM, stream, m.q, m.k, m.v, a);
    if constexpr (KIND == kShared || KIND == kAlternate) {
        if (err != cudaSuccess) return err;
        constexpr bool ALT = KIND == kAlternate;
        const int64_t rows = static_cast<int64_t>(a.total_q) * a.group * a.heads_kv;
        if (rows <= 4 * sm_count())
            return launch_pdl(packed_combine_kernel<T, D, ALT, true>, dim3(static_cast<unsigned>(rows)),
                              dim3(32 * join_warps(true)), 0, stream, a, ctas);
        return launch_pdl(packed_combine_kernel<T, D, ALT, false>,
                          dim3(static_cast<unsigned>((rows + 2 * join_warps(false) - 1) / (2 * join_warps(false)))),
                          dim3(32 * join_warps(false)), 0, stream, a, ctas);
    }
    return err;
}

template <typename T, int D>
cudaError_t pa_launch(const PackedAttnMaps &m, const PackedAttnArgs &a, int kind, int ctas,
                      cudaStream_t stream) {
    return kind == kWhole    ? pa_launch_kind<T, D, kWhole>(m, a, ctas, stream)
           : kind == kTwins  ? pa_launch_kind<T, D, kTwins>(m, a, ctas, stream)
           : kind == kShared ? pa_launch_kind<T, D, kShared>(m, a, ctas, stream)
                             : pa_launch_kind<T, D, kAlternate>(m, a, ctas, stream);
}

}  // namespace
}  // namespace vta
