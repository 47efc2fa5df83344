// packed_attn.cu -- the entry points packed_attn_fwd and packed_attn_workspace
// of rpe_attn.h: argument checks, the split of the work, tensor maps and the
// launch. The kernels are in packed_attn.cuh.
#include "rpe_attn.h"
#include "vta_internal.h"
#include "sm103_ptx.cuh"

#include <cmath>
#include <cstdint>

namespace vta {
namespace {

// How a call is split, from sizes that the host knows.
struct Plan {
    int kind;  // 0 whole items, 1 pieces of two tiles, 2 pieces of one, 3 whole items, short ones by two heads
    int ctas, tile_tokens, ws_rows;
    int64_t max_items;
    size_t item_at, ml_at, o_at, bytes;  // workspace offsets and size (pieces)
};

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

Plan make_plan(int64_t total_q, int64_t total_k, int batch, int heads_q, int heads_kv, int d) {
    Plan p{};
    const int group = heads_q / heads_kv, sms = sm_count();
    p.tile_tokens = 128 / group;
    // items of one and of two tiles of 128 rows: at most one part per sequence
    const int64_t ones = least(total_q, total_q / p.tile_tokens + batch) * heads_kv;
    const int64_t pairs = least(total_q, total_q / (2 * p.tile_tokens) + batch) * heads_kv;
    // One tile where a sequence's queries fill half of one at most and its keys
    // outnumber them (a second tile would have nothing to do); two tiles, in
    // pieces, where whole items would leave SMs idle and keys are long enough
    // to share out.
    const bool thin = total_q <= static_cast<int64_t>(batch) * p.tile_tokens / 2 && total_k >= 4 * total_q;
    const bool few = pairs < 2 * sms && total_k >= 512 * static_cast<int64_t>(batch);
    // Two heads of a short sequence at once where sequences have a tile and a half
    // at most on average (one tile each: 41 us instead of 65; two each: 73 instead
    // of 69) and the items are more than one round of the SMs.
    const bool brief = heads_kv > 1 && 2 * total_q <= 3 * static_cast<int64_t>(batch) * p.tile_tokens &&
                       pairs >= 2 * sms;
    p.kind = thin ? 2 : few ? 1 : brief ? 3 : 0;
    const bool pieces = p.kind == 1 || p.kind == 2;
    p.ctas = static_cast<int>(pieces ? sms : least(pairs, sms));
    if (!pieces) return p;
    p.max_items = thin ? ones : pairs;
    p.ws_rows = static_cast<int>(least(128, group * least(p.tile_tokens, total_q)));
    const int D = d <= 64 ? 64 : 128;
    const size_t rows = static_cast<size_t>(p.max_items + p.ctas) * 2 * p.ws_rows;
    p.item_at = 64 + static_cast<size_t>(p.max_items) * 16;
    p.ml_at = (p.item_at + static_cast<size_t>(total_q) * sizeof(int32_t) + 127) & ~static_cast<size_t>(127);
    p.o_at = (p.ml_at + rows * sizeof(float2) + 127) & ~static_cast<size_t>(127);
    p.bytes = p.o_at + rows * D * sizeof(float);
    return p;
}

int check_sizes(int64_t total_q, int64_t total_k, int batch, int heads_q, int heads_kv, int d,
                int dtype) {
    if (total_q < 0 || total_k < 0 || batch < 0 || heads_q < 1 || heads_kv < 1 || d < 1 ||
        heads_q % heads_kv != 0)
        return RPE_ERR_INVALID_ARG;
    if (dtype != RPE_DTYPE_BF16 && dtype != RPE_DTYPE_F32 && dtype != RPE_DTYPE_F16)
        return RPE_ERR_INVALID_ARG;
    if (dtype == RPE_DTYPE_F32 || d > 128 || d % 8 != 0 || heads_q / heads_kv > 128 ||
        heads_q > 65536 || batch >= (1 << 24) || total_q >= (1 << 30) || total_k >= (1 << 30))
        return RPE_ERR_UNSUPPORTED;
    return RPE_OK;
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A view whose rows TMA (and 16-byte stores) can reach.
bool good_view(const rpe_view *v, int64_t tokens, int heads) {
    if (v == nullptr || v->data == nullptr || !aligned(v->data, 16)) return false;
    if (tokens > 1 && (v->token_stride <= 0 || v->token_stride % 8 != 0)) return false;
    return heads <= 1 || (v->head_stride > 0 && v->head_stride % 8 == 0);
}

bool token_map(CUtensorMap *map, int dtype, const rpe_view &v, int64_t tokens, int heads, int d,
               int box_heads, int box_tokens) {
    // the stride of an axis with one entry is free: any multiple of 16 bytes
    const uint64_t hs = static_cast<uint64_t>(heads > 1 ? v.head_stride : 8 * ((d + 7) / 8)) * 2;
    const uint64_t ts = static_cast<uint64_t>(tokens > 1 ? v.token_stride : 8 * ((d + 7) / 8)) * 2;
    const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                              static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {hs, ts};
    const uint32_t box[3] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
    return encode_tensor_map(map,
                             dtype == RPE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                             3, v.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace
}  // namespace vta

using namespace vta;

extern "C" {

int packed_attn_workspace(int64_t total_q, int64_t total_k, int batch, int heads_q, int heads_kv,
                          int d, int dtype, size_t *bytes) {
    if (bytes == nullptr) return RPE_ERR_INVALID_ARG;
    const int rc = check_sizes(total_q, total_k, batch, heads_q, heads_kv, d, dtype);
    if (rc != RPE_OK) return rc;
    *bytes = total_q == 0 || batch == 0
                 ? 0
                 : make_plan(total_q, total_k, batch, heads_q, heads_kv, d).bytes;
    return RPE_OK;
}

int packed_attn_fwd(const rpe_view *q, const rpe_view *k, const rpe_view *v, const rpe_view *out,
                    float *lse, const int32_t *cu_q, const int32_t *cu_k, const int32_t *k_lens,
                    int batch, int64_t total_q, int64_t total_k, int heads_q, int heads_kv, int d,
                    float scale, unsigned flags, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream) {
    const int rc = check_sizes(total_q, total_k, batch, heads_q, heads_kv, d, dtype);
    if (rc == RPE_ERR_INVALID_ARG) return rc;
    if ((flags & ~static_cast<unsigned>(RPE_ATTN_CAUSAL)) != 0 || !std::isfinite(scale) ||
        scale <= 0.f)
        return RPE_ERR_INVALID_ARG;
    if (rc != RPE_OK) return rc;
    if (total_q == 0 || batch == 0) return RPE_OK;  // no row to write
    if (!good_view(q, total_q, heads_q) || !good_view(out, total_q, heads_q) ||
        (total_k > 0 && (!good_view(k, total_k, heads_kv) || !good_view(v, total_k, heads_kv))))
        return RPE_ERR_INVALID_ARG;
    if (cu_q == nullptr || cu_k == nullptr || !aligned(cu_q, 4) || !aligned(cu_k, 4) ||
        !aligned(k_lens, 4) || !aligned(lse, 4))
        return RPE_ERR_INVALID_ARG;
    const Plan p = make_plan(total_q, total_k, batch, heads_q, heads_kv, d);
    if (p.bytes > 0 && (workspace == nullptr || !aligned(workspace, 128) || workspace_bytes < p.bytes))
        return RPE_ERR_INVALID_ARG;
    if (p.bytes > 0 && (p.max_items > INT32_MAX / 2 || total_q * heads_q > INT32_MAX - 64))
        return RPE_ERR_UNSUPPORTED;

    PackedAttnArgs a{};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.k_lens = k_lens;
    a.batch = batch;
    a.total_q = static_cast<int>(total_q);
    a.total_k = static_cast<int>(total_k);
    a.heads_kv = heads_kv;
    a.group = heads_q / heads_kv;
    a.d = d;
    a.tile_tokens = p.tile_tokens;
    a.causal = (flags & RPE_ATTN_CAUSAL) ? 1 : 0;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.out = out->data;
    a.out_token = total_q > 1 ? out->token_stride : 0;
    a.out_head = heads_q > 1 ? out->head_stride : 0;
    a.lse = lse;
    if (p.bytes > 0) {
        char *ws = static_cast<char *>(workspace);
        a.workspace = ws;
        a.ws_item = reinterpret_cast<int32_t *>(ws + p.item_at);
        a.ws_ml = reinterpret_cast<float2 *>(ws + p.ml_at);
        a.ws_o = reinterpret_cast<float *>(ws + p.o_at);
        a.ws_rows = p.ws_rows;
        a.max_items = static_cast<int>(p.max_items);
    }
    PackedAttnMaps m;
    // without any key the maps read q's first row instead (every score is masked)
    const rpe_view none{q->data, 0, 0, 0};
    const int64_t rows_k = total_k > 0 ? total_k : 1;
    const int heads_m = total_k > 0 ? heads_kv : 1, keys = d <= 64 ? 96 : 128;  // of a key tile
    if (!token_map(&m.q, dtype, *q, total_q, heads_q, d, a.group, p.tile_tokens) ||
        !token_map(&m.k, dtype, total_k > 0 ? *k : none, rows_k, heads_m, d, 1, keys) ||
        !token_map(&m.v, dtype, total_k > 0 ? *v : none, rows_k, heads_m, d, 1, keys))
        return RPE_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!status_word_ready(st)) return RPE_ERR_UNSUPPORTED;
    a.status = device_status_word();
    if (a.status == nullptr) return RPE_ERR_CUDA;
    const bool bf16 = dtype == RPE_DTYPE_BF16;
    const cudaError_t err = d <= 64 ? launch_packed_attn_d64(m, a, bf16, p.kind, p.ctas, st)
                                    : launch_packed_attn_d128(m, a, bf16, p.kind, p.ctas, st);
    return err == cudaSuccess ? RPE_OK : RPE_ERR_CUDA;
}

}  // extern "C"
