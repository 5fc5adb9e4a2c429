// attention_api.hip -- the C ABI of the attention block on the MXFP4 cache
// (declared in include/w4a8.h): arguments are validated on the host before
// anything is enqueued, as in api.hip.
#include <math.h>

#include "w4a8_internal.h"

using namespace w4a8;

namespace {

constexpr int64_t kMaxCount = (int64_t)1 << 30;
constexpr int kMaxHeads = 1024;
constexpr int kSegmentTiles = 16;   // at most what a segment counts for beside its tiles (attention.hip)

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline w4a8_status hip_status(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP; }
inline bool known_dim(int d) { return d == 64 || d == 128 || d == 256; }
inline bool known_type(w4a8_float t) { return t == W4A8_BF16 || t == W4A8_FP16; }

// log2 of the page, or -1
int page_shift_of(int page) {
    for (int s = 4; s <= 10; ++s)
        if (page == 1 << s) return s;
    return -1;
}

w4a8_status check_cache(const w4a8_kv_cache* c) {
    if (!c || !c->k_codes || !c->k_e8m0 || !c->v_codes || !c->v_e8m0) return W4A8_ERR_INVALID_ARG;
    if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > kMaxHeads) return W4A8_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_e8m0, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_e8m0, 16))
        return W4A8_ERR_INVALID_ARG;
    if (!known_dim(c->head_dim) || page_shift_of(c->page) < 0 || c->pages >= ((int64_t)1 << 40) / c->page)
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    return W4A8_OK;
}

// 16-bit heads: 2-byte aligned, heads of head_dim contiguous values
w4a8_status check_heads(const uint16_t* p, int64_t st, int64_t sh, int heads) {
    if (!p || heads < 1 || heads > kMaxHeads || st < 0 || sh < 0 || !aligned(p, 2)) return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}

w4a8_status check_turn(const float* q_w, const float* k_w, float eps, const float* cos_sin, int64_t cos_rows,
                       const int64_t* positions, int rot, int head_dim) {
    if (!aligned(q_w, 4) || !aligned(k_w, 4) || !(eps >= 0.0f) || !isfinite(eps) || rot < 0) return W4A8_ERR_INVALID_ARG;
    if (rot % 16 != 0 || rot > head_dim) return W4A8_ERR_UNSUPPORTED_SHAPE;
    if (rot && (!cos_sin || !positions || cos_rows < 1 || !aligned(cos_sin, 4) || !aligned(positions, 8)))
        return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}

}  // namespace

extern "C" {

w4a8_status w4a8_qk_norm_rope(w4a8_float type, const uint16_t* d_q, int64_t q_stride_token, int64_t q_stride_head,
                              int q_heads, const uint16_t* d_k, int64_t k_stride_token, int64_t k_stride_head,
                              int k_heads, int64_t tokens, int head_dim, const float* d_q_weight,
                              const float* d_k_weight, float eps, const float* d_cos_sin, int64_t cos_rows,
                              const int64_t* d_positions, int rot, int interleaved, uint16_t* d_q_out,
                              uint16_t* d_k_out, void* stream) {
    if (!known_type(type) || tokens < 1 || (!d_q && !d_k)) return W4A8_ERR_INVALID_ARG;
    if (!d_q && q_heads != 0) return W4A8_ERR_INVALID_ARG;
    if (!d_k && k_heads != 0) return W4A8_ERR_INVALID_ARG;
    w4a8_status st = W4A8_OK;
    if (d_q && (st = check_heads(d_q, q_stride_token, q_stride_head, q_heads)) != W4A8_OK) return st;
    if (d_k && (st = check_heads(d_k, k_stride_token, k_stride_head, k_heads)) != W4A8_OK) return st;
    if ((d_q && (!d_q_out || !aligned(d_q_out, 16))) || (d_k && (!d_k_out || !aligned(d_k_out, 16))))
        return W4A8_ERR_INVALID_ARG;
    if (!known_dim(head_dim) || tokens >= kMaxCount / (q_heads + k_heads)) return W4A8_ERR_UNSUPPORTED_SHAPE;
    st = check_turn(d_q_weight, d_k_weight, eps, d_cos_sin, cos_rows, d_positions, rot, head_dim);
    if (st != W4A8_OK) return st;
    HeadRows a{};
    a.q = d_q, a.q_st = q_stride_token, a.q_sh = q_stride_head, a.hq = q_heads;
    a.k = d_k, a.k_st = k_stride_token, a.k_sh = k_stride_head, a.hk = k_heads;
    a.tokens = tokens;
    a.q_weight = d_q_weight, a.k_weight = d_k_weight, a.eps = eps;
    a.cos_sin = d_cos_sin, a.cs_rows = cos_rows, a.positions = d_positions, a.rot = rot;
    a.interleaved = interleaved != 0;
    a.q_out = d_q_out, a.k_out = d_k_out;
    a.cache.head_dim = head_dim;
    if (head_rows_threads(a) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_head_rows(a, type == W4A8_FP16, as_stream(stream)));
}

w4a8_status w4a8_kv_append_mxfp4(const w4a8_kv_cache* cache, w4a8_float type, const uint16_t* d_k,
                                 int64_t k_stride_token, int64_t k_stride_head, const uint16_t* d_v,
                                 int64_t v_stride_token, int64_t v_stride_head, int64_t tokens,
                                 const int64_t* d_slots, w4a8_exp_mode mode, const float* d_k_weight, float eps,
                                 const float* d_cos_sin, int64_t cos_rows, const int64_t* d_positions, int rot,
                                 int interleaved, const uint16_t* d_q, int64_t q_stride_token,
                                 int64_t q_stride_head, int q_heads, const float* d_q_weight, uint16_t* d_q_out,
                                 void* stream) {
    w4a8_status st = check_cache(cache);
    if (st != W4A8_OK) return st;
    const int hk = cache->kv_heads;
    if (!known_type(type) || tokens < 1 || !d_slots || !aligned(d_slots, 8)) return W4A8_ERR_INVALID_ARG;
    if (mode != W4A8_EXP_OCP && mode != W4A8_EXP_NOCLIP) return W4A8_ERR_INVALID_ARG;
    if ((st = check_heads(d_k, k_stride_token, k_stride_head, hk)) != W4A8_OK) return st;
    if ((st = check_heads(d_v, v_stride_token, v_stride_head, hk)) != W4A8_OK) return st;
    if (!d_q && q_heads != 0) return W4A8_ERR_INVALID_ARG;
    if (d_q) {
        if ((st = check_heads(d_q, q_stride_token, q_stride_head, q_heads)) != W4A8_OK) return st;
        if (!d_q_out || !aligned(d_q_out, 16)) return W4A8_ERR_INVALID_ARG;
    }
    if (tokens >= kMaxCount / (q_heads + 2 * hk)) return W4A8_ERR_UNSUPPORTED_SHAPE;
    st = check_turn(d_q_weight, d_k_weight, eps, d_cos_sin, cos_rows, d_positions, rot, cache->head_dim);
    if (st != W4A8_OK) return st;
    HeadRows a{};
    a.q = d_q, a.q_st = q_stride_token, a.q_sh = q_stride_head, a.hq = q_heads;
    a.k = d_k, a.k_st = k_stride_token, a.k_sh = k_stride_head, a.hk = hk;
    a.v = d_v, a.v_st = v_stride_token, a.v_sh = v_stride_head, a.hv = hk;
    a.tokens = tokens;
    a.q_weight = d_q_weight, a.k_weight = d_k_weight, a.eps = eps;
    a.cos_sin = d_cos_sin, a.cs_rows = cos_rows, a.positions = d_positions, a.rot = rot;
    a.interleaved = interleaved != 0;
    a.q_out = d_q_out;
    a.cache = *cache;
    a.page_shift = page_shift_of(cache->page);
    a.slots = d_slots;
    a.mode = (int)mode;
    if (head_rows_threads(a) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_head_rows(a, type == W4A8_FP16, as_stream(stream)));
}

w4a8_status w4a8_kv_read_mxfp4(const w4a8_kv_cache* cache, int64_t tokens, const int64_t* d_slots, uint16_t* d_k_out,
                               uint16_t* d_v_out, void* stream) {
    const w4a8_status st = check_cache(cache);
    if (st != W4A8_OK) return st;
    if (tokens < 1 || !d_slots || !d_k_out || !d_v_out || !aligned(d_slots, 8) || !aligned(d_k_out, 16) ||
        !aligned(d_v_out, 16))
        return W4A8_ERR_INVALID_ARG;
    if (tokens >= kMaxCount / (2 * cache->kv_heads) || kv_read_threads(*cache, tokens) >= kGridThreads)
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_kv_read(*cache, page_shift_of(cache->page), tokens, d_slots, d_k_out, d_v_out,
                                     as_stream(stream)));
}

static bool attention_shape(int64_t seqs, int64_t max_q, int q_heads, int kv_heads) {
    return seqs >= 1 && max_q >= 1 && kv_heads >= 1 && q_heads >= 1 && q_heads <= kMaxHeads && q_heads % kv_heads == 0;
}

size_t w4a8_attention_workspace_bytes(int64_t seqs, int64_t max_q, int q_heads, int kv_heads, int head_dim) {
    if (!attention_shape(seqs, max_q, q_heads, kv_heads) || !known_dim(head_dim)) return 0;
    if (seqs >= kMaxCount || max_q >= kMaxCount / (seqs * q_heads)) return 0;
    return attention_workspace_bytes(seqs, max_q, q_heads, kv_heads, head_dim);
}

size_t w4a8_attention_counter_bytes(void) { return attention_counter_bytes(); }

w4a8_status w4a8_attention_mxfp4(const w4a8_kv_cache* cache, w4a8_float type, const uint16_t* d_q,
                                 int64_t q_stride_token, int64_t q_stride_head, int q_heads, int64_t tokens,
                                 int64_t seqs, const int32_t* d_cu_q, int64_t max_q, const int32_t* d_block_table,
                                 int64_t table_stride, int64_t table_width, const int32_t* d_context_lens,
                                 float scale, int causal, int window, uint16_t* d_out, void* d_ws, size_t ws_bytes,
                                 void* stream) {
    w4a8_status st = check_cache(cache);
    if (st != W4A8_OK) return st;
    if (!known_type(type) || !attention_shape(seqs, max_q, q_heads, cache->kv_heads)) return W4A8_ERR_INVALID_ARG;
    if ((st = check_heads(d_q, q_stride_token, q_stride_head, q_heads)) != W4A8_OK) return st;
    if (tokens < 1 || !d_block_table || !d_context_lens || !d_out || table_width < 1 || table_stride < table_width ||
        !aligned(d_block_table, 4) || !aligned(d_context_lens, 4) || !aligned(d_cu_q, 4) || !aligned(d_out, 16))
        return W4A8_ERR_INVALID_ARG;
    if (!isfinite(scale) || window < 0 || (window && !causal)) return W4A8_ERR_INVALID_ARG;
    if (!d_cu_q && (tokens != seqs || max_q != 1)) return W4A8_ERR_INVALID_ARG;
    if (tokens >= kMaxCount / q_heads || seqs >= kMaxCount || max_q >= kMaxCount / (seqs * q_heads) ||
        table_width >= kMaxCount / cache->page ||
        (table_width * cache->page + 63) / 64 + kSegmentTiles >= kMaxCount / (seqs * cache->kv_heads))
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    const size_t need = attention_workspace_bytes(seqs, max_q, q_heads, cache->kv_heads, cache->head_dim);
    if (need && (!d_ws || ws_bytes < need || !aligned(d_ws, 256))) return W4A8_ERR_WORKSPACE;
    AttnArgs a{};
    a.cache = *cache;
    a.page_shift = page_shift_of(cache->page);
    a.q = d_q, a.q_st = q_stride_token, a.q_sh = q_stride_head;
    a.out = d_out;
    a.hq = q_heads, a.group = q_heads / cache->kv_heads;
    a.tokens = tokens;
    a.seqs = (int)seqs, a.max_q = (int)max_q;
    a.cu_q = d_cu_q;
    a.table = d_block_table, a.table_stride = table_stride, a.table_width = (int)table_width;
    a.context = d_context_lens;
    a.scale = scale;
    a.causal = causal != 0, a.window = window;
    a.ws = static_cast<uint8_t*>(d_ws);
    if (attention_threads(a, type == W4A8_FP16) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_attention(a, type == W4A8_FP16, as_stream(stream)));
}

}  // extern "C"
