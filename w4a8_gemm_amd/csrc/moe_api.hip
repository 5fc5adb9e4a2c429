// moe_api.hip -- the C ABI of the expert half of a layer (declared in
// include/w4a8.h): arguments are validated on the host before anything is
// enqueued, as in api.hip.
#include <math.h>

#include "w4a8_internal.h"

using namespace w4a8;

namespace {

constexpr int64_t kMaxCount = (int64_t)1 << 30;
constexpr int64_t kMaxHidden = 32768;
constexpr int kMaxExperts = 1024, kMaxTopK = 32, kMaxGroups = 64;
constexpr int64_t kMaxWidth = 65536;       // hidden and inter of the experts
constexpr int64_t kMaxChunks = 1 << 15;    // a grid's second dimension holds 2^16 - 1

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline w4a8_status hip_status(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP; }

}  // namespace

extern "C" {

w4a8_status w4a8_residual_norm(w4a8_float type, const uint16_t* d_y, int64_t ld_y, int64_t tokens, int64_t hidden,
                               const float* d_post_weight, const uint16_t* d_gate, int64_t gate_stride_token,
                               int64_t gate_stride_col, float scale, const void* d_residual, int residual_fp32,
                               int64_t ld_residual, void* d_residual_out, int64_t ld_residual_out,
                               const float* d_weight, float eps, uint16_t* d_out, uint8_t* d_x_fp8, float* d_x_scale,
                               void* stream) {
    if ((type != W4A8_BF16 && type != W4A8_FP16) || !d_y || tokens < 1 || hidden < 1) return W4A8_ERR_INVALID_ARG;
    if (!d_residual_out && !d_out && !d_x_fp8) return W4A8_ERR_INVALID_ARG;
    if ((d_x_fp8 != nullptr) != (d_x_scale != nullptr)) return W4A8_ERR_INVALID_ARG;
    const size_t ra = d_residual && residual_fp32 ? 4 : 2;
    if (!aligned(d_y, 2) || !aligned(d_gate, 2) || !aligned(d_out, 2) || !aligned(d_residual, ra) ||
        !aligned(d_residual_out, ra) || !aligned(d_post_weight, 4) || !aligned(d_weight, 4) || !aligned(d_x_scale, 4))
        return W4A8_ERR_INVALID_ARG;
    if (!isfinite(scale) || !isfinite(eps) || !(eps >= 0.0f)) return W4A8_ERR_INVALID_ARG;
    if (ld_y < 0 || (d_residual && ld_residual < 0) || (d_residual_out && ld_residual_out < hidden && tokens > 1))
        return W4A8_ERR_INVALID_ARG;
    if (d_gate && (gate_stride_token < 0 || gate_stride_col < 0 || gate_stride_col > 1)) return W4A8_ERR_INVALID_ARG;
    if (hidden > kMaxHidden || tokens >= kMaxCount || tokens >= ((int64_t)1 << 40) / hidden)
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    NormArgs a{};
    a.y = d_y, a.ldy = ld_y;
    a.tokens = tokens, a.hidden = (int)hidden;
    a.post_weight = d_post_weight;
    a.gate = d_gate, a.gate_st = gate_stride_token, a.gate_sc = gate_stride_col;
    a.scale = scale;
    a.residual = d_residual, a.residual_fp32 = d_residual && residual_fp32, a.ldr = ld_residual;
    a.residual_out = d_residual_out, a.ldro = ld_residual_out;
    a.weight = d_weight, a.eps = eps;
    a.out = d_out, a.x8 = d_x_fp8, a.xs = d_x_scale;
    if (residual_norm_threads(a) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_residual_norm(a, type == W4A8_FP16, as_stream(stream)));
}

w4a8_status w4a8_moe_route(w4a8_float type, const void* d_logits, int64_t ld, int64_t tokens, int experts, int top_k,
                           w4a8_score score, const float* d_bias, int groups, int groups_kept, int group_top,
                           int renormalize, float scale, int32_t* d_ids, float* d_weights, void* stream) {
    if (type != W4A8_BF16 && type != W4A8_FP16 && type != W4A8_FP32) return W4A8_ERR_INVALID_ARG;
    if (score != W4A8_SCORE_SOFTMAX && score != W4A8_SCORE_SIGMOID) return W4A8_ERR_INVALID_ARG;
    if (!d_logits || !d_ids || !d_weights || tokens < 1 || experts < 1 || top_k < 1 || groups < 1 || groups_kept < 1 ||
        ld < 0 || !isfinite(scale) || group_top < 1 || group_top > 2)
        return W4A8_ERR_INVALID_ARG;
    if (!aligned(d_logits, type == W4A8_FP32 ? 4 : 2) || !aligned(d_bias, 4) || !aligned(d_ids, 4) || !aligned(d_weights, 4))
        return W4A8_ERR_INVALID_ARG;
    if (experts > kMaxExperts || top_k > kMaxTopK || top_k > experts || groups > kMaxGroups || experts % groups ||
        groups_kept > groups || tokens >= kMaxCount / top_k)
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    RouteArgs a{};
    a.logits = d_logits, a.ld = ld, a.tokens = tokens;
    a.experts = experts, a.top_k = top_k, a.score = (int)score, a.bias = d_bias;
    a.groups = groups, a.groups_kept = groups_kept, a.group_top = group_top;
    a.renormalize = renormalize != 0, a.scale = scale;
    a.ids = d_ids, a.weights = d_weights;
    if (moe_route_threads(a) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    return hip_status(launch_moe_route(a, type, as_stream(stream)));
}

static bool moe_shape(int64_t tokens, int top_k, int64_t hidden, int64_t inter) {
    return hidden >= 128 && hidden <= kMaxWidth && hidden % 128 == 0 && tokens >= 1 && top_k >= 1 && top_k <= kMaxTopK && inter >= 128 && inter <= kMaxWidth && inter % 128 == 0 &&
           tokens < kMaxCount / top_k && tokens <= kMaxChunks * moe_chunk_tokens(top_k);
}

size_t w4a8_moe_workspace_bytes(int64_t tokens, int top_k, int64_t hidden, int64_t inter) {
    return moe_shape(tokens, top_k, hidden, inter) ? moe_workspace_bytes(tokens * top_k, hidden, inter) : 0;
}

w4a8_status w4a8_moe_mxfp4(const w4a8_experts_mxfp4* experts, const uint8_t* d_x_fp8, const float* d_x_scale,
                           int64_t tokens, const int32_t* d_ids, const float* d_weights, int top_k, w4a8_act act,
                           uint16_t* d_out, void* d_ws, size_t ws_bytes, void* stream) {
    if (!experts || !experts->up_w || !experts->up_s || !experts->down_w || !experts->down_s || !d_x_fp8 || !d_x_scale ||
        !d_ids || !d_weights || !d_out || tokens < 1 || top_k < 1 || experts->experts < 1 || experts->hidden < 1 ||
        experts->inter < 1)
        return W4A8_ERR_INVALID_ARG;
    if (act != W4A8_ACT_SILU && act != W4A8_ACT_GELU_TANH) return W4A8_ERR_INVALID_ARG;
    if (!aligned(experts->up_w, 16) || !aligned(experts->up_s, 16) || !aligned(experts->down_w, 16) ||
        !aligned(experts->down_s, 16) || !aligned(d_x_fp8, 16) || !aligned(d_x_scale, 4) || !aligned(d_ids, 4) ||
        !aligned(d_weights, 4) || !aligned(d_out, 8))
        return W4A8_ERR_INVALID_ARG;
    if (experts->experts > kMaxExperts || top_k > experts->experts ||
        !moe_shape(tokens, top_k, experts->hidden, experts->inter))
        return W4A8_ERR_UNSUPPORTED_SHAPE;
    MoeArgs a{};
    a.e = *experts;
    a.x8 = d_x_fp8, a.xs = d_x_scale, a.tokens = tokens;
    a.ids = d_ids, a.weights = d_weights, a.top_k = top_k, a.act = (int)act;
    a.out = d_out, a.ws = static_cast<uint8_t*>(d_ws);
    return launch_moe(a, ws_bytes, as_stream(stream));
}

}  // extern "C"
