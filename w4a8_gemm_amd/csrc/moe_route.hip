// moe_route.hip -- each token's experts from the router's logits.
//
// A wave takes a token: lane L holds the experts L, L + 64, ...  Each round of the
// choice takes the largest key of the wave (unsigned keys in the scores' order, so
// a maximum is one instruction a step) and, of those that hold it, the lowest
// expert.
//
// Without bias and groups the choice goes by the logits themselves.  With them it
// goes by scores in fp64: which expert a token meets should follow from the inputs,
// not from how an exponential or a sum was rounded.  Weights are sums and
// exponentials in the same precision, but for the sigmoids of experts chosen by their logits,
// which are fp64 too.
#include <type_traits>

#include "wave_ops.h"

#pragma clang fp contract(off)

namespace w4a8 {
namespace {

constexpr int kRouteWaves = 4;   // tokens to a workgroup

// keys in the order of the values, 0 for one that may not be chosen
__device__ __forceinline__ uint32_t key_of(float v) {
    if (!(v > -__builtin_inff())) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 counts as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
    if (!(v > -__builtin_inf())) return 0u;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return wave_reduce(v, Max()); }
// the lanes that hold the largest key, which is not 0; none if all are.  The low halves are looked at only
// where several lanes share the high one.
__device__ __forceinline__ uint64_t lanes_of_max(uint64_t v) {
    const uint32_t hi = (uint32_t)(v >> 32);
    const uint32_t most = wave_max(hi);
    uint64_t have = most ? __ballot(hi == most) : 0;
    if (have & (have - 1)) {
        const bool in = (have >> (threadIdx.x & 63)) & 1;
        const uint32_t top = wave_max(in ? (uint32_t)v : 0u);
        have = __ballot(in && (uint32_t)v == top);
    }
    return have;
}

// A chosen expert's sigmoid where the choice went by the logits, its lane's alone: in fp64, as 1 + exp(-logit) leaves
// fp32 below a logit of -88, and of such scores renormalized ones are not zeros.
__device__ __forceinline__ double chosen_sigmoid(int id, float logit) { return id >= 0 ? 1.0 / (1.0 + exp(-(double)logit)) : 0.0; }
__device__ __forceinline__ float scaled_share(double w, double sum, const RouteArgs& a) {
    return (float)((a.renormalize ? (sum > 0.0 ? w / sum : 0.0) : w) * (double)a.scale);
}

__device__ __forceinline__ float exponential(float v) { return expf(v); }
__device__ __forceinline__ double exponential(double v) { return exp(v); }

template <w4a8_float TYPE>
__device__ __forceinline__ float load_logit(const void* row, int i) {
    if (TYPE == W4A8_FP32) return static_cast<const float*>(row)[i];
    const uint16_t h = static_cast<const uint16_t*>(row)[i];
    return TYPE == W4A8_FP16 ? f16_to_f32(h) : bf16_to_f32(h);
}

// NL: experts per lane.  S: type of the scores (double: the choice goes by them)
template <w4a8_float TYPE, int NL, typename S>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
    constexpr bool kByScore = sizeof(S) == 8;
    using Key = std::conditional_t<kByScore, uint64_t, uint32_t>;
    __shared__ double line[kByScore ? kRouteWaves : 1][kByScore ? 64 * NL : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t token = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (token >= a.tokens) return;   // whole waves; no barrier of the workgroup follows
    const void* row = static_cast<const uint8_t*>(a.logits) + token * a.ld * (TYPE == W4A8_FP32 ? 4 : 2);
    const float inf = __builtin_inff();
    float logit[NL];
    S p[NL];
    Key key[NL];
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane + 64 * i;
        const float v = e < a.experts ? load_logit<TYPE>(row, e) : -inf;
        logit[i] = v == v ? v : -inf;
        top = fmaxf(top, logit[i]);
    }
    S total = 1;
    if (a.score == W4A8_SCORE_SOFTMAX) {
        top = wave_reduce(top, Max());
        total = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // equal to the top, infinity included: 1; off: 0
            const S d = logit[i] == top ? S(0) : S(logit[i]) - S(top);
            p[i] = logit[i] > -inf ? exponential(d) : S(0);
            total += p[i];
        }
        total = wave_reduce(total, Add());
        if (!(total > 0)) total = 1;
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if constexpr (kByScore)
                p[i] = S(1) / (S(1) + exponential(-S(logit[i])));
            else
                p[i] = logit[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        if constexpr (kByScore) {
            if (a.score == W4A8_SCORE_SOFTMAX) p[i] = p[i] / total;
            const int e = lane + 64 * i;
            const double by = a.bias && e < a.experts ? p[i] + (double)a.bias[e] : p[i];
            key[i] = logit[i] > -inf ? key_of(by) : 0;
            if (a.groups > 1) line[wave][e] = key[i] ? by : -__builtin_inf();
        } else {
            key[i] = key_of(logit[i]);
        }
    }
    if constexpr (kByScore) {
        if (a.groups > 1) {
            // 2^by lanes to a group: its largest scores.  The wave's own lines: its LDS accesses are in order.
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int size = a.experts / a.groups, by = __builtin_clz(a.groups - 1) - 26;
            const int g = lane >> by;
            double first = -__builtin_inf(), second = first;
            if (g < a.groups)
#pragma unroll 4
                for (int i = lane & ((1 << by) - 1); i < size; i += 1 << by) {
                    const double v = line[wave][g * size + i];
                    second = fmax(second, fmin(first, v));
                    first = fmax(first, v);
                }
            for (int off = 1; off < 1 << by; off <<= 1) {
                const double f = __shfl_xor(first, off), t = __shfl_xor(second, off);
                second = fmax(fmin(first, f), fmax(second, t));
                first = fmax(first, f);
            }
            const double sum = a.group_top == 2 && size > 1 ? first + second : first;
            // a group with too few experts is behind all others
            const uint64_t group = sum > -__builtin_inf() ? key_of(sum) : 0;
            // its place: the groups that are better, or as good and before it
            int place = 0;
            for (int o = 0; o < a.groups; ++o) {
                const uint64_t other = lane_value(group, o << by);
                place += other > group || (other == group && o < g);
            }
            const uint64_t best = __ballot(g < a.groups && place < a.groups_kept);   // a group's first lane speaks for it
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int e = lane + 64 * i;
                if (e < a.experts && !((best >> ((e / size) << by)) & 1)) key[i] = 0;
            }
        }
    }
    int id = -1;
    S mine = 0, sum = 0;
    for (int j = 0; j < a.top_k; ++j) {
        int at = -1;
        S w = 0;
        if constexpr (kByScore) {
            // a lane's largest, of equals the lowest expert; the lane, and of several the one with the lowest expert
            Key best = 0;
            int held = 0;
            S value = 0;
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (key[i] > best) best = key[i], held = i, value = p[i];
            const uint64_t have = lanes_of_max(best);
            if (have == 0) break;   // the same in all lanes: nothing is left
            int from = __builtin_ctzll(have);
            if (have & (have - 1)) from = ~wave_max((have >> lane) & 1 ? ~(uint32_t)(64 * held + lane) : 0u) & 63;
            at = 64 * (int)lane_value((uint32_t)held, from) + from;
            w = lane_value(value, from);
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (lane == from && held == i) key[i] = 0;
        } else {
            // one reduction, then the lanes that hold it, for each held expert (the other way 3.2 us for one
            // token's eight of 128, this way 2.9 to 3.1)
            Key best = 0;
#pragma unroll
            for (int i = 0; i < NL; ++i) best = key[i] > best ? key[i] : best;
            best = wave_max(best);
            if (best == 0) break;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                if (at >= 0) continue;
                const uint64_t have = __ballot(key[i] == best);
                if (!have) continue;
                const int from = __builtin_ctzll(have);
                at = 64 * i + from;
                w = lane_value(p[i], from);
                if (lane == from) key[i] = 0;
            }
        }
        sum += w;
        if (lane == j) id = at, mine = w;
    }
    float weight;
    if (!kByScore && a.score == W4A8_SCORE_SIGMOID) {
        const double w = chosen_sigmoid(id, (float)mine);
        weight = scaled_share(w, wave_reduce(w, Add()), a);
    } else {
        if constexpr (!kByScore) mine = mine / total, sum = sum / total;
        if (a.renormalize) mine = sum > 0 ? mine / sum : S(0);
        weight = (float)(mine * S(a.scale));
    }
    if (lane < a.top_k) {
        a.ids[token * a.top_k + lane] = id;
        a.weights[token * a.top_k + lane] = weight;
    }
}

// Many tokens or few experts, where the choice goes by the logits: four tokens to a wave, 16 lanes each, lane L of
// them with the experts L, L + 16, ...; a round's instructions serve four tokens (16384 tokens, 8 of 128
// experts, one launch after another: 8.4 us, a wave per token 11.5, both bound by their instructions).
template <w4a8_float TYPE, int NL>
__global__ __launch_bounds__(64 * kRouteWaves) void route_rows_kernel(RouteArgs a) {
    const int sub = threadIdx.x & 15;
    const int64_t token = ((int64_t)blockIdx.x * (64 * kRouteWaves) + threadIdx.x) >> 4;
    const int64_t at = token < a.tokens ? token : a.tokens - 1;   // lanes past the last compute it again
    const void* row = static_cast<const uint8_t*>(a.logits) + at * a.ld * (TYPE == W4A8_FP32 ? 4 : 2);
    const float inf = __builtin_inff();
    float p[NL];
    uint32_t key[NL];
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = sub + 16 * i;
        const float v = e < a.experts ? load_logit<TYPE>(row, e) : -inf;
        p[i] = v == v ? v : -inf;
        key[i] = key_of(p[i]);
        top = fmaxf(top, p[i]);
    }
    float total = 1.0f;
    if (a.score == W4A8_SCORE_SOFTMAX) {
        top = row_reduce(top, Max());
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const float d = p[i] == top ? 0.0f : p[i] - top;
            p[i] = p[i] > -inf ? expf(d) : 0.0f;
            total += p[i];
        }
        total = row_reduce(total, Add());
        if (!(total > 0.0f)) total = 1.0f;
    }
    int id = -1;
    float mine = 0.0f, sum = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) best = max(best, key[i]);
        best = row_reduce(best, Max());
        // ~expert, the largest: the lowest expert of those that hold it; 0 for none
        uint32_t which = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) which = max(which, key[i] == best ? ~(uint32_t)(sub + 16 * i) : 0u);
        which = row_reduce(which, Max());
        float w = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (which == ~(uint32_t)(sub + 16 * i)) {
                key[i] = 0;
                w = p[i];
            }
        w = row_reduce(w, Add());   // of one lane (its logit, for a sigmoid), and zeros
        if (best == 0) w = 0.0f;
        sum += w;
        if (sub == j && best) id = (int)~which, mine = w;
    }
    if (a.score == W4A8_SCORE_SIGMOID) {
        const double q = chosen_sigmoid(id, mine);
        mine = scaled_share(q, row_reduce(q, Add()), a);
    } else {
        mine = mine / total, sum = sum / total;
        if (a.renormalize) mine = sum > 0.0f ? mine / sum : 0.0f;
        mine *= a.scale;
    }
    if (sub < a.top_k && token < a.tokens) {
        a.ids[token * a.top_k + sub] = id;
        a.weights[token * a.top_k + sub] = mine;
    }
}

// 16 lanes to a token hold up to 16 experts each, one after the other, where a wave holds 4: with more experts it takes more
// tokens than the CUs' waves for them to be ahead.  Time of 16 lanes over a wave's: up to 32 experts 0.80 to 0.97 for any tokens;
// 64 experts 1.02 to 1.04 for 1024 tokens, 0.97 to 1.02 for 2048, 0.54 to 0.63 for 16384; 128 1.15 for 1024, 1.00 to 1.06 for
// 3001, 0.91 to 0.99 for 4096, 0.72 to 0.74 for 16384; 256 1.3 for 1024, 1.05 for 4096, 0.91 to 0.93 for 8192.
bool by_rows(const RouteArgs& a) {
    return !a.bias && a.groups == 1 && a.experts <= 256 && a.top_k <= 16 &&
           (a.experts <= 32 || a.tokens >= (a.experts <= 64 ? 2048 : a.experts <= 128 ? 4096 : 8192));
}

template <w4a8_float TYPE>
hipError_t launch_rows(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.tokens + 4 * kRouteWaves - 1) / (4 * kRouteWaves))), block(64 * kRouteWaves);
#define W4A8_ROUTE(NL) hipLaunchKernelGGL((route_rows_kernel<TYPE, NL>), grid, block, 0, stream, a)
    if (a.experts <= 16) W4A8_ROUTE(1);
    else if (a.experts <= 32) W4A8_ROUTE(2);
    else if (a.experts <= 64) W4A8_ROUTE(4);
    else if (a.experts <= 128) W4A8_ROUTE(8);
    else W4A8_ROUTE(16);
#undef W4A8_ROUTE
    return hipGetLastError();
}

template <w4a8_float TYPE, typename S>
hipError_t launch_type(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.tokens + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
#define W4A8_ROUTE(NL) hipLaunchKernelGGL((route_kernel<TYPE, NL, S>), grid, block, 0, stream, a)
    if (a.experts <= 64) W4A8_ROUTE(1);
    else if (a.experts <= 128) W4A8_ROUTE(2);
    else if (a.experts <= 256) W4A8_ROUTE(4);
    else if (a.experts <= 512) W4A8_ROUTE(8);
    else W4A8_ROUTE(16);
#undef W4A8_ROUTE
    return hipGetLastError();
}

}  // namespace

int64_t moe_route_threads(const RouteArgs& a) { return (a.tokens + kRouteWaves - 1) / kRouteWaves * 64 * kRouteWaves; }

hipError_t launch_moe_route(const RouteArgs& a, w4a8_float type, hipStream_t stream) {
    const bool by_score = a.bias || a.groups > 1;
    if (by_rows(a))
        return type == W4A8_FP32   ? launch_rows<W4A8_FP32>(a, stream)
               : type == W4A8_FP16 ? launch_rows<W4A8_FP16>(a, stream)
                                   : launch_rows<W4A8_BF16>(a, stream);
    switch (type) {
        case W4A8_FP32: return by_score ? launch_type<W4A8_FP32, double>(a, stream) : launch_type<W4A8_FP32, float>(a, stream);
        case W4A8_FP16: return by_score ? launch_type<W4A8_FP16, double>(a, stream) : launch_type<W4A8_FP16, float>(a, stream);
        default: return by_score ? launch_type<W4A8_BF16, double>(a, stream) : launch_type<W4A8_BF16, float>(a, stream);
    }
}

}  // namespace w4a8
