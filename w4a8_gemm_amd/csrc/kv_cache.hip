// kv_cache.hip -- head norms with the position rotation, and the paged MXFP4
// KV cache: appending tokens' keys and values, reading rows back.
//
// A row is one head of one token, head_dim = 64, 128 or 256 values.  For
// queries and keys
//   x <- x * (mean(x^2) + eps)^-1/2 * w               (with a weight)
//   (a, b) <- (a c - b s, b c + a s)                  (the first `rot` values, in
//             pairs (i, i + rot/2), or (2i, 2i + 1) interleaved; c, s the token's
//             row of the table)
// then rounded to 16 bits (queries; keys outside the cache) or encoded like a
// weight: per 32 values the exponent of the ocp or noclip rule, codes to the
// nearest e2m1 value with ties to the even index.  Values are encoded as they
// come.  Cache layout: codes [pages][kv_heads][page][head_dim / 2], exponent
// bytes [pages][kv_heads][head_dim / 32][page]: a key's row is contiguous (an
// fp4 matrix operand's lane reads 16 bytes of it), and so are the exponents of
// neighbouring tokens for one 32-block.
//
// Queries are normed and turned in fp32.  Keys bound for the cache are normed
// and turned in fp64 and rounded once to fp32 before they are encoded: the code
// of a value next to the border of two codes then follows from the inputs
// alone, not from the order of fp32 operations.
#include "w4a8_internal.h"

#pragma clang fp contract(off)

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

template <bool FP16>
__device__ __forceinline__ float widen(uint32_t h) {
    return FP16 ? f16_to_f32(h) : bf16_to_f32(h);
}
template <bool FP16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (FP16) {
        const _Float16 x = (_Float16)a, y = (_Float16)b;
        return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
    } else {
        const __bf16 x = (__bf16)a, y = (__bf16)b;
        return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
    }
}

// sum over the GL lanes of a row
template <int GL, typename T>
__device__ __forceinline__ T row_sum(T v) {
#pragma unroll
    for (int off = GL / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// Lane L of a row's GL = D/8 lanes holds values 8L .. 8L+7.  rot is a multiple
// of 16, so a lane is inside or outside the rotated part as a whole, and the
// partner values of split pairs lie rot/16 lanes away.
template <int D, typename T>
__device__ __forceinline__ void norm_rotate(T (&x)[8], int L, const float* __restrict__ w, float eps,
                                            const float* __restrict__ cs, int rot, bool interleaved, bool bad_pos) {
    constexpr int GL = D / 8;
    if (w) {
        float wv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[j] = w[8 * L + j];
        T sq = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq += x[j] * x[j];
        const T ms = row_sum<GL>(sq) * (T)(1.0 / D) + (T)eps;
        const T r = sizeof(T) == 8 ? (T)rsqrt((double)ms) : (T)rsqrtf((float)ms);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * (T)wv[j];
    }
    if (rot == 0) return;
    const int half = rot >> 1;
    if (interleaved) {
        if (8 * L < rot) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T c = (T)cs[4 * L + j], s = (T)cs[half + 4 * L + j];
                const T a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * c - b * s;
                x[2 * j + 1] = b * c + a * s;
            }
        }
    } else {
        const int hl = rot >> 4;   // lanes of one half
        const bool first = L < hl;
        const int self = (int)(threadIdx.x & 63);
        const int from = first ? self + hl : (L < 2 * hl ? self - hl : self);
        T y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __shfl(x[j], from);
        if (8 * L < rot) {
            const int i = 8 * (first ? L : L - hl);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const T c = (T)cs[i + j], s = (T)cs[half + i + j];
                x[j] = first ? x[j] * c - y[j] * s : x[j] * c + y[j] * s;
            }
        }
    }
    // a position outside the table: NaN rather than some other token's angles
    if (bad_pos && 8 * L < rot) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (T)__builtin_nanf("");
    }
}

// Eight values of a 32-block (lanes 4i .. 4i+3 of the wave hold one block) ->
// their codes, and the block's exponent byte.  A block that holds a non-finite
// value is stored as NaN: byte 255, codes 0.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], int mode, uint32_t* e8m0) {
    uint32_t most = 0;   // magnitudes compared as integers: a NaN is above infinity
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    most = max(most, (uint32_t)__shfl_xor((int)most, 1));
    most = max(most, (uint32_t)__shfl_xor((int)most, 2));
    if (most >= 0x7F800000u) {
        *e8m0 = 255u;
        return 0u;
    }
    const int e = block_exponent(__uint_as_float(most), mode);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, normal: e <= 126
    uint32_t p = to_e2m1<0>(0u, v[0] * inv, v[1] * inv);
    p = to_e2m1<1>(p, v[2] * inv, v[3] * inv);
    p = to_e2m1<2>(p, v[4] * inv, v[5] * inv);
    p = to_e2m1<3>(p, v[6] * inv, v[7] * inv);
    *e8m0 = (uint32_t)(e + 127);
    return fold_neg_zero(p);
}

template <bool FP16, bool VEC>
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
    uint32_t d[4];
    if (VEC) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = widen<FP16>(d[j] & 0xFFFFu);
        x[2 * j + 1] = widen<FP16>(d[j] >> 16);
    }
}
template <bool FP16>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(narrow2<FP16>(x[0], x[1]), narrow2<FP16>(x[2], x[3]),
                                              narrow2<FP16>(x[4], x[5]), narrow2<FP16>(x[6], x[7]));
}

// One row per group of D/8 lanes, the rows of a token neighbours (queries, keys,
// values in this order), so that its table row is read once from memory.
template <int D, bool FP16, bool VEC>
__global__ __launch_bounds__(kThreads) void head_rows_kernel(const HeadRows a) {
    constexpr int GL = D / 8;
    const int L = threadIdx.x % GL;
    const uint32_t f = blockIdx.x * (uint32_t)(kThreads / GL) + threadIdx.x / GL;
    const uint32_t per = (uint32_t)(a.hq + a.hk + a.hv);
    const uint32_t token = f / per;
    int h = (int)(f - token * per);
    if (token >= (uint32_t)a.tokens) return;   // whole groups
    const int what = h < a.hq ? 0 : h < a.hq + a.hk ? 1 : 2;
    h -= what == 0 ? 0 : what == 1 ? a.hq : a.hq + a.hk;
    int64_t slot = 0;
    if (a.slots && what > 0) {
        slot = a.slots[token];
        if (slot < 0 || slot >= (a.cache.pages << a.page_shift)) return;   // padding
    }
    float x[8];
    const uint16_t* src = what == 0 ? a.q + token * a.q_st + h * a.q_sh
                          : what == 1 ? a.k + token * a.k_st + h * a.k_sh
                                      : a.v + token * a.v_st + h * a.v_sh;
    load8<FP16, VEC>(src + 8 * L, x);
    if (what < 2) {
        const float* w = what == 0 ? a.q_weight : a.k_weight;
        const float* cs = nullptr;
        bool bad = false;
        if (a.rot) {
            int64_t pos = a.positions[token];
            bad = pos < 0 || pos >= a.cs_rows;
            cs = a.cos_sin + (bad ? 0 : pos) * a.rot;
        }
        if (what == 1 && a.slots) {
            double y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (double)x[j];
            norm_rotate<D>(y, L, w, a.eps, cs, a.rot, a.interleaved, bad);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)y[j];
        } else {
            norm_rotate<D>(x, L, w, a.eps, cs, a.rot, a.interleaved, bad);
            uint16_t* out = what == 0 ? a.q_out + ((int64_t)token * a.hq + h) * D : a.k_out + ((int64_t)token * a.hk + h) * D;
            store8<FP16>(out + 8 * L, x);
            return;
        }
    }
    uint32_t e;
    const uint32_t codes = encode8(x, a.mode, &e);
    const int64_t page = slot >> a.page_shift;
    const int row = (int)(slot & ((1 << a.page_shift) - 1));
    const int64_t head = page * a.cache.kv_heads + h;
    uint8_t* cd = what == 1 ? a.cache.k_codes : a.cache.v_codes;
    uint8_t* ex = what == 1 ? a.cache.k_e8m0 : a.cache.v_e8m0;
    *reinterpret_cast<uint32_t*>(cd + ((head << a.page_shift) + row) * (D / 2) + 4 * L) = codes;
    if ((L & 3) == 0) ex[((head * (D / 32) + L / 4) << a.page_shift) + row] = (uint8_t)e;
}

// Rows of the cache as bf16 (exact: an e2m1 value has two significant bits);
// zeros where the slot is outside the cache.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(const w4a8_kv_cache c, int page_shift, int64_t tokens,
                                                           const int64_t* __restrict__ slots,
                                                           uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
    constexpr int GL = D / 8;
    const int L = threadIdx.x % GL;
    const uint32_t f = blockIdx.x * (uint32_t)(kThreads / GL) + threadIdx.x / GL;
    const uint32_t per = 2u * (uint32_t)c.kv_heads;
    const uint32_t token = f / per;
    if (token >= (uint32_t)tokens) return;
    const uint32_t r = f - token * per;
    const bool val = r >= (uint32_t)c.kv_heads;
    const int h = (int)(val ? r - c.kv_heads : r);
    const int64_t slot = slots[token];
    float x[8] = {};
    if (slot >= 0 && slot < (c.pages << page_shift)) {
        const int64_t head = (slot >> page_shift) * c.kv_heads + h;
        const int row = (int)(slot & ((1 << page_shift) - 1));
        const uint8_t* cd = val ? c.v_codes : c.k_codes;
        const uint8_t* ex = val ? c.v_e8m0 : c.k_e8m0;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(cd + ((head << page_shift) + row) * (D / 2) + 4 * L);
        const uint32_t e = ex[((head * (D / 32) + L / 4) << page_shift) + row];
        // 2^(e - 127): a subnormal at e = 0, NaN at 255
        const float s = e == 255u ? __builtin_nanf("") : e ? __uint_as_float(e << 23) : 0x1p-127f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t n = (w >> (4 * j)) & 15u;
            x[j] = (n & 8u ? -e2m1_mag(n & 7u) : e2m1_mag(n & 7u)) * s;
        }
    }
    uint16_t* out = (val ? v_out : k_out) + ((int64_t)token * c.kv_heads + h) * D + 8 * L;
    store8<false>(out, x);
}

template <int D>
hipError_t rows_dim(const HeadRows& a, bool fp16, bool vec, hipStream_t s) {
    constexpr int G = kThreads / (D / 8);
    const int64_t rows = a.tokens * (a.hq + a.hk + a.hv);
    const dim3 grid((unsigned)((rows + G - 1) / G));
    if (fp16) {
        if (vec) head_rows_kernel<D, true, true><<<grid, kThreads, 0, s>>>(a);
        else head_rows_kernel<D, true, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (vec) head_rows_kernel<D, false, true><<<grid, kThreads, 0, s>>>(a);
        else head_rows_kernel<D, false, false><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_head_rows(const HeadRows& a, bool fp16, hipStream_t stream) {
    // 16-byte loads where every row of every input starts on 16 bytes
    const auto vec16 = [](const uint16_t* p, int64_t st, int64_t sh) {
        return !p || (((uintptr_t)p | (uintptr_t)(2 * st) | (uintptr_t)(2 * sh)) & 15) == 0;
    };
    const bool vec = vec16(a.q, a.q_st, a.q_sh) && vec16(a.k, a.k_st, a.k_sh) && vec16(a.v, a.v_st, a.v_sh);
    switch (a.cache.head_dim) {
        case 64: return rows_dim<64>(a, fp16, vec, stream);
        case 128: return rows_dim<128>(a, fp16, vec, stream);
        default: return rows_dim<256>(a, fp16, vec, stream);
    }
}

hipError_t launch_kv_read(const w4a8_kv_cache& c, int page_shift, int64_t tokens, const int64_t* slots, uint16_t* k_out,
                          uint16_t* v_out, hipStream_t stream) {
    const int64_t rows = tokens * 2 * c.kv_heads;
    const int G = kThreads / (c.head_dim / 8);
    const dim3 grid((unsigned)((rows + G - 1) / G));
    switch (c.head_dim) {
        case 64: kv_read_kernel<64><<<grid, kThreads, 0, stream>>>(c, page_shift, tokens, slots, k_out, v_out); break;
        case 128: kv_read_kernel<128><<<grid, kThreads, 0, stream>>>(c, page_shift, tokens, slots, k_out, v_out); break;
        default: kv_read_kernel<256><<<grid, kThreads, 0, stream>>>(c, page_shift, tokens, slots, k_out, v_out); break;
    }
    return hipGetLastError();
}

}  // namespace w4a8
