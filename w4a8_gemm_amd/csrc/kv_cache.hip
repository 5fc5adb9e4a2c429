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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// eight 16-bit values at any 2-byte alignment (strided views of a fused
// projection may start anywhere): one 16-byte load either way
struct __attribute__((packed, aligned(2))) Half8 {
    u32x4 d;
};

template <bool FP16>
__device__ __forceinline__ void widen8(u32x4 d, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = FP16 ? f16_to_f32(d[j] & 0xFFFFu) : bf16_to_f32(d[j] & 0xFFFFu);
        x[2 * j + 1] = FP16 ? f16_to_f32(d[j] >> 16) : __uint_as_float(d[j] & 0xFFFF0000u);
    }
}
template <bool FP16>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = FP16 ? pack_f16(x[2 * j], x[2 * j + 1]) : pack_bf16(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<u32x4*>(p) = v;
}

// sum over the GL lanes of a row, in lanes' registers but for the last step
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ float swap16(float v) {
    return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), (0x10 << 10) | 0x1f));
}
__device__ __forceinline__ double swap16(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_swizzle((int)(uint32_t)b, (0x10 << 10) | 0x1f);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_swizzle((int)(uint32_t)(b >> 32), (0x10 << 10) | 0x1f);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
template <int GL, typename T>
__device__ __forceinline__ T row_sum(T v) {
    v += dpp<0xB1>(v);                       // lanes ^ 1
    v += dpp<0x4E>(v);                       // lanes ^ 2
    v += dpp<0x141>(v);                      // the mirrored half row: the other four of eight
    if (GL >= 16) v += dpp<0x140>(v);        // the mirrored row: the other eight of sixteen
    if (GL >= 32) v += swap16(v);
    return v;
}

// What a lane multiplies its values by: the weight, the rotation and its partner's.
//   y[j] = r (x[j] a[j] + x'[j] b[j]),   x' the pairs' other values, r the norm
// For first values a = w c, b = -w' s; for second ones a = w c, b = w' s; outside
// the rotation a = w, b = 0 and x' = 0.  Lane L of a row's GL = D/8 lanes holds
// values 8L .. 8L+7; rot is a multiple of 16, so a lane is inside or outside the
// rotation as a whole, and the partners of split pairs lie rot/16 lanes away.
template <typename T>
struct Factors {
    T a[8], b[8];
};
typedef float f32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(4))) Float4 {   // a 16-byte load at any 4-byte alignment
    f32x4 v;
};
__device__ __forceinline__ void load_floats(const float* p, float (&x)[8]) {
    const f32x4 u = reinterpret_cast<const Float4*>(p)[0].v, v = reinterpret_cast<const Float4*>(p)[1].v;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = u[j], x[4 + j] = v[j];
}
template <typename T>
__device__ __forceinline__ Factors<T> factors(int L, const float* __restrict__ w, const float* __restrict__ cs, int rot,
                                              bool interleaved, bool bad_pos) {
    Factors<T> f;
    const int half = rot >> 1;
    const bool in = 8 * L < rot, first = 8 * L < half;
    const int other = interleaved || !in ? L : first ? L + (rot >> 4) : L - (rot >> 4);
    float wa[8], wb[8], c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wa[j] = wb[j] = 1.0f;
    if (w) {
        load_floats(w + 8 * L, wa);
        load_floats(w + 8 * other, wb);
    }
    if (in) {
        if (interleaved) {
            const f32x4 u = reinterpret_cast<const Float4*>(cs + 4 * L)->v, v = reinterpret_cast<const Float4*>(cs + half + 4 * L)->v;
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = u[j / 2], s[j] = j & 1 ? v[j / 2] : -v[j / 2];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float t = wb[j];
                wb[j] = wb[j + 1], wb[j + 1] = t;
            }
        } else {
            const int i = 8 * (first ? L : other);
            load_floats(cs + i, c);
            load_floats(cs + half + i, s);
            if (first)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = -s[j];
        }
        if (bad_pos)   // rather than some other token's angles
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = __builtin_nanf("");
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f.a[j] = (T)wa[j] * (T)c[j];
        f.b[j] = (T)wb[j] * (T)s[j];
    }
    return f;
}

__device__ __forceinline__ float fma_t(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double fma_t(double a, double b, double c) { return fma(a, b, c); }

// A row: d the lane's eight values, p the pairs' other ones
template <int D, typename T, bool FP16>
__device__ __forceinline__ void turn_row(u32x4 d, u32x4 p, const Factors<T>& f, bool norm, float eps, float (&y)[8]) {
    float x[8], o[8];
    widen8<FP16>(d, x);
    widen8<FP16>(p, o);
    T r = 1;
    if (norm) {
        T sq = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fma_t((T)x[j], (T)x[j], sq);
        const T ms = row_sum<D / 8>(sq) * (T)(1.0 / D) + (T)eps;
        r = sizeof(T) == 8 ? (T)rsqrt((double)ms) : (T)rsqrtf((float)ms);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (float)(fma_t((T)x[j], f.a[j], (T)o[j] * f.b[j]) * r);
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

// A wave takes up to HPU heads of one kind (one cached key head: its fp64 work is
// the longest) of 64 / (D/8) neighbouring tokens, one token to a group of D/8
// lanes: the wave takes one path, the factors are made once for its heads, their
// loads are in flight together, and neighbouring tokens' exponent bytes are
// written together.  Bound by HBM from some thousand tokens on: 16384 tokens x 28 heads
// of 256 dims 87 us, 5.4 TB/s; the append of 16381 (24 / 4 heads) 102 us, where the
// cached keys' fp64 weighs too; a single token is the launch.
template <int HPU, bool CACHE>
struct Units {
    int q, k, v;
    __host__ __device__ Units(const HeadRows& a)
        : q((a.hq + HPU - 1) / HPU), k(CACHE ? a.hk : (a.hk + HPU - 1) / HPU), v((a.hv + HPU - 1) / HPU) {}
    __host__ __device__ int all() const { return q + k + v; }
};
constexpr int64_t token_blocks(int64_t tokens, int D) { return (tokens + 512 / D - 1) / (512 / D); }

template <int D, bool FP16, int HPU, bool CACHE>
__global__ __launch_bounds__(kThreads) void head_rows_kernel(const HeadRows a) {
    constexpr int GL = D / 8, TB = 64 / GL;
    const int lane = threadIdx.x & 63, L = lane % GL;
    const Units<HPU, CACHE> n(a);
    const uint32_t wave = blockIdx.x * (kThreads / 64) + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t block = wave / (uint32_t)n.all();
    const int u = (int)(wave - block * (uint32_t)n.all());
    const int64_t token = (int64_t)block * TB + lane / GL;
    if (token >= a.tokens) return;             // whole groups
    const int what = u < n.q ? 0 : u < n.q + n.k ? 1 : 2;
    const bool cached = CACHE && what > 0;
    const int per = CACHE && what == 1 ? 1 : HPU;
    const int h0 = per * (u - (what == 0 ? 0 : what == 1 ? n.q : n.q + n.k));
    const int count = min(per, (what == 0 ? a.hq : what == 1 ? a.hk : a.hv) - h0);
    int64_t slot = 0;
    if (cached) {
        slot = a.slots[token];
        if (slot < 0 || slot >= (a.cache.pages << a.page_shift)) return;   // padding
    }
    const int64_t sh = what == 0 ? a.q_sh : what == 1 ? a.k_sh : a.v_sh;
    const uint16_t* src = (what == 0 ? a.q + token * a.q_st : what == 1 ? a.k + token * a.k_st : a.v + token * a.v_st) + h0 * sh + 8 * L;
    u32x4 d[HPU];
#pragma unroll
    for (int i = 0; i < HPU; ++i)
        if (i < count) d[i] = reinterpret_cast<const Half8*>(src + i * sh)->d;

    const float* w = what == 0 ? a.q_weight : a.k_weight;
    const float* cs = nullptr;
    bool bad = false;
    if (a.rot && what < 2) {
        const int64_t pos = a.positions[token];
        bad = pos < 0 || pos >= a.cs_rows;
        cs = a.cos_sin + (bad ? 0 : pos) * a.rot;
    }
    // the pairs' other values: two to a dword, or those of the lane rot/16 away
    const int far = a.rot >> 4;
    const int from = 4 * (L < far ? lane + far : L < 2 * far ? lane - far : lane);
    const uint32_t in = 8 * L < a.rot ? ~0u : 0u;
    auto partner = [&](u32x4 v) {
        u32x4 p;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[j] = in & (a.interleaved ? (v[j] >> 16) | (v[j] << 16) : (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[j]));
        return p;
    };
    if (!CACHE || !cached) {
        const Factors<float> fa = factors<float>(L, w, cs, a.rot, a.interleaved, bad);
        uint16_t* out = (what == 0 ? a.q_out + ((int64_t)token * a.hq + h0) * D : a.k_out + ((int64_t)token * a.hk + h0) * D) + 8 * L;
#pragma unroll
        for (int i = 0; i < HPU; ++i)
            if (i < count) {
                float y[8];
                turn_row<D, float, FP16>(d[i], partner(d[i]), fa, w != nullptr, a.eps, y);
                store8<FP16>(out + i * D, y);
            }
        return;
    }
    const int64_t page = slot >> a.page_shift;
    const int row = (int)(slot & ((1 << a.page_shift) - 1));
    uint8_t* cd = what == 1 ? a.cache.k_codes : a.cache.v_codes;
    uint8_t* ex = what == 1 ? a.cache.k_e8m0 : a.cache.v_e8m0;
    auto put = [&](int i, const float (&x)[8]) {
        uint32_t e;
        const uint32_t codes = encode8(x, a.mode, &e);
        const int64_t head = page * a.cache.kv_heads + h0 + i;
        *reinterpret_cast<uint32_t*>(cd + ((head << a.page_shift) + row) * (D / 2) + 4 * L) = codes;
        if ((L & 3) == 0) ex[((head * (D / 32) + L / 4) << a.page_shift) + row] = (uint8_t)e;
    };
    if (what == 1) {
        const Factors<double> fa = factors<double>(L, w, cs, a.rot, a.interleaved, bad);
        float y[8];
        turn_row<D, double, FP16>(d[0], partner(d[0]), fa, w != nullptr, a.eps, y);
        put(0, y);
    } else {
#pragma unroll
        for (int i = 0; i < HPU; ++i)
            if (i < count) {
                float y[8];
                widen8<FP16>(d[i], y);
                put(i, y);
            }
    }
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

template <int D, int HPU>
hipError_t rows_go(const HeadRows& a, bool fp16, hipStream_t s) {
    const auto grid = [&](int units) {
        return dim3((unsigned)((token_blocks(a.tokens, D) * units + kThreads / 64 - 1) / (kThreads / 64)));
    };
    if (a.slots) {
        const dim3 g = grid(Units<HPU, true>(a).all());
        if (fp16) head_rows_kernel<D, true, HPU, true><<<g, kThreads, 0, s>>>(a);
        else head_rows_kernel<D, false, HPU, true><<<g, kThreads, 0, s>>>(a);
    } else {
        const dim3 g = grid(Units<HPU, false>(a).all());
        if (fp16) head_rows_kernel<D, true, HPU, false><<<g, kThreads, 0, s>>>(a);
        else head_rows_kernel<D, false, HPU, false><<<g, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}
// four heads to a wave where that still leaves every CU two workgroups (28 heads of 256
// dims, one and four: 512 tokens 6.1 and 6.2 us, 1024 tokens 9.7 and 9.2, 16384 tokens
// 129 and 87; appended with the read back 16381 tokens 247 and 121)
bool four_heads(const HeadRows& a) {
    const int64_t waves = token_blocks(a.tokens, a.cache.head_dim) * ((a.hq + 3) / 4 + (a.hk + 3) / 4 + (a.hv + 3) / 4);
    return waves >= (int64_t)device_cus() * 2 * (kThreads / 64);
}
template <int D>
hipError_t rows_dim(const HeadRows& a, bool fp16, hipStream_t s) {
    return four_heads(a) ? rows_go<D, 4>(a, fp16, s) : rows_go<D, 1>(a, fp16, s);
}

}  // namespace

int64_t head_rows_threads(const HeadRows& a) {
    const int units = four_heads(a) ? (a.slots ? Units<4, true>(a).all() : Units<4, false>(a).all())
                                    : (a.slots ? Units<1, true>(a).all() : Units<1, false>(a).all());
    return 64 * token_blocks(a.tokens, a.cache.head_dim) * units + kThreads;
}
int64_t kv_read_threads(const w4a8_kv_cache& c, int64_t tokens) {
    return tokens * 2 * c.kv_heads * (c.head_dim / 8) + kThreads;
}

hipError_t launch_head_rows(const HeadRows& a, bool fp16, hipStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: return rows_dim<64>(a, fp16, stream);
        case 128: return rows_dim<128>(a, fp16, stream);
        default: return rows_dim<256>(a, fp16, stream);
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
