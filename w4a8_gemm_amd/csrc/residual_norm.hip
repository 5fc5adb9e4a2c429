// residual_norm.hip -- the norms around a block, with its gate and residual sum,
// and the per-token fp8 codes of the result.
//
//   u = y [(mean y^2 + eps)^-1/2 post_weight] [gate]
//   r = residual + scale u                          (stored, rounded once)
//   h = r (mean r^2 + eps)^-1/2 weight              (16-bit values, and / or codes
//                                                    e4m3(h / s), s = max |h| / 448)
//
// Everything between the loads and the outputs stays in registers as fp32: a row
// is read once and each output written once, so rows in number are bound by HBM,
// a few rows by the launch and by the chain load -> sum -> sum -> max.  The codes
// come from h before its rounding to 16 bits: one rounding, and a scale that no
// 16-bit rounding of the largest value moves.
//
// A thread holds R runs of eight values, thread i the runs i, i + T, ... of its
// row's T threads.  T = 64: a wave per row, four rows to a workgroup, sums within
// the wave; else a workgroup per row whose waves join sums through LDS.  Rows need
// no alignment (16-byte loads at element alignment); the last, shorter run of a
// row whose length is no multiple of eight goes element by element.
#include "wave_ops.h"

#pragma clang fp contract(off)

namespace w4a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) Half8 { u32x4 d; };
struct __attribute__((packed, aligned(4))) Float4 { f32x4 v; };
struct __attribute__((packed, aligned(1))) Byte8 { u32x2 d; };

constexpr int kMaxWaves = 16;

template <bool FP16>
__device__ __forceinline__ float widen(uint16_t h) {
    return FP16 ? f16_to_f32(h) : bf16_to_f32(h);
}
template <bool FP16>
__device__ __forceinline__ uint16_t narrow(float f) {
    return (uint16_t)(FP16 ? pack_f16(f, 0.0f) : pack_bf16(f, 0.0f));
}
template <bool FP16>
__device__ __forceinline__ void widen8(u32x4 d, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = widen<FP16>((uint16_t)(d[j] & 0xFFFFu));
        x[2 * j + 1] = widen<FP16>((uint16_t)(d[j] >> 16));
    }
}

// Values [at, at + 8) of a row of n, zeros past its end.  The load is the same for all lanes, of a row's last
// eight where the run is shorter; those lanes shift it, so that no second load is waited for.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int at, int n) {
    if (n < 8) {   // the same for all threads
        u32x4 d = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (at + j < n) d[j >> 1] |= (uint32_t)row[at + j] << (16 * (j & 1));
        return d;
    }
    u32x4 d = reinterpret_cast<const Half8*>(row + min(at, n - 8))->d;
    const int past = at + 8 - n;
    if (past > 0) {
        uint64_t lo = d[0] | (uint64_t)d[1] << 32, hi = d[2] | (uint64_t)d[3] << 32;
        if (past >= 4) lo = hi, hi = 0;
        if (past >= 8) lo = 0;
        const int by = 16 * (past & 3);
        if (by) lo = lo >> by | hi << (64 - by), hi >>= by;
        d = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    return d;
}
__device__ __forceinline__ void load8(const float* row, int at, int n, float (&x)[8]) {
    if (n < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = at + j < n ? row[at + j] : 0.0f;
        return;
    }
    const float* from = row + min(at, n - 8);
    const f32x4 u = reinterpret_cast<const Float4*>(from)->v, v = reinterpret_cast<const Float4*>(from + 4)->v;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = u[j], x[4 + j] = v[j];
    const int past = at + 8 - n;
    if (past > 0) {
#pragma unroll
        for (int b = 1; b <= 4; b *= 2)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (past & b) x[j] = j + b < 8 ? x[j + b] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (past >= 8) x[j] = 0.0f;
    }
}
template <bool FP16>
__device__ __forceinline__ void store8(uint16_t* row, int at, int n, const float (&x)[8]) {
    if (at + 8 <= n) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = FP16 ? pack_f16(x[2 * j], x[2 * j + 1]) : pack_bf16(x[2 * j], x[2 * j + 1]);
        reinterpret_cast<Half8*>(row + at)->d = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at + j < n) row[at + j] = narrow<FP16>(x[j]);
}
__device__ __forceinline__ void store8(float* row, int at, int n, const float (&x)[8]) {
    if (at + 8 <= n) {
        reinterpret_cast<Float4*>(row + at)->v = f32x4{x[0], x[1], x[2], x[3]};
        reinterpret_cast<Float4*>(row + at + 4)->v = f32x4{x[4], x[5], x[6], x[7]};
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at + j < n) row[at + j] = x[j];
}
// e4m3 codes of eight values of magnitude up to 448 (a rounding error over it included)
__device__ __forceinline__ void store_codes(uint8_t* row, int at, int n, const float (&x)[8]) {
    u32x2 d;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * q], x[4 * q + 1], 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * q + 2], x[4 * q + 3], c, true);
        d[q] = (uint32_t)c;
    }
    if (at + 8 <= n) {
        reinterpret_cast<Byte8*>(row + at)->d = d;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at + j < n) row[at + j] = (uint8_t)(d[j >> 2] >> (8 * (j & 3)));
}

// sum (or, of magnitudes' bits, maximum) over a row's threads, zero for none; `part` is this
// reduction's own words of LDS
template <typename T, typename F>
__device__ __forceinline__ T threads_reduce(T v, F f, bool one_wave, T* part) {
    v = wave_reduce(v, f);
    if (one_wave) return v;
    const int waves = blockDim.x >> 6, lane = threadIdx.x & (kMaxWaves - 1);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return row_reduce(lane < waves ? part[lane] : T(0), f);
}

template <bool FP16, int R>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a, bool one_wave) {
    __shared__ float sums[2][kMaxWaves];
    __shared__ uint32_t tops[kMaxWaves];
    const int threads = one_wave ? 64 : blockDim.x, tid = one_wave ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = one_wave ? (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= a.tokens) return;   // whole waves, and no barrier follows where rows are waves
    const int n = a.hidden;
    const float over_n = 1.0f / (float)n;

    const uint16_t* y = a.y + row * a.ldy;
    u32x4 raw[R];
    float x[R][8], old[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = load8(y, 8 * (tid + i * threads), n);
    if (a.residual) {
        if (a.residual_fp32) {
            const float* p = static_cast<const float*>(a.residual) + row * a.ldr;
#pragma unroll
            for (int i = 0; i < R; ++i) load8(p, 8 * (tid + i * threads), n, old[i]);
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(a.residual) + row * a.ldr;
#pragma unroll
            for (int i = 0; i < R; ++i) widen8<FP16>(load8(p, 8 * (tid + i * threads), n), old[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) old[i][j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) widen8<FP16>(raw[i], x[i]);

    if (a.post_weight) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __builtin_fmaf(x[i][j], x[i][j], s);
        s = threads_reduce(s, Add(), one_wave, sums[0]);
        const float k = 1.0f / __builtin_sqrtf(s * over_n + a.eps);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float w[8];
            load8(a.post_weight, 8 * (tid + i * threads), n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = x[i][j] * k * w[j];
        }
    }
    if (a.gate) {
        const uint16_t* g = a.gate + row * a.gate_st;
        if (a.gate_sc) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float w[8];
                widen8<FP16>(load8(g, 8 * (tid + i * threads), n), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] *= w[j];
            }
        } else {
            const float w = widen<FP16>(g[0]);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] *= w;
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        // past the row's end everything is zero, unless a NaN scale of the row made it NaN
        const int left = n - 8 * (tid + i * threads);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[i][j] = j < left ? __builtin_fmaf(x[i][j], a.scale, old[i][j]) : 0.0f;
            s = __builtin_fmaf(x[i][j], x[i][j], s);
        }
    }
    if (a.residual_out) {
        if (a.residual_fp32) {
            float* p = static_cast<float*>(a.residual_out) + row * a.ldro;
#pragma unroll
            for (int i = 0; i < R; ++i) store8(p, 8 * (tid + i * threads), n, x[i]);
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.residual_out) + row * a.ldro;
#pragma unroll
            for (int i = 0; i < R; ++i) store8<FP16>(p, 8 * (tid + i * threads), n, x[i]);
        }
    }
    if (!a.out && !a.x8) return;

    s = threads_reduce(s, Add(), one_wave, sums[1]);
    const float k = 1.0f / __builtin_sqrtf(s * over_n + a.eps);
    uint32_t top = 0u;   // bits of |h|: NaN over infinity over the finite ones
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float w[8];
        const int at = 8 * (tid + i * threads);
        if (a.weight)
            load8(a.weight, at, n, w);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[i][j] = x[i][j] * k * w[j];
            if (at + j < n) top = max(top, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
        }
    }
    if (a.out) {
        uint16_t* p = a.out + row * n;
#pragma unroll
        for (int i = 0; i < R; ++i) store8<FP16>(p, 8 * (tid + i * threads), n, x[i]);
    }
    if (!a.x8) return;
    top = threads_reduce(top, Max(), one_wave, tops);
    // s = amax / 448, the codes by its reciprocal: below 2^-110 that would pass fp32
    const float amax = top == 0u ? 448.0f : __uint_as_float(max(top, __float_as_uint(0x1p-110f)));
    const float to_code = 448.0f / amax;
    if (tid == 0) a.xs[row] = amax / 448.0f;
    uint8_t* p = a.x8 + row * n;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= to_code;
        store_codes(p, 8 * (tid + i * threads), n, x[i]);
    }
}

struct NormShape {
    int threads, r;   // threads of a row (64: a wave, four rows to a workgroup) and runs of each
};
// Many rows: two runs to a thread (16384 rows of 5120: 106 us, with one 129, with four 111), but one where a
// row has no more than a wave's (16384 rows of 256: 15 us, with two 23).  Few rows wait for their latency:
// one run (a row of 5120: 3.5 us, with two 4.0).  Between, two runs take of one's time 1.00 to 1.12 at 512 rows, 0.85 to 1.09 at
// 1024 and 0.89 to 1.05 at 2048 (hidden 520 to 8192).  More where 16 waves are too few.
NormShape norm_shape(const NormArgs& a) {
    const int runs = (a.hidden + 7) / 8;
    int r = runs <= 64 || a.tokens < 1024 ? 1 : 2;
    while ((runs + 64 * r - 1) / (64 * r) > kMaxWaves) r *= 2;
    return {64 * ((runs + 64 * r - 1) / (64 * r)), r};
}

template <bool FP16, int R>
hipError_t launch_norm(const NormArgs& a, int threads, hipStream_t stream) {
    const bool one_wave = threads == 64;
    const int64_t groups = one_wave ? (a.tokens + 3) / 4 : a.tokens;
    hipLaunchKernelGGL((residual_norm_kernel<FP16, R>), dim3((unsigned)groups), dim3(one_wave ? 256 : threads), 0, stream, a,
                       one_wave);
    return hipGetLastError();
}
template <bool FP16>
hipError_t launch_norm_type(const NormArgs& a, hipStream_t stream) {
    const NormShape s = norm_shape(a);
    switch (s.r) {
        case 1: return launch_norm<FP16, 1>(a, s.threads, stream);
        case 2: return launch_norm<FP16, 2>(a, s.threads, stream);
        default: return launch_norm<FP16, 4>(a, s.threads, stream);
    }
}

}  // namespace

int64_t residual_norm_threads(const NormArgs& a) {
    const int threads = norm_shape(a).threads;
    return threads == 64 ? (a.tokens + 3) / 4 * 256 : a.tokens * threads;
}

hipError_t launch_residual_norm(const NormArgs& a, bool fp16, hipStream_t stream) {
    return fp16 ? launch_norm_type<true>(a, stream) : launch_norm_type<false>(a, stream);
}

}  // namespace w4a8
