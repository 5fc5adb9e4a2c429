// wave_ops.h -- reductions over a wavefront by lane swaps in registers.
//
// Four swaps (lanes ^ 1, ^ 2, the mirrored half row, the mirrored row) give every lane its
// row of 16's result; the four rows are then read as scalars.  About a dozen instructions,
// where six exchanges through LDS wait for each other.
#pragma once

#include "w4a8_internal.h"

namespace w4a8 {

template <int CTRL>
__device__ __forceinline__ uint32_t swap_lanes(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float swap_lanes(float v) {
    return __uint_as_float(swap_lanes<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double swap_lanes(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = swap_lanes<CTRL>((uint32_t)b), hi = swap_lanes<CTRL>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, lo | hi << 32);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) { return __uint_as_float(lane_value(__float_as_uint(v), lane)); }
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    return lane_value((uint32_t)v, lane) | (uint64_t)lane_value((uint32_t)(v >> 32), lane) << 32;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, v), lane));
}

// over each row of 16 lanes, in all of them
template <typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F f) {
    v = f(v, swap_lanes<0xB1>(v));
    v = f(v, swap_lanes<0x4E>(v));
    v = f(v, swap_lanes<0x141>(v));
    return f(v, swap_lanes<0x140>(v));
}
// over the wave, in all lanes
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, F f) {
    v = row_reduce(v, f);
    return f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
}
struct Add {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

}  // namespace w4a8
