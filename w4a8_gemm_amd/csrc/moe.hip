// moe.hip -- a mixture of experts' gated products on MXFP4 weights.
//
//   g, u = x W_up[e]^T (halves),  v = act(g) u,  out[t] = sum_j w[t, j] v[t, j] W_down[e]^T
//
// with up to some hundreds of tokens per expert: both products read each weight of the experts
// met, and are bound by that until units are full (8 experts, hidden 4096, inter 8192: their 428 MB
// take 69 us at 6.2 TB/s, the products of 502 slots 49 us at 1.4 PFLOP/s in bf16 and 10 at 3.2 in fp8).  The weights are in the
// fragment order of the prepared linears (gemm_prepared.hip), so a wave's 16-row tile of 128 k is one
// 1 KiB load.  The second product takes it as the e2m1 operand of one block-scaled 16x16x128 instruction, whose e4m3
// operand is 16 slots' v (a slot: token t, j); the first widens it and the slots' activations to bf16.
//
// Between the products v is held as e4m3 with a power of two per 32 values, which the matrix
// instruction takes as the operand's scale: a scale per token would need the maximum over
// all of inter, which no workgroup of the first product sees.
//
// Slots, at most 2048 at a time (more tokens: more chunks in the same launches), are listed by
// expert by every workgroup of the first product itself (2 to 4 us), which spares a launch and the
// wait for it, and read by the second's as the last one left them (1 us); runs of slots of one
// expert are the units of all kernels.  A unit's slots are the columns of its products; which
// column a slot takes has no influence on its result, but the kernel does, by roundings, and so
// do the sizes that choose it.
//
//                    up to 64 slots                          more
//   first product    up_kernel<true>, the list in registers  up_tile_kernel, the columns in LDS, or, with few
//                                                            items, up_kernel<false>, which splits K over waves
//   second product   down_kernel: a workgroup per 16         down_tile_kernel: a unit and 256 columns of the output
//                    columns has all slots' partial sums      to a workgroup, partial sums to device memory;
//                    in LDS and adds them                     join_kernel adds them (also for few slots, where
//                                                             inter is long and hidden short)
//
// The partial sums of a token are added in the order of j, K parts of a slot first: no atomics.
#include <math.h>

#include <type_traits>

#include "w4a8_internal.h"

namespace w4a8 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFmtFp8 = 0, kFmtFp4 = 4;
constexpr int kMaxExperts = 1024;
constexpr int kUpThreads = 512, kDownThreads = 1024;

__device__ __forceinline__ v8i frag_fp4(uint4 q) { return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0}; }
__device__ __forceinline__ v8i frag_fp8(u32x4 lo, u32x4 hi) {
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
// The second product's: scales in the low byte of each dword.  Here the instruction's cut (widen_fp8) is left as it is, as in the
// linears: no code is chosen by the sums, and 2^-14 of a step's largest product is under what bf16 shows of them
// (a token's error 0.00166 of its result, the rounding's).
__device__ __forceinline__ v4f product(v8i w, v8i x, v4f c, uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, kFmtFp4, kFmtFp8, 0, (int)sw, 0, (int)sx);
}

// ---------------------------------------------------------------------------
// slots by expert
// ---------------------------------------------------------------------------
struct alignas(16) MoePlan {
    uint16_t list[kMoeSlots];           // slots (of the chunk) by expert, in order
    uint32_t unit[kMoeSlots];           // first place | (slots - 1) << 11 | expert << 18
    float scale[2][64];                 // token scales of a unit's columns, of every other item
    uint32_t part[16];                  // of two sums over 512 threads
    int units;
};
// what the first product's last workgroup leaves of it for the second, in the workspace
struct alignas(16) StoredPlan {
    uint32_t unit[kMoeSlots];           // with the second product's slots to a unit
    uint16_t list[kMoeSlots];
    int units;
};
__device__ __forceinline__ int unit_first(uint32_t u) { return u & 2047; }
__device__ __forceinline__ int unit_slots(uint32_t u) { return ((u >> 11) & 127) + 1; }
__device__ __forceinline__ int unit_expert(uint32_t u) { return u >> 18; }

// lanes with the same id, which is in [0, experts) or -1: compared bit by bit over the wave
__device__ __forceinline__ uint64_t equal_lanes(int id, int experts) {
    const int bits = 32 - __builtin_clz(experts);   // 2^bits > experts: -1 is no other's low bits
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t on = __ballot((id >> b) & 1);
        same &= (id >> b) & 1 ? on : ~on;
    }
    return same;
}

// LDS that make_plan works in: how many slots of each 64 each expert has, and their first places
size_t plan_scratch(int64_t slots, int64_t experts) { return (size_t)(((slots + 63) / 64 + 2) * ((experts + 3) / 4 * 4)); }

// sum of v over the threads before this one, and over all NT; `part` is this sum's own words of LDS
template <int NT>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* part, uint32_t& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t incl = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t w = __shfl_up(incl, off);
        if (lane >= off) incl += w;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    uint32_t before = incl - v;
    all = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        const uint32_t w = part[i];
        if (i < wave) before += w;
        all += w;
    }
    return before;
}

// All NT threads; `slots` of the chunk, its ids; US: slots to a unit (at most 64).  Slots keep their
// order within an expert, so that all workgroups agree on the units: each wave ranks 64 slots
// by the equal ids before them, and the counts of the 64s are summed up for each expert.  No
// atomics.  `out`, where given: also for units of out_us slots.
template <int NT, int US>
__device__ void make_plan(MoePlan& p, uint8_t* scratch, const int32_t* ids, int slots, int experts, StoredPlan* out, int out_us) {
    constexpr int kPer = kMoeSlots / NT, kExp = kMaxExperts / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e4 = (experts + 3) / 4 * 4, lots = (slots + 63) / 64;
    uint8_t* count = scratch;                                          // [64 slots][expert]
    uint16_t* first = reinterpret_cast<uint16_t*>(scratch + lots * e4);
    int id[kPer], rank[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid + i * NT;
        id[i] = s < slots ? ids[s] : -1;
        if ((uint32_t)id[i] >= (uint32_t)experts) id[i] = -1;
    }
    for (int i = tid; i < lots * e4 / 4; i += NT) reinterpret_cast<uint32_t*>(count)[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int lot = wave + i * (NT / 64);
        if (lot >= lots) break;   // the same for the wave
        const uint64_t same = equal_lanes(id[i], experts);
        rank[i] = __popcll(same & ((1ull << lane) - 1));
        if (id[i] >= 0 && rank[i] == 0) count[lot * e4 + id[i]] = (uint8_t)__popcll(same);
    }
    __syncthreads();
    // an expert's counts, summed over the 64s before each, and exclusive sums over the experts of slots
    // (low half) and units (high half)
    uint32_t mine[kExp], sum = 0;
#pragma unroll
    for (int i = 0; i < kExp; ++i) {
        const int e = tid * kExp + i;
        uint32_t c = 0;
        if (e < experts)
            for (int l = 0; l < lots; ++l) c += count[l * e4 + e];
        mine[i] = c | ((c + US - 1) / US) << 16;
        sum += mine[i];
    }
    uint32_t all;
    uint32_t before = sum_before<NT>(sum, p.part, all);
    if (tid == 0) p.units = (int)(all >> 16);
    if (out) {   // the same for all threads
        uint32_t mine_out = 0;
#pragma unroll
        for (int i = 0; i < kExp; ++i) mine_out += ((mine[i] & 0xFFFFu) + out_us - 1) / out_us;
        uint32_t u = sum_before<NT>(mine_out, p.part + NT / 64, all), at = before & 0xFFFFu;
        if (tid == 0) out->units = (int)all;
#pragma unroll
        for (int i = 0; i < kExp; ++i) {
            const int c = mine[i] & 0xFFFFu;
            for (int k = 0; k < c; k += out_us, ++u)
                out->unit[u] = (at + k) | (uint32_t)(min(c - k, out_us) - 1) << 11 | (uint32_t)(tid * kExp + i) << 18;
            at += c;
        }
    }
#pragma unroll
    for (int i = 0; i < kExp; ++i) {
        const int e = tid * kExp + i, c = mine[i] & 0xFFFFu, at = before & 0xFFFFu;
        int u = before >> 16;
        if (e < experts) first[e] = (uint16_t)at;
        for (int k = 0; k < c; k += US, ++u)
            p.unit[u] = (uint32_t)(at + k) | (uint32_t)(min(c - k, US) - 1) << 11 | (uint32_t)e << 18;
        before += mine[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (id[i] < 0) continue;
        int at = first[id[i]] + rank[i];
        for (int l = 0; l < wave + i * (NT / 64); ++l) at += count[l * e4 + id[i]];
        p.list[at] = (uint16_t)(tid + i * NT);
    }
    __syncthreads();
    if (out)
        for (int i = tid; i < (slots + 1) / 2; i += NT) reinterpret_cast<uint32_t*>(out->list)[i] = reinterpret_cast<uint32_t*>(p.list)[i];
}

// the plan as the first product left it: read in one round, units to the most that there can be
template <int NT, int US>
__device__ void read_plan(MoePlan& p, const StoredPlan& from, int slots, int experts) {
    const int most = min(slots, experts + slots / US), lists = (slots + 7) / 8, units = (most + 3) / 4;
    const int i = threadIdx.x;
    uint4 list, unit;
    if (i < lists) list = reinterpret_cast<const uint4*>(from.list)[i];
    if (i < units) unit = reinterpret_cast<const uint4*>(from.unit)[i];
    if (i == 0) p.units = from.units;
    if (i < lists) reinterpret_cast<uint4*>(p.list)[i] = list;
    if (i < units) reinterpret_cast<uint4*>(p.unit)[i] = unit;
    __syncthreads();
}

// Up to 64 slots: every wave lists them in its registers, lane s holding slot s.  No LDS, no
// barrier, and the units come in the same order in every wave.
constexpr int kWaveSlots = 64;
struct WaveList {
    int id;              // the slot's expert, -1 if it has none
    int rank;            // how many slots of the same expert come before it
    uint64_t starts;     // slots that begin a unit of 16
    __device__ __forceinline__ int units() const { return __popcll(starts); }
};
__device__ __forceinline__ WaveList wave_list(const int32_t* ids, int slots, int experts) {
    const int lane = threadIdx.x & 63;
    const uint64_t before = (1ull << lane) - 1;
    WaveList r;
    r.id = lane < slots ? ids[lane] : -1;
    if ((uint32_t)r.id >= (uint32_t)experts) r.id = -1;
    r.rank = __popcll(equal_lanes(r.id, experts) & before);
    r.starts = __ballot(r.id >= 0 && (r.rank & 15) == 0);
    return r;
}
// A unit of up to 16 slots as a wave has it: lanes n, n + 16, ... have the slot of column n, those
// past cols the last one's
struct Unit {
    int expert, cols, slot;
};
__device__ __forceinline__ Unit wave_unit(const WaveList& l, int u) {
    const int lane = threadIdx.x & 63;
    const bool here = ((l.starts >> lane) & 1) && __popcll(l.starts & ((1ull << lane) - 1)) == u;
    const int at = __builtin_ctzll(__ballot(here));
    const int first = __builtin_amdgcn_readlane(l.rank, at);
    Unit r;
    r.expert = __builtin_amdgcn_readlane(l.id, at);
    const bool in = l.id == r.expert && l.rank >= first && l.rank < first + 16;
    r.cols = __popcll(__ballot(in));
    // each slot to the lane of its column (the others to lanes that are not read)
    const int got = __builtin_amdgcn_ds_permute(4 * (in ? l.rank - first : 16 + (lane & 15)), lane);
    r.slot = __builtin_amdgcn_ds_bpermute(4 * min(lane & 15, r.cols - 1), got);
    return r;
}
__device__ __forceinline__ Unit plan_unit(const MoePlan& p, int u) {
    const uint32_t v = uniform(p.unit[u]);
    const int cols = unit_slots(v);
    return {unit_expert(v), cols, p.list[unit_first(v) + min((int)(threadIdx.x & 15), cols - 1)]};
}

// n / d for n d < 2^32, by a product
struct Divisor {
    uint32_t d, m;
    Divisor() = default;
    explicit Divisor(int64_t by) : d((uint32_t)by), m(by > 1 ? (uint32_t)((1ull << 32) / (uint64_t)by + 1) : 0) {}
    __device__ __forceinline__ int quotient(int n) const { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }
    __device__ __forceinline__ int rest(int n, int q) const { return n - q * (int)d; }
};
struct MoeShape {
    int64_t tokens, hidden, inter;
    int experts, top_k, chunk;          // tokens of a chunk
    Divisor by_top_k;                   // a slot's token
    int h_steps, i_steps;               // 128-wide steps of hidden and inter
    int64_t e_stride;                   // exponent bytes of a slot of v: 16 per 4 steps, [step / 4][k / 32 % 4][step % 4]
    uint8_t *v, *ve;                    // v's codes [slots][inter] and exponents
};
struct UpArgs {
    MoeShape m;
    const uint8_t *w, *s, *x8;
    const float* xs;
    const int32_t* ids;
    int act, kw;
    Divisor by_blocks, by_kw;           // items of a unit; K parts
    int plan_at;                        // of the plan in LDS; before it the kernel's own, and the plan's making
    StoredPlan* plans;                  // of each chunk, for the second product
    int plan_slots;                     // to a unit of it
};
struct DownArgs {
    MoeShape m;
    const uint8_t *w, *s;
    const int32_t* ids;
    const float* weights;
    uint16_t* out;
    int rows;                           // of partial sums that LDS holds, the slots' weights after them
};
struct DownTileArgs {
    MoeShape m;
    const uint8_t *w, *s;
    const int32_t* ids;
    const float* weights;
    uint16_t* out;
    float* sums;
    int ks;                             // K parts
    Divisor by_items;                   // items of a unit: K parts x groups of columns, the parts first
    int plan_at;
    const StoredPlan* plans;
};

// ---------------------------------------------------------------------------
// up
// ---------------------------------------------------------------------------
// exp and 1 / x by the hardware's instructions, each within a unit in the last place: g to 2^6 comes out
// within 2^-17, and v is rounded to four bits
__device__ __forceinline__ float activated(float g, int act) {
    float z = g;
    if (act != W4A8_ACT_SILU) z = 1.5957691216057308f * (g + 0.044715f * g * g * g);   // (1 + tanh(z / 2)) / 2
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// The first product's operands are widened to bf16, exact as both are, and its products added in fp32
// by the bf16 instruction.  The e2m1 x e4m3 instruction that takes them as they are aligns its 128 products to
// the largest and cuts what lies 2^-14 below it.  That is far under what bf16 outputs show, but v is rounded to
// four bits next, and a value that the cut takes over the border of two codes moves by a whole step: a
// step of a large value is that token's error (up to 0.0135 of its result, 0.0018 with widened operands;
// 77 tokens, 3 of 32 experts, 640 x 384), and large products that cancel take the small ones with them.  It costs
// four instructions of half the time for one, and the conversions, which the weights' arrival hides but for full
// units (64 tokens, 8 of 128 experts, 2048 x 768: 63 us cut, 61 widened, with the empty column tiles left out;
// 251 tokens, 2 of 8, 4096 x 8192: 113 cut, 130 to 139 widened).
__device__ __forceinline__ v8bf widen_fp8(uint32_t a, uint32_t b) {
    const auto two = [](uint32_t codes, auto high) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, decltype(high)::value));
    };
    const u32x4 r = {two(a, std::false_type{}), two(a, std::true_type{}), two(b, std::false_type{}), two(b, std::true_type{})};
    return __builtin_bit_cast(v8bf, r);
}
// of the scale the conversion reads the exponent field alone: 2^(byte - 127), for byte 0 too
__device__ __forceinline__ v8bf widen_fp4(uint32_t codes, float scale) {
    const auto two = [&](auto at) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, decltype(at)::value));
    };
    const u32x4 r = {two(std::integral_constant<int, 0>{}), two(std::integral_constant<int, 1>{}),
                     two(std::integral_constant<int, 2>{}), two(std::integral_constant<int, 3>{})};
    return __builtin_bit_cast(v8bf, r);
}
// the exponent byte of step s % 4 of a scale dword, for widen_fp4
__device__ __forceinline__ float scale_at(uint32_t sc, int s) { return __uint_as_float(((sc >> (8 * (s & 3))) & 0xFFu) << 23); }
__device__ __forceinline__ v4f product_wide(v8bf w, v8bf x, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0); }

// Loads through a buffer resource: a scalar base and offset beside one vector offset, and zeros for
// offsets past its end.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kNowhere = 0x7FFFFFFF;   // past every resource's end
constexpr int kOnce = 2;                    // the non-temporal hint (load_stream16)

struct UpStep {
    u32x4 w[4];            // gate rows i0 .. +15 and +16 .. +31, then the up rows
    uint32_t s[4];
    u32x4 x[2];
};

// Four values of v of a lane, from the sums of a gate's and an up tile; the bits of the largest magnitude
struct Quad {
    float v[4];
    uint32_t top;
};
__device__ __forceinline__ Quad quad_of(const v4f& gate, const v4f& up, float sx, int act) {
    Quad q;
    q.top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q.v[i] = activated(sx * gate[i], act) * (sx * up[i]);
        q.top = max(q.top, __float_as_uint(q.v[i]) & 0x7FFFFFFFu);
    }
    return q;
}
// over the four lanes of a column
__device__ __forceinline__ uint32_t column_top(uint32_t top) {
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    return max(top, (uint32_t)__shfl_xor((int)top, 32));
}
// the block's exponent: the least e with top <= 448 2^e = 1.75 2^(e + 8), at least -127
__device__ __forceinline__ int block_power(uint32_t top) {
    return max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -127);
}
__device__ __forceinline__ void store_quad(const MoeShape& m, const Quad& q, uint32_t top, int64_t row, int at) {
    const float to_code = __uint_as_float((uint32_t)(127 - block_power(top)) << 23);   // 2^-e, -e <= 127
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[0] * to_code, q.v[1] * to_code, 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(q.v[2] * to_code, q.v[3] * to_code, c, true);
    *reinterpret_cast<int*>(m.v + row * m.inter + at) = top < 0x7F800000u ? c : 0x7F7F7F7F;
}
__device__ __forceinline__ void store_power(const MoeShape& m, uint32_t top, int64_t row, int blk) {
    // block blk: k / 32 % 4 = blk % 4 of step blk / 4
    m.ve[row * m.e_stride + (blk >> 4) * 16 + (blk & 3) * 4 + ((blk >> 2) & 3)] =
        top < 0x7F800000u ? (uint8_t)(block_power(top) + 127) : 255;
}
// v of 32 of inter (block blk) for 16 columns, from the sums of its four tiles: a lane has 4 values of each half
__device__ __forceinline__ void store_v(const MoeShape& m, const v4f (&r)[4], float sx, int act, int64_t row, int blk, int g,
                                        bool mine) {
    const Quad a = quad_of(r[0], r[2], sx, act), b = quad_of(r[1], r[3], sx, act);
    const uint32_t top = column_top(max(a.top, b.top));
    if (!mine) return;
    store_quad(m, a, top, row, 32 * blk + 4 * g);
    store_quad(m, b, top, row, 32 * blk + 16 + 4 * g);
    if (g == 0) store_power(m, top, row, blk);
}

// An item is a unit of 16 slots and 32 of inter, two tiles each of the gate's and the up rows, so that v's
// blocks of 32 are whole in a wave; kw waves share its K and are joined in LDS.  The columns are read from the
// cache as they are, gathered, no copy in LDS.
//
// WAVE: up to 64 slots, listed by every wave; else listed in LDS.  Bound by how many bytes a CU has under way:
// two steps of 5 KiB to a wave, two workgroups to a CU, of the registers that the widening leaves (one token
// of eight experts, hidden 2048, inter 768: 13.5 MB in 7.5 us, of which 3 are the start, the list and the first loads' way;
// eight tokens, 78.8 MB in 20.2 us, 3.9 TB/s).
template <bool WAVE>
__global__ __launch_bounds__(kUpThreads, 4) void up_kernel(UpArgs a) {
    constexpr int D = 2;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    MoePlan& p = *reinterpret_cast<MoePlan*>(lds + a.plan_at);
    v4f* join = reinterpret_cast<v4f*>(lds);   // [wave][tile][lane]
    const MoeShape& m = a.m;
    const int64_t t0 = (int64_t)blockIdx.y * m.chunk;
    const int tokens = (int)min((int64_t)m.chunk, m.tokens - t0), slots = tokens * m.top_k;
    WaveList list;
    if constexpr (WAVE)
        list = wave_list(a.ids, slots, m.experts);
    else
        make_plan<kUpThreads, 16>(p, lds, a.ids + t0 * m.top_k, slots, m.experts,
                                  blockIdx.x == gridDim.x - 1 ? a.plans + blockIdx.y : nullptr, a.plan_slots);

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int kw = a.kw, mine = a.by_kw.quotient(wave), part = wave - mine * kw, per_wg = 8 / kw;   // kw: 1, 2, 4 or 8
    const int blocks = (int)(m.inter / 32), items = (WAVE ? list.units() : p.units) * blocks;
    const int c_pad = (m.h_steps + 3) / 4;
    const int64_t tiles_i = m.inter / 16;
    const int s0 = m.h_steps * part / kw, s1 = m.h_steps * (part + 1) / kw;
    const __amdgpu_buffer_rsrc_t x = resource(a.x8 + t0 * m.hidden, (uint32_t)(tokens * m.hidden));
    for (int base = blockIdx.x * per_wg; base < items; base += gridDim.x * per_wg) {   // the same in all waves
        const bool live = base + mine < items;
        const int item = live ? base + mine : 0, of = a.by_blocks.quotient(item), blk = a.by_blocks.rest(item, of);
        const Unit u = WAVE ? wave_unit(list, of) : plan_unit(p, of);
        const int t = m.by_top_k.quotient(u.slot);
        const uint32_t xo = (uint32_t)t * (uint32_t)m.hidden + 32 * g;
        const float sx = a.xs[t0 + t];
        __amdgpu_buffer_rsrc_t wr[4], sr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t tile = (2 * u.expert + (q >> 1)) * tiles_i + 2 * blk + (q & 1);
            wr[q] = resource(a.w + tile * c_pad * 4096, c_pad * 4096);
            sr[q] = resource(a.s + tile * c_pad * 256, c_pad * 256);
        }
        v4f acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = v4f{0.f, 0.f, 0.f, 0.f};
        const auto load = [&](int s, UpStep& r) {
            r.x[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(x, xo, 128 * s, 0));
            r.x[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(x, xo + 16, 128 * s, 0));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r.s[q] = __builtin_amdgcn_raw_buffer_load_b32(sr[q], 4 * lane, (s >> 2) * 256, 0);
                r.w[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr[q], 16 * lane, s * 1024, kOnce));
            }
        };
        const auto compute = [&](int s, const UpStep& r) {
            // a lane's 32 k are those of its weights, 32 g to 32 g + 31 of the step
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4& from = r.x[i / 2];
                const v8bf c = widen_fp8(from[2 * (i & 1)], from[2 * (i & 1) + 1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = product_wide(widen_fp4(r.w[q][i], scale_at(r.s[q], s)), c, acc[q]);
            }
        };
        if (live) {
            UpStep ring[D];
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (s0 + d < s1) load(s0 + d, ring[d]);
            for (int s = s0; s < s1; s += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (s + d < s1) compute(s + d, ring[d]);
                    if (s + d + D < s1) load(s + d + D, ring[d]);
                }
            }
        }
        if (kw > 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q) join[(wave * 4 + q) * 64 + lane] = acc[q];
            __syncthreads();
        }
        if (live && part == 0) {
            if (kw > 1) {   // the parts in order, seven reads at a time
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v4f f[7];
#pragma unroll
                    for (int k = 1; k < 8; ++k) f[k - 1] = join[((wave + min(k, kw - 1)) * 4 + q) * 64 + lane];
#pragma unroll
                    for (int k = 1; k < 8; ++k)
                        if (k < kw) acc[q] += f[k - 1];
                }
            }
            store_v(m, acc, sx, a.act, t0 * m.top_k + u.slot, blk, g, n < u.cols);
        }
        if (kw > 1) __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------
struct DownStep {
    uint4 w;
    uint32_t s;
    u32x4 x[2];
    uint32_t e;
};

// Up to 64 slots.  A workgroup has 16 columns of the output and all slots: no partial sum leaves the CU, and no
// third launch is needed.  Its waves take the units, or K parts of them where units are few; six steps in
// flight.  Bound like the first product (one token of eight experts: 7.0 MB in 6.2 us; eight tokens:
// 40.6 MB in 16.5 us, as the 128 workgroups of hidden 2048 fill half the CUs).
__global__ __launch_bounds__(kDownThreads) void down_kernel(DownArgs a) {
    constexpr int D = 6, kWaves = kDownThreads / 64;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const MoeShape& m = a.m;
    const int tokens = (int)m.tokens, slots = tokens * m.top_k;
    // LDS: partial sums [slot][K part][16 columns], the slots' weights
    float4* part = reinterpret_cast<float4*>(lds);
    const float* lds_sums = reinterpret_cast<const float*>(lds);
    float* share = reinterpret_cast<float*>(lds + (size_t)a.rows * 64);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const WaveList list = wave_list(a.ids, slots, m.experts);
    const int units = list.units();
    int ks = 1;   // K parts: as many as give every wave one, while there are few units
    while (2 * ks * units <= kWaves && 2 * ks * slots <= a.rows && 2 * ks <= min(kWaves, m.i_steps)) ks *= 2;
    // slots without an expert add nothing
    if ((int)threadIdx.x < slots) {
        share[lane] = list.id >= 0 ? a.weights[lane] : 0.0f;
        if (list.id < 0)
            for (int k = 0; k < 4 * ks; ++k) part[4 * lane * ks + k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int c_pad = (m.i_steps + 3) / 4;
    for (int item = wave; item < units * ks; item += kWaves) {
        const int k = item % ks;
        const Unit u = wave_unit(list, item / ks);
        const int64_t tile = u.expert * (m.hidden / 16) + blockIdx.x;
        const uint8_t* wp = a.w + tile * c_pad * 4096;
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(a.s) + tile * c_pad * 64;
        const uint32_t xo = (uint32_t)u.slot * (uint32_t)m.inter + 16 * g, eo = (uint32_t)u.slot * (uint32_t)m.e_stride + 4 * g;
        v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
        const auto load = [&](int s, DownStep& r) {
            r.w = load_stream16(reinterpret_cast<const uint4*>(wp + s * 1024) + lane);
            r.s = (sp + (s >> 2) * 64)[lane];
            r.x[0] = *reinterpret_cast<const u32x4*>(m.v + 128 * s + xo);
            r.x[1] = *reinterpret_cast<const u32x4*>(m.v + 128 * s + 64 + xo);
            r.e = *reinterpret_cast<const uint32_t*>(m.ve + (s >> 2) * 16 + eo);
        };
        const auto compute = [&](int s, const DownStep& r) {
            acc = product(frag_fp4(r.w), frag_fp8(r.x[0], r.x[1]), acc, r.s >> (8 * (s & 3)), r.e >> (8 * (s & 3)));
        };
        const int s0 = m.i_steps * k / ks, s1 = m.i_steps * (k + 1) / ks;
        DownStep ring[D];
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            if (s0 + d < s1) load(s0 + d, ring[d]);
        for (int s = s0; s < s1; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d + D - 1 < s1) load(s + d + D - 1, ring[(d + D - 1) % D]);
                if (s + d < s1) compute(s + d, ring[d]);
            }
        }
        if (n < u.cols) part[(u.slot * ks + k) * 4 + g] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
    __syncthreads();
    // a column of a token to a thread: its slots in order, eight reads at a time
    if ((int)threadIdx.x < 16 * tokens) {
        const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
        const float* sums = lds_sums + c;
        float sum = 0.0f;
        for (int j0 = 0; j0 < m.top_k; j0 += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            for (int k = 0; k < ks; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += sums[16 * ((t * m.top_k + min(j0 + j, m.top_k - 1)) * ks + k)];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < m.top_k) sum = __builtin_fmaf(share[t * m.top_k + j0 + j], v[j], sum);
        }
        a.out[(int64_t)t * m.hidden + 16 * blockIdx.x + c] = (uint16_t)pack_bf16(sum, 0.0f);
    }
}

// ---------------------------------------------------------------------------
// both products with the columns in LDS
// ---------------------------------------------------------------------------
// A workgroup takes a unit and eight waves' worth of weight rows; the unit's columns (up to
// 16 MT) are staged for all eight in LDS, 512 k (a chunk of the scales) at a time, two
// buffers.  A wave's weights of D steps are in flight: each step's registers are
// asked for again, D steps on, as soon as its products are issued, and the next chunk's
// columns are asked for before them, so that waiting for those leaves the weights in flight.
// Every step of a chunk is computed: past K the columns are zeros, and the weights those of the
// last step.  The first product, which widens its operands, takes a unit's own column tiles (1, 2 or 4) by code of
// their own; the second all MT: those without slots cost products that the weights' arrival
// hides, conditions on them cost copies of the sums.
constexpr int kTileThreads = 512;
constexpr int kUpColumns = 64;      // of the first product's units

template <int OPSEL>
__device__ __forceinline__ v4f product_at(v8i w, v8i x, v4f c, uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, kFmtFp4, kFmtFp8, OPSEL, (int)sw, OPSEL, (int)sx);
}
// 16-byte pieces of a column's 512, swapped within 256 by the column, so that the 16 columns of a
// read meet all banks
__device__ __forceinline__ int piece(int column, int c) { return column * 512 + 16 * (c ^ (column & 15)); }

template <int MT>
struct Stage {                 // what a thread brings of a chunk: piece tid % 32 of the columns tid / 32 + 16 i
    u32x4 r[MT];
    static __device__ __forceinline__ int column(int i) { return (int)threadIdx.x / 32 + 16 * i; }
    // row: the columns' offsets from x, kNowhere past the last; width of a row in bytes
    template <int I0 = 0, int I1 = MT>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, const uint32_t (&row)[MT], int chunk, int width) {
        const int c = 16 * (threadIdx.x % 32), at = chunk * 512;
#pragma unroll
        for (int i = I0; i < I1; ++i)
            r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(x, at + c < width ? row[i] + c : kNowhere, at, 0));
    }
    // the first chunk, with zeros past the unit's last column in both buffers: their products cost least
    __device__ __forceinline__ void store_first(uint8_t* to, uint8_t* other, int cols) const {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int at = piece(column(i), threadIdx.x % 32);
            *reinterpret_cast<u32x4*>(to + at) = r[i];
            if (column(i) >= cols) *reinterpret_cast<u32x4*>(other + at) = r[i];
        }
    }
    template <int I0 = 0, int I1 = MT>
    __device__ __forceinline__ void store(uint8_t* to, int cols) const {
#pragma unroll
        for (int i = I0; i < I1; ++i)
            if (column(i) < cols) *reinterpret_cast<u32x4*>(to + piece(column(i), threadIdx.x % 32)) = r[i];
    }
};
// Where a lane finds its two pieces of step s of column 16 j + n: pieces 8 s + g and 8 s + 4 + g, whose
// swap leaves four addresses, and constants beside them.
struct ColumnReader {
    int at[4];
    __device__ __forceinline__ ColumnReader() {
        const int n = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = n * 512 + 16 * ((g ^ n) ^ (4 * i));
    }
    __device__ __forceinline__ v8i read(const uint8_t* from, int j, int s) const {
        const int more = 16 * 512 * j + 256 * (s >> 1), i = 2 * (s & 1);
        return frag_fp8(*reinterpret_cast<const u32x4*>(from + at[i] + more),
                        *reinterpret_cast<const u32x4*>(from + at[i + 1] + more));
    }
};
// f(integral_constant<int, 0>) .. <3>: the steps of a chunk
template <typename F>
__device__ __forceinline__ void each_step(F f) {
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
}

// a slot's exponents of the four steps from `quad`'s; past K, where none were written, 2^0
__device__ __forceinline__ u32x4 exponents(const uint8_t* row, int quad, int steps) {
    u32x4 e = *reinterpret_cast<const u32x4*>(row + 16 * quad);
    const int left = steps - 4 * quad;
    if (left < 4) {
        const uint32_t keep = (1u << (8 * left)) - 1;
#pragma unroll
        for (int g = 0; g < 4; ++g) e[g] = (e[g] & keep) | (0x7F7F7F7Fu & ~keep);
    }
    return e;
}

// The sums as they stand here: without it the compiler moves a step's products behind the loads
// that are to take their operands' registers.
template <int Q, int MT>
__device__ __forceinline__ void hold(v4f (&acc)[Q][MT]) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int j = 0; j < MT; ++j) asm volatile("" : "+v"(acc[q][j]));
}

// Two weight tiles of a wave: codes of D steps (2 or 4) and scale dwords of a chunk
template <int D, int HINT>
struct Tiles {
    __amdgpu_buffer_rsrc_t w[2], s[2];
    uint4 q[D][2];
    uint32_t sc[2], next[2];
    __device__ __forceinline__ void at(int r, const uint8_t* wt, const uint8_t* st, int64_t tile, int c_pad) {
        w[r] = resource(wt + tile * c_pad * 4096, c_pad * 4096);
        s[r] = resource(st + tile * c_pad * 256, c_pad * 256);
    }
    __device__ __forceinline__ void load(int step, int to) {   // to: step % D
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int r = 0; r < 2; ++r)
            q[to][r] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(w[r], 16 * lane, step * 1024, HINT));
    }
    __device__ __forceinline__ void load_scales(int chunk) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int r = 0; r < 2; ++r) next[r] = __builtin_amdgcn_raw_buffer_load_b32(s[r], 4 * lane, chunk * 256, 0);
    }
    // of the chunk that was asked for; then the next one's asked for
    __device__ __forceinline__ void take_scales() {
#pragma unroll
        for (int r = 0; r < 2; ++r) sc[r] = next[r];
    }
};

// Where a lane finds eight of its k, from 32 g + 8 i on, of step s of column 16 j + n, for the bf16 products: in piece
// 8 s + 2 g + i / 2.
struct WideReader {
    int at[4];
    __device__ __forceinline__ WideReader() {
        const int n = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = n * 512 + 16 * ((2 * g + (i & 1) + 8 * (i >> 1)) ^ n);
    }
    __device__ __forceinline__ uint2 read(const uint8_t* from, int j, int s, int i) const {
        return *reinterpret_cast<const uint2*>(from + at[2 * (s & 1) + i / 2] + 16 * 512 * j + 256 * (s >> 1) + 8 * (i & 1));
    }
};

// An item of the first product: the unit's NT column tiles.  A wave has 16 of inter, a tile each of the gate's and the up
// rows, and the waves of a pair agree on their block's largest value through LDS.
template <int NT, int HINT>
__device__ __forceinline__ void up_item(const UpArgs& a, const MoePlan& p, uint8_t* lds, float* scale, __amdgpu_buffer_rsrc_t x,
                                        int64_t t0, uint32_t u, int blk) {
    constexpr int kBuf = kUpColumns * 512, D = 2;   // steps of weights in flight
    const MoeShape& m = a.m;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const WideReader cr;
    const int first = unit_first(u), cols = unit_slots(u), steps = m.h_steps, chunks = (steps + 3) / 4;
    const int64_t tiles_i = m.inter / 16;
    Stage<NT> st;
    uint32_t row[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int col = st.column(i);
        row[i] = col < cols ? (uint32_t)m.by_top_k.quotient(p.list[first + col]) * (uint32_t)m.hidden : kNowhere;
    }
    st.load(x, row, 0, (int)m.hidden);
    float sx = 0.0f;
    if ((int)threadIdx.x < cols) sx = a.xs[t0 + m.by_top_k.quotient(p.list[first + threadIdx.x])];
    Tiles<D, HINT> w;
#pragma unroll
    for (int q = 0; q < 2; ++q) w.at(q, a.w, a.s, (2 * unit_expert(u) + q) * tiles_i + blk, chunks);
    w.load_scales(0);
#pragma unroll
    for (int s = 0; s < D; ++s) w.load(min(s, steps - 1), s);
    v4f acc[2][NT];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[q][j] = v4f{0.f, 0.f, 0.f, 0.f};
    st.store_first(lds, lds + kBuf, cols);
    if ((int)threadIdx.x < cols) scale[threadIdx.x] = sx;
    __syncthreads();
    const auto products = [&](const uint8_t* buf, auto step) {
        constexpr int s = decltype(step)::value;
        float sw[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) sw[q] = scale_at(w.sc[q], s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // eight of a lane's 32 k
            v8bf wide[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) wide[q] = widen_fp4((&w.q[s % D][q].x)[i], sw[q]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint2 codes = cr.read(buf, j, s, i);
                const v8bf b = widen_fp8(codes.x, codes.y);
#pragma unroll
                for (int q = 0; q < 2; ++q) acc[q][j] = product_wide(wide[q], b, acc[q][j]);
                __builtin_amdgcn_sched_barrier(0);   // no more than a tile's columns in registers
            }
        }
    };
    for (int c = 0; c + 1 < chunks; ++c) {
        w.take_scales();
        w.load_scales(c + 1);
        each_step([&](auto step) {
            constexpr int s = decltype(step)::value;
            // half of the next chunk's columns at a time, for the registers
            if constexpr (s == 0) st.template load<0, (NT + 1) / 2>(x, row, c + 1, (int)m.hidden);
            if constexpr (s == 2) st.template load<(NT + 1) / 2, NT>(x, row, c + 1, (int)m.hidden);
            __builtin_amdgcn_sched_barrier(0);
            products(lds + (c & 1) * kBuf, step);
            hold(acc);
            __builtin_amdgcn_sched_barrier(0);
            w.load(min(4 * c + s + D, steps - 1), s % D);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (s == 1) st.template store<0, (NT + 1) / 2>(lds + ((c + 1) & 1) * kBuf, cols);
            if constexpr (s == 3) st.template store<(NT + 1) / 2, NT>(lds + ((c + 1) & 1) * kBuf, cols);
            __builtin_amdgcn_sched_barrier(0);
        });
        __syncthreads();
    }
    w.take_scales();
    each_step([&](auto step) {
        constexpr int s = decltype(step)::value;
        products(lds + ((chunks - 1) & 1) * kBuf, step);
        hold(acc);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (s + D < 4) w.load(min(4 * (chunks - 1) + s + D, steps - 1), s % D);
    });
    __syncthreads();   // before the next item's first columns
    uint32_t* tops = reinterpret_cast<uint32_t*>(lds);   // [wave][column]
    Quad v[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        v[j] = quad_of(acc[0][j], acc[1][j], scale[16 * j + n], a.act);
        v[j].top = column_top(v[j].top);
        if (g == 0) tops[wave * 16 * NT + 16 * j + n] = v[j].top;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const uint32_t top = max(v[j].top, tops[(wave ^ 1) * 16 * NT + 16 * j + n]);
        if (16 * j + n >= cols) continue;
        const int64_t at = t0 * m.top_k + p.list[first + 16 * j + n];
        store_quad(m, v[j], top, at, 16 * blk + 4 * g);
        if (g == 0 && !(wave & 1)) store_power(m, top, at, blk >> 1);
    }
    __syncthreads();
}

// Units of up to 64 slots and 128 of inter to a workgroup, whose waves are all live (inter is a multiple of 128).  Sums of
// two times four tiles, two steps of weights and half a chunk's columns fill the 128 registers that two
// workgroups to a CU leave a wave.  64 tokens of 8 in 128 experts, hidden 2048, inter 768: 179 MB in 35.0 us, 5.1 TB/s; 251 tokens
// of 2 in 8, hidden 4096, inter 8192: 383 MB (some experts have two units) in 85 us, 4.5 TB/s, the matrix pipe a third
// and the vector pipe a quarter of the time: waves wait for columns, weights and each other in turn, which neither more
// weights in flight nor columns widened once on their way to LDS change much (131 for 134 us of the call; 64 tokens 62 for 60).
template <int HINT>
__global__ __launch_bounds__(kTileThreads, 4) void up_tile_kernel(UpArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    MoePlan& p = *reinterpret_cast<MoePlan*>(lds + a.plan_at);
    const MoeShape& m = a.m;
    const int64_t t0 = (int64_t)blockIdx.y * m.chunk;
    const int tokens = (int)min((int64_t)m.chunk, m.tokens - t0), slots = tokens * m.top_k;
    make_plan<kTileThreads, kUpColumns>(p, lds, a.ids + t0 * m.top_k, slots, m.experts,
                                        blockIdx.x == gridDim.x - 1 ? a.plans + blockIdx.y : nullptr, a.plan_slots);

    const int items = p.units * (int)(m.inter / 128);
    const __amdgpu_buffer_rsrc_t x = resource(a.x8 + t0 * m.hidden, (uint32_t)(tokens * m.hidden));
    float* scale = p.scale[1];
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        scale = p.scale[scale == p.scale[1] ? 0 : 1];   // a slow wave may still read the last item's
        const int of = a.by_blocks.quotient(item), blk = a.by_blocks.rest(item, of) * 8 + uniform(threadIdx.x >> 6);
        const uint32_t u = uniform(p.unit[of]);
        const int tiles = (unit_slots(u) + 15) / 16;   // the same for all threads
        if (tiles == 1)
            up_item<1, HINT>(a, p, lds, scale, x, t0, u, blk);
        else if (tiles == 2)
            up_item<2, HINT>(a, p, lds, scale, x, t0, u, blk);
        else
            up_item<4, HINT>(a, p, lds, scale, x, t0, u, blk);
    }
}

// The second product's share of K part k of every slot, to partial sums [K part][slot][hidden] in
// device memory: fp32, as the sum over the slots that follows is of terms of both signs.  A wave has two tiles of
// output columns.  64 tokens of 8 in 128 experts, hidden 2048, inter 768: 95.9 MB in 20.8 us, 4.6 TB/s; 251
// tokens of 2 in 8, hidden 4096, inter 8192: 177 MB in 40.4 us, 4.4 TB/s.
template <int MT, int D, int WAVES, int HINT>
__global__ __launch_bounds__(kTileThreads, WAVES) void down_tile_kernel(DownTileArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int kCols = 16 * MT * 512, kBuf = kCols + 16 * MT * 16;   // columns, then their exponents
    MoePlan& p = *reinterpret_cast<MoePlan*>(lds + a.plan_at);
    const MoeShape& m = a.m;
    const int64_t t0 = (int64_t)blockIdx.y * m.chunk;
    const int tokens = (int)min((int64_t)m.chunk, m.tokens - t0), slots = tokens * m.top_k;
    read_plan<kTileThreads, 16 * MT>(p, a.plans[blockIdx.y], slots, m.experts);

    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const ColumnReader cr;
    const int tiles = (int)(m.hidden / 16), groups = (tiles + 15) / 16, items = p.units * groups * a.ks;
    const int steps = m.i_steps, chunks = (steps + 3) / 4;
    const __amdgpu_buffer_rsrc_t x = resource(m.v + t0 * m.top_k * m.inter, (uint32_t)(slots * m.inter));
    const uint8_t* xe = m.ve + t0 * m.top_k * m.e_stride;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int of = a.by_items.quotient(item), rest = a.by_items.rest(item, of);
        const int k = rest & (a.ks - 1), grp = rest >> (31 - __builtin_clz(a.ks));   // ks: a power of two
        const uint32_t u = uniform(p.unit[of]);
        const int first = unit_first(u), cols = unit_slots(u), tile = grp * 16 + 2 * wave;
        const bool live = tile < tiles;   // tiles are even; a wave past the last pair computes that one again
        const int c0 = chunks * k / a.ks, c1 = chunks * (k + 1) / a.ks;
        Stage<MT> st;
        uint32_t row[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int col = st.column(i);
            row[i] = col < cols ? (uint32_t)p.list[first + col] * (uint32_t)m.inter : kNowhere;
        }
        const bool has_e = (int)threadIdx.x < cols;
        const uint8_t* ep = xe + (uint32_t)p.list[first + min((int)threadIdx.x, cols - 1)] * (uint32_t)m.e_stride;
        u32x4 er{};
        st.load(x, row, c0, (int)m.inter);
        if (has_e) er = exponents(ep, c0, steps);
        Tiles<D, HINT> w;
#pragma unroll
        for (int q = 0; q < 2; ++q) w.at(q, a.w, a.s, (int64_t)unit_expert(u) * tiles + (live ? tile : tiles - 2) + q, chunks);
        w.load_scales(c0);
#pragma unroll
        for (int s = 0; s < D; ++s) w.load(min(4 * c0 + s, steps - 1), s);
        v4f acc[2][MT];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[q][j] = v4f{0.f, 0.f, 0.f, 0.f};
        const auto put_e = [&](uint8_t* to) {
            if (has_e) *reinterpret_cast<u32x4*>(to + kCols + 16 * threadIdx.x) = er;
        };
        st.store_first(lds, lds + kBuf, cols);
        put_e(lds);
        __syncthreads();
        uint32_t e[MT];
        const auto read_e = [&](const uint8_t* buf) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
                e[j] = *reinterpret_cast<const uint32_t*>(buf + kCols + 16 * (16 * j + n) + 4 * g);
        };
        const auto products = [&](const uint8_t* buf, auto step) {
            constexpr int s = decltype(step)::value;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const v8i b = cr.read(buf, j, s);
#pragma unroll
                for (int q = 0; q < 2; ++q) acc[q][j] = product_at<s>(frag_fp4(w.q[s % D][q]), b, acc[q][j], w.sc[q], e[j]);
                if (j % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
        };
        for (int c = c0; c + 1 < c1; ++c) {
            const uint8_t* buf = lds + ((c - c0) & 1) * kBuf;
            st.load(x, row, c + 1, (int)m.inter);
            if (has_e) er = exponents(ep, c + 1, steps);
            w.take_scales();
            w.load_scales(c + 1);
            read_e(buf);
            each_step([&](auto step) {
                constexpr int s = decltype(step)::value;
                products(buf, step);
                hold(acc);
                __builtin_amdgcn_sched_barrier(0);
                w.load(min(4 * c + s + D, steps - 1), s % D);
                __builtin_amdgcn_sched_barrier(0);
            });
            st.store(lds + ((c - c0 + 1) & 1) * kBuf, cols);
            put_e(lds + ((c - c0 + 1) & 1) * kBuf);
            __syncthreads();
        }
        w.take_scales();
        const uint8_t* buf = lds + ((c1 - 1 - c0) & 1) * kBuf;
        read_e(buf);
        each_step([&](auto step) {
            constexpr int s = decltype(step)::value;
            products(buf, step);
            hold(acc);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (s + D < 4) w.load(min(4 * (c1 - 1) + s + D, steps - 1), s % D);
        });
        __syncthreads();   // before the next item's first columns
        if (live) {
            float* to = a.sums + ((int64_t)k * m.tokens * m.top_k + t0 * m.top_k) * m.hidden + 16 * tile + 4 * g;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (16 * j + n >= cols) continue;
                const int64_t slot = p.list[first + 16 * j + n];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    *reinterpret_cast<float4*>(to + slot * m.hidden + 16 * q) =
                        make_float4(acc[q][j][0], acc[q][j][1], acc[q][j][2], acc[q][j][3]);
            }
        }
    }
}

// out from the partial sums: four columns of a token to a thread, its slots in order.  They come from the L2
// that the last kernel left them in, or from memory (512 x 2048: 4.7 us, 502 x 4096: 5.2, of which some 3 are the launch).
__global__ __launch_bounds__(256) void join_kernel(DownTileArgs a) {
    const MoeShape& m = a.m;
    const int64_t quads = m.hidden / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= m.tokens * quads) return;
    const int64_t t = i / quads, col = 4 * (i - t * quads);
    // eight slots' loads at a time; of a slot without an expert the sums hold anything
    v4f sum = v4f{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < m.top_k; j0 += 8) {
        float w[8];
        v4f v[8];
        bool on[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t s = t * m.top_k + min(j0 + j, m.top_k - 1);
            on[j] = j0 + j < m.top_k && (uint32_t)a.ids[s] < (uint32_t)m.experts;
            w[j] = a.weights[s];
            v[j] = *reinterpret_cast<const v4f*>(a.sums + s * m.hidden + col);
        }
        for (int k = 1; k < a.ks; ++k) {
            v4f more[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                more[j] = *reinterpret_cast<const v4f*>(a.sums + ((int64_t)k * m.tokens * m.top_k + t * m.top_k + min(j0 + j, m.top_k - 1)) * m.hidden + col);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += more[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = on[j] ? __builtin_fmaf(w[j], v[j][c], sum[c]) : sum[c];
    }
    *reinterpret_cast<uint2*>(a.out + t * m.hidden + col) = make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
int64_t exponent_stride(int64_t inter) { return (inter + 511) / 512 * 16; }
// Rows of the partial sums: one for each slot, or for up to four K parts of them within kSumRows
constexpr int64_t kSumRows = 2048;
int64_t moe_sum_rows(int64_t slots) { return slots >= kSumRows ? slots : 4 * slots < kSumRows ? 4 * slots : kSumRows; }
// Stored plans: of at least the chunks, which have 2048 / top_k tokens, 2017 slots or more
int64_t moe_plans(int64_t slots) { return slots / 2017 + 1; }

struct MoeGrid {
    bool few, up_tiles;             // few: the kernels for up to 64 slots
    int down_mt;                    // column tiles of the second product's units
    bool up_shared, down_shared;    // several units of an expert read its weights
    int kw, rows, ks;
    unsigned up, down, join, chunks;
    size_t up_at, down_at;          // LDS of the kernels before the plan
};

// Units of w slots that an expert takes, were its slots normal about `each` with that variance: the mean of ceil(c / w)
double expected_units(double each, int w) {
    if (each > 8.0 * w) return each / w + 0.5;
    double units = 0.0;
    for (int j = 0; j * w < each + 6.0 * sqrt(each) + 1.0; ++j) units += 0.5 * erfc((j * w + 0.5 - each) / sqrt(2.0 * each));
    return units;
}

MoeGrid moe_grid(const MoeArgs& a) {
    MoeGrid g{};
    const int64_t chunk = moe_chunk_tokens(a.top_k), cus = device_cus();
    g.chunks = (unsigned)((a.tokens + chunk - 1) / chunk);
    const int64_t slots = (a.tokens < chunk ? a.tokens : chunk) * a.top_k, experts = a.e.experts;
    // experts met, about: were the slots spread at random
    const int64_t met = (int64_t)((double)experts * (1.0 - pow(1.0 - 1.0 / (double)experts, (double)slots)) + 0.5);
    const int64_t down_groups = (a.e.hidden / 16 + 15) / 16;
    const int64_t each = slots / experts;   // slots of an expert, on average, were none left out
    const bool small = slots <= kWaveSlots;
    // Up to 64 slots: the down kernel's workgroups, one for each 16 columns, read inter of each expert met at some
    // 30 GB/s, the tile kernels' together at 5.5 TB/s, but with a list of the slots and a third launch, 6 us
    // (seven tokens of 7 in 60 experts, hidden 512, inter 7936: 72 us for 15 + 5; hidden 2048, inter 768,
    // eight tokens of 8 in 128: 17 us for 11 + 5)
    const double read = (double)met * (double)a.e.inter * 8.5;   // bytes of 16 columns
    g.few = small && read / 30e3 < read * (double)(a.e.hidden / 16) / 5.5e6 + 6.0;
    // The second product's K parts, 2 or 4 within moe_sum_rows, while items are fewer than the CUs: parts cost their partial
    // sums (microseconds of the call with 1, 2 and 4: 32 items, inter 8192 53, 44, 42; 60, 7936 57, 50, 50; 128, 4096
    // 42, 45, 46; 128, 8192 92, 93, 94, and with units of 64 136, 142, 157)
    const int64_t chunks_k = (a.e.inter + 511) / 512;
    const auto parts = [&](int mt) {
        const int64_t items = met * (each / (16 * mt) + 1) * down_groups;
        int ks = 1;
        while (ks < 4 && 2 * ks * items < cus && 2 * ks * a.tokens * a.top_k <= kSumRows && 4 * ks <= chunks_k) ks *= 2;
        return ks;
    };
    // Its units, of 32 slots, two workgroups to a CU, or of 64, one: by the rounds that the items take.  As times of a K part's
    // chunk, two workgroups of 32 side by side are 1, one alone 0.6, one of 64 0.84.  Over 418 sizes (4 to 256 experts of 1 to
    // 250 slots, hidden 1024 to 8192, inter 512 to 14336) the calls come out 0.5 % over the better of the two on average and 7 %
    // at most; with 32 always 1.2 % and 11 %.  Times of the call (32 | 64): 8 experts, 4096 x 8192, 48 slots of an
    // expert 108 | 114, 60 146 | 137, 100 183 | 174; 16 experts, 4096 x 4096, 44 slots 115 | 109, 64 142 | 146, 80 171 | 189.
    const auto rounds = [&](int mt) {
        const int ks = parts(mt);
        const double items = (double)experts * expected_units((double)slots / (double)experts, 16 * mt) * (double)(down_groups * ks);
        const double chunks = (double)chunks_k / ks;
        if (mt == 4) return chunks * 0.84 * ceil(items / (double)cus);
        const double pairs = items / (double)(2 * cus), whole = floor(pairs), rest = pairs - whole;
        return chunks * (whole + (rest == 0.0 ? 0.0 : rest <= 0.5 ? 0.6 : 1.0));
    };
    g.down_mt = !g.few && rounds(4) < rounds(2) ? 4 : 2;
    // Weights that several units read are left in the caches, the others' loads have the hint.  First product (with | without):
    // 60 slots of an expert, 16 experts, 2048 x 1408 44.8 | 46.4, 80 56.1 | 55.8, 8 experts 37.3 | 36.2; 72, 8 experts,
    // 4096 x 8192 -2 %.  Second, units of 32: 20 slots, 32 experts, 4096 x 4096 172 | 176, 28 188 | 188, 32 200 | 193,
    // 48 252 | 226.
    g.up_shared = each >= kUpColumns, g.down_shared = each >= 24;
    // With few items the tile kernel leaves CUs idle, which up_kernel's K parts fill (microseconds of the call, tiles | K parts:
    // 64 items, 4096 x 512, 150 tokens 37 | 30; 96, 4096 x 1536, 100 43 | 39, 1024 x 1024, 300 26.0 | 26.2; 128,
    // 1024 x 1024, 66 19 | 21; 192, 4096 x 1536, 150 44 | 54)
    const int64_t up_items = met * (each / kUpColumns + 1) * (a.e.inter / 128);
    g.up_tiles = !small && up_items >= 112;
    const auto units = [&](int64_t columns) {
        const int64_t most = slots < experts ? slots : experts + slots / columns;
        return most < slots ? most : slots;
    };
    const size_t scratch = g.few ? 0 : (plan_scratch(slots, experts) + 15) / 16 * 16;
    const auto at = [&](int64_t bytes) { return (size_t)bytes > scratch ? (size_t)bytes : scratch; };
    // as many workgroups of the tile kernels as the CUs hold at once: each lists the slots only once
    const auto grid = [&](int64_t groups, int64_t room) { return (unsigned)(groups < room ? groups : room); };
    if (g.up_tiles) {
        g.up = grid(units(kUpColumns) * (a.e.inter / 128), 2 * cus);
        g.up_at = at(2 * kUpColumns * 512);
    } else {
        const int64_t items = units(16) * (a.e.inter / 32), steps = a.e.hidden / 128;
        // K parts while there is about a workgroup for each CU, and four where a wave would have eight steps or more
        // (microseconds with 1, 2, 4 and 8: hidden 2048, one token of eight experts 14.4, 10.9, 10.2, 5.9, four
        // 15.5, 12.3, 13.4, 12.9, eight 18.5, 22.0, 19.9, 20.6; hidden 2688, 73 workgroups 24.4, 17.9, 12.9,
        // 12.5; hidden 4096, 256 workgroups 37, 46, 32, 37)
        g.kw = 1;
        while (g.kw < 8 && 2 * g.kw <= steps && (items * 2 * g.kw <= 9 * cus || (steps >= 32 && g.kw < 4))) g.kw *= 2;
        const int64_t groups = (items * g.kw + 7) / 8;
        g.up = (unsigned)(groups < 3 * cus ? groups : 3 * cus);
        g.up_at = at(g.kw > 1 ? 8 * 4 * 1024 : 0);
    }
    if (g.few) {
        g.down = (unsigned)(a.e.hidden / 16);
        g.rows = (int)(16 * slots);
        g.down_at = (size_t)g.rows * 64 + (size_t)slots * 4;
    } else {
        g.ks = parts(g.down_mt);
        g.down = grid(units(16 * g.down_mt) * down_groups * g.ks, 2 * cus);
        g.down_at = (size_t)(2 * 16 * g.down_mt * (512 + 16));
        g.join = (unsigned)((a.tokens * (a.e.hidden / 4) + 255) / 256);
    }
    return g;
}

// dynamic LDS past 64 KB has to be asked for
hipError_t raise_lds(const void* f, size_t bytes) {
    return bytes <= 64 * 1024 ? hipSuccess : hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
}
template <typename A>
hipError_t launch_one(void (*f)(A), unsigned x, unsigned y, int threads, size_t bytes, hipStream_t stream, const A& a) {
    const hipError_t e = raise_lds((const void*)f, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(f, dim3(x, y), dim3(threads), bytes, stream, a);
    return hipGetLastError();
}

hipError_t launch_up(const MoeGrid& g, UpArgs a, hipStream_t stream) {
    a.plan_at = (int)g.up_at;
    if (g.few) return launch_one(up_kernel<true>, g.up, 1, kUpThreads, g.up_at, stream, a);
    const size_t bytes = g.up_at + sizeof(MoePlan);
    if (!g.up_tiles) return launch_one(up_kernel<false>, g.up, g.chunks, kUpThreads, bytes, stream, a);
    return launch_one(g.up_shared ? up_tile_kernel<0> : up_tile_kernel<kOnce>, g.up, g.chunks, kTileThreads, bytes, stream, a);
}

hipError_t launch_down(const MoeGrid& g, const DownArgs& a, float* sums, const StoredPlan* plans, hipStream_t stream) {
    if (g.few) return launch_one(down_kernel, g.down, 1, kDownThreads, g.down_at, stream, a);
    const DownTileArgs d{a.m, a.w, a.s, a.ids, a.weights, a.out, sums, g.ks, Divisor((a.m.hidden / 16 + 15) / 16 * g.ks), (int)g.down_at, plans};
    const hipError_t e = launch_one(g.down_mt == 4     ? down_tile_kernel<4, 4, 2, 0>
                                    : g.down_shared ? down_tile_kernel<2, 4, 4, 0>
                                                    : down_tile_kernel<2, 4, 4, kOnce>,
                                    g.down, g.chunks, kTileThreads, g.down_at + sizeof(MoePlan), stream, d);
    return e != hipSuccess ? e : launch_one(join_kernel, g.join, 1, 256, 0, stream, d);
}

}  // namespace

// v's codes and exponents, then (16-byte aligned) the partial sums and the plans
size_t moe_workspace_bytes(int64_t slots, int64_t hidden, int64_t inter) {
    return (size_t)(slots * (inter + exponent_stride(inter)) + moe_sum_rows(slots) * hidden * 4) + (size_t)moe_plans(slots) * sizeof(StoredPlan);
}

static int64_t threads(const MoeGrid& g) {
    const int64_t up = (int64_t)g.chunks * g.up * kUpThreads, down = (int64_t)g.chunks * g.down * kDownThreads;
    const int64_t join = (int64_t)g.join * 256, most = up > down ? up : down;
    return most > join ? most : join;
}

w4a8_status launch_moe(const MoeArgs& a, size_t ws_bytes, hipStream_t stream) {
    const MoeGrid g = moe_grid(a);
    if (threads(g) >= kGridThreads) return W4A8_ERR_UNSUPPORTED_SHAPE;
    if (!a.ws || ws_bytes < moe_workspace_bytes(a.tokens * a.top_k, a.e.hidden, a.e.inter) || (uintptr_t)a.ws % 256 != 0)
        return W4A8_ERR_WORKSPACE;
    MoeShape m{};
    m.tokens = a.tokens, m.hidden = a.e.hidden, m.inter = a.e.inter;
    m.by_top_k = Divisor(a.top_k);
    m.experts = a.e.experts, m.top_k = a.top_k, m.chunk = (int)moe_chunk_tokens(a.top_k);
    m.h_steps = (int)(a.e.hidden / 128), m.i_steps = (int)(a.e.inter / 128);
    m.e_stride = exponent_stride(a.e.inter);
    const int64_t slots = a.tokens * a.top_k;
    m.v = a.ws, m.ve = a.ws + slots * a.e.inter;
    float* sums = reinterpret_cast<float*>(m.ve + slots * m.e_stride);
    StoredPlan* plans = reinterpret_cast<StoredPlan*>(sums + moe_sum_rows(slots) * a.e.hidden);
    const hipError_t e = launch_up(g, {m, a.e.up_w, a.e.up_s, a.x8, a.xs, a.ids, a.act, g.kw, Divisor(a.e.inter / (g.up_tiles ? 128 : 32)),
                                       Divisor(g.up_tiles ? 1 : g.kw), 0, plans, 16 * g.down_mt}, stream);
    if (e != hipSuccess) return W4A8_ERR_HIP;
    return launch_down(g, {m, a.e.down_w, a.e.down_s, a.ids, a.weights, a.out, g.rows}, sums, plans, stream) == hipSuccess ? W4A8_OK : W4A8_ERR_HIP;
}

}  // namespace w4a8
