// moe.hip -- a mixture of experts' gated products on MXFP4 weights, two kernels.
//
//   g, u = x W_up[e]^T (halves),  v = act(g) u,  out[t] = sum_j w[t, j] v[t, j] W_down[e]^T
//
// with few tokens per expert: both products read each weight of the experts met once
// and are bound by that.  The weights are in the fragment order of the prepared
// linears (gemm_prepared.hip), so a wave's 16-row tile of 128 k is one 1 KiB load and
// the e2m1 operand of one block-scaled 16x16x128 product; the activations of up to 16
// tokens are its e4m3 operand, read from the cache as they are (their rows are
// gathered, no copy in LDS: a tile's 2 KiB meet its 4 or 1 KiB of weights).
//
// Between the products v is held as e4m3 with a power of two per 32 values, which the
// matrix instruction takes as the operand's scale: a scale per token would need the
// maximum over all of inter, which no workgroup of the first kernel sees.
//
// Slots (token t, j), at most 2048 at a time (more tokens: more chunks in the same
// launches), are listed by expert in LDS by every workgroup; runs of up to 16 MT
// slots of one expert are the units of both kernels.  A unit's slots are the columns of
// its products; which column a slot takes has no influence on its result.
//
//   up    an item is a unit and 32 of inter (two tiles each of gate and up rows), its
//         K shared by KW waves and joined in LDS; v's blocks of 32 are then whole in a wave
//   down  a workgroup per 16 columns of the output, its waves over the units (and parts
//         of K where units are few); every slot's 16 partial sums meet in LDS, and are
//         added in the order of j: no atomics, no third kernel
#include "w4a8_internal.h"

namespace w4a8 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFmtFp8 = 0, kFmtFp4 = 4, kUnitScale = 127;
constexpr int kMaxExperts = 1024;
constexpr int kUpThreads = 512, kDownThreads = 1024;

__device__ __forceinline__ v8i frag_fp4(uint4 q) { return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0}; }
__device__ __forceinline__ v8i frag_fp8(u32x4 lo, u32x4 hi) {
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
// scales in the low byte of each dword
__device__ __forceinline__ v4f product(v8i w, v8i x, v4f c, uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, kFmtFp4, kFmtFp8, 0, (int)sw, 0, (int)sx);
}

// ---------------------------------------------------------------------------
// slots by expert
// ---------------------------------------------------------------------------
struct alignas(16) MoePlan {
    uint32_t count[kMaxExperts + 1];    // slots of each expert, then its first place in `list` (and the end of the last)
    uint16_t list[kMoeSlots];           // slots (of the chunk) by expert
    uint32_t unit[kMoeSlots];           // first place | (slots - 1) << 11 | expert << 17
    uint32_t part[16];
    int units, several;                 // several: some expert has more than one unit
};
__device__ __forceinline__ int unit_first(uint32_t u) { return u & 2047; }
__device__ __forceinline__ int unit_slots(uint32_t u) { return ((u >> 11) & 63) + 1; }
__device__ __forceinline__ int unit_expert(uint32_t u) { return u >> 17; }

// All NT threads; `slots` of the chunk, its ids; US: slots to a unit (at most 64).  The atomics
// list an expert's slots in any order.  Where workgroups share an expert of several units
// (ORDER) they have to agree on which slots are whose: such an expert's are sorted, each
// slot counting the smaller ones.
template <int NT, int US, bool ORDER>
__device__ void make_plan(MoePlan& p, const int32_t* ids, int slots, int experts) {
    constexpr int kPer = kMoeSlots / NT, kExp = kMaxExperts / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < experts; e += NT) p.count[e] = 0;
    if (tid == 0) p.several = 0;
    __syncthreads();
    int id[kPer], at[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = tid + i * NT;
        id[i] = s < slots ? ids[s] : -1;
        if ((uint32_t)id[i] >= (uint32_t)experts) id[i] = -1;
        if (id[i] >= 0) at[i] = (int)atomicAdd(&p.count[id[i]], 1u);
    }
    __syncthreads();
    // exclusive sums over the experts of slots (low half) and units (high half)
    uint32_t mine[kExp], sum = 0;
#pragma unroll
    for (int i = 0; i < kExp; ++i) {
        const int e = tid * kExp + i;
        const uint32_t c = e < experts ? p.count[e] : 0u;
        mine[i] = c | ((c + US - 1) / US) << 16;
        sum += mine[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t v = __shfl_up(incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 63) p.part[wave] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int i = 0; i < wave; ++i) before += p.part[i];
    if (tid == NT - 1) p.units = (int)((before + sum) >> 16), p.count[experts] = (before + sum) & 0xFFFFu;
#pragma unroll
    for (int i = 0; i < kExp; ++i) {
        const int e = tid * kExp + i, c = mine[i] & 0xFFFFu, first = before & 0xFFFFu;
        int u = before >> 16;
        if (e < experts) p.count[e] = first;
        if (ORDER && c > US) p.several = 1;
        for (int k = 0; k < c; k += US, ++u)
            p.unit[u] = (uint32_t)(first + k) | (uint32_t)(min(c - k, US) - 1) << 11 | (uint32_t)e << 17;
        before += mine[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (id[i] >= 0) p.list[p.count[id[i]] + at[i]] = (uint16_t)(tid + i * NT);
    __syncthreads();
    if constexpr (ORDER) {
        if (!p.several) return;   // the same in all threads
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (id[i] < 0) continue;
            const int first = p.count[id[i]], end = p.count[id[i] + 1], s = tid + i * NT;
            if (end - first <= US) {
                id[i] = -1;
                continue;
            }
            at[i] = first;
            for (int k = first; k < end; ++k) at[i] += p.list[k] < s;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (id[i] >= 0) p.list[at[i]] = (uint16_t)(tid + i * NT);
        __syncthreads();
    }
}

struct MoeShape {
    int64_t tokens, hidden, inter;
    int experts, top_k, chunk;          // tokens of a chunk
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
};
struct DownArgs {
    MoeShape m;
    const uint8_t *w, *s;
    const int32_t* ids;
    const float* weights;
    uint16_t* out;
    int rows;                           // of partial sums that LDS holds
};

// ---------------------------------------------------------------------------
// up
// ---------------------------------------------------------------------------
__device__ __forceinline__ float activated(float g, int act) {
    if (act == W4A8_ACT_SILU) return g / (1.0f + expf(-g));
    const float t = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-2.0f * t));   // (1 + tanh t) / 2
}

template <int MT>
struct UpStep {
    uint4 w[4];            // gate rows i0 .. +15 and +16 .. +31, then the up rows
    uint32_t s[4];
    u32x4 x[MT][2];
};

template <int MT>
__global__ __launch_bounds__(kUpThreads) void up_kernel(UpArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    MoePlan& p = *reinterpret_cast<MoePlan*>(lds);
    float4* join = reinterpret_cast<float4*>(lds + sizeof(MoePlan));   // [wave][tile][MT][lane]
    const MoeShape& m = a.m;
    const int64_t t0 = (int64_t)blockIdx.y * m.chunk;
    const int tokens = (int)min((int64_t)m.chunk, m.tokens - t0), slots = tokens * m.top_k;
    make_plan<kUpThreads, 16 * MT, true>(p, a.ids + t0 * m.top_k, slots, m.experts);

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int kw = a.kw, part = wave % kw, per_wg = 8 / kw;
    const int blocks = (int)(m.inter / 32), items = p.units * blocks;
    const int c_pad = (m.h_steps + 3) / 4;
    const int64_t tiles_i = m.inter / 16;
    const int s0 = m.h_steps * part / kw, s1 = m.h_steps * (part + 1) / kw;
    for (int base = blockIdx.x * per_wg; base < items; base += gridDim.x * per_wg) {   // the same in all waves
        const int item = base + wave / kw;
        const bool live = item < items;
        const uint32_t u = uniform(p.unit[live ? item / blocks : 0]);
        const int blk = live ? item % blocks : 0, cols = unit_slots(u);
        int slot[MT];
        const uint8_t* x = a.x8 + t0 * m.hidden;
        uint32_t xo[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            slot[j] = p.list[unit_first(u) + min(16 * j + n, cols - 1)];
            xo[j] = (uint32_t)(slot[j] / m.top_k) * (uint32_t)m.hidden + 16 * g;
        }
        const uint8_t *wp[4];
        const uint32_t* sp[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t tile = (2 * unit_expert(u) + (q >> 1)) * tiles_i + 2 * blk + (q & 1);
            wp[q] = a.w + tile * c_pad * 4096;
            sp[q] = reinterpret_cast<const uint32_t*>(a.s) + tile * c_pad * 64;
        }
        v4f acc[4][MT];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[q][j] = v4f{0.f, 0.f, 0.f, 0.f};
        const auto load = [&](int s, UpStep<MT>& r) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r.w[q] = load_stream16(reinterpret_cast<const uint4*>(wp[q] + s * 1024) + lane);
                r.s[q] = (sp[q] + (s >> 2) * 64)[lane];
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                r.x[j][0] = *reinterpret_cast<const u32x4*>(x + 128 * s + xo[j]);
                r.x[j][1] = *reinterpret_cast<const u32x4*>(x + 128 * s + 64 + xo[j]);
            }
        };
        const auto compute = [&](int s, const UpStep<MT>& r) {
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const v8i x = frag_fp8(r.x[j][0], r.x[j][1]);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[q][j] = product(frag_fp4(r.w[q]), x, acc[q][j], r.s[q] >> (8 * (s & 3)), kUnitScale);
            }
        };
        if (live && s0 < s1) {
            UpStep<MT> ring[2];
            load(s0, ring[0]);
            for (int s = s0; s < s1; s += 2) {
                if (s + 1 < s1) load(s + 1, ring[1]);
                compute(s, ring[0]);
                if (s + 2 < s1) load(s + 2, ring[0]);
                if (s + 1 < s1) compute(s + 1, ring[1]);
            }
        }
        if (kw > 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    join[((wave * 4 + q) * MT + j) * 64 + lane] = make_float4(acc[q][j][0], acc[q][j][1], acc[q][j][2], acc[q][j][3]);
            __syncthreads();
        }
        // column tile j of the item by the wave of part j % kw: parts in order
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (!live || j % kw != part) continue;
            v4f r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (kw == 1) {
                    r[q] = acc[q][j];
                    continue;
                }
                r[q] = v4f{0.f, 0.f, 0.f, 0.f};
                for (int k = 0; k < kw; ++k) {
                    const float4 f = join[(((wave - part + k) * 4 + q) * MT + j) * 64 + lane];
                    r[q] += v4f{f.x, f.y, f.z, f.w};
                }
            }
            const float sx = a.xs[t0 + slot[j] / m.top_k];
            float v[2][4];
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[h][i] = activated(sx * r[h][i], a.act) * (sx * r[2 + h][i]);
                    top = max(top, __float_as_uint(v[h][i]) & 0x7FFFFFFFu);
                }
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            // the least e with top <= 448 2^e = 1.75 2^(e + 8)
            const int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -127);
            const bool finite = top < 0x7F800000u;
            const float to_code = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, -e <= 127
            if (16 * j + n >= cols) continue;
            const int64_t row = t0 * m.top_k + slot[j];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[h][0] * to_code, v[h][1] * to_code, 0, false);
                c = __builtin_amdgcn_cvt_pk_fp8_f32(v[h][2] * to_code, v[h][3] * to_code, c, true);
                *reinterpret_cast<int*>(m.v + row * m.inter + 32 * blk + 16 * h + 4 * g) = finite ? c : 0x7F7F7F7F;
            }
            if (g == 0)   // block blk: k / 32 % 4 = blk % 4 of step blk / 4
                m.ve[row * m.e_stride + (blk >> 4) * 16 + (blk & 3) * 4 + ((blk >> 2) & 3)] = finite ? (uint8_t)(e + 127) : 255;
        }
        if (kw > 1) __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------
template <int MT>
struct DownStep {
    uint4 w;
    uint32_t s;
    u32x4 x[MT][2];
    uint32_t e[MT];
};

template <int MT>
__global__ __launch_bounds__(kDownThreads) void down_kernel(DownArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    MoePlan& p = *reinterpret_cast<MoePlan*>(lds);
    float4* part = reinterpret_cast<float4*>(lds + sizeof(MoePlan));   // [slot][K part][16 columns]
    const MoeShape& m = a.m;
    const int64_t t0 = (int64_t)blockIdx.y * m.chunk;
    const int tokens = (int)min((int64_t)m.chunk, m.tokens - t0), slots = tokens * m.top_k;
    const int32_t* ids = a.ids + t0 * m.top_k;
    make_plan<kDownThreads, 16 * MT, false>(p, ids, slots, m.experts);

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    constexpr int kWaves = kDownThreads / 64;
    int ks = 1;   // K parts: as many as give every wave one, while there are few units
    while (2 * ks * p.units <= kWaves && 2 * ks * slots <= a.rows && 2 * ks <= min(kWaves, m.i_steps)) ks *= 2;
    const int c_pad = (m.i_steps + 3) / 4;
    for (int item = wave; item < p.units * ks; item += kWaves) {
        const uint32_t u = uniform(p.unit[item / ks]);
        const int k = item % ks, cols = unit_slots(u);
        const int64_t tile = unit_expert(u) * (m.hidden / 16) + blockIdx.x;
        const uint8_t* wp = a.w + tile * c_pad * 4096;
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(a.s) + tile * c_pad * 64;
        const uint8_t *x = m.v + t0 * m.top_k * m.inter, *e = m.ve + t0 * m.top_k * m.e_stride;
        int slot[MT];
        uint32_t xo[MT], eo[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            slot[j] = p.list[unit_first(u) + min(16 * j + n, cols - 1)];
            xo[j] = (uint32_t)slot[j] * (uint32_t)m.inter + 16 * g;
            eo[j] = (uint32_t)slot[j] * (uint32_t)m.e_stride + 4 * g;
        }
        v4f acc[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
        const auto load = [&](int s, DownStep<MT>& r) {
            r.w = load_stream16(reinterpret_cast<const uint4*>(wp + s * 1024) + lane);
            r.s = (sp + (s >> 2) * 64)[lane];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                r.x[j][0] = *reinterpret_cast<const u32x4*>(x + 128 * s + xo[j]);
                r.x[j][1] = *reinterpret_cast<const u32x4*>(x + 128 * s + 64 + xo[j]);
                r.e[j] = *reinterpret_cast<const uint32_t*>(e + (s >> 2) * 16 + eo[j]);
            }
        };
        const auto compute = [&](int s, const DownStep<MT>& r) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
                acc[j] = product(frag_fp4(r.w), frag_fp8(r.x[j][0], r.x[j][1]), acc[j], r.s >> (8 * (s & 3)),
                                 r.e[j] >> (8 * (s & 3)));
        };
        const int s0 = m.i_steps * k / ks, s1 = m.i_steps * (k + 1) / ks;
        DownStep<MT> ring[2];
        load(s0, ring[0]);
        for (int s = s0; s < s1; s += 2) {
            if (s + 1 < s1) load(s + 1, ring[1]);
            compute(s, ring[0]);
            if (s + 2 < s1) load(s + 2, ring[0]);
            if (s + 1 < s1) compute(s + 1, ring[1]);
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
            if (16 * j + n < cols) part[(slot[j] * ks + k) * 4 + g] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    }
    __syncthreads();
    // four columns of a token to a thread: its slots in order
    for (int i = threadIdx.x; i < 4 * tokens; i += kDownThreads) {
        const int t = i >> 2, q = i & 3;
        v4f sum = v4f{0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < m.top_k; ++j) {
            const int s = t * m.top_k + j;
            if ((uint32_t)ids[s] >= (uint32_t)m.experts) continue;
            v4f v = v4f{0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < ks; ++k) {
                const float4 f = part[(s * ks + k) * 4 + q];
                v += v4f{f.x, f.y, f.z, f.w};
            }
            const float w = a.weights[t0 * m.top_k + s];
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = __builtin_fmaf(w, v[c], sum[c]);
        }
        *reinterpret_cast<uint2*>(a.out + (t0 + t) * m.hidden + 16 * blockIdx.x + 4 * q) =
            make_uint2(pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3]));
    }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
struct MoeGrid {
    int mt, kw, rows;
    unsigned up, down, chunks;
    size_t up_lds, down_lds;
};
int64_t exponent_stride(int64_t inter) { return (inter + 511) / 512 * 16; }

MoeGrid moe_grid(const MoeArgs& a) {
    MoeGrid g{};
    const int64_t chunk = moe_chunk_tokens(a.top_k);
    g.chunks = (unsigned)((a.tokens + chunk - 1) / chunk);
    const int64_t slots = (a.tokens < chunk ? a.tokens : chunk) * a.top_k;
    // column tiles of a unit by the slots that an expert has on average
    const int64_t each = slots / a.e.experts;
    g.mt = each <= 8 ? 1 : each <= 24 ? 2 : 4;
    const int64_t most = slots < a.e.experts ? slots : a.e.experts + slots / (16 * g.mt);
    const int64_t units = most < slots ? most : slots, items = units * (a.e.inter / 32);
    const int64_t steps = a.e.hidden / 128;
    g.kw = 8;
    while (g.kw > 1 && (items * g.kw > 4096 || g.kw > steps || g.kw * g.mt > 16)) g.kw /= 2;
    const int64_t groups = (items * g.kw + 7) / 8, room = 2 * (int64_t)device_cus();
    g.up = (unsigned)(groups < room ? groups : room);
    g.down = (unsigned)(a.e.hidden / 16);
    g.up_lds = sizeof(MoePlan) + (g.kw > 1 ? (size_t)8 * 4 * g.mt * 1024 : 0);
    // K parts of few slots: to 1024 rows
    g.rows = (int)(slots >= 1024 ? slots : 16 * slots < 1024 ? 16 * slots : 1024);
    g.down_lds = sizeof(MoePlan) + (size_t)g.rows * 64;
    return g;
}

// dynamic LDS past 64 KB has to be asked for
hipError_t raise_lds(const void* f, size_t bytes) {
    return bytes <= 64 * 1024 ? hipSuccess : hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
}

template <int MT>
hipError_t launch_mt(const MoeGrid& g, const UpArgs& up, const DownArgs& down, hipStream_t stream) {
    hipError_t e = raise_lds((const void*)up_kernel<MT>, g.up_lds);
    if (e == hipSuccess) e = raise_lds((const void*)down_kernel<MT>, g.down_lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(up_kernel<MT>, dim3(g.up, g.chunks), dim3(kUpThreads), g.up_lds, stream, up);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(down_kernel<MT>, dim3(g.down, g.chunks), dim3(kDownThreads), g.down_lds, stream, down);
    return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(int64_t slots, int64_t inter) {
    return (size_t)(slots * (inter + exponent_stride(inter)));
}

int64_t moe_threads(const MoeArgs& a) {
    const MoeGrid g = moe_grid(a);
    return (int64_t)g.chunks * ((int64_t)g.up * kUpThreads > (int64_t)g.down * kDownThreads ? (int64_t)g.up * kUpThreads
                                                                                             : (int64_t)g.down * kDownThreads);
}

hipError_t launch_moe(const MoeArgs& a, hipStream_t stream) {
    const MoeGrid g = moe_grid(a);
    MoeShape m{};
    m.tokens = a.tokens, m.hidden = a.e.hidden, m.inter = a.e.inter;
    m.experts = a.e.experts, m.top_k = a.top_k, m.chunk = (int)moe_chunk_tokens(a.top_k);
    m.h_steps = (int)(a.e.hidden / 128), m.i_steps = (int)(a.e.inter / 128);
    m.e_stride = exponent_stride(a.e.inter);
    m.v = a.ws, m.ve = a.ws + a.tokens * a.top_k * a.e.inter;
    const UpArgs up{m, a.e.up_w, a.e.up_s, a.x8, a.xs, a.ids, a.act, g.kw};
    const DownArgs down{m, a.e.down_w, a.e.down_s, a.ids, a.weights, a.out, g.rows};
    switch (g.mt) {
        case 1: return launch_mt<1>(g, up, down, stream);
        case 2: return launch_mt<2>(g, up, down, stream);
        default: return launch_mt<4>(g, up, down, stream);
    }
}

}  // namespace w4a8
