// attention.hip -- softmax attention of new tokens over the paged MXFP4 cache.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - max),  j over the
//   keys that the query's mask leaves; zeros where it leaves none.
//
// One pass over the keys with a running maximum and sum.  The rows of a
// key/value head are its group's heads of every query token (row = token *
// group + head), so a key's bytes are read once for all of them.
//
// q.k runs on the block-scaled matrix instructions straight from the cache: 16
// bytes of a key's row and its exponent byte are an fp4 operand and its scale,
// nothing is decoded.  The queries are the e4m3 operand, as a sum of pieces
//   q 2^(7-e) = x0 + x1 / 16 + x2 / 256,  e = the row's exponent,
// each piece the e4m3 rounding of what the ones before left.  Two pieces hold
// the 8 significant bits of bf16 and three the 11 of fp16 (values 2^13 and more
// below the row's largest are off by up to 2^-21 of it).  The pieces' 1, 1/16,
// 1/256 are the operand's scale; 2^(e-7) and the softmax scale multiply the
// fp32 score.
//
// p.v runs in bf16: an e2m1 value times a power of two is exact in it, p is
// rounded to bf16 (relative 2^-9, as the output's own rounding; fp16 queries
// take p as two bf16 pieces, relative 2^-17).  Scores, sums and outputs
// accumulate in fp32.
//
// Values whose exponent byte is 253 or more (NaN blocks; magnitudes at the end
// of bf16's range) count as NaN: their key's score becomes NaN, and the value
// itself zero, so that a masked key never reaches the sum, whatever the cache
// holds there.  A block-table entry outside the cache does the same.
#include <type_traits>

#include "w4a8_internal.h"

#pragma clang fp contract(off)

namespace w4a8 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8h __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kFmtFp8 = 0, kFmtFp4 = 4;
constexpr int kTile = 64;             // keys per step of a wave (decode) or workgroup (prompts)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLazy = 8.0f;         // the running maximum follows when a score passes it by this (log2)

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// What a sequence asks for.  Lengths come from device memory and are not
// trusted: queries stay inside the q tensor, keys inside the block table.
struct Seq {
    int ctx, q0, qlen, q_all;   // keys, first query token, query tokens (at most max_q) and as given
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int s) {
    Seq r;
    const int most = a.table_width << a.page_shift;
    r.ctx = min(max(a.context[s], 0), most);
    if (a.cu_q) {
        const int t = (int)a.tokens;
        r.q0 = min(max(a.cu_q[s], 0), t);
        r.q_all = max(min(a.cu_q[s + 1], t) - r.q0, 0);
        r.qlen = min(r.q_all, a.max_q);
    } else {
        r.q0 = s;
        r.q_all = r.qlen = 1;
    }
    return r;
}
// keys [lo, hi) that the query token t of a sequence sees
__device__ __forceinline__ int key_hi(const AttnArgs& a, const Seq& s, int t) {
    return a.causal ? min(s.ctx, s.ctx - s.q_all + t + 1) : s.ctx;
}
__device__ __forceinline__ int key_lo(const AttnArgs& a, const Seq& s, int t) {
    return a.window ? max(0, s.ctx - s.q_all + t + 1 - a.window) : 0;
}

// A query value's e4m3 pieces, four values per dword.
template <int PC>
__device__ __forceinline__ void pieces4(const float* x, uint32_t* out) {
    float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int p = 0; p < PC; ++p) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], w, true);
        out[p] = (uint32_t)w;
        if (p + 1 < PC) {
            const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            r[0] = (r[0] - lo[0]) * 16.0f;
            r[1] = (r[1] - lo[1]) * 16.0f;
            r[2] = (r[2] - hi[0]) * 16.0f;
            r[3] = (r[3] - hi[1]) * 16.0f;
        }
    }
}

// sixteen 16-bit query values from p
template <bool FP16>
__device__ __forceinline__ void load_q16(const uint16_t* p, bool vec, float* x) {
    uint32_t d[8];
    if (vec) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[0], v = reinterpret_cast<const uint4*>(p)[1];
        d[0] = u.x, d[1] = u.y, d[2] = u.z, d[3] = u.w, d[4] = v.x, d[5] = v.y, d[6] = v.z, d[7] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[2 * j] = FP16 ? f16_to_f32(d[j] & 0xFFFFu) : bf16_to_f32(d[j] & 0xFFFFu);
        x[2 * j + 1] = FP16 ? f16_to_f32(d[j] >> 16) : bf16_to_f32(d[j] >> 16);
    }
}
// the power of two that takes the row's largest magnitude (bits) to [128, 256),
// and what undoes it in the score; a non-finite row's scores are NaN
__device__ __forceinline__ float row_power(uint32_t most, float scale, float* mult) {
    if (most >= 0x7F800000u) {
        *mult = __builtin_nanf("");
        return 0.0f;   // the pieces stay finite
    }
    const int e = max((int)(most >> 23) - 127, -119);
    *mult = scale * kLog2e * ldexpf(1.0f, e - 7);
    return __uint_as_float((uint32_t)(127 + 7 - e) << 23);
}

// byte mask of a dword's bytes >= 253
__device__ __forceinline__ uint32_t bad_bytes(uint32_t x) {
    const uint32_t f = ((x & 0x7F7F7F7Fu) + 0x03030303u) & x & 0x80808080u;
    return (f << 1) - (f >> 7);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}
// p as bf16 pieces: the rounded values, and (PC == 3) the rounded rest
template <int PC>
__device__ __forceinline__ void pack_p(const float* p, uint32_t* hi, uint32_t* lo) {
    *hi = pack_bf16(p[0], p[1]);
    if (PC == 3) *lo = pack_bf16(p[0] - __uint_as_float(*hi << 16), p[1] - __uint_as_float(*hi & 0xFFFF0000u));
}

// bf16 pairs of the e2m1 codes of byte B of x, times the power of two s
template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t x, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, B));
}
// an exponent byte in place of an fp32's exponent: 2^(byte - 127)
template <int B>
__device__ __forceinline__ float byte_scale(uint32_t x) {
    const uint32_t s = B == 3 ? x >> 1 : B == 2 ? x << 7 : B == 1 ? x << 15 : x << 23;
    return __uint_as_float(s & 0x7F800000u);
}

template <bool FP16>
__device__ __forceinline__ uint32_t out_pair(float a, float b) {
    if constexpr (FP16) {
        const _Float16 x = (_Float16)a, y = (_Float16)b;
        return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
    } else {
        return pack_bf16(a, b);
    }
}

// ===========================================================================
// Few query rows per key/value head (single tokens, drafts): the keys stream.
//
// All sequences' tiles of 64 keys, head after head, form one line that is cut
// into equal runs, one per workgroup; a run may cross segments (one sequence's
// one head), and a segment cut by runs is joined by a second kernel.  The cut
// follows the lengths in device memory, so the grid depends on none of them.
//
// A wave takes every fourth tile of its workgroup's run.  Rows of 16 queries are
// the columns of the 16x16 products:
//   S^T = K Q^T: tile u of four holds keys 4r + u (r = row), so that a lane reads
//     the exponents of its four keys as one dword and picks by opsel;
//   lane (n, g) then holds query n's scores of keys 16g .. 16g+15;
//   O^T = V^T P^T: the product's k-slots are filled in that order, so P moves
//     between no lanes, and lane (n, g) reads from keys 16g .. 16g+15 the D/16
//     values of dims n D/16 ..: the transpose happens in its own registers.
// ===========================================================================
template <int D>
struct VWord;   // D/16 e2m1 codes
template <> struct VWord<64> { typedef uint16_t T; static constexpr int N = 1; };
template <> struct VWord<128> { typedef uint32_t T; static constexpr int N = 1; };
template <> struct VWord<256> { typedef uint2 T; static constexpr int N = 2; };
__device__ __forceinline__ uint32_t vword(uint16_t v, int) { return v; }
__device__ __forceinline__ uint32_t vword(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t vword(uint2 v, int i) { return i ? v.y : v.x; }

// tiles of a sequence: at least one while it has queries, so that rows without
// a key are written
__device__ __forceinline__ int first_tile(const AttnArgs& a, const Seq& s) { return key_lo(a, s, 0) / kTile; }
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int s) {
    const Seq q = seq_of(a, s);
    return q.qlen ? max(1, (q.ctx + kTile - 1) / kTile - first_tile(a, q)) : 0;
}

struct Line {       // the cut: total tiles over heads, tiles per workgroup
    int total, run;
};
__device__ __forceinline__ Line line_of(const AttnArgs& a, int workgroups) {
    const int lane = threadIdx.x & 63;
    int t = 0;
    for (int s = lane; s < a.seqs; s += 64) t += tiles_of(a, s);
#pragma unroll
    for (int off = 32; off; off >>= 1) t += __shfl_xor(t, off);
    Line l;
    l.total = t * a.cache.kv_heads;
    // a run gives every wave a tile
    l.run = max((l.total + workgroups - 1) / workgroups, 4);
    return l;
}
// The sequence whose tiles hold position `at` of the line, its first position
// and tiles per head (at < total).
__device__ __forceinline__ void seq_at(const AttnArgs& a, int at, int* seq, int* start, int* tiles) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
        const int n = s0 + lane < a.seqs ? tiles_of(a, s0 + lane) : 0;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(incl, off);
            if (lane >= off) incl += o;
        }
        const int first = base + (incl - n) * a.cache.kv_heads;
        const uint64_t hit = __ballot(n > 0 && at >= first && at < first + n * a.cache.kv_heads);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            *seq = s0 + l;
            *start = __shfl(first, l);
            *tiles = __shfl(n, l);
            return;
        }
        base += __shfl(incl, 63) * a.cache.kv_heads;
    }
    *seq = a.seqs;
    *start = base;
    *tiles = 0;
}

// floats of one partial result: rows x (D outputs, then maximum and sum)
__host__ __device__ constexpr int64_t part_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

template <int D, int NT, int PC>
__global__ __launch_bounds__(256, 2) void decode_kernel(const AttnArgs a, const int workgroups) {
    constexpr int KS = D >= 128 ? D / 128 : 1;      // 128-deep products per score
    constexpr int QP = D >= 128 ? PC : PC - 1;      // q operands per 128 (D = 64: pieces side by side)
    constexpr int DT = D / 16;                      // output tiles
    typedef typename VWord<D>::T VT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int hk = a.cache.kv_heads, ps = a.page_shift;
    __shared__ float sm_m[4][NT * 16], sm_l[4][NT * 16];
    __shared__ v4f sm_o[2][NT * DT][64];

    const Line line = line_of(a, workgroups);
    int pos = (int)blockIdx.x * line.run;
    if ((int64_t)blockIdx.x * line.run >= line.total) return;
    const int end = min(pos + line.run, line.total);
    int sq, start, tiles;
    seq_at(a, pos, &sq, &start, &tiles);
    if (sq >= a.seqs) return;

    while (pos < end) {
        const int head = (pos - start) / tiles;
        const int t0 = (pos - start) - head * tiles;
        const int cnt = min(tiles - t0, end - pos);
        const Seq s = seq_of(a, sq);
        const int rows = s.qlen * a.group;
        const int first = first_tile(a, s);
        const int32_t* table = a.table + (int64_t)sq * a.table_stride;

        // ---- queries ----
        v8i qf[NT][KS][QP];
        float mult[NT];
        int hi[NT], lo[NT];
        const bool vec = (((uintptr_t)a.q | (uintptr_t)(2 * a.q_st) | (uintptr_t)(2 * a.q_sh)) & 15) == 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = min(nt * 16 + n, rows - 1);
            const int tok = row / a.group, h = row - tok * a.group;
            hi[nt] = key_hi(a, s, tok);
            lo[nt] = key_lo(a, s, tok);
            const uint16_t* src = a.q + (int64_t)(s.q0 + tok) * a.q_st + (int64_t)(head * a.group + h) * a.q_sh;
            constexpr int C = D / 64;               // runs of 16 values per lane
            float x[C][16];
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                load_q16<PC == 3>(src + 64 * c + 16 * g, vec, x[c]);
#pragma unroll
                for (int j = 0; j < 16; ++j) most = max(most, __float_as_uint(x[c][j]) & 0x7FFFFFFFu);
            }
            most = max(most, (uint32_t)__shfl_xor((int)most, 16));
            most = max(most, (uint32_t)__shfl_xor((int)most, 32));
            const float up = row_power(most, a.scale, &mult[nt]);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float y[4];
                    uint32_t w[PC];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = up != 0.0f ? x[c][4 * j + i] * up : 0.0f;
                    pieces4<PC>(y, w);
                    if constexpr (D >= 128) {
                        // run c: bytes 0-15 (d = 128 s + 16 g ..) or 16-31 (128 s + 64 + 16 g ..)
#pragma unroll
                        for (int p = 0; p < PC; ++p) qf[nt][c >> 1][p][4 * (c & 1) + j] = (int)w[p];
                    } else {
                        // k < 64: the first piece, k >= 64: the second; then the third alone
                        qf[nt][0][0][j] = (int)w[0];
                        qf[nt][0][0][4 + j] = (int)w[1];
                        if constexpr (PC == 3) {
                            qf[nt][0][1][j] = (int)w[2];
                            qf[nt][0][1][4 + j] = 0;
                        }
                    }
                }
        }

        v4f o[NT][DT];
        float m[NT], mu[NT], l[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = neg_inf();
            mu[nt] = 0.0f;
            l[nt] = 0.0f;
#pragma unroll
            for (int j = 0; j < DT; ++j) o[nt][j] = v4f{0, 0, 0, 0};
        }

        // ---- keys ----
        uint4 kc[KS][4];
        uint32_t ke[KS];
        VT vc[16];
        uint4 ve;
        const int last_key = s.ctx - 1;             // ctx >= 1 wherever it is used
        int pk = 0, pv = 0;                         // block-table entries of the next tile
        // the page of a lane's four keys, and of its sixteen values; keys past the
        // context take the last one's (they are masked)
        auto load_pages = [&](int t) {
            pk = table[min(t * kTile + 4 * n, last_key) >> ps];
            pv = table[min(t * kTile + 16 * g, last_key) >> ps];
        };
        auto load_k = [&](int t) {
            const bool ok = (uint32_t)pk < (uint64_t)a.cache.pages;
            const int64_t ph = (int64_t)(ok ? pk : 0) * hk + head;
            const int row = (t * kTile + 4 * n) & ((1 << ps) - 1);
            const uint8_t* c = a.cache.k_codes + ((ph << ps) + row) * (D / 2) + 16 * (D == 64 ? g & 1 : g);
            const uint8_t* e = a.cache.k_e8m0 + ((ph * (D / 32) + (D == 64 ? g & 1 : g)) << ps) + row;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
#pragma unroll
                for (int u = 0; u < 4; ++u) kc[k][u] = *reinterpret_cast<const uint4*>(c + 64 * k + u * (D / 2));
                ke[k] = *reinterpret_cast<const uint32_t*>(e + ((int64_t)(4 * k) << ps));
                if (!ok) ke[k] = 0xFFFFFFFFu;
            }
        };
        auto load_v = [&](int t) {
            const bool ok = (uint32_t)pv < (uint64_t)a.cache.pages;
            const int64_t ph = (int64_t)(ok ? pv : 0) * hk + head;
            const int row = (t * kTile + 16 * g) & ((1 << ps) - 1);
            const uint8_t* c = a.cache.v_codes + ((ph << ps) + row) * (D / 2) + n * (D / 32);
            const uint8_t* e = a.cache.v_e8m0 + ((ph * (D / 32) + n / (512 / D)) << ps) + row;
#pragma unroll
            for (int k = 0; k < 16; ++k) vc[k] = *reinterpret_cast<const VT*>(c + k * (D / 2));
            ve = *reinterpret_cast<const uint4*>(e);
        };

        const int t_end = first + t0 + cnt;
        int t = first + t0 + wave;
        const bool any = s.ctx > 0;
        // every row sees all keys of [all_lo, all_hi)
        const int all_hi = a.causal ? s.ctx - s.q_all + 1 : s.ctx;
        const int all_lo = key_lo(a, s, s.qlen - 1);
        if (any && t < t_end) {
            load_pages(t);
            load_k(t);
            load_v(t);
            if (t + 4 < t_end) load_pages(t + 4);
        }
        for (; any && t < t_end; t += 4) {
            const bool more = t + 4 < t_end;
            float sc[NT][4][4];                     // [tile u][i]: key 16 g + 4 i + u
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                v4f acc[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int p = 0; p < QP; ++p) {
                        // D = 64: k >= 64 holds the next piece, its scale comes from lanes g = 2, 3
                        const int qs = D == 64 ? (p ? 119 : g < 2 ? 127 : 123) : 127 - 4 * p;
                        auto dot = [&](auto U) {
                            constexpr int u = decltype(U)::value;
                            const v8i kf = {(int)kc[k][u].x, (int)kc[k][u].y, (int)kc[k][u].z, (int)kc[k][u].w, 0, 0, 0, 0};
                            acc[u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf, qf[nt][k][p], acc[u], kFmtFp4,
                                                                                      kFmtFp8, u, (int)ke[k], 0, qs);
                        };
                        dot(std::integral_constant<int, 0>{});
                        dot(std::integral_constant<int, 1>{});
                        dot(std::integral_constant<int, 2>{});
                        dot(std::integral_constant<int, 3>{});
                    }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[nt][u][i] = acc[u][i] * mult[nt];
            }
            if (more) load_k(t + 4);

            // value blocks that count as NaN: rare, so found for the wave at once
            const uint32_t bad[4] = {bad_bytes(ve.x), bad_bytes(ve.y), bad_bytes(ve.z), bad_bytes(ve.w)};
            if (__any((bad[0] | bad[1] | bad[2] | bad[3]) != 0)) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {       // over the head's blocks: the 16 lanes of g
                    b[i] = bad[i];
#pragma unroll
                    for (int off = 1; off < 16; off <<= 1) b[i] |= (uint32_t)__shfl_xor((int)b[i], off);
                }
                ve.x &= ~bad[0], ve.y &= ~bad[1], ve.z &= ~bad[2], ve.w &= ~bad[3];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if ((b[i] >> (8 * u)) & 1u) sc[nt][u][i] = __builtin_nanf("");
            }
            const int key0 = t * kTile;
            if (key0 + kTile > all_hi || key0 < all_lo) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 16 * g + 4 * i + u;
                            if (key >= hi[nt] || key < lo[nt]) sc[nt][u][i] = neg_inf();
                        }
            }
            // ---- running maximum, probabilities ----
            uint32_t pf[NT][2][4], pl[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mx = neg_inf();
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, sc[nt][u][i]);
                if (__any(mx > m[nt] + kLazy)) {
                    mx = fmaxf(mx, __shfl_xor(mx, 16));
                    mx = fmaxf(mx, __shfl_xor(mx, 32));
                    const float mn = fmaxf(m[nt], mx);
                    const float un = mn == neg_inf() ? 0.0f : mn;
                    const float f = exp2f(m[nt] - un);   // 0 where there was none
                    m[nt] = mn;
                    mu[nt] = un;
                    l[nt] *= f;
#pragma unroll
                    for (int j = 0; j < DT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nt][j][i] *= f;
                }
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    float p[8];                     // slots: tile 2 st (i = 0..3), tile 2 st + 1
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[e] = __builtin_amdgcn_exp2f(sc[nt][2 * st + e / 4][e % 4] - mu[nt]);
                        l[nt] += p[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) pack_p<PC>(p + 2 * e, &pf[nt][st][e], &pl[nt][st][e]);
                }
            }
            // ---- values ----
            const uint32_t vs[4] = {ve.x, ve.y, ve.z, ve.w};
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                float vscale[8];                    // slot e: key 4 (e % 4) + 2 st + e / 4
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w = vs[e % 4];
                    vscale[e] = st == 0 ? (e < 4 ? byte_scale<0>(w) : byte_scale<1>(w)) : (e < 4 ? byte_scale<2>(w) : byte_scale<3>(w));
                }
                auto pair = [&](auto B, int word) {   // output tiles 2 b, 2 b + 1 of this word
                    constexpr int b = decltype(B)::value;
                    uint32_t c[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) c[e] = fp4_pair<b>(vword(vc[4 * (e % 4) + 2 * st + e / 4], word), vscale[e]);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                        uint32_t vf[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) vf[e] = __builtin_amdgcn_perm(c[2 * e + 1], c[2 * e], sel);
                        const v8h av = __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(vf));
                        const int j = 8 * word + 2 * b + odd;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            o[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pf[nt][st])), o[nt][j], 0, 0, 0);
                            if (PC == 3)
                                o[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pl[nt][st])), o[nt][j], 0, 0, 0);
                        }
                    }
                };
#pragma unroll
                for (int word = 0; word < VWord<D>::N; ++word) {
                    pair(std::integral_constant<int, 0>{}, word);
                    pair(std::integral_constant<int, 1>{}, word);
                    if constexpr (D >= 128) {
                        pair(std::integral_constant<int, 2>{}, word);
                        pair(std::integral_constant<int, 3>{}, word);
                    }
                }
            }
            if (more) load_v(t + 4);
            if (t + 8 < t_end) load_pages(t + 8);
        }

        // ---- the four waves' results ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] += __shfl_xor(l[nt], 16);
            l[nt] += __shfl_xor(l[nt], 32);
            if (g == 0) {
                sm_m[wave][nt * 16 + n] = m[nt];
                sm_l[wave][nt * 16 + n] = l[nt];
            }
        }
        __syncthreads();
        float mt[NT], lt[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mt[nt] = neg_inf();
#pragma unroll
            for (int w = 0; w < 4; ++w) mt[nt] = fmaxf(mt[nt], sm_m[w][nt * 16 + n]);
            const float u = mt[nt] == neg_inf() ? 0.0f : mt[nt];
            lt[nt] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) lt[nt] += sm_l[w][nt * 16 + n] * exp2f(sm_m[w][nt * 16 + n] - u);
            const float f = exp2f(m[nt] - u);   // 0 without a key (NaN outputs stay NaN)
#pragma unroll
            for (int j = 0; j < DT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][j][i] *= f;
        }
        for (int half = 2; half; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < DT; ++j) sm_o[wave - half][nt * DT + j][lane] = o[nt][j];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < DT; ++j) o[nt][j] += sm_o[wave][nt * DT + j][lane];
            }
            __syncthreads();
        }
        if (wave == 0) {
            const bool whole = cnt == tiles;
            // partial results: slot 0 of a workgroup continues a segment, slot 1 begins one
            float* part = reinterpret_cast<float*>(a.ws) + (2 * (int64_t)blockIdx.x + (t0 == 0 ? 1 : 0)) * part_floats(NT * 16, D);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = nt * 16 + n;
                if (row >= rows) continue;
                if (whole) {
                    const int tok = row / a.group, h = row - tok * a.group;
                    uint16_t* dst = a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + h) * D;
                    const float inv = lt[nt] == 0.0f ? 0.0f : 1.0f / lt[nt];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < DT; j += 2)
                            *reinterpret_cast<uint32_t*>(dst + DT * (4 * g + i) + j) =
                                out_pair<PC == 3>(o[nt][j][i] * inv, o[nt][j + 1][i] * inv);
                } else {
                    float* dst = part + (int64_t)row * D;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < DT; j += 4)
                            *reinterpret_cast<v4f*>(dst + DT * (4 * g + i) + j) =
                                v4f{o[nt][j][i], o[nt][j + 1][i], o[nt][j + 2][i], o[nt][j + 3][i]};
                    if (g == 0) {
                        part[(int64_t)NT * 16 * D + row] = mt[nt];
                        part[(int64_t)NT * 16 * (D + 1) + row] = lt[nt];
                    }
                }
            }
        }
        pos += cnt;
        if (pos < end && t0 + cnt == tiles && head == hk - 1) {
            start += tiles * hk;
            for (tiles = 0; tiles == 0;) {
                if (++sq >= a.seqs) return;
                tiles = tiles_of(a, sq);
            }
        }
    }
}

// Joins a row's partial results: pieces [0, pieces) at part(i), weights
// 2^(m_i - max).  Four waves share the pieces; lane L holds D/64 outputs.
template <int D, bool FP16, typename PART>
__device__ __forceinline__ void join_row(int pieces, int rows, int row, uint16_t* dst, PART part) {
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ float sm[4][64 * C], sl[4], smx[4];
    float mx = neg_inf();
    for (int i = threadIdx.x; i < pieces; i += 256) mx = fmaxf(mx, part(i)[(int64_t)rows * D + row]);
#pragma unroll
    for (int off = 32; off; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    if (lane == 0) smx[wave] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(smx[0], smx[1]), fmaxf(smx[2], smx[3]));
    const float u = mx == neg_inf() ? 0.0f : mx;
    float acc[C] = {}, l = 0.0f;
#pragma unroll 4
    for (int i = wave; i < pieces; i += 4) {
        const float* p = part(i);
        const float w = exp2f(p[(int64_t)rows * D + row] - u);
        const float pl = p[(int64_t)rows * (D + 1) + row];
        l += pl * w;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] += p[(int64_t)row * D + C * lane + c] * w;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) sm[wave][C * lane + c] = acc[c];
    if (lane == 0) sl[wave] = l;
    __syncthreads();
    if (wave == 0) {
        l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = C * lane + c;
            const float v = ((sm[0][at] + sm[1][at]) + (sm[2][at] + sm[3][at])) * inv;
            dst[at] = (uint16_t)out_pair<FP16>(v, v);
        }
    }
}

// one workgroup per segment (sequence and head) and row
template <int D, bool FP16>
__global__ __launch_bounds__(256) void decode_join_kernel(const AttnArgs a, const int workgroups, const int nt16) {
    const uint32_t pair = blockIdx.x / (uint32_t)(a.max_q * a.group);
    const int row = (int)(blockIdx.x - pair * (uint32_t)(a.max_q * a.group));
    const int sq = pair / a.cache.kv_heads, head = pair - sq * a.cache.kv_heads;
    const Seq s = seq_of(a, sq);
    if (row >= s.qlen * a.group) return;
    const Line line = line_of(a, workgroups);
    // the segment's place in the line
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int i = lane; i < sq; i += 64) before += tiles_of(a, i);
#pragma unroll
    for (int off = 32; off; off >>= 1) before += __shfl_xor(before, off);
    const int tiles = tiles_of(a, sq);
    const int g0 = before * a.cache.kv_heads + head * tiles, g1 = g0 + tiles;
    const int w0 = g0 / line.run, w1 = (g1 - 1) / line.run;
    if (w0 == w1) return;   // written whole
    const int tok = row / a.group, h = row - tok * a.group;
    uint16_t* dst = a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + h) * D;
    const float* ws = reinterpret_cast<const float*>(a.ws);
    const int64_t size = part_floats(nt16, D);
    join_row<D, FP16>(w1 - w0 + 1, nt16, row, dst, [&](int i) { return ws + (2 * (int64_t)(w0 + i) + (i == 0 ? 1 : 0)) * size; });
}

// ===========================================================================
// Many query rows (prompts, chunks of prompts): the matrix pipe is the bound.
//
// A workgroup of NW waves holds 32 NW rows of one segment, a wave 32 of them as
// the columns of 32x32 products; 64 keys per step, shared through LDS: the
// keys' codes as they are (fp4 operand), the values widened to bf16 and
// transposed once for all waves.  The copies for the next step are in flight
// while a step computes; two LDS buffers, one barrier per step.  Where there
// are too few workgroups for the chip the keys are split in `ks` parts and
// joined by a second kernel.
// ===========================================================================
template <int D, int NW>
struct PrefillLds {
    uint8_t k[kTile * D / 2];                // row key, 16-byte units XOR-swizzled
    uint8_t e[2 * 2 * 32 * (D / 64)];        // [32-key tile][h][row][64-step]
    uint16_t v[D * kTile];                   // [d][slot], 16-byte units XOR-swizzled
};

template <int D, int PC, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void prefill_kernel(const AttnArgs a, const int tiles_max, const int ks) {
    constexpr int TH = 64 * NW;
    constexpr int S = D / 64;                       // 64-deep products per score
    constexpr int DT = D / 32;                      // 32-wide output tiles
    constexpr int KU = D / 32;                      // 16-byte units of a key
    constexpr int KI = kTile * KU, VI = kTile / 4 * (D / 8);
    constexpr int KN = (KI + TH - 1) / TH, VN = (VI + TH - 1) / TH;
    constexpr int EI = kTile / 4 * KU;              // dwords of exponents
    __shared__ PrefillLds<D, NW> lds[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int hk = a.cache.kv_heads, ps = a.page_shift;

    // the rows' last tiles first: with causal masks they are the longest
    const int pairs = a.seqs * hk;
    int bid = blockIdx.x;
    const int part = bid % ks;
    bid /= ks;
    const int pair = bid % pairs, tile = tiles_max - 1 - bid / pairs;
    const int sq = pair / hk, head = pair - sq * hk;
    const Seq s = seq_of(a, sq);
    const int rows = s.qlen * a.group;
    const int row0 = tile * 32 * NW;
    if (row0 >= rows) return;
    const int32_t* table = a.table + (int64_t)sq * a.table_stride;

    // keys of the workgroup, of its part, and of this wave
    const int tok_last = (min(row0 + 32 * NW, rows) - 1) / a.group;
    const int k_lo = key_lo(a, s, row0 / a.group) / kTile;
    const int k_hi = (max(key_hi(a, s, tok_last), 0) + kTile - 1) / kTile;
    const int k_n = max(k_hi - k_lo, 0);
    const int t_begin = k_lo + (int)((int64_t)k_n * part / ks), t_end = k_lo + (int)((int64_t)k_n * (part + 1) / ks);
    const int wrow0 = row0 + 32 * wave;
    const bool live = wrow0 < rows;
    const int wtok0 = min(wrow0, rows - 1) / a.group, wtok1 = min(wrow0 + 31, rows - 1) / a.group;
    const int w_hi = live ? key_hi(a, s, wtok1) : 0, w_lo = key_lo(a, s, wtok0);   // any row sees [w_lo, w_hi)
    const int all_hi = key_hi(a, s, wtok0), all_lo = key_lo(a, s, wtok1);          // every row sees [all_lo, all_hi)

    // ---- queries ----
    const int row = min(wrow0 + n, rows - 1);
    const int tok = row / a.group, hh = row - tok * a.group;
    const int r_hi = key_hi(a, s, tok), r_lo = key_lo(a, s, tok);
    v8i qf[S][PC];
    float mult;
    {
        const bool vec = (((uintptr_t)a.q | (uintptr_t)(2 * a.q_st) | (uintptr_t)(2 * a.q_sh)) & 15) == 0;
        const uint16_t* src = a.q + (int64_t)(s.q0 + tok) * a.q_st + (int64_t)(head * a.group + hh) * a.q_sh;
        uint32_t most = 0;
        for (int c = 0; c < 2 * S; ++c) {
            float x[16];
            load_q16<PC == 3>(src + 32 * c + 16 * h, vec, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) most = max(most, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const float up = row_power(most, a.scale, &mult);
#pragma unroll
        for (int c = 0; c < 2 * S; ++c) {
            float x[16];
            load_q16<PC == 3>(src + 32 * c + 16 * h, vec, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[4];
                uint32_t w[PC];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = up != 0.0f ? x[4 * j + i] * up : 0.0f;
                pieces4<PC>(y, w);
#pragma unroll
                for (int p = 0; p < PC; ++p) qf[c >> 1][p][4 * (c & 1) + j] = (int)w[p];
            }
        }
    }

    v16f o[DT];
    float m = neg_inf(), mu = 0.0f, l = 0.0f;
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;

    // ---- a step's copies: into registers, then (values widened) into LDS ----
    uint4 kc[KN];
    uint32_t vc[VN][4], vs[VN], ke = 0, kev = 0;
    auto page_of = [&](int key, bool* ok) {
        const int p = table[min(key, s.ctx - 1) >> ps];
        *ok = (uint32_t)p < (uint64_t)a.cache.pages;
        return (int64_t)(*ok ? p : 0) * hk + head;
    };
    const int mask = (1 << ps) - 1;
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int it = TH - 1 - tid + i * TH;   // from the end: few values, other threads
            if (it < KI) {
                const int key = t * kTile + it / KU, u = it % KU;
                bool ok;
                const int64_t ph = page_of(key, &ok);
                kc[i] = *reinterpret_cast<const uint4*>(a.cache.k_codes + ((ph << ps) + (key & mask)) * (D / 2) + 16 * u);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int it = tid + i * TH;
            if (it < VI) {
                const int q = it & 15, oct = it >> 4;
                const int key = t * kTile + 4 * q;
                bool ok;
                const int64_t ph = page_of(key, &ok);
                const uint8_t* c = a.cache.v_codes + ((ph << ps) + (key & mask)) * (D / 2) + 4 * oct;
#pragma unroll
                for (int j = 0; j < 4; ++j) vc[i][j] = *reinterpret_cast<const uint32_t*>(c + j * (D / 2));
                vs[i] = *reinterpret_cast<const uint32_t*>(a.cache.v_e8m0 + ((ph * KU + oct / 4) << ps) + (key & mask));
            }
        }
        if (tid < EI) {
            const int q = tid & 15, b = tid >> 4;
            const int key = t * kTile + 4 * q;
            bool ok;
            const int64_t ph = page_of(key, &ok);
            const int64_t at = ((ph * KU + b) << ps) + (key & mask);
            ke = *reinterpret_cast<const uint32_t*>(a.cache.k_e8m0 + at);
            kev = *reinterpret_cast<const uint32_t*>(a.cache.v_e8m0 + at);
            if (!ok) ke = 0xFFFFFFFFu;
        }
    };
    auto stage = [&](PrefillLds<D, NW>& b) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int it = TH - 1 - tid + i * TH;
            if (it < KI) {
                const int key = it / KU, u = it % KU;
                constexpr int RP = 256 / (D / 2);   // rows per 256 bytes of banks
                *reinterpret_cast<uint4*>(b.k + key * (D / 2) + 16 * (u ^ ((key / RP) & (KU - 1)))) = kc[i];
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int it = tid + i * TH;
            if (it < VI) {
                const int q = it & 15, oct = it >> 4;
                const uint32_t sb = vs[i] & ~bad_bytes(vs[i]);
                const float sc[4] = {byte_scale<0>(sb), byte_scale<1>(sb), byte_scale<2>(sb), byte_scale<3>(sb)};
                // the slots of keys 4q .. 4q+3: unit 2 (q / 4) + (q & 1), half (q / 2) & 1
                const int unit = 2 * (q >> 2) + (q & 1), half = (q >> 1) & 1;
                auto put = [&](auto B) {
                    constexpr int bb = decltype(B)::value;
                    uint32_t c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[j] = fp4_pair<bb>(vc[i][j], sc[j]);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const int d = 8 * oct + 2 * bb + odd;
                        const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                        *reinterpret_cast<uint2*>(b.v + d * kTile + 8 * (unit ^ ((d >> 1) & 7)) + 4 * half) =
                            make_uint2(__builtin_amdgcn_perm(c[1], c[0], sel), __builtin_amdgcn_perm(c[3], c[2], sel));
                    }
                };
                put(std::integral_constant<int, 0>{});
                put(std::integral_constant<int, 1>{});
                put(std::integral_constant<int, 2>{});
                put(std::integral_constant<int, 3>{});
            }
        }
        if (tid < EI) {
            const int q = tid & 15, blk = tid >> 4;
            const uint32_t e = ke | bad_bytes(kev);
            uint8_t* dst = b.e + ((((q >> 3) * 2 + (blk & 1)) * 32 + 4 * (q & 7)) * S) + (blk >> 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[j * S] = (uint8_t)(e >> (8 * j));
        }
    };

    if (t_begin < t_end) {
        fetch(t_begin);
        stage(lds[0]);
    }
    __syncthreads();
    for (int t = t_begin; t < t_end; ++t) {
        const PrefillLds<D, NW>& b = lds[(t - t_begin) & 1];
        const bool more = t + 1 < t_end;
        if (more) fetch(t + 1);
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            const int key0 = t * kTile + 32 * kt;
            if (key0 >= w_hi || key0 + 32 <= w_lo) continue;   // nothing here for this wave
            // ---- scores of 32 keys: register i of lane (n, h) is key 8 (i / 4) + 4 h + i % 4 ----
            v16f sc;
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
            const int key = 32 * kt + n;
            constexpr int RP = 256 / (D / 2);
            const uint8_t* krow = b.k + key * (D / 2);
            const int sw = (key / RP) & (KU - 1);
            const uint8_t* ep = b.e + ((kt * 2 + h) * 32 + n) * S;
            const int es = S == 4 ? *reinterpret_cast<const int*>(ep) : S == 2 ? *reinterpret_cast<const uint16_t*>(ep) : *ep;
            auto dot = [&](auto ST) {
                constexpr int st = decltype(ST)::value;
                const uint4 kq = *reinterpret_cast<const uint4*>(krow + 16 * ((2 * st + h) ^ sw));
                const v8i kf = {(int)kq.x, (int)kq.y, (int)kq.z, (int)kq.w, 0, 0, 0, 0};
#pragma unroll
                for (int p = 0; p < PC; ++p)
                    sc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf, qf[st][p], sc, kFmtFp4, kFmtFp8, st, es, 0,
                                                                        127 - 4 * p);
            };
            dot(std::integral_constant<int, 0>{});
            if constexpr (S > 1) dot(std::integral_constant<int, 1>{});
            if constexpr (S > 2) {
                dot(std::integral_constant<int, 2>{});
                dot(std::integral_constant<int, 3>{});
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] *= mult;
            if (key0 + 32 > all_hi || key0 < all_lo) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int k = key0 + 8 * (i / 4) + 4 * h + i % 4;
                    if (k >= r_hi || k < r_lo) sc[i] = neg_inf();
                }
            }
            // ---- running maximum, probabilities ----
            float mx = neg_inf();
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[i]);
            if (__any(mx > m + kLazy)) {
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mn = fmaxf(m, mx);
                const float un = mn == neg_inf() ? 0.0f : mn;
                const float f = exp2f(m - un);
                m = mn;
                mu = un;
                l *= f;
#pragma unroll
                for (int j = 0; j < DT; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[j][i] *= f;
            }
            uint32_t pf[2][4], pl[2][4];
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float p[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        p[x] = __builtin_amdgcn_exp2f(sc[8 * st + 2 * e + x] - mu);
                        l += p[x];
                    }
                    pack_p<PC>(p, &pf[st][e], &pl[st][e]);
                }
            // ---- values ----
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int j = 0; j < DT; ++j) {
                    const int d = 32 * j + n;
                    const v8h av = *reinterpret_cast<const v8h*>(b.v + d * kTile + 8 * ((4 * kt + 2 * st + h) ^ ((d >> 1) & 7)));
                    o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pf[st])), o[j], 0, 0, 0);
                    if (PC == 3)
                        o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pl[st])), o[j], 0, 0, 0);
                }
        }
        if (more) stage(lds[(t + 1 - t_begin) & 1]);
        __syncthreads();
    }

    l += __shfl_xor(l, 32);
    if (wrow0 + n >= rows) return;
    if (ks == 1) {
        uint16_t* dst = a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + hh) * D;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint2*>(dst + 32 * j + 8 * i + 4 * h) =
                    make_uint2(out_pair<PC == 3>(o[j][4 * i] * inv, o[j][4 * i + 1] * inv),
                               out_pair<PC == 3>(o[j][4 * i + 2] * inv, o[j][4 * i + 3] * inv));
    } else {
        float* p = reinterpret_cast<float*>(a.ws) +
                   (((int64_t)pair * tiles_max + tile) * ks + part) * part_floats(32 * NW, D);
        const int r = 32 * wave + n;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<v4f*>(p + (int64_t)r * D + 32 * j + 8 * i + 4 * h) =
                    v4f{o[j][4 * i], o[j][4 * i + 1], o[j][4 * i + 2], o[j][4 * i + 3]};
        if (h == 0) {
            p[(int64_t)32 * NW * D + r] = m;
            p[(int64_t)32 * NW * (D + 1) + r] = l;
        }
    }
}

template <int D, bool FP16>
__global__ __launch_bounds__(256) void prefill_join_kernel(const AttnArgs a, const int tiles_max, const int ks, const int tile_rows) {
    const uint32_t pair = blockIdx.x / (uint32_t)(a.max_q * a.group);
    const int row = (int)(blockIdx.x - pair * (uint32_t)(a.max_q * a.group));
    const int sq = pair / a.cache.kv_heads, head = pair - sq * a.cache.kv_heads;
    const Seq s = seq_of(a, sq);
    if (row >= s.qlen * a.group) return;
    const int tile = row / tile_rows;
    const int tok = row / a.group, h = row - tok * a.group;
    uint16_t* dst = a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + h) * D;
    const float* ws = reinterpret_cast<const float*>(a.ws);
    const int64_t size = part_floats(tile_rows, D);
    join_row<D, FP16>(ks, tile_rows, row - tile * tile_rows, dst,
                      [&](int i) { return ws + (((int64_t)pair * tiles_max + tile) * ks + i) * size; });
}

// ---------------------------------------------------------------------------
// routes (host)
// ---------------------------------------------------------------------------
struct Plan {
    bool decode;
    int nt;              // decode: 16-row tiles
    int workgroups;      // decode: runs of the line
    int nw;              // prompts: waves
    int tiles;           // prompts: row tiles per segment
    int ks;              // prompts: parts of the keys
};
// rows per key/value head up to which the decode kernel serves: its outputs fill
// 4 NT D/16 registers
constexpr int decode_rows(int D) { return D == 256 ? 32 : 64; }
constexpr int decode_tiles(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
int decode_workgroups() { return 2 * device_cus(); }
constexpr int prefill_waves(int D, bool fp16) { return D == 256 && fp16 ? 4 : 8; }

Plan plan_attention(int64_t seqs, int64_t max_q, int hq, int hk, int D, bool fp16) {
    Plan p{};
    const int64_t rows = max_q * (hq / hk);
    if (rows <= decode_rows(D)) {
        p.decode = true;
        p.nt = decode_tiles(rows);
        p.workgroups = decode_workgroups();
        return p;
    }
    p.nw = prefill_waves(D, fp16);
    p.tiles = (int)((rows + 32 * p.nw - 1) / (32 * p.nw));
    const int64_t grid = seqs * hk * p.tiles, cus = device_cus();
    p.ks = (int)(grid >= cus ? 1 : cus / grid);
    return p;
}

template <int D, int NT>
hipError_t go_decode(const AttnArgs& a, const Plan& p, bool fp16, hipStream_t st) {
    if (fp16) decode_kernel<D, NT, 3><<<p.workgroups, 256, 0, st>>>(a, p.workgroups);
    else decode_kernel<D, NT, 2><<<p.workgroups, 256, 0, st>>>(a, p.workgroups);
    return hipGetLastError();
}
template <int D>
hipError_t go_dim(const AttnArgs& a, const Plan& p, bool fp16, hipStream_t st) {
    hipError_t e;
    const dim3 join((unsigned)((int64_t)a.seqs * a.cache.kv_heads * a.max_q * a.group));
    if (p.decode) {
        if (p.nt == 1) e = go_decode<D, 1>(a, p, fp16, st);
        else if (p.nt == 2) e = go_decode<D, 2>(a, p, fp16, st);
        else if constexpr (D < 256) e = go_decode<D, 4>(a, p, fp16, st);
        else e = hipErrorInvalidValue;
        if (e != hipSuccess) return e;
        if (fp16) decode_join_kernel<D, true><<<join, 256, 0, st>>>(a, p.workgroups, 16 * p.nt);
        else decode_join_kernel<D, false><<<join, 256, 0, st>>>(a, p.workgroups, 16 * p.nt);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((int64_t)a.seqs * a.cache.kv_heads * p.tiles * p.ks));
    if (fp16) prefill_kernel<D, 3, D == 256 ? 4 : 8><<<grid, 64 * p.nw, 0, st>>>(a, p.tiles, p.ks);
    else prefill_kernel<D, 2, 8><<<grid, 64 * p.nw, 0, st>>>(a, p.tiles, p.ks);
    e = hipGetLastError();
    if (e != hipSuccess || p.ks == 1) return e;
    if (fp16) prefill_join_kernel<D, true><<<join, 256, 0, st>>>(a, p.tiles, p.ks, 32 * p.nw);
    else prefill_join_kernel<D, false><<<join, 256, 0, st>>>(a, p.tiles, p.ks, 32 * p.nw);
    return hipGetLastError();
}

}  // namespace

// Enough for every call of at most these sizes: fewer queries take the decode
// kernel (two partial results per run), fewer row tiles are split over the keys
// (at most one partial result per CU).
size_t attention_workspace_bytes(int64_t seqs, int64_t max_q, int hq, int hk, int D) {
    const int64_t rows = max_q * (hq / hk), most = decode_rows(D);
    int64_t floats = 2 * (int64_t)decode_workgroups() * part_floats(16 * decode_tiles(rows < most ? rows : most), D);
    if (rows > most) {
        const int64_t split = (int64_t)device_cus() * part_floats(32 * prefill_waves(D, false), D);
        if (split > floats) floats = split;
    }
    return (size_t)floats * 4;
}

hipError_t launch_attention(const AttnArgs& a, bool fp16, hipStream_t stream) {
    const Plan p = plan_attention(a.seqs, a.max_q, a.hq, a.cache.kv_heads, a.cache.head_dim, fp16);
    switch (a.cache.head_dim) {
        case 64: return go_dim<64>(a, p, fp16, stream);
        case 128: return go_dim<128>(a, p, fp16, stream);
        default: return go_dim<256>(a, p, fp16, stream);
    }
}

}  // namespace w4a8
