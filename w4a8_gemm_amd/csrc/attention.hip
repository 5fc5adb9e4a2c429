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
// p.v runs in bf16, where an e2m1 value times a power of two is exact, with p as
// the sum of two bf16 pieces (relative 2^-16): few query rows take them in about the
// time of one, as the keys' bytes bound them (the two cases below 67 and 71 us, 67 and
// 70 with one; 30 rows with 256 dims 59 for 54, 56 with 128 dims 85 for 74).  Prompts
// of bf16 queries, which the matrix pipe bounds, round p to one piece, relative 2^-8 at most
// as the output's own rounding: two took 1482 us for 880 in prompts of 8191 and 3533
// tokens (24 / 4 heads of 256 dims, whose registers spill) and 2654 for 2030 in two of
// 8192 unmasked (32 / 8 of 128).  Scores, sums and outputs accumulate in fp32.
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

// Sixteen 16-bit query values from p, in 8 dwords: 16-byte loads at any 2-byte
// alignment (strided views of a fused projection may start anywhere).
struct __attribute__((packed, aligned(2))) Half8 {
    uint32_t d[4];
};
__device__ __forceinline__ void load_q16(const uint16_t* p, uint32_t* d) {
    const Half8 u = reinterpret_cast<const Half8*>(p)[0], v = reinterpret_cast<const Half8*>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = u.d[j], d[4 + j] = v.d[j];
}
// the largest magnitude among 8 dwords of values, as fp32 bits
template <bool FP16>
__device__ __forceinline__ uint32_t most_of(const uint32_t* d, uint32_t most) {
    uint32_t m = 0;   // 16-bit patterns order like the magnitudes, NaN above infinity
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, max(d[j] & 0x7FFFu, (d[j] >> 16) & 0x7FFFu));
    if (FP16 && m >= 0x7C00u) return 0x7F800000u;
    return max(most, FP16 ? __float_as_uint(f16_to_f32(m)) : m << 16);
}
template <bool FP16>
__device__ __forceinline__ void widen4(const uint32_t* d, float* x) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        x[2 * j] = FP16 ? f16_to_f32(d[j] & 0xFFFFu) : bf16_to_f32(d[j] & 0xFFFFu);
        x[2 * j + 1] = FP16 ? f16_to_f32(d[j] >> 16) : bf16_to_f32(d[j] >> 16);
    }
}
// What a row's values are multiplied by before they are split: the power of two
// that takes its largest magnitude (fp32 bits) to [128, 256), with the softmax
// scale's sign; `mult`, positive, makes scores in log2 of the products.  A
// non-finite row's mult is NaN, and its pieces are zero.
__device__ __forceinline__ float row_power(uint32_t most, const AttnArgs& a, float* mult) {
    if (most >= 0x7F800000u) {
        *mult = __builtin_nanf("");
        return 0.0f;
    }
    if (a.scale == 0.0f) {
        *mult = 1.0f;
        return 0.0f;
    }
    const int e = max((int)(most >> 23) - 127, -119);
    *mult = fmaxf(a.scale_log2 * __uint_as_float((uint32_t)(127 - 7 + e) << 23), 0x1p-126f);
    const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
    return a.scale < 0.0f ? -up : up;
}

// byte mask of a dword's bytes >= 253
__device__ __forceinline__ uint32_t bad_bytes(uint32_t x) {
    const uint32_t f = ((x & 0x7F7F7F7Fu) + 0x03030303u) & x & 0x80808080u;
    return (f << 1) - (f >> 7);
}

// p as bf16 pieces: the rounded values, and (TWO) the rounded rest
template <bool TWO>
__device__ __forceinline__ void pack_p(const float* p, uint32_t* hi, uint32_t* lo) {
    *hi = pack_bf16(p[0], p[1]);
    if (TWO) *lo = pack_bf16(p[0] - __uint_as_float(*hi << 16), p[1] - __uint_as_float(*hi & 0xFFFF0000u));
}

// bf16 pairs of the e2m1 codes of byte B of x, times the power of two s
template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t x, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, B));
}
// an exponent byte in place of an fp32's exponent: 2^(byte - 127) to the conversions,
// which read that field alone, 0 too
template <int B>
__device__ __forceinline__ float byte_scale(uint32_t x) {
    const uint32_t s = B == 3 ? x >> 1 : B == 2 ? x << 7 : B == 1 ? x << 15 : x << 23;
    return __uint_as_float(s & 0x7F800000u);
}

template <bool FP16>
__device__ __forceinline__ uint32_t out_pair(float a, float b) {
    return FP16 ? pack_f16(a, b) : pack_bf16(a, b);
}

// ===========================================================================
// Few query rows per key/value head (single tokens, drafts): the keys stream.
//
// All sequences' tiles of 64 keys, head after head, form one line that is cut
// into equal runs, one per workgroup; a run may cross segments (one sequence's
// one head), and a segment that several runs share is joined by the last of
// them to arrive (below).  The cut follows the lengths in device memory, so the
// grid depends on none of them.
//
// A wave takes every NW-th tile of its workgroup's run.  Rows of 16 queries are
// the columns of the 16x16 products:
//   S^T = K Q^T: tile u of four holds keys 4r + u (r = row), so that a lane reads
//     the exponents of its four keys as one dword and picks by opsel;
//   lane (n, g) then holds query n's scores of keys 16g .. 16g+15;
//   O^T = V^T P^T: the product's k-slots are filled in that order, so P moves
//     between no lanes, and lane (n, g) reads from keys 16g .. 16g+15 the D/16
//     values of dims n D/16 ..: the transpose happens in its own registers.
// The next tile's loads are issued as soon as this one's registers are free:
// exponents and keys after the scores, values after the products.  Loads return
// in order, so nothing that is needed early is asked for late: the block-table
// entries of a run lie in LDS.  Bound by HBM: 64 sequences to 8192 keys (32 / 8 heads
// of 128 dims, 308 MB) take 67 us, three to 131072 keys (24 / 4 of 256, 316 MB) 71 us;
// the stream itself runs at 6 TB/s.
// ===========================================================================
template <int D>
struct VWord;   // D/16 e2m1 codes
template <> struct VWord<64> { typedef uint16_t T; static constexpr int N = 1; };
template <> struct VWord<128> { typedef uint32_t T; static constexpr int N = 1; };
template <> struct VWord<256> { typedef uint2 T; static constexpr int N = 2; };
__device__ __forceinline__ uint32_t vword(uint16_t v, int) { return v; }
__device__ __forceinline__ uint32_t vword(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t vword(uint2 v, int i) { return i ? v.y : v.x; }

// Tiles of a sequence: at least one while it has queries, so that rows without
// a key are written.  Its place on the line is longer by what a segment costs
// beside its tiles (queries in, results out: about the time of kSegment tiles),
// in whole steps of the four waves: short segments then get workgroups of their
// own, and a run through several of them takes no longer than the others.
constexpr int kSegment = 8;
__device__ __forceinline__ int first_tile(const AttnArgs& a, const Seq& s) { return key_lo(a, s, 0) / kTile; }
__device__ __forceinline__ int tiles_of(const AttnArgs& a, const Seq& q) {
    return max(1, (q.ctx + kTile - 1) / kTile - first_tile(a, q));
}
template <int NW>
__device__ __forceinline__ int place_of(const AttnArgs& a, int s) {
    const Seq q = seq_of(a, s);
    return q.qlen ? (tiles_of(a, q) + kSegment + NW - 1) & ~(NW - 1) : 0;
}
__device__ __forceinline__ int wave_scan(int v) {   // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// A workgroup's run [pos, end) of the line, and the sequence that holds its
// start: first position and length per head.
struct Run {
    int run;                 // per workgroup
    int pos, end;
    int seq, start, place;
};
// tiles of a wave up to which segments are not cut: a join takes as long
constexpr int kWhole = 2;
template <int NW>
__device__ __forceinline__ Run run_of(const AttnArgs& a, int workgroups) {
    const int lane = threadIdx.x & 63, hk = a.cache.kv_heads;
    const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    Run r;
    int n = lane < a.seqs ? place_of<NW>(a, lane) : 0, longest = n;
    int incl = wave_scan(n);
    int64_t t = __shfl(incl, 63);
    for (int s0 = 64; s0 < a.seqs; s0 += 64) {
        const int v = s0 + lane < a.seqs ? place_of<NW>(a, s0 + lane) : 0;
        longest = max(longest, v);
        t += __shfl(wave_scan(v), 63);
    }
    r.start = r.place = 0;
    if ((int64_t)a.seqs * hk <= workgroups && !__any(longest > NW * kWhole + kSegment)) {   // a workgroup each
        r.seq = (int)blockIdx.x / hk;
        r.place = r.seq < a.seqs ? uniform(place_of<NW>(a, r.seq)) : 0;
        if (r.place == 0) r.seq = a.seqs;
        r.pos = ((int)blockIdx.x - r.seq * hk) * r.place;
        r.run = r.place;
        r.end = r.pos + r.place;
        return r;
    }
    const int total = uniform((int)t * hk);
    r.run = uniform(max((total + workgroups - 1) / workgroups, NW));   // a tile for every wave
    const int64_t pos = (int64_t)blockIdx.x * r.run;
    r.pos = (int)min(pos, (int64_t)total);
    r.end = min(r.pos + r.run, total);
    r.seq = a.seqs;
    if (r.pos >= total) return r;
    int base = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
        if (s0) {
            n = s0 + lane < a.seqs ? place_of<NW>(a, s0 + lane) : 0;
            incl = wave_scan(n);
        }
        const int first = base + (incl - n) * hk;
        const uint64_t hit = __ballot(n > 0 && r.pos >= first && r.pos < first + n * hk);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            r.seq = s0 + l;
            r.start = uniform(__shfl(first, l));
            r.place = uniform(__shfl(n, l));
            break;
        }
        base += uniform(__shfl(incl, 63)) * hk;
    }
    return r;
}

// ---- joining the pieces of a segment ----
//
// Piece i of a segment belongs to workgroup w0 + i; its result (rows x D
// unnormalized outputs, the rows' maxima, their sums) lies in slot 2 w + 1 of
// the workspace where the segment begins in that run, else in slot 2 w.  Up to
// kJoin pieces are joined by the last of them to arrive, more in two rounds of
// about the root of their number.  Always in the pieces' order, so the result
// does not depend on which came last.  Nobody waits: a workgroup that is not last
// goes on.
constexpr int kJoin = 16;
constexpr int kJoinMost = 64;           // of one round: two rounds join 4096
__host__ __device__ constexpr int64_t part_floats(int rows, int D) { return (int64_t)rows * (D + 2); }
__host__ __device__ constexpr int64_t counter_words(int workgroups) { return (int64_t)2 * 2 * workgroups; }

__device__ __forceinline__ float ws_get(__amdgpu_buffer_rsrc_t ws, uint32_t at) {
    return __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(ws, (int)at, 0, 16));
}
__device__ __forceinline__ void ws_put(__amdgpu_buffer_rsrc_t ws, uint32_t at, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v), ws, (int)at, 0, 16);
}

// Joins `count` results (the j-th at slot(j)) of `rows` live rows: into slot(0),
// or normalized into the output.  R = rows of a slot; ml: 2 R kJoinMost floats.
template <int D, int R, int TH, bool FP16, typename SLOT, typename OUT>
__device__ __forceinline__ void join_pieces(__amdgpu_buffer_rsrc_t ws, SLOT slot, int count, int rows, bool final, OUT out,
                                            float* ml) {
    constexpr int C = D / 4;                // threads per row
    constexpr int RG = TH / C;
    constexpr int B = 8;                    // results in flight
    const int tid = threadIdx.x, c = tid % C;
    auto fetch = [&](sk_i32x4* v, int row, int j0) {
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (j0 + j < count) v[j] = sk_get4(ws, slot(j0 + j) + 4u * (uint32_t)(row * D + 4 * c));
    };
    int row = tid / C;
    sk_i32x4 v[B];
    if (row < rows) fetch(v, row, 0);
    for (int i = tid; i < rows * count; i += TH) {
        const int j = i / rows, r = i - j * rows;
        ml[j * R + r] = ws_get(ws, slot(j) + 4u * (uint32_t)(R * D + r));
        ml[(kJoinMost + j) * R + r] = ws_get(ws, slot(j) + 4u * (uint32_t)(R * D + R + r));
    }
    __syncthreads();
    for (; row < rows; row += RG) {
        float mx = neg_inf(), sum = 0.0f, acc[4] = {0, 0, 0, 0};
        for (int j = 0; j < count; ++j) mx = fmaxf(mx, ml[j * R + row]);
        const float u = mx == neg_inf() ? 0.0f : mx;
        for (int j0 = 0; j0 < count; j0 += B) {
            sk_i32x4 x[B];
#pragma unroll
            for (int j = 0; j < B; ++j) x[j] = v[j];
            if (j0 + B < count) fetch(v, row, j0 + B);
            else if (row + RG < rows) fetch(v, row + RG, 0);
#pragma unroll
            for (int j = 0; j < B; ++j)
                if (j0 + j < count) {
                    const float w = exp2f(ml[(j0 + j) * R + row] - u);
                    sum += ml[(kJoinMost + j0 + j) * R + row] * w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] += __int_as_float(x[j][i]) * w;
                }
        }
        if (final) {
            const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(out(row) + 4 * c) =
                make_uint2(out_pair<FP16>(acc[0] * f, acc[1] * f), out_pair<FP16>(acc[2] * f, acc[3] * f));
        } else {
            sk_put4(ws, slot(0) + 4u * (uint32_t)(row * D + 4 * c), acc[0], acc[1], acc[2], acc[3]);
            if (c == 0) {
                ws_put(ws, slot(0) + 4u * (uint32_t)(R * D + row), mx);
                ws_put(ws, slot(0) + 4u * (uint32_t)(R * D + R + row), sum);
            }
        }
    }
}

// waves per SIMD of four-wave workgroups: the outputs of many rows need the registers
// of two; with 64 dims there are registers for three, and the third hides changes of
// segments (3200 segments of 1620 keys on average 104 -> 96 us; with 128 dims it spills,
// and 512 segments took 72 us for 67)
constexpr int decode_waves(int D, int NT) { return NT * (D / 16) > 16 || NT == 4 ? 1 : NT == 1 && D == 64 ? 3 : 2; }
constexpr int kWavesMost = 3;

// NW waves to a workgroup.  Eight, one workgroup to a CU, where few segments have
// tiles for all of them: the runs are half as many pieces to join, and all waves keep
// step (of two workgroups the older is served first: equal runs ended after 40 and 55
// us).  Three contexts to 131072 keys 75 -> 71 us, eight of 4000 14.9 -> 13.7 us.  Four,
// two or three workgroups to a CU, where runs cross segments, so that one streams while
// another changes segments (16 sequences of four drafts on 8192 keys, 26.6 us with eight,
// 24.7 with four), and for short contexts (one of 1021 keys: 15.8 and 13.9 us).
template <int D, int NT, int PC, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 2 : decode_waves(D, NT)) void decode_kernel(const AttnArgs a, const int workgroups) {
    constexpr int KS = D >= 128 ? D / 128 : 1;      // 128-deep products per score
    constexpr int QP = D >= 128 ? PC : PC - 1;      // q operands per 128 (D = 64: pieces side by side)
    constexpr int DT = D / 16;                      // output tiles
    constexpr int C = D / 64;                       // runs of 16 query values per lane
    constexpr int R = NT * 16, TH = 64 * NW;
    typedef typename VWord<D>::T VT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int hk = a.cache.kv_heads, ps = a.page_shift;
    // queries while the keys stream; then the waves' results, rows padded by 16
    // bytes; then the joined pieces' maxima and sums
    constexpr int kRow = D + 4;
    constexpr int kQBytes = NT * KS * QP * 2048, kOBytes = NW * R * kRow * 4, kMBytes = 2 * R * kJoinMost * 4;
    constexpr int kBytes = kQBytes > kOBytes ? (kQBytes > kMBytes ? kQBytes : kMBytes) : (kOBytes > kMBytes ? kOBytes : kMBytes);
    __shared__ __attribute__((aligned(16))) uint8_t smem[kBytes];
    __shared__ float sm_m[NW][R], sm_l[NW][R];
    __shared__ uint32_t sm_flag;
    __shared__ int32_t sm_table[16 * kTile + 1];
    uint4* const sm_q = reinterpret_cast<uint4*>(smem);                 // [nt][k][p][half][lane]
    float* const sm_o = reinterpret_cast<float*>(smem);                 // [wave][row][kRow]
    uint32_t* const counters = reinterpret_cast<uint32_t*>(a.ws);
    float* const parts = reinterpret_cast<float*>(a.ws) + a.ws_skip;

    Run r = run_of<NW>(a, workgroups);
    if (r.seq >= a.seqs) return;

    while (r.pos < r.end) {
        const int head = (r.pos - r.start) / r.place;
        const int t0 = (r.pos - r.start) - head * r.place;
        const int span = min(r.place - t0, r.end - r.pos);      // on the line
        const Seq s = seq_of(a, r.seq);
        const int tiles = tiles_of(a, s);
        const int cnt = min(span, tiles - t0);                  // tiles among it
        r.pos += span;
        const int seq = r.seq, start = r.start, r_place = r.place;
        if (r.pos < r.end && t0 + span == r.place && head == hk - 1) {   // the next sequence with queries
            r.start += r.place * hk;
            for (r.place = 0; r.place == 0 && ++r.seq < a.seqs;) r.place = place_of<NW>(a, r.seq);
            if (r.seq >= a.seqs) r.end = r.pos;
        }
        if (cnt <= 0) continue;
        const int rows = s.qlen * a.group;
        const int first = first_tile(a, s);
        const int32_t* table = a.table + (int64_t)seq * a.table_stride;
        const int t_end = s.ctx > 0 ? first + t0 + cnt : 0;
        int t = first + t0 + wave;

        uint4 kc[KS][4];
        uint32_t ke[KS], k_bad = 0;
        VT vc[16];
        uint4 ve_next;
        const int last_key = s.ctx - 1;             // ctx >= 1 wherever it is used
        int page0 = 0;                              // the first of the block-table entries in LDS
        auto fill_table = [&](int from, int to) {   // those of tiles [from, to)
            page0 = (from * kTile) >> ps;
            const int count = (min(to * kTile - 1, last_key) >> ps) - page0 + 1;
            for (int i = threadIdx.x; i < count; i += TH) sm_table[i] = table[page0 + i];
        };
        // the page of a lane's four keys, and of its sixteen values; keys past the
        // context take the last one's (they are masked).  An entry outside the cache
        // makes its keys' scales NaN, at the product: a select here would wait for them.
        auto load_k = [&](int at) {
            const int pk = sm_table[(min(at * kTile + 4 * n, last_key) >> ps) - page0];
            const int pv = sm_table[(min(at * kTile + 16 * g, last_key) >> ps) - page0];
            {
                const int64_t ph = (int64_t)((uint32_t)pv < (uint64_t)a.cache.pages ? pv : 0) * hk + head;
                const int row = (at * kTile + 16 * g) & ((1 << ps) - 1);
                ve_next = *reinterpret_cast<const uint4*>(a.cache.v_e8m0 + ((ph * (D / 32) + n / (512 / D)) << ps) + row);
            }
            const bool ok = (uint32_t)pk < (uint64_t)a.cache.pages;
            k_bad = ok ? 0u : 0xFFFFFFFFu;
            const int64_t ph = (int64_t)(ok ? pk : 0) * hk + head;
            const int row = (at * kTile + 4 * n) & ((1 << ps) - 1);
            const uint8_t* c = a.cache.k_codes + ((ph << ps) + row) * (D / 2) + 16 * (D == 64 ? g & 1 : g);
            const uint8_t* e = a.cache.k_e8m0 + ((ph * (D / 32) + (D == 64 ? g & 1 : g)) << ps) + row;
#pragma unroll
            for (int k = 0; k < KS; ++k) ke[k] = *reinterpret_cast<const uint32_t*>(e + ((int64_t)(4 * k) << ps));
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < KS; ++k) kc[k][u] = *reinterpret_cast<const uint4*>(c + 64 * k + u * (D / 2));
        };
        auto load_v = [&](int at) {
            const int pv = sm_table[(min(at * kTile + 16 * g, last_key) >> ps) - page0];
            const int64_t ph = (int64_t)((uint32_t)pv < (uint64_t)a.cache.pages ? pv : 0) * hk + head;
            const int row = (at * kTile + 16 * g) & ((1 << ps) - 1);
            const uint8_t* c = a.cache.v_codes + ((ph << ps) + row) * (D / 2) + n * (D / 32);
#pragma unroll
            for (int k = 0; k < 16; ++k) vc[k] = *reinterpret_cast<const VT*>(c + k * (D / 2));
        };
        // tiles whose entries are in LDS together
        const int chunk = 16 << ps;
        int c_end = min(t_end, first + t0 + chunk);

        // ---- queries: every wave finds its rows' powers, and converts its share ----
        float mult[NT];
        int hi[NT], lo[NT];
        uint32_t x[NT][C][8], most[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = min(nt * 16 + n, rows - 1);
            const int tok = row / a.group, h = row - tok * a.group;
            hi[nt] = key_hi(a, s, tok);
            lo[nt] = key_lo(a, s, tok);
            const uint16_t* src = a.q + (int64_t)(s.q0 + tok) * a.q_st + (int64_t)(head * a.group + h) * a.q_sh + 16 * g;
#pragma unroll
            for (int c = 0; c < C; ++c) load_q16(src + 64 * c, x[nt][c]);
        }
        if (first + t0 < t_end) fill_table(first + t0, c_end);
        __syncthreads();                            // the table; the last segment's results are out
        // all of the queries are waited for here: past the branch their wait would be one
        // for the keys
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            most[nt] = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) most[nt] = most_of<PC == 3>(x[nt][c], most[nt]);
            asm volatile("" : "+v"(most[nt]));
        }
        if (t < c_end) {                            // the first tile's loads run meanwhile
            load_k(t);
            load_v(t);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            most[nt] = max(most[nt], (uint32_t)__shfl_xor((int)most[nt], 16));
            most[nt] = max(most[nt], (uint32_t)__shfl_xor((int)most[nt], 32));
            const float up = row_power(most[nt], a, &mult[nt]);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (((nt * C + c) & (NW - 1)) != wave) continue;
                uint32_t w[PC][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float y[4];
                    uint32_t v[PC];
                    widen4<PC == 3>(x[nt][c] + 2 * j, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = up != 0.0f ? y[i] * up : 0.0f;
                    pieces4<PC>(y, v);
#pragma unroll
                    for (int p = 0; p < PC; ++p) w[p][j] = v[p];
                }
                auto put = [&](int k, int p, int half, const uint32_t* v) {
                    sm_q[(((nt * KS + k) * QP + p) * 2 + half) * 64 + lane] = make_uint4(v[0], v[1], v[2], v[3]);
                };
                if constexpr (D >= 128) {
                    // run c: bytes 0-15 (d = 128 k + 16 g ..) or 16-31 (128 k + 64 + 16 g ..)
#pragma unroll
                    for (int p = 0; p < PC; ++p) put(c >> 1, p, c & 1, w[p]);
                } else {
                    // k < 64: the first piece, k >= 64: the second; then the third alone
                    put(0, 0, 0, w[0]);
                    put(0, 0, 1, w[1]);
                    if constexpr (PC == 3) {
                        const uint32_t zero[4] = {0, 0, 0, 0};
                        put(0, 1, 0, w[2]);
                        put(0, 1, 1, zero);
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
        __syncthreads();

        // ---- keys ----
        // every row sees all keys of [all_lo, all_hi)
        const int all_hi = a.causal ? s.ctx - s.q_all + 1 : s.ctx;
        const int all_lo = key_lo(a, s, s.qlen - 1);
        auto step = [&](auto MORE) {                // tile t; the wave's next one is in LDS's table
            constexpr bool more = decltype(MORE)::value;
            const int key0 = t * kTile;
            const bool masked = key0 + kTile > all_hi || key0 < all_lo;
            uint4 ve = ve_next;
#pragma unroll
            for (int k = 0; k < KS; ++k) ke[k] |= k_bad;
            // value blocks that count as NaN are rare, so found for the wave at once; then over
            // the head's blocks, the 16 lanes of g
            uint32_t bad[4] = {bad_bytes(ve.x), bad_bytes(ve.y), bad_bytes(ve.z), bad_bytes(ve.w)};
            const bool any_bad = __any((bad[0] | bad[1] | bad[2] | bad[3]) != 0);
            if (any_bad) {
                ve.x &= ~bad[0], ve.y &= ~bad[1], ve.z &= ~bad[2], ve.w &= ~bad[3];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int off = 1; off < 16; off <<= 1) bad[i] |= (uint32_t)__shfl_xor((int)bad[i], off);
            }
            uint32_t pf[NT][2][4], pl[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // ---- scores [tile u][i]: key 16 g + 4 i + u ----
                v4f acc[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u] = v4f{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int p = 0; p < QP; ++p) {
                        // D = 64: k >= 64 holds the next piece, its scale comes from lanes g = 2, 3
                        const int qs = D == 64 ? (p ? 119 : g < 2 ? 127 : 123) : 127 - 4 * p;
                        const uint4* qp = sm_q + ((nt * KS + k) * QP + p) * 128 + lane;
                        const uint4 q0 = qp[0], q1 = qp[64];
                        const v8i qf = {(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, (int)q1.x, (int)q1.y, (int)q1.z, (int)q1.w};
                        auto dot = [&](auto U) {
                            constexpr int u = decltype(U)::value;
                            const v8i kf = {(int)kc[k][u].x, (int)kc[k][u].y, (int)kc[k][u].z, (int)kc[k][u].w, 0, 0, 0, 0};
                            acc[u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf, qf, acc[u], kFmtFp4, kFmtFp8, u,
                                                                                      (int)ke[k], 0, qs);
                        };
                        dot(std::integral_constant<int, 0>{});
                        dot(std::integral_constant<int, 1>{});
                        dot(std::integral_constant<int, 2>{});
                        dot(std::integral_constant<int, 3>{});
                    }
                __builtin_amdgcn_sched_barrier(0);
                if (nt == NT - 1 && more) load_k(t + NW);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[u][i] *= mult[nt];
                if (any_bad) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((bad[i] >> (8 * u)) & 1u) acc[u][i] = __builtin_nanf("");
                }
                if (masked) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 16 * g + 4 * i + u;
                            if (key >= hi[nt] || key < lo[nt]) acc[u][i] = neg_inf();
                        }
                }
                // ---- running maximum, probabilities ----
                float mx = neg_inf();
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, acc[u][i]);
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
                        p[e] = __builtin_amdgcn_exp2f(acc[2 * st + e / 4][e % 4] - mu[nt]);
                        l[nt] += p[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) pack_p<true>(p + 2 * e, &pf[nt][st][e], &pl[nt][st][e]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
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
                            o[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pl[nt][st])), o[nt][j], 0, 0, 0);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);   // one pair's words at a time, or they fill the registers
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
            if (more) load_v(t + NW);
        };
        while (true) {
            if (t < c_end) {
                for (; t + NW < c_end; t += NW) {
                    step(std::true_type{});
                    // all waves have a next tile: in step (loads in flight are not awaited)
                    if (NW == 8 && t - wave + 2 * NW <= c_end) __builtin_amdgcn_s_barrier();
                }
                step(std::false_type{});
                t += NW;
            }
            if (c_end >= t_end) break;
            __syncthreads();                        // the next tiles' entries
            const int c0 = c_end;
            c_end = min(t_end, c0 + chunk);
            fill_table(c0, c_end);
            __syncthreads();
            if (t < c_end) {
                load_k(t);
                load_v(t);
            }
        }

        // ---- the waves' results ----
        __syncthreads();                            // the queries are read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] += __shfl_xor(l[nt], 16);
            l[nt] += __shfl_xor(l[nt], 32);
            const int row = nt * 16 + n;
            if (row < rows) {
                if (g == 0) {
                    sm_m[wave][row] = m[nt];
                    sm_l[wave][row] = l[nt];
                }
                float* dst = sm_o + (wave * R + row) * kRow + 4 * DT * g;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < DT; j += 4)
                        *reinterpret_cast<v4f*>(dst + DT * i + j) = v4f{o[nt][j][i], o[nt][j + 1][i], o[nt][j + 2][i], o[nt][j + 3][i]};
            }
        }
        __syncthreads();
        const bool whole = cnt == tiles;
        auto out_row = [&](int row) {
            const int tok = row / a.group, h = row - tok * a.group;
            return a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + h) * D;
        };
        constexpr uint32_t kPart = (uint32_t)(4 * part_floats(R, D));
        const __amdgpu_buffer_rsrc_t ws = sk_rsrc(parts);
        const uint32_t mine = (2u * blockIdx.x + (t0 == 0 ? 1u : 0u)) * kPart;
        for (int i = threadIdx.x; i < rows * (D / 4); i += TH) {
            const int row = i / (D / 4), c = i - row * (D / 4);
            float mx = neg_inf(), sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm_m[w][row]);
            const float u = mx == neg_inf() ? 0.0f : mx;
            v4f acc = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = exp2f(sm_m[w][row] - u);    // 0 without a key (NaN outputs stay NaN)
                sum += sm_l[w][row] * f;
                acc += *reinterpret_cast<const v4f*>(sm_o + (w * R + row) * kRow + 4 * c) * f;
            }
            if (whole) {
                const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<uint2*>(out_row(row) + 4 * c) =
                    make_uint2(out_pair<PC == 3>(acc[0] * f, acc[1] * f), out_pair<PC == 3>(acc[2] * f, acc[3] * f));
            } else {
                sk_put4(ws, mine + 4u * (uint32_t)(row * D + 4 * c), acc[0], acc[1], acc[2], acc[3]);
                if (c == 0) {
                    ws_put(ws, mine + 4u * (uint32_t)(R * D + row), mx);
                    ws_put(ws, mine + 4u * (uint32_t)(R * D + R + row), sum);
                }
            }
        }
        if (!whole) {
            const int g0 = start + head * r_place, w0 = g0 / r.run;
            int pieces = (g0 + tiles - 1) / r.run - w0 + 1, at = (int)blockIdx.x - w0, step = 1;
            int fan = pieces;
            if (pieces > kJoin)
                for (fan = kJoin / 2; fan * fan < pieces;) ++fan;
            for (int level = 0; pieces > 1; ++level) {
                const int lead = at / fan * fan;            // among this round's
                const int count = min(fan, pieces - lead);
                // the j-th result's slot: its first run's
                auto id = [&](int j) {
                    const int p = (lead + j) * step;
                    return 2u * (uint32_t)(w0 + p) + (p == 0 ? 1u : 0u);
                };
                if (!sk_arrive(counters + (int64_t)level * 2 * workgroups + id(0), count, &sm_flag)) break;
                const bool final = pieces <= fan;
                join_pieces<D, R, TH, PC == 3>(ws, [&](int j) { return id(j) * kPart; }, count, rows, final, out_row,
                                           reinterpret_cast<float*>(smem));
                pieces = (pieces + fan - 1) / fan;
                at /= fan;
                step *= fan;
            }
            __syncthreads();                        // the flag is read
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

// ===========================================================================
// Many query rows (prompts, chunks of prompts): the matrix pipe is the bound.
//
// A workgroup of NW waves holds 32 NW rows of one segment, a wave 32 of them as
// the columns of 32x32 products; KT keys per step, shared through LDS: the
// keys' codes as they are (fp4 operand), the values widened to bf16 and
// transposed once for all waves.
//
// A wave's step has two halves: products (outputs of the step before, scores of
// this one) and the rest (probabilities, its share of widening the values).
// Waves w and w + 4 share a SIMD, so with eight waves the second four run half a
// step behind: while one wave of a SIMD multiplies, the other exponentiates.  Half
// steps are kept apart by barriers.  Prompts of 8191 and 3533 tokens (24 / 4 heads of
// 256 dims) take 885 us, 1105 TFLOP/s, the matrix pipe busy in 45 % of the cycles; two
// of 8192 unmasked with 32 / 8 heads of 128 dims 2.05 ms, 1075 TFLOP/s.
// In half step x (tile i):
//   first four waves    x = 2i: products(i)           x = 2i+1: rest(i), widen(i)
//   second four waves   x = 2i: rest(i-1), widen(i)   x = 2i+1: products(i)
// products(i) reads keys i and values i-1; widen(i) makes values i (over i-2) and
// the exponents of keys i+1 (over i-1), which the half step before read last.
//
// Codes and exponents come by direct copies to LDS, kAhead steps before their
// use, into rings of eight tiles (two steps and four tiles with 256 dims): keys
// i+1+kAhead and values i+kAhead are asked for in widen(i), and what widen(i+1)
// and products(i+1) read is waited for before the barrier that ends it.
//
// Where there are too few workgroups for the chip the keys are cut into up to
// `ks` parts, joined by a second kernel.
// ===========================================================================
// keys per step: with 256 dims the outputs and queries leave registers for the
// scores of 32
constexpr int prefill_keys(int D) { return D == 256 ? 32 : 64; }
constexpr int kTable = 1024;
// the queries' last piece lies in LDS where two waves of a SIMD share its
// registers with the outputs of 256 dims
constexpr bool prefill_q_lds(int D, int NW) { return D == 256 && NW == 8; }
template <int D, int NW>
struct PrefillLds {
    static constexpr int KT = prefill_keys(D);
    static constexpr bool kQ = prefill_q_lds(D, NW);
    static constexpr int kAhead = kQ ? 2 : 3, kRing = kQ ? 4 : 8;
    uint8_t k[kRing][KT * D / 2];            // row key, 16-byte units XOR-swizzled
    uint8_t vr[kRing][KT * D / 2];           // the values' codes, likewise
    uint8_t er[kRing][2][KT * D / 32];       // exponents of keys and values, [32-block][key]
    uint8_t e[2][KT * 2 * (D / 64)];         // the keys' as scale operands: [32-key tile][h][row][64-step]
    uint16_t v[2][D * KT];                   // values: [d][slot], 16-byte units XOR-swizzled
    uint4 q[kQ ? NW : 1][kQ ? D / 64 : 1][2][64];   // [wave][64-step][half][lane]
    int32_t table[kTable + 1];
};

// Copies of 16 or 4 bytes a lane from p to LDS at base + lane's place.  Inline, as
// the compiler would drain them before every LDS read; awaited by wait_copies.
// No register is written, so none can be reused under a copy in flight.  m0 takes a
// wait state to reach the copy that reads it; the compiler adds none in asm.
__device__ __forceinline__ void copy16(const uint8_t* p, uint32_t base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const uint8_t* p, uint32_t base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(base) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {   // at most N of this wave's still in flight
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_at(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(p));
}

// N times: a matrix product, then an LDS read
template <int N>
__device__ __forceinline__ void sched_pairs() {
    if constexpr (N > 0) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        sched_pairs<N - 1>();
    }
}

// The key tiles [lo, lo + n) that a workgroup's rows [row0, row0 + count) see, and
// the parts that they are cut into: of `ks`, as many as have kPartSteps of them
// (a part costs the time of about as many beside its own; three prompts of 17
// tokens cut into 21 parts took 24 us, uncut 17).
constexpr int kPartSteps = 16;
struct Span {
    int lo, n, parts;
};
template <int D>
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int row0, int count, int ks) {
    constexpr int KT = prefill_keys(D);
    const int last = (min(row0 + count, s.qlen * a.group) - 1) / a.group;
    Span r;
    r.lo = key_lo(a, s, row0 / a.group) / KT;
    r.n = max((max(key_hi(a, s, last), 0) + KT - 1) / KT - r.lo, 0);
    r.parts = min(ks, max(r.n / kPartSteps, 1));
    return r;
}

template <int D, int PC, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void prefill_kernel(const AttnArgs a, const int tiles_max, const int ks) {
    constexpr int TH = 64 * NW;
    constexpr int S = D / 64;                       // 64-deep products per score
    constexpr int DT = D / 32;                      // 32-wide output tiles
    constexpr int KU = D / 32;                      // 16-byte units of a key
    constexpr int KT = prefill_keys(D), NK = KT / 32;
    constexpr int KQ = KT / 4;                      // groups of four keys
    constexpr int KI = KT * KU / 64;                // copies of a wave for a tile's keys (or values)
    constexpr int EI = KQ * KU;                     // dwords of exponents
    constexpr int VI = KQ * (D / 4), VN = (VI + TH - 1) / TH;   // four keys by four dims each
    constexpr int KR = 256 / (D / 2), VR = 256 / (2 * KT);      // rows per 256 bytes of LDS banks
    static_assert(KI <= 4 && EI <= 64, "the copies' shares below");
    typedef PrefillLds<D, NW> Lds;
    constexpr int kRing = Lds::kRing, kAhead = Lds::kAhead;
    constexpr int PR = Lds::kQ ? PC - 1 : PC;       // pieces of the queries in registers
    __shared__ __attribute__((aligned(16))) Lds lds;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = NW == 8 ? wave >> 2 : 0;
    const int n = lane & 31, h = lane >> 5;
    const int hk = a.cache.kv_heads, ps = a.page_shift;

    // The rows' last tiles first: with causal masks they are the longest.  The pair
    // moves on from tile to tile, so that the XCDs (workgroup mod 8) share the
    // sequences of different lengths alike.
    const int pairs = a.seqs * hk;
    int bid = blockIdx.x;
    const int part = bid % ks;
    bid /= ks;
    const int turn = bid / pairs;
    const int pair = (bid + turn) % pairs, tile = tiles_max - 1 - turn;
    const int sq = pair / hk, head = pair - sq * hk;
    const Seq s = seq_of(a, sq);
    const int rows = s.qlen * a.group;
    const int row0 = tile * 32 * NW;
    if (row0 >= rows) return;
    const int32_t* table = a.table + (int64_t)sq * a.table_stride;

    // keys of the workgroup, of its part, and of this wave
    const Span span = span_of<D>(a, s, row0, 32 * NW, ks);
    if (part >= span.parts) return;
    const int t_begin = span.lo + (int)((int64_t)span.n * part / span.parts);
    const int t_end = span.lo + (int)((int64_t)span.n * (part + 1) / span.parts);
    const int wrow0 = row0 + 32 * wave;
    const bool live = wrow0 < rows;
    const int wtok0 = min(wrow0, rows - 1) / a.group, wtok1 = min(wrow0 + 31, rows - 1) / a.group;
    const int w_hi = live ? key_hi(a, s, wtok1) : 0, w_lo = key_lo(a, s, wtok0);   // any row sees [w_lo, w_hi)
    const int all_hi = key_hi(a, s, wtok0), all_lo = key_lo(a, s, wtok1);          // every row sees [all_lo, all_hi)

    // ---- queries ----
    const int row = min(wrow0 + n, rows - 1);
    const int tok = row / a.group, hh = row - tok * a.group;
    const int r_hi = key_hi(a, s, tok), r_lo = key_lo(a, s, tok);
    v8i qf[S][PR];
    float mult;
    {
        const uint16_t* src = a.q + (int64_t)(s.q0 + tok) * a.q_st + (int64_t)(head * a.group + hh) * a.q_sh;
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < 2 * S; ++c) {
            uint32_t x[8];
            load_q16(src + 32 * c + 16 * h, x);
            most = most_of<PC == 3>(x, most);
        }
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const float up = row_power(most, a, &mult);
        if (r_hi <= r_lo) mult = 1.0f;              // no keys: zeros, whatever the query holds
#pragma unroll
        for (int c = 0; c < 2 * S; ++c) {
            uint32_t x[8];
            load_q16(src + 32 * c + 16 * h, x);
            uint32_t last[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[4];
                uint32_t w[PC];
                widen4<PC == 3>(x + 2 * j, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = up != 0.0f ? y[i] * up : 0.0f;
                pieces4<PC>(y, w);
#pragma unroll
                for (int p = 0; p < PR; ++p) qf[c >> 1][p][4 * (c & 1) + j] = (int)w[p];
                last[j] = w[PC - 1];
            }
            if constexpr (Lds::kQ) lds.q[wave][c >> 1][c & 1][lane] = make_uint4(last[0], last[1], last[2], last[3]);
        }
    }

    v16f o[DT], sc[NK];
    uint32_t pf[NK][2][4], pl[NK][2][4];            // [32-key tile][16-key step]: probabilities, fp16: their rest
    float m = neg_inf(), mu = 0.0f, l = 0.0f;
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;

    // ---- copies of tile t (absolute) into ring slot r ----
    const int mask = (1 << ps) - 1, last_key = s.ctx - 1;
    int page0 = 0;                                  // the first of the table's entries in LDS
    auto entry = [&](int key) { return lds.table[(min(key, last_key) >> ps) - page0]; };
    auto head_of = [&](int p) { return (int64_t)((uint32_t)p < (uint64_t)a.cache.pages ? p : 0) * hk + head; };
    auto copy_codes = [&](const uint8_t* codes, uint8_t* ring, int t, int c, bool value) {
        const int slot = 64 * c + lane, kr = slot / KU, u = slot % KU;      // LDS: row, physical unit
        const int key = t * KT + kr;
        // keys: swizzled by the row, values by the group of four
        const int from = u ^ ((value ? kr / 4 : kr / KR) & (KU - 1));
        copy16(codes + ((head_of(entry(key)) << ps) + (key & mask)) * (D / 2) + 16 * from, lds_at(ring + 1024 * c));
    };
    auto copy_exps = [&](const uint8_t* exps, uint8_t* ring, int t) {
        if (lane < EI) {
            const int key = t * KT + 4 * (lane % KQ);
            copy4(exps + ((head_of(entry(key)) * KU + lane / KQ) << ps) + (key & mask), lds_at(ring));
        }
    };
    // The waves' shares: with eight waves the first four copy keys, the second four
    // values; each at most one of codes, and one wave of each also exponents.
    const int cw = NW == 8 ? wave & 3 : wave;
    const bool my_k = group == 0 && cw < KI, my_v = (NW == 4 || group == 1) && cw < KI;
    const bool my_ke = NW == 8 ? wave == 0 : wave == 0, my_ve = NW == 8 ? wave == 4 : wave == 1;
    constexpr int kEach = NW == 8 ? 1 : 2;          // copies of codes per wave and step
    auto ask_k = [&](int t, int r) {
        if (my_k) copy_codes(a.cache.k_codes, lds.k[r & (kRing - 1)], t, cw, false);
        if (my_ke) copy_exps(a.cache.k_e8m0, lds.er[r & (kRing - 1)][0], t);
    };
    auto ask_v = [&](int t, int r) {
        if (my_v) copy_codes(a.cache.v_codes, lds.vr[r & (kRing - 1)], t, cw, true);
    };
    auto ask_ve = [&](int t, int r) {
        if (my_ve) copy_exps(a.cache.v_e8m0, lds.er[r & (kRing - 1)][1], t);
    };

    // ---- exponents of the keys of tile i as scale operands ----
    auto scales = [&](int i, int t) {
        if (tid < EI) {
            const int q = tid % KQ, blk = tid / KQ;
            const uint8_t(*r)[KT * D / 32] = lds.er[i & (kRing - 1)];
            const bool ok = (uint32_t)entry(t * KT + 4 * q) < (uint64_t)a.cache.pages;
            const uint32_t ke = *reinterpret_cast<const uint32_t*>(r[0] + 4 * tid);
            const uint32_t kv = *reinterpret_cast<const uint32_t*>(r[1] + 4 * tid);
            const uint32_t e = ok ? ke | bad_bytes(kv) : 0xFFFFFFFFu;
            uint8_t* dst = lds.e[i & 1] + ((((q >> 3) * 2 + (blk & 1)) * 32 + 4 * (q & 7)) * S) + (blk >> 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[j * S] = (uint8_t)(e >> (8 * j));
        }
    };
    // ---- values of tile i widened: a thread four keys by four dims ----
    auto widen = [&](int i) {
        uint16_t* const dst = lds.v[i & 1];
        const uint8_t* const raw = lds.vr[i & (kRing - 1)];
        const uint8_t* const exps = lds.er[i & (kRing - 1)][1];
#pragma unroll
        for (int w = 0; w < VN; ++w) {
            const int it = tid + w * TH;
            if (it < VI) {
                const int q = it % KQ, c = it / KQ;             // dims 4c .. 4c+3
                const uint32_t sv = *reinterpret_cast<const uint32_t*>(exps + (c >> 3) * KT + 4 * q);
                const uint32_t sb = sv & ~bad_bytes(sv);
                const float f[4] = {byte_scale<0>(sb), byte_scale<1>(sb), byte_scale<2>(sb), byte_scale<3>(sb)};
                const uint8_t* src = raw + 4 * q * (D / 2) + 16 * ((c >> 3) ^ (q & (KU - 1))) + 2 * (c & 7);
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint16_t*>(src + j * (D / 2));
                // the slots of keys 4q .. 4q+3: unit 2 (q / 4) + (q & 1), half (q / 2) & 1
                const int unit = 2 * (q >> 2) + (q & 1), half = (q >> 1) & 1;
                auto put = [&](auto B) {
                    constexpr int bb = decltype(B)::value;
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fp4_pair<bb>(x[j], f[j]);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const int d = 4 * c + 2 * bb + odd;
                        const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                        *reinterpret_cast<uint2*>(dst + d * KT + 8 * (unit ^ ((d / VR) & (KT / 8 - 1))) + 4 * half) =
                            make_uint2(__builtin_amdgcn_perm(y[1], y[0], sel), __builtin_amdgcn_perm(y[3], y[2], sel));
                    }
                };
                put(std::integral_constant<int, 0>{});
                put(std::integral_constant<int, 1>{});
            }
        }
    };

    // ---- products ----
    auto outputs = [&](int i, int kt) {             // of tile i
        const uint16_t* bv = lds.v[i & 1];
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int j = 0; j < DT; ++j) {
                const int d = 32 * j + n;
                const v8h av = *reinterpret_cast<const v8h*>(bv + d * KT + 8 * ((4 * kt + 2 * st + h) ^ ((d / VR) & (KT / 8 - 1))));
                o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pf[kt][st])), o[j], 0, 0, 0);
                if (PC == 3)
                    o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        av, __builtin_bit_cast(v8h, *reinterpret_cast<const uint4*>(pl[kt][st])), o[j], 0, 0, 0);
            }
    };
    // scores of 32 keys: register x of lane (n, h) is key 8 (x / 4) + 4 h + x % 4
    auto scores = [&](int i, int kt) {
        const int key = 32 * kt + n;
        const uint8_t* krow = lds.k[i & (kRing - 1)] + key * (D / 2);
        const int sw = (key / KR) & (KU - 1);
        const uint8_t* ep = lds.e[i & 1] + ((kt * 2 + h) * 32 + n) * S;
        const int es = S == 4 ? *reinterpret_cast<const int*>(ep) : S == 2 ? *reinterpret_cast<const uint16_t*>(ep) : *ep;
        v16f acc;
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[x] = 0.0f;
        auto dot = [&](auto ST) {
            constexpr int st = decltype(ST)::value;
            const uint4 kq = *reinterpret_cast<const uint4*>(krow + 16 * ((2 * st + h) ^ sw));
            const v8i kf = {(int)kq.x, (int)kq.y, (int)kq.z, (int)kq.w, 0, 0, 0, 0};
#pragma unroll
            for (int p = 0; p < PC; ++p) {
                v8i qp;
                if (Lds::kQ && p == PC - 1) {
                    const uint4 q0 = lds.q[wave][st][0][lane], q1 = lds.q[wave][st][1][lane];
                    qp = v8i{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, (int)q1.x, (int)q1.y, (int)q1.z, (int)q1.w};
                } else
                    qp = qf[st][p];
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kf, qp, acc, kFmtFp4, kFmtFp8, st, es, 0, 127 - 4 * p);
            }
        };
        dot(std::integral_constant<int, 0>{});
        if constexpr (S > 1) dot(std::integral_constant<int, 1>{});
        if constexpr (S > 2) {
            dot(std::integral_constant<int, 2>{});
            dot(std::integral_constant<int, 3>{});
        }
        sc[kt] = acc;
    };
    // ---- running maximum, probabilities of the tile at key0 ----
    auto rest = [&](int key0) {
        if (key0 + KT > all_hi || key0 < all_lo) {
#pragma unroll
            for (int kt = 0; kt < NK; ++kt)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int k = key0 + 32 * kt + 8 * (x / 4) + 4 * h + x % 4;
                    if (k >= r_hi || k < r_lo) sc[kt][x] = neg_inf();
                }
        }
        float mx = neg_inf();
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int x = 0; x < 16; ++x) mx = fmaxf(mx, sc[kt][x]);
        mx *= mult;                                 // positive, or NaN with the row
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
                for (int x = 0; x < 16; ++x) o[j][x] *= f;
        }
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float p[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        p[x] = __builtin_amdgcn_exp2f(fmaf(sc[kt][8 * st + 2 * e + x], mult, -mu));
                        l += p[x];
                    }
                    pack_p<PC == 3>(p, &pf[kt][st][e], &pl[kt][st][e]);
                }
    };

    // runs of tiles whose block-table entries fit in LDS
    const int chunk = (kTable << ps) / KT;
    for (int c0 = t_begin; c0 < t_end; c0 += chunk) {
        const int tiles = min(chunk, t_end - c0);
        page0 = (c0 * KT) >> ps;
        const int count = (min((c0 + tiles) * KT - 1, last_key) >> ps) - page0 + 1;
        for (int i = tid; i < count; i += TH) lds.table[i] = table[page0 + i];
        __syncthreads();
        for (int i = 0; i <= kAhead; ++i)
            if (i < tiles) {
                ask_k(c0 + i, i);
                ask_ve(c0 + i, i);
                if (i < kAhead) ask_v(c0 + i, i);
            }
        wait_copies<0>();
        __syncthreads();
        scales(0, c0);
        __syncthreads();
        auto ahead = [&](int i) {                   // the copies and widening of step i
            const bool more = i + 1 + kAhead < tiles;
            if (more) {
                ask_k(c0 + i + 1 + kAhead, i + 1 + kAhead);
                ask_ve(c0 + i + 1 + kAhead, i + 1 + kAhead);
            }
            if (i + kAhead < tiles) ask_v(c0 + i + kAhead, i + kAhead);
            return more;
        };
        auto finish = [&](int i, bool more) {
            if (i + 1 < tiles) scales(i + 1, c0 + i + 1);
            if (i < tiles) widen(i);
            if (!more) wait_copies<0>();
            else if (my_ke || my_ve) wait_copies<(kEach + 1) * (kAhead - 1)>();
            else wait_copies<kEach * (kAhead - 1)>();
        };
        if (group) {
            const bool more = ahead(0);
            finish(0, more);
            __syncthreads();
        }
        auto idle = [&](int i) {
            __syncthreads();
            const bool more = ahead(i + group);
            finish(i + group, more);
            __syncthreads();
        };
        // the tiles in which this wave sees a key
        const int see_lo = min(max(w_lo / KT - c0, 0), tiles);
        const int see_hi = w_hi > w_lo ? min(max((w_hi + KT - 1) / KT - c0, see_lo), tiles) : see_lo;
        int i = 0;
        for (; i < see_lo; ++i) idle(i);
        if (Lds::kQ && i < see_hi)
#pragma unroll
            for (int kt = 0; kt < NK; ++kt) scores(i, kt);
        for (; i < see_hi; ++i) {
            if (!Lds::kQ)
#pragma unroll
                for (int kt = 0; kt < NK; ++kt) scores(i, kt);
            // here, or the compiler sinks the products past the barrier to their first use
#pragma unroll
            for (int kt = 0; kt < NK; ++kt) asm volatile("" : "+v"(sc[kt]));
            __syncthreads();
            const bool more = ahead(i + group);
            rest((c0 + i) * KT);
#pragma unroll
            for (int kt = 0; kt < NK; ++kt)
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        asm volatile("" : "+v"(pf[kt][st][e]));
                        if (PC == 3) asm volatile("" : "+v"(pl[kt][st][e]));
                    }
            finish(i + group, more);
            __syncthreads();
            if constexpr (Lds::kQ) {
                // With the scores of the next tile (past the last one they are of whatever the
                // rings hold, and not used) in one block, whose LDS reads run kDeep ahead of
                // its products: left to itself the compiler waits for each read.
                constexpr int kReads = NK * (2 * DT + S + 2 * S + 1), kProducts = NK * (2 * DT + S * PC), kDeep = 4;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int kt = 0; kt < NK; ++kt) outputs(i, kt);
#pragma unroll
                for (int kt = 0; kt < NK; ++kt) scores(i + 1, kt);
                __builtin_amdgcn_sched_group_barrier(0x100, kDeep, 0);
                sched_pairs<(kReads - kDeep < kProducts ? kReads - kDeep : kProducts)>();
                __builtin_amdgcn_sched_barrier(0);
            } else {
#pragma unroll
                for (int kt = 0; kt < NK; ++kt) outputs(i, kt);
            }
        }
        for (; i < tiles; ++i) idle(i);
        __syncthreads();                            // the rings and the table are free
        if (NW == 8 && !group) __syncthreads();
    }

    l += __shfl_xor(l, 32);
    if (wrow0 + n >= rows) return;
    if (span.parts == 1) {
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
        float* p = reinterpret_cast<float*>(a.ws) + a.ws_skip +
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

// A workgroup joins `per` rows of a pair, one after another.
template <int D, bool FP16>
__global__ __launch_bounds__(256) void prefill_join_kernel(const AttnArgs a, const int tiles_max, const int ks, const int tile_rows,
                                                           const int per) {
    const uint32_t blocks = (uint32_t)((a.max_q * a.group + per - 1) / per);
    const uint32_t pair = blockIdx.x / blocks;
    const int row0 = (int)(blockIdx.x - pair * blocks) * per;
    const int sq = pair / a.cache.kv_heads, head = pair - sq * a.cache.kv_heads;
    const Seq s = seq_of(a, sq);
    const float* ws = reinterpret_cast<const float*>(a.ws) + a.ws_skip;
    const int64_t size = part_floats(tile_rows, D);
    for (int row = row0; row < min(row0 + per, s.qlen * a.group); ++row) {
        const int tile = row / tile_rows;
        const int parts = span_of<D>(a, s, tile * tile_rows, tile_rows, ks).parts;
        if (parts == 1) continue;
        const int tok = row / a.group, h = row - tok * a.group;
        uint16_t* dst = a.out + ((int64_t)(s.q0 + tok) * a.hq + head * a.group + h) * D;
        join_row<D, FP16>(parts, tile_rows, row - tile * tile_rows, dst,
                          [&](int i) { return ws + (((int64_t)pair * tiles_max + tile) * ks + i) * size; });
        __syncthreads();                            // join_row's LDS is read
    }
}

// ---------------------------------------------------------------------------
// routes (host)
// ---------------------------------------------------------------------------
struct Plan {
    bool decode;
    int nt;              // decode: 16-row tiles
    int workgroups;      // decode: runs of the line
    int nw;              // waves of a workgroup
    int tiles;           // prompts: row tiles per segment
    int ks;              // prompts: parts of the keys
};
// rows per key/value head up to which the decode kernel serves: its outputs fill
// 4 NT D/16 registers
constexpr int decode_rows(int D) { return D == 256 ? 32 : 64; }
constexpr int decode_tiles(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
constexpr int prefill_waves(int D, bool fp16) { return D == 256 && fp16 ? 4 : 8; }

// Parts of the keys: what fills whole rounds of the CUs best, fewest first; a
// step up has to fill a tenth more; `most` for the longest context.  Two rounds and
// more of row tiles are not cut.  (Two chunks of 512 tokens on 30000 keys, 96 row
// tiles: 789 us with two parts, 675 with five.)
constexpr int kSplitRounds = 3;
int split_of(int64_t grid, int64_t cus, int64_t most) {
    if (grid >= 2 * cus) return 1;
    int best = 1;
    double fill = 0;
    for (int64_t ks = 1; ks <= most && grid * ks <= kSplitRounds * cus; ++ks) {
        const int64_t rounds = (grid * ks + cus - 1) / cus;
        const double f = (double)(grid * ks) / (double)(rounds * cus);
        if (f > 1.1 * fill) best = (int)ks, fill = f;
    }
    return best;
}

Plan plan_attention(int64_t seqs, int64_t max_q, int64_t keys, int hq, int hk, int D, bool fp16) {
    Plan p{};
    const int64_t rows = max_q * (hq / hk);
    if (rows <= decode_rows(D)) {
        p.decode = true;
        p.nt = decode_tiles(rows);
        const int64_t tiles = seqs * hk * ((keys + kTile - 1) / kTile), cus = device_cus();
        p.nw = decode_waves(D, p.nt) >= 2 && 4 * seqs * hk <= cus && tiles >= 8 * cus ? 8 : 4;
        p.workgroups = (int)cus * (p.nw == 4 ? decode_waves(D, p.nt) : 1);
        return p;
    }
    p.nw = prefill_waves(D, fp16);
    p.tiles = (int)((rows + 32 * p.nw - 1) / (32 * p.nw));
    p.ks = split_of(seqs * hk * p.tiles, device_cus(), keys / (prefill_keys(D) * kPartSteps));
    return p;
}

template <int D, int NT, int NW>
hipError_t go_waves(const AttnArgs& a, const Plan& p, bool fp16, hipStream_t st) {
    if (fp16) decode_kernel<D, NT, 3, NW><<<p.workgroups, 64 * NW, 0, st>>>(a, p.workgroups);
    else decode_kernel<D, NT, 2, NW><<<p.workgroups, 64 * NW, 0, st>>>(a, p.workgroups);
    return hipGetLastError();
}
template <int D, int NT>
hipError_t go_decode(const AttnArgs& a, const Plan& p, bool fp16, hipStream_t st) {
    if constexpr (decode_waves(D, NT) >= 2)
        if (p.nw == 8) return go_waves<D, NT, 8>(a, p, fp16, st);
    return go_waves<D, NT, 4>(a, p, fp16, st);
}
template <int D>
hipError_t go_dim(const AttnArgs& a, const Plan& p, bool fp16, hipStream_t st) {
    hipError_t e;
    if (p.decode) {
        if (p.nt == 1) return go_decode<D, 1>(a, p, fp16, st);
        if (p.nt == 2) return go_decode<D, 2>(a, p, fp16, st);
        if constexpr (D < 256) return go_decode<D, 4>(a, p, fp16, st);
        return hipErrorInvalidValue;
    }
    const dim3 grid((unsigned)((int64_t)a.seqs * a.cache.kv_heads * p.tiles * p.ks));
    if (fp16) prefill_kernel<D, 3, D == 256 ? 4 : 8><<<grid, 64 * p.nw, 0, st>>>(a, p.tiles, p.ks);
    else prefill_kernel<D, 2, 8><<<grid, 64 * p.nw, 0, st>>>(a, p.tiles, p.ks);
    e = hipGetLastError();
    if (e != hipSuccess || p.ks == 1) return e;
    // rows per workgroup: about eight of them on a CU, most with nothing to join where contexts are short
    const int64_t pairs = (int64_t)a.seqs * a.cache.kv_heads, rows = (int64_t)a.max_q * a.group;
    const int64_t share = pairs * rows / (8 * (int64_t)device_cus());
    const int per = (int)(share < 1 ? 1 : share > 8 ? 8 : share);
    const dim3 join((unsigned)(pairs * ((rows + per - 1) / per)));
    if (fp16) prefill_join_kernel<D, true><<<join, 256, 0, st>>>(a, p.tiles, p.ks, 32 * p.nw, per);
    else prefill_join_kernel<D, false><<<join, 256, 0, st>>>(a, p.tiles, p.ks, 32 * p.nw, per);
    return hipGetLastError();
}

}  // namespace

// The joins' counters, then enough for every call of at most these sizes: fewer
// queries take the decode kernel (two partial results per run), fewer row tiles
// are split over the keys (at most kSplitRounds partial results per CU).
size_t attention_counter_bytes() { return (size_t)(4 * counter_words(kWavesMost * device_cus())); }
size_t attention_workspace_bytes(int64_t seqs, int64_t max_q, int hq, int hk, int D) {
    const int64_t rows = max_q * (hq / hk), most = decode_rows(D);
    int64_t floats = 2 * kWavesMost * (int64_t)device_cus() * part_floats(16 * decode_tiles(rows < most ? rows : most), D);
    if (rows > most) {
        const int64_t split = (int64_t)kSplitRounds * device_cus() * part_floats(32 * prefill_waves(D, false), D);
        if (split > floats) floats = split;
    }
    return attention_counter_bytes() + (size_t)floats * 4;
}

namespace {
Plan plan_of(const AttnArgs& a, bool fp16) {
    // the most keys that a sequence's queries see
    const int64_t room = (int64_t)a.table_width << a.page_shift, reach = (int64_t)a.window + a.max_q;
    return plan_attention(a.seqs, a.max_q, a.window && reach < room ? reach : room, a.hq, a.cache.kv_heads, a.cache.head_dim, fp16);
}
}  // namespace

int64_t attention_threads(const AttnArgs& a, bool fp16) {
    const Plan p = plan_of(a, fp16);
    return p.decode ? (int64_t)64 * p.nw * p.workgroups : (int64_t)a.seqs * a.cache.kv_heads * p.tiles * p.ks * 64 * p.nw;
}

hipError_t launch_attention(const AttnArgs& args, bool fp16, hipStream_t stream) {
    AttnArgs a = args;
    a.ws_skip = (int64_t)attention_counter_bytes() / 4;
    a.scale_log2 = fabsf(a.scale) * kLog2e;
    const int64_t room = (int64_t)a.table_width << a.page_shift;
    if (a.window >= room) a.window = 0;             // none; key_lo's differences stay above -2^31
    const Plan p = plan_of(a, fp16);
    switch (a.cache.head_dim) {
        case 64: return go_dim<64>(a, p, fp16, stream);
        case 128: return go_dim<128>(a, p, fp16, stream);
        default: return go_dim<256>(a, p, fp16, stream);
    }
}

}  // namespace w4a8
