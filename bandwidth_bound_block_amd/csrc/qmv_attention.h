// Attention of new tokens over a quantized paged cache: what its kernels and
// entry points share, and the streaming kernel for few rows of queries.
//
// Mathematics.  Scores are block sums, s = sum_b d_b (q . c)_b (+ m_b sum q),
// with the codes c small integers, exact in fp16, as are 16-bit queries (bf16
// ones after a power of two per row): v_mfma_f32_16x16x32_f16 multiplies 16
// keys by 16 query rows over one block of 32 values, and one multiply-add per
// score applies the block's scale.  The softmax runs over the keys with a
// running maximum and sum.  For the second product V's codes become fp16
// values, and the weights go from the result registers of the first straight
// into the operand of the second: with two tiles t of 16 keys, a lane has
// after the first product the keys 16 t + 4 g + r (g = lane / 16, r < 4) of
// query lane % 16, and the second takes in lane group g eight keys in any
// order as long as both operands have the same.  With bf16 queries the weights
// and values are rounded to fp16 (2^-11; the outputs to 2^-8).  With fp16 or
// fp32 queries they are pairs of fp16 pieces, fp32 queries too: fp16 outputs
// had twice the error of their own rounding without.  That costs little here
// (131000 tokens: 41 us, bf16 34) and twice the time where arithmetic is the
// bound.  Weights go up to 2^14 (kALow), so that small ones keep their digits.
//
// The transposition that V needs (a lane multiplies eight keys of one place of
// the head) happens inside the lane: it loads the same few values of its eight
// keys and pairs neighbouring keys' halves with v_perm.
//
// Work.  Units are (request, key/value head, tile of rows), each with its own
// number of 32-key blocks; all units' blocks in a row are cut into equal
// shares, one workgroup each, so one long request fills the GPU and many
// ragged ones leave no tail, without a length on the host.  A workgroup's
// four waves split each unit's blocks of the share.  What does not end a unit
// goes to the workspace and is joined by a second launch.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "qmv_block_decode.h"
#include "qmv_cache.h"

namespace qmv {

constexpr int kAWaves = 4, kAT = 64 * kAWaves;
constexpr int kAShares = 1024;      // workgroups of the streaming kernel at most
constexpr int kABlock = 32;
// A part of a unit costs its blocks and a beginning and an end (queries, the
// first loads' latency, the meeting of the waves) of about this many: units
// count as that much longer, the additional blocks first.  With 4, 8 and 16: 64
// requests of 200..8000 tokens 73, 64 and 56 us, 200 of 20..500 tokens 57, 52
// and 50, 16 x 5 fp32 queries 37.2, 35.4 and 34.5, one request of 131000 43, 41
// and 41; one of 700 the same.
constexpr int kABegin = 8;

struct AttnArgs {
    CacheSide k, v;
    int64_t n_pages;
    int32_t page_shift, H, G, R;
    uint32_t g_mul, g_shift;        // row / G = row * g_mul >> (31 + g_shift)
    const void* q;
    int64_t qst, qsh;
    bool qvec;
    int64_t n_tokens, max_q;
    const int32_t* table;
    int64_t max_pages;
    const int32_t* lens;
    const int32_t* q_begin;
    float scale;
    int32_t window;
    const float* sinks;
    void* out;
    int32_t x_type;
    // workspace of the streaming kernel
    int64_t* prefix;                // [R + 1]: blocks of all units before request r's; [R + 1]: a share's blocks
    int32_t stream_to, tile_over;   // a request's rows up to which the streaming kernel takes it, over which the tile kernel
    float* tile_part;               // split tiles: [splits][n_tokens][heads][D], then (maximum, sum) of each
    float* part;                    // [2 * shares][rows][D], then maxima and sums [2 * shares][rows] each
};

// Rows of queries of a unit of the streaming kernel: one tile of 16, or two
// where a request can have more and the registers allow.
inline int stream_tiles(int64_t max_rows, int D) { return max_rows > 16 && D < 256 ? 2 : 1; }

// Per K format and pieces: launch the streaming kernel and the joining one.
int32_t attn_stream_q8_0_1(const AttnArgs& a, int D, hipStream_t st);
int32_t attn_stream_q8_0_2(const AttnArgs& a, int D, hipStream_t st);
int32_t attn_stream_q4_0_1(const AttnArgs& a, int D, hipStream_t st);
int32_t attn_stream_q4_0_2(const AttnArgs& a, int D, hipStream_t st);
int32_t attn_stream_q4_1_1(const AttnArgs& a, int D, hipStream_t st);
int32_t attn_stream_q4_1_2(const AttnArgs& a, int D, hipStream_t st);
// Rows of a tile of the kernel for many rows.
inline int tile_rows(int D, int32_t x_type) { return D * (x_type == QMV_X_BF16 ? 1 : 2) <= 256 ? 256 : 128; }
// Per pieces: launch the kernel for many rows, its tiles split over the keys.
int32_t attn_tile_1(const AttnArgs& a, int D, int splits, hipStream_t st);
int32_t attn_tile_2(const AttnArgs& a, int D, int splits, hipStream_t st);

namespace {

constexpr float kANone = -0x1p127f; // the maximum of no score: scores are less than 2^126 either way
// The running maximum is kept this much lower than the largest score, in units
// of log 2: weights go up to 2^14 (fp16 holds 65504), so that those far below
// the largest keep their digits.  As numbers of up to 1 they were 0 from 2^-25
// on, and beside one key with nearly all the weight and no value the output was
// lost (18 nats under it: two thirds); now from 2^-39 on, 27 nats.
constexpr float kALow = 14.f;
// Scores (times log2 e) from which on fp32 has no halves: a score's product
// and its maximum, rounded, may differ by any power of two, so that weights
// are infinite or all 0.  A part whose maximum is that far from 0 is done
// again in the careful pass, where both are rounded alike before their
// difference, which is 0 for the largest, and the maximum is kept as it is.
// (Looked for in every step it costs 1% to 4%.)
constexpr float kAFar = 0x1p24f;
__device__ __forceinline__ float lowered(float most) { return most - (__builtin_fabsf(most) < kAFar ? kALow : 0.f); }
__device__ __forceinline__ bool is_far(float m) { return __builtin_fabsf(m) >= kAFar && m > kANone; }

struct Req {
    int64_t q0;                     // first query token
    int n, len;                     // query tokens (max_q at most), keys up to the last one's
    int lo, blk0, nblk;             // first key seen, first block, blocks of a unit
    int tiles;                      // tiles of rows
    __device__ int cost() const { return nblk + kABegin; }
    bool bad;
};
template <int NT>
__device__ __forceinline__ Req request(const AttnArgs& a, int r) {
    Req o;
    int64_t b, e;
    if (a.q_begin) {
        b = min(max((int64_t)a.q_begin[r], (int64_t)0), a.n_tokens);
        e = min(max((int64_t)a.q_begin[r + 1], b), a.n_tokens);
    } else {
        b = r * a.max_q;
        e = b + a.max_q;
    }
    o.q0 = b;
    o.n = (int)min(e - b, a.max_q);
    const int len = a.lens[r];
    o.bad = len < 0 || len > (a.max_pages << a.page_shift);
    // queries past max_q are left out with their own keys, which no other query sees: the others stand where they stood
    o.len = o.bad ? 0 : (int)(len - (e - b - o.n));
    o.lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)o.len - o.n - a.window + 1) : 0;
    o.blk0 = o.lo / kABlock;
    o.nblk = max(1, (int)(((int64_t)o.len + kABlock - 1) / kABlock) - o.blk0);
    const int rows = o.n * a.G;                                          // n_tokens * G < 2^31
    o.tiles = rows > a.stream_to ? 0 : (int)(((int64_t)rows + 16 * NT - 1) / (16 * NT));
    return o;
}

// a / b for uniform numbers that nearly always have 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// max and sum over the four lane groups that hold a query
__device__ __forceinline__ float groups_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// Where a workgroup's share lies among all units' blocks.  By every wave for
// itself, 64 requests at a time: nothing passes between waves.
struct Share {
    int64_t total, size;
    int r;               // the request that holds the share's first block
    int64_t first;       // blocks before it
};
template <int NT>
__device__ __forceinline__ int64_t blocks_of(const AttnArgs& a, int r, int64_t& units) {
    if (r >= a.R) return 0;
    const Req q = request<NT>(a, r);
    units += (int64_t)q.tiles * a.H;
    return (int64_t)q.cost() * q.tiles * a.H;
}
template <int NT>
__device__ __forceinline__ Share find_share(const AttnArgs& a, int wg, int wgs) {
    const int lane = threadIdx.x & 63;
    const auto scan = [&](int64_t v) {          // inclusive, over the lanes
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t t = __shfl_up(v, o);
            if (lane >= o) v += t;
        }
        return v;
    };
    const auto last = [&](int64_t v, int l) {
        return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane((int)v, l));
    };
    Share s;
    int64_t units = 0, mine = blocks_of<NT>(a, lane, units), at = scan(mine);
    s.total = last(at, 63);
    for (int r0 = 64; r0 < a.R; r0 += 64) s.total += last(scan(blocks_of<NT>(a, r0 + lane, units)), 63);
    units = last(scan(units), 63);
    // at least a block for each wave, where units have as many
    s.size = max(quotient(s.total + wgs - 1, wgs), max(min(quotient(s.total, max(units, (int64_t)1)), (int64_t)kAWaves), (int64_t)1));
    const int64_t pos = wg * s.size;
    s.r = 0;
    s.first = 0;
    int64_t before = 0;
    for (int r0 = 0;;) {
        const int64_t first = before + at - mine;
        if (wg == 0 && r0 + lane < a.R && threadIdx.x < 64) a.prefix[r0 + lane] = first;
        const uint64_t who = __ballot(mine > 0 && pos >= first && pos < first + mine);
        if (who) {
            const int l = __builtin_ctzll(who);
            s.r = r0 + l;
            s.first = last(first, l);
            if (wg != 0) break;
        }
        before += last(at, 63);
        r0 += 64;
        if (r0 >= a.R) break;
        mine = blocks_of<NT>(a, r0 + lane, units);
        at = scan(mine);
    }
    if (wg == 0 && threadIdx.x == 0) {
        a.prefix[a.R] = s.total;
        a.prefix[a.R + 1] = s.size;
    }
    return s;
}

// Eight elements of the queries from element i on: as they are stored, bf16 (P 1), or fp16 or fp32 (P 2).
template <int P>
__device__ __forceinline__ void load_q8(const AttnArgs& a, int64_t i, uint32_t (&w)[4 * P]) {
    const bool f32 = P == 2 && a.x_type == QMV_X_F32;
    const uint8_t* p = static_cast<const uint8_t*>(a.q) + i * (f32 ? 4 : 2);
    if (a.qvec) {
#pragma unroll
        for (int k = 0; k < P; ++k) {
            if (k && !f32) continue;
            const u32x4 u = reinterpret_cast<const u32x4*>(p)[k];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * k + j] = u[j];
        }
    } else if (f32) {
#pragma unroll
        for (int j = 0; j < 4 * P; ++j) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = reinterpret_cast<const uint16_t*>(p)[2 * j] | (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * j + 1] << 16;
    }
}
template <int P>
__device__ __forceinline__ void widen_q8(const AttnArgs& a, const uint32_t (&w)[4 * P], float (&x)[8]) {
    if constexpr (P == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __builtin_bit_cast(float, w[j] << 16);
            x[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xffff0000u);
        }
    } else if (a.x_type == QMV_X_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_bit_cast(float, w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = (float)as_h2(w[j])[0];
            x[2 * j + 1] = (float)as_h2(w[j])[1];
        }
    }
}
// row / G of a row of a request's queries (query token times G + head of the group), for rows below 2^31.
__device__ __forceinline__ int token_of(const AttnArgs& a, int row) {
    return (int)(((uint64_t)(uint32_t)row * a.g_mul) >> (31 + a.g_shift));
}
__device__ __forceinline__ void store_out4(const AttnArgs& a, int64_t i, f32x4 x) {    // i a multiple of 4
    if (a.x_type == QMV_X_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + i) = x;
    } else if (a.x_type == QMV_X_F16) {
        const _Float16 e[4] = {(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
        __builtin_memcpy(static_cast<_Float16*>(a.out) + i, e, 8);
    } else {
        const __bf16 e[4] = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
        __builtin_memcpy(static_cast<__bf16*>(a.out) + i, e, 8);
    }
}

// A sink's logit in units of log 2.  Past fp32 it is its largest number, which
// no score comes near: the difference of two infinities would be NaN.
__device__ __forceinline__ float sink_of(const AttnArgs& a, int hq) {
    const float sk = a.sinks[hq] * 1.44269504088896341f;
    return sk > 0x1.fffffep127f ? 0x1.fffffep127f : sk;
}
// Sums x and l relative to the maximum m, of query head hq, to outputs.
__device__ __forceinline__ void finish(const AttnArgs& a, int hq, float m, float l, f32x4& x, bool bad) {
    if (a.sinks) {
        const float sk = sink_of(a, hq), top = fmaxf(m, sk);
        const float f = __builtin_amdgcn_exp2f(m - top);
        x *= f;
        l = l * f + __builtin_amdgcn_exp2f(sk - top);
    }
    const float inv = bad ? __builtin_nanf("") : l == 0.f ? 0.f : 1.f / l;      // a query that sees nothing: sums of 0
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= inv;
}

// A row's power of two: |q| 2^shift < 2^15 throughout.  A row that is not
// finite gives NaN.
__device__ __forceinline__ int row_shift(float amax) {
    return amax > 0.f ? 14 - (int)((__builtin_bit_cast(uint32_t, amax) >> 23) & 255) + 127 : 0;
}
// What sums over a row of queries times 2^shift, in units of 2^unit, are
// multiplied by: the rest of the scale, for scores in units of log 2.  Not 0, as what is out of sight is -inf times it.  Sums are
// less than 2^15 * 65024 * 256 units (< 2^39): up to 2^87 scores stay within
// fp32, and more would change nothing (two sums are a unit's 2^-48 apart at
// least, or alike).
__device__ __forceinline__ float row_factor(const AttnArgs& a, int shift, int unit) {
    return fminf(fmaxf(__builtin_ldexpf(a.scale, -shift - unit) * 1.44269504088896341f, 1e-37f), __builtin_ldexpf(1.f, 87 - unit));
}

constexpr int row_bytes_of(int F, int D) { return F == QMV_Q8_0 ? D : D / 2; }

// A stage: 32 keys' codes, values' codes, scales and minimums in a wave's own
// part of LDS, loaded straight into it in 16-byte chunks.  The chunks lie so
// that no read meets bank conflicts of more than two:
//   K  rows in order of the keys; in rows of 8 chunks or more chunk q at
//      place q ^ (key mod chunks);
//   V  the row of key 16 t + 4 g + r at 16 t + 4 g + (r + g) mod 4: the four
//      lane groups read four rows that differ modulo 4;
//   then [plane][block][t][half] chunks of 8 keys' scales.
template <int KF, int VF, int NB>
struct Stage {
    static constexpr int D = 32 * NB;
    static constexpr int kKRow = row_bytes_of(KF, D), kVRow = row_bytes_of(VF, D);
    static constexpr int kKC = kKRow / 16, kVC = kVRow / 16;             // chunks of a row
    static constexpr int kKSwz = kKC >= 8 ? kKC - 1 : 0;
    static constexpr int kKP = KF == QMV_Q4_1 ? 2 : 1, kVP = VF == QMV_Q4_1 ? 2 : 1;      // planes
    static constexpr int kV = 32 * kKRow, kS = kV + 32 * kVRow;          // offsets
    static constexpr int kSC = 4 * NB * (kKP + kVP);                     // scale chunks
    static constexpr int kBytes = kS + 16 * kSC;
    static constexpr int kKL = kKRow / 32, kVL = kVRow / 32, kSL = (kSC + 63) / 64;      // loads
    static constexpr int kLoads = kKL + kVL + kSL;
    static constexpr int kKW = kKRow / 16;                               // words of K a lane has of a key
    static constexpr int kVW = kVRow >= 64 ? kVRow / 64 : 1;             // words of V a lane has of a key
    static constexpr int kVB = NB == 8 ? 2 : 1;                          // blocks that a lane's places are of
};

// LDS reads with their wait in one asm: for plain reads the compiler waits for
// all loads into LDS on their way.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {      // N consecutive words
    static_assert(N == 2 || N == 4);
    if constexpr (N == 2) {
        uint2 a;
        asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(a) : "v"(at) : "memory");
        w[0] = a.x; w[1] = a.y;
    } else {
        u32x4 a;
        asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(a) : "v"(at) : "memory");
        w[0] = a[0]; w[1] = a[1]; w[2] = a[2]; w[3] = a[3];
    }
}
// 16-byte chunks at N addresses.
__device__ __forceinline__ void lds_chunks2(uint32_t a, uint32_t b, u32x4& x, u32x4& y) {
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x), "=&v"(y) : "v"(a), "v"(b) : "memory");
}
// N pairs of words, STEP bytes apart.
template <int N, int STEP>
__device__ __forceinline__ void lds_pairs(uint32_t at, uint2 (&w)[N]) {
    static_assert(N == 1 || N == 2 || N == 4 || N == 8);
    if constexpr (N == 1) {
        asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(w[0]) : "v"(at) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ds_read_b64 %0, %2\n\tds_read_b64 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0]), "=&v"(w[1]) : "v"(at), "n"(STEP) : "memory");
    } else if constexpr (N == 4) {
        asm volatile("ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:%5\n\tds_read_b64 %2, %4 offset:%6\n\t"
                     "ds_read_b64 %3, %4 offset:%7\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3])
                     : "v"(at), "n"(STEP), "n"(2 * STEP), "n"(3 * STEP) : "memory");
    } else {
        uint2 a[4], b[4];
        lds_pairs<4, STEP>(at, a);
        lds_pairs<4, STEP>(at + 4 * STEP, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = a[i];
            w[4 + i] = b[i];
        }
    }
}
// Values' words of the keys 4 g + r of both tiles: rows at four addresses, the second tile STEP bytes on.
template <int BYTES, int STEP>
__device__ __forceinline__ void lds_values(const uint32_t (&at)[4], uint32_t (&w)[8][BYTES <= 4 ? 1 : BYTES / 4]) {
    if constexpr (BYTES == 2) {
        asm volatile("ds_read_u16 %0, %8\n\tds_read_u16 %1, %9\n\tds_read_u16 %2, %10\n\tds_read_u16 %3, %11\n\t"
                     "ds_read_u16 %4, %8 offset:%12\n\tds_read_u16 %5, %9 offset:%12\n\tds_read_u16 %6, %10 offset:%12\n\t"
                     "ds_read_u16 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0][0]), "=&v"(w[1][0]), "=&v"(w[2][0]), "=&v"(w[3][0]), "=&v"(w[4][0]), "=&v"(w[5][0]),
                       "=&v"(w[6][0]), "=&v"(w[7][0])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(STEP) : "memory");
    } else if constexpr (BYTES == 4) {
        asm volatile("ds_read_b32 %0, %8\n\tds_read_b32 %1, %9\n\tds_read_b32 %2, %10\n\tds_read_b32 %3, %11\n\t"
                     "ds_read_b32 %4, %8 offset:%12\n\tds_read_b32 %5, %9 offset:%12\n\tds_read_b32 %6, %10 offset:%12\n\t"
                     "ds_read_b32 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(w[0][0]), "=&v"(w[1][0]), "=&v"(w[2][0]), "=&v"(w[3][0]), "=&v"(w[4][0]), "=&v"(w[5][0]),
                       "=&v"(w[6][0]), "=&v"(w[7][0])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(STEP) : "memory");
    } else if constexpr (BYTES == 8) {
        uint2 x[8];
        asm volatile("ds_read_b64 %0, %8\n\tds_read_b64 %1, %9\n\tds_read_b64 %2, %10\n\tds_read_b64 %3, %11\n\t"
                     "ds_read_b64 %4, %8 offset:%12\n\tds_read_b64 %5, %9 offset:%12\n\tds_read_b64 %6, %10 offset:%12\n\t"
                     "ds_read_b64 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(STEP) : "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i][0] = x[i].x;
            w[i][1] = x[i].y;
        }
    } else {
        u32x4 x[8];
        asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
                     "ds_read_b128 %4, %8 offset:%12\n\tds_read_b128 %5, %9 offset:%12\n\tds_read_b128 %6, %10 offset:%12\n\t"
                     "ds_read_b128 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
                     : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(STEP) : "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = x[i][j];
    }
}
// A barrier for LDS alone: this wave's stores to memory are not waited for.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

typedef __attribute__((address_space(3))) void* lds_ptr;
// 16 bytes a lane from p to LDS at `to` + 16 lane.
__device__ __forceinline__ void load_chunks(const uint8_t* p, uint8_t* to) {
    __builtin_amdgcn_global_load_lds(p, (lds_ptr)to, 16, 0, 0);
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p);
}

// 0xffff in each half of w that is an infinity or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((((w & 0x7c007c00u) + 0x04000400u) >> 15) & 0x00010001u) * 0xffffu;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) { return (a & b) | c; }

// One of the eight fp16 values that an octet of codes stands for, of two
// neighbouring keys side by side.
template <int F>
__device__ __forceinline__ f16x2 scaled(f16x2 c, f16x2 d, f16x2 m) {
    if constexpr (F == QMV_Q4_1) return __builtin_elementwise_fma(c, d, m);
    else return c * d;
}
// What scaled() leaves, as a second fp16 piece.  c d is exact in two pieces;
// with a minimum, the error of the sum of its first piece and m as well (the
// six steps are exact).  With care also where c d is past fp16 though c d + m
// is not (a block with values near both ends of the range), which gives NaN
// without: those steps on halves, and twice their outcome.
template <int F, bool CARE>
__device__ __forceinline__ f16x2 scaled_rest(f16x2 c, f16x2 d, f16x2 m, f16x2& first) {
#pragma clang fp contract(off)
    if constexpr (F == QMV_Q4_1) {      // fused into other multiply-adds these steps would not be exact
        f16x2 back = h2(1.f);
        if constexpr (CARE) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool wide = __builtin_fabsf((float)d[i]) >= 4096.f;       // 15 * 4096 < 65504
                d[i] = wide ? d[i] * (_Float16)0.5f : d[i];
                m[i] = wide ? m[i] * (_Float16)0.5f : m[i];
                back[i] = wide ? (_Float16)2.f : (_Float16)1.f;
            }
        }
        const f16x2 p = c * d, e = __builtin_elementwise_fma(c, d, -p);
        const f16x2 s = p + m, z = s - p;
        const f16x2 rest = (p - (s - z)) + (m - z) + e;
        first = CARE ? s * back : s;
        return CARE ? rest * back : rest;
    } else {
        first = c * d;
        return __builtin_elementwise_fma(c, d, -first);
    }
}

__device__ __forceinline__ f16x8 pack8(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Waves per SIMD, and so workgroups per compute unit: what the accumulators and
// queries leave of the registers, and the rings of LDS.  Three with small
// heads (64 requests of 200..8000 tokens: 42 us, two 47), two with heads of
// 128 (one request of 131000 tokens: 38 us, three 50, whose shares are smaller
// and begin and end more often; 64 requests 65 and 70).  One instead of two, by
// P NT NB = 8: with pairs of pieces it is slower (131000 fp16 49 us for 41, 64
// requests fp16 115 for 82, 16 x 5 fp32 39.6 for 35.8).  With bf16 queries it
// would be faster, as two spill registers in the loop over blocks (240 to 630
// bytes a lane with heads of 128 and two tiles, up to 800 with heads of 256):
// 64 x 5 queries of four heads 128 us for 133 (Q8_0 135 for 178), 16 x 5 45 for
// 53, heads of 256 64 requests 79 for 97, one of 131000 57 for 79.
template <int KF, int VF, int P, int NB, int NT>
constexpr int stream_waves() {
    constexpr int lds = std::max(2 * Stage<KF, VF, NB>::kBytes, 16 * NT * 68 * 4) * kAWaves + 1024;
    return std::min(P * NT * NB <= 2 ? 3 : P * NT * NB <= 8 ? 2 : 1, kLdsMax / lds);
}

template <int KF, int VF, int P, int NB, int NT>
__global__ __launch_bounds__(kAT, (stream_waves<KF, VF, P, NB, NT>())) void attn_stream_kernel(const AttnArgs a) {
    constexpr int D = 32 * NB, NV = D / 16;             // NV: tiles of 16 places of the head
    constexpr int kRows = 16 * NT;
    typedef Stage<KF, VF, NB> S;
    constexpr int kRing = kAWaves * 2 * S::kBytes, kMeet = kAWaves * kRows * 68 * 4;
    __shared__ __align__(16) uint8_t s_mem[kRing > kMeet ? kRing : kMeet];      // the waves' rings, then their sums
    float (*s_o)[kRows][68] = reinterpret_cast<float (*)[kRows][68]>(s_mem);
    __shared__ float s_m[kAWaves][kRows], s_l[kAWaves][kRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, g = lane >> 4;
    const float inf = __builtin_inff(), nan = __builtin_nanf("");
    // Codes of V are taken as fp16 kBase + c (8 bits: 1024 + 128 + c), with c or c - 8 the code.  Without minimums and with
    // bf16 queries the base goes with the scale, d (kBase + c) - d kBase in one multiply-add; d kBase is rounded, and what
    // that adds to the sums is one product of the weights and the rounding errors, which are exact.  Where d kBase is no
    // number (|V| past 7000), the sums are not either and the careful pass takes the base off first.
    // K's codes go into the product as they are, the integers c 2^-24 that fp16 has below its normal numbers (odd pairs of
    // 4-bit codes 16 times as large).  The matrix cores multiply those to about 2^-20: with pairs of pieces they go in times 2^14.
    constexpr int kUnitLog = P == 2 ? -10 : -24;
    constexpr float kUnit = P == 2 ? 0x1p-10f : 0x1p-24f;
    constexpr bool kOffset = P == 1 && VF != QMV_Q4_1;
    constexpr float kBase = VF == QMV_Q8_0 ? 1152.f : VF == QMV_Q4_0 ? 72.f : 64.f;
    uint32_t mask = 0x00f000f0u, magic = 0x54005400u;
    asm("" : "+s"(mask));        // in registers: one multiply-free instruction takes a code out
    asm("" : "+v"(magic));
    const uint32_t window = a.window > 0 ? a.window : 0x80000000u;

    // ---- the share: blocks [pos, end) of all units' in a row
    const Share share = find_share<NT>(a, blockIdx.x, gridDim.x);
    int64_t pos = blockIdx.x * share.size;
    const int64_t end = min(pos + share.size, share.total);
    int r = share.r;
    int64_t first = share.first;        // of request r's units
    bool tail = true;               // the share's first segment

    while (pos < end) {
        const Req rq = request<NT>(a, r);
        const int64_t mine = (int64_t)rq.cost() * rq.tiles * a.H;
        if (pos >= first + mine) {  // the next request (those without queries have no blocks)
            first += mine;
            ++r;
            continue;
        }
        const int64_t unit = quotient(pos - first, rq.cost());
        const int h = rq.tiles == 1 ? (int)unit : (int)quotient(unit, rq.tiles), tile = (int)(unit - (int64_t)h * rq.tiles);
        const int64_t ubase = first + unit * rq.cost();
        const int b0 = max((int)(pos - ubase) - kABegin, 0);
        const int b1 = (int)(min(end - ubase, (int64_t)rq.cost())) - kABegin;
        pos = min(end, ubase + rq.cost());
        if (b1 <= b0) continue;         // the unit's first block is the next share's
        const bool whole = b0 == 0 && b1 == rq.nblk;

        // ---- queries on their way: B operand, lane n16 = row, places 32 b + 8 g .. + 7
        uint32_t qw[NT][NB][4 * P];
        int qpos[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = tile * kRows + 16 * nt + n16;
            const bool have = row < rq.n * a.G;
            const int i = have ? token_of(a, row) : 0, hq = h * a.G + (have ? row - i * a.G : 0);
            const int64_t base = (rq.q0 + i) * a.qst + hq * a.qsh;
#pragma unroll
            for (int b = 0; b < NB; ++b) load_q8<P>(a, base + 32 * b + 8 * g, qw[nt][b]);
            qpos[nt] = have ? rq.len - rq.n + i : -1;    // -1: sees nothing
        }

        // ---- this wave's blocks
        const int per = (b1 - b0 + kAWaves - 1) / kAWaves;
        const int w0 = __builtin_amdgcn_readfirstlane(min(b0 + wave * per, b1));
        const int w1 = __builtin_amdgcn_readfirstlane(min(w0 + per, b1));
        const int32_t* table = a.table + (int64_t)r * a.max_pages;
        const int full_to = rq.len - rq.n + 1;                       // keys before it are seen by every query
        const int full_from = a.window > 0 ? max(0, rq.len - a.window) : 0;    // from it on, too
        // lane's parts of the loads' addresses
        const uint8_t* kbase = a.k.pages + h * a.k.head_bytes;
        const uint8_t* vbase = a.v.pages + h * a.v.head_bytes;
        uint8_t* ring = s_mem + wave * 2 * S::kBytes;
        const uint32_t ring_at = lds_address(ring);
        const int vb = NB == 4 ? n16 & 3 : NB == 2 ? (n16 >> 1) & 1 : 2 * (n16 & 3);      // the block (or two) of the lane's places of V
        const int kl = (lane / S::kKC) * S::kKRow + (((lane % S::kKC) ^ ((lane / S::kKC) & S::kKSwz)) * 16);
        constexpr int kVPer = 64 / S::kVC, kVParts = kVPer >= 16 ? 1 : 16 / kVPer;      // keys of a load, loads of a tile
        int vl[kVParts];
#pragma unroll
        for (int i = 0; i < kVParts; ++i) {
            const int row = (lane / S::kVC + kVPer * i) & 15, gg = row >> 2;
            vl[i] = (4 * gg + ((row - gg) & 3)) * S::kVRow + (lane % S::kVC) * 16;
        }
        int sl[S::kSL];
        bool sside[S::kSL], st[S::kSL];
#pragma unroll
        for (int i = 0; i < S::kSL; ++i) {
            const int c = lane + 64 * i, pl = c / (4 * NB), b = c / 4 % NB;
            sside[i] = pl >= S::kKP;
            st[i] = (c >> 1) & 1;
            const int plane = (sside[i] ? pl - S::kKP : pl) * NB + b;
            sl[i] = (((sside[i] ? S::kVRow : S::kKRow) + 2 * plane) << a.page_shift) + 16 * (c & 1);
        }
        // Loads of block blk (of the 32 from c0 on) into half `half` of the ring.
        int entries = -1;       // pages of the 64 tiles from block c0 on; -1: absent, -2: out of range
        const auto load = [&](int blk, int c0, int half) {
            uint8_t* to = ring + half * S::kBytes;
            const uint8_t *kp[2], *vp[2], *sp[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t e = max(__builtin_amdgcn_readlane(entries, (2 * (blk - c0) + t) & 63), 0);
                const int off = ((rq.blk0 + blk) * kABlock + 16 * t) & ((1 << a.page_shift) - 1);
                const uint8_t *ke = kbase + e * a.k.page_bytes, *ve = vbase + e * a.v.page_bytes;
                kp[t] = ke + off * S::kKRow;
                vp[t] = ve + off * S::kVRow;
                sp[0][t] = ke + 2 * off;
                sp[1][t] = ve + 2 * off;
            }
#pragma unroll
            for (int i = 0; i < S::kKL; ++i) {
                constexpr int kPer = 64 / S::kKC;      // keys of a load
                const uint8_t* p = S::kKL == 1 ? (lane < 32 ? kp[0] : kp[1]) : kp[i >= S::kKL / 2];
                const int at = S::kKL == 1 ? kl & 511
                                           : (kl ^ (S::kKC == 16 ? (4 * i & 15) * 16 : 0)) +
                                                 (S::kKL > 1 ? i % (S::kKL / 2) : 0) * (kPer * S::kKRow);
                load_chunks(p + at, to + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < S::kVL; ++i) {
                const uint8_t* p = S::kVL == 1 ? (lane < 32 ? vp[0] : vp[1]) : vp[i >= S::kVL / 2];
                load_chunks(p + vl[S::kVL == 1 ? 0 : i % (S::kVL / 2)], to + S::kV + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < S::kSL; ++i) {
                const uint8_t* p = sside[i] ? (st[i] ? sp[1][1] : sp[1][0]) : (st[i] ? sp[0][1] : sp[0][0]);
                if (64 * i + 64 <= S::kSC || lane < S::kSC - 64 * i) load_chunks(p + sl[i], to + S::kS + 1024 * i);
            }
        };
        // The pages of 32 blocks, and the first two blocks on their way.
        const auto begin = [&](int c0) {
            const int at = (rq.blk0 + c0) * kABlock + 16 * lane;
            entries = -1;
            if (at < rq.len && at + 16 > rq.lo && c0 + lane / 2 < w1) {
                entries = table[at >> a.page_shift];
                if (entries < 0 || entries >= a.n_pages) entries = -2;
            }
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
                if (c0 + i < min(c0 + 32, w1)) load(c0 + i, c0, i);
        };
        if (w0 < w1) begin(w0);

        // ---- queries in fp16 pieces
        f16x8 qh[NT][NB], ql[P == 2 ? NT : 1][P == 2 ? NB : 1];
        float qsum[NT][NB], fac[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float amax = 0.f;
            bool fin = true;
            float w[NB][8];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                widen_q8<P>(a, qw[nt][b], w[b]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    amax = fmaxf(amax, __builtin_fabsf(w[b][j]));
                    fin &= __builtin_fabsf(w[b][j]) < inf;
                }
            }
            amax = groups_max(amax);
            const int sh = row_shift(amax);
            fac[nt] = row_factor(a, sh, kUnitLog);
            if (groups_max(fin ? 0.f : 1.f) != 0.f) fac[nt] = __builtin_nanf("");
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = __builtin_ldexpf(w[b][j], sh);
                    const _Float16 hi = (_Float16)x, lo = (_Float16)(x - (float)hi);
                    // odd pairs of 4-bit codes stay where they are in the word, 16 times as large
                    const _Float16 f = KF != QMV_Q8_0 && (j & 2) ? (_Float16)0.0625f : (_Float16)1.f;
                    qh[nt][b][j] = hi * f;
                    s += (float)hi;
                    if constexpr (P == 2) {
                        ql[nt][b][j] = lo * f;
                        s += (float)lo;
                    }
                }
                qsum[nt][b] = groups_sum(s) * kUnit;
            }
        }

        float m[NT], l[NT];
        f32x4 o[NT][NV];
        // All of the wave's blocks; `care`: with values that are not finite by themselves, and scores far from 0.
        const auto pass = [&](auto care) {
            constexpr bool careful = decltype(care)::value, offset = kOffset && !careful;
            f32x4 poison[NT][S::kVB], corr[NT][S::kVB];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt] = kANone;
                l[nt] = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) o[nt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < S::kVB; ++v) poison[nt][v] = corr[nt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            // 32 blocks at a time.  A step reads its stage, has the stage after the next loaded in its place, and computes.
            for (int c0 = w0; c0 < w1; c0 += 32) {
                const int c1 = min(c0 + 32, w1);
                if (careful || c0 > w0) begin(c0);
#pragma unroll 1
                for (int blk = c0; blk < c1; ++blk) {
                    const int half = (blk - c0) & 1;
                    uint32_t vw[8][S::kVW];
                    uint2 vs[2][S::kVB], vmn[2][S::kVB];
                    f32x4 s[NT][2];
                    // this stage has landed; the next may be on its way (loads return in order)
                    if (blk + 1 < c1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kLoads) : "memory");
                    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    const uint32_t from = ring_at + half * S::kBytes;
                    // scores: rows of the result are keys 4 g + r of tile t; the codes' bias comes from the operand added
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t kw[S::kKW];
                        uint2 ks[NB], km[NB];
                        const uint32_t row = from + (16 * t + n16) * S::kKRow;
                        if constexpr (S::kKW == 2 || S::kKW == 4) {
                            lds_words<S::kKW>(row + g * (S::kKRow / 4), kw);
                        } else {
                            // the lane's chunks, each at its place in the row
#pragma unroll
                            for (int c = 0; c < S::kKW / 4; c += 2) {
                                const int q = g * (S::kKC / 4) + c, z = n16 & S::kKSwz;
                                u32x4 x, y;
                                lds_chunks2(row + 16 * (q ^ z), row + 16 * ((q + 1) ^ z), x, y);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    kw[4 * c + k] = x[k];
                                    kw[4 * c + 4 + k] = y[k];
                                }
                            }
                        }
                        const uint32_t sc = from + S::kS + 32 * t + 8 * g;
                        lds_pairs<NB, 64>(sc, ks);
                        if constexpr (KF == QMV_Q4_1) lds_pairs<NB, 64>(sc + 64 * NB, km);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) s[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            f16x8 c;
                            if constexpr (KF == QMV_Q8_0) {
                                const uint32_t x = kw[2 * b] ^ 0x80808080u, y = kw[2 * b + 1] ^ 0x80808080u;
                                c = pack8(as_h2(__builtin_amdgcn_perm(x, x, 0x0c010c00u)), as_h2(__builtin_amdgcn_perm(x, x, 0x0c030c02u)),
                                          as_h2(__builtin_amdgcn_perm(y, y, 0x0c010c00u)), as_h2(__builtin_amdgcn_perm(y, y, 0x0c030c02u)));
                            } else {
                                const uint32_t x = kw[b], y = x >> 8;
                                c = pack8(as_h2(x & 0x000f000fu), as_h2(x & 0x00f000f0u), as_h2(y & 0x000f000fu), as_h2(y & 0x00f000f0u));
                            }
                            if constexpr (P == 2) c *= (_Float16)16384.f;
                            const f16x2 d0 = as_h2(ks[b].x), d1 = as_h2(ks[b].y);
                            constexpr float bias = KF == QMV_Q8_0 ? 128.f : KF == QMV_Q4_0 ? 8.f : 0.f;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const float z0 = -bias * qsum[nt][b];
                                f32x4 z = f32x4{z0, z0, z0, z0};
                                if constexpr (P == 2) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(c, ql[nt][b], z, 0, 0, 0);
                                z = __builtin_amdgcn_mfma_f32_16x16x32_f16(c, qh[nt][b], z, 0, 0, 0);
                                f32x4& y = s[nt][t];
                                y[0] = __builtin_fmaf((float)d0[0], z[0], y[0]);
                                y[1] = __builtin_fmaf((float)d0[1], z[1], y[1]);
                                y[2] = __builtin_fmaf((float)d1[0], z[2], y[2]);
                                y[3] = __builtin_fmaf((float)d1[1], z[3], y[3]);
                                if constexpr (KF == QMV_Q4_1) {
                                    const f16x2 m0 = as_h2(km[b].x), m1 = as_h2(km[b].y);
                                    y[0] = __builtin_fmaf((float)m0[0], qsum[nt][b], y[0]);
                                    y[1] = __builtin_fmaf((float)m0[1], qsum[nt][b], y[1]);
                                    y[2] = __builtin_fmaf((float)m1[0], qsum[nt][b], y[2]);
                                    y[3] = __builtin_fmaf((float)m1[1], qsum[nt][b], y[3]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t vc = from + S::kS + 32 * t + 8 * g + 64 * NB * S::kKP + 64 * vb;
                        lds_pairs<S::kVB, 64>(vc, vs[t]);
                        if constexpr (VF == QMV_Q4_1) lds_pairs<S::kVB, 64>(vc + 64 * NB, vmn[t]);
                    }
                    uint32_t at[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = from + S::kV + (4 * g + ((i + g) & 3)) * S::kVRow + n16 * (S::kVRow / 16);
                    lds_values<S::kVRow / 16, 16 * S::kVRow>(at, vw);
                    if (blk + 2 < c1) load(blk + 2, c0, half);

                    const int key0 = (rq.blk0 + blk) * kABlock;
                    const int e0 = __builtin_amdgcn_readlane(entries, (2 * (blk - c0)) & 63);
                    const int e1 = __builtin_amdgcn_readlane(entries, (2 * (blk - c0) + 1) & 63);
                    const bool plain = key0 + 32 <= full_to && key0 >= full_from && e0 >= 0 && e1 >= 0;
                    if (careful || !plain) {
                        // pages out of range
                        if (e0 == -2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[nt][0] = f32x4{nan, nan, nan, nan};
                        if (e1 == -2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[nt][1] = f32x4{nan, nan, nan, nan};
                        // keys out of a query's sight: 0 <= position - key < window
                        f16x8 sees[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int back = qpos[nt] - key0 - 4 * g;
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const bool seen = (uint32_t)(back - 16 * t - i) < window;
                                    s[nt][t][i] = seen ? s[nt][t][i] : -inf;
                                    sees[nt][4 * t + i] = seen ? (_Float16)1.f : (_Float16)0.f;
                                }
                        }
                        // absent keys, whose bytes are any: scales and minimums of 0
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int n = (t ? e1 : e0) < 0 ? 0 : rq.len - key0 - 16 * t - 4 * g;
                            const uint32_t m0 = n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u, m1 = n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
#pragma unroll
                            for (int k = 0; k < S::kVB; ++k) {
                                vs[t][k].x &= m0;
                                vs[t][k].y &= m1;
                                if constexpr (VF == QMV_Q4_1) {
                                    vmn[t][k].x &= m0;
                                    vmn[t][k].y &= m1;
                                }
                            }
                        }
                        if constexpr (careful) {
                            // values that are not finite: which rows see one, block by block; 0 in their place
#pragma unroll
                            for (int k = 0; k < S::kVB; ++k) {
                                uint32_t sick[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    uint32_t& d = j & 1 ? vs[j / 2][k].y : vs[j / 2][k].x;
                                    uint32_t& mn = j & 1 ? vmn[j / 2][k].y : vmn[j / 2][k].x;
                                    uint32_t odd = not_finite(d);
                                    if constexpr (VF == QMV_Q4_1) {
                                        odd |= not_finite(mn);
                                        mn &= ~odd;
                                    }
                                    d &= ~odd;
                                    sick[j] = odd & 0x3c003c00u;
                                }
                                const f16x8 x = pack8(as_h2(sick[0]), as_h2(sick[1]), as_h2(sick[2]), as_h2(sick[3]));
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    poison[nt][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, sees[nt], poison[nt][k], 0, 0, 0);
                            }
                        }
                    }
                    // softmax: running maximum (kALow under it) and sum, in units of log 2
                    f16x8 ph[NT], pl[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float top = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                                          fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
                        if constexpr (careful) top = fmaxf(lowered(groups_max(top * fac[nt])), m[nt]);
                        else top = fmaxf(groups_max(__builtin_fmaf(top, fac[nt], -kALow)), m[nt]);
                        if (__any(top > m[nt])) {
                            const float f = __builtin_amdgcn_exp2f(m[nt] - top);
                            l[nt] *= f;
#pragma unroll
                            for (int v = 0; v < NV; ++v) o[nt][v] *= f;
                            if constexpr (offset)
#pragma unroll
                                for (int k = 0; k < S::kVB; ++k) corr[nt][k] *= f;
                            m[nt] = top;
                        }
                        float unit = fac[nt];
                        if constexpr (careful) {
                            const bool far = is_far(m[nt]);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) s[nt][t][i] *= far ? unit : 1.f;
                            unit = far ? 1.f : unit;
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][t][i], unit, -m[nt]));
                                const _Float16 hi = (_Float16)p;
                                ph[nt][4 * t + i] = hi;
                                if constexpr (P == 2) {
                                    l[nt] += p;
                                    pl[nt][4 * t + i] = (_Float16)(p - (float)hi);
                                }
                            }
                        if constexpr (P == 1)      // the sum of the weights as they are multiplied
#pragma unroll
                            for (int i = 0; i < 8; i += 2)
                                l[nt] = __builtin_amdgcn_fdot2(f16x2{ph[nt][i], ph[nt][i + 1]}, h2(1.f), l[nt], false);
                    }
                    // values: tile v of the result's places, keys in the order of the weights
                    f16x2 vd[4][S::kVB], ve[4][S::kVB];      // pairs of keys 2 j, 2 j + 1: scales, and minimums or offsets
#pragma unroll
                    for (int k = 0; k < S::kVB; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            vd[j][k] = as_h2(j & 1 ? vs[j / 2][k].y : vs[j / 2][k].x);
                            if constexpr (VF == QMV_Q4_1) ve[j][k] = as_h2(j & 1 ? vmn[j / 2][k].y : vmn[j / 2][k].x);
                            else if constexpr (offset) ve[j][k] = vd[j][k] * h2(-kBase);
                            else ve[j][k] = h2(0.f);
                        }
                        if constexpr (offset) {
                            // what the offsets' rounding adds to the block's values, for one more product
                            const f16x8 x = pack8(__builtin_elementwise_fma(vd[0][k], h2(kBase), ve[0][k]),
                                                  __builtin_elementwise_fma(vd[1][k], h2(kBase), ve[1][k]),
                                                  __builtin_elementwise_fma(vd[2][k], h2(kBase), ve[2][k]),
                                                  __builtin_elementwise_fma(vd[3][k], h2(kBase), ve[3][k]));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                corr[nt][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, ph[nt], corr[nt][k], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const int k = S::kVB == 2 ? v / 8 : 0;
                        f16x2 x[4], rest[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // the code plus kRaw, of the two keys side by side
                            f16x2 c;
                            if constexpr (VF == QMV_Q8_0) {
                                constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
                                c = as_h2((__builtin_amdgcn_perm(vw[2 * j + 1][v / 4], vw[2 * j][v / 4], sel[v % 4]) ^ 0x00800080u) |
                                          0x64006400u);
                            } else {
                                // value 2 e is nibble e of a word's low half, 2 e + 1 of the high one; a lane that has half
                                // an octet (NB 2) has four nibbles
                                const int wd = NB == 8 ? v / 8 : 0, e = NB == 2 ? v : v % 8 >> 1;
                                const uint32_t both = __builtin_amdgcn_perm(vw[2 * j + 1][wd], vw[2 * j][wd],
                                                                            NB != 2 && (v & 1) ? 0x07060302u : 0x05040100u);
                                c = as_h2(and_or(e == 0 ? both << 4 : e == 1 ? both : e == 2 ? both >> 4 : both >> 8, mask, magic));
                            }
                            if constexpr (!offset) {
                                c = c - h2(kBase);
                                if constexpr (P == 2) rest[j] = scaled_rest<VF, careful>(c, vd[j][k], ve[j][k], x[j]);
                                else x[j] = scaled<VF>(c, vd[j][k], ve[j][k]);
                            } else {
                                x[j] = __builtin_elementwise_fma(c, vd[j][k], ve[j][k]);
                            }
                        }
                        const f16x8 vh = pack8(x[0], x[1], x[2], x[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (P == 2) {
                                const f16x8 vl2 = pack8(rest[0], rest[1], rest[2], rest[3]);
                                o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl2, ph[nt], o[nt][v], 0, 0, 0);
                                o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, pl[nt], o[nt][v], 0, 0, 0);
                            }
                            o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, ph[nt], o[nt][v], 0, 0, 0);
                        }
                    }
                }
            }
            if constexpr (offset || careful)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const int k = S::kVB == 2 ? v / 8 : 0;
                        if constexpr (offset) o[nt][v] -= corr[nt][k];
                        if constexpr (careful)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[nt][v][i] = poison[nt][k][i] > 0.f ? nan : o[nt][v][i];
                    }
        };
        pass(std::false_type{});
        bool odd = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            odd |= is_far(m[nt]);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) odd |= !(__builtin_fabsf(o[nt][v][i]) < inf);
        }
        // 0 times a value that is not finite, of a key that a row does not see: again, with such values by themselves.  Scores
        // that were far from 0 before the maximum came near it: their weights, infinite or not, were multiplied by 0 there
        if (__builtin_expect(__any(odd), 0)) pass(std::true_type{});

        // ---- the waves' parts meet
        __syncthreads();        // the last segment's reads of LDS
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = groups_sum(l[nt]);
            if (g == 0) {
                s_m[wave][16 * nt + n16] = m[nt];
                s_l[wave][16 * nt + n16] = l[nt];
            }
        }
        __syncthreads();
        float all_m[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = 16 * nt + n16;
            all_m[nt] = fmaxf(fmaxf(s_m[0][n], s_m[1][n]), fmaxf(s_m[2][n], s_m[3][n]));
            const float f = __builtin_amdgcn_exp2f(m[nt] - all_m[nt]);
#pragma unroll
            for (int v = 0; v < NV; ++v) o[nt][v] *= f;
        }
        // rows of the sums: thread tid / 16 (+ 16), four places tid % 16
        const int64_t slot = 2 * (int64_t)blockIdx.x + (tail ? 0 : 1);
        const int64_t slots = 2 * (int64_t)gridDim.x;
        float* pm = a.part + slots * kRows * D;
        constexpr int kPieces = D / 64;
#pragma unroll
        for (int pc = 0; pc < kPieces; ++pc) {
            if (pc) __syncthreads();
            // result row i of lane group g: place(s) of block and octet by NB (the order of a row's octets)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float* to = s_o[wave][16 * nt + n16];
                if constexpr (NB == 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int v = 0; v < NV; ++v)      // half an octet a lane: four bytes, or every other value
                            to[32 * (i >> 1) + 8 * g + (VF == QMV_Q8_0 ? 4 * (i & 1) + v : 2 * v + (i & 1))] = o[nt][v][i];
                } else if constexpr (NB == 4) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int v = 0; v < NV; v += 4)
                            *reinterpret_cast<f32x4*>(to + 32 * i + 8 * g + v) =
                                f32x4{o[nt][v][2 * pc + i], o[nt][v + 1][2 * pc + i], o[nt][v + 2][2 * pc + i], o[nt][v + 3][2 * pc + i]};
                } else {
#pragma unroll
                    for (int v = 0; v < NV; v += 4)
                        *reinterpret_cast<f32x4*>(to + 32 * (v / 8) + 8 * g + v % 8) =
                            f32x4{o[nt][v][pc], o[nt][v + 1][pc], o[nt][v + 2][pc], o[nt][v + 3][pc]};
                }
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int n = 16 * nt + tid / 16, c = 4 * (tid % 16);
                const int row = tile * kRows + n;
                if (row >= rq.n * a.G) continue;
                f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
                float mm = fmaxf(fmaxf(s_m[0][n], s_m[1][n]), fmaxf(s_m[2][n], s_m[3][n])), ll = 0.f;
#pragma unroll
                for (int w = 0; w < kAWaves; ++w) {
                    x += *reinterpret_cast<const f32x4*>(&s_o[w][n][c]);
                    ll += s_l[w][n] * __builtin_amdgcn_exp2f(s_m[w][n] - mm);
                }
                if (whole) {
                    const int i = token_of(a, row), hq = h * a.G + row - i * a.G;
                    finish(a, hq, mm, ll, x, rq.bad);
                    store_out4(a, ((rq.q0 + i) * a.H * a.G + hq) * D + 64 * pc + c, x);
                } else {
                    *reinterpret_cast<f32x4*>(a.part + (slot * kRows + n) * D + 64 * pc + c) = x;
                    if (pc == 0 && c == 0) {
                        pm[slot * kRows + n] = mm;
                        pm[(slots + slot) * kRows + n] = ll;
                    }
                }
            }
        }
        tail = false;
        lds_barrier();          // the rings take the place of the sums
    }
}

// The parts of the units that no single workgroup had: a workgroup per row.
// A row's parts are read by kAT / (D / 4) threads side by side, which meet in
// LDS in a fixed order.
template <int D, int NT>
__global__ __launch_bounds__(kAT) void attn_join_kernel(const AttnArgs a, int shares, int rows) {
    constexpr int kRows = 16 * NT, kCols = D / 4, kPer = kAT / kCols;
    __shared__ f32x4 s_x[kPer][kCols];
    __shared__ float s_l[kPer];
    const int r = blockIdx.y;
    const Req rq = request<NT>(a, r);
    const int64_t share = a.prefix[a.R + 1], first = a.prefix[r];
    const int64_t slots = 2 * (int64_t)shares;
    const float* pm = a.part + slots * kRows * D;
    const float* pl = pm + slots * kRows;
    const int64_t work = (int64_t)rq.tiles * a.H * rows;
    for (int64_t at = blockIdx.x; at < work; at += gridDim.x) {
        const int64_t unit = quotient(at, rows);
        const int n = (int)(at - unit * rows);
        const int64_t u0 = first + unit * rq.cost(), u1 = u0 + rq.cost();
        const int64_t s0 = quotient(u0 + kABegin, share), s1 = quotient(u1 - 1, share);
        if (s0 == s1) continue;
        const int h = (int)quotient(unit, rq.tiles), tile = (int)(unit - (int64_t)h * rq.tiles);
        const int row = tile * kRows + n;
        if (row >= rq.n * a.G) continue;
        const int c = threadIdx.x % kCols, part = threadIdx.x / kCols;
        // the unit's first part is its workgroup's last unless no other unit is before it in the share
        const auto slot_of = [&](int64_t s) { return (2 * s + (s == s0 && u0 > s * share ? 1 : 0)) * kRows + n; };
        float m = kANone;
        for (int64_t s = s0 + (threadIdx.x & 63); s <= s1; s += 64) m = fmaxf(m, pm[slot_of(s)]);
#pragma unroll
        for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
        // eight parts' loads at a time: one by one 128 parts of a row took 9.1 us, most of it waiting, now 5.9
        constexpr int kLoads = 8;
        for (int64_t s = s0 + part; s <= s1; s += kLoads * kPer) {
            float mm[kLoads], ll[kLoads];
            f32x4 xx[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const bool there = s + k * kPer <= s1;
                const int64_t i = slot_of(there ? s + k * kPer : s);
                mm[k] = there ? pm[i] : -__builtin_inff();
                ll[k] = pl[i];
                xx[k] = *reinterpret_cast<const f32x4*>(a.part + i * D + 4 * c);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                if (k && s + k * kPer > s1) break;
                const float f = __builtin_amdgcn_exp2f(mm[k] - m);
                l += ll[k] * f;
                x += xx[k] * f;
            }
        }
        __syncthreads();
        s_x[part][c] = x;
        if (c == 0) s_l[part] = l;
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int k = 1; k < kPer; ++k) {
                x += s_x[k][c];
                l += s_l[k];
            }
            const int i = token_of(a, row), hq = h * a.G + row - i * a.G;
            finish(a, hq, m, l, x, rq.bad);
            store_out4(a, ((rq.q0 + i) * a.H * a.G + hq) * D + 4 * c, x);
        }
    }
}

template <int KF, int VF, int P, int NB, int NT>
int32_t launch_stream_n(const AttnArgs& a, hipStream_t st) {
    const char* name = "qmv_cache_attention";
    constexpr int shares = 256 * stream_waves<KF, VF, P, NB, NT>();     // all at once on the GPU
    static_assert(shares <= kAShares);
    hipLaunchKernelGGL((attn_stream_kernel<KF, VF, P, NB, NT>), dim3(shares), dim3(kAT), 0, st, a);
    if (const int32_t e = check_launch(name)) return e;
    const int64_t most = std::min<int64_t>(a.max_q * a.G, a.stream_to);
    const int rows = (int)std::min<int64_t>(16 * NT, most);
    const int64_t work = a.H * ((most + 16 * NT - 1) / (16 * NT)) * rows;
    const unsigned x = (unsigned)std::min<int64_t>(work, std::max<int64_t>(1, 65536 / a.R));
    hipLaunchKernelGGL((attn_join_kernel<32 * NB, NT>), dim3(x, a.R), dim3(kAT), 0, st, a, shares, rows);
    return check_launch(name);
}
template <int KF, int VF, int P>
int32_t launch_stream_d(const AttnArgs& a, int D, hipStream_t st) {
    const bool two = stream_tiles(a.max_q * a.G, D) == 2;
    switch (D) {
    case 64: return two ? launch_stream_n<KF, VF, P, 2, 2>(a, st) : launch_stream_n<KF, VF, P, 2, 1>(a, st);
    case 128: return two ? launch_stream_n<KF, VF, P, 4, 2>(a, st) : launch_stream_n<KF, VF, P, 4, 1>(a, st);
    default: return launch_stream_n<KF, VF, P, 8, 1>(a, st);
    }
}
template <int KF, int P>
int32_t launch_stream(const AttnArgs& a, int D, hipStream_t st) {
    switch (a.v.fmt) {
    case QMV_Q8_0: return launch_stream_d<KF, QMV_Q8_0, P>(a, D, st);
    case QMV_Q4_0: return launch_stream_d<KF, QMV_Q4_0, P>(a, D, st);
    default: return launch_stream_d<KF, QMV_Q4_1, P>(a, D, st);
    }
}

}  // namespace
}  // namespace qmv
