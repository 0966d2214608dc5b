// Block-quantized matrix x many tokens on the matrix cores (gfx950): the
// tile kernel of the grouped products and of projections past 8 tokens.
//
// y[t][i] = sum_j DEQ(W)[i][j] x[t][j].  A 32-weight block contributes
// d * sum_e q_e x_e (+ mu * sum_e x_e for formats with a minimum), q_e the
// block's codes as small signed integers: exact in bf16 and in fp16.  So
// v_mfma_f32_32x32x16 with the codes as one operand and the activations as
// the other gives the exact products summed in fp32, and the block's scale
// multiplies the 32 x 32 results in fp32 afterwards.  Nothing is rounded to
// 16 bits:
//  * 16-bit activations are the operand themselves (bf16 or fp16 MFMA);
//  * fp32 activations are split into three bf16 pieces, hi = RN(x), mid =
//    RN(x - hi), lo = RN(x - hi - mid): 24 bits, three MFMAs a block half
//    into one accumulator.
// Formats with a minimum carry codes about the pivot code k next to the zero
// of D c - M, and mu = D k - M: where c != k, |mu| is at most |w|, so no two
// large terms cancel.  Q6_K has a scale per 16 weights, one MFMA's depth.
//
// Operands: the activations are the MFMA's rows (A), the weight rows its
// columns (B), so that lane l holds results of one weight row, l % 32, for 16
// tokens, and scales them all by one register.
//
// Many tokens (2048 through 14336 x 4096, bf16 in and out): Q4_0 336 us (716
// TF/s), Q8_0 367, Q4_1 434, Q4_K 440, Q6_K 551.  Parts of Q4_0's left out in
// turn (395 us with fp32 outputs): MFMAs alone 175, with the scalings and
// reads of x beside them 246, staging x 102, decoding 52, staging weights 28:
// at two waves a SIMD these add up more than they overlap (counters: vector
// instructions 49% of the issue slots, the matrix pipe busy 25%).  Few tokens
// (single ones through 128 experts of 2048 x 8192): weights stream at 5.0
// TB/s in Q8_0, 4.0 Q4_0, 3.6 Q4_1 and Q6_K, 3.2 Q4_K; no pipe is full (with 9
// tokens through 1536 x 2048 Q4_0 the vector pipe 47%, the matrix pipe 12%,
// LDS bank conflicts 22% of the cycles).
#pragma once
#include <type_traits>

#include "qmv_block_decode.h"
#include "qmv_group.h"

namespace qmv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Calls fn(std::integral_constant<int, J>{}) for J = 0..N-1 in order.
template <class Fn, int... Js>
__device__ __forceinline__ void static_for(std::integer_sequence<int, Js...>, Fn&& fn) {
    (fn(std::integral_constant<int, Js>{}), ...);
}

__device__ __forceinline__ uint32_t fbits(float f) { return __builtin_bit_cast(uint32_t, f); }

// --------------------------------------------------------------- operands
// XOp<XT>: the MFMA of an activation type, and pairs of codes in its type.
template <class XT> struct XOp {
    static constexpr int kPieces = 1;
    // two floats that are exact in bf16
    __device__ static uint32_t pair(float a, float b) { return __builtin_amdgcn_perm(fbits(b), fbits(a), 0x07060302u); }
    __device__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
};
template <> struct XOp<float> : XOp<__bf16> {
    static constexpr int kPieces = 3;
};
template <> struct XOp<_Float16> {
    static constexpr int kPieces = 1;
    __device__ static uint32_t pair(float a, float b) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    }
    __device__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
};

// --------------------------------------------------------------- weights
// A wave reads its 32 rows eight blocks at a time: 16-byte pieces of a row
// with neighbouring lanes on neighbouring pieces, kept in registers while the
// eight blocks before them are computed, then copied to the wave's part of
// LDS (its slot).  Loads by block and lane instead (64 lanes on 64 lines) ran
// at 2.4 TB/s for Q4_0 and 1.5 for Q6_K whatever the number of waves: the
// cache looks up about one lane's line a cycle.
//
// Rows start on 2 bytes (34-, 18- and 210-byte units), pieces on words: the
// slot's row r holds the bytes from 0 or 2 (sh) bytes before the row's.  The
// loads go through a buffer that ends with the word that holds the matrix's
// last byte: words past it read 0, and no word without a byte of the matrix
// is read.
//
// Unit<F> is a format's step of two blocks, 2 J and 2 J + 1 of the eight (J
// 0..3), of the lane's row, in three parts, so that a step can be decoded
// bit by bit among the MFMAs of the step before it: read() takes its words
// from the slot; scales() gives the blocks' scales d[b][.] (one, or one per
// 16 weights), mu of block 2 J + lh, and what codes() needs; codes() gives
// the codes of block b that MFMA h takes from lane half lh, elements
// at(h, lh) .. + 7, as signed bytes.
//   kRow    bytes of eight blocks;  kCpr  pieces of a row;  kPitch  bytes of
//   a slot's row, an odd number of 16-byte units.
// weight() is the weight of column c of the row at `row` in memory, in fp32.
template <class F> struct Unit;

__device__ __forceinline__ uint32_t lds4(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint16_t lds2(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
// The words that hold N - 1 words from p, p 0 or 2 (sh) bytes past a word,
// and the i-th of those.
template <int N>
__device__ __forceinline__ void lds_span(const uint8_t* p, uint32_t sh, uint32_t (&w)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = lds4(p - sh + 4 * i);
}
template <int N>
__device__ __forceinline__ uint32_t word_of(const uint32_t (&w)[N], int i, uint32_t sh) {
    return __builtin_amdgcn_alignbyte(w[i + 1], w[i], sh);
}
// Exchanges the upper 32 lanes of a with the lower 32 of b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// v of lane l % 32 (a) and of lane l % 32 + 32 (b), in both.
__device__ __forceinline__ void both_halves(uint32_t v, uint32_t& a, uint32_t& b) {
    a = b = v;
    swap_halves(a, b);
}
__device__ __forceinline__ void both_halves(float v, float& a, float& b) {
    uint32_t x, y;
    both_halves(fbits(v), x, y);
    a = __builtin_bit_cast(float, x);
    b = __builtin_bit_cast(float, y);
}
// c - k per byte, c and k in 0..15: no borrow crosses a byte
__device__ __forceinline__ uint32_t less_pivot(uint32_t c, uint32_t k4) {
    return ((c | 0x80808080u) - k4) ^ 0x80808080u;
}
// the code nearest the zero of D c - M (any code gives the same exact value)
__device__ __forceinline__ float pivot(float D, float M) {
    // fmax/fmin return the number for a NaN operand (D = M = 0): k = 0
    return __builtin_fminf(__builtin_fmaxf(__builtin_rintf(M * __builtin_amdgcn_rcpf(D)), 0.f), 15.f);
}

template <> struct Unit<Q8_0> {
    static constexpr int kSub = 1, kRow = 272, kCpr = 18, kPitch = 304;
    static constexpr bool kSums = false;
    __device__ static float weight(const uint8_t* row, int c) {
        const uint8_t* blk = row + 34 * (c >> 5);
        return half_bits_to_float(ld2(blk)) * (float)(int8_t)blk[2 + (c & 31)];
    }
    __device__ static constexpr int at(int h, int lh) { return 16 * lh + 8 * h; }
    struct Raw {
        uint32_t w[2][5];
        uint16_t d[2];
    };
    template <int J>
    __device__ static void read(const uint8_t* row, uint32_t sh, int lh, Raw& r) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint8_t* blk = row + sh + 34 * (2 * J + b);     // 2 b (mod 4) past sh
            lds_span(blk + 2 + 16 * lh, (sh + 2 * b + 2) & 2, r.w[b]);
            r.d[b] = lds2(blk);
        }
    }
    template <int J>
    __device__ static void scales(const Raw& r, uint32_t, int, float (&d)[2][kSub], float&, uint32_t (&)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) d[b][0] = half_bits_to_float(r.d[b]);
    }
    template <int J>
    __device__ static void codes(const Raw& r, uint32_t sh, int b, int h, const uint32_t (&)[2], uint32_t (&q)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) q[i] = word_of(r.w[b], 2 * h + i, (sh + 2 * b + 2) & 2);
    }
};

template <> struct Unit<Q4_0> {
    static constexpr int kSub = 1, kRow = 144, kCpr = 10, kPitch = 176;
    static constexpr bool kSums = false;
    __device__ static float weight(const uint8_t* row, int c) {
        const uint8_t* blk = row + 18 * (c >> 5);
        return half_bits_to_float(ld2(blk)) * (float)((blk[2 + (c & 15)] >> (c & 16 ? 4 : 0) & 15) - 8);
    }
    __device__ static constexpr int at(int h, int lh) { return 16 * h + 8 * lh; }
    struct Raw {
        uint32_t w[2][3];
        uint16_t d[2];
    };
    template <int J>
    __device__ static void read(const uint8_t* row, uint32_t sh, int lh, Raw& r) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint8_t* blk = row + sh + 18 * (2 * J + b);     // 2 b (mod 4) past sh
            lds_span(blk + 2 + 8 * lh, (sh + 2 * b + 2) & 2, r.w[b]);
            r.d[b] = lds2(blk);
        }
    }
    // codes are 16 (c - 8); d / 16 is exact
    template <int J>
    __device__ static void scales(const Raw& r, uint32_t, int, float (&d)[2][kSub], float&, uint32_t (&)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) d[b][0] = half_bits_to_float(r.d[b]) * 0.0625f;
    }
    template <int J>
    __device__ static void codes(const Raw& r, uint32_t sh, int b, int h, const uint32_t (&)[2], uint32_t (&q)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = word_of(r.w[b], i, (sh + 2 * b + 2) & 2);
            q[i] = ((h ? c : c << 4) ^ 0x80808080u) & 0xf0f0f0f0u;
        }
    }
};

template <> struct Unit<Q4_1> {
    static constexpr int kSub = 1, kRow = 160, kCpr = 10, kPitch = 176;
    static constexpr bool kSums = true;
    __device__ static float weight(const uint8_t* row, int c) {
        const uint8_t* blk = row + 20 * (c >> 5);
        return __builtin_fmaf(half_bits_to_float(ld2(blk)), (float)(blk[4 + (c & 15)] >> (c & 16 ? 4 : 0) & 15),
                              half_bits_to_float(ld2(blk + 2)));
    }
    __device__ static constexpr int at(int h, int lh) { return 16 * h + 8 * lh; }
    struct Raw {
        uint32_t w[2][2], dm;
    };
    template <int J>
    __device__ static void read(const uint8_t* row, uint32_t, int lh, Raw& r) {
        r.dm = lds4(row + 20 * (2 * J + lh));
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) r.w[b][i] = lds4(row + 20 * (2 * J + b) + 4 + 8 * lh + 4 * i);
    }
    template <int J>
    __device__ static void scales(const Raw& r, uint32_t, int, float (&d)[2][kSub], float& mu, uint32_t (&k4)[2]) {
        const float D = half_bits_to_float(r.dm), m = half_bits_to_float(r.dm >> 16);
        const float k = pivot(D, -m);
        mu = __builtin_fmaf(D, k, m);
        both_halves((uint32_t)k * 0x01010101u, k4[0], k4[1]);
        both_halves(D, d[0][0], d[1][0]);
    }
    template <int J>
    __device__ static void codes(const Raw& r, uint32_t, int b, int h, const uint32_t (&k4)[2], uint32_t (&q)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) q[i] = less_pivot((h ? r.w[b][i] >> 4 : r.w[b][i]) & 0x0f0f0f0fu, k4[b]);
    }
};

// Super-block formats: the eight blocks are a super-block.
struct Q4KTile {};
template <> struct Unit<Q4KTile> {
    static constexpr int kSub = 1, kRow = 144, kCpr = 9, kPitch = 144;
    static constexpr bool kSums = true;
    __device__ static float weight(const uint8_t* row, int c) {
        const uint8_t* sb = row + 144 * (c >> 8);
        const int b = c >> 5 & 7, k = b & 3;
        const uint32_t f1 = sb[4 + k], f2 = sb[8 + k], f3 = sb[12 + k];
        const uint32_t sc = b < 4 ? f1 & 63u : (f3 & 15u) | (f1 >> 2 & 48u);
        const uint32_t mn = b < 4 ? f2 & 63u : (f3 >> 4) | (f2 >> 2 & 48u);
        const uint32_t q = sb[16 + 32 * (b >> 1) + (c & 31)] >> (b & 1 ? 4 : 0) & 15;
        return __builtin_fmaf(half_bits_to_float(ld2(sb)) * (float)sc, (float)q,
                              -(half_bits_to_float(ld2(sb + 2)) * (float)mn));
    }
    __device__ static constexpr int at(int h, int lh) { return 16 * lh + 8 * h; }
    struct Raw {
        u32x4 head, c;
    };
    template <int J>
    __device__ static void read(const uint8_t* row, uint32_t, int lh, Raw& r) {
        r.head = *reinterpret_cast<const u32x4*>(row);
        r.c = *reinterpret_cast<const u32x4*>(row + 16 + 32 * J + 16 * lh);
    }
    template <int J>
    __device__ static void scales(const Raw& r, uint32_t, int lh, float (&d)[2][kSub], float& mu, uint32_t (&k4)[2]) {
        const int t = 8 * ((2 * J & 3) + lh);                 // block 2 J + lh: byte J % 4 of the fields
        const uint32_t h1 = r.head.y >> t, h2 = r.head.z >> t, h3 = r.head.w >> t;
        const uint32_t sc = J < 2 ? (h1 & 63u) : ((h3 & 15u) | ((h1 >> 2) & 48u));
        const uint32_t mn = J < 2 ? (h2 & 63u) : (((h3 >> 4) & 15u) | ((h2 >> 2) & 48u));
        const float D = half_bits_to_float(r.head.x) * (float)sc;          // exact
        const float M = half_bits_to_float(r.head.x >> 16) * (float)mn;    // exact
        const float k = pivot(D, M);
        mu = __builtin_fmaf(D, k, -M);
        both_halves((uint32_t)k * 0x01010101u, k4[0], k4[1]);
        both_halves(D, d[0][0], d[1][0]);
    }
    template <int J>
    __device__ static void codes(const Raw& r, uint32_t, int b, int h, const uint32_t (&k4)[2], uint32_t (&q)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) q[i] = less_pivot((b ? r.c[2 * h + i] >> 4 : r.c[2 * h + i]) & 0x0f0f0f0fu, k4[b]);
    }
};

struct Q6KTile {};
template <> struct Unit<Q6KTile> {
    static constexpr int kSub = 2, kRow = 210, kCpr = 14, kPitch = 240;
    static constexpr bool kSums = false;
    __device__ static float weight(const uint8_t* row, int c) {
        const uint8_t* sb = row + 210 * (c >> 8);
        const int h = c >> 7 & 1, q = c >> 5 & 3, l = c & 31;       // half of the super-block, its quarter
        const uint32_t lo = sb[64 * h + 32 * (q & 1) + l] >> (q & 2 ? 4 : 0) & 15;
        const uint32_t hi = sb[128 + 32 * h + l] >> (2 * q) & 3;
        return half_bits_to_float(ld2(sb + 208)) * (float)(int8_t)sb[192 + (c >> 4 & 15)] * (float)((int)(lo | hi << 4) - 32);
    }
    __device__ static constexpr int at(int h, int lh) { return 16 * h + 8 * lh; }     // an MFMA is one scale's 16 weights
    struct Raw {
        uint32_t lo[2][2][3], hi[2][3], sc[2];     // [b][h], [h]
        uint16_t d;
    };
    template <int J>
    __device__ static void read(const uint8_t* row, uint32_t sh, int lh, Raw& r) {
        const uint8_t* sb = row + sh;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lds_span(sb + 128 + 32 * (J >> 1) + 16 * h + 8 * lh, sh, r.hi[h]);
#pragma unroll
            for (int b = 0; b < 2; ++b) lds_span(sb + 64 * (J >> 1) + 32 * b + 16 * h + 8 * lh, sh, r.lo[b][h]);
        }
        lds_span(sb + 192 + 4 * J, sh, r.sc);
        r.d = lds2(sb + 208);
    }
    // codes are 4 (c - 32); d sc / 4 is exact
    template <int J>
    __device__ static void scales(const Raw& r, uint32_t sh, int, float (&d)[2][kSub], float&, uint32_t (&)[2]) {
        const uint32_t sc = word_of(r.sc, 0, sh);
        const float d4 = half_bits_to_float(r.d) * 0.25f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) d[b][h] = d4 * (float)(int8_t)(sc >> (8 * (2 * b + h)));
    }
    template <int J>
    __device__ static void codes(const Raw& r, uint32_t sh, int b, int h, const uint32_t (&)[2], uint32_t (&q)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = word_of(r.lo[b][h], i, sh);
            const uint32_t hi = (word_of(r.hi[h], i, sh) ^ 0xaaaaaaaau) << (6 - 2 * (2 * (J & 1) + b));
            q[i] = ((J & 1 ? lo >> 2 : lo << 2) & 0x3c3c3c3cu) | (hi & 0xc0c0c0c0u);
        }
    }
};

// --------------------------------------------------------------- activations
// Eight activations of one token: loads (16-byte where `vec`), and their
// pieces as MFMA operands.
template <class XT> struct X8 {
    u32x4 v;
    __device__ void load(const XT* p, bool vec) {
        if (vec) {
            v = *reinterpret_cast<const u32x4*>(p);
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
        }
    }
    __device__ void zero() { v = u32x4{0, 0, 0, 0}; }
    __device__ void pieces(u32x4 (&p)[1]) const { p[0] = v; }
    __device__ float sum() const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<XT, __bf16>::value) {
                s += __builtin_bit_cast(float, v[i] << 16);
                s += __builtin_bit_cast(float, v[i] & 0xffff0000u);
            } else {
                s += half_bits_to_float(v[i]);
                s += half_bits_to_float(v[i] >> 16);
            }
        }
        return s;
    }
};
template <> struct X8<float> {
    float v[8];
    __device__ void load(const float* p, bool vec) {
        if (vec) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i];
        }
    }
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ void pieces(u32x4 (&p)[3]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
                p[k][i] = w;
                a -= __builtin_bit_cast(float, w << 16);           // exact
                b -= __builtin_bit_cast(float, w & 0xffff0000u);
            }
        }
    }
    __device__ float sum() const {
        return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
};

// mu (SIDE 0) or a block sum of x (SIDE 1) as eight bf16 of an MFMA operand:
// three pieces each, h, m and l, in six places whose products add up to
// mu * sum but for terms of 2^-24 of it: hh, mh, hm, mm, lh, hl.
template <int SIDE>
__device__ __forceinline__ u32x4 min_operand(float v) {
    const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, 0.f}, bf16x2));
    float r = v - __builtin_bit_cast(float, h << 16);
    const uint32_t m = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{r, 0.f}, bf16x2));
    r -= __builtin_bit_cast(float, m << 16);
    const uint32_t l = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{r, 0.f}, bf16x2));
    return SIDE == 0 ? u32x4{h | (m << 16), h | (m << 16), l | (h << 16), 0}
                     : u32x4{h | (h << 16), m | (m << 16), h | (l << 16), 0};
}

// --------------------------------------------------------------- the kernel
struct TileDev {
    const uint8_t* W;
    int64_t estride;
    int rows, nb, row_tiles, row_unit;
    const int32_t* plan;
    int n_items, n_groups, top_k, plan_tile;
    const void* x;
    int64_t xs_tok, xs_slot;
    void* y;
    int y_type;
    int64_t ldy;
    int swiglu, vec, yvec;
    int tiles_at, order_at;
    LoraTile lora;
};

__device__ __forceinline__ void store_y(void* y, int y_type, int64_t at, float v) {
    if (y_type == QMV_X_F32) {
        static_cast<float*>(y)[at] = v;
    } else if (y_type == QMV_X_F16) {
        static_cast<_Float16*>(y)[at] = (_Float16)v;
    } else {
        static_cast<__bf16*>(y)[at] = (__bf16)v;
    }
}

// Up to four neighbouring outputs (`left` of them exist), in one store where
// every output row is on four elements.
__device__ __forceinline__ void store_y4(void* y, int y_type, int64_t at, f32x4 v, int left, bool vec) {
    if (!vec || left < 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left) store_y(y, y_type, at + k, v[k]);
        return;
    }
    if (y_type == QMV_X_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(y) + at) = v;
        return;
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        w[k] = y_type == QMV_X_F16
                   ? __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, f16x2))
                   : __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, bf16x2));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = uint2{w[0], w[1]};
}

// The kernel's arguments and the lane's number, read at this place.
__device__ __forceinline__ const TileDev& again_args() {
    auto p = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    return *reinterpret_cast<const TileDev*>(p);
}
__device__ __forceinline__ int again_lane() {
    int all = -1;
    asm volatile("" : "+s"(all));
    return (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}

__device__ __forceinline__ bool finite(f32x4 v) {
    const float inf = __builtin_inff();
    return __builtin_fabsf(v[0]) < inf && __builtin_fabsf(v[1]) < inf && __builtin_fabsf(v[2]) < inf &&
           __builtin_fabsf(v[3]) < inf;
}

// An element of B.
__device__ __forceinline__ float lora_b(const LoraTile& l, int64_t at) {
    return l.b_type == QMV_X_F32   ? static_cast<const float*>(l.B)[at]
           : l.b_type == QMV_X_F16 ? (float)static_cast<const _Float16*>(l.B)[at]
                                   : (float)static_cast<const __bf16*>(l.B)[at];
}

constexpr int kLoraRanks = 64;                       // ranks staged at a time
constexpr int kLoraPitch = 2 * kLoraRanks + 16;      // bytes of a token's piece, an odd number of 16-byte units

// The adapters' part of a tile, added to acc: token j of the tile (item
// first + j) gains B_a v_j for a = s_adapter[j].  For each adapter among the
// tile's tokens, its 32 rows of B are multiplied with the v of every 32
// tokens that hold one of its own, and the sums taken over for those tokens
// alone.  v and B are split into three bf16 pieces each (bf16 B has one); the
// products left out are 2^-24 of the sum.  v is staged in `lds` by the whole
// workgroup; of the KG waves that share the rows, wave wk takes every KG-th
// adapter (their sums meet in the epilogue).  An adapter's rows are loaded
// while those of the one before are multiplied: 40 requests of 101 tokens
// would else wait for 25 loads a tile, one after the other.
template <int TN, int KG, int THREADS>
__device__ __forceinline__ void add_adapters(const LoraTile& l, const int* s_adapter, int first, int count, int n_items,
                                             int rows, int row, int wk, uint8_t* lds, f32x16 (&acc)[TN / 32]) {
    constexpr int kSteps = kLoraRanks / 16;
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    for (int c0 = 0; c0 < l.rank; c0 += kLoraRanks) {
        const int ranks = min(kLoraRanks, l.rank - c0);
        const int steps = (ranks + 15) >> 4;
        __syncthreads();
        // fours of ranks, zeros past the last up to whole steps; all loads first
        constexpr int kQuads = TN * 4 * kSteps / THREADS;
        f32x4 x[kQuads];
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const int i = tid + q * THREADS, j = i / (4 * kSteps), r = 4 * (i % (4 * kSteps));
            x[q] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (j < count && r < ranks) {
                const float* v = l.v + (int64_t)(first + j) * l.rank + c0 + r;
                for (int p = 0; p < l.parts; ++p, v += (int64_t)n_items * l.rank) {
                    if (l.rank % 4 == 0) {
                        x[q] += *reinterpret_cast<const f32x4*>(v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (r + k < ranks) x[q][k] += v[k];
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const int i = tid + q * THREADS, j = i / (4 * kSteps), r = 4 * (i % (4 * kSteps));
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                uint32_t w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[q][2 * e], x[q][2 * e + 1]}, bf16x2));
                    x[q][2 * e] -= __builtin_bit_cast(float, w[e] << 16);
                    x[q][2 * e + 1] -= __builtin_bit_cast(float, w[e] & 0xffff0000u);
                }
                *reinterpret_cast<uint2*>(lds + (k * TN + j) * kLoraPitch + 2 * r) = uint2{w[0], w[1]};
            }
        }
        __syncthreads();
        uint32_t todo[TN / 32];
        int id[TN / 32];
#pragma unroll
        for (int t = 0; t < TN / 32; ++t) {
            id[t] = s_adapter[32 * t + lr];
            todo[t] = (uint32_t)__ballot(32 * t + lr < count && (unsigned)id[t] < (unsigned)l.n_adapters);
        }
        // the next adapter of this wave's turn (-1: none), its tokens
        int turn = 0;
        auto next_adapter = [&](uint32_t (&own)[TN / 32]) __attribute__((always_inline)) {
            while (true) {
                int ad = -1;
#pragma unroll
                for (int t = 0; t < TN / 32; ++t)
                    if (ad < 0 && todo[t]) ad = __builtin_amdgcn_readlane(id[t], __builtin_ctz(todo[t]));
#pragma unroll
                for (int t = 0; t < TN / 32; ++t) {
                    own[t] = (uint32_t)__ballot(id[t] == ad) & todo[t];
                    todo[t] &= ~own[t];
                }
                if (ad < 0 || turn++ % KG == wk) return ad;
            }
        };
        auto load_b = [&](int ad, u32x4 (&w)[kSteps]) __attribute__((always_inline)) {
            if (!l.b16 || ad < 0) return;
            const uint16_t* b = static_cast<const uint16_t*>(l.B) + ((int64_t)ad * rows + row) * l.rank + c0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int r0 = 16 * s + 8 * lh;
                w[s] = u32x4{0, 0, 0, 0};
                if (r0 < ranks) w[s] = *reinterpret_cast<const u32x4*>(b + r0);
            }
        };
        uint32_t own[TN / 32], own2[TN / 32];
        u32x4 w[kSteps], w2[kSteps];
        int ad = next_adapter(own);
        load_b(ad, w);
        while (ad >= 0) {
            const int ad2 = next_adapter(own2);
            load_b(ad2, w2);
            const int64_t brow = ((int64_t)ad * rows + row) * l.rank + c0;
            u32x4 bp[kSteps][3];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (s >= steps) continue;
                X8<float> b;
                if (l.b16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool half = l.b_type == QMV_X_F16;
                        b.v[2 * i] = half ? half_bits_to_float(w[s][i]) : __builtin_bit_cast(float, w[s][i] << 16);
                        b.v[2 * i + 1] = half ? half_bits_to_float(w[s][i] >> 16)
                                              : __builtin_bit_cast(float, w[s][i] & 0xffff0000u);
                    }
                } else {
                    const int r0 = 16 * s + 8 * lh;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float f = lora_b(l, brow + min(r0 + i, ranks - 1));
                        b.v[i] = r0 + i < ranks ? f : 0.f;
                    }
                }
                b.pieces(bp[s]);
            }
#pragma unroll
            for (int t = 0; t < TN / 32; ++t) {
                if (!own[t]) continue;
                f32x16 sum;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] = 0.f;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    if (s >= steps) continue;
#pragma unroll
                    for (int k = 2; k >= 0; --k) {
                        const u32x4 vp = *reinterpret_cast<const u32x4*>(lds + (k * TN + 32 * t + lr) * kLoraPitch +
                                                                         32 * s + 16 * lh);
                        sum = XOp<__bf16>::mfma(vp, bp[s][0], sum);
                        if (l.b_type == QMV_X_BF16) continue;
                        if (k < 2) sum = XOp<__bf16>::mfma(vp, bp[s][1], sum);
                        if (k < 1) sum = XOp<__bf16>::mfma(vp, bp[s][2], sum);
                    }
                }
                const uint32_t mine = own[t] >> (4 * lh);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (mine >> (8 * (i >> 2) + (i & 3)) & 1) acc[t][i] += sum[i];
            }
            ad = ad2;
#pragma unroll
            for (int t = 0; t < TN / 32; ++t) own[t] = own2[t];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) w[s] = w2[s];
        }
    }
}

constexpr int kXcds = 8;          // workgroups go to the XCDs in turn
constexpr int kTokGroup = 8;      // token tiles that an XCD takes together
constexpr int kRowGroup = 32;     // compute units of an XCD: most row tiles of a unit
// A wave takes 32 weight rows by TN tokens.  Its step is two blocks of each
// row, decoded by the lanes that multiply them, so no wave waits for
// another's weights.  KG waves of a workgroup share 32 rows and take their
// eight-block pieces of the row (four steps) in turn; their sums are added in
// a fixed order at the end: where there are few rows, that keeps enough loads
// in flight (KG 8 in workgroups of eight waves).  Activations are staged in
// LDS in chunks of CHS steps for each of the KG.
template <class F, class XT, int TN, int KG>
struct TileShape {
    static constexpr int kP = XOp<XT>::kPieces;
    static constexpr int kWaves = KG > 4 ? KG : 4;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kTM = 32 * kWaves / KG;
    static constexpr int kTS = TN / 32;
    static constexpr int kCHS = TN > 32 || kP > 1 || KG > 1 ? 1 : 2;
    // Loads return in order, so a wait for activations that were asked for
    // after a round's weights is a wait for those weights too.  With four
    // chunks (a round) of activations on their way the weights have a round's
    // time: 9 tokens through 4096 x 14336, KG 4: Q8_0 63 us against 97 with
    // one chunk, Q4_K 72 against 94 with two.  That takes the third wave's
    // registers, which KG 4 and 8 have no use for; at KG 2 it pays for Q8_0
    // (101 tokens through 14336 x 4096 76 us against 96), not for Q4_K (78
    // against 76) or Q6_K (95 against 89).
    static constexpr bool kDeep = kP == 1 && (KG > 2 || (KG == 2 && Unit<F>::kCpr > 14));
    // waves of a SIMD that the registers are cut for; few tokens leave the
    // decoding as the bound, and it takes more waves to keep that going.
    // fp32 pieces with KG 4 fill the LDS with one workgroup
    static constexpr int kOcc = kP > 1 && KG > 2 ? 1 : TN > 32 || kP > 1 || kDeep ? 2 : 3;
    // whether a step is decoded during the one before it; for few tokens
    // Q6_K's words and a second set of operands would take the third wave
    // (64 tokens through 128 experts 180 us against 200)
    static constexpr bool kAhead = TN > 32 || Unit<F>::kSub == 1;
    static constexpr int kCH = kCHS * KG;
    // chunks of activations on their way besides the one being staged
    static constexpr int kXAhead = kDeep                                                 ? 4
                                   : kP > 1 && KG > 2                                    ? 2
                                   : TN < 128 && kP == 1 && Unit<F>::kCpr <= 10          ? 2
                                                                                         : 1;     // as registers allow
    static constexpr int kXL = TN * 8 * kCH / kThreads;         // 8-column pieces of x per thread and chunk
    static constexpr int kPitch = 128 * kCH + 16;                   // bytes of a staged token: an odd number of 16-byte units, so 8 tokens hit distinct banks
    static constexpr int kX = kP * TN * kPitch;
    static constexpr int kM = Unit<F>::kSums ? 2 * kCH * TN * 16 : 0;
    static constexpr int kBuf = kX + kM;
    static constexpr int kSlot = 32 * Unit<F>::kPitch;              // of a wave
    static constexpr int kOutPitch = kTM + 4;                       // floats
    static constexpr int kOut = KG * TN * kOutPitch * 4;
    static constexpr int kMain = 2 * kBuf + kWaves * kSlot;
    static constexpr int kLora = 3 * TN * kLoraPitch;
    static constexpr int kLds = kMain > kOut ? kMain : kOut;
    // workgroups that a compute unit holds: by registers, and by LDS with what
    // the kernel has of its own (under 1 KB at 32 tokens)
    static constexpr int kWgs = std::min(4 * kOcc / kWaves, kLdsMax / (kLds + 1024));
    static_assert(kXL >= 1 && kCHS >= 1, "every thread stages, every wave computes");
};

// LORA: the tokens carry adapters (and there is no plan).
template <class F, class XT, int TN, int KG, bool LORA>
__global__ __launch_bounds__((TileShape<F, XT, TN, KG>::kThreads), (TileShape<F, XT, TN, KG>::kOcc)) void tile_kernel(
    const TileDev a) {
    using S = TileShape<F, XT, TN, KG>;
    using U = Unit<F>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int s_item[TN], s_adapter[LORA ? TN : 1], s_group;
    __shared__ int64_t s_x[TN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int split = a.plan_tile / TN;      // workgroups along a plan's tile (1 without a plan)
    int tok_tiles;
    if (a.plan) {
        // a plan of other items or groups than the call's is not followed
        if (a.plan[0] != kPlanMagic || a.plan[1] != a.n_items || a.plan[2] != a.n_groups || a.plan[3] != a.plan_tile)
            return;
        tok_tiles = a.plan[4] * split;
    } else {
        tok_tiles = (a.n_items + TN - 1) / TN;
    }
    const int xcd = blockIdx.x % kXcds, turn = blockIdx.x / kXcds;
    int rt, tt;
    if (split == 1) {
        // Tiles in runs, one run to an XCD, and within it kTokGroup token
        // tiles side by side down the rows: the tiles an XCD works on at one
        // time share their weights and activations in its L2.
        const int total = tok_tiles * a.row_tiles;
        if ((int)blockIdx.x >= total) return;
        const int id = xcd * (total / kXcds) + min(xcd, total % kXcds) + turn;
        const int t0 = id / (kTokGroup * a.row_tiles) * kTokGroup;
        const int tw = min(kTokGroup, tok_tiles - t0);
        const int in = id - t0 * a.row_tiles;
        rt = in / tw;
        tt = t0 + in % tw;
    } else {
        // A plan's tile that is split has parts past its items, which are
        // empty.  Units of all parts of a tile by row_unit row tiles go to
        // the XCDs in turn, so that these are as busy as each other, and
        // within a unit a part's rows follow each other (side by side, the
        // busy workgroups all came to every fourth compute unit: 66 us
        // against 21).
        const int size = split * a.row_unit, units = (a.row_tiles + a.row_unit - 1) / a.row_unit;
        const int unit = turn / size * kXcds + xcd, at = turn % size;
        rt = unit % units * a.row_unit + at % a.row_unit;
        tt = unit / units * split + at / a.row_unit;
        if (tt >= tok_tiles || rt >= a.row_tiles) return;
    }

    const int out_rows = a.swiglu ? S::kTM / 2 : S::kTM;
    const int row0 = rt * out_rows;
    int group = 0, start = tt * TN, count = min(TN, a.n_items - start);
    if (a.plan) {
        const int* t = a.plan + a.tiles_at + 4 * (tt / split);
        const int skip = tt % split * TN;
        group = t[0];
        start = t[1] + skip;
        count = min(TN, t[2] - skip);
        if (count <= 0) return;
    }
    const int lr = lane & 31, lh = lane >> 5;
    const int wk = wave % KG, wr = wave / KG * 32;       // the wave's share of the row, and its rows
    auto matrix_row = [&](int r) __attribute__((always_inline)) {      // row r of the tile
        return a.swiglu ? (r < out_rows ? 0 : a.rows) + min(row0 + (r & (out_rows - 1)), a.rows - 1)
                        : min(row0 + r, a.rows - 1);
    };
    // Weights: eight blocks (four steps) of the row at a time.
    const int sups = (a.nb + 7) >> 3;                    // pieces of eight blocks of a row
    const int rounds = (sups + KG - 1) / KG;
    auto sup_of = [&](int s) __attribute__((always_inline)) { return min(KG * s + wk, sups - 1); };
    const uint32_t pitch = (uint32_t)(a.nb / 8 * U::kRow + a.nb % 8 * (U::kRow / 8));
    const int first = matrix_row(wr);                    // the wave's rows are at and after it
    const uint8_t* W = a.W + min(group, a.n_groups - 1) * a.estride;
    const uintptr_t wbase = reinterpret_cast<uintptr_t>(W + (int64_t)first * pitch);
    const uintptr_t wend = reinterpret_cast<uintptr_t>(W + (int64_t)(a.swiglu ? 2 * a.rows : a.rows) * pitch);
    const int64_t wlen = (int64_t)(((wend + 3) & ~(uintptr_t)3) - (wbase & ~(uintptr_t)3));
    const __amdgpu_buffer_rsrc_t wbuf = raw_buffer(reinterpret_cast<const void*>(wbase & ~(uintptr_t)3),
                                                   (uint32_t)min(wlen, (int64_t)0xfffffffc));
    const uint32_t wsh = (uint32_t)(wbase & 2);
    constexpr int kLoads = (32 * U::kCpr + 63) / 64;
    // the lane's pieces: row and byte of the row, where in the matrix, where in the slot
    uint32_t woff[kLoads];
    int wput[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const int p = min(64 * k + lane, 32 * U::kCpr - 1), r = p / U::kCpr, byte = 16 * (p % U::kCpr);
        // whole words of 16 past the row's own start: & ~3 leaves the piece's
        woff[k] = wsh + (uint32_t)(matrix_row(wr + r) - first) * pitch + byte;
        wput[k] = r * U::kPitch + byte;
    }
    const uint32_t wown = wsh + (uint32_t)(matrix_row(wr + lr) - first) * pitch;
    u32x4 wreg[kLoads];
    auto load_w = [&](int s) __attribute__((always_inline)) {
        const int at = sup_of(s) * U::kRow;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b128(wbuf, (int)((woff[k] + at) & ~3u), 0, 0);
            wreg[k] = u32x4{v[0], v[1], v[2], v[3]};
        }
    };
    uint8_t* slot = lds + 2 * S::kBuf + wave * S::kSlot;
    const uint8_t* slot_row = slot + lr * U::kPitch;
    auto put_w = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) *reinterpret_cast<u32x4*>(slot + wput[k]) = wreg[k];
    };
    load_w(0);

    if (tid == 0) s_group = group;
    if (tid < TN) {
        const int at = start + min(tid, count - 1);
        const int item = a.plan ? a.plan[a.order_at + at] : at;
        const int tok = a.top_k == 1 ? item : item / a.top_k;
        s_item[tid] = item;
        s_x[tid] = tok * a.xs_tok + (item - tok * a.top_k) * a.xs_slot;
        if constexpr (LORA) s_adapter[tid] = a.lora.ids[at];
    }
    __syncthreads();
    if (a.plan && group >= a.n_groups) {   // ids that are no group
        for (int i = tid; i < count * out_rows; i += S::kThreads) {
            const int r = row0 + i % out_rows;
            if (r < a.rows)
                store_y(a.y, a.y_type, (int64_t)s_item[i / out_rows] * a.ldy + r, __builtin_nanf(""));
        }
        return;
    }

    // This thread's activations: eight columns (of step xs, share xk) of kXL
    // tokens.  Chunk c is steps kCHS (c % (4 / kCHS)).. of round c / (4 / kCHS).
    const int xc = tid % (8 * S::kCH), xt = tid / (8 * S::kCH);
    const int xk = xc / (8 * S::kCHS), xw = xc % (8 * S::kCHS);
    constexpr int kXStep = S::kThreads / (8 * S::kCH);
    constexpr int kParts = 4 / S::kCHS;
    const XT* xp[S::kXL];
#pragma unroll
    for (int i = 0; i < S::kXL; ++i) {
        xp[i] = static_cast<const XT*>(a.x) + s_x[xt + kXStep * i];
    }
    const bool vec = a.vec != 0;
    struct XRegs {
        X8<XT> x[S::kXL];
    };
    auto column = [&](int c) __attribute__((always_inline)) {
        return 256 * (KG * (c / kParts) + xk) + 64 * S::kCHS * (c % kParts) + 8 * xw;
    };
    // Past the row the last eight columns, put as zeros.
    auto load_x = [&](int c, XRegs& g) __attribute__((always_inline)) {
        const int at = min(column(c), 32 * a.nb - 8);
#pragma unroll
        for (int i = 0; i < S::kXL; ++i)
            if (xt + kXStep * i < count) g.x[i].load(xp[i] + at, vec);
    };
    auto put_x = [&](int c, XRegs& g) __attribute__((always_inline)) {
        uint8_t* buf = lds + (c & 1) * S::kBuf;
        // only the row's last round can hold columns past it
        if (256 * KG * (c / kParts + 1) > 32 * a.nb) {
            asm volatile("");
            if (column(c) >= 32 * a.nb) {
#pragma unroll
                for (int i = 0; i < S::kXL; ++i) g.x[i].zero();
            }
        }
#pragma unroll
        for (int i = 0; i < S::kXL; ++i) {
            u32x4 p[S::kP];
            g.x[i].pieces(p);
#pragma unroll
            for (int k = 0; k < S::kP; ++k)
                *reinterpret_cast<u32x4*>(buf + (k * TN + xt + kXStep * i) * S::kPitch + 16 * xc) = p[k];
        }
        if constexpr (U::kSums) {
            // a block's sum is over four neighbouring lanes (eight columns
            // each) and then in all four; the k-th of them writes the k-th
            // of up to four tokens' sums
#pragma unroll
            for (int i0 = 0; i0 < S::kXL; i0 += 4) {
                float own = 0.f;
#pragma unroll
                for (int k = 0; k < 4 && i0 + k < S::kXL; ++k) {
                    float t = g.x[i0 + k].sum();
                    t += dpp_mov<0xB1>(t);
                    t += dpp_mov<0x4E>(t);
                    own = (xc & 3) == k ? t : own;
                }
                if ((xc & 3) + i0 < S::kXL)
                    *reinterpret_cast<u32x4*>(buf + S::kX + ((xc >> 2) * TN + xt + kXStep * (i0 + (xc & 3))) * 16) =
                        min_operand<1>(own);
            }
        }
    };

    f32x16 acc[S::kTS];
#pragma unroll
    for (int t = 0; t < S::kTS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;

    // A step's operands: codes by block and MFMA, scales, mu.
    struct Ops {
        u32x4 op[2][2];
        float d[2][U::kSub], mu;
    };
    typename U::Raw raw;
    Ops ops[2];
    uint32_t k4[2];
    auto row_sh = [&](int s) __attribute__((always_inline)) { return (wown + sup_of(s) * U::kRow) & 2; };
    auto read_raw = [&](auto jc, int s) __attribute__((always_inline)) {
        U::template read<decltype(jc)::value>(slot_row, row_sh(s), lh, raw);
    };
    auto decode_scales = [&](auto jc, int s, Ops& o) __attribute__((always_inline)) {
        constexpr int J = decltype(jc)::value;
        o.mu = 0.f;
        U::template scales<J>(raw, row_sh(s), lh, o.d, o.mu, k4);
        // past the row the scales are 0 (and so are the activations); the
        // asm keeps this a branch, which only a row's last round takes
        if (8 * (KG * s + wk) + 8 > a.nb) {
            asm volatile("");
            const int blk = 8 * (KG * s + wk) + 2 * J;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (blk + b >= a.nb) {
#pragma unroll
                    for (int h = 0; h < U::kSub; ++h) o.d[b][h] = 0.f;
                }
            if (blk + lh >= a.nb) o.mu = 0.f;
        }
    };
    auto decode_codes = [&](auto jc, int s, auto pc, Ops& o) __attribute__((always_inline)) {
        constexpr int b = decltype(pc)::value >> 1, h = decltype(pc)::value & 1;
        uint32_t q[2];
        U::template codes<decltype(jc)::value>(raw, row_sh(s), b, h, k4, q);
        o.op[b][h] = u32x4{XOp<XT>::pair(sbyte(q[0], 0), sbyte(q[0], 1)), XOp<XT>::pair(sbyte(q[0], 2), sbyte(q[0], 3)),
                           XOp<XT>::pair(sbyte(q[1], 0), sbyte(q[1], 1)), XOp<XT>::pair(sbyte(q[1], 2), sbyte(q[1], 3))};
        asm volatile("" : "+v"(o.op[b][h]));      // here, not where the next step uses it
    };

    // Step J of round s, the sc0-th of those staged in buf.  For each block
    // and 32 tokens (a piece) its MFMAs, between the scalings of the piece
    // before it (16 fused multiply-adds a lane, about as long as the two
    // MFMAs) and the decoding of the next step (round sn) in four parts: the
    // matrix and the vector pipe run side by side, with two pieces' results
    // live.
    auto compute = [&](auto jc, int sn, int sc0, const uint8_t* buf) __attribute__((always_inline)) {
        constexpr int J = decltype(jc)::value;
        const std::integral_constant<int, (J + 1) & 3> jn;
        const Ops& cur = ops[S::kAhead ? J & 1 : 0];
        Ops& next = ops[S::kAhead ? (J + 1) & 1 : 0];
        const uint8_t* xq0 = buf + lr * S::kPitch + 128 * sc0 + 2 * U::at(0, 1) * lh;
        constexpr int kPieces = 2 * S::kTS;
        constexpr int kMf = 2 * S::kP;                        // MFMAs of a piece
        f32x16 dot[2][U::kSub];
        u32x4 xq[2][S::kP][2];
        auto read_x = [&](auto nc) __attribute__((always_inline)) {
            constexpr int e = decltype(nc)::value, b = e / S::kTS, t = e % S::kTS;
#pragma unroll
            for (int k = 0; k < S::kP; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xq[e & 1][k][h] =
                        *reinterpret_cast<const u32x4*>(xq0 + (k * TN + 32 * t) * S::kPitch + 64 * b + 2 * U::at(h, 0));
        };
        read_x(std::integral_constant<int, 0>{});
        if constexpr (S::kAhead) {
            decode_scales(jn, sn, next);
            decode_codes(jn, sn, std::integral_constant<int, 0>{}, next);
        }
        constexpr int kSlots = (kPieces + 1) * kMf;
        // the wave that multiplies goes before those that stage and decode
        // (2048 tokens x 14336 x 4096 Q4_0 397 -> 386 us, weights for single
        // tokens 137 -> 127)
        __builtin_amdgcn_s_setprio(1);
        static_for(std::make_integer_sequence<int, kPieces + 1>{}, [&](auto nc) __attribute__((always_inline)) {
            constexpr int e = decltype(nc)::value;
            constexpr int b = e / S::kTS;
            constexpr int pe = e > 0 ? e - 1 : 0, pb = pe / S::kTS, pt = pe % S::kTS;
            if constexpr (e + 1 < kPieces) read_x(std::integral_constant<int, e + 1>{});
            static_for(std::make_integer_sequence<int, kMf>{}, [&](auto mc) __attribute__((always_inline)) {
                constexpr int m = decltype(mc)::value;
                constexpr int h = m / S::kP, k = m % S::kP;
                if constexpr (e < kPieces) {
                    constexpr int o = U::kSub == 2 ? h : 0;
                    f32x16 c;
                    if constexpr (k == 0 && (U::kSub == 2 || h == 0)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) c[i] = 0.f;
                    } else {
                        c = dot[e & 1][o];
                    }
                    dot[e & 1][o] = XOp<XT>::mfma(xq[e & 1][k][h], cur.op[b][h], c);
                }
                if constexpr (e > 0) {
                    // the m-th share of the piece before
                    constexpr int all = 16 * U::kSub, i0 = all * m / kMf, i1 = all * (m + 1) / kMf;
#pragma unroll
                    for (int i = i0; i < i1; ++i)
                        acc[pt][i & 15] = __builtin_fmaf(cur.d[pb][i >> 4], dot[pe & 1][i >> 4][i & 15], acc[pt][i & 15]);
                }
                static_for(std::make_integer_sequence<int, 3>{}, [&](auto tc) __attribute__((always_inline)) {
                    constexpr int t = decltype(tc)::value + 1;
                    if constexpr (S::kAhead && e * kMf + m == kSlots * t / 4 - 1)
                        decode_codes(jn, sn, std::integral_constant<int, t>{}, next);
                });
                __builtin_amdgcn_sched_barrier(0x4 | 0x10);            // scalar and global memory may pass
            });
            // the scalings stay here (they are used a step later only)
            if constexpr (e > 0) asm volatile("" : "+v"(acc[pt]));
        });
        __builtin_amdgcn_s_setprio(0);
        if constexpr (U::kSums) {
            // mu times the block sums of x, both blocks of the step in one MFMA
            const u32x4 mw = min_operand<0>(cur.mu);
            const u32x4* mx = reinterpret_cast<const u32x4*>(buf + S::kX) + (2 * sc0 + lh) * TN + lr;
#pragma unroll
            for (int t = 0; t < S::kTS; ++t) acc[t] = XOp<__bf16>::mfma(mx[32 * t], mw, acc[t]);
        }
    };

    // One barrier a chunk: the buffer of chunk c + 1 was last read in chunk
    // c - 1, before the barrier that ended it.
    {
        XRegs gx[S::kXAhead];                  // chunk c in gx[c % kXAhead]
#pragma unroll
        for (int k = 0; k < S::kXAhead; ++k)
#pragma unroll
            for (int i = 0; i < S::kXL; ++i) gx[k].x[i].zero();       // tokens past the tile's stay 0
#pragma unroll
        for (int k = 0; k < S::kXAhead; ++k) load_x(k, gx[k]);
        auto decode = [&](auto jc, int s, Ops& o) __attribute__((always_inline)) {
            decode_scales(jc, s, o);
            static_for(std::make_integer_sequence<int, 4>{},
                       [&](auto pc) __attribute__((always_inline)) { decode_codes(jc, s, pc, o); });
        };
        if constexpr (S::kAhead) {
            const std::integral_constant<int, 0> j0;
            put_w();
            load_w(1);
            read_raw(j0, 0);
            decode(j0, 0, ops[0]);
            read_raw(std::integral_constant<int, 1>{}, 0);
        }
        put_x(0, gx[0]);
        load_x(S::kXAhead, gx[0]);
        __syncthreads();
        for (int s = 0; s < rounds; ++s) {
            static_for(std::make_integer_sequence<int, 4>{}, [&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                const int c = kParts * s + j / S::kCHS;
                // the slot changes once its last step's words are read (LDS
                // keeps a wave's order)
                if constexpr (!S::kAhead) {
                    if constexpr (j == 0) {
                        put_w();
                        load_w(s + 1);
                    }
                    read_raw(jc, s);
                    decode(jc, s, ops[0]);
                }
                compute(jc, j == 3 ? s + 1 : s, S::kCHS * wk + j % S::kCHS, lds + (c & 1) * S::kBuf);
                if constexpr (S::kAhead) {
                    // the words of the step after next
                    if constexpr (j == 2) {
                        put_w();
                        load_w(s + 2);
                    }
                    read_raw(std::integral_constant<int, (j + 2) & 3>{}, j >= 2 ? s + 1 : s);
                }
                if constexpr (j % S::kCHS == S::kCHS - 1) {
                    // past the last chunk: not read
                    XRegs& g = gx[(j / S::kCHS + 1) % S::kXAhead];
                    put_x(c + 1, g);
                    load_x(c + 1 + S::kXAhead, g);
                    __syncthreads();
                }
            });
        }
    }
    if constexpr (LORA)
        add_adapters<TN, KG, S::kThreads>(a.lora, s_adapter, start, count, a.n_items, a.rows,
                                          min(row0 + wr + lr, a.rows - 1), wk, lds, acc);
    __syncthreads();

    // results through LDS, so that stores run along the rows
    float* out = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < S::kTS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            out[(wk * TN + 32 * t + 8 * (i >> 2) + 4 * lh + (i & 3)) * S::kOutPitch + wr + lr] = acc[t][i];
    __syncthreads();
    // four rows a thread; rows of a tile are a power of two
    const int quads = out_rows >> 2, qshift = __builtin_ctz(quads);
    const int all_quads = count << qshift;
    auto result = [&](int j, int rr) __attribute__((always_inline)) {
        f32x4 v = *reinterpret_cast<const f32x4*>(out + j * S::kOutPitch + rr);
#pragma unroll
        for (int k = 1; k < KG; ++k) v += *reinterpret_cast<const f32x4*>(out + (k * TN + j) * S::kOutPitch + rr);
        return v;
    };
    float open = 0.f;             // NaN once an output of this thread's is not finite
    for (int i = tid; i < all_quads; i += S::kThreads) {
        const int j = i >> qshift, r = (i & (quads - 1)) << 2;
        f32x4 v = result(j, r);
        if (a.swiglu) {
            const f32x4 u = result(j, out_rows + r);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = silu(v[k]) * u[k];      // of a sum that is not finite: not finite
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) open = __builtin_fmaf(v[k], 0.f, open);
        if constexpr (LORA) {
            if (s_adapter[j] < -1 || s_adapter[j] >= a.lora.n_adapters) v = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
        }
        store_y4(a.y, a.y_type, (int64_t)s_item[j] * a.ldy + row0 + r, v, a.rows - row0 - r, a.yvec != 0);
    }
    if (__ballot(open != 0.f) == 0) return;

    // Sums that are not finite.  An infinite activation (and a finite one
    // that the first bf16 piece or a block's sum of codes takes past the
    // largest float) meets zero codes, pieces of NaN and both terms of a
    // minimum: NaN where the weights' own products give an infinity, or a
    // number.  These outputs are computed again from the weights one by one,
    // by the whole wave.  A token with a NaN keeps its NaN.  What this needs
    // of the arguments and the lane's number is read again: held through the
    // main loop it took four registers.  Where all sums are finite the test
    // for it costs up to 1% (block of 2048 tokens 485.3 -> 489 us, 101 tokens
    // with 40 adapters 96.9 -> 98.2).
    const TileDev& b = again_args();
    const int l64 = again_lane();
    const uint8_t* wmat = b.W + min(s_group, b.n_groups - 1) * b.estride;
    const int64_t row_bytes = (int64_t)(b.nb / 8 * U::kRow + b.nb % 8 * (U::kRow / 8));
    int looked = -1;              // the token looked through last, whether it holds a NaN
    bool nan_in = false;
    for (int i0 = 64 * wave; i0 < all_quads; i0 += S::kThreads) {
        const int i = min(i0 + l64, all_quads - 1), j = i >> qshift, r = (i & (quads - 1)) << 2;
        bool again = !finite(result(j, r));
        if (b.swiglu) again |= !finite(result(j, out_rows + r));
        if constexpr (LORA) again &= s_adapter[j] >= -1 && s_adapter[j] < b.lora.n_adapters;
        for (uint64_t todo = __ballot(again && i0 + l64 < all_quads); todo; todo &= todo - 1) {
            const int from = __builtin_ctzll(todo);
            const int jj = __builtin_amdgcn_readlane(j, from), rr = row0 + __builtin_amdgcn_readlane(r, from);
            const XT* x = static_cast<const XT*>(b.x) + s_x[jj];
            if (looked != jj) {
                looked = jj;
                bool n = false;
                for (int c = l64; c < 32 * b.nb; c += 64) {
                    const float f = XIn<XT>::load1(x + c);
                    n |= f != f;
                }
                nan_in = __ballot(n) != 0;
            }
            if (nan_in) continue;
            for (int row = rr; row < min(rr + 4, b.rows); ++row) {
                float v = 0.f;
                for (int up = 0; up < (b.swiglu ? 2 : 1); ++up) {
                    const uint8_t* wr = wmat + (up ? b.rows + row : row) * row_bytes;
                    float s = 0.f;
                    for (int blk = l64; blk < b.nb; blk += 64)
#pragma unroll 8
                        for (int c = 32 * blk; c < 32 * blk + 32; ++c)
                            s = __builtin_fmaf(U::weight(wr, c), XIn<XT>::load1(x + c), s);
                    if constexpr (LORA) {
                        const int ad = s_adapter[jj];
                        for (int k = l64; ad >= 0 && k < b.lora.rank; k += 64) {
                            float t = 0.f;
                            for (int p = 0; p < b.lora.parts; ++p)
                                t += b.lora.v[((int64_t)p * b.n_items + s_item[jj]) * b.lora.rank + k];
                            s = __builtin_fmaf(lora_b(b.lora, ((int64_t)ad * b.rows + row) * b.lora.rank + k), t, s);
                        }
                    }
#pragma unroll
                    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
                    v = up ? silu(v) * s : s;
                }
                if (l64 == 0) store_y(b.y, b.y_type, (int64_t)s_item[jj] * b.ldy + row, v);
            }
        }
    }
}

template <class F, class XT, int TN, int KG, bool LORA>
int32_t launch_tile(const TileCall& c, int plan_tile, hipStream_t st) {
    using S = TileShape<F, XT, TN, KG>;
    if (!c.plan) plan_tile = TN;
    const int out_rows = c.swiglu ? S::kTM / 2 : S::kTM;
    TileDev d;
    d.W = c.W;
    d.estride = c.estride;
    d.rows = (int)c.rows;
    d.nb = (int)(c.cols / 32);
    d.row_tiles = (int)((c.rows + out_rows - 1) / out_rows);
    d.plan = c.plan;
    d.n_items = (int)c.n_items;
    d.n_groups = c.n_groups;
    d.top_k = c.top_k;
    d.plan_tile = plan_tile;      // without a plan, TN
    d.x = c.x;
    d.xs_tok = c.xs_tok;
    d.xs_slot = c.xs_slot;
    d.y = c.y;
    d.y_type = c.y_type;
    d.ldy = c.ldy;
    d.swiglu = c.swiglu;
    d.yvec = c.ldy % 4 == 0 && aligned(c.y, c.y_type == QMV_X_F32 ? 16 : 8);
    const int per16 = 16 / (int)sizeof(XT);
    d.vec = aligned(c.x, 16) && c.xs_tok % per16 == 0 && c.xs_slot % per16 == 0;
    d.tiles_at = (int)plan_tiles_at(c.n_groups);
    d.order_at = c.plan ? (int)plan_order_at(c.n_items, c.n_groups) : 0;
    d.lora = c.lora;
    const int units = (d.row_tiles + kRowGroup - 1) / kRowGroup;
    d.row_unit = (d.row_tiles + units - 1) / units;
    const int split = plan_tile / TN;
    const int64_t whole = c.plan ? plan_tile_bound(c.n_items, c.n_groups, plan_tile) : (c.n_items + plan_tile - 1) / plan_tile;
    int64_t grid;
    if (split == 1)
        grid = whole * d.row_tiles;
    else
        grid = (whole * units + kXcds - 1) / kXcds * kXcds * split * d.row_unit;
    if (grid > 0xffffffffll / S::kThreads)        // a launch's threads are counted in 32 bits
        return fail(QMV_EINVAL, "qmv: %lld tiles exceed a launch", (long long)grid);
    auto kern = tile_kernel<F, XT, TN, KG, LORA>;
    size_t dyn_max = 0;
    if (const int32_t e = lds_limit(reinterpret_cast<const void*>(kern), kLdsMax, "qmv", &dyn_max)) return e;
    const size_t lds = std::max<size_t>(S::kLds, LORA ? S::kLora : 0);
    if (lds > dyn_max) return fail(QMV_EHIP, "qmv: the tile kernel's LDS exceeds the device's");
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(S::kThreads), lds, st, d);
    return check_launch("qmv");
}

template <class F, class XT, int TN, int KG>
int32_t launch_tile_s(const TileCall& c, int tile, hipStream_t st) {
    return c.lora.rank ? launch_tile<F, XT, TN, KG, true>(c, tile, st) : launch_tile<F, XT, TN, KG, false>(c, tile, st);
}

// Which tile.  TN 128 by 128 rows (fp32 activations, of three times the LDS
// and MFMAs: 64) where the plan's tiles are of 128 and one workgroup each
// fills the GPU, else TN 32.  bf16 x, 32 experts of 1536 x 2048, exactly 64 /
// 96 / 128 / 192 / 256 tokens each: TN 128 45 / 46 / 48 / 83 / 85 us in Q4_0
// and 53 / 56 / 58 / 91 / 94 in Q8_0, TN 32 34 / 52 / 61 / 110 / 116 and 53 /
// 74 / 84 / 161 / 162.  A tile costs the same for 1 token as for 128: with
// 128 tokens each on average half the experts take two, TN 128 89 (Q4_0) and
// 93 (Q8_0) against 78 and 110; with 160 82 and 90 against 110 and 162.
// Under that, 512 tokens through 6144 x 4096 (192 wide tiles): TN 128 68
// (Q4_0) and 75 (Q8_0), TN 32 59 and 87.
//
// With TN 32, waves of a workgroup share rows (KG) where one per 32 rows and
// tile would leave the SIMDs short of waves: as many as have all workgroups
// on the GPU at once.  20 tokens, bf16, n x 4096, the number of waves on
// either side of each border:
//   KG 8 to 4 past 256   Q8_0 256: 17.2 / 18.4 us, 448: 31.8 / 24.2;  Q4_K 18.1 / 20.5, 32.9 / 26.0
//   KG 4 to 2 past 512   Q8_0 512: 24.7 / 27.5, 576: 36.5 / 34.8;  Q4_0 20.1 / 22.5, 31.0 / 27.7;  Q6_K 28.7 / 32.3, 42.4 / 43.3
//   KG 2 to 1 past 1024 in Q8_0 (two workgroups each, the others three)
//                        1024: 36.4 / 41.1, 1152: 55.7 / 53.1
//        past 1536       Q4_0 1536: 36.5 / 43.3, 1600: 50.3 / 43.3;  Q6_K 58.3 / 73.8, 78.2 / 73.9
// 101 tokens with 40 adapters through 4096 x 14336 (512 waves): Q4_K KG 4 97,
// KG 8 114, KG 2 115, Q8_0 82, 98, 102; through 14336 x 4096 (1792) KG 2 / 1
// 90 / 78 and 87 / 73.  fp32 (a workgroup of KG 4 each):
//   KG 4 to 2 past 256   Q8_0 256: 26.7 / 33.9, 448: 48.9 / 36.1
//   KG 2 to 1 past 512 where LDS holds one workgroup (Q8_0, Q6_K)
//                        Q8_0 512: 37.3 / 60.6, 576: 68.0 / 61.5
//        from 2048       Q4_0 1536: 70.2 / 86.0, 2048 (n x 2048): 48.1 / 47.2;  Q4_K 2048: 55.5 / 49.2
template <class F, class XT>
int32_t launch_tile_n(const TileCall& c, hipStream_t st) {
    constexpr bool kWideX = std::is_same<XT, float>::value;
    constexpr int kWide = kWideX ? 64 : 128;
    const int tile = plan_tile(c.n_items, c.plan ? c.n_groups : 1);
    // a group's items on average; at most as many groups as items
    const int64_t groups = c.plan ? std::min<int64_t>(c.n_groups, c.n_items) : 1;
    const int64_t matrix_rows = c.swiglu ? 2 * c.rows : c.rows;
    const int64_t each = c.n_items / groups, cus = device_cu_count();
    const int64_t wide = groups * ((each + kWide - 1) / kWide) * ((matrix_rows + 127) / 128);
    if (tile == 128 && wide >= cus) return launch_tile_s<F, XT, kWide, 1>(c, tile, st);
    const int64_t waves = groups * ((each + 31) / 32) * ((matrix_rows + 31) / 32);
    // KG 4 and 8 have 16 gate rows and 16 up rows in a wave: their bytes have
    // to be within the 32-bit offsets from its first row
    const bool near = !c.swiglu || c.rows * (c.cols / 32) < (1ll << 25);
    constexpr int kTwo = TileShape<F, XT, 32, 2>::kWgs;
    if constexpr (kWideX) {
        if (waves <= cus && near) return launch_tile_s<F, XT, 32, 4>(c, tile, st);
        if (kTwo > 1 ? waves < 8 * cus : waves <= 2 * cus) return launch_tile_s<F, XT, 32, 2>(c, tile, st);
    } else {
        if (waves <= cus && near) return launch_tile_s<F, XT, 32, 8>(c, tile, st);
        if (waves <= 2 * cus && near) return launch_tile_s<F, XT, 32, 4>(c, tile, st);
        if (waves <= 2 * kTwo * cus) return launch_tile_s<F, XT, 32, 2>(c, tile, st);
    }
    return launch_tile_s<F, XT, 32, 1>(c, tile, st);
}

template <class F>
int32_t launch_tile_x(const TileCall& c, hipStream_t st) {
    switch (c.x_type) {
    case QMV_X_F32: return launch_tile_n<F, float>(c, st);
    case QMV_X_F16: return launch_tile_n<F, _Float16>(c, st);
    default: return launch_tile_n<F, __bf16>(c, st);
    }
}

}  // namespace
}  // namespace qmv
