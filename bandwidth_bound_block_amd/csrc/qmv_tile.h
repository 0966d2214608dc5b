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
#pragma once
#include <type_traits>

#include "qmv_block_decode.h"
#include "qmv_group.h"

namespace qmv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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
// Experts may follow each other at 2-byte strides (34- and 18-byte blocks),
// while the blocks' fetches go by the block's parity in a matrix that starts
// on a word: where this one starts 2 bytes past it, the block before the
// first does.
template <class F>
__device__ __forceinline__ void fetch_even(const uint8_t* W, int64_t g, typename F::Raw& r) {
    const int odd = (int)(reinterpret_cast<uintptr_t>(W) & 2) >> 1;
    F::fetch(W - odd * F::kBytes, g + odd, r);
}

// Unit<F>: one 32-weight block of one row.  fetch() issues its loads,
// decode() leaves the 32 codes in weight order as signed bytes, the scale of
// each kSub-th of the block, and mu.
template <class F> struct Unit;

template <> struct Unit<Q8_0> {
    static constexpr int kSub = 1;
    static constexpr bool kSums = false;
    using Raw = Q8_0::Raw;
    __device__ static void fetch(const uint8_t* W, int row, int nb, int blk, Raw& r) {
        fetch_even<Q8_0>(W, (int64_t)row * nb + blk, r);
    }
    __device__ static void decode(const Raw& r, int, uint32_t (&q)[8], float (&s)[kSub], float&) {
        float m;
        Q8_0::decode(r, s[0], m, q);
    }
};

template <> struct Unit<Q4_0> {
    static constexpr int kSub = 1;
    static constexpr bool kSums = false;
    using Raw = Q4_0::Raw;
    __device__ static void fetch(const uint8_t* W, int row, int nb, int blk, Raw& r) {
        fetch_even<Q4_0>(W, (int64_t)row * nb + blk, r);
    }
    // 16 (c - 8) as signed bytes; d / 16 is exact
    __device__ static void decode(const Raw& r, int, uint32_t (&q)[8], float (&s)[kSub], float&) {
        float d, m;
        uint32_t c[8];
        Q4_0::decode(r, d, m, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) signed_nibbles(c[i], q[i], q[4 + i]);
        s[0] = d * 0.0625f;
    }
};

// c - k per byte, c and k in 0..15: no borrow crosses a byte
__device__ __forceinline__ uint32_t less_pivot(uint32_t c, uint32_t k4) {
    return ((c | 0x80808080u) - k4) ^ 0x80808080u;
}
// the code nearest the zero of D c - M (any code gives the same exact value)
__device__ __forceinline__ float pivot(float D, float M) {
    // fmax/fmin return the number for a NaN operand (D = M = 0): k = 0
    return __builtin_fminf(__builtin_fmaxf(__builtin_rintf(M * __builtin_amdgcn_rcpf(D)), 0.f), 15.f);
}

template <> struct Unit<Q4_1> {
    static constexpr int kSub = 1;
    static constexpr bool kSums = true;
    using Raw = Q4_1::Raw;
    __device__ static void fetch(const uint8_t* W, int row, int nb, int blk, Raw& r) {
        Q4_1::fetch(W, (int64_t)row * nb + blk, r);
    }
    __device__ static void decode(const Raw& r, int, uint32_t (&q)[8], float (&s)[kSub], float& mu) {
        float d, m;
        uint32_t c[8];
        Q4_1::decode(r, d, m, c);
        const float k = pivot(d, -m);
        const uint32_t k4 = (uint32_t)k * 0x01010101u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = less_pivot(c[i] & 0x0f0f0f0fu, k4);
            q[4 + i] = less_pivot((c[i] >> 4) & 0x0f0f0f0fu, k4);
        }
        s[0] = d;
        mu = __builtin_fmaf(d, k, m);
    }
};

// Super-block formats: blk = 8 * super-block + J.
struct Q4KTile {};
template <> struct Unit<Q4KTile> {
    static constexpr int kSub = 1;
    static constexpr bool kSums = true;
    struct Raw {
        u32x4 h, a, b;
    };
    __device__ static void fetch(const uint8_t* W, int row, int nb, int blk, Raw& r) {
        const uint8_t* sb = W + ((int64_t)row * (nb >> 3) + (blk >> 3)) * 144;
        const int o = 16 + 32 * ((blk & 7) >> 1);
        r.h = *reinterpret_cast<const u32x4*>(sb);
        r.a = *reinterpret_cast<const u32x4*>(sb + o);
        r.b = *reinterpret_cast<const u32x4*>(sb + o + 16);
    }
    __device__ static void decode(const Raw& r, int blk, uint32_t (&q)[8], float (&s)[kSub], float& mu) {
        const int J = blk & 7, t = 8 * (J & 3);
        const uint32_t h1 = r.h.y >> t, h2 = r.h.z >> t, h3 = r.h.w >> t;
        const uint32_t sc = J < 4 ? (h1 & 63u) : ((h3 & 15u) | ((h1 >> 2) & 48u));
        const uint32_t mn = J < 4 ? (h2 & 63u) : (((h3 >> 4) & 15u) | ((h2 >> 2) & 48u));
        const float D = half_bits_to_float(r.h.x) * (float)sc;          // exact
        const float M = half_bits_to_float(r.h.x >> 16) * (float)mn;    // exact
        const float k = pivot(D, M);
        const uint32_t k4 = (uint32_t)k * 0x01010101u;
        const uint32_t c[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        const int sh = 4 * (J & 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = less_pivot((c[i] >> sh) & 0x0f0f0f0fu, k4);
        s[0] = D;
        mu = __builtin_fmaf(D, k, -M);
    }
};

struct Q6KTile {};
template <> struct Unit<Q6KTile> {
    static constexpr int kSub = 2;
    static constexpr bool kSums = false;
    // The super-block starts sh = 0 or 2 bytes past a word; words from
    // sb - sh (inside the matrix: sh = 2 only past its first super-block).
    struct Raw {
        u32x4 l0, l1, h0, h1;
        uint32_t l8, h8, sc, d, sh;
    };
    __device__ static void fetch(const uint8_t* W, int row, int nb, int blk, Raw& r) {
        const uint8_t* sb = W + ((int64_t)row * (nb >> 3) + (blk >> 3)) * 210;
        const int sh = (int)(reinterpret_cast<uintptr_t>(sb) & 2);
        const int J = blk & 7;
        const uint8_t* pl = sb - sh + 64 * (J >> 2) + 32 * (J & 1);
        const uint8_t* ph = sb - sh + 128 + 32 * (J >> 2);
        r.l0 = ld16(pl);
        r.l1 = ld16(pl + 16);
        r.l8 = ld4(pl + 32);
        r.h0 = ld16(ph);
        r.h1 = ld16(ph + 16);
        r.h8 = ld4(ph + 32);
        r.sc = ld2(sb + 192 + 2 * J);
        r.d = ld2(sb + 208);
        r.sh = (uint32_t)sh;
    }
    // 4 (c - 32) as signed bytes; d sc / 4 is exact
    __device__ static void decode(const Raw& r, int blk, uint32_t (&q)[8], float (&s)[kSub], float&) {
        const int qt = blk & 3;
        const uint32_t l[9] = {r.l0.x, r.l0.y, r.l0.z, r.l0.w, r.l1.x, r.l1.y, r.l1.z, r.l1.w, r.l8};
        const uint32_t h[9] = {r.h0.x, r.h0.y, r.h0.z, r.h0.w, r.h1.x, r.h1.y, r.h1.z, r.h1.w, r.h8};
        const int sl = qt < 2 ? 0 : 4, su = 6 - 2 * qt;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = __builtin_amdgcn_alignbyte(l[i + 1], l[i], r.sh) >> sl;
            const uint32_t hi = (__builtin_amdgcn_alignbyte(h[i + 1], h[i], r.sh) ^ 0xaaaaaaaau) << su;
            q[i] = ((lo << 2) & 0x3c3c3c3cu) | (hi & 0xc0c0c0c0u);
        }
        const float d4 = half_bits_to_float(r.d) * 0.25f;
        s[0] = d4 * (float)(int8_t)(r.sc & 0xff);
        s[1] = d4 * (float)(int8_t)(r.sc >> 8);
    }
};

// --------------------------------------------------------------- slots
// Eight blocks of each of a wave's 32 rows, loaded as 16-byte pieces with
// neighbouring lanes on neighbouring pieces, kept in registers while the
// blocks before them are computed, then copied to the wave's part of LDS
// (its slot), where each lane takes its block.  Loads by block and lane
// instead (64 lanes on 64 lines) run at 2.4 TB/s for Q4_0 and 1.5 for Q6_K
// whatever the number of waves: the cache looks up one lane's line a cycle.
// kCpr: pieces of a row; kPitch: bytes of a row in the slot, an odd number of
// 16-byte units.  take() leaves what Unit<F>::fetch would.
template <class F, int BYTES, int PITCH>
struct SlotOf {
    static constexpr int kRow = BYTES, kCpr = BYTES / 16, kPitch = PITCH;
    static constexpr int kLoads = (32 * kCpr + 63) / 64;
    struct Regs {
        u32x4 v[kLoads];
    };
    // the lane's piece k: row and byte of the row
    __device__ static int row_of(int k, int lane) { return min(64 * k + lane, 32 * kCpr - 1) / kCpr; }
    __device__ static int byte_of(int k, int lane) { return min(64 * k + lane, 32 * kCpr - 1) % kCpr * 16; }
    __device__ static void load(const uint8_t* W, const uint32_t (&off)[kLoads], uint32_t, int sup, Regs& r) {
        const uint8_t* p = W + (int64_t)sup * kRow;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) r.v[k] = *reinterpret_cast<const u32x4*>(p + off[k]);
    }
    __device__ static void put(const Regs& r, uint8_t* slot, const uint8_t*, uint32_t, int, int lane) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            *reinterpret_cast<u32x4*>(slot + row_of(k, lane) * kPitch + byte_of(k, lane)) = r.v[k];
    }
};
template <class F> struct Slot;
template <> struct Slot<Q8_0> : SlotOf<Q8_0, 272, 272> {
    __device__ static void take(const uint8_t* row, const uint8_t*, int l, Q8_0::Raw& r) { Q8_0::from_lds(row, l, r); }
};
template <> struct Slot<Q4_0> : SlotOf<Q4_0, 144, 144> {
    __device__ static void take(const uint8_t* row, const uint8_t*, int l, Q4_0::Raw& r) { Q4_0::from_lds(row, l, r); }
};
template <> struct Slot<Q4_1> : SlotOf<Q4_1, 160, 176> {
    __device__ static void take(const uint8_t* row, const uint8_t*, int l, Q4_1::Raw& r) { Q4_1::from_lds(row, l, r); }
};
template <> struct Slot<Q4KTile> : SlotOf<Q4KTile, 144, 144> {
    __device__ static void take(const uint8_t* row, const uint8_t*, int l, Unit<Q4KTile>::Raw& r) {
        const u32x4* q = reinterpret_cast<const u32x4*>(row + 16 + 32 * (l >> 1));
        r.h = *reinterpret_cast<const u32x4*>(row);
        r.a = q[0];
        r.b = q[1];
    }
};
// Q6_K: 13 pieces from the word the super-block starts in (0 or 2 bytes
// before it), and its last four bytes on their own: every load stays inside.
template <> struct Slot<Q6KTile> : SlotOf<Q6KTile, 210, 240> {
    struct Regs {
        u32x4 v[kLoads];
        uint32_t t0, t1;
    };
    __device__ static void load(const uint8_t* W, const uint32_t (&off)[kLoads], uint32_t own, int sup, Regs& r) {
        const uint8_t* p = W + (int64_t)sup * kRow;
#pragma unroll
        for (int k = 0; k < kLoads; ++k)     // off: of the piece; whole words before it do not change the parity
            r.v[k] = ld16(reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p + off[k]) & ~(uintptr_t)3));
        r.t0 = ld2(p + own + 206);
        r.t1 = ld2(p + own + 208);
    }
    __device__ static void put(const Regs& r, uint8_t* slot, const uint8_t* W, uint32_t own, int sup, int lane) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            *reinterpret_cast<u32x4*>(slot + row_of(k, lane) * kPitch + byte_of(k, lane)) = r.v[k];
        const bool odd = (reinterpret_cast<uintptr_t>(W + (int64_t)sup * kRow + own) & 2) != 0;
        *reinterpret_cast<uint32_t*>(slot + (lane & 31) * kPitch + 208) = odd ? (r.t0 | (r.t1 << 16)) : r.t1;
    }
    // at: the super-block's address
    __device__ static void take(const uint8_t* row, const uint8_t* at, int l, Unit<Q6KTile>::Raw& r) {
        const int sh = (int)(reinterpret_cast<uintptr_t>(at) & 2);
        const uint8_t* pl = row + 64 * (l >> 2) + 32 * (l & 1);
        const uint8_t* ph = row + 128 + 32 * (l >> 2);
        r.l0 = *reinterpret_cast<const u32x4*>(pl);
        r.l1 = *reinterpret_cast<const u32x4*>(pl + 16);
        r.l8 = ld4(pl + 32);
        r.h0 = *reinterpret_cast<const u32x4*>(ph);
        r.h1 = *reinterpret_cast<const u32x4*>(ph + 16);
        r.h8 = ld4(ph + 32);
        r.sc = ld2(row + sh + 192 + 2 * l);
        r.d = ld2(row + sh + 208);
        r.sh = (uint32_t)sh;
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
    int rows, nb, row_tiles;
    const int32_t* plan;
    int n_items, n_groups, top_k, plan_tile;
    const void* x;
    int64_t xs_tok, xs_slot;
    void* y;
    int y_type;
    int64_t ldy;
    int swiglu, vec;
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

// Exchanges the upper 32 lanes of a with the lower 32 of b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// v of lane l % 32 (a) and of lane l % 32 + 32 (b), in both.
__device__ __forceinline__ void both_halves(float v, float& a, float& b) {
    uint32_t x = fbits(v), y = fbits(v);
    swap_halves(x, y);
    a = __builtin_bit_cast(float, x);
    b = __builtin_bit_cast(float, y);
}

constexpr int kTileWaves = 4;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kLoraRanks = 64;                       // ranks staged at a time
constexpr int kLoraPitch = 2 * kLoraRanks + 16;      // bytes of a token's piece, an odd number of 16-byte units

// The adapters' part of a tile, added to acc: token j of the tile (item
// first + j) gains B_a v_j for a = s_adapter[j].  For each adapter among the
// tile's tokens, its 32 rows of B are multiplied with the v of every 32
// tokens that hold one of its own, and the sums taken over for those tokens
// alone.  v and B are split into three bf16 pieces each (bf16 B has one); the
// products left out are 2^-24 of the sum.  v is staged in `lds` by the whole
// workgroup; waves with add false only stage.
template <int TN>
__device__ __forceinline__ void add_adapters(const LoraTile& l, const int* s_adapter, int first, int count, int n_items,
                                             int rows, int row, bool add, uint8_t* lds, f32x16 (&acc)[TN / 32]) {
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    for (int c0 = 0; c0 < l.rank; c0 += kLoraRanks) {
        const int ranks = min(kLoraRanks, l.rank - c0);
        const int steps = (ranks + 15) >> 4;
        __syncthreads();
        // pairs of ranks, zeros past the last up to whole steps
        for (int i = tid; i < TN * 8 * steps; i += kTileThreads) {
            const int j = i / (8 * steps), r = 2 * (i % (8 * steps));
            float a = 0.f, b = 0.f;
            if (j < count) {
                const float* v = l.v + (int64_t)(first + j) * l.rank + c0 + r;
                for (int p = 0; p < l.parts; ++p, v += (int64_t)n_items * l.rank) {
                    if (r < ranks) a += v[0];
                    if (r + 1 < ranks) b += v[1];
                }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
                *reinterpret_cast<uint32_t*>(lds + (k * TN + j) * kLoraPitch + 2 * r) = w;
                a -= __builtin_bit_cast(float, w << 16);
                b -= __builtin_bit_cast(float, w & 0xffff0000u);
            }
        }
        __syncthreads();
        if (!add) continue;
        uint32_t todo[TN / 32];
        int id[TN / 32];
#pragma unroll
        for (int t = 0; t < TN / 32; ++t) {
            id[t] = s_adapter[32 * t + lr];
            todo[t] = (uint32_t)__ballot(32 * t + lr < count && (unsigned)id[t] < (unsigned)l.n_adapters);
        }
        while (true) {
            int ad = -1;
#pragma unroll
            for (int t = 0; t < TN / 32; ++t)
                if (ad < 0 && todo[t]) ad = __builtin_amdgcn_readlane(id[t], __builtin_ctz(todo[t]));
            if (ad < 0) break;
            const int64_t brow = ((int64_t)ad * rows + row) * l.rank + c0;
            uint32_t own[TN / 32];
#pragma unroll
            for (int t = 0; t < TN / 32; ++t) {
                own[t] = (uint32_t)__ballot(id[t] == ad) & todo[t];
                todo[t] &= ~own[t];
            }
            u32x4 bp[kLoraRanks / 16][3];
#pragma unroll
            for (int s = 0; s < kLoraRanks / 16; ++s) {
                if (s >= steps) continue;
                const int r0 = 16 * s + 8 * lh;
                X8<float> b;
                if (l.vec && r0 + 8 <= ranks) {
                    if (l.b_type == QMV_X_F32) {
                        b.load(static_cast<const float*>(l.B) + brow + r0, true);
                    } else {
                        const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(l.B) + brow + r0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool half = l.b_type == QMV_X_F16;
                            b.v[2 * i] = half ? half_bits_to_float(w[i]) : __builtin_bit_cast(float, w[i] << 16);
                            b.v[2 * i + 1] =
                                half ? half_bits_to_float(w[i] >> 16) : __builtin_bit_cast(float, w[i] & 0xffff0000u);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t at = brow + min(r0 + i, ranks - 1);
                        const float w = l.b_type == QMV_X_F32   ? static_cast<const float*>(l.B)[at]
                                        : l.b_type == QMV_X_F16 ? (float)static_cast<const _Float16*>(l.B)[at]
                                                                : (float)static_cast<const __bf16*>(l.B)[at];
                        b.v[i] = r0 + i < ranks ? w : 0.f;
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
                for (int s = 0; s < kLoraRanks / 16; ++s) {
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
        }
    }
}

constexpr int kXcds = 8;          // workgroups go to the XCDs in turn
constexpr int kTokGroup = 8;      // token tiles that an XCD takes together
// A wave takes 32 weight rows by TN tokens.  Its step is two blocks of each
// row: lane l holds block l / 32 of row l % 32, decodes it alone, and one
// exchange of lane halves turns the two blocks' codes into MFMA operands, so
// no wave waits for another's weights.  KG waves of a workgroup share 32 rows
// and take their eight-block pieces of the row (four steps) in turn; their
// sums are added in a fixed order at the end: where there are few rows, that
// keeps enough loads in flight.  Activations are staged in LDS in chunks of
// CHS steps for each of the KG.  SLOT: weights by whole lines through LDS;
// otherwise (rows off 16 bytes, or of part of eight blocks) by each lane.
template <class F, class XT, int TN, int KG, bool SLOT>
struct TileShape {
    static constexpr int kP = XOp<XT>::kPieces;
    static constexpr int kTM = 32 * kTileWaves / KG;
    static constexpr int kTS = TN / 32;
    static constexpr int kCHS = TN > 32 || kP > 1 || KG > 1 ? 1 : 2;
    // waves of a SIMD that the registers are cut for; few tokens leave the
    // decoding as the bound, and it takes four waves to keep that going
    static constexpr int kOcc = TN > 32 ? 2 : (kP > 1 ? 3 : 4);
    static constexpr int kCH = kCHS * KG;
    static constexpr int kXL = TN * 8 * kCH / kTileThreads;         // 8-column pieces of x per thread and chunk
    static constexpr int kPitch = 128 * kCH + 16;                   // bytes of a staged token: an odd number of 16-byte units, so 8 tokens hit distinct banks
    static constexpr int kX = kP * TN * kPitch;
    static constexpr int kM = Unit<F>::kSums ? 2 * kCH * TN * 16 : 0;
    static constexpr int kBuf = kX + kM;
    static constexpr int kSlot = SLOT ? 32 * Slot<F>::kPitch : 0;   // of a wave
    static constexpr int kOutPitch = kTM + 4;                       // floats
    static constexpr int kOut = KG * TN * kOutPitch * 4;
    static constexpr int kMain = 2 * kBuf + kTileWaves * kSlot;
    static constexpr int kLora = 3 * TN * kLoraPitch;
    static constexpr int kLds = kMain > kOut ? kMain : kOut;
    static_assert(kXL >= 1 && kCHS >= 1, "every thread stages, every wave computes");
};

// LORA: the tokens carry adapters (and there is no plan).
template <class F, class XT, int TN, int KG, bool SLOT, bool LORA>
__global__ __launch_bounds__(kTileThreads, (TileShape<F, XT, TN, KG, SLOT>::kOcc)) void tile_kernel(const TileDev a) {
    using S = TileShape<F, XT, TN, KG, SLOT>;
    using U = Unit<F>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int s_item[TN], s_adapter[LORA ? TN : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int split = a.plan_tile / TN;      // workgroups along a plan's tile
    int tok_tiles;
    if (a.plan) {
        // a plan of other items or groups than the call's is not followed
        if (a.plan[0] != kPlanMagic || a.plan[1] != a.n_items || a.plan[2] != a.n_groups || a.plan[3] != a.plan_tile)
            return;
        tok_tiles = a.plan[4] * split;
    } else {
        tok_tiles = (a.n_items + TN - 1) / TN;
    }
    const int total = tok_tiles * a.row_tiles;
    if ((int)blockIdx.x >= total) return;
    // Tiles in runs, one run to an XCD, and within it kTokGroup token tiles
    // side by side down the rows: the tiles an XCD works on at one time
    // share their weights and activations in its L2.
    const int xcd = blockIdx.x % kXcds;
    const int id = xcd * (total / kXcds) + min(xcd, total % kXcds) + blockIdx.x / kXcds;
    const int t0 = id / (kTokGroup * a.row_tiles) * kTokGroup;
    const int tw = min(kTokGroup, tok_tiles - t0);
    const int in = id - t0 * a.row_tiles;
    const int rt = in / tw, tt = t0 + in % tw;

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
    const int wrow = matrix_row(wr + lr);
    const uint8_t* W = a.W + min(group, a.n_groups - 1) * a.estride;

    // Weights: eight blocks (four steps) of the row at a time.
    constexpr bool kWhole = SLOT && KG == 1;             // no step passes the row's end
    const int sups = (a.nb + 7) >> 3;                    // pieces of eight blocks of a row
    const int rounds = (sups + KG - 1) / KG;
    auto sup_of = [&](int s) __attribute__((always_inline)) { return KG * s + wk; };
    // SLOT: pieces of 16 bytes; otherwise the lane's blocks of steps n, n + 1
    using SL = Slot<F>;
    typename SL::Regs wreg;
    uint32_t woff[SL::kLoads], wown = 0;
    typename U::Raw r0, r1;
    auto block_of = [&](int n) __attribute__((always_inline)) { return 8 * sup_of(n >> 2) + 2 * (n & 3) + lh; };
    auto load_slot = [&](int s) __attribute__((always_inline)) {
        SL::load(W, woff, wown, min(sup_of(s), sups - 1), wreg);
    };
    auto load_lane = [&](int n, typename U::Raw& r) __attribute__((always_inline)) {
        U::fetch(W, wrow, a.nb, min(block_of(n), a.nb - 1), r);
    };
    uint8_t* slot = lds + 2 * S::kBuf + wave * S::kSlot;
    if constexpr (SLOT) {
        const uint32_t pitch = (uint32_t)(sups * SL::kRow);
#pragma unroll
        for (int k = 0; k < SL::kLoads; ++k)
            woff[k] = (uint32_t)matrix_row(wr + SL::row_of(k, lane)) * pitch + (uint32_t)SL::byte_of(k, lane);
        wown = (uint32_t)wrow * pitch;
        load_slot(0);
    } else {
        load_lane(0, r0);
        load_lane(1, r1);
    }

    if (tid < TN) {
        const int at = start + min(tid, count - 1);
        s_item[tid] = a.plan ? a.plan[a.order_at + at] : at;
        if constexpr (LORA) s_adapter[tid] = a.lora.ids[at];
    }
    __syncthreads();
    if (a.plan && group >= a.n_groups) {   // ids that are no group
        for (int i = tid; i < count * out_rows; i += kTileThreads) {
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
    constexpr int kXStep = kTileThreads / (8 * S::kCH);
    constexpr int kParts = 4 / S::kCHS;
    const XT* xp[S::kXL];
#pragma unroll
    for (int i = 0; i < S::kXL; ++i) {
        const int p = s_item[xt + kXStep * i];
        xp[i] = static_cast<const XT*>(a.x) + (int64_t)(p / a.top_k) * a.xs_tok + (int64_t)(p % a.top_k) * a.xs_slot;
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
        for (int i = 0; i < S::kXL; ++i) g.x[i].load(xp[i] + at, vec);
    };
    auto put_x = [&](int c, XRegs& g) __attribute__((always_inline)) {
        uint8_t* buf = lds + (c & 1) * S::kBuf;
        // only the row's last round can hold columns past it
        if (!kWhole && 256 * KG * (c / kParts + 1) > 32 * a.nb && column(c) >= 32 * a.nb) {
#pragma unroll
            for (int i = 0; i < S::kXL; ++i) g.x[i].zero();
        }
#pragma unroll
        for (int i = 0; i < S::kXL; ++i) {
            const int tok = xt + kXStep * i;
            u32x4 p[S::kP];
            g.x[i].pieces(p);
#pragma unroll
            for (int k = 0; k < S::kP; ++k)
                *reinterpret_cast<u32x4*>(buf + (k * TN + tok) * S::kPitch + 16 * xc) = p[k];
            if constexpr (U::kSums) {
                float t = g.x[i].sum();      // of 8 columns; four lanes hold a block's 32
                t += dpp_mov<0xB1>(t);
                t += dpp_mov<0x4E>(t);
                if ((xc & 3) == 0)
                    *reinterpret_cast<u32x4*>(buf + S::kX + ((xc >> 2) * TN + tok) * 16) = min_operand<1>(t);
            }
        }
    };

    f32x16 acc[S::kTS];
#pragma unroll
    for (int t = 0; t < S::kTS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;

    // Step n of the wave, the sc0-th of those staged in buf: decode, then for
    // each block and 32 tokens (a piece) its MFMAs, between the scalings of
    // the piece before it: a piece's results are 16 fused multiply-adds a
    // lane, about as long as its two MFMAs, so the two pipes run side by side
    // with two pieces' results live.
    auto compute = [&](int n, int sc0, const uint8_t* buf, const typename U::Raw& raw) __attribute__((always_inline)) {
        const int blk = block_of(n);
        uint32_t q[8], op[16];
        float sc[U::kSub], mu = 0.f, d[2][U::kSub];
        U::decode(raw, blk, q, sc, mu);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            op[2 * j] = XOp<XT>::pair(sbyte(q[j], 0), sbyte(q[j], 1));
            op[2 * j + 1] = XOp<XT>::pair(sbyte(q[j], 2), sbyte(q[j], 3));
        }
        // lanes hold codes 8m..8m+7 of their block in op[4m..4m+3]; after the
        // exchange op[0..3], op[8..11] are the first block's operands and
        // op[4..7], op[12..15] the second's
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) swap_halves(op[8 * h + j], op[8 * h + 4 + j]);
        const bool live = kWhole || blk < a.nb;        // past the row: its scale is 0
#pragma unroll
        for (int h = 0; h < U::kSub; ++h) both_halves(live ? sc[h] : 0.f, d[0][h], d[1][h]);

        const uint8_t* xq0 = buf + lr * S::kPitch + 128 * sc0 + 16 * lh;
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
                        *reinterpret_cast<const u32x4*>(xq0 + (k * TN + 32 * t) * S::kPitch + 64 * b + 32 * h);
        };
        read_x(std::integral_constant<int, 0>{});
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
                    constexpr int w = 8 * h + 4 * b;
                    f32x16 c;
                    if constexpr (k == 0 && (U::kSub == 2 || h == 0)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) c[i] = 0.f;
                    } else {
                        c = dot[e & 1][o];
                    }
                    dot[e & 1][o] = XOp<XT>::mfma(xq[e & 1][k][h], u32x4{op[w], op[w + 1], op[w + 2], op[w + 3]}, c);
                }
                if constexpr (e > 0) {
                    // the m-th share of the piece before
                    constexpr int all = 16 * U::kSub, i0 = all * m / kMf, i1 = all * (m + 1) / kMf;
#pragma unroll
                    for (int i = i0; i < i1; ++i)
                        acc[pt][i & 15] = __builtin_fmaf(d[pb][i >> 4], dot[pe & 1][i >> 4][i & 15], acc[pt][i & 15]);
                }
                __builtin_amdgcn_sched_barrier(0x4 | 0x10);            // scalar and global memory may pass
            });
            // the scalings stay here (they are used a step later only)
            if constexpr (e > 0) asm volatile("" : "+v"(acc[pt]));
        });
        if constexpr (U::kSums) {
            // mu times the block sums of x, both blocks of the step in one MFMA
            const u32x4 mw = min_operand<0>(live ? mu : 0.f);
            const u32x4* mx = reinterpret_cast<const u32x4*>(buf + S::kX) + (2 * sc0 + lh) * TN + lr;
#pragma unroll
            for (int t = 0; t < S::kTS; ++t) acc[t] = XOp<__bf16>::mfma(mx[32 * t], mw, acc[t]);
        }
    };

    // One barrier a chunk: the buffer of chunk c + 1 was last read in chunk
    // c - 1, before the barrier that ended it.
    {
        XRegs gx;
        load_x(0, gx);
        put_x(0, gx);
        load_x(1, gx);
        __syncthreads();
        for (int s = 0; s < rounds; ++s) {
            if constexpr (SLOT) {
                // the slot's last reads are this wave's own: LDS keeps their order
                SL::put(wreg, slot, W, wown, min(sup_of(s), sups - 1), lane);
                load_slot(s + 1);
            }
            static_for(std::make_integer_sequence<int, 4>{}, [&](auto jc) __attribute__((always_inline)) {
                constexpr int j = decltype(jc)::value;
                const int c = kParts * s + j / S::kCHS;
                const uint8_t* buf = lds + (c & 1) * S::kBuf;
                const int sc0 = S::kCHS * wk + j % S::kCHS;
                const int n = 4 * s + j;
                if constexpr (SLOT) {
                    typename U::Raw r;
                    SL::take(slot + lr * SL::kPitch, W + wown + (int64_t)min(sup_of(s), sups - 1) * SL::kRow, 2 * j + lh, r);
                    compute(n, sc0, buf, r);
                } else {
                    compute(n, sc0, buf, j & 1 ? r1 : r0);
                    load_lane(n + 2, j & 1 ? r1 : r0);
                }
                if constexpr (j % S::kCHS == S::kCHS - 1) {
                    put_x(c + 1, gx);                // past the last chunk: not read
                    load_x(c + 2, gx);
                    __syncthreads();
                }
            });
        }
    }
    if constexpr (LORA)
        add_adapters<TN>(a.lora, s_adapter, start, count, a.n_items, a.rows, min(row0 + wr + lr, a.rows - 1), wk == 0,
                         lds, acc);
    __syncthreads();

    // results through LDS, so that stores run along the rows
    float* out = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int t = 0; t < S::kTS; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            out[(wk * TN + 32 * t + 8 * (i >> 2) + 4 * lh + (i & 3)) * S::kOutPitch + wr + lr] = acc[t][i];
    __syncthreads();
    auto result = [&](int j, int r) __attribute__((always_inline)) {
        float v = out[j * S::kOutPitch + r];
#pragma unroll
        for (int k = 1; k < KG; ++k) v += out[(k * TN + j) * S::kOutPitch + r];
        return v;
    };
    for (int i = tid; i < count * out_rows; i += kTileThreads) {
        const int j = i / out_rows, r = i % out_rows;
        if (row0 + r >= a.rows) continue;
        float v = result(j, r);
        if (a.swiglu) v = silu(v) * result(j, out_rows + r);
        if constexpr (LORA)
            if (s_adapter[j] < -1 || s_adapter[j] >= a.lora.n_adapters) v = __builtin_nanf("");
        store_y(a.y, a.y_type, (int64_t)s_item[j] * a.ldy + row0 + r, v);
    }
}

template <class F, class XT, int TN, int KG, bool SLOT, bool LORA>
int32_t launch_tile(const TileCall& c, int plan_tile, hipStream_t st) {
    using S = TileShape<F, XT, TN, KG, SLOT>;
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
    d.plan_tile = plan_tile;
    d.x = c.x;
    d.xs_tok = c.xs_tok;
    d.xs_slot = c.xs_slot;
    d.y = c.y;
    d.y_type = c.y_type;
    d.ldy = c.ldy;
    d.swiglu = c.swiglu;
    const int per16 = 16 / (int)sizeof(XT);
    d.vec = aligned(c.x, 16) && c.xs_tok % per16 == 0 && c.xs_slot % per16 == 0;
    d.tiles_at = (int)plan_tiles_at(c.n_groups);
    d.order_at = c.plan ? (int)plan_order_at(c.n_items, c.n_groups) : 0;
    d.lora = c.lora;
    const int64_t tiles = c.plan ? plan_tile_bound(c.n_items, c.n_groups, plan_tile) * (plan_tile / TN)
                                 : (c.n_items + TN - 1) / TN;
    if (tiles * d.row_tiles > 0x7fffffff)
        return fail(QMV_EINVAL, "qmv: %lld tiles exceed a launch", (long long)(tiles * d.row_tiles));
    auto kern = tile_kernel<F, XT, TN, KG, SLOT, LORA>;
    size_t dyn_max = 0;
    if (const int32_t e = lds_limit(reinterpret_cast<const void*>(kern), kLdsMax, "qmv", &dyn_max)) return e;
    const size_t lds = std::max<size_t>(S::kLds, LORA ? S::kLora : 0);
    if (lds > dyn_max) return fail(QMV_EHIP, "qmv: the tile kernel's LDS exceeds the device's");
    hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * d.row_tiles)), dim3(kTileThreads), lds, st, d);
    return check_launch("qmv");
}

// Whole lines where the rows are whole pieces of eight blocks on 16 bytes
// (Q6_K: any; its pieces are 210 bytes) and the lanes' offsets fit 32 bits.
template <class F>
bool slots_fit(const TileCall& c) {
    constexpr int kRow = Slot<F>::kRow;
    const int64_t matrix_rows = c.swiglu ? 2 * c.rows : c.rows;
    if (c.cols % 256 || matrix_rows * (c.cols / 256) * kRow > 0xffffffffll) return false;
    return kRow % 16 != 0 || (aligned(c.W, 16) && c.estride % 16 == 0);
}

template <class F, class XT, int TN, int KG>
int32_t launch_tile_s(const TileCall& c, int tile, hipStream_t st) {
    if (c.lora.rank)
        return slots_fit<F>(c) ? launch_tile<F, XT, TN, KG, true, true>(c, tile, st)
                               : launch_tile<F, XT, TN, KG, false, true>(c, tile, st);
    return slots_fit<F>(c) ? launch_tile<F, XT, TN, KG, true, false>(c, tile, st)
                           : launch_tile<F, XT, TN, KG, false, false>(c, tile, st);
}

// fp32 activations take three times the LDS and MFMAs: 64 tokens by 256 rows
// where 16-bit ones take 128 by 128.
template <class F, class XT>
int32_t launch_tile_n(const TileCall& c, hipStream_t st) {
    constexpr int kWide = std::is_same<XT, float>::value ? 64 : 128;
    const int tile = c.plan ? plan_tile(c.n_items, c.n_groups) : plan_tile(c.n_items, 1);
    // waves that one per 32 rows and tile would be: a group's items on
    // average, at most as many groups as items
    const int64_t groups = c.plan ? std::min<int64_t>(c.n_groups, c.n_items) : 1;
    const int64_t matrix_rows = c.swiglu ? 2 * c.rows : c.rows;
    const int64_t wide = groups * ((c.n_items / groups + kWide - 1) / kWide) * ((matrix_rows + 127) / 128);
    if (tile == 128 && wide >= device_cu_count()) return launch_tile_s<F, XT, kWide, 1>(c, tile, st);
    if (const char* e = getenv("KG")) {   // TEMP
        const int kg = atoi(e);
        if constexpr (!std::is_same<XT, float>::value) if (kg == 4) return launch_tile_s<F, XT, 32, 4>(c, tile, st);
        if (kg == 2) return launch_tile_s<F, XT, 32, 2>(c, tile, st);
        if (kg == 1) return launch_tile_s<F, XT, 32, 1>(c, tile, st);
    }
    const int64_t waves = groups * ((c.n_items / groups + 31) / 32) * ((matrix_rows + 31) / 32);
    if constexpr (!std::is_same<XT, float>::value)
        if (waves < 4 * device_cu_count() && !c.swiglu) return launch_tile_s<F, XT, 32, 4>(c, tile, st);
    if (waves < 8 * device_cu_count()) return launch_tile_s<F, XT, 32, 2>(c, tile, st);
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
