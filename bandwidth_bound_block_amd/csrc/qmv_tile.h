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

constexpr int kTileBlks = 2;      // 32-weight blocks of a step
constexpr int kTilePitch = 64 * kTileBlks + 16;   // bytes of a staged row: an odd number of 16-byte units, so 8 rows hit distinct banks
constexpr int kXcds = 8;          // workgroups go to the XCDs in turn
constexpr int kTokGroup = 8;      // token tiles that an XCD takes together

// A workgroup of kNW waves: kTM weight rows (one block of one row per thread
// and step) by TN tokens; a wave takes 32 kRS rows by 32 kTS tokens.
template <class F, class XT, int TN>
struct TileShape {
    static constexpr int kP = XOp<XT>::kPieces;
    static constexpr int kNW = TN == 64 ? 8 : 4;
    static constexpr int kNT = 64 * kNW;
    static constexpr int kTM = kNT / kTileBlks;
    static constexpr int kWt = TN == 32 ? 1 : 2;                    // waves along the tokens
    static constexpr int kWr = kNW / kWt;                           // waves along the rows
    static constexpr int kRS = kTM / kWr / 32;
    static constexpr int kTS = TN / kWt / 32;
    static constexpr int kXL = TN * 8 / kNT;                        // 8-column pieces of x per thread and step 
    static constexpr int kW = kTM * kTilePitch;
    static constexpr int kX = kP * TN * kTilePitch;
    static constexpr int kS = kTileBlks * Unit<F>::kSub * kTM * 4;
    static constexpr int kM = Unit<F>::kSums ? kTileBlks * (kTM + TN) * 16 : 0;
    static constexpr int kBuf = kW + kX + kS + kM;
    static constexpr int kOutPitch = kTM + 4;                       // floats
    static constexpr int kLds = 2 * kBuf > TN * kOutPitch * 4 ? 2 * kBuf : TN * kOutPitch * 4;
    static_assert(kXL >= 1 && kRS >= 1 && kTS >= 1, "every thread stages");
};

template <class F, class XT, int TN>
__global__ __launch_bounds__((TN == 64 ? 512 : 256), 2) void tile_kernel(const TileDev a) {
    using S = TileShape<F, XT, TN>;
    using U = Unit<F>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int s_item[TN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Tiles in runs, one run to an XCD, and within it kTokGroup token tiles
    // side by side down the rows: the tiles an XCD works on at one time
    // share their weights and activations in its L2.
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
    for (int j = tid; j < TN; j += S::kNT) {
        const int at = start + min(j, count - 1);
        s_item[j] = a.plan ? a.plan[a.order_at + at] : at;
    }
    __syncthreads();
    if (a.plan && group >= a.n_groups) {   // ids that are no group
        for (int i = tid; i < count * out_rows; i += S::kNT) {
            const int r = row0 + i % out_rows;
            if (r < a.rows)
                store_y(a.y, a.y_type, (int64_t)s_item[i / out_rows] * a.ldy + r, __builtin_nanf(""));
        }
        return;
    }

    // this thread's block of a step: row tid / 2 of the tile, block tid % 2
    const int ur = tid >> 1, ub = tid & 1;
    int wrow;
    if (a.swiglu)
        wrow = (ur < out_rows ? 0 : a.rows) + min(row0 + (ur & (out_rows - 1)), a.rows - 1);
    else
        wrow = min(row0 + ur, a.rows - 1);
    const uint8_t* W = a.W + group * a.estride;
    // and its activations: eight columns of kXL tokens
    const int xc = tid & 7, xt = tid >> 3;
    const XT* xp[S::kXL];
#pragma unroll
    for (int i = 0; i < S::kXL; ++i) {
        const int p = s_item[xt + S::kNT / 8 * i];
        xp[i] = static_cast<const XT*>(a.x) + (int64_t)(p / a.top_k) * a.xs_tok + (int64_t)(p % a.top_k) * a.xs_slot +
                8 * xc;
    }
    const bool vec = a.vec != 0;
    struct Stage {
        typename U::Raw w;
        X8<XT> x[S::kXL];
    };
    // Whole steps; a row of an odd number of blocks has half a step more.
    const int steps = a.nb / kTileBlks;
    auto load = [&](int s, Stage& g) __attribute__((always_inline)) {
        s = min(s, steps - 1);        // past the last: the last again, unused
        U::fetch(W, wrow, a.nb, kTileBlks * s + ub, g.w);
#pragma unroll
        for (int i = 0; i < S::kXL; ++i) g.x[i].load(xp[i] + 64 * s, vec);
    };
    auto put = [&](int s, int blk, bool live, const Stage& g) __attribute__((always_inline)) {
        uint8_t* buf = lds + (s & 1) * S::kBuf;
        uint32_t q[8];
        float sc[U::kSub], mu = 0.f;
        U::decode(g.w, blk, q, sc, mu);
        u32x4* w = reinterpret_cast<u32x4*>(buf + ur * kTilePitch + 64 * ub);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = u32x4{XOp<XT>::pair(sbyte(q[2 * i], 0), sbyte(q[2 * i], 1)),
                         XOp<XT>::pair(sbyte(q[2 * i], 2), sbyte(q[2 * i], 3)),
                         XOp<XT>::pair(sbyte(q[2 * i + 1], 0), sbyte(q[2 * i + 1], 1)),
                         XOp<XT>::pair(sbyte(q[2 * i + 1], 2), sbyte(q[2 * i + 1], 3))};
        float* sp = reinterpret_cast<float*>(buf + S::kW + S::kX);
#pragma unroll
        for (int h = 0; h < U::kSub; ++h) sp[(ub * U::kSub + h) * S::kTM + ur] = live ? sc[h] : 0.f;
        u32x4* mp = reinterpret_cast<u32x4*>(buf + S::kW + S::kX + S::kS);     // [block][rows], [block][tokens]
        if constexpr (U::kSums) mp[ub * S::kTM + ur] = min_operand<0>(live ? mu : 0.f);
#pragma unroll
        for (int i = 0; i < S::kXL; ++i) {
            const int tok = xt + S::kNT / 8 * i;
            u32x4 p[S::kP];
            g.x[i].pieces(p);
#pragma unroll
            for (int k = 0; k < S::kP; ++k)
                *reinterpret_cast<u32x4*>(buf + S::kW + (k * TN + tok) * kTilePitch + 16 * xc) = p[k];
            if constexpr (U::kSums) {
                float t = g.x[i].sum();      // of 8 columns; four lanes hold a block's 32
                t += dpp_mov<0xB1>(t);
                t += dpp_mov<0x4E>(t);
                if ((xc & 3) == 0) mp[kTileBlks * S::kTM + (xc >> 2) * TN + tok] = min_operand<1>(t);
            }
        }
    };

    const int wr = (wave / S::kWt) * 32 * S::kRS, wt = (wave % S::kWt) * 32 * S::kTS;
    const int lr = lane & 31, lh = lane >> 5;
    f32x16 acc[S::kRS][S::kTS];
#pragma unroll
    for (int r = 0; r < S::kRS; ++r)
#pragma unroll
        for (int t = 0; t < S::kTS; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[r][t][i] = 0.f;

    // The MFMAs of one 32 x 32 piece of a block go between the scalings of
    // the piece before it: a piece's results are 16 fused multiply-adds a
    // lane, about as long as its two MFMAs, and the two pipes then run side
    // by side with no more than two pieces' results live.  Operands are read
    // from LDS one piece (weights) or one block (activations) ahead.
    auto compute = [&](int s) __attribute__((always_inline)) {
        const uint8_t* buf = lds + (s & 1) * S::kBuf;
        const float* sp = reinterpret_cast<const float*>(buf + S::kW + S::kX) + wr + lr;
        const uint8_t* wp = buf + (wr + lr) * kTilePitch + 16 * lh;
        const uint8_t* xq0 = buf + S::kW + (wt + lr) * kTilePitch + 16 * lh;
        constexpr int kPer = S::kRS * S::kTS;          // pieces of a block
        constexpr int kPieces = kTileBlks * kPer;
        constexpr int kMf = 2 * S::kP;                 // MFMAs of a piece
        f32x16 dot[2][U::kSub];
        float d[2][U::kSub];
        u32x4 wq[2][2], xq[2][S::kP][S::kTS][2];
        auto read_w = [&](auto nc) __attribute__((always_inline)) {     // block and rows number nc
            constexpr int n = decltype(nc)::value, b = n / S::kRS, r = n % S::kRS;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wq[n & 1][h] = *reinterpret_cast<const u32x4*>(wp + 32 * r * kTilePitch + 64 * b + 32 * h);
#pragma unroll
            for (int h = 0; h < U::kSub; ++h) d[n & 1][h] = sp[(b * U::kSub + h) * S::kTM + 32 * r];
        };
        auto read_x = [&](auto bc) __attribute__((always_inline)) {
            constexpr int b = decltype(bc)::value;
#pragma unroll
            for (int k = 0; k < S::kP; ++k)
#pragma unroll
                for (int u = 0; u < S::kTS; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        xq[b & 1][k][u][h] =
                            *reinterpret_cast<const u32x4*>(xq0 + (k * TN + 32 * u) * kTilePitch + 64 * b + 32 * h);
        };
        read_x(std::integral_constant<int, 0>{});
        read_w(std::integral_constant<int, 0>{});
        float dp[U::kSub];                             // scales of the piece before
        static_for(std::make_integer_sequence<int, kPieces + 1>{}, [&](auto nc) __attribute__((always_inline)) {
            constexpr int n = decltype(nc)::value;
            constexpr int b = n / kPer, r = n / S::kTS % S::kRS, t = n % S::kTS, wn = n / S::kTS;
            constexpr int pn = n > 0 ? n - 1 : 0, pr = pn / S::kTS % S::kRS, pt = pn % S::kTS;
            if constexpr (n > 0) {
#pragma unroll
                for (int h = 0; h < U::kSub; ++h) dp[h] = d[(pn / S::kTS) & 1][h];
            }
            static_for(std::make_integer_sequence<int, kMf>{}, [&](auto mc) __attribute__((always_inline)) {
                constexpr int m = decltype(mc)::value;
                constexpr int h = m / S::kP, k = m % S::kP;
                if constexpr (n < kPieces) {
                    constexpr int o = U::kSub == 2 ? h : 0;
                    f32x16 c;
                    if constexpr (k == 0 && (U::kSub == 2 || h == 0)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) c[i] = 0.f;
                    } else {
                        c = dot[n & 1][o];
                    }
                    dot[n & 1][o] = XOp<XT>::mfma(xq[b & 1][k][t][h], wq[wn & 1][h], c);
                }
                if constexpr (n > 0) {
                    // the m-th share of the piece before
                    constexpr int all = 16 * U::kSub, i0 = all * m / kMf, i1 = all * (m + 1) / kMf;
#pragma unroll
                    for (int i = i0; i < i1; ++i)
                        acc[pr][pt][i & 15] = __builtin_fmaf(dp[i >> 4], dot[pn & 1][i >> 4][i & 15], acc[pr][pt][i & 15]);
                }
                // operands of the next rows and block, once the last piece
                // that reads their registers is past
                if constexpr (m == 0 && n < kPieces && t == 0 && wn + 1 < kTileBlks * S::kRS)
                    read_w(std::integral_constant<int, wn + 1>{});
                if constexpr (m == kMf - 1 && n < kPieces && r == 0 && t == 0 && b + 1 < kTileBlks)
                    read_x(std::integral_constant<int, b + 1>{});
                __builtin_amdgcn_sched_barrier(0x4 | 0x10);            // scalar and global memory may pass
            });
            // the scalings stay here (they are used a step later only)
            if constexpr (n > 0) asm volatile("" : "+v"(acc[pr][pt]));
        });
        if constexpr (U::kSums) {
            // mu times the block sums of x, both blocks of the step in one MFMA
            const u32x4* mp = reinterpret_cast<const u32x4*>(buf + S::kW + S::kX + S::kS);
            u32x4 mw[S::kRS], mx[S::kTS];
#pragma unroll
            for (int r = 0; r < S::kRS; ++r) mw[r] = mp[lh * S::kTM + wr + 32 * r + lr];
#pragma unroll
            for (int t = 0; t < S::kTS; ++t) mx[t] = mp[kTileBlks * S::kTM + lh * TN + wt + 32 * t + lr];
#pragma unroll
            for (int r = 0; r < S::kRS; ++r)
#pragma unroll
                for (int t = 0; t < S::kTS; ++t) acc[r][t] = XOp<__bf16>::mfma(mx[t], mw[r], acc[r][t]);
        }
    };

    // One barrier a step: the buffer of step s + 1 was last read in step
    // s - 1, before the barrier that ended it.  A step's loads are issued two
    // steps before they are put in LDS.
    if (steps > 0) {
        Stage g0, g1;
        load(0, g0);
        load(1, g1);
        put(0, ub, true, g0);
        load(2, g0);
        __syncthreads();
        for (int s = 0; s < steps; s += 2) {
            compute(s);
            put(s + 1, kTileBlks * (s + 1) + ub, true, g1);      // past the last step: not read
            load(s + 3, g1);
            __syncthreads();
            if (s + 1 >= steps) break;
            compute(s + 1);
            put(s + 2, kTileBlks * (s + 2) + ub, true, g0);
            load(s + 4, g0);
            __syncthreads();
        }
    }
    if (a.nb % kTileBlks) {
        // the last block; activations and scales past the row are 0
        Stage g;
        U::fetch(W, wrow, a.nb, a.nb - 1, g.w);
#pragma unroll
        for (int i = 0; i < S::kXL; ++i) {
            if (xc < 4)
                g.x[i].load(xp[i] + 64 * steps, vec);
            else
                g.x[i].zero();
        }
        __syncthreads();
        put(steps, a.nb - 1, ub == 0, g);
        __syncthreads();
        compute(steps);
        __syncthreads();
    }

    // results through LDS, so that stores run along the rows
    float* out = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int r = 0; r < S::kRS; ++r)
#pragma unroll
        for (int t = 0; t < S::kTS; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                out[(wt + 32 * t + 8 * (i >> 2) + 4 * lh + (i & 3)) * S::kOutPitch + wr + 32 * r + lr] = acc[r][t][i];
    __syncthreads();
    for (int i = tid; i < count * out_rows; i += S::kNT) {
        const int j = i / out_rows, r = i % out_rows;
        if (row0 + r >= a.rows) continue;
        float v = out[j * S::kOutPitch + r];
        if (a.swiglu) v = silu(v) * out[j * S::kOutPitch + out_rows + r];
        store_y(a.y, a.y_type, (int64_t)s_item[j] * a.ldy + row0 + r, v);
    }
}

template <class F, class XT, int TN>
int32_t launch_tile(const TileCall& c, int plan_tile, hipStream_t st) {
    using S = TileShape<F, XT, TN>;
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
    const int64_t tiles = c.plan ? plan_tile_bound(c.n_items, c.n_groups, plan_tile) * (plan_tile / TN)
                                 : (c.n_items + TN - 1) / TN;
    if (tiles * d.row_tiles > 0x7fffffff)
        return fail(QMV_EINVAL, "qmv: %lld tiles exceed a launch", (long long)(tiles * d.row_tiles));
    auto kern = tile_kernel<F, XT, TN>;
    size_t dyn_max = 0;
    if (const int32_t e = lds_limit(reinterpret_cast<const void*>(kern), kLdsMax, "qmv", &dyn_max)) return e;
    if ((size_t)S::kLds > dyn_max) return fail(QMV_EHIP, "qmv: the tile kernel's LDS exceeds the device's");
    hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * d.row_tiles)), dim3(S::kNT), S::kLds, st, d);
    return check_launch("qmv");
}

// fp32 activations take three times the LDS and MFMAs: 64 tokens by 256 rows
// where 16-bit ones take 128 by 128.
template <class F, class XT>
int32_t launch_tile_n(const TileCall& c, hipStream_t st) {
    const int tile = c.plan ? plan_tile(c.n_items, c.n_groups) : plan_tile(c.n_items, 1);
    if (tile == 32) return launch_tile<F, XT, 32>(c, 32, st);
    if constexpr (std::is_same<XT, float>::value)
        return launch_tile<F, XT, 64>(c, tile, st);
    else
        return launch_tile<F, XT, 128>(c, tile, st);
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
