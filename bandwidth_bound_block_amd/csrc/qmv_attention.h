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
// order as long as both operands have the same.  fp32 queries, weights and
// values are pairs of fp16 pieces.
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

#include "qmv_block_decode.h"
#include "qmv_cache.h"

namespace qmv {

constexpr int kAWaves = 4, kAT = 64 * kAWaves;
constexpr int kAShares = 1024;      // workgroups of the streaming kernel at most
constexpr int kAMinBlocks = 8;      // blocks of 32 keys of a share at least
constexpr int kABlock = 32;

struct AttnArgs {
    CacheSide k, v;
    int64_t n_pages;
    int32_t page_shift, H, G, R;
    const void* q;
    int64_t qst, qsh;
    bool qvec;
    int64_t n_tokens, max_q;
    const int32_t* table;
    int64_t max_pages;
    const int32_t* lens;
    const int32_t* q_begin;
    float scale;                    // times log2(e)
    int32_t window;
    const float* sinks;
    void* out;
    int32_t x_type;
    // workspace of the streaming kernel
    int64_t* prefix;                // [R + 1]: blocks of all units before request r's; [R + 1]: a share's blocks
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

namespace {

constexpr float kANone = -1e30f;    // the maximum of no score

struct Req {
    int64_t q0;                     // first query token
    int n, len;                     // query tokens, keys
    int lo, blk0, nblk;             // first key seen, first block, blocks of a unit
    int tiles;                      // tiles of rows
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
    o.len = o.bad ? 0 : len;
    o.lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)o.len - o.n - a.window + 1) : 0;
    o.blk0 = o.lo / kABlock;
    o.nblk = max(1, (int)(((int64_t)o.len + kABlock - 1) / kABlock) - o.blk0);
    o.tiles = (int)(((int64_t)o.n * a.G + 16 * NT - 1) / (16 * NT));     // n_tokens * G < 2^31
    return o;
}

// Sum over the waves of a workgroup; every thread gets it.
__device__ __forceinline__ int64_t group_sum64(int64_t v, int64_t* lds) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    int64_t s = 0;
    for (int w = 0; w < kAWaves; ++w) s += lds[w];
    return s;
}

// max over the four lane groups that hold a query
__device__ __forceinline__ float groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float groups_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ float load_q(const void* p, int32_t type, int64_t i) {
    return type == QMV_X_F32   ? static_cast<const float*>(p)[i]
           : type == QMV_X_F16 ? (float)static_cast<const _Float16*>(p)[i]
                               : XIn<__bf16>::load1(static_cast<const __bf16*>(p) + i);
}
__device__ __forceinline__ void load_q8(const AttnArgs& a, int64_t i, float (&w)[8]) {
    if (a.qvec) {
        if (a.x_type == QMV_X_F32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + i);
            const float4 x = p[0], y = p[1];
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w; w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + i);
            const uint32_t s[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (a.x_type == QMV_X_F16) {
                    w[2 * j] = half_bits_to_float(s[j]);
                    w[2 * j + 1] = half_bits_to_float(s[j] >> 16);
                } else {
                    w[2 * j] = __builtin_bit_cast(float, s[j] << 16);
                    w[2 * j + 1] = __builtin_bit_cast(float, s[j] & 0xffff0000u);
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = load_q(a.q, a.x_type, i + j);
    }
}
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t i, float x) {
    if (a.x_type == QMV_X_F32) static_cast<float*>(a.out)[i] = x;
    else if (a.x_type == QMV_X_F16) static_cast<_Float16*>(a.out)[i] = (_Float16)x;
    else static_cast<__bf16*>(a.out)[i] = (__bf16)x;
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

// A row's power of two: |q| 2^shift < 2^15 throughout (0 for fp16 queries).
// At most 2^60: scores of smaller rows are 0 to fp32 beside any others.
__device__ __forceinline__ int row_shift(float amax, int32_t type) {
    if (type == QMV_X_F16 || !(amax > 0.f)) return 0;
    return min(14 - (int)((__builtin_bit_cast(uint32_t, amax) >> 23) & 255) + 127, 60);
}

// Loads of one lane for 32 keys: two tiles of 16.
template <int F, int N> struct Codes;    // N octets
template <int N> struct Codes<QMV_Q8_0, N> { uint2 w[N]; };
template <int N> struct Codes<QMV_Q4_0, N> { uint32_t w[N]; };
template <int N> struct Codes<QMV_Q4_1, N> { uint32_t w[N]; };

template <int KF, int VF, int NB>
struct Raw {
    static constexpr int kVW = VF == QMV_Q8_0 ? NB / 2 : NB >= 4 ? NB / 4 : 1;    // words of V a key
    static constexpr int kVB = NB == 8 ? 2 : 1;                                    // blocks of V a lane has
    Codes<KF, NB> k[2];
    uint2 ks[2][NB], km[2][KF == QMV_Q4_1 ? NB : 1];
    uint32_t v[8][kVW];
    uint2 vs[2][kVB], vm[2][VF == QMV_Q4_1 ? kVB : 1];
};

template <int F> constexpr int row_bytes_of(int D) { return F == QMV_Q8_0 ? D : D / 2; }

// One of the eight fp16 values that an octet of codes stands for, of two
// neighbouring keys side by side.
template <int F>
__device__ __forceinline__ f16x2 scaled(f16x2 c, f16x2 d, f16x2 m) {
    if constexpr (F == QMV_Q4_1) return __builtin_elementwise_fma(c, d, m);
    else return c * d;
}
// What scaled() leaves, as a second fp16 piece.  c d is exact in two pieces;
// with a minimum, the error of the sum of its first piece and m as well (the
// six steps are exact).
template <int F>
__device__ __forceinline__ f16x2 scaled_rest(f16x2 c, f16x2 d, f16x2 m, f16x2& first) {
#pragma clang fp contract(off)
    if constexpr (F == QMV_Q4_1) {      // fused into other multiply-adds these steps would not be exact
        const f16x2 p = c * d, e = __builtin_elementwise_fma(c, d, -p);
        const f16x2 s = p + m, z = s - p;
        const f16x2 rest = (p - (s - z)) + (m - z) + e;
        first = s;
        return rest;
    } else {
        first = c * d;
        return __builtin_elementwise_fma(c, d, -first);
    }
}

__device__ __forceinline__ f16x8 pack8(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int KF, int VF, int P, int NB, int NT>
__global__ __launch_bounds__(kAT) void attn_stream_kernel(const AttnArgs a) {
    constexpr int D = 32 * NB, NV = D / 16;             // NV: tiles of 16 places of the head
    constexpr int kRows = 16 * NT;
    constexpr int kKRow = row_bytes_of<KF>(D), kVRow = row_bytes_of<VF>(D);
    typedef Raw<KF, VF, NB> RawT;
    __shared__ int64_t s_scan[kAWaves];
    __shared__ int64_t s_at[4];
    __shared__ __align__(16) float s_o[kAWaves][kRows][68];
    __shared__ float s_m[kAWaves][kRows], s_l[kAWaves][kRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n16 = lane & 15, g = lane >> 4;
    const float inf = __builtin_inff();

    // ---- the share: blocks [pos, end) of all units' in a row
    int64_t total = 0;
    for (int r0 = 0; r0 < a.R; r0 += kAT) {
        int64_t mine = 0;
        if (r0 + tid < a.R) {
            const Req q = request<NT>(a, r0 + tid);
            mine = (int64_t)q.nblk * q.tiles * a.H;
        }
        total += group_sum64(mine, s_scan);
    }
    const int64_t share = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kAMinBlocks);
    int64_t pos = blockIdx.x * share;
    const int64_t end = min(pos + share, total);
    if (blockIdx.x != 0 && pos >= end) return;
    // the request that holds pos, and for the second launch where each begins
    {
        int64_t before = 0;
        if (tid < 4) s_at[tid] = -1;
        for (int r0 = 0; r0 < a.R; r0 += kAT) {
            int64_t mine = 0;
            if (r0 + tid < a.R) {
                const Req q = request<NT>(a, r0 + tid);
                mine = (int64_t)q.nblk * q.tiles * a.H;
            }
            int64_t at = mine;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int64_t t = __shfl_up(at, o);
                if (lane >= o) at += t;
            }
            __syncthreads();
            if (lane == 63) s_scan[wave] = at;
            __syncthreads();
            int64_t off = before;
            for (int w = 0; w < kAWaves; ++w) {
                if (w < wave) off += s_scan[w];
                before += s_scan[w];
            }
            const int64_t first = off + at - mine;
            if (r0 + tid < a.R) {
                if (blockIdx.x == 0) a.prefix[r0 + tid] = first;
                if (mine > 0 && pos >= first && pos < first + mine) {
                    s_at[0] = r0 + tid;
                    s_at[1] = first;
                }
            }
            if (blockIdx.x != 0 && before > pos) break;
        }
        if (blockIdx.x == 0 && tid == 0) {
            a.prefix[a.R] = total;
            a.prefix[a.R + 1] = share;
        }
        __syncthreads();
    }
    int r = (int)s_at[0];
    int64_t first = s_at[1];        // of request r's units
    bool tail = true;               // the share's first segment

    while (pos < end) {
        const Req rq = request<NT>(a, r);
        const int64_t mine = (int64_t)rq.nblk * rq.tiles * a.H;
        if (pos >= first + mine) {  // the next request (those without queries have no blocks)
            first += mine;
            ++r;
            continue;
        }
        const int64_t unit = (pos - first) / rq.nblk;
        const int tile = (int)(unit % rq.tiles), h = (int)(unit / rq.tiles);
        const int64_t ubase = first + unit * rq.nblk;
        const int b0 = (int)(pos - ubase);
        const int b1 = (int)(min(end - ubase, (int64_t)rq.nblk));
        const bool whole = b0 == 0 && b1 == rq.nblk;

        // ---- queries: B operand, lane n16 = row, places 32 b + 8 g .. + 7
        f16x8 qh[NT][NB], ql[P == 2 ? NT : 1][P == 2 ? NB : 1];
        float qsum[NT][NB], fac[NT];
        int qpos[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const unsigned row = tile * kRows + 16 * nt + n16;
            const bool have = row < (unsigned)(rq.n * a.G);
            const int i = have ? row / (unsigned)a.G : 0, hq = h * a.G + (have ? row - i * a.G : 0);
            const int64_t base = (rq.q0 + i) * a.qst + hq * a.qsh;
            float w[NB][8], amax = 0.f;
            bool fin = true;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                load_q8(a, base + 32 * b + 8 * g, w[b]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    amax = fmaxf(amax, __builtin_fabsf(w[b][j]));
                    fin &= __builtin_fabsf(w[b][j]) < inf;
                }
            }
            amax = groups_max(amax);
            const int sh = row_shift(amax, a.x_type);
            fac[nt] = fmaxf(__builtin_ldexpf(a.scale, -sh), 1e-37f);      // not 0: what is out of sight is -inf times it
            if (groups_max(fin ? 0.f : 1.f) != 0.f) fac[nt] = __builtin_nanf("");
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = __builtin_ldexpf(w[b][j], sh);
                    const _Float16 hi = (_Float16)x;
                    qh[nt][b][j] = hi;
                    s += (float)hi;
                    if constexpr (P == 2) {
                        const _Float16 lo = (_Float16)(x - (float)hi);
                        ql[nt][b][j] = lo;
                        s += (float)lo;
                    }
                }
                qsum[nt][b] = KF == QMV_Q4_1 ? groups_sum(s) : 0.f;
            }
            qpos[nt] = have ? rq.len - rq.n + i : -1;    // -1: sees nothing
        }

        // ---- this wave's blocks
        const int per = (b1 - b0 + kAWaves - 1) / kAWaves;
        const int w0 = __builtin_amdgcn_readfirstlane(min(b0 + wave * per, b1));
        const int w1 = __builtin_amdgcn_readfirstlane(min(w0 + per, b1));
        const int32_t* table = a.table + (int64_t)r * a.max_pages;
        const int full_to = rq.len - rq.n + 1;                       // keys before it are seen by every query
        const int full_from = a.window > 0 ? max(0, rq.len - a.window) : 0;    // from it on, too
        float m[NT], l[NT];
        f32x4 o[NT][NV];
        f32x4 poison[NT][RawT::kVB];
        bool careful = false;
        for (;;) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt] = kANone;
                l[nt] = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) o[nt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < RawT::kVB; ++v) poison[nt][v] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            int entries = 0;
            const auto refill = [&](int blk) {       // pages of the 64 tiles from block blk on; -1: absent, -2: out of range
                const int s = (rq.blk0 + blk) * kABlock + 16 * lane;
                int e = -1;
                if (s < rq.len && s + 16 > rq.lo && blk + lane / 2 < w1) {
                    e = table[s >> a.page_shift];
                    if (e < 0 || e >= a.n_pages) e = -2;
                }
                entries = e;
            };
            const auto load = [&](int blk, RawT& w) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int e = max(__builtin_amdgcn_readlane(entries, (2 * (blk - w0) + t) & 63), 0);
                    const int key0 = (rq.blk0 + blk) * kABlock + 16 * t;
                    const int off = key0 & ((1 << a.page_shift) - 1);
                    const uint8_t* kp = a.k.pages + e * a.k.page_bytes + h * a.k.head_bytes;
                    const uint8_t* vp = a.v.pages + e * a.v.page_bytes + h * a.v.head_bytes;
                    const uint8_t* kc = kp + (off + n16) * kKRow + g * (kKRow / 4);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if constexpr (KF == QMV_Q8_0) w.k[t].w[b] = reinterpret_cast<const uint2*>(kc)[b];
                        else w.k[t].w[b] = reinterpret_cast<const uint32_t*>(kc)[b];
                    }
                    const uint8_t* ks = kp + ((int64_t)kKRow << a.page_shift) + 2 * (off + 4 * g);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        w.ks[t][b] = *reinterpret_cast<const uint2*>(ks + ((int64_t)(2 * b) << a.page_shift));
                        if constexpr (KF == QMV_Q4_1)
                            w.km[t][b] = *reinterpret_cast<const uint2*>(ks + ((int64_t)(2 * (NB + b)) << a.page_shift));
                    }
                    const uint8_t* vc = vp + (off + 4 * g) * kVRow + n16 * (kVRow / 16);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < RawT::kVW; ++j) {
                            if constexpr (VF != QMV_Q8_0 && NB == 2)
                                w.v[4 * t + i][j] = *reinterpret_cast<const uint16_t*>(vc + i * kVRow);
                            else
                                w.v[4 * t + i][j] = reinterpret_cast<const uint32_t*>(vc + i * kVRow)[j];
                        }
                    // the block (or two) of this lane's places
                    const int vb = NB == 4 ? n16 & 3 : NB == 2 ? (n16 >> 1) & 1 : 2 * (n16 & 3);
                    const uint8_t* vs = vp + ((int64_t)kVRow << a.page_shift) + 2 * (off + 4 * g);
#pragma unroll
                    for (int j = 0; j < RawT::kVB; ++j) {
                        w.vs[t][j] = *reinterpret_cast<const uint2*>(vs + ((int64_t)(2 * (vb + j)) << a.page_shift));
                        if constexpr (VF == QMV_Q4_1)
                            w.vm[t][j] = *reinterpret_cast<const uint2*>(vs + ((int64_t)(2 * (NB + vb + j)) << a.page_shift));
                    }
                }
            };
            const auto compute = [&](int blk, const RawT& w) {
                const int key0 = (rq.blk0 + blk) * kABlock;
                const int e0 = __builtin_amdgcn_readlane(entries, (2 * (blk - w0)) & 63);
                const int e1 = __builtin_amdgcn_readlane(entries, (2 * (blk - w0) + 1) & 63);
                const bool plain = key0 + 32 <= full_to && key0 >= full_from && e0 >= 0 && e1 >= 0 && !careful;
                // scores: rows of the result are keys 4 g + r of tile t
                f32x4 s[NT][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        f16x8 c;
                        if constexpr (KF == QMV_Q8_0) {
                            const uint32_t x = w.k[t].w[b].x ^ 0x80808080u, y = w.k[t].w[b].y ^ 0x80808080u;
                            c = pack8(byte_pair<0, 1>(x, y), byte_pair<2, 3>(x, y), byte_pair<4, 5>(x, y), byte_pair<6, 7>(x, y));
                        } else {
                            constexpr float bias = KF == QMV_Q4_0 ? 8.f : 0.f;
                            const uint32_t x = w.k[t].w[b];
                            c = pack8(nibble_pair(x, 0, bias), nibble_pair(x, 1, bias), nibble_pair(x, 2, bias),
                                      nibble_pair(x, 3, bias));
                        }
                        const f16x2 d0 = as_h2(w.ks[t][b].x), d1 = as_h2(w.ks[t][b].y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
                            if constexpr (P == 2) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(c, ql[nt][b], z, 0, 0, 0);
                            z = __builtin_amdgcn_mfma_f32_16x16x32_f16(c, qh[nt][b], z, 0, 0, 0);
                            f32x4& y = s[nt][t];
                            y[0] = __builtin_fmaf((float)d0[0], z[0], y[0]);
                            y[1] = __builtin_fmaf((float)d0[1], z[1], y[1]);
                            y[2] = __builtin_fmaf((float)d1[0], z[2], y[2]);
                            y[3] = __builtin_fmaf((float)d1[1], z[3], y[3]);
                            if constexpr (KF == QMV_Q4_1) {
                                const f16x2 m0 = as_h2(w.km[t][b].x), m1 = as_h2(w.km[t][b].y);
                                y[0] = __builtin_fmaf((float)m0[0], qsum[nt][b], y[0]);
                                y[1] = __builtin_fmaf((float)m0[1], qsum[nt][b], y[1]);
                                y[2] = __builtin_fmaf((float)m1[0], qsum[nt][b], y[2]);
                                y[3] = __builtin_fmaf((float)m1[1], qsum[nt][b], y[3]);
                            }
                        }
                    }
                }
                f16x2 vd[4][RawT::kVB], vm[4][RawT::kVB];      // pairs of keys 2 j, 2 j + 1
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < RawT::kVB; ++k) {
                        vd[j][k] = as_h2(j & 1 ? w.vs[j / 2][k].y : w.vs[j / 2][k].x);
                        if constexpr (VF == QMV_Q4_1) vm[j][k] = as_h2(j & 1 ? w.vm[j / 2][k].y : w.vm[j / 2][k].x);
                        else vm[j][k] = h2(0.f);
                    }
                if (!plain) {
                    // keys out of a query's sight, absent keys (their bytes are any) and pages out of range
                    f16x8 sick[RawT::kVB];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 16 * t + 4 * g + i, e = t ? e1 : e0;
                            const bool there = e >= 0 && key < rq.len;
                            const int j = 2 * t + i / 2;
#pragma unroll
                            for (int k = 0; k < RawT::kVB; ++k) {
                                const bool odd = there && !(__builtin_fabsf((float)vd[j][k][i & 1]) < inf &&
                                                            __builtin_fabsf((float)vm[j][k][i & 1]) < inf);
                                sick[k][4 * t + i] = odd ? (_Float16)1.f : (_Float16)0.f;
                                if (!there || (careful && odd)) {
                                    vd[j][k][i & 1] = (_Float16)0.f;
                                    vm[j][k][i & 1] = (_Float16)0.f;
                                }
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const bool seen = key <= qpos[nt] && (a.window <= 0 || key > qpos[nt] - a.window);
                                s[nt][t][i] = seen ? (e == -2 ? __builtin_nanf("") : s[nt][t][i]) : -inf;
                            }
                        }
                    if (careful) {      // which rows see a value that is not finite, block by block
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            f16x8 sees;
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int key = key0 + 16 * t + 4 * g + i;
                                    sees[4 * t + i] = key <= qpos[nt] && (a.window <= 0 || key > qpos[nt] - a.window)
                                                          ? (_Float16)1.f : (_Float16)0.f;
                                }
#pragma unroll
                            for (int k = 0; k < RawT::kVB; ++k)
                                poison[nt][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(sick[k], sees, poison[nt][k], 0, 0, 0);
                        }
                    }
                }
                // softmax: running maximum and sum, in units of log 2
                f16x8 ph[NT], pl[P == 2 ? NT : 1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float top = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                                      fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
                    top = fmaxf(groups_max(top * fac[nt]), m[nt]);
                    if (__any(top > m[nt])) {
                        const float f = __builtin_amdgcn_exp2f(m[nt] - top);
                        l[nt] *= f;
#pragma unroll
                        for (int v = 0; v < NV; ++v) o[nt][v] *= f;
                        m[nt] = top;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][t][i], fac[nt], -m[nt]));
                            l[nt] += p;
                            const _Float16 hi = (_Float16)p;
                            ph[nt][4 * t + i] = hi;
                            if constexpr (P == 2) pl[nt][4 * t + i] = (_Float16)(p - (float)hi);
                        }
                }
                // values: tile v of the result's places, keys in the order of the weights
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    f16x2 c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (VF == QMV_Q8_0) {
                            const uint32_t x = w.v[2 * j][v / 4] ^ 0x80808080u, y = w.v[2 * j + 1][v / 4] ^ 0x80808080u;
                            c[j] = v % 4 == 0 ? byte_pair<0, 4>(x, y) : v % 4 == 1 ? byte_pair<1, 5>(x, y)
                                   : v % 4 == 2 ? byte_pair<2, 6>(x, y) : byte_pair<3, 7>(x, y);
                        } else {
                            constexpr float bias = VF == QMV_Q4_0 ? 8.f : 0.f;
                            // halves of the two keys' words side by side; value 2 e is nibble e of the low half, 2 e + 1 of the
                            // high one; a lane that has half an octet (NB 2) has four nibbles
                            const int wd = NB == 8 ? v / 8 : 0, u = v % 8;
                            const uint32_t x = w.v[2 * j][wd], y = w.v[2 * j + 1][wd];
                            if constexpr (NB == 2) c[j] = nibble_pair(x | y << 16, u, bias);
                            else c[j] = nibble_pair(__builtin_amdgcn_perm(y, x, u & 1 ? 0x07060302u : 0x05040100u), u >> 1, bias);
                        }
                    }
                    const int k = RawT::kVB == 2 ? v / 8 : 0;
                    f16x2 first[4], rest[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (P == 2) rest[j] = scaled_rest<VF>(c[j], vd[j][k], vm[j][k], first[j]);
                        else first[j] = scaled<VF>(c[j], vd[j][k], vm[j][k]);
                    }
                    const f16x8 vh = pack8(first[0], first[1], first[2], first[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (P == 2) {
                            const f16x8 vl = pack8(rest[0], rest[1], rest[2], rest[3]);
                            o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl, ph[nt], o[nt][v], 0, 0, 0);
                            o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, pl[nt], o[nt][v], 0, 0, 0);
                        }
                        o[nt][v] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, ph[nt], o[nt][v], 0, 0, 0);
                    }
                }
            };
            for (int c0 = w0; c0 < w1; c0 += 32) {
                refill(c0);
                const int c1 = min(c0 + 32, w1);
                RawT x, y;
                load(c0, x);
                for (int blk = c0; blk < c1; blk += 2) {
                    load(min(blk + 1, c1 - 1), y);
                    compute(blk, x);
                    if (blk + 1 < c1) {
                        load(min(blk + 2, c1 - 1), x);
                        compute(blk + 1, y);
                    }
                }
            }
            if (careful) break;
            bool odd = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i) odd |= !(__builtin_fabsf(o[nt][v][i]) < inf);
            // 0 times a value that is not finite, of a key that a row does not see: again, with such values by themselves
            if (!__any(odd)) break;
            careful = true;
        }
        if (careful) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (poison[nt][RawT::kVB == 2 ? v / 8 : 0][i] > 0.f) o[nt][v][i] = __builtin_nanf("");
        }

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
                const unsigned row = tile * kRows + n;
                if (row >= (unsigned)(rq.n * a.G)) continue;
                f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
                float mm = fmaxf(fmaxf(s_m[0][n], s_m[1][n]), fmaxf(s_m[2][n], s_m[3][n])), ll = 0.f;
#pragma unroll
                for (int w = 0; w < kAWaves; ++w) {
                    x += *reinterpret_cast<const f32x4*>(&s_o[w][n][c]);
                    ll += s_l[w][n] * __builtin_amdgcn_exp2f(s_m[w][n] - mm);
                }
                if (whole) {
                    const unsigned i = row / (unsigned)a.G;
                    const int hq = h * a.G + (int)(row - i * a.G);
                    if (a.sinks) {
                        const float sk = a.sinks[hq] * 1.44269504088896341f, top = fmaxf(mm, sk);
                        const float f = __builtin_amdgcn_exp2f(mm - top);
                        x *= f;
                        ll = ll * f + __builtin_amdgcn_exp2f(sk - top);
                    }
                    const float inv = 1.f / ll;
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = rq.bad ? __builtin_nanf("") : ll == 0.f ? 0.f : x[k] * inv;
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
        pos += b1 - b0;
    }
}

// The parts of the units that no single workgroup had: a workgroup per
// (request, head, tile).
template <int D, int NT>
__global__ __launch_bounds__(kAT) void attn_join_kernel(const AttnArgs a, int shares) {
    constexpr int kRows = 16 * NT;
    const int r = blockIdx.y;
    const Req rq = request<NT>(a, r);
    const int64_t share = a.prefix[a.R + 1], first = a.prefix[r];
    for (int64_t unit = blockIdx.x; unit < (int64_t)rq.tiles * a.H; unit += gridDim.x) {
        const int64_t u0 = first + unit * rq.nblk, u1 = u0 + rq.nblk;
        const int64_t s0 = u0 / share, s1 = (u1 - 1) / share;
        if (s0 == s1) continue;
        const int tile = (int)(unit % rq.tiles), h = (int)(unit / rq.tiles);
        const int64_t slots = 2 * (int64_t)shares;
        const float* pm = a.part + slots * kRows * D;
        const float* pl = pm + slots * kRows;
        constexpr int kCols = D / 4, kPer = kAT / kCols;      // rows at a time
        for (int n = threadIdx.x / kCols; n < kRows; n += kPer) {
            const unsigned row = tile * kRows + n;
            if (row >= (unsigned)(rq.n * a.G)) break;
            const int c = 4 * (threadIdx.x % kCols);
            float m = kANone;
            // the unit's first part is its workgroup's last unless it begins the share
            const auto slot_of = [&](int64_t s) { return 2 * s + (s == s0 && u0 != s * share ? 1 : 0); };
            for (int64_t s = s0; s <= s1; ++s) m = fmaxf(m, pm[slot_of(s) * kRows + n]);
            f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
            float l = 0.f;
            for (int64_t s = s0; s <= s1; ++s) {
                const int64_t at = slot_of(s) * kRows + n;
                const float f = __builtin_amdgcn_exp2f(pm[at] - m);
                l += pl[at] * f;
                x += *reinterpret_cast<const f32x4*>(a.part + at * D + c) * f;
            }
            const unsigned i = row / (unsigned)a.G;
            const int hq = h * a.G + (int)(row - i * a.G);
            if (a.sinks) {
                const float sk = a.sinks[hq] * 1.44269504088896341f, top = fmaxf(m, sk);
                const float f = __builtin_amdgcn_exp2f(m - top);
                x *= f;
                l = l * f + __builtin_amdgcn_exp2f(sk - top);
            }
            const float inv = 1.f / l;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = rq.bad ? __builtin_nanf("") : l == 0.f ? 0.f : x[k] * inv;
            store_out4(a, ((rq.q0 + i) * a.H * a.G + hq) * D + c, x);
        }
    }
}

template <int KF, int VF, int P, int NB, int NT>
int32_t launch_stream_n(const AttnArgs& a, hipStream_t st) {
    const char* name = "qmv_cache_attention";
    hipLaunchKernelGGL((attn_stream_kernel<KF, VF, P, NB, NT>), dim3(kAShares), dim3(kAT), 0, st, a);
    if (const int32_t e = check_launch(name)) return e;
    const int64_t units = (int64_t)a.H * ((a.max_q * a.G + 16 * NT - 1) / (16 * NT));
    const unsigned x = (unsigned)std::min<int64_t>(units, std::max<int64_t>(1, 65536 / a.R));
    hipLaunchKernelGGL((attn_join_kernel<32 * NB, NT>), dim3(x, a.R), dim3(kAT), 0, st, a, kAShares);
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
