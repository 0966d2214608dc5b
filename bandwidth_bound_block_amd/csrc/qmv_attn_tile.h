// The kernel for many rows of queries: pieces of prompts.
//
// A workgroup has 32 rows of queries a wave (row = query token times G + head
// of the group) and one key/value head, and goes over the keys KT at a time.
// It makes fp16 values of the codes once for all its rows and lays them in
// LDS, keys as rows, values transposed, each in the order that the matrix
// cores take them: v_mfma_f32_32x32x16_f16 gives a lane, for one query, the
// keys 8 j + 4 h + r (h = lane / 32, j, r < 4) of 32, and the second product
// takes them from there as its operand, so the values' rows are in that order.
//
// The waves are two groups, one of each on every SIMD, half a step apart:
// while one group multiplies (weights by values of a step, then queries by
// keys of the next), the other does its softmax and turns codes into values,
// the first group the keys', the second the values'.  All waves in step left
// the matrix and the vector pipes waiting for each other: 458 us against 386
// for 2048 bf16 queries behind 6144 keys, 32 heads of 128, Q4_0.  That is
// 622 TF/s (327 us, 735, where calls follow each other); what bounds it is the
// vector work beside the products (exponentials and their scales, codes to
// values), about as long as they are.  Codes are on their way two phases before
// they are used.  fp16 and fp32 queries (P 2) take three products for one,
// 720..790 us.  Few tiles are split over the keys and joined by a second launch.
#pragma once
#include "qmv_attention.h"

namespace qmv {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D, int P>
struct Tile {
    static constexpr int kWaves = D * P <= 256 ? 8 : 4, kThreads = 64 * kWaves, kGroup = kThreads / 2, kRows = 32 * kWaves;
    static constexpr int NB = D / 32;
    static constexpr int KT = D * P <= 128 ? 64 : 32;           // keys of a step
    static constexpr int kSubs = KT / 16;
    // bytes of a row in LDS, a key's places or a place's keys: 16 rows at any of their 16-byte chunks meet all banks once
    static constexpr int kKRow = 2 * D + 16, kVRow = 2 * KT + 16;
    static constexpr int kKBytes = KT * kKRow, kVBytes = D * kVRow;
    static constexpr int kBuf = P * (kKBytes + kVBytes);
    static constexpr int kVItems = (D / 8) * (KT / 4);          // (octet, four keys)
};

// What one thread has of a step: of keys 16-byte chunks of codes, of values
// four keys' octets, with their scales and minimums.
template <int D, int P, bool W8>
struct RawK {
    static constexpr int kRow = W8 ? D : D / 2, kC = kRow / 16, kOct = W8 ? 2 : 4;      // chunks of a row, octets of a chunk
    static constexpr int kAll = Tile<D, P>::KT * kC, N = (kAll + Tile<D, P>::kGroup - 1) / Tile<D, P>::kGroup;
    u32x4 w[N];
    uint32_t d[N][kOct], m[N][kOct];
};
template <int D, int P, bool W8>
struct RawV {
    static constexpr int kRow = W8 ? D : D / 2, N = (Tile<D, P>::kVItems + Tile<D, P>::kGroup - 1) / Tile<D, P>::kGroup;
    uint32_t w[N][4][W8 ? 2 : 1];
    uint2 d[N], m[N];
    int there[N];
};

template <int D, int P>
struct TileStep {
    typedef Tile<D, P> T;
    static constexpr int NB = T::NB, kVItems = T::kVItems;
    // Entry of tile `sub` (below kSubs, of the lane) of the step whose first tile is sub0.
    __device__ static int entry(int entries, int sub0, int sub) {
        int e = __builtin_amdgcn_readlane(entries, sub0);
#pragma unroll
        for (int i = 1; i < T::kSubs; ++i) {
            const int x = __builtin_amdgcn_readlane(entries, sub0 + i);
            e = sub == i ? x : e;
        }
        return e;
    }
    // K: chunks of 16 bytes of the step's codes, KT * (row / 16) of them over the group's threads (t: thread of the group);
    // neighbouring lanes have neighbouring keys, whose rows in LDS lie over all banks.
    template <int C>
    __device__ static void k_place(int t, int n, int& key, int& q) {
        constexpr int kPer = 64 / C;        // keys of a wave's chunks
        const int lane = t & 63, w = (t >> 6) + n * (T::kGroup / 64);
        key = w * kPer + lane % kPer;
        q = lane / kPer;
    }
    // minimums: the plane offset of the minimums, 0 without them (the scales are read in their place)
    template <bool W8>
    __device__ static void load(const uint8_t* base, int64_t page_bytes, int page_shift, uint32_t minimums, int t, int entries, int sub0,
                                int key0, int, RawK<D, P, W8>& w) {
        typedef RawK<D, P, W8> R;
#pragma unroll
        for (int n = 0; n < R::N; ++n) {
            int key, q;
            k_place<R::kC>(t, n, key, q);
            if (R::kAll < T::kGroup) key &= T::KT - 1;      // threads past the last do the first's again
            const int e = max(entry(entries, sub0, key >> 4), 0);
            const uint32_t off = (key0 + key) & ((1 << page_shift) - 1);
            const uint8_t* p = base + e * page_bytes;
            w.w[n] = *reinterpret_cast<const u32x4*>(p + (off * R::kRow + 16 * q));
            const uint32_t s = ((R::kRow + 2 * (R::kOct * q % NB)) << page_shift) + 2 * off;
#pragma unroll
            for (int i = 0; i < R::kOct; ++i) {
                if (i >= NB) {                              // two blocks: the others are these
                    w.d[n][i] = w.d[n][i % NB];
                    w.m[n][i] = w.m[n][i % NB];
                    continue;
                }
                w.d[n][i] = *reinterpret_cast<const uint16_t*>(p + (s + (uint32_t(2 * i) << page_shift)));
                if constexpr (!W8) w.m[n][i] = *reinterpret_cast<const uint16_t*>(p + (s + (uint32_t(2 * i) << page_shift) + minimums));
                else w.m[n][i] = 0;
            }
        }
    }
    template <bool W8, bool CARE>
    __device__ static void store(int t, uint8_t* buf, bool mins, const RawK<D, P, W8>& w, _Float16*) {
        typedef RawK<D, P, W8> R;
        const f16x2 bias = h2(W8 ? 1152.f : mins ? 1024.f : 1032.f);
        uint32_t mask = 0x000f000fu, magic = 0x64006400u;
        asm("" : "+s"(mask));
        asm("" : "+v"(magic));
#pragma unroll
        for (int n = 0; n < R::N; ++n) {
            int key, q;
            k_place<R::kC>(t, n, key, q);
            if (R::kAll < T::kGroup && t >= R::kAll) break;
            uint8_t* row = buf + key * T::kKRow;
#pragma unroll
            for (int i = 0; i < R::kOct; ++i) {
                const int p = q * R::kOct + i, g = p / NB, b = p % NB;
                f16x2 x[4], rest[4];
                const f16x2 d = as_h2(w.d[n][i] * 0x10001u), m = as_h2(mins ? w.m[n][i] * 0x10001u : 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f16x2 c;
                    if constexpr (W8) c = as_h2((__builtin_amdgcn_perm(0, w.w[n][2 * i + j / 2], j & 1 ? 0x0c030c02u : 0x0c010c00u) ^ 0x00800080u) | magic);
                    else c = as_h2(and_or(w.w[n][i] >> (4 * j), mask, magic));
                    c -= bias;
                    if constexpr (P == 2) rest[j] = scaled_rest<W8 ? QMV_Q8_0 : QMV_Q4_1, CARE>(c, d, m, x[j]);
                    else x[j] = scaled<W8 ? QMV_Q8_0 : QMV_Q4_1>(c, d, m);
                }
                uint8_t* to = row + 16 * (4 * b + g);
                *reinterpret_cast<f16x8*>(to) = pack8(x[0], x[1], x[2], x[3]);
                if constexpr (P == 2) *reinterpret_cast<f16x8*>(to + T::kKBytes) = pack8(rest[0], rest[1], rest[2], rest[3]);
            }
        }
    }
    // V: (octet p, four keys) items; neighbouring lanes have neighbouring keys, then octets whose rows are on other banks.
    __device__ static void v_place(int t, int n, int& p, int& key, int& g, int& b) {
        const int it = (t + n * T::kGroup) & (kVItems - 1), o = it / (T::KT / 4);
        key = 4 * (it % (T::KT / 4));
        g = o % 4;
        b = o / 4;
        p = g * NB + b;
    }
    template <bool W8>
    __device__ static void load(const uint8_t* base, int64_t page_bytes, int page_shift, uint32_t minimums, int t, int entries, int sub0,
                                int key0, int len, RawV<D, P, W8>& w) {
        typedef RawV<D, P, W8> R;
#pragma unroll
        for (int n = 0; n < R::N; ++n) {
            int p, key, g, b;
            v_place(t, n, p, key, g, b);
            const int en = entry(entries, sub0, key >> 4), e = max(en, 0);
            const uint32_t off = (key0 + key) & ((1 << page_shift) - 1);
            const uint8_t* pg = base + e * page_bytes;
            const uint8_t* c = pg + (off * R::kRow + (W8 ? 8 : 4) * p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (W8) {
                    const uint2 u = *reinterpret_cast<const uint2*>(c + i * R::kRow);
                    w.w[n][i][0] = u.x;
                    w.w[n][i][1] = u.y;
                } else {
                    w.w[n][i][0] = *reinterpret_cast<const uint32_t*>(c + i * R::kRow);
                }
            }
            const uint32_t s = ((R::kRow + 2 * b) << page_shift) + 2 * off;
            w.d[n] = *reinterpret_cast<const uint2*>(pg + s);
            if constexpr (!W8) w.m[n] = *reinterpret_cast<const uint2*>(pg + (s + minimums));
            w.there[n] = en < 0 ? 0 : len - key0 - key;      // keys of these that are there
        }
    }
    template <bool W8, bool CARE>
    __device__ static void store(int t, uint8_t* buf, bool mins, const RawV<D, P, W8>& w, _Float16* sick) {
        typedef RawV<D, P, W8> R;
        const f16x2 bias = h2(W8 ? 1152.f : mins ? 1024.f : 1032.f);
        uint32_t mask = 0x000f000fu, magic = 0x64006400u;
        asm("" : "+s"(mask));
        asm("" : "+v"(magic));
#pragma unroll
        for (int n = 0; n < R::N; ++n) {
            int p, key, g, b;
            v_place(t, n, p, key, g, b);
            if (kVItems < T::kGroup && t >= kVItems) break;
            // the keys' place in a row: 16 u + 8 jj + 4 h + r at 16 u + 8 h + 4 jj + r
            const int place = (key & ~15) | (key & 4) << 1 | (key & 8) >> 1;
            // absent keys, whose bytes are any: scales and minimums of 0
            const uint32_t k0 = w.there[n] >= 2 ? ~0u : w.there[n] == 1 ? 0xffffu : 0u;
            const uint32_t k1 = w.there[n] >= 4 ? ~0u : w.there[n] == 3 ? 0xffffu : 0u;
            uint32_t d0 = w.d[n].x & k0, d1 = w.d[n].y & k1, m0 = 0, m1 = 0;
            if constexpr (!W8) {
                m0 = mins ? w.m[n].x & k0 : 0u;
                m1 = mins ? w.m[n].y & k1 : 0u;
            }
            if constexpr (CARE) {
                const uint32_t o0 = not_finite(d0) | not_finite(m0), o1 = not_finite(d1) | not_finite(m1);
                d0 &= ~o0;
                d1 &= ~o1;
                m0 &= ~o0;
                m1 &= ~o1;
                if (g == 0) *reinterpret_cast<uint2*>(sick + b * T::KT + place) = uint2{o0 & 0x3c003c00u, o1 & 0x3c003c00u};
            }
            uint8_t* to = buf + (32 * b + 8 * g) * T::kVRow + 2 * place;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f16x2 x[2], y[2], rest[2];        // value e of the keys 0, 1 and 2, 3
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (W8) {
                        constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
                        x[j] = as_h2((__builtin_amdgcn_perm(w.w[n][2 * j + 1][e / 4], w.w[n][2 * j][e / 4], sel[e % 4]) ^ 0x00800080u) | magic);
                    } else {
                        const uint32_t u = __builtin_amdgcn_perm(w.w[n][2 * j + 1][0], w.w[n][2 * j][0], e & 1 ? 0x07060302u : 0x05040100u);
                        x[j] = as_h2(and_or(u >> (4 * (e >> 1)), mask, magic));
                    }
                    x[j] -= bias;
                    const f16x2 d = as_h2(j ? d1 : d0), m = as_h2(j ? m1 : m0);
                    if constexpr (P == 2) rest[j] = scaled_rest<W8 ? QMV_Q8_0 : QMV_Q4_1, CARE>(x[j], d, m, y[j]);
                    else y[j] = scaled<W8 ? QMV_Q8_0 : QMV_Q4_1>(x[j], d, m);
                }
                *reinterpret_cast<uint2*>(to + e * T::kVRow) = uint2{as_u(y[0]), as_u(y[1])};
                if constexpr (P == 2) *reinterpret_cast<uint2*>(to + e * T::kVRow + T::kVBytes) = uint2{as_u(rest[0]), as_u(rest[1])};
            }
        }
    }
};

// N products whose operands (P fp16 pieces) come from LDS, read kAhead
// products before they are multiplied.  Left to the compiler every product
// waits for its own read (3500 cycles for 32 products of 32 cycles).
template <int P, int N, class Read, class Multiply>
__device__ __forceinline__ void products(const Read& read, const Multiply& multiply) {
    constexpr int B = 2, kAhead = N < 12 / P ? N : 12 / P;
    static_assert(N % B == 0 && kAhead % B == 0);
    f16x8 x[kAhead + B][P];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) read(i, x[i]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < N; b += B) {
#pragma unroll
        for (int i = b + kAhead; i < b + kAhead + B; ++i)
            if (i < N) read(i, x[i % (kAhead + B)]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = b; i < b + B; ++i) multiply(i, x[i % (kAhead + B)]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Parts that a request's tiles are split into: no more than leave four blocks
// of 32 keys to each.  A part that has less costs more than it takes over: 123
// tokens of 5 requests, none before them, took 61 us in 10 parts each, now 39.
__device__ __forceinline__ int parts_of(const Req& rq, int splits) { return min(splits, max(1, rq.nblk / 4)); }

template <int D, int P, bool K8, bool V8>
__global__ __launch_bounds__((Tile<D, P>::kThreads), (Tile<D, P>::kWaves / 4)) void attn_tile_kernel(const AttnArgs a) {
    typedef Tile<D, P> T;
    typedef TileStep<D, P> S;
    constexpr int NB = D / 32, KT = T::KT, NT = KT / 32;
    __shared__ __align__(16) uint8_t s_buf[2][T::kBuf];
    __shared__ __align__(16) _Float16 s_sick[2][NB][KT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n32 = lane & 31, hh = lane >> 5;
    const bool second = wave >= T::kWaves / 2;        // the group that has the values
    const int gt = tid % T::kGroup;
    const float inf = __builtin_inff(), nan = __builtin_nanf("");
    const uint32_t window = a.window > 0 ? a.window : 0x80000000u;

    const int r = blockIdx.y, split = blockIdx.z;
    const Req rq = request<1>(a, r);
    const int rows = rq.n * a.G;
    const int parts = parts_of(rq, gridDim.z);
    if (rows <= a.tile_over || split >= parts) return;
    const int tiles = (rows + T::kRows - 1) / T::kRows;
    const int h = blockIdx.x % a.H, order = blockIdx.x / a.H;
    // the last tiles first: they see the most keys
    for (int tile = tiles - 1 - order; tile >= 0; tile -= gridDim.x / a.H) {
        const int row0 = tile * T::kRows;
        const int i_first = token_of(a, row0), i_last = token_of(a, min(row0 + T::kRows, rows) - 1);
        const int p_first = rq.len - rq.n + i_first, p_last = rq.len - rq.n + i_last;
        const int k_lo = a.window > 0 ? max(0, p_first - a.window + 1) : 0, k_hi = p_last + 1;      // keys that some row sees
        const int blk0 = k_lo / KT, blks = max(0, (k_hi + KT - 1) / KT - blk0);
        const int c_lo = blk0 + (int)((int64_t)blks * split / parts), c_hi = blk0 + (int)((int64_t)blks * (split + 1) / parts);

        // ---- queries: B operand, lane n32 = row, places 16 s + 8 hh .. + 7
        const int wrow = row0 + 32 * wave;              // the wave's first
        const int row = wrow + n32;
        const bool have = row < rows;
        const int qi = have ? token_of(a, row) : 0, hq = h * a.G + (have ? row - qi * a.G : 0);
        const int qpos = have ? rq.len - rq.n + qi : -1;
        f16x8 qh[D / 16], ql[P == 2 ? D / 16 : 1];
        float fac;
        {
            const int64_t base = (rq.q0 + qi) * a.qst + hq * a.qsh;
            float amax = 0.f;
            bool fin = true;
            uint32_t w[D / 16][4 * P];
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                load_q8<P>(a, base + 16 * s + 8 * hh, w[s]);
                float x[8];
                widen_q8<P>(a, w[s], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    amax = fmaxf(amax, __builtin_fabsf(x[j]));
                    fin &= __builtin_fabsf(x[j]) < inf;
                }
            }
            amax = fmaxf(amax, __shfl_xor(amax, 32));
            const int sh = row_shift(amax);
            fac = row_factor(a, sh, 0);
            const int odd = fin ? 0 : 1;
            if (odd | __shfl_xor(odd, 32)) fac = nan;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                float x[8];
                widen_q8<P>(a, w[s], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = __builtin_ldexpf(x[j], sh);
                    const _Float16 hi = (_Float16)y;
                    qh[s][j] = hi;
                    if constexpr (P == 2) ql[s][j] = (_Float16)(y - (float)hi);
                }
            }
        }
        // positions of the wave's first and last row
        const int wave_last = __builtin_amdgcn_readfirstlane(rq.len - rq.n + token_of(a, min(wrow + 32, rows) - 1));
        const int wave_first = __builtin_amdgcn_readfirstlane(rq.len - rq.n + token_of(a, min(wrow, rows - 1)));
        const bool wave_has = wrow < rows;
        // whether some of the wave's rows see keys of a block
        const auto sees_some = [&](int blk) {
            return wave_has && blk * KT <= wave_last && (a.window <= 0 || blk * KT + KT > wave_first - a.window + 1);
        };

        const int32_t* table = a.table + (int64_t)r * a.max_pages;
        float m, l;
        f32x16 o[NB];
        // All of the split's blocks, by the first group (Raw: keys) and by the second (values); `care`: with values that are
        // not finite by themselves, and scores far from 0.
        const auto pass = [&](auto care, auto raw) {
            constexpr bool careful = decltype(care)::value;
            typedef decltype(raw) Raw;
            constexpr bool second = std::is_same_v<Raw, RawV<D, P, V8>>;
            // the group's side of the cache
            const CacheSide& side = second ? a.v : a.k;
            const uint8_t* base = side.pages + h * side.head_bytes;
            const int64_t page_bytes = side.page_bytes;
            const int page_shift = a.page_shift;
            const bool mins = side.fmt == QMV_Q4_1;
            const uint32_t minimums = mins ? (2 * NB) << page_shift : 0;
            f32x16 poison;
            m = kANone;
            l = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                poison[i] = 0.f;
#pragma unroll
                for (int v = 0; v < NB; ++v) o[v][i] = 0.f;
            }
            int entries = -1, from = -1;       // pages of 64 tiles of 16 keys from block `from` on; -1: absent, -2: out of range
            Raw w;
            uint32_t bad = 0;                  // tiles of 16 keys out of range: 4 bits a block, the latest loaded lowest
            const auto load = [&](int blk) {
                bad <<= 4;
                if (blk >= c_hi) return;
                if (from < 0 || blk >= from + 64 / T::kSubs) {
                    from = blk;
                    const int at = blk * KT + 16 * lane;
                    entries = -1;
                    if (at < min(rq.len, k_hi) && at + 16 > k_lo && at < c_hi * KT) {
                        entries = table[at >> page_shift];
                        if (entries < 0 || entries >= a.n_pages) entries = -2;
                    }
                }
                const int sub0 = (blk - from) * T::kSubs, key0 = blk * KT;
#pragma unroll
                for (int i = 0; i < T::kSubs; ++i) bad |= __builtin_amdgcn_readlane(entries, sub0 + i) == -2 ? 1u << i : 0u;
                S::load(base, page_bytes, page_shift, minimums, gt, entries, sub0, key0, rq.len, w);
            };
            const auto store = [&](int blk) {
                if (blk >= c_hi) return;
                S::template store<second ? V8 : K8, careful>(gt, s_buf[blk & 1] + (second ? P * T::kKBytes : 0), mins, w,
                                                             &s_sick[blk & 1][0][0]);
            };
            f32x16 s[NT];
            f16x8 ph[NT][2], pl[P == 2 ? NT : 1][2];
            // Queries by keys of block blk, and weights by values of block blk.
            const auto read_k = [&](int blk, int n, f16x8 (&k)[P]) {
                const uint8_t* p = s_buf[blk & 1] + (32 * (n % NT) + n32) * T::kKRow + 32 * (n / NT) + 16 * hh;
#pragma unroll
                for (int i = 0; i < P; ++i) k[i] = *reinterpret_cast<const f16x8*>(p + i * T::kKBytes);
            };
            const auto mul_k = [&](int n, const f16x8 (&k)[P]) {
                const int t = n % NT, d = n / NT;
                if constexpr (P == 2) {
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[1], qh[d], s[t], 0, 0, 0);
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[0], ql[d], s[t], 0, 0, 0);
                }
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[0], qh[d], s[t], 0, 0, 0);
            };
            const auto read_v = [&](int blk, int n, f16x8 (&x)[P]) {
                const uint8_t* p = s_buf[blk & 1] + P * T::kKBytes + (32 * (n % NB) + n32) * T::kVRow + 32 * (n / NB) + 16 * hh;
#pragma unroll
                for (int i = 0; i < P; ++i) x[i] = *reinterpret_cast<const f16x8*>(p + i * T::kVBytes);
            };
            const auto mul_v = [&](int n, const f16x8 (&x)[P]) {
                const int v = n % NB, t = n / NB / 2, u = n / NB % 2;
                if constexpr (P == 2) {
                    o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[1], ph[t][u], o[v], 0, 0, 0);
                    o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[0], pl[t][u], o[v], 0, 0, 0);
                }
                o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[0], ph[t][u], o[v], 0, 0, 0);
            };
            constexpr int kNK = NT * D / 16, kNV = NT * 2 * NB;
            const auto clear = [&] {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
            };
            const auto scores = [&](int blk) {
                clear();
                products<P, kNK>([&](int n, f16x8 (&k)[P]) { read_k(blk, n, k); }, mul_k);
            };
            const auto values = [&](int blk) { products<P, kNV>([&](int n, f16x8 (&x)[P]) { read_v(blk, n, x); }, mul_v); };
            const auto values_scores = [&](int blk) {
                clear();
                products<P, kNV + kNK>(
                    [&](int n, f16x8 (&x)[P]) {
                        if (n < kNV) read_v(blk, n, x);
                        else read_k(blk + 1, n - kNV, x);
                    },
                    [&](int n, const f16x8 (&x)[P]) {
                        if (n < kNV) mul_v(n, x);
                        else mul_k(n - kNV, x);
                    });
            };
            const auto softmax = [&](int blk, uint32_t odd) {
                if (!sees_some(blk)) return;
                const int key0 = blk * KT;
                const bool plain = key0 + KT <= wave_first + 1 && (a.window <= 0 || key0 > wave_last - a.window) && !odd;
                if (careful || !plain) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int back = qpos - key0 - 32 * t - 4 * hh;      // position less key 8 j + r
                        f16x8 sees[2];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const bool seen = (uint32_t)(back - 8 * (i / 4) - i % 4) < window;
                            s[t][i] = seen ? (odd >> (2 * t + i / 8) & 1 ? nan : s[t][i]) : -inf;
                            sees[i / 8][i % 8] = seen ? (_Float16)1.f : (_Float16)0.f;
                        }
                        if constexpr (careful)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                f16x8 x;
#pragma unroll
                                for (int i = 0; i < 8; ++i) x[i] = (_Float16)0.f;
                                if (n32 < NB) x = *reinterpret_cast<const f16x8*>(&s_sick[blk & 1][n32 % NB][32 * t + 16 * u + 8 * hh]);
                                poison = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, sees[u], poison, 0, 0, 0);
                            }
                    }
                }
                float top = -inf;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
                const uint32_t tw = __builtin_bit_cast(uint32_t, careful ? top * fac : __builtin_fmaf(top, fac, -kALow));
                const auto x = __builtin_amdgcn_permlane32_swap(tw, tw, false, false);
                top = fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1]));
                top = fmaxf(careful ? lowered(top) : top, m);
                if (__any(top > m)) {
                    const float f = __builtin_amdgcn_exp2f(m - top);
                    l *= f;
#pragma unroll
                    for (int v = 0; v < NB; ++v) o[v] *= f;
                    m = top;
                }
                float unit = fac;
                if constexpr (careful) {
                    const bool far = is_far(m);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[t][i] *= far ? unit : 1.f;
                    unit = far ? 1.f : unit;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][8 * u + i], unit, -m));
                            const _Float16 hi = (_Float16)p;
                            ph[t][u][i] = hi;
                            if constexpr (P == 2) {
                                l += p;
                                pl[t][u][i] = (_Float16)(p - (float)hi);
                            }
                        }
                        if constexpr (P == 1)      // the sum of the weights as they are multiplied
#pragma unroll
                            for (int i = 0; i < 8; i += 2) l = __builtin_amdgcn_fdot2(f16x2{ph[t][u][i], ph[t][u][i + 1]}, h2(1.f), l, false);
                    }
            };

            // Phase 2 j: the first group weighs block j and stores the keys of j + 1, the second multiplies the values of j - 1 and
            // the keys of j; phase 2 j + 1: the first multiplies the values of j and the keys of j + 1, the second weighs j and
            // stores the values of j + 1.  Buffers hold two blocks: the keys of j are read in phases 2 j - 1 and 2 j, the values
            // of j in 2 j + 1 and 2 j + 2, and each is stored in a phase between the last reads of its buffer and its own first.
            if (c_lo < c_hi) {
                lds_barrier();             // the last pass's reads
                load(c_lo);
                store(c_lo);
                load(c_lo + 1);
                lds_barrier();
                if (!second && sees_some(c_lo)) scores(c_lo);
                lds_barrier();
                if (second) {
                    if (sees_some(c_lo)) scores(c_lo);
                    lds_barrier();
                }
#pragma unroll 1
                for (int blk = c_lo; blk < c_hi; ++blk) {
                    softmax(blk, (bad >> 4) & 15);
                    store(blk + 1);
                    lds_barrier();
                    load(blk + 2);      // here: the phases take about as long as each other
                    __builtin_amdgcn_s_setprio(1);
                    const bool now = sees_some(blk), next = blk + 1 < c_hi && sees_some(blk + 1);
                    if (now && next) values_scores(blk);
                    else if (now) values(blk);
                    else if (next) scores(blk + 1);
                    __builtin_amdgcn_s_setprio(0);
                    lds_barrier();
                }
                if (!second) lds_barrier();
            }
            if constexpr (careful) {
                // rows 8 j + 4 hh + r of the product are blocks: a lane has four of its query's, the other half the others
#pragma unroll
                for (int v = 0; v < NB; ++v) {
                    const float mine = poison[v % 4], other = __shfl_xor(mine, 32);
                    const bool odd = (v / 4 == hh ? mine : other) > 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[v][i] = odd ? nan : o[v][i];
                }
            }
        };
        if (second) pass(std::false_type{}, RawV<D, P, V8>());
        else pass(std::false_type{}, RawK<D, P, K8>());
        bool odd = is_far(m);
#pragma unroll
        for (int v = 0; v < NB; ++v)
#pragma unroll
            for (int i = 0; i < 16; ++i) odd |= !(__builtin_fabsf(o[v][i]) < inf);
        // 0 times a value that is not finite, of a key that a row does not see, or scores far from 0: again, with care
        if (__builtin_expect(__syncthreads_or(odd), 0)) {
            if (second) pass(std::true_type{}, RawV<D, P, V8>());
            else pass(std::true_type{}, RawK<D, P, K8>());
        }

        // ---- outputs: places 32 v + 8 j + 4 hh + r of the lane's row
        const float ll = l + __shfl_xor(l, 32);
        if (have) {
            if (parts == 1) {
                float f = 1.f, total = ll;
                if (a.sinks) {
                    const float sk = sink_of(a, hq), top = fmaxf(m, sk);
                    f = __builtin_amdgcn_exp2f(m - top);
                    total = ll * f + __builtin_amdgcn_exp2f(sk - top);
                }
                const float inv = rq.bad ? nan : total == 0.f ? 0.f : f / total;
                const int64_t to = ((rq.q0 + qi) * a.H * a.G + hq) * D + 4 * hh;
#pragma unroll
                for (int v = 0; v < NB; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        store_out4(a, to + 32 * v + 8 * j,
                                   f32x4{o[v][4 * j] * inv, o[v][4 * j + 1] * inv, o[v][4 * j + 2] * inv, o[v][4 * j + 3] * inv});
            } else {
                const int64_t at = split * a.n_tokens * a.H * a.G + (rq.q0 + qi) * a.H * a.G + hq;
                float* x = a.tile_part + at * D + 4 * hh;
#pragma unroll
                for (int v = 0; v < NB; ++v)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<f32x4*>(x + 32 * v + 8 * j) = f32x4{o[v][4 * j], o[v][4 * j + 1], o[v][4 * j + 2], o[v][4 * j + 3]};
                if (hh == 0) {
                    float* ml = a.tile_part + gridDim.z * a.n_tokens * a.H * a.G * D + 2 * at;
                    ml[0] = m;
                    ml[1] = ll;
                }
            }
        }
    }
}

// Joins the parts of split tiles: D / 4 threads a row.
template <int D>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(const AttnArgs a, int splits) {
    constexpr int kCols = D / 4, kPer = 256 / kCols;
    const int r = blockIdx.y;
    const Req rq = request<1>(a, r);
    const int parts = parts_of(rq, splits);
    if (rq.n * a.G <= a.tile_over || parts == 1) return;
    const int64_t rows = (int64_t)rq.n * a.G * a.H, all = a.n_tokens * a.G * a.H;
    for (int64_t w = (int64_t)blockIdx.x * kPer + threadIdx.x / kCols; w < rows; w += (int64_t)gridDim.x * kPer) {
        const int64_t at = rq.q0 * a.G * a.H + w;
        const int hq = (int)(w % (a.G * a.H)), c = 4 * (threadIdx.x % kCols);
        const float* ml = a.tile_part + splits * all * D;
        // the loads of a few parts at a time
        constexpr int kLoads = 4;
        float m = kANone, l = 0.f;
#pragma unroll kLoads
        for (int s = 0; s < parts; ++s) m = fmaxf(m, ml[2 * (s * all + at)]);
        f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < parts; s += kLoads) {
            float2 y[kLoads];
            f32x4 z[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int64_t i = min(s + k, parts - 1) * all + at;
                y[k] = *reinterpret_cast<const float2*>(ml + 2 * i);
                z[k] = *reinterpret_cast<const f32x4*>(a.tile_part + i * D + c);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const float f = s + k < parts ? __builtin_amdgcn_exp2f(y[k].x - m) : 0.f;
                l += y[k].y * f;
                x += z[k] * f;
            }
        }
        finish(a, hq, m, l, x, rq.bad);
        store_out4(a, at * D + c, x);
    }
}

template <int D, int P, bool K8, bool V8>
int32_t launch_tile_n(const AttnArgs& a, int splits, hipStream_t st) {
    const char* name = "qmv_cache_attention";
    const int64_t most = (a.max_q * a.G + Tile<D, P>::kRows - 1) / Tile<D, P>::kRows;
    const int64_t x = std::min<int64_t>(most, std::max<int64_t>(1, (int64_t(1) << 22) / ((int64_t)a.H * a.R * splits)));
    hipLaunchKernelGGL((attn_tile_kernel<D, P, K8, V8>), dim3((unsigned)(x * a.H), a.R, splits), dim3(Tile<D, P>::kThreads), 0, st, a);
    if (const int32_t e = check_launch(name)) return e;
    if (splits == 1) return QMV_OK;
    const int64_t rows = a.max_q * a.G * a.H * (D / 4) / 256 + 1;
    hipLaunchKernelGGL((attn_tile_join_kernel<D>), dim3((unsigned)std::min<int64_t>(rows, std::max<int64_t>(1, 65536 / a.R)), a.R),
                       dim3(256), 0, st, a, splits);
    return check_launch(name);
}

template <int D, int P>
int32_t launch_tile(const AttnArgs& a, int splits, hipStream_t st) {
    const bool k8 = a.k.fmt == QMV_Q8_0, v8 = a.v.fmt == QMV_Q8_0;
    if (k8) return v8 ? launch_tile_n<D, P, true, true>(a, splits, st) : launch_tile_n<D, P, true, false>(a, splits, st);
    return v8 ? launch_tile_n<D, P, false, true>(a, splits, st) : launch_tile_n<D, P, false, false>(a, splits, st);
}

}  // namespace
}  // namespace qmv
