// The kernel for many rows of queries: pieces of prompts.
//
// A workgroup has 32 rows of queries a wave (row = query token times G + head
// of the group) and one key/value head, and goes over the keys KT at a time.
// Its threads make fp16 values of the codes once for all its rows and lay them
// in LDS, keys as rows, values transposed, each in the order that the matrix
// cores take them: v_mfma_f32_32x32x16_f16 gives a lane, for one query, the
// keys 8 j + 4 h + r (h = lane / 32, j, r < 4) of 32, and the second product
// takes them from there as its operand, so the values' rows are in that order.
// The next keys' codes are on their way meanwhile; two buffers, one barrier a
// step.  Few tiles are split over the keys and joined by a second launch.
#pragma once
#include "qmv_attention.h"

namespace qmv {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D, int P>
struct Tile {
    static constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 32 * kWaves;
    static constexpr int NB = D / 32;
    static constexpr int KT = D * P <= 128 ? 64 : 32;           // keys of a step
    static constexpr int kSubs = KT / 16;
    static constexpr int kKRow = 2 * D, kVRow = 2 * KT;         // bytes of a row in LDS: a key's places, a place's keys
    static constexpr int kKBytes = KT * kKRow, kVBytes = D * kVRow;
    static constexpr int kBuf = P * (kKBytes + kVBytes);
    static constexpr int kKChunks = KT * (D / 16) / kThreads > 1 ? KT * (D / 16) / kThreads : 1;      // 16-byte chunks of codes a thread, 8 bits
    static constexpr int kVItems = (D / 8) * (KT / 4);          // (octet, four keys)
};

// Chunk c (16 bytes) of row r, rows of N chunks, at a place without bank conflicts for 16 neighbouring rows.
template <int N>
__device__ __forceinline__ int chunk_place(int r, int c) {
    if constexpr (N >= 16) return c ^ (r & 15);
    else if constexpr (N == 8) return c ^ ((r >> 1) & 7);
    else return c ^ ((r >> 2) & 3);
}

// Raw codes and scales of one step, of one thread.
struct RawStep {
    u32x4 k[2];          // two chunks of 16 bytes
    uint32_t kd[4], km[4];
    uint32_t v[4][2];
    uint2 vd, vm;
};

template <int D, int P>
struct TileStep {
    typedef Tile<D, P> T;
    static constexpr int NB = T::NB;
    // K: chunks of 16 bytes of the step's codes, KT * (row / 16) of them over the threads.
    template <int F>
    __device__ static void load_k(const AttnArgs& a, int h, int entries, int sub0, int key0, RawStep& w) {
        constexpr int kRow = row_bytes_of(F, D), kC = kRow / 16, kAll = T::KT * kC;
#pragma unroll
        for (int n = 0; n < (kAll + T::kThreads - 1) / T::kThreads; ++n) {
            const int c = threadIdx.x + n * T::kThreads, key = c / kC, q = c % kC;
            const int64_t e = max(__shfl(entries, sub0 + (key >> 4)), 0);
            if (kAll < T::kThreads && c >= kAll) break;
            const int off = (key0 + key) & ((1 << a.page_shift) - 1);
            const uint8_t* p = a.k.pages + e * a.k.page_bytes + h * a.k.head_bytes;
            w.k[n] = *reinterpret_cast<const u32x4*>(p + off * kRow + 16 * q);
            const uint8_t* s = p + ((int64_t)kRow << a.page_shift) + 2 * off;
            constexpr int kOct = F == QMV_Q8_0 ? 2 : 4;      // octets of a chunk
#pragma unroll
            for (int i = 0; i < kOct; ++i) {
                const int b = (q * kOct + i) % NB;
                w.kd[kOct * n + i] = *reinterpret_cast<const uint16_t*>(s + ((int64_t)(2 * b) << a.page_shift));
                if constexpr (F == QMV_Q4_1)
                    w.km[kOct * n + i] = *reinterpret_cast<const uint16_t*>(s + ((int64_t)(2 * (NB + b)) << a.page_shift));
            }
        }
    }
    template <int F>
    __device__ static void store_k(uint8_t* buf, const RawStep& w) {
        constexpr int kRow = row_bytes_of(F, D), kC = kRow / 16, kAll = T::KT * kC;
#pragma unroll
        for (int n = 0; n < (kAll + T::kThreads - 1) / T::kThreads; ++n) {
            const int c = threadIdx.x + n * T::kThreads, key = c / kC, q = c % kC;
            if (kAll < T::kThreads && c >= kAll) break;
            constexpr int kOct = F == QMV_Q8_0 ? 2 : 4;
#pragma unroll
            for (int i = 0; i < kOct; ++i) {
                const int p = q * kOct + i, g = p / NB, b = p % NB;
                f16x2 x[4], first[4], rest[4];
                if constexpr (F == QMV_Q8_0) {
                    const uint32_t u = w.k[n][2 * i] ^ 0x80808080u, v = w.k[n][2 * i + 1] ^ 0x80808080u;
                    x[0] = byte_pair<0, 1>(u, v); x[1] = byte_pair<2, 3>(u, v); x[2] = byte_pair<4, 5>(u, v); x[3] = byte_pair<6, 7>(u, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = nibble_pair(w.k[n][i], j, F == QMV_Q4_0 ? 8.f : 0.f);
                }
                const f16x2 d = as_h2(w.kd[kOct * n + i] * 0x10001u), m = as_h2(F == QMV_Q4_1 ? w.km[kOct * n + i] * 0x10001u : 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (P == 2) rest[j] = scaled_rest<F>(x[j], d, m, first[j]);
                    else first[j] = scaled<F>(x[j], d, m);
                }
                uint8_t* to = buf + key * T::kKRow + 16 * chunk_place<D / 8>(key, 4 * b + g);
                *reinterpret_cast<f16x8*>(to) = pack8(first[0], first[1], first[2], first[3]);
                if constexpr (P == 2) *reinterpret_cast<f16x8*>(to + T::kKBytes) = pack8(rest[0], rest[1], rest[2], rest[3]);
            }
        }
    }
    // V: (octet p, four keys) items.
    template <int F>
    __device__ static void load_v(const AttnArgs& a, int h, int entries, int sub0, int key0, int len, RawStep& w) {
        constexpr int kRow = row_bytes_of(F, D);
        const int it = threadIdx.x % T::kVItems, p = it % (D / 8), key = 4 * (it / (D / 8));
        const int en = __shfl(entries, sub0 + (key >> 4));
        if (T::kVItems < T::kThreads && threadIdx.x >= T::kVItems) return;
        const int64_t e = max(en, 0);
        const int off = (key0 + key) & ((1 << a.page_shift) - 1), b = p % NB;
        const uint8_t* pg = a.v.pages + e * a.v.page_bytes + h * a.v.head_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F == QMV_Q8_0) {
                const uint2 u = *reinterpret_cast<const uint2*>(pg + (off + i) * kRow + 8 * p);
                w.v[i][0] = u.x;
                w.v[i][1] = u.y;
            } else {
                w.v[i][0] = *reinterpret_cast<const uint32_t*>(pg + (off + i) * kRow + 4 * p);
            }
        }
        const uint8_t* s = pg + ((int64_t)kRow << a.page_shift) + 2 * off;
        w.vd = *reinterpret_cast<const uint2*>(s + ((int64_t)(2 * b) << a.page_shift));
        if constexpr (F == QMV_Q4_1) w.vm = *reinterpret_cast<const uint2*>(s + ((int64_t)(2 * (NB + b)) << a.page_shift));
        // absent keys, whose bytes are any: scales and minimums of 0
        const int n = en < 0 ? 0 : len - key0 - key;
        const uint32_t m0 = n >= 2 ? ~0u : n == 1 ? 0xffffu : 0u, m1 = n >= 4 ? ~0u : n == 3 ? 0xffffu : 0u;
        w.vd.x &= m0;
        w.vd.y &= m1;
        if constexpr (F == QMV_Q4_1) {
            w.vm.x &= m0;
            w.vm.y &= m1;
        }
    }
    template <int F, bool CARE>
    __device__ static void store_v(uint8_t* buf, RawStep& w, _Float16* sick) {
        if (T::kVItems < T::kThreads && threadIdx.x >= T::kVItems) return;
        const int it = threadIdx.x % T::kVItems, p = it % (D / 8), key = 4 * (it / (D / 8));
        const int g = p / NB, b = p % NB;
        // the keys' place in a row: 16 u + 8 jj + 4 h + r at 16 u + 8 h + 4 jj + r
        const int place = (key & ~15) | (key & 4) << 1 | (key & 8) >> 1;
        if constexpr (CARE) {
            uint32_t o0 = not_finite(w.vd.x), o1 = not_finite(w.vd.y);
            if constexpr (F == QMV_Q4_1) {
                o0 |= not_finite(w.vm.x);
                o1 |= not_finite(w.vm.y);
                w.vm.x &= ~o0;
                w.vm.y &= ~o1;
            }
            w.vd.x &= ~o0;
            w.vd.y &= ~o1;
            if (g == 0) *reinterpret_cast<uint2*>(sick + b * T::KT + place) = uint2{o0 & 0x3c003c00u, o1 & 0x3c003c00u};
        }
        const f16x2 d0 = as_h2(w.vd.x), d1 = as_h2(w.vd.y);
        const f16x2 m0 = as_h2(F == QMV_Q4_1 ? w.vm.x : 0u), m1 = as_h2(F == QMV_Q4_1 ? w.vm.y : 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f16x2 x0, x1;        // value e of the keys 0, 1 and 2, 3
            if constexpr (F == QMV_Q8_0) {
                constexpr uint32_t sel[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
                x0 = as_h2((__builtin_amdgcn_perm(w.v[1][e / 4], w.v[0][e / 4], sel[e % 4]) ^ 0x00800080u) | 0x64006400u) - h2(1152.f);
                x1 = as_h2((__builtin_amdgcn_perm(w.v[3][e / 4], w.v[2][e / 4], sel[e % 4]) ^ 0x00800080u) | 0x64006400u) - h2(1152.f);
            } else {
                const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
                const float bias = F == QMV_Q4_0 ? 8.f : 0.f;
                x0 = nibble_pair(__builtin_amdgcn_perm(w.v[1][0], w.v[0][0], sel), e >> 1, bias);
                x1 = nibble_pair(__builtin_amdgcn_perm(w.v[3][0], w.v[2][0], sel), e >> 1, bias);
            }
            const int dim = 32 * b + 8 * g + e;
            uint8_t* to = buf + dim * T::kVRow + 16 * chunk_place<T::KT / 8>(dim, place >> 3) + (place & 4) * 2;
            f16x2 y0, y1;
            if constexpr (P == 2) {
                const f16x2 r0 = scaled_rest<F>(x0, d0, m0, y0), r1 = scaled_rest<F>(x1, d1, m1, y1);
                *reinterpret_cast<uint2*>(to + T::kVBytes) = uint2{as_u(r0), as_u(r1)};
            } else {
                y0 = scaled<F>(x0, d0, m0);
                y1 = scaled<F>(x1, d1, m1);
            }
            *reinterpret_cast<uint2*>(to) = uint2{as_u(y0), as_u(y1)};
        }
    }
};

template <int D, int P>
__global__ __launch_bounds__(256, (D * P <= 128 ? 2 : 1)) void attn_tile_kernel(const AttnArgs a) {
    typedef Tile<D, P> T;
    typedef TileStep<D, P> S;
    constexpr int NB = D / 32, KT = T::KT, NT = KT / 32;
    __shared__ __align__(16) uint8_t s_buf[2][T::kBuf];
    __shared__ __align__(16) _Float16 s_sick[NB][KT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n32 = lane & 31, hh = lane >> 5;
    const float inf = __builtin_inff(), nan = __builtin_nanf("");
    const uint32_t window = a.window > 0 ? a.window : 0x80000000u;

    const int r = blockIdx.y, split = blockIdx.z, splits = gridDim.z;
    const Req rq = request<1>(a, r);
    const int rows = rq.n * a.G;
    if (rows <= a.tile_over) return;
    const int tiles = (rows + T::kRows - 1) / T::kRows;
    const int h = blockIdx.x % a.H, order = blockIdx.x / a.H;
    // the last tiles first: they see the most keys
    for (int tile = tiles - 1 - order; tile >= 0; tile -= gridDim.x / a.H) {
        const int row0 = tile * T::kRows;
        const int i_first = token_of(a, row0), i_last = token_of(a, min(row0 + T::kRows, rows) - 1);
        const int p_first = rq.len - rq.n + i_first, p_last = rq.len - rq.n + i_last;
        const int k_lo = a.window > 0 ? max(0, p_first - a.window + 1) : 0, k_hi = p_last + 1;      // keys that some row sees
        const int blk0 = k_lo / KT, blks = max(0, (k_hi + KT - 1) / KT - blk0);
        const int c_lo = blk0 + (int)((int64_t)blks * split / splits), c_hi = blk0 + (int)((int64_t)blks * (split + 1) / splits);

        // ---- queries: B operand, lane n32 = row, places 16 s + 8 hh .. + 7
        const int row = row0 + 32 * wave + n32;
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
                widen_q8<P>(w[s], a.x_type == QMV_X_F16, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    amax = fmaxf(amax, __builtin_fabsf(x[j]));
                    fin &= __builtin_fabsf(x[j]) < inf;
                }
            }
            amax = fmaxf(amax, __shfl_xor(amax, 32));
            const int sh = row_shift(amax);
            fac = fmaxf(__builtin_ldexpf(a.scale, -sh), 1e-37f);
            const int odd = fin ? 0 : 1;
            if (odd | __shfl_xor(odd, 32)) fac = nan;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                float x[8];
                widen_q8<P>(w[s], a.x_type == QMV_X_F16, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = __builtin_ldexpf(x[j], sh);
                    const _Float16 hi = (_Float16)y;
                    qh[s][j] = hi;
                    if constexpr (P == 2) ql[s][j] = (_Float16)(y - (float)hi);
                }
            }
        }
        const int wave_last = __builtin_amdgcn_readfirstlane(
            rq.len - rq.n + token_of(a, max(min(row0 + 32 * wave + 32, rows) - 1, 0)));       // last position of the wave's rows
        const int wave_first = __builtin_amdgcn_readfirstlane(rq.len - rq.n + token_of(a, min(row0 + 32 * wave, rows - 1)));

        const int32_t* table = a.table + (int64_t)r * a.max_pages;
        float m, l;
        f32x16 o[NB];
        const auto pass = [&](auto care) {
            constexpr bool careful = decltype(care)::value;
            m = kANone;
            l = 0.f;
#pragma unroll
            for (int v = 0; v < NB; ++v)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[v][i] = 0.f;
            f32x16 poison;
#pragma unroll
            for (int i = 0; i < 16; ++i) poison[i] = 0.f;
            int entries = -1, from = -1;       // pages of 64 tiles of 16 keys from block `from` on; -1: absent, -2: out of range
            const auto pages = [&](int blk) {
                if (from >= 0 && blk < from + 64 / T::kSubs) return;
                from = blk;
                const int at = blk * KT + 16 * lane;
                entries = -1;
                if (at < min(rq.len, k_hi) && at + 16 > k_lo && at < c_hi * KT) {
                    entries = table[at >> a.page_shift];
                    if (entries < 0 || entries >= a.n_pages) entries = -2;
                }
            };
            RawStep w;
            int bad_next = 0, bad = 0;         // tiles of 16 keys out of range
            const auto load = [&](int blk) {
                pages(blk);
                const int sub0 = (blk - from) * T::kSubs, key0 = blk * KT;
                bad_next = 0;
#pragma unroll
                for (int i = 0; i < T::kSubs; ++i) bad_next |= __builtin_amdgcn_readlane(entries, sub0 + i) == -2 ? 1 << i : 0;
                switch (a.k.fmt) {
                case QMV_Q8_0: S::template load_k<QMV_Q8_0>(a, h, entries, sub0, key0, w); break;
                case QMV_Q4_0: S::template load_k<QMV_Q4_0>(a, h, entries, sub0, key0, w); break;
                default: S::template load_k<QMV_Q4_1>(a, h, entries, sub0, key0, w); break;
                }
                switch (a.v.fmt) {
                case QMV_Q8_0: S::template load_v<QMV_Q8_0>(a, h, entries, sub0, key0, rq.len, w); break;
                case QMV_Q4_0: S::template load_v<QMV_Q4_0>(a, h, entries, sub0, key0, rq.len, w); break;
                default: S::template load_v<QMV_Q4_1>(a, h, entries, sub0, key0, rq.len, w); break;
                }
            };
            const auto store = [&](int half) {
                uint8_t* kb = s_buf[half];
                uint8_t* vb = kb + P * T::kKBytes;
                switch (a.k.fmt) {
                case QMV_Q8_0: S::template store_k<QMV_Q8_0>(kb, w); break;
                case QMV_Q4_0: S::template store_k<QMV_Q4_0>(kb, w); break;
                default: S::template store_k<QMV_Q4_1>(kb, w); break;
                }
                switch (a.v.fmt) {
                case QMV_Q8_0: S::template store_v<QMV_Q8_0, careful>(vb, w, &s_sick[0][0]); break;
                case QMV_Q4_0: S::template store_v<QMV_Q4_0, careful>(vb, w, &s_sick[0][0]); break;
                default: S::template store_v<QMV_Q4_1, careful>(vb, w, &s_sick[0][0]); break;
                }
            };
            if (c_lo < c_hi) {
                __syncthreads();           // the last pass's reads
                load(c_lo);
                store(c_lo & 1);
                bad = bad_next;
                __syncthreads();
            }
            for (int blk = c_lo; blk < c_hi; ++blk) {
                const bool more = blk + 1 < c_hi;
                if (more) load(blk + 1);
                const int key0 = blk * KT;
                const uint8_t* kb = s_buf[blk & 1];
                const uint8_t* vb = kb + P * T::kKBytes;
                // a wave whose rows see none of the keys has nothing to do
                if (key0 <= wave_last && (a.window <= 0 || key0 + KT > wave_first - a.window + 1)) {
                    const bool plain = key0 + KT <= wave_first + 1 && (a.window <= 0 || key0 > wave_last - a.window) && !bad;
                    f32x16 s[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            const int key = 32 * t + n32;
                            const uint8_t* p = kb + key * T::kKRow + 16 * chunk_place<D / 8>(key, 2 * d + hh);
                            const f16x8 k = *reinterpret_cast<const f16x8*>(p);
                            if constexpr (P == 2) {
                                const f16x8 k2 = *reinterpret_cast<const f16x8*>(p + T::kKBytes);
                                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k2, qh[d], s[t], 0, 0, 0);
                                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, ql[d], s[t], 0, 0, 0);
                            }
                            s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qh[d], s[t], 0, 0, 0);
                        }
                    }
                    if (careful || !plain) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int back = qpos - key0 - 32 * t - 4 * hh;      // position less key 8 j + r
                            f16x8 sees[2];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const bool seen = (uint32_t)(back - 8 * (i / 4) - i % 4) < window;
                                s[t][i] = seen ? (bad >> (2 * t + i / 8) & 1 ? nan : s[t][i]) : -inf;
                                sees[i / 8][i % 8] = seen ? (_Float16)1.f : (_Float16)0.f;
                            }
                            if constexpr (careful)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    f16x8 x;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) x[i] = (_Float16)0.f;
                                    if (n32 < NB) x = *reinterpret_cast<const f16x8*>(&s_sick[n32 % NB][32 * t + 16 * u + 8 * hh]);
                                    poison = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, sees[u], poison, 0, 0, 0);
                                }
                        }
                    }
                    float top = -inf;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
                    top *= fac;
                    {
                        const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, top), __builtin_bit_cast(uint32_t, top),
                                                                        false, false);
                        top = fmaxf(fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1])), m);
                    }
                    if (__any(top > m)) {
                        const float f = __builtin_amdgcn_exp2f(m - top);
                        l *= f;
#pragma unroll
                        for (int v = 0; v < NB; ++v) o[v] *= f;
                        m = top;
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            f16x8 ph, pl;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][8 * u + i], fac, -m));
                                l += p;
                                const _Float16 hi = (_Float16)p;
                                ph[i] = hi;
                                if constexpr (P == 2) pl[i] = (_Float16)(p - (float)hi);
                            }
#pragma unroll
                            for (int v = 0; v < NB; ++v) {
                                const int dim = 32 * v + n32;
                                const uint8_t* p = vb + dim * T::kVRow + 16 * chunk_place<KT / 8>(dim, 4 * t + 2 * u + hh);
                                const f16x8 x = *reinterpret_cast<const f16x8*>(p);
                                if constexpr (P == 2) {
                                    const f16x8 x2 = *reinterpret_cast<const f16x8*>(p + T::kVBytes);
                                    o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x2, ph, o[v], 0, 0, 0);
                                    o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, pl, o[v], 0, 0, 0);
                                }
                                o[v] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, ph, o[v], 0, 0, 0);
                            }
                        }
                }
                bad = bad_next;
                if constexpr (careful) __syncthreads();        // one array of flags
                if (more) store((blk + 1) & 1);
                __syncthreads();
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
        pass(std::false_type{});
        bool odd = false;
#pragma unroll
        for (int v = 0; v < NB; ++v)
#pragma unroll
            for (int i = 0; i < 16; ++i) odd |= !(__builtin_fabsf(o[v][i]) < inf);
        // 0 times a value that is not finite, of a key that a row does not see: again, with such values by themselves
        if (__builtin_expect(__syncthreads_or(odd), 0)) pass(std::true_type{});

        // ---- outputs: places 32 v + 8 j + 4 hh + r of the lane's row
        l += __shfl_xor(l, 32);
        if (have) {
            if (splits == 1) {
                float f = 1.f;
                float ll = l;
                if (a.sinks) {
                    const float sk = a.sinks[hq] * 1.44269504088896341f, top = fmaxf(m, sk);
                    f = __builtin_amdgcn_exp2f(m - top);
                    ll = l * f + __builtin_amdgcn_exp2f(sk - top);
                }
                const float inv = rq.bad ? nan : ll == 0.f ? 0.f : f / ll;
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
                    float* ml = a.tile_part + splits * a.n_tokens * a.H * a.G * D + 2 * at;
                    ml[0] = m;
                    ml[1] = l;
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
    if (rq.n * a.G <= a.tile_over) return;
    const int64_t rows = (int64_t)rq.n * a.G * a.H, all = a.n_tokens * a.G * a.H;
    for (int64_t w = (int64_t)blockIdx.x * kPer + threadIdx.x / kCols; w < rows; w += (int64_t)gridDim.x * kPer) {
        const int64_t at = rq.q0 * a.G * a.H + w;
        const int hq = (int)(w % (a.G * a.H)), c = 4 * (threadIdx.x % kCols);
        const float* ml = a.tile_part + splits * all * D;
        float m = kANone, l = 0.f;
        for (int s = 0; s < splits; ++s) m = fmaxf(m, ml[2 * (s * all + at)]);
        f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * (s * all + at)] - m);
            l += ml[2 * (s * all + at) + 1] * f;
            x += *reinterpret_cast<const f32x4*>(a.tile_part + (s * all + at) * D + c) * f;
        }
        finish(a, hq, m, l, x, rq.bad);
        store_out4(a, at * D + c, x);
    }
}

template <int D, int P>
int32_t launch_tile(const AttnArgs& a, int splits, hipStream_t st) {
    const char* name = "qmv_cache_attention";
    const int64_t most = (a.max_q * a.G + Tile<D, P>::kRows - 1) / Tile<D, P>::kRows;
    const int64_t x = std::min<int64_t>(most, std::max<int64_t>(1, (int64_t(1) << 23) / ((int64_t)a.H * a.R * splits)));
    hipLaunchKernelGGL((attn_tile_kernel<D, P>), dim3((unsigned)(x * a.H), a.R, splits), dim3(256), 0, st, a);
    if (const int32_t e = check_launch(name)) return e;
    if (splits == 1) return QMV_OK;
    const int64_t rows = a.max_q * a.G * a.H * (D / 4) / 256 + 1;
    hipLaunchKernelGGL((attn_tile_join_kernel<D>), dim3((unsigned)std::min<int64_t>(rows, std::max<int64_t>(1, 65536 / a.R)), a.R),
                       dim3(256), 0, st, a, splits);
    return check_launch(name);
}

}  // namespace
}  // namespace qmv
