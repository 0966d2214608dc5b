// Log probabilities of given tokens, entropy and the most probable tokens of
// rows of logits.
//
// With m the row's largest logit, z = l - m and T the sum of e^z without one
// largest term, log p = z - log1p(T) and the entropy log1p(T) + A / (1 + T),
// A = sum e^z (-z): sums of terms of one sign, so fp32 keeps the digits of a
// row that is nearly certain.
//
// Two launches: every chunk of 8192 logits gives its maximum, T and A
// relative to it, and the maxima of groups of 64 logits; then a workgroup per
// row joins the chunks.  Top tokens: the top_k-th largest of those maxima is
// reached by the top_k most probable tokens, so only the few groups whose
// maximum reaches it have candidates, whose logits the second launch reads
// again; places among the candidates are counted.  Candidates found in the
// first launch (ballots and a sort of lanes' maxima in every chunk) took 299
// us for 500 x 151936, where the two launches now take 33 us (152 MB at 4.6
// TB/s, with 82% of the vector issue slots taken) and 15 us (reads that wait
// for one another), together 43; one row of 128256 takes 4 and 7 us.
#include <algorithm>
#include <type_traits>

#include "qmv_block_decode.h"
#include "qmv_host.h"

namespace qmv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLT = 256;
constexpr int kLWaves = kLT / 64;
// Logits of a thread: the first launch takes 30.7 us for 500 rows of 151936
// bf16 logits, with 16 a thread 32.6; for one row of 128256 4.5 and 3.9, with
// 64 it was 5.9.
constexpr int kLPer = 32;
// Logits of a group: those of kLGroup / kLPer threads.  With 32, 64 and 128: 500
// rows of 151936, top 20, 44.2, 43.2 and 44.7 us, 500 of 32000 22.7, 22.6 and 24.3.
constexpr int kLGroup = 64;
constexpr int kLTop = 32;
// Groups that reach the bound, and candidates, of a row that LDS holds, in 12
// KB (registers, not these, bound the workgroups of a compute unit).  A row with
// more (many equal logits, or fewer tokens than top_k beside a finite mask) is
// scanned once for each of its top tokens: 500 rows of 151936 with 8 tokens,
// the rest at the type's lowest value, take 4140 us for the top 20, 41 for the
// top 5; with -infinity in their place 39.
constexpr int kLCands = 1024;
constexpr int kLKeep = 16;                    // maxima of groups that a thread keeps in registers

struct ChunkStat {
    float m, t, a;       // maximum; sum of e^(l - m) without one largest term; sum of e^(l - m) (m - l).  NaN in t: no distribution
    float pad;
};
struct LogprobArgs {
    const void* logits;
    int64_t ld, rows;
    int V, chunks, top;
    const int32_t* targets;
    int n_targets;
    float* logprobs;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprobs;
    ChunkStat* stat;     // [rows][chunks]
    float* most;         // [rows][chunks][groups]: largest logit of each group
};

// Pieces of 16 bytes of a row: thread t of a chunk has pieces t, t + 256, ..  A
// row may begin at any element; the hardware takes such addresses.
template <class LT> constexpr int kVecOf = 16 / sizeof(LT);
typedef uint32_t piece_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t piece_a2 __attribute__((ext_vector_type(4), aligned(2)));
template <class LT>
__device__ __forceinline__ u32x4 load_piece(const LT* p) {
    if constexpr (sizeof(LT) == 4) return *reinterpret_cast<const piece_a4*>(p);
    else return *reinterpret_cast<const piece_a2*>(p);
}

// e^z for z <= 0, and 0 for what is below -1000: the rounding of z log2(e) is a
// relative error of |z| 2^-24.
__device__ __forceinline__ float exp_neg32(float z) {
    return __builtin_amdgcn_exp2f(fmaxf(z, -1000.f) * 1.44269504088896341f);
}

// The larger one, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A value over all lanes: neighbours, quads, eights, rows of 16 by moves within a row of lanes, then rows and halves.  By
// way of LDS (__shfl_xor) these steps were a quarter of the first launch's instructions.
template <class Op>
__device__ __forceinline__ float over_wave(float v, const Op& op) {
    const auto moved = [](float x, auto how) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(how)::value, 0xf, 0xf, true));
    };
    v = op(v, moved(v, std::integral_constant<int, 0xb1>{}));      // lane ^ 1
    v = op(v, moved(v, std::integral_constant<int, 0x4e>{}));      // lane ^ 2
    v = op(v, moved(v, std::integral_constant<int, 0x141>{}));     // mirrored within 8
    v = op(v, moved(v, std::integral_constant<int, 0x140>{}));     // mirrored within 16
    const uint32_t a = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = op(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return op(__builtin_bit_cast(float, (uint32_t)h[0]), __builtin_bit_cast(float, (uint32_t)h[1]));
}
__device__ __forceinline__ float wave_sum(float s) {
    return over_wave(s, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float m) {
    return over_wave(m, [](float a, float b) { return fmaxf(a, b); });
}
// A number that grows with x, and for equal x with a smaller id; +0 and -0 are equal.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    return (uint64_t)(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) << 32 | ~(uint32_t)id;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
// Every lane gets a wave's values in descending order.
__device__ __forceinline__ float wave_sort(float v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
            const float o = __shfl_xor(v, j);
            const bool up = (lane & k) == 0, low = (lane & j) == 0;
            v = up == low ? fmaxf(v, o) : fminf(v, o);
        }
    return v;
}

template <class LT>
__global__ __launch_bounds__(kLT) void logprobs_chunk_kernel(const LogprobArgs a) {
    constexpr int kVec = kVecOf<LT>, kN = kLPer / kVec;
    const int c = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inf = __builtin_inff();
    __shared__ float wm[kLWaves], wt[kLWaves], wa[kLWaves], wc[kLWaves];
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const LT* l = static_cast<const LT*>(a.logits) + row * a.ld;
        const int u0 = c * (kLT * kLPer) + kVec * (int)threadIdx.x;
        float f[kLPer];
        u32x4 w[kN];
        const bool whole = (c + 1) * (kLT * kLPer) <= a.V;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const int u = u0 + kVec * kLT * k;
            if (whole || u + kVec <= a.V) {
                w[k] = load_piece(l + u);
            } else {                       // the row's last piece, or one behind it
                constexpr uint32_t none = sizeof(LT) == 4 || std::is_same_v<LT, __bf16> ? 0xff80u : 0xfc00u;      // -inf's high half
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(LT) == 4) {
                        w[k][j] = u + j < a.V ? reinterpret_cast<const uint32_t*>(l)[u + j] : none << 16;
                    } else {
                        const uint16_t* b = reinterpret_cast<const uint16_t*>(l) + u + 2 * j;
                        w[k][j] = (u + 2 * j < a.V ? b[0] : none) | (u + 2 * j + 1 < a.V ? b[1] : none) << 16;
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const u32x4 x = w[k];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t y = x[j];
                if constexpr (sizeof(LT) == 4) {
                    f[4 * k + j] = __builtin_bit_cast(float, y);
                } else if constexpr (std::is_same_v<LT, _Float16>) {
                    f[8 * k + 2 * j] = half_bits_to_float(y);
                    f[8 * k + 2 * j + 1] = half_bits_to_float(y >> 16);
                } else {
                    f[8 * k + 2 * j] = __builtin_bit_cast(float, y << 16);
                    f[8 * k + 2 * j + 1] = __builtin_bit_cast(float, y & 0xffff0000u);
                }
            }
        }
        float mine = -inf;
#pragma unroll
        for (int i = 0; i < kLPer; ++i) mine = max_or_nan(mine, f[i]);
        const int64_t at = row * a.chunks + c;
        if (a.top) {
            constexpr int kThreads = kLGroup / kLPer;
            float g = mine;
#pragma unroll
            for (int o = 1; o < kThreads; o <<= 1) g = fmaxf(g, __shfl_xor(g, o));
            if (threadIdx.x % kThreads == 0) a.most[at * (kLT / kThreads) + threadIdx.x / kThreads] = g;
        }
        float m = over_wave(mine, max_or_nan);
        __syncthreads();          // the last row's reads
        if (lane == 0) wm[wave] = m;
        __syncthreads();
        m = max_or_nan(max_or_nan(wm[0], wm[1]), max_or_nan(wm[2], wm[3]));
        // largest terms are 1 each and are counted: beside them the small ones would lose their digits
        float t = 0.f, e_a = 0.f;
        float count = 0.f;
        const bool good = m > -inf && m < inf;
        if (good && __any(mine == m)) {
#pragma unroll
            for (int i = 0; i < kLPer; ++i) {
                const float z = fmaxf(f[i] - m, -1000.f), e = __builtin_amdgcn_exp2f(z * 1.44269504088896341f);
                const bool top = z == 0.f;
                count += top ? 1.f : 0.f;
                t += top ? 0.f : e;
                e_a = __builtin_fmaf(e, -z, e_a);
            }
            count = wave_sum(count);
        } else if (good) {        // most waves: what is left out here was a third of the launch's instructions
#pragma unroll
            for (int i = 0; i < kLPer; ++i) {
                const float z = fmaxf(f[i] - m, -1000.f), e = __builtin_amdgcn_exp2f(z * 1.44269504088896341f);
                t += e;
                e_a = __builtin_fmaf(e, -z, e_a);
            }
        }
        t = wave_sum(t);
        e_a = wave_sum(e_a);
        if (lane == 0) {
            wt[wave] = t;
            wa[wave] = e_a;
            wc[wave] = count;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            ChunkStat s;
            s.m = m;
            s.t = good ? (wt[0] + wt[1]) + (wt[2] + wt[3]) + (wc[0] + wc[1] + wc[2] + wc[3] - 1.f)
                  : m == -inf ? 0.f : __builtin_nanf("");
            s.a = (wa[0] + wa[1]) + (wa[2] + wa[3]);
            s.pad = 0.f;
            a.stat[at] = s;
        }
    }
}

template <class LT>
__global__ __launch_bounds__(kLT) void logprobs_row_kernel(const LogprobArgs a) {
    constexpr int kVec = kVecOf<LT>, kThreads = kLGroup / kLPer, kGroups = kLT / kThreads, kPieces = kLGroup / kVec;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inf = __builtin_inff();
    __shared__ float s_m, s_log, s_bad, s_bound;
    __shared__ __align__(16) float s_b[kLWaves * kLTop];
    __shared__ __align__(16) uint64_t s_key[kLCands];
    __shared__ int s_n, s_c, s_id[kLCands];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const ChunkStat* st = a.stat + row * a.chunks;
        const float* most = a.most + row * a.chunks * kGroups;
        const int groups = a.top ? a.chunks * kGroups : 0;
        float g[kLKeep];      // on their way while the chunks are joined
#pragma unroll
        for (int k = 0; k < kLKeep; ++k) {
            const int i = threadIdx.x + k * kLT;
            g[k] = i < groups ? most[i] : -inf;
        }
        const LT* l = static_cast<const LT*>(a.logits) + row * a.ld;
        int target = -1;
        if ((int)threadIdx.x < a.n_targets) target = a.targets[row * a.n_targets + threadIdx.x];
        const float l_target = (unsigned)target < (unsigned)a.V ? XIn<LT>::load1(l + target) : __builtin_nanf("");
        __syncthreads();
        if (wave == 0) {
            const ChunkStat none = {-inf, 0.f, 0.f, 0.f}, first = lane < a.chunks ? st[lane] : none;
            float m = first.m, bad = first.t >= 0.f ? 0.f : 1.f;
            int lead = lane;      // the first chunk with the largest gives the term left out
            for (int c = lane + 64; c < a.chunks; c += 64) {
                if (st[c].m > m) lead = c;
                m = fmaxf(m, st[c].m);
                if (!(st[c].t >= 0.f)) bad = 1.f;
            }
            const float own = m;
            m = wave_max(m);
            bad = __any(bad != 0.f) || !(m > -inf) ? 1.f : 0.f;
            if (own != m) lead = 0x7fffffff;
#pragma unroll
            for (int o = 32; o; o >>= 1) lead = min(lead, __shfl_xor(lead, o));
            float t = 0.f, e_a = 0.f;
            for (int c = lane; c < a.chunks; c += 64) {
                const ChunkStat s = c < 64 ? first : st[c];
                if (!(s.m > -inf)) continue;
                const float z = s.m - m, e = exp_neg32(z), all = 1.f + s.t;
                t += c == lead ? s.t : e * all;
                if (e > 0.f) e_a += e * (s.a - z * all);
            }
            t = wave_sum(t);
            e_a = wave_sum(e_a);
            const float log_t = log1pf(t);
            if (lane == 0) {
                s_m = m;
                s_log = log_t;
                s_bad = bad;
                s_n = s_c = 0;
                if (a.entropy) a.entropy[row] = bad != 0.f ? __builtin_nanf("") : log_t + e_a / (1.f + t);
            }
        }
        // the top-th largest of the threads' maxima, each of a group of its own, bounds the row's from below
        if (a.top) {
            float mine = g[0];
#pragma unroll
            for (int k = 1; k < kLKeep; ++k) mine = fmaxf(mine, g[k]);
            for (int i = threadIdx.x + kLKeep * kLT; i < groups; i += kLT) mine = fmaxf(mine, most[i]);
            mine = wave_sort(mine);
            if (lane < a.top) s_b[wave * a.top + lane] = mine;
        }
        __syncthreads();
        if ((int)threadIdx.x < kLWaves * a.top) {
            const float v = s_b[threadIdx.x];
            int place = 0;
#pragma unroll 4
            for (int j = 0; j < a.top; ++j) {
                const f32x4 o = reinterpret_cast<const f32x4*>(s_b)[j];
#pragma unroll
                for (int k = 0; k < kLWaves; ++k) place += o[k] > v || (o[k] == v && kLWaves * j + k < (int)threadIdx.x);
            }
            if (place == a.top - 1) s_bound = v;
        }
        const float m = s_m, log_t = s_log;
        const bool bad = s_bad != 0.f;
        for (int i = threadIdx.x; i < a.n_targets; i += kLT) {
            const int64_t at = row * a.n_targets + i;
            float v = l_target;
            if (i >= kLT) {
                const int x = a.targets[at];
                v = (unsigned)x < (unsigned)a.V ? XIn<LT>::load1(l + x) : __builtin_nanf("");
            }
            a.logprobs[at] = bad ? __builtin_nanf("") : (v - m) - log_t;
        }
        if (!a.top) continue;
        const int64_t out = row * a.top;
        __syncthreads();
        const float bound = s_bound;
        auto reached = [&](float v, int i) {
            if (bad || !(v >= bound && v > -inf)) return;
            const int at = atomicAdd(&s_n, 1);
            if (at < kLCands) s_id[at] = i;
        };
#pragma unroll
        for (int k = 0; k < kLKeep; ++k) reached(g[k], threadIdx.x + k * kLT);
        for (int i = threadIdx.x + kLKeep * kLT; i < groups; i += kLT) reached(most[i], i);
        __syncthreads();
        int n = s_n;
        // the groups' logits that reach it, piece by piece
        for (int w = threadIdx.x; w < (n <= kLCands ? n * kPieces : 0); w += kLT) {
            const int i = s_id[w / kPieces], k = w % kPieces;
            const int id = i / kGroups * (kLT * kLPer) + kVec * (i % kGroups * kThreads + k % kThreads + kLT * (k / kThreads));
            float x[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] = id + j < a.V ? XIn<LT>::load1(l + id + j) : -inf;
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (x[j] >= bound && x[j] > -inf) {
                    const int at = atomicAdd(&s_c, 1);
                    if (at < kLCands) s_key[at] = order_key(x[j], id + j);
                }
        }
        __syncthreads();
        const int found = s_c;
        if (n <= kLCands && found <= kLCands) {      // the order they came in does not matter: a place is a count
            n = found;
            for (int i = threadIdx.x; i < n; i += kLT) {
                const uint64_t key = s_key[i];
                int place = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) place += s_key[j] > key;
                if (place < a.top) {
                    a.top_tokens[out + place] = (int)~(uint32_t)key;
                    a.top_logprobs[out + place] = (key_value(key) - m) - log_t;
                }
            }
        } else {
            // many equal ones: the largest of the row behind the last one taken, top times
            float last_v = inf;
            int last_id = -1;
            for (n = 0; n < a.top; ++n) {
                float v = -inf;
                int id = 0x7fffffff;
                for (int i = threadIdx.x; i < a.V; i += kLT) {
                    const float x = XIn<LT>::load1(l + i);
                    if ((x < last_v || (x == last_v && i > last_id)) && x > v) {       // the first of equal ones: i goes up
                        v = x;
                        id = i;
                    }
                }
#pragma unroll
                for (int o = 32; o; o >>= 1) {
                    const float ov = __shfl_xor(v, o);
                    const int oi = __shfl_xor(id, o);
                    if (ov > v || (ov == v && oi < id)) {
                        v = ov;
                        id = oi;
                    }
                }
                __syncthreads();
                if (lane == 0) {
                    s_b[wave] = v;
                    s_id[wave] = id;
                }
                __syncthreads();
                for (int w = 0; w < kLWaves; ++w)
                    if (s_b[w] > v || (s_b[w] == v && s_id[w] < id)) {
                        v = s_b[w];
                        id = s_id[w];
                    }
                if (!(v > -inf)) break;
                if (threadIdx.x == 0) {
                    a.top_tokens[out + n] = id;
                    a.top_logprobs[out + n] = (v - m) - log_t;
                }
                last_v = v;
                last_id = id;
            }
        }
        for (int i = n + (int)threadIdx.x; i < a.top; i += kLT) {
            a.top_tokens[out + i] = -1;
            a.top_logprobs[out + i] = bad ? __builtin_nanf("") : -inf;
        }
    }
}

constexpr int64_t kLRows = 1 << 20, kLVocab = 1 << 22;
int64_t chunks_of(int64_t vocab) {
    return (vocab + kLT * kLPer - 1) / (kLT * kLPer);
}
bool sizes_ok(int64_t rows, int64_t vocab, int32_t top) {
    return rows >= 1 && rows <= kLRows && vocab >= 1 && vocab <= kLVocab && rows * chunks_of(vocab) < (1 << 28) && top >= 0 &&
           top <= kLTop;
}

template <class LT>
int32_t launch_logprobs(const LogprobArgs& a, hipStream_t st) {
    const char* name = "qmv_logprobs";
    hipLaunchKernelGGL((logprobs_chunk_kernel<LT>), dim3(a.chunks, (unsigned)std::min<int64_t>(a.rows, 65535)), dim3(kLT), 0, st, a);
    if (const int32_t e = check_launch(name)) return e;
    hipLaunchKernelGGL((logprobs_row_kernel<LT>), dim3((unsigned)a.rows), dim3(kLT), 0, st, a);
    return check_launch(name);
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_logprobs_workspace_bytes(int64_t n_rows, int64_t vocab, int32_t top_k) {
    using namespace qmv;
    if (!sizes_ok(n_rows, vocab, top_k)) return 0;
    return (size_t)(n_rows * chunks_of(vocab)) * (sizeof(ChunkStat) + (top_k ? 4 * (size_t)(kLT * kLPer / kLGroup) : 0));
}

extern "C" int32_t qmv_logprobs(const void* logits, int32_t logits_type, int64_t ld, int64_t n_rows, int64_t vocab,
                                const int32_t* targets, int32_t n_targets, float* logprobs, float* entropy, int32_t top_k,
                                int32_t* top_tokens, float* top_logprobs, void* workspace, size_t workspace_bytes,
                                void* stream) {
    using namespace qmv;
    const char* name = "qmv_logprobs";
    if (!logits || !workspace || (n_targets > 0 && (!targets || !logprobs)) || (top_k > 0 && (!top_tokens || !top_logprobs)))
        return fail(QMV_EINVAL, "%s: null pointer", name);
    if (logits_type != QMV_X_F32 && logits_type != QMV_X_F16 && logits_type != QMV_X_BF16)
        return fail(QMV_EINVAL, "%s: unknown logits_type %d", name, (int)logits_type);
    if (n_targets < 0 || n_targets > 1024) return fail(QMV_EINVAL, "%s: n_targets must be 0..1024", name);
    if (!sizes_ok(n_rows, vocab, top_k))
        return fail(QMV_EINVAL, "%s: n_rows must be 1..2^20, vocab 1..2^22, their chunks below 2^28, top_k 0..%d", name, kLTop);
    if (n_rows > 1 && ld < vocab) return fail(QMV_EINVAL, "%s: ld must be >= vocab", name);
    const size_t need = qmv_logprobs_workspace_bytes(n_rows, vocab, top_k);
    if (workspace_bytes < need)
        return fail(QMV_EINVAL, "%s: the workspace needs %zu bytes, got %zu", name, need, workspace_bytes);
    const int le = logits_type == QMV_X_F32 ? 4 : 2;
    if (!aligned(logits, le) || !aligned(targets, 4) || !aligned(logprobs, 4) || !aligned(entropy, 4) || !aligned(top_tokens, 4) ||
        !aligned(top_logprobs, 4) || !aligned(workspace, 16))
        return fail(QMV_EALIGN, "%s: a pointer is not aligned to its elements (workspace: 16 bytes)", name);
    LogprobArgs a{};
    a.logits = logits;
    a.ld = n_rows > 1 ? ld : vocab;
    a.rows = n_rows;
    a.V = (int)vocab;
    a.chunks = (int)chunks_of(vocab);
    a.top = top_k;
    a.targets = targets;
    a.n_targets = n_targets;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.stat = static_cast<ChunkStat*>(workspace);
    a.most = reinterpret_cast<float*>(a.stat + n_rows * a.chunks);
    const hipStream_t st = as_stream(stream);
    switch (logits_type) {
    case QMV_X_F32: return launch_logprobs<float>(a, st);
    case QMV_X_F16: return launch_logprobs<_Float16>(a, st);
    default: return launch_logprobs<__bf16>(a, st);
    }
}
