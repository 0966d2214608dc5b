// Log probabilities of given tokens, entropy and the most probable tokens of
// rows of logits.
//
// With m the row's largest logit, z = l - m and T the sum of e^z without one
// largest term, log p = z - log1p(T) and the entropy log1p(T) + A / (1 + T),
// A = sum e^z (-z): sums of terms of one sign, so fp32 keeps the digits of a
// row that is nearly certain.
//
// Two launches: every chunk of 4096 logits gives its maximum, T and A relative
// to it, and its top_k in order; then a workgroup per row joins the chunks.
// Top tokens: each wave sorts its 64 lanes' maxima, the k-th of them is
// reached by at least k logits, so only logits that reach the largest such
// bound are candidates, a little more than k; their places are counted
// against each other.
#include <algorithm>

#include "qmv_block_decode.h"
#include "qmv_host.h"

namespace qmv {
namespace {

constexpr int kLT = 256;
constexpr int kLWaves = kLT / 64;
constexpr int kLPer = 16;
constexpr int kLChunk = kLT * kLPer;
constexpr int kLTop = 32;
constexpr int kLCands = 2048;            // candidates of a row that are counted in LDS

struct ChunkStat {
    float m, t, a;       // maximum; sum of e^(l - m) without one largest term; sum of e^(l - m) (m - l).  NaN in t: no distribution
    float pad;
};
struct LogprobArgs {
    const void* logits;
    int64_t ld, rows;
    int V, chunks, top, vec;
    const int32_t* targets;
    int n_targets;
    float* logprobs;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprobs;
    ChunkStat* stat;     // [rows][chunks]
    float* best;         // [rows][chunks][top]: largest logits in order, then -inf
    int32_t* best_id;
};

// e^x for x <= 0, relative error about 2^-22: x log2(e) in two parts, since an
// error of the exponent is one of the result.
__device__ __forceinline__ float exp_neg32(float x) {
    const float hi = x * 1.44269504088896341f;
    const float lo = __builtin_fmaf(x, 1.44269504088896341f, -hi) + x * 1.92596299e-8f;
    // x = -inf: lo is NaN, and the result 0
    return hi < -160.f ? 0.f : __builtin_amdgcn_exp2f(hi) * __builtin_fmaf(lo, 0.69314718f, 1.f);
}

__device__ __forceinline__ float wave_sum(float s) {
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    return s;
}
__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
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
    const int c = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inf = __builtin_inff();
    __shared__ float wm[kLWaves], wt[kLWaves], wa[kLWaves], wb[kLWaves], wc[kLWaves];
    __shared__ int wbad[kLWaves], s_n;
    __shared__ float s_v[kLChunk];
    __shared__ int s_id[kLChunk];
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const LT* l = static_cast<const LT*>(a.logits) + row * a.ld;
        const int v0 = c * kLChunk;
        float f[kLPer];
#pragma unroll
        for (int k = 0; k < kLPer / 4; ++k) {
            const int v = v0 + 4 * ((int)threadIdx.x + kLT * k);
            if (a.vec && v + 3 < a.V) {
                const float4 w = XIn<LT>::load4(l + v);
                f[4 * k] = w.x; f[4 * k + 1] = w.y; f[4 * k + 2] = w.z; f[4 * k + 3] = w.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * k + j] = v + j < a.V ? XIn<LT>::load1(l + v + j) : -inf;
            }
        }
        float mine = -inf;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kLPer; ++i) {
            mine = fmaxf(mine, f[i]);
            bad |= !(f[i] < inf);
        }
        float m = wave_max(mine);
        float bound = -inf;
        if (a.top) bound = __shfl(wave_sort(mine), a.top - 1);
        __syncthreads();          // the last row's reads
        if (lane == 0) {
            wm[wave] = m;
            wb[wave] = bound;
        }
        bad = __any(bad);
        if (lane == 0) wbad[wave] = bad;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        m = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
        bound = fmaxf(fmaxf(wb[0], wb[1]), fmaxf(wb[2], wb[3]));
        bad = wbad[0] | wbad[1] | wbad[2] | wbad[3];
        float t = 0.f, e_a = 0.f;
        int tops = 0;
        if (m > -inf) {
#pragma unroll
            for (int i = 0; i < kLPer; ++i) {
                const float z = f[i] - m, e = exp_neg32(z);
                tops += f[i] == m;
                t += f[i] == m ? 0.f : e;
                e_a += e > 0.f ? e * -z : 0.f;
            }
        }
        t = wave_sum(t);
        e_a = wave_sum(e_a);
        const float count = wave_sum((float)tops);
        if (lane == 0) {
            wt[wave] = t;
            wa[wave] = e_a;
            wc[wave] = count;
        }
        if (a.top) {
            // candidates, those equal to the bound among them
#pragma unroll
            for (int i = 0; i < kLPer; ++i) {
                const bool in = f[i] >= bound && f[i] > -inf;
                const uint64_t who = __ballot(in);
                if (!who) continue;
                int at = 0;
                if (lane == __builtin_ctzll(who)) at = atomicAdd(&s_n, __popcll(who));
                at = __builtin_amdgcn_readlane(at, __builtin_ctzll(who)) + __builtin_popcountll(who & ((uint64_t(1) << lane) - 1));
                if (in) {
                    s_v[at] = f[i];
                    s_id[at] = v0 + 4 * ((int)threadIdx.x + kLT * (i >> 2)) + (i & 3);
                }
            }
        }
        __syncthreads();
        const int64_t at = row * a.chunks + c;
        if (threadIdx.x == 0) {
            ChunkStat s;
            s.m = m;
            // the other largest terms, each 1, come last: beside 1 the small ones would lose their digits
            s.t = bad ? __builtin_nanf("")
                  : m > -inf ? (wt[0] + wt[1]) + (wt[2] + wt[3]) + (wc[0] + wc[1] + wc[2] + wc[3] - 1.f) : 0.f;
            s.a = (wa[0] + wa[1]) + (wa[2] + wa[3]);
            s.pad = 0.f;
            a.stat[at] = s;
        }
        if (a.top) {
            const int n = s_n;
            for (int i = threadIdx.x; i < n; i += kLT) {
                const float v = s_v[i];
                const int id = s_id[i];
                int place = 0;
                for (int j = 0; j < n; ++j) place += s_v[j] > v || (s_v[j] == v && s_id[j] < id);
                if (place < a.top) {
                    a.best[at * a.top + place] = v;
                    a.best_id[at * a.top + place] = id;
                }
            }
            for (int i = n + threadIdx.x; i < a.top; i += kLT) {
                a.best[at * a.top + i] = -inf;
                a.best_id[at * a.top + i] = -1;
            }
        }
    }
}

template <class LT>
__global__ __launch_bounds__(kLT) void logprobs_row_kernel(const LogprobArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inf = __builtin_inff();
    __shared__ float s_m, s_log, s_bad, s_b[kLWaves], s_v[kLCands];
    __shared__ int s_n, s_id[kLCands];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const ChunkStat* st = a.stat + row * a.chunks;
        __syncthreads();
        if (wave == 0) {
            float m = -inf, bad = 0.f;
            for (int c = lane; c < a.chunks; c += 64) {
                m = fmaxf(m, st[c].m);
                if (!(st[c].t >= 0.f)) bad = 1.f;
            }
            m = wave_max(m);
            bad = wave_max(bad);
            if (!(m > -inf)) bad = 1.f;
            // the first chunk with the largest gives the term left out
            int lead = 0x7fffffff;
            for (int c = lane; c < a.chunks; c += 64)
                if (st[c].m == m && c < lead) lead = c;
#pragma unroll
            for (int o = 32; o; o >>= 1) lead = min(lead, __shfl_xor(lead, o));
            float t = 0.f, e_a = 0.f;
            for (int c = lane; c < a.chunks; c += 64) {
                const ChunkStat s = st[c];
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
                if (a.entropy) a.entropy[row] = bad != 0.f ? __builtin_nanf("") : log_t + e_a / (1.f + t);
            }
        }
        __syncthreads();
        const float m = s_m, log_t = s_log;
        const bool bad = s_bad != 0.f;
        for (int i = threadIdx.x; i < a.n_targets; i += kLT) {
            const int64_t at = row * a.n_targets + i;
            const int x = a.targets[at];
            float v = __builtin_nanf("");
            if (!bad && (unsigned)x < (unsigned)a.V)
                v = (XIn<LT>::load1(static_cast<const LT*>(a.logits) + row * a.ld + x) - m) - log_t;
            a.logprobs[at] = v;
        }
        if (!a.top) continue;
        const int64_t out = row * a.top;
        const float* best = a.best + row * a.chunks * a.top;
        const int* best_id = a.best_id + row * a.chunks * a.top;
        // entries of the chunks' lists that reach the top-th of a wave's chunk maxima
        if (threadIdx.x == 0) s_n = 0;
        float mine = -inf;
        for (int c = threadIdx.x; c < a.chunks; c += kLT) mine = fmaxf(mine, st[c].m);
        const float bound = __shfl(wave_sort(mine), a.top - 1);
        if (lane == 0) s_b[wave] = bound;
        __syncthreads();
        const float reach = fmaxf(fmaxf(s_b[0], s_b[1]), fmaxf(s_b[2], s_b[3]));
        const int entries = bad ? 0 : a.chunks * a.top;
        for (int i = threadIdx.x; i < entries; i += kLT) {
            const float v = best[i];
            if (v >= reach && v > -inf) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kLCands) {
                    s_v[at] = v;
                    s_id[at] = best_id[i];
                }
            }
        }
        __syncthreads();
        const int n = s_n;
        if (n <= kLCands) {      // the order they came in does not matter: a place is a count
            for (int i = threadIdx.x; i < n; i += kLT) {
                const float v = s_v[i];
                const int id = s_id[i];
                int place = 0;
                for (int j = 0; j < n; ++j) place += s_v[j] > v || (s_v[j] == v && s_id[j] < id);
                if (place < a.top) {
                    a.top_tokens[out + place] = id;
                    a.top_logprobs[out + place] = (v - m) - log_t;
                }
            }
        } else if (wave == 0) {
            // many equal ones: the largest behind the last one taken, top times
            float last_v = inf;
            int last_id = -1;
            for (int k = 0; k < a.top; ++k) {
                float v = -inf;
                int id = 0x7fffffff;
                for (int i = lane; i < entries; i += 64) {
                    const float x = best[i];
                    const int y = best_id[i];
                    if ((x < last_v || (x == last_v && y > last_id)) && (x > v || (x == v && y < id))) {
                        v = x;
                        id = y;
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
                if (lane == 0) {
                    a.top_tokens[out + k] = id;
                    a.top_logprobs[out + k] = (v - m) - log_t;
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
int64_t chunks_of(int64_t vocab) { return (vocab + kLChunk - 1) / kLChunk; }
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
    return (size_t)(n_rows * chunks_of(vocab)) * (sizeof(ChunkStat) + 8 * (size_t)top_k);
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
    a.vec = aligned(logits, 4 * le) && (n_rows == 1 || ld % 4 == 0);
    a.targets = targets;
    a.n_targets = n_targets;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.stat = static_cast<ChunkStat*>(workspace);
    a.best = reinterpret_cast<float*>(a.stat + n_rows * a.chunks);
    a.best_id = reinterpret_cast<int32_t*>(a.best + n_rows * a.chunks * top_k);
    const hipStream_t st = as_stream(stream);
    switch (logits_type) {
    case QMV_X_F32: return launch_logprobs<float>(a, st);
    case QMV_X_F16: return launch_logprobs<_Float16>(a, st);
    default: return launch_logprobs<__bf16>(a, st);
    }
}
