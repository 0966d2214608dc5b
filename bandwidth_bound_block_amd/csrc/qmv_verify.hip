// Verification of drafted tokens against the target's probabilities.
//
// Request r has n = n_draft[r] drafted tokens x_0..x_{n-1} and the target's
// logits at rows 0..n.  With p_i = softmax(logits row i) and q_i the draft's
// distribution at i (all of it on x_i where no draft probabilities are
// given), tokens are kept in order while u_i q_i(x_i) < p_i(x_i).  At the
// first that is not, i, one token is drawn from max(p_i - q_i, 0); if all
// are kept, one from p_n: the first v whose running sum of weights passes
// u_last times their total.  The tokens so chosen are distributed as the
// target's own.
//
// Three launches: (1) every row's maximum and sum of exponentials, in chunks
// of the vocabulary; (2) the decisions, made alike by every workgroup of a
// request, and the chunk sums of the drawn row's weights; (3) the chunk and
// the place in it.  (3) by the last workgroup of (2) took longer: the fences
// it needs write the L2s back (139 us against 26 + 27 with the same bodies
// for 64 requests of 151936 tokens).  There the three take 47, 22 and 11 us;
// the first reads 190 MB (fp32 logits of 64 x 1..8 rows) at 4.0 TB/s with 68%
// of the vector issue slots taken by fp64 exponentials, the others are bound
// by those and by latency: 1 request of 4 drafts and 128256 tokens takes 4, 6
// and 8 us.  Exponentials and sums are in
// fp64: the outputs are comparisons, and with fp32 sums (1e-7 off) over a
// vocabulary of 1.5e5 about one draw in thirty could fall on the wrong side
// of a border between two tokens of mean mass.
#include <algorithm>

#include "qmv_block_decode.h"
#include "qmv_host.h"

namespace qmv {
namespace {

struct Decision;
constexpr int kVT = 256;                 // threads
constexpr int kVWaves = kVT / 64;
constexpr int kVPer = 16;                // logits a thread holds
constexpr int kVChunk = kVT * kVPer;     // logits of a workgroup
constexpr int kVDrafts = 64;             // most drafted tokens of a request
constexpr int kVMaxChunks = 1024;        // most chunks of a vocabulary

struct VerifyArgs {
    const void* logits;
    int64_t ls_req, ls_row;
    const float* q;
    int64_t qs_req, qs_row;
    const int32_t* drafted;
    const int32_t* n_draft;
    const float* u;
    const float* u_last;
    int D, V, chunks, vec, qvec;
    double2* part;         // [requests][D + 1][chunks]: maximum, sum of exp(l - maximum)
    double2* sums;         // [requests][chunks]: sum of max(p - q, 0), sum of p, times the row's sum
    Decision* made;        // [requests]
    int32_t* tokens;
    int32_t* kept;
};

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int r) { return min(max(a.n_draft[r], 0), a.D); }

// e^x for x <= 0 to 5e-14: x = n ln 2 + f, |f| <= ln 2 / 2 (the rounding of
// ln 2 adds n 2.3e-17), e^f by the Taylor polynomial of degree 20 economized
// to degree 9 (its terms past that in Chebyshev polynomials of f / (ln 2 / 2)
// dropped: 1.9e-14 of e^f), times 2^n.  The Taylor polynomial of degree 9
// itself costs the same and is up to 7e-12 off, always one way; degree 10
// and ln 2 in two parts (1e-15) take the largest batch from 79 to 83 us.
// Below -746 the value is less than half of the smallest number; NaN stays
// NaN.
__device__ __forceinline__ double exp_neg(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634074);
    const double f = __builtin_fma(n, -0x1.62e42fefa39efp-1, x);
    double p = 0x1.72faf16b7bd05p-19;
    p = __builtin_fma(p, f, 0x1.a17df2ec2bc60p-16);
    p = __builtin_fma(p, f, 0x1.a01978c559bacp-13);
    p = __builtin_fma(p, f, 0x1.6c162bb5db14bp-10);
    p = __builtin_fma(p, f, 0x1.1111112dd6fbap-7);
    p = __builtin_fma(p, f, 0x1.55555588b972bp-5);
    p = __builtin_fma(p, f, 0x1.555555554b752p-3);
    p = __builtin_fma(p, f, 0x1.ffffffffe74e3p-2);
    p = __builtin_fma(p, f, 0x1.000000000001ep+0);
    p = __builtin_fma(p, f, 0x1.000000000003dp+0);
    p = __builtin_ldexp(p, (int)n);
    return x < -746.0 ? 0.0 : p;
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    return s;
}
__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
}

// Elements v..v+3 of a row; those past its end are `pad`.
template <class LT>
__device__ __forceinline__ void load_quad(const LT* p, int v, int V, bool vec, float pad, float* f) {
    if (vec && v + 3 < V) {
        const float4 w = XIn<LT>::load4(p + v);
        f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v + j < V ? XIn<LT>::load1(p + v + j) : pad;
    }
}

// Quads of a chunk: thread t holds elements 4 (t + 256 k) .. + 3, k < 4, so
// that a wave's loads run along the row.  Elements past the row are `pad`.
template <class LT>
__device__ __forceinline__ void load_chunk(const LT* p, int v0, int V, bool vec, float pad, float (&f)[kVPer]) {
#pragma unroll
    for (int k = 0; k < kVPer / 4; ++k)
        load_quad<LT>(p, v0 + 4 * ((int)threadIdx.x + kVT * k), V, vec, pad, f + 4 * k);
}

// (1) maximum and sum of a chunk of a row
template <class LT>
__global__ __launch_bounds__(kVT) void verify_stats_kernel(const VerifyArgs a) {
    const int c = blockIdx.x, row = blockIdx.y, r = blockIdx.z;
    if (row > drafts_of(a, r)) return;
    const LT* l = static_cast<const LT*>(a.logits) + r * a.ls_req + row * a.ls_row;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float inf = __builtin_inff();
    float f[kVPer];
    load_chunk<LT>(l, c * kVChunk, a.V, a.vec, -inf, f);
    float m = -inf;
#pragma unroll
    for (int i = 0; i < kVPer; ++i) m = fmaxf(m, f[i]);     // passes NaN over: they come back in the sum
    __shared__ float wm[kVWaves];
    __shared__ double ws[kVWaves];
    m = wave_max(m);
    if (lane == 0) wm[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    double s = 0.0;
    if (m == -inf) {                                        // nothing, or NaN
#pragma unroll
        for (int i = 0; i < kVPer; ++i)
            if (f[i] != f[i]) s = __builtin_nan("");
    } else {
#pragma unroll
        for (int i = 0; i < kVPer; ++i) s += exp_neg((double)f[i] - (double)m);
    }
    s = wave_sum(s);
    if (lane == 0) ws[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        a.part[((int64_t)r * (a.D + 1) + row) * a.chunks + c] =
            double2{(double)m, (ws[0] + ws[1]) + (ws[2] + ws[3])};
}

// What a request's rows come to: kept tokens, and the drawn row.
struct Decision {
    int kept, x;           // x: the rejected token where all of q is on it, else -1
    bool all;
    double m, s;           // the drawn row's maximum and sum
};

// By one whole workgroup; every thread gets the same.  A row that is no
// distribution (NaN, +inf, or -inf throughout) keeps nothing: its sum is NaN
// or 0, and no comparison with it holds.
template <class LT>
__device__ __forceinline__ Decision decide(const VerifyArgs& a, int r) {
    __shared__ double rm[kVDrafts + 1], rs[kVDrafts + 1], rp[kVDrafts], rl[kVDrafts];
    __shared__ int rx[kVDrafts];
    const int n = drafts_of(a, r);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = wave; i <= n; i += kVWaves) {
        const double2* p = a.part + ((int64_t)r * (a.D + 1) + i) * a.chunks;
        float m = -__builtin_inff();
        for (int c = lane; c < a.chunks; c += 64) m = fmaxf(m, (float)p[c].x);
        m = wave_max(m);
        double s = 0.0;
        for (int c = lane; c < a.chunks; c += 64) {
            const double2 v = p[c];
            // a chunk of -inf adds nothing unless it holds a NaN
            if (v.y != 0.0) s += v.x == (double)m ? v.y : v.y * exp_neg(v.x - (double)m);
        }
        s = wave_sum(s);
        if (lane == 0) {
            rm[i] = (double)m;
            rs[i] = s;
        }
    }
    // token i by thread i; the first that is not kept ends them
    __shared__ int s_kept, s_x;
    if (threadIdx.x < 64) {
        bool keep = true;
        int x = -1;
        if (lane < n) {
            x = a.drafted[(int64_t)r * a.D + lane];
            keep = false;
            if ((unsigned)x < (unsigned)a.V) {
                const float l = XIn<LT>::load1(static_cast<const LT*>(a.logits) + r * a.ls_req + lane * a.ls_row + x);
                const float qx = a.q ? a.q[r * a.qs_req + lane * a.qs_row + x] : 1.f;
                const float u = a.u[(int64_t)r * a.D + lane];
                rp[lane] = (double)u * (double)qx;
                rl[lane] = (double)l;
                keep = true;
            } else {
                x = -1;
            }
        }
        rx[lane] = keep ? x : -1;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        bool keep = lane >= n || rx[lane] >= 0;
        if (lane < n && keep) keep = rp[lane] * rs[lane] < exp_neg(rl[lane] - rm[lane]);
        const uint64_t no = __ballot(!keep);
        if (lane == 0) {
            s_kept = no ? __builtin_ctzll(no) : n;
            s_x = !a.q && no ? rx[s_kept] : -1;
        }
    }
    __syncthreads();
    Decision d;
    d.kept = s_kept;
    d.all = d.kept == n;
    d.x = s_x;
    d.m = rm[d.kept];
    d.s = rs[d.kept];
    return d;
}

// Weights of the drawn row times its sum: left of q, and whole.
__device__ __forceinline__ double left_of(const Decision& d, double p, float q, int v) {
    if (d.all) return p;
    const double t = v == d.x ? d.s : (double)q * d.s;
    return fmax(p - t, 0.0);
}

// (2) chunk sums of the drawn row's weights
template <class LT>
__global__ __launch_bounds__(kVT) void verify_weights_kernel(const VerifyArgs a) {
    const int c = blockIdx.x, r = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Decision d = decide<LT>(a, r);
    float f[kVPer], q[kVPer];
    load_chunk<LT>(static_cast<const LT*>(a.logits) + r * a.ls_req + d.kept * a.ls_row, c * kVChunk, a.V, a.vec,
                   -__builtin_inff(), f);
    if (a.q && !d.all) {
        load_chunk<float>(a.q + r * a.qs_req + d.kept * a.qs_row, c * kVChunk, a.V, a.qvec, 0.f, q);
    } else {
#pragma unroll
        for (int i = 0; i < kVPer; ++i) q[i] = 0.f;
    }
    double sl = 0.0, sp = 0.0;
#pragma unroll
    for (int i = 0; i < kVPer; ++i) {
        const int v = c * kVChunk + 4 * ((int)threadIdx.x + kVT * (i >> 2)) + (i & 3);
        const double p = exp_neg((double)f[i] - d.m);
        sp += p;
        sl += left_of(d, p, q[i], v);
    }
    __shared__ double2 w[kVWaves];
    sl = wave_sum(sl);
    sp = wave_sum(sp);
    if (lane == 0) w[wave] = double2{sl, sp};
    __syncthreads();
    if (threadIdx.x == 0) {
        a.sums[(int64_t)r * a.chunks + c] =
            double2{(w[0].x + w[1].x) + (w[2].x + w[3].x), (w[0].y + w[1].y) + (w[2].y + w[3].y)};
        if (c == 0) a.made[r] = d;
    }
}

// (3) the token drawn, and the outputs of request r
template <class LT>
__global__ __launch_bounds__(kVT) void verify_draw_kernel(const VerifyArgs a) {
    const int r = blockIdx.x;
    const Decision d = a.made[r];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __shared__ int s_chunk, s_whole, s_token;
    __shared__ double s_before, s_goal, wsum[kVWaves], cl[kVMaxChunks], cp[kVMaxChunks];
    const double2* sums = a.sums + (int64_t)r * a.chunks;
    for (int c = tid; c < a.chunks; c += kVT) {
        cl[c] = sums[c].x;
        cp[c] = sums[c].y;
    }
    __syncthreads();
    if (wave == 0) {
        // each lane a run of chunks; totals and places by scans over the lanes
        const int per = (a.chunks + 63) / 64, c0 = min(lane * per, a.chunks), c1 = min(c0 + per, a.chunks);
        double tl = 0.0, tp = 0.0;
        for (int c = c0; c < c1; ++c) {
            tl += cl[c];
            tp += cp[c];
        }
        const double all_left = wave_sum(tl), all_p = wave_sum(tp);
        // p = q leaves nothing: the draw is from p
        const bool whole = !(all_left > 0.0);
        const double total = whole ? all_p : all_left, own = whole ? tp : tl;
        const double goal = (double)a.u_last[r] * total;
        double at = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double t = __shfl_up(at, o);
            if (lane >= o) at += t;
        }
        at -= own;
        // the first chunk that passes the goal, and the last with weight if
        // rounding passes them all
        int found = -1, last = -1;
        double before = 0.0, before_last = 0.0;
        for (int c = c0; c < c1; ++c) {
            const double w = whole ? cp[c] : cl[c];
            if (w > 0.0) {
                last = c;
                before_last = at;
                if (found < 0 && at + w > goal) {
                    found = c;
                    before = at;
                }
            }
            at += w;
        }
        const uint64_t f = __ballot(found >= 0), l = __ballot(last >= 0);
        const bool any = total > 0.0 && total < (double)__builtin_inff() && d.s > 0.0 && l != 0;
        const int who = f ? __builtin_ctzll(f) : (l ? 63 - __builtin_clzll(l) : 0);
        if (lane == who) {
            s_chunk = any ? (f ? found : last) : -1;
            s_before = f ? before : before_last;
            s_goal = goal;
            s_whole = whole;
            s_token = -1;
        }
    }
    __syncthreads();
    if (s_chunk >= 0) {
        // 16 neighbouring tokens a thread
        const int v0 = s_chunk * kVChunk + kVPer * tid;
        const LT* l = static_cast<const LT*>(a.logits) + r * a.ls_req + d.kept * a.ls_row;
        const float* q = a.q && !d.all ? a.q + r * a.qs_req + d.kept * a.qs_row : nullptr;
        double w[kVPer], own = 0.0;
        float f[kVPer], g[kVPer];
#pragma unroll
        for (int k = 0; k < kVPer; k += 4) {
            load_quad<LT>(l, v0 + k, a.V, a.vec, -__builtin_inff(), f + k);
            if (q) load_quad<float>(q, v0 + k, a.V, a.qvec, 0.f, g + k);
        }
#pragma unroll
        for (int i = 0; i < kVPer; ++i) {
            const double p = exp_neg((double)f[i] - d.m);
            w[i] = s_whole ? p : left_of(d, p, q ? g[i] : 0.f, v0 + i);
            own += w[i];
        }
        double in = own;                    // inclusive scan over the threads
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double t = __shfl_up(in, o);
            if (lane >= o) in += t;
        }
        if (lane == 63) wsum[wave] = in;
        __syncthreads();
        double at = s_before + (in - own);
        for (int k = 0; k < wave; ++k) at += wsum[k];
        int last = -1, found = -1;
#pragma unroll
        for (int i = 0; i < kVPer; ++i) {
            at += w[i];
            if (w[i] > 0.0) {
                last = v0 + i;
                if (found < 0 && at > s_goal) found = v0 + i;
            }
        }
        // the first found; the last with weight if rounding passes them all
        __shared__ int s_found, s_last;
        if (tid == 0) {
            s_found = 0x7fffffff;
            s_last = -1;
        }
        __syncthreads();
        if (found >= 0) atomicMin(&s_found, found);
        if (last >= 0) atomicMax(&s_last, last);
        __syncthreads();
        if (tid == 0) s_token = s_found < 0x7fffffff ? s_found : s_last;
        __syncthreads();
    }
    for (int i = tid; i <= a.D; i += kVT)
        a.tokens[(int64_t)r * (a.D + 1) + i] =
            i < d.kept ? a.drafted[(int64_t)r * a.D + i] : (i == d.kept ? s_token : -1);
    if (tid == 0) a.kept[r] = d.kept;
}

template <class LT>
int32_t launch_verify(const VerifyArgs& a, int requests, hipStream_t st) {
    hipLaunchKernelGGL((verify_stats_kernel<LT>), dim3(a.chunks, a.D + 1, requests), dim3(kVT), 0, st, a);
    if (const int32_t e = check_launch("qmv_spec_verify")) return e;
    hipLaunchKernelGGL((verify_weights_kernel<LT>), dim3(a.chunks, requests), dim3(kVT), 0, st, a);
    if (const int32_t e = check_launch("qmv_spec_verify")) return e;
    hipLaunchKernelGGL((verify_draw_kernel<LT>), dim3(requests), dim3(kVT), 0, st, a);
    return check_launch("qmv_spec_verify");
}

constexpr int64_t kVRequests = 65535, kVVocab = 1 << 22;
static_assert(kVVocab / kVChunk <= kVMaxChunks, "a request's chunk sums fit LDS");
bool sizes_ok(int64_t requests, int32_t drafts, int64_t vocab) {
    return requests >= 1 && requests <= kVRequests && drafts >= 1 && drafts <= kVDrafts && vocab >= 1 && vocab <= kVVocab;
}
int64_t chunks_of(int64_t vocab) { return (vocab + kVChunk - 1) / kVChunk; }

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_spec_verify_workspace_bytes(int64_t n_requests, int32_t max_drafts, int64_t vocab) {
    using namespace qmv;
    if (!sizes_ok(n_requests, max_drafts, vocab)) return 0;
    return (size_t)(n_requests * (max_drafts + 2) * chunks_of(vocab)) * 16 + (size_t)n_requests * sizeof(Decision);
}

extern "C" int32_t qmv_spec_verify(const void* logits, int32_t logits_type, int64_t logits_stride_request,
                                   int64_t logits_stride_row, const float* draft_probs, int64_t probs_stride_request,
                                   int64_t probs_stride_row, const int32_t* draft_tokens, const int32_t* n_draft,
                                   const float* u_accept, const float* u_last, int64_t n_requests, int32_t max_drafts,
                                   int64_t vocab, int32_t* tokens, int32_t* n_kept, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    using namespace qmv;
    const char* name = "qmv_spec_verify";
    if (!logits || !draft_tokens || !n_draft || !u_accept || !u_last || !tokens || !n_kept || !workspace)
        return fail(QMV_EINVAL, "%s: null pointer", name);
    if (logits_type != QMV_X_F32 && logits_type != QMV_X_F16 && logits_type != QMV_X_BF16)
        return fail(QMV_EINVAL, "%s: unknown logits_type %d", name, (int)logits_type);
    if (!sizes_ok(n_requests, max_drafts, vocab))
        return fail(QMV_EINVAL, "%s: n_requests must be 1..65535, max_drafts 1..%d, vocab 1..2^22", name, kVDrafts);
    if (logits_stride_row < vocab || (n_requests > 1 && logits_stride_request < vocab))
        return fail(QMV_EINVAL, "%s: the logits' strides must be >= vocab", name);
    if (draft_probs && ((max_drafts > 1 && probs_stride_row < vocab) || (n_requests > 1 && probs_stride_request < vocab)))
        return fail(QMV_EINVAL, "%s: the draft probabilities' strides must be >= vocab", name);
    const size_t need = qmv_spec_verify_workspace_bytes(n_requests, max_drafts, vocab);
    if (workspace_bytes < need)
        return fail(QMV_EINVAL, "%s: the workspace needs %zu bytes, got %zu", name, need, workspace_bytes);
    const int le = logits_type == QMV_X_F32 ? 4 : 2;
    if (!aligned(logits, le) || !aligned(draft_probs, 4) || !aligned(draft_tokens, 4) || !aligned(n_draft, 4) ||
        !aligned(u_accept, 4) || !aligned(u_last, 4) || !aligned(tokens, 4) || !aligned(n_kept, 4) ||
        !aligned(workspace, 16))
        return fail(QMV_EALIGN, "%s: a pointer is not aligned to its elements (workspace: 16 bytes)", name);
    VerifyArgs a;
    a.logits = logits;
    a.ls_req = logits_stride_request;
    a.ls_row = logits_stride_row;
    a.q = draft_probs;
    a.qs_req = probs_stride_request;
    a.qs_row = probs_stride_row;
    a.drafted = draft_tokens;
    a.n_draft = n_draft;
    a.u = u_accept;
    a.u_last = u_last;
    a.D = max_drafts;
    a.V = (int)vocab;
    a.chunks = (int)chunks_of(vocab);
    a.vec = aligned(logits, 4 * le) && a.ls_req % 4 == 0 && a.ls_row % 4 == 0;
    a.qvec = aligned(draft_probs, 16) && a.qs_req % 4 == 0 && a.qs_row % 4 == 0;
    a.part = static_cast<double2*>(workspace);
    a.sums = a.part + n_requests * (max_drafts + 1) * a.chunks;
    a.made = reinterpret_cast<Decision*>(a.sums + n_requests * a.chunks);
    a.tokens = tokens;
    a.kept = n_kept;
    const hipStream_t st = as_stream(stream);
    switch (logits_type) {
    case QMV_X_F32: return launch_verify<float>(a, (int)n_requests, st);
    case QMV_X_F16: return launch_verify<_Float16>(a, (int)n_requests, st);
    default: return launch_verify<__bf16>(a, (int)n_requests, st);
    }
}
