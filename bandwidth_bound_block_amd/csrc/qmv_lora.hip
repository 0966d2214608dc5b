// A projection of shared quantized weights with a low-rank adapter per token:
// y_t = DEQ(W) x_t + s_a B_a (A_a x_t), a = adapter_ids[t].
//
// The base product is the library's own (the matvec kernels up to 8 tokens,
// the tile kernel past that); the adapters are two narrow products in fp32:
// v_t = s_a A_a x_t, then y_t += B_a v_t.
#include <algorithm>

#include "qmv_block_decode.h"
#include "qmv_group.h"

namespace qmv {
namespace {

// v[t][r] = scales[a] * sum_k A[a][r][k] x[t][k]: a wave per (token, rank row).
template <class XT, class AT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const XT* __restrict__ x, int64_t ldx,
                                                          const AT* __restrict__ A, const float* __restrict__ scales,
                                                          const int32_t* __restrict__ ids, int n_adapters, int rank,
                                                          int K, float* __restrict__ v) {
    const int t = blockIdx.x, r = blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (r >= rank) return;
    const int a = ids[t];
    if ((unsigned)a >= (unsigned)n_adapters) return;
    const AT* ar = A + ((int64_t)a * rank + r) * K;
    const XT* xt = x + t * ldx;
    float s = 0.f;
    for (int k = lane; k < K; k += 64) s = __builtin_fmaf(XIn<AT>::load1(ar + k), XIn<XT>::load1(xt + k), s);
    s = segment_sum<64>(s);
    if (lane == 0) v[(int64_t)t * rank + r] = scales[a] * s;
}

// y[t][n] += sum_r B[a][n][r] v[t][r]; NaN for an id that is no adapter.
template <class AT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const AT* __restrict__ B, const int32_t* __restrict__ ids,
                                                          int n_adapters, int rank, int N,
                                                          const float* __restrict__ v, float* __restrict__ y,
                                                          int64_t ldy) {
    const int t = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x;
    const int a = ids[t];
    if (n >= N || a == -1) return;
    float* o = y + t * ldy + n;
    if ((unsigned)a >= (unsigned)n_adapters) {
        *o = __builtin_nanf("");
        return;
    }
    const AT* b = B + ((int64_t)a * N + n) * rank;
    const float* vt = v + (int64_t)t * rank;
    float s = 0.f;
    for (int r = 0; r < rank; ++r) s = __builtin_fmaf(XIn<AT>::load1(b + r), vt[r], s);
    *o += s;
}

struct LoraCall {
    const void* x;
    int32_t x_type;
    int64_t ldx, T, N, K;
    const void *A, *B;
    int32_t a_type, n_adapters, rank;
    const float* scales;
    const int32_t* ids;
    float* y;
    int64_t ldy;
    float* v;
};

template <class XT, class AT>
int32_t shrink(const LoraCall& c, hipStream_t st) {
    hipLaunchKernelGGL((lora_shrink_kernel<XT, AT>), dim3((unsigned)c.T, (unsigned)((c.rank + 3) / 4)), dim3(256), 0, st,
                       (const XT*)c.x, c.ldx, (const AT*)c.A, c.scales, c.ids, c.n_adapters, c.rank, (int)c.K, c.v);
    return check_launch("qmv_lora");
}
template <class AT>
int32_t shrink_x(const LoraCall& c, hipStream_t st) {
    switch (c.x_type) {
    case QMV_X_F32: return shrink<float, AT>(c, st);
    case QMV_X_F16: return shrink<_Float16, AT>(c, st);
    default: return shrink<__bf16, AT>(c, st);
    }
}
template <class AT>
int32_t expand(const LoraCall& c, hipStream_t st) {
    hipLaunchKernelGGL((lora_expand_kernel<AT>), dim3((unsigned)c.T, (unsigned)((c.N + 255) / 256)), dim3(256), 0, st,
                       (const AT*)c.B, c.ids, c.n_adapters, c.rank, (int)c.N, c.v, c.y, c.ldy);
    return check_launch("qmv_lora");
}

constexpr int64_t kLoraTokens = 1 << 20;
constexpr int kLoraRank = 128, kLoraAdapters = 1024;

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_lora_workspace_bytes(int64_t n_tokens, int32_t rank, int32_t n_adapters) {
    using namespace qmv;
    if (n_tokens < 1 || n_tokens > kLoraTokens || rank < 1 || rank > kLoraRank || n_adapters < 1 ||
        n_adapters > kLoraAdapters)
        return 0;
    return (size_t)n_tokens * rank * 4;
}

extern "C" int32_t qmv_lora(qmv_fmt fmt, const void* W, int64_t n_rows, int64_t n_cols, const void* x, int32_t x_type,
                            int64_t ldx, int64_t n_tokens, const void* A, const void* B, int32_t a_type,
                            int32_t n_adapters, int32_t rank, const float* scales, const int32_t* adapter_ids,
                            float* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace qmv;
    const char* name = "qmv_lora";
    int uw, ub;
    if (!fmt_unit(fmt, &uw, &ub)) return fail(QMV_EUNSUPPORTED, "%s: unknown format %d", name, (int)fmt);
    if (!W || !x || !A || !B || !scales || !adapter_ids || !y || !workspace)
        return fail(QMV_EINVAL, "%s: null pointer", name);
    if (!x_type_ok(x_type) || !x_type_ok(a_type)) return fail(QMV_EINVAL, "%s: unknown element type", name);
    if (n_rows < 1 || n_rows > (1 << 24)) return fail(QMV_EINVAL, "%s: n_rows must be 1..2^24", name);
    if (n_cols < uw || n_cols % uw || n_cols > 35424)
        return fail(QMV_EINVAL, "%s: n_cols must be a multiple of %d in %d..35424", name, uw, uw);
    if (n_tokens < 1 || n_tokens > kLoraTokens) return fail(QMV_EINVAL, "%s: n_tokens must be 1..2^20", name);
    if (n_adapters < 1 || n_adapters > kLoraAdapters)
        return fail(QMV_EINVAL, "%s: n_adapters must be 1..%d", name, kLoraAdapters);
    if (rank < 1 || rank > kLoraRank) return fail(QMV_EINVAL, "%s: rank must be 1..%d", name, kLoraRank);
    if (n_tokens > 1 && (ldx < n_cols || ldy < n_rows))
        return fail(QMV_EINVAL, "%s: ldx must be >= n_cols and ldy >= n_rows", name);
    if (workspace_bytes < qmv_lora_workspace_bytes(n_tokens, rank, n_adapters))
        return fail(QMV_EINVAL, "%s: the workspace needs %zu bytes, got %zu", name,
                    qmv_lora_workspace_bytes(n_tokens, rank, n_adapters), workspace_bytes);
    if (!aligned(W, fmt_align(fmt))) return fail(QMV_EALIGN, "%s: W must be %d-byte aligned", name, fmt_align(fmt));
    if (!aligned(x, x_elem(x_type)) || !aligned(A, x_elem(a_type)) || !aligned(B, x_elem(a_type)) ||
        !aligned(scales, 4) || !aligned(adapter_ids, 4) || !aligned(y, 4) || !aligned(workspace, 16))
        return fail(QMV_EALIGN, "%s: a pointer is not aligned to its elements (workspace: 16 bytes)", name);
    const hipStream_t st = as_stream(stream);
    LoraCall c{x, x_type, ldx, n_tokens, n_rows, n_cols, A, B, a_type, n_adapters, rank, scales, adapter_ids, y, ldy,
               static_cast<float*>(workspace)};
    int32_t rc;
    if (n_tokens <= 8) {
        rc = format_ops(fmt)->matvec(name, W, n_rows, n_cols, x, x_type, n_tokens > 1 ? ldx : n_cols,
                                     (int32_t)n_tokens, y, n_tokens > 1 ? ldy : n_rows, stream, QMV_PATH_AUTO);
    } else {
        TileCall t{};
        t.W = static_cast<const uint8_t*>(W);
        t.rows = n_rows;
        t.cols = n_cols;
        t.n_items = n_tokens;
        t.n_groups = 1;
        t.top_k = 1;
        t.x = x;
        t.x_type = x_type;
        t.xs_tok = ldx;
        t.y = y;
        t.y_type = QMV_X_F32;
        t.ldy = ldy;
        rc = tile_product(fmt, t, st);
    }
    if (rc != QMV_OK) return rc;
    switch (a_type) {
    case QMV_X_F32: rc = shrink_x<float>(c, st); break;
    case QMV_X_F16: rc = shrink_x<_Float16>(c, st); break;
    default: rc = shrink_x<__bf16>(c, st);
    }
    if (rc != QMV_OK) return rc;
    switch (a_type) {
    case QMV_X_F32: return expand<float>(c, st);
    case QMV_X_F16: return expand<_Float16>(c, st);
    default: return expand<__bf16>(c, st);
    }
}
