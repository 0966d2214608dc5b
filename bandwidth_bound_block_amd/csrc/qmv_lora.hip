// A projection of shared quantized weights with a low-rank adapter per token:
// y_t = DEQ(W) x_t + s_a B_a (A_a x_t), a = adapter_ids[t].
//
// The base product is the library's own: the matvec kernels up to 8 tokens,
// the tile kernel past that.  The adapters are two narrow products in fp32
// accuracy: v_t = s_a A_a x_t by one launch, in parts of the columns, and
// y_t += B_a v_t, in the tile kernel's last step or (up to 8 tokens) by a
// launch of its own.
//
// 4096 x 4096 Q4_0, 1 token, rank 16: 4 + 5 + 4 us, all latency.  8 tokens of
// 8 adapters, fp32, 6144 x 4096 Q8_0: 6 + 20 + 4, the FMA matvec's 8 columns.
// 101 tokens of 40 requests, 4096 x 14336 Q4_K, rank 8: 14 for v (each
// workgroup's adapters one after the other) and 92 for the tiles.
#include <algorithm>

#include "qmv_tile.h"

namespace qmv {
namespace {

// Operands of the narrow products as MFMA pieces: fp16 by fp16 in its own
// type; otherwise bf16 pieces that hold the value to 24 bits (fp16: two, its
// 11 bits exactly).
template <class T, bool F16> struct Piece;
template <bool F16> struct Piece<__bf16, F16> {
    static constexpr int kN = 1;
    __device__ static void of(const X8<__bf16>& x, u32x4 (&p)[1]) { p[0] = x.v; }
};
template <> struct Piece<_Float16, true> {
    static constexpr int kN = 1;
    __device__ static void of(const X8<_Float16>& x, u32x4 (&p)[1]) { p[0] = x.v; }
};
template <> struct Piece<_Float16, false> {
    static constexpr int kN = 2;
    __device__ static void of(const X8<_Float16>& x, u32x4 (&p)[2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = half_bits_to_float(x.v[i]), b = half_bits_to_float(x.v[i] >> 16);
            const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
            p[0][i] = h;
            p[1][i] = XOp<__bf16>::pair(a - __builtin_bit_cast(float, h << 16),
                                        b - __builtin_bit_cast(float, h & 0xffff0000u));
        }
    }
};
template <bool F16> struct Piece<float, F16> {
    static constexpr int kN = 3;
    __device__ static void of(const X8<float>& x, u32x4 (&p)[3]) { x.pieces(p); }
};

// The sum of x[k] a[k] over a part's columns: 512 of every 512 * parts.
template <class XT, class AT>
__device__ __forceinline__ float part_sum(const XT* x, const AT* a, int64_t K, int part, int parts) {
    float s = 0.f;
    for (int64_t c0 = 512 * part; c0 < K; c0 += 512 * parts)
#pragma unroll 8
        for (int64_t c = c0; c < min(c0 + 512, K); ++c) s = __builtin_fmaf(XIn<XT>::load1(x + c), XIn<AT>::load1(a + c), s);
    return s;
}

// v[part][t][r] = scales[a] * sum over the part's columns of A[a][r][k] x[t][k].
// A workgroup takes 32 tokens and a part of the columns; its four waves take
// groups of 128 columns in turn, and the sums of an adapter's rows with all
// 32 tokens are kept for its own tokens.  Workgroup z of gridDim.z takes
// every gridDim.z-th of the adapters among the tokens.  RT: rank rows in 32s.
template <class XT, class AT, int RT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const XT* __restrict__ x, int64_t ldx,
                                                          const AT* __restrict__ A, const float* __restrict__ scales,
                                                          const int32_t* __restrict__ ids, int T, int n_adapters,
                                                          int rank, int nb, int xvec, int avec, float* __restrict__ v) {
    constexpr bool kF16 = std::is_same<XT, _Float16>::value && std::is_same<AT, _Float16>::value;
    using PX = Piece<XT, kF16>;
    using PA = Piece<AT, kF16>;
    using Op = typename std::conditional<kF16, XOp<_Float16>, XOp<__bf16>>::type;
    __shared__ float red[4][32][32 * RT + 1];
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int part = blockIdx.y, parts = gridDim.y;
    const int t0 = blockIdx.x * 32, count = min(32, T - t0);
    const int tok = t0 + min(lr, count - 1);
    const int id = ids[tok];
    const XT* xr = x + tok * ldx + 8 * lh;
    const int64_t K = 32 * (int64_t)nb;
    uint32_t todo = (uint32_t)__ballot(lr < count && (unsigned)id < (unsigned)n_adapters);
    for (unsigned turn = 0; todo; ++turn) {
        const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t own = (uint32_t)__ballot(id == ad) & todo;
        todo &= ~own;
        if (turn % gridDim.z != blockIdx.z) continue;
        const AT* ar[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) ar[r] = A + ((int64_t)ad * rank + min(32 * r + lr, rank - 1)) * K + 8 * lh;
        f32x16 acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[r][i] = 0.f;
        for (int g = part * 4 + wave; 4 * g < nb; g += 4 * parts) {
            X8<XT> xv[8];
            X8<AT> av[RT][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // sixteens of columns; past the row the last ones, as zeros
                const int c = 128 * g + 16 * j;
                const int at = min(c, (int)K - 16);
                xv[j].load(xr + at, xvec);
                if (c >= K) xv[j].zero();
#pragma unroll
                for (int r = 0; r < RT; ++r) av[r][j].load(ar[r] + at, avec);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u32x4 px[PX::kN];
                PX::of(xv[j], px);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    u32x4 pa[PA::kN];
                    PA::of(av[r][j], pa);
#pragma unroll
                    for (int k = PX::kN - 1; k >= 0; --k)
#pragma unroll
                        for (int m = PA::kN - 1; m >= 0; --m)
                            if (k + m <= 2) acc[r] = Op::mfma(px[k], pa[m], acc[r]);
                }
            }
        }
        __syncthreads();          // the last adapter's sums are read
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) red[wave][8 * (i >> 2) + 4 * lh + (i & 3)][32 * r + lr] = acc[r][i];
        __syncthreads();
        const float sc = scales[ad];
        for (int i = tid; i < 32 * rank; i += 256) {
            const int j = i / rank, r = i % rank;
            if (!(own >> j & 1)) continue;
            float s = (red[0][j][r] + red[1][j][r]) + (red[2][j][r] + red[3][j][r]);
            // an infinity's pieces are NaN: its products one by one
            if (!(__builtin_fabsf(s) < __builtin_inff()))
                s = part_sum<XT, AT>(x + (int64_t)(t0 + j) * ldx, A + ((int64_t)ad * rank + r) * K, K, part, parts);
            v[((int64_t)part * T + t0 + j) * rank + r] = sc * s;
        }
    }
}

// Sum of a row's weights times x, one by one.
template <class F, class XT>
__device__ float row_sum(const uint8_t* W, int64_t n, int nb, const XT* x) {
    const uint8_t* row = W + n * (int64_t)(nb / 8 * Unit<F>::kRow + nb % 8 * (Unit<F>::kRow / 8));
    float s = 0.f;
    for (int b = 0; b < nb && s == s; ++b)
#pragma unroll 8
        for (int c = 32 * b; c < 32 * b + 32; ++c) s = __builtin_fmaf(Unit<F>::weight(row, c), XIn<XT>::load1(x + c), s);
    return s;
}

// y[t][n] += sum_r B[a][n][r] v[t][r]; NaN for an id that is no adapter.  A
// base sum that is not finite (an infinite activation's pieces are NaN in the
// matrix-core matvec) is computed again first.
template <class F, class AT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const AT* __restrict__ B, const int32_t* __restrict__ ids,
                                                          int n_adapters, int rank, int parts, int T, int N, int vec,
                                                          const float* __restrict__ v, float* __restrict__ y,
                                                          int64_t ldy, const uint8_t* __restrict__ W, int nb,
                                                          const void* __restrict__ x, int x_type, int64_t ldx) {
    __shared__ float sv[128];
    const int t = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x;
    const int a = ids[t];
    const bool good = (unsigned)a < (unsigned)n_adapters;
    if (good && (int)threadIdx.x < rank) {
        float s = 0.f;
        for (int p = 0; p < parts; ++p) s += v[((int64_t)p * T + t) * rank + threadIdx.x];
        sv[threadIdx.x] = s;
    }
    __syncthreads();
    if (n >= N) return;
    float* o = y + t * ldy + n;
    if (!good && a != -1) {
        *o = __builtin_nanf("");
        return;
    }
    float s = 0.f;
    if (good) {
        const AT* b = B + ((int64_t)a * N + n) * rank;
        if (vec) {
            for (int r = 0; r < rank; r += 4) {
                const float4 w = XIn<AT>::load4(b + r);
                s = __builtin_fmaf(w.x, sv[r], s);
                s = __builtin_fmaf(w.y, sv[r + 1], s);
                s = __builtin_fmaf(w.z, sv[r + 2], s);
                s = __builtin_fmaf(w.w, sv[r + 3], s);
            }
        } else {
            for (int r = 0; r < rank; ++r) s = __builtin_fmaf(XIn<AT>::load1(b + r), sv[r], s);
        }
    }
    float base = *o;
    if (!(__builtin_fabsf(base) < __builtin_inff())) {
        base = x_type == QMV_X_F32   ? row_sum<F, float>(W, n, nb, static_cast<const float*>(x) + t * ldx)
               : x_type == QMV_X_F16 ? row_sum<F, _Float16>(W, n, nb, static_cast<const _Float16*>(x) + t * ldx)
                                     : row_sum<F, __bf16>(W, n, nb, static_cast<const __bf16*>(x) + t * ldx);
    } else if (a == -1) {
        return;
    }
    *o = base + s;
}

struct LoraCall {
    const void *W, *x;
    int32_t x_type;
    int64_t ldx, T, N, K;
    const void *A, *B;
    int32_t a_type, n_adapters, rank, parts;
    const float* scales;
    const int32_t* ids;
    float* y;
    int64_t ldy;
    float* v;
};

// Parts of the columns: enough workgroups for the GPU where there are few
// tokens, and at least one group of 128 columns for every wave.
int lora_parts(int64_t T, int64_t K) {
    const int64_t tiles = (T + 31) / 32, most = (K + 511) / 512;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, most), 128 / tiles));
}

template <class XT, class AT, int RT>
int32_t shrink(const LoraCall& c, hipStream_t st) {
    const int xvec = aligned(c.x, 16) && c.ldx % (16 / (int)sizeof(XT)) == 0, avec = aligned(c.A, 16);
    const int64_t tiles = (c.T + 31) / 32;
    // adapters side by side, up to about 1024 workgroups in all
    const int64_t most = std::min<int64_t>(std::min<int64_t>(32, c.T), c.n_adapters);
    const unsigned side = (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, 1024 / (tiles * c.parts)));
    hipLaunchKernelGGL((lora_shrink_kernel<XT, AT, RT>), dim3((unsigned)tiles, (unsigned)c.parts, side), dim3(256), 0, st,
                       (const XT*)c.x, c.ldx, (const AT*)c.A, c.scales, c.ids, (int)c.T, c.n_adapters, c.rank,
                       (int)(c.K / 32), xvec, avec, c.v);
    return check_launch("qmv_lora");
}
template <class XT, class AT>
int32_t shrink_r(const LoraCall& c, hipStream_t st) {
    if (c.rank <= 32) return shrink<XT, AT, 1>(c, st);
    if (c.rank <= 64) return shrink<XT, AT, 2>(c, st);
    return shrink<XT, AT, 4>(c, st);
}
template <class AT>
int32_t shrink_x(const LoraCall& c, hipStream_t st) {
    switch (c.x_type) {
    case QMV_X_F32: return shrink_r<float, AT>(c, st);
    case QMV_X_F16: return shrink_r<_Float16, AT>(c, st);
    default: return shrink_r<__bf16, AT>(c, st);
    }
}
template <class F, class AT>
int32_t expand_f(const LoraCall& c, hipStream_t st) {
    const int vec = c.rank % 4 == 0 && aligned(c.B, XIn<AT>::kVecAlign);
    hipLaunchKernelGGL((lora_expand_kernel<F, AT>), dim3((unsigned)c.T, (unsigned)((c.N + 255) / 256)), dim3(256), 0, st,
                       (const AT*)c.B, c.ids, c.n_adapters, c.rank, c.parts, (int)c.T, (int)c.N, vec, c.v, c.y, c.ldy,
                       (const uint8_t*)c.W, (int)(c.K / 32), c.x, c.x_type, c.ldx);
    return check_launch("qmv_lora");
}
template <class AT>
int32_t expand(qmv_fmt fmt, const LoraCall& c, hipStream_t st) {
    switch (fmt) {
    case QMV_Q8_0: return expand_f<Q8_0, AT>(c, st);
    case QMV_Q4_0: return expand_f<Q4_0, AT>(c, st);
    case QMV_Q4_1: return expand_f<Q4_1, AT>(c, st);
    case QMV_Q4_K: return expand_f<Q4KTile, AT>(c, st);
    default: return expand_f<Q6KTile, AT>(c, st);
    }
}

constexpr int64_t kLoraTokens = 1 << 20;
constexpr int64_t kMatvecTokens = 8, kMatvecCols = 35424;     // the base is the matvec, whose rows have to fit LDS
constexpr int64_t kTileCols = 1 << 24;
constexpr int kLoraRank = 128, kLoraAdapters = 1024;

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_lora_workspace_bytes(int64_t n_tokens, int32_t rank, int32_t n_adapters) {
    using namespace qmv;
    if (n_tokens < 1 || n_tokens > kLoraTokens || rank < 1 || rank > kLoraRank || n_adapters < 1 ||
        n_adapters > kLoraAdapters)
        return 0;
    // v in at most as many parts as the longest rows have
    return (size_t)n_tokens * rank * 4 * lora_parts(n_tokens, kTileCols);
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
    if (n_tokens < 1 || n_tokens > kLoraTokens) return fail(QMV_EINVAL, "%s: n_tokens must be 1..2^20", name);
    const int64_t most_cols = n_tokens > kMatvecTokens ? kTileCols : kMatvecCols;
    if (n_cols < uw || n_cols % uw || n_cols > most_cols)
        return fail(QMV_EINVAL, "%s: n_cols must be a multiple of %d in %d..%lld for %lld tokens", name, uw, uw,
                    (long long)most_cols, (long long)n_tokens);
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
    LoraCall c{W, x, x_type, ldx, n_tokens, n_rows, n_cols, A, B, a_type, n_adapters, rank, lora_parts(n_tokens, n_cols),
               scales, adapter_ids, y, ldy, static_cast<float*>(workspace)};
    int32_t rc;
    switch (a_type) {
    case QMV_X_F32: rc = shrink_x<float>(c, st); break;
    case QMV_X_F16: rc = shrink_x<_Float16>(c, st); break;
    default: rc = shrink_x<__bf16>(c, st);
    }
    if (rc != QMV_OK) return rc;
    if (n_tokens > kMatvecTokens) {
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
        t.lora = LoraTile{B, adapter_ids, c.v, a_type, n_adapters, rank, c.parts,
                          a_type != QMV_X_F32 && rank % 8 == 0 && aligned(B, 16)};
        return tile_product(fmt, t, st);
    }
    // fp32 activations by the FMA kernels: the matrix-core matvec holds them
    // to 16 bits only
    rc = format_ops(fmt)->matvec(name, W, n_rows, n_cols, x, x_type, n_tokens > 1 ? ldx : n_cols, (int32_t)n_tokens, y,
                                 n_tokens > 1 ? ldy : n_rows, stream, x_type == QMV_X_F32 ? QMV_PATH_FMA : QMV_PATH_AUTO);
    if (rc != QMV_OK) return rc;
    switch (a_type) {
    case QMV_X_F32: return expand<float>(fmt, c, st);
    case QMV_X_F16: return expand<_Float16>(fmt, c, st);
    default: return expand<__bf16>(fmt, c, st);
    }
}
