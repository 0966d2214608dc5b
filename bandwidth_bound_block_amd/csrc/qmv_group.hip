// Products grouped by expert for any number of tokens: the plan (a stable
// counting sort of the (token, slot) items by group), the entry points of the
// tiled product, and the weighted sum over a token's slots.
#include <algorithm>

#include "qmv_block_decode.h"
#include "qmv_group.h"

namespace qmv {

// One plan serves every product of its routing, of any format and activation
// type; their borders lie apart, and 48 between them.  Routed at random, tiles
// of 32 / of 128: 128 experts of 1536 x 2048, 48 and 64 tokens each on average,
// bf16: Q4_0 122 / 129 and 149 / 137 us, Q8_0 191 / 169 and 223 / 175, Q4_K 156
// / 177 and 184 / 183, Q6_K 193 / 268 and 247 / 272; fp32: Q4_0 404 / 193 and
// 457 / 260.  8 experts of 4096 x 4096: Q4_0 46 / 64 and 56 / 65, Q8_0 54 / 72
// and 86 / 74, Q6_K 75 / 117 and 98 / 118; fp32: Q4_0 125 / 72.  32 experts of
// 1536 x 2048, 32 and 40 tokens each: Q4_0 34 / 43 and 32 / 44, Q8_0 50 / 51
// and 52 / 52, Q6_K 51 / 80 and 53 / 81.
int plan_tile(int64_t n_items, int n_groups) { return n_items >= 48 * (int64_t)n_groups ? 128 : 32; }

bool fmt_unit(qmv_fmt fmt, int* weights, int* bytes) {
    switch (fmt) {
    case QMV_Q8_0: *weights = 32; *bytes = 34; return true;
    case QMV_Q4_0: *weights = 32; *bytes = 18; return true;
    case QMV_Q4_1: *weights = 32; *bytes = 20; return true;
    case QMV_Q4_K: *weights = 256; *bytes = 144; return true;
    case QMV_Q6_K: *weights = 256; *bytes = 210; return true;
    default: return false;
    }
}

int32_t tile_product(qmv_fmt fmt, const TileCall& c, hipStream_t st) {
    switch (fmt) {
    case QMV_Q8_0: return tile_q8_0(c, st);
    case QMV_Q4_0: return tile_q4_0(c, st);
    case QMV_Q4_1: return tile_q4_1(c, st);
    case QMV_Q4_K: return tile_q4_k(c, st);
    default: return tile_q6_k(c, st);
    }
}

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanWgs = 64;             // at most: each reads all ids

// Inclusive scan over the workgroup; `part` holds kPlanWaves ints.
__device__ __forceinline__ int scan_wg(int v, int* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 63) part[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += part[w];
    return v;
}

// The plan.  A workgroup counts all items by group and puts down its own
// chunk of them, so nothing is passed between workgroups (one alone is bound
// by its ballots).  Of the chunk
// a wave has a run of neighbouring items.  Groups in turn, within a group the
// chunks and the waves in turn, give the wave its first places; it puts its
// items down 64 at a time, after those of their group it has put before and
// those in lower lanes (found with one ballot per id bit).  So the order
// within a group is the items' own, and the plan's bits do not depend on
// timing.  128 groups: 72 items 4.7 us, 4096 6.7, 16384 8.8 (by one workgroup
// 7.5 and 18); 65536 items of 256 groups 15.6 (63).
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t* __restrict__ ids, int n, int E, int tile,
                                                            int tiles_at, int order_at, int32_t* __restrict__ plan) {
    extern __shared__ int sh[];
    const int G = E + 1;
    int* base = sh;                        // [G] items before the chunk, then the chunk's first places
    int* all = sh + G;                     // [G] items after it, then all
    int* wcnt = sh + 2 * G;                // [waves][G] a wave's items, then places used by earlier waves and this one
    __shared__ int part[kPlanWaves];
    constexpr int kAhead = 8;              // loads of a lane on their way
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int k = tid; k < (kPlanWaves + 2) * G; k += kPlanThreads) sh[k] = 0;
    __syncthreads();
    int* mine = wcnt + wave * G;
    // chunk and run are whole ballots
    const int run = (n + gridDim.x * kPlanThreads - 1) / (gridDim.x * kPlanThreads) * 64;
    const int c0 = (int)min((int64_t)n, (int64_t)blockIdx.x * run * kPlanWaves);
    const int c1 = min(n, c0 + run * kPlanWaves);
    const int i0 = min(c1, c0 + wave * run), i1 = min(c1, i0 + run);
    int id[kAhead];
    // `step` apart from i + the thread's own; those from `to` on are not read
    auto load = [&](int i, int step, int to) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const unsigned v = i + step * k < to ? (unsigned)ids[i + step * k] : 0u;
            id[k] = v < (unsigned)E ? (int)v : E;
        }
    };
    auto count = [&](int* into, int from, int to, int step) __attribute__((always_inline)) {
        for (int i = from; i < to; i += step * kAhead) {
            load(i, step, to);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i + step * k < to) atomicAdd(&into[id[k]], 1);
        }
    };
    count(base, tid, c0, kPlanThreads);
    count(all, c1 + tid, n, kPlanThreads);
    count(mine, i0 + lane, i1, 64);
    __syncthreads();
    for (int g = tid; g < G; g += kPlanThreads) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = wcnt[w * G + g];
            wcnt[w * G + g] = s;
            s += c;
        }
        all[g] += base[g] + s;
    }
    __syncthreads();
    // offsets and tiles; at most 1025 groups: one per thread, and the last
    // group (no group's items) by the scan's total
    const int c = tid < E ? all[tid] : 0;
    const int t = (c + tile - 1) / tile;
    const int end = scan_wg(c, part);
    const int tend = scan_wg(t, part);
    const int bad = all[E];
    int32_t* offs = plan + kPlanHeader;
    int4* tl = reinterpret_cast<int4*>(plan + tiles_at);
    __syncthreads();
    const bool lists = blockIdx.x == 0;
    if (tid < E) base[tid] += end - c;
    if (tid == kPlanThreads - 1) base[E] += end;      // holds the totals over the groups
    if (lists && tid < E) {
        offs[tid] = end - c;
        for (int k = 0; k < t; ++k)
            tl[tend - t + k] = int4{tid, end - c + k * tile, min(tile, c - k * tile), 0};
    }
    if (lists && tid == kPlanThreads - 1) {
        offs[E] = end;
        offs[E + 1] = n;
        const int tb = (bad + tile - 1) / tile;
        for (int k = 0; k < tb; ++k) tl[tend + k] = int4{E, end + k * tile, min(tile, bad - k * tile), 0};
        plan[0] = kPlanMagic;
        plan[1] = n;
        plan[2] = E;
        plan[3] = tile;
        plan[4] = tend + tb;
    }
    __syncthreads();
    int bits = 1;
    while ((1 << bits) < G) ++bits;
    for (int i = i0; i < i1; i += 64 * kAhead) {
        load(i + lane, 64, i1);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + 64 * k >= i1) break;
            const int at = i + 64 * k + lane;
            const bool in = at < i1;
            uint64_t same = __ballot(in);
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot((id[k] >> b) & 1);
                same &= (id[k] >> b) & 1 ? m : ~m;
            }
            const int below = __popcll(same & ((1ull << lane) - 1));
            if (in) plan[order_at + base[id[k]] + mine[id[k]] + below] = at;
            // every lane has read its group's count before one adds to it
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (in && below == 0) mine[id[k]] += __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// out[t][n] = sum_s w[t][s] y[t][s][n], an fp32 fused multiply-add chain in
// slot order; four columns a thread, in turns where a launch's threads (2^32)
// do not reach.
template <class YT>
__device__ __forceinline__ float4 y4(const YT* p, int left, bool vec) {
    if (vec) return XIn<YT>::load4(p);
    float4 v = {0.f, 0.f, 0.f, 0.f};
    v.x = XIn<YT>::load1(p);
    if (left > 1) v.y = XIn<YT>::load1(p + 1);
    if (left > 2) v.z = XIn<YT>::load1(p + 2);
    if (left > 3) v.w = XIn<YT>::load1(p + 3);
    return v;
}
template <class OT> __device__ __forceinline__ OT narrow(float v) { return (OT)v; }

template <class YT, class OT>
__global__ __launch_bounds__(256) void weighted_sum_kernel(const YT* __restrict__ y, const float* __restrict__ w,
                                                           int64_t tokens, int top_k, int64_t n, int64_t quads,
                                                           OT* __restrict__ out, int vec) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < tokens * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / quads, c = 4 * (i - t * quads);
        const int left = (int)min((int64_t)4, n - c);
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < top_k; ++s) {
            const float4 v = y4<YT>(y + (t * top_k + s) * n + c, left, vec);
            const float f = w[t * top_k + s];
            a[0] = __builtin_fmaf(f, v.x, a[0]);
            a[1] = __builtin_fmaf(f, v.y, a[1]);
            a[2] = __builtin_fmaf(f, v.z, a[2]);
            a[3] = __builtin_fmaf(f, v.w, a[3]);
        }
        for (int k = 0; k < left; ++k) out[t * n + c + k] = narrow<OT>(a[k]);
    }
}

template <class YT>
int32_t launch_sum(const YT* y, const float* w, int64_t T, int S, int64_t n, void* out, int32_t ot, hipStream_t st) {
    const int64_t quads = (n + 3) / 4, blocks = std::min<int64_t>((T * quads + 255) / 256, 0xffffffff / 256);
    const int vec = n % 4 == 0 && aligned(y, XIn<YT>::kVecAlign);
    const dim3 g((unsigned)blocks), b(256);
    switch (ot) {
    case QMV_X_F32:
        hipLaunchKernelGGL((weighted_sum_kernel<YT, float>), g, b, 0, st, y, w, T, S, n, quads, (float*)out, vec);
        break;
    case QMV_X_F16:
        hipLaunchKernelGGL((weighted_sum_kernel<YT, _Float16>), g, b, 0, st, y, w, T, S, n, quads, (_Float16*)out, vec);
        break;
    default:
        hipLaunchKernelGGL((weighted_sum_kernel<YT, __bf16>), g, b, 0, st, y, w, T, S, n, quads, (__bf16*)out, vec);
    }
    return check_launch("qmv_moe_weighted_sum");
}

bool plan_sizes_ok(int64_t n_items, int32_t n_groups) {
    return n_items >= 1 && n_items <= kMaxItems && n_groups >= 1 && n_groups <= kMaxGroups;
}

int32_t grouped_entry(const char* name, bool swiglu, qmv_fmt fmt, const void* W, int64_t estride, int32_t E,
                      int64_t rows, int64_t cols, const void* plan, int64_t T, int32_t S, const void* x,
                      int32_t x_type, int64_t xs_tok, int64_t xs_slot, void* y, int32_t y_type, void* stream) {
    int uw, ub;
    if (!fmt_unit(fmt, &uw, &ub)) return fail(QMV_EUNSUPPORTED, "%s: unknown format %d", name, (int)fmt);
    if (!W || !plan || !x || !y) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (!x_type_ok(x_type)) return fail(QMV_EINVAL, "%s: unknown x_type %d", name, (int)x_type);
    if (!x_type_ok(y_type)) return fail(QMV_EINVAL, "%s: unknown output type %d", name, (int)y_type);
    if (E < 1 || E > kMaxGroups) return fail(QMV_EINVAL, "%s: n_experts must be 1..%d, got %d", name, kMaxGroups, (int)E);
    if (rows < 1 || rows > (1 << 28)) return fail(QMV_EINVAL, "%s: n_rows must be 1..2^28", name);
    if (cols < uw || cols % uw || cols > (1 << 24))
        return fail(QMV_EINVAL, "%s: n_cols must be a multiple of %d in %d..2^24", name, uw, uw);
    if (T < 1 || S < 1 || S > 1024 || T > kMaxItems / S)
        return fail(QMV_EINVAL, "%s: n_tokens * top_k must be 1..2^24 with top_k 1..1024", name);
    const int64_t need = (swiglu ? 2 : 1) * rows * (cols / uw * ub);
    if (E > 1 && estride < need)
        return fail(QMV_EINVAL, "%s: expert_stride_bytes %lld is less than an expert's %lld bytes", name,
                    (long long)estride, (long long)need);
    if (T > 1 && xs_tok < cols) return fail(QMV_EINVAL, "%s: x_stride_token is less than n_cols", name);
    if (xs_slot != 0 && xs_slot < cols) return fail(QMV_EINVAL, "%s: x_stride_slot must be 0 or >= n_cols", name);
    const int wa = fmt_align(fmt), sa = fmt_stride_align(fmt);
    if (!aligned(W, wa) || (E > 1 && estride % sa))
        return fail(QMV_EALIGN, "%s: W must be %d-byte aligned and expert_stride_bytes a multiple of %d", name, wa, sa);
    if (!aligned(plan, 16)) return fail(QMV_EALIGN, "%s: plan must be 16-byte aligned", name);
    if (!aligned(x, x_elem(x_type)) || !aligned(y, x_elem(y_type)))
        return fail(QMV_EALIGN, "%s: x and the output must be aligned to their element size", name);
    TileCall c{};
    c.W = static_cast<const uint8_t*>(W);
    c.estride = E > 1 ? estride : 0;
    c.rows = rows;
    c.cols = cols;
    c.plan = static_cast<const int32_t*>(plan);
    c.n_items = T * S;
    c.n_groups = E;
    c.top_k = S;
    c.x = x;
    c.x_type = x_type;
    c.xs_tok = xs_tok;
    c.xs_slot = xs_slot;
    c.y = y;
    c.y_type = y_type;
    c.ldy = rows;
    c.swiglu = swiglu;
    return tile_product(fmt, c, as_stream(stream));
}

int32_t make_plan(const char* name, const int32_t* ids, int64_t n, int32_t E, int32_t* plan, hipStream_t st) {
    const size_t lds = sizeof(int) * (size_t)(E + 1) * (kPlanWaves + 2);
    size_t dyn_max = 0;
    if (const int32_t e = lds_limit(reinterpret_cast<const void*>(plan_kernel), kLdsMax, name, &dyn_max)) return e;
    if (lds > dyn_max) return fail(QMV_EINVAL, "%s: %d groups exceed the LDS", name, (int)E);
    const unsigned wgs = (unsigned)std::min<int64_t>(kPlanWgs, (n + kPlanThreads - 1) / kPlanThreads);
    hipLaunchKernelGGL(plan_kernel, dim3(wgs), dim3(kPlanThreads), lds, st, ids, (int)n, (int)E, plan_tile(n, E),
                       (int)plan_tiles_at(E), (int)plan_order_at(n, E), plan);
    return check_launch(name);
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_group_plan_bytes(int64_t n_items, int32_t n_groups) {
    if (!qmv::plan_sizes_ok(n_items, n_groups)) return 0;
    return 4 * (size_t)(qmv::plan_order_at(n_items, n_groups) + n_items);
}

extern "C" int32_t qmv_group_plan(const int32_t* group_ids, int64_t n_items, int32_t n_groups, void* plan,
                                  size_t plan_bytes, void* stream) {
    using namespace qmv;
    const char* name = "qmv_group_plan";
    if (!group_ids || !plan) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (!plan_sizes_ok(n_items, n_groups))
        return fail(QMV_EINVAL, "%s: n_items must be 1..2^24 and n_groups 1..%d", name, kMaxGroups);
    if (plan_bytes < qmv_group_plan_bytes(n_items, n_groups))
        return fail(QMV_EINVAL, "%s: the plan needs %zu bytes, got %zu", name, qmv_group_plan_bytes(n_items, n_groups),
                    plan_bytes);
    if (!aligned(group_ids, 4) || !aligned(plan, 16))
        return fail(QMV_EALIGN, "%s: group_ids must be 4-byte and plan 16-byte aligned", name);
    return make_plan(name, group_ids, n_items, n_groups, static_cast<int32_t*>(plan), as_stream(stream));
}

extern "C" int32_t qmv_moe_grouped(qmv_fmt fmt, const void* W_experts, int64_t expert_stride_bytes, int32_t n_experts,
                                   int64_t n_rows, int64_t n_cols, const void* plan, int64_t n_tokens, int32_t top_k,
                                   const void* x, int32_t x_type, int64_t x_stride_token, int64_t x_stride_slot,
                                   void* y, int32_t y_type, void* stream) {
    return qmv::grouped_entry("qmv_moe_grouped", false, fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols,
                              plan, n_tokens, top_k, x, x_type, x_stride_token, x_stride_slot, y, y_type, stream);
}

extern "C" int32_t qmv_moe_grouped_swiglu(qmv_fmt fmt, const void* W_experts, int64_t expert_stride_bytes,
                                          int32_t n_experts, int64_t n_ff, int64_t n_cols, const void* plan,
                                          int64_t n_tokens, int32_t top_k, const void* x, int32_t x_type,
                                          int64_t x_stride_token, int64_t x_stride_slot, void* h, int32_t h_type,
                                          void* stream) {
    return qmv::grouped_entry("qmv_moe_grouped_swiglu", true, fmt, W_experts, expert_stride_bytes, n_experts, n_ff,
                              n_cols, plan, n_tokens, top_k, x, x_type, x_stride_token, x_stride_slot, h, h_type,
                              stream);
}

extern "C" int32_t qmv_moe_weighted_sum(const void* y, int32_t y_type, const float* weights, int64_t n_tokens,
                                        int32_t top_k, int64_t n_rows, void* out, int32_t out_type, void* stream) {
    using namespace qmv;
    const char* name = "qmv_moe_weighted_sum";
    if (!y || !weights || !out) return fail(QMV_EINVAL, "%s: null pointer", name);
    if (!x_type_ok(y_type) || !x_type_ok(out_type)) return fail(QMV_EINVAL, "%s: unknown element type", name);
    if (n_tokens < 1 || top_k < 1 || top_k > 1024 || n_tokens > kMaxItems / top_k)
        return fail(QMV_EINVAL, "%s: n_tokens * top_k must be 1..2^24 with top_k 1..1024", name);
    if (n_rows < 1 || n_rows > (1 << 28)) return fail(QMV_EINVAL, "%s: n_rows must be 1..2^28", name);
    if (!aligned(y, x_elem(y_type)) || !aligned(weights, 4) || !aligned(out, x_elem(out_type)))
        return fail(QMV_EALIGN, "%s: y, weights and out must be aligned to their element size", name);
    const hipStream_t st = as_stream(stream);
    switch (y_type) {
    case QMV_X_F32: return launch_sum((const float*)y, weights, n_tokens, top_k, n_rows, out, out_type, st);
    case QMV_X_F16: return launch_sum((const _Float16*)y, weights, n_tokens, top_k, n_rows, out, out_type, st);
    default: return launch_sum((const __bf16*)y, weights, n_tokens, top_k, n_rows, out, out_type, st);
    }
}
