// Entry points of attention over a quantized cache.
#include <cmath>

#include "qmv_attention.h"

namespace qmv {
namespace {

size_t round16(size_t n) { return (n + 15) & ~size_t(15); }

bool sizes_ok(const qmv_cache& c, int64_t R, int64_t T, int32_t heads, int64_t max_q) {
    return R >= 1 && R <= 65535 && T >= 1 && T <= (1 << 24) && heads >= 1 && heads % c.n_kv_heads == 0 &&
           heads / c.n_kv_heads <= 1024 && max_q >= 1 && max_q <= T && T * (heads / c.n_kv_heads) < (int64_t(1) << 31);
}
size_t stream_bytes(const qmv_cache& c, int64_t R, int32_t heads, int64_t max_q) {
    const int64_t rows = 16 * stream_tiles(max_q * (heads / c.n_kv_heads), c.head_dim);
    return round16((size_t)(R + 2) * 8) + (size_t)(2 * kAShares * rows * (c.head_dim + 2)) * 4;
}

// Rows of a request up to which the streaming kernel takes it.  Requests behind
// 900..4000 tokens, 8 key/value heads of 128, 8 query heads each, streaming and
// tile kernel: of 24 rows 16 requests 54 and 109 us, 64 142 and 240; of 32 rows 57 and
// 110, 149 and 230; of 40 rows 82 and 97, 254 and 230; of 64 rows 84 and 95,
// 258 and 228; of 128 rows 138 and 93, 479 and 232.  One request behind 8000, 4
// query heads each: 24 rows 30 and 26, 40 rows 35 and 28.  fp16 queries would
// go further: 40 rows 92 and 202, 307 and 542; 64 rows 95 and 194, 319 and 539;
// 128 rows 167 and 194, 612 and 581.
constexpr int kFewRows = 32;
// Parts that the tile kernel's tiles are split into over the keys, where there
// are fewer tiles than the GPU runs at once: a workgroup for each of 256 compute
// units.  With half as many, 200 tokens behind 8000 take 101 us for 68, 512
// behind 4000 102 for 69; small mixed steps less (54 us, 52).  At most 32: with 16,
// 64 tokens behind 30000 take 96 us for 68, with both limits many short ones
// the same (5 x 123 tokens 29 us, 29).
int tile_splits(const qmv_cache& c, int64_t T, int32_t heads, int64_t max_q, int32_t x_type) {
    const int64_t G = heads / c.n_kv_heads;
    if (max_q * G <= kFewRows) return 0;
    const int64_t rows = tile_rows(c.head_dim, x_type), tiles = c.n_kv_heads * ((T * G + rows - 1) / rows);
    return (int)std::min<int64_t>(std::max<int64_t>(1, 256 / tiles), 32);
}
// Room for the split tiles' rows.  The splits times the tiles are 256 at most, of
// 256 rows at most, and a row is split 32 times at most: a bound that grows
// with the sizes, as the splits themselves do not.
size_t tile_bytes(const qmv_cache& c, int64_t T, int32_t heads, int64_t max_q) {
    if (max_q * (heads / c.n_kv_heads) <= kFewRows) return 0;
    return round16((size_t)std::min<int64_t>(32 * T * heads, 256 * 256) * (c.head_dim + 2) * 4);
}

}  // namespace
}  // namespace qmv

extern "C" size_t qmv_cache_attention_workspace_bytes(const qmv_cache* cache, int64_t n_requests, int64_t n_tokens,
                                                      int32_t n_heads, int64_t max_q) {
    using namespace qmv;
    if (!cache || !qmv_cache_page_bytes(QMV_Q8_0, cache->n_kv_heads, cache->head_dim, cache->page_size) ||
        !sizes_ok(*cache, n_requests, n_tokens, n_heads, max_q))
        return 0;
    return stream_bytes(*cache, n_requests, n_heads, max_q) + tile_bytes(*cache, n_tokens, n_heads, max_q);
}

extern "C" int32_t qmv_cache_attention(const qmv_cache* cache, const void* q, int32_t x_type, int64_t q_stride_token,
                                       int64_t q_stride_head, int64_t n_tokens, int32_t n_heads, const int32_t* page_table,
                                       int64_t max_pages, const int32_t* kv_lens, const int32_t* q_begin,
                                       int64_t n_requests, int64_t max_q, float scale, int32_t window, const float* sinks,
                                       void* out, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace qmv;
    const char* name = "qmv_cache_attention";
    if (const int32_t e = check_cache(name, cache)) return e;
    if (!q || !page_table || !kv_lens || !out || !workspace) return fail(QMV_EINVAL, "%s: null pointer", name);
    const int xe = type_bytes(x_type);
    if (!xe) return fail(QMV_EINVAL, "%s: unknown x_type %d", name, (int)x_type);
    if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 || n_heads / cache->n_kv_heads > 1024)
        return fail(QMV_EINVAL, "%s: n_heads must be a multiple of n_kv_heads, at most 1024 times as many", name);
    if (!sizes_ok(*cache, n_requests, n_tokens, n_heads, max_q))
        return fail(QMV_EINVAL, "%s: n_requests must be 1..65535, n_tokens 1..2^24 (times n_heads / n_kv_heads below 2^31), max_q "
                                "1..n_tokens", name);
    if (!q_begin && n_requests * max_q != n_tokens)
        return fail(QMV_EINVAL, "%s: without q_begin, n_tokens must be n_requests * max_q", name);
    if (max_pages < 1 || max_pages > (int64_t(1) << 30) / cache->page_size)
        return fail(QMV_EINVAL, "%s: max_pages must be >= 1 with max_pages * page_size <= 2^30", name);
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(QMV_EINVAL, "%s: scale must be finite and > 0", name);
    if (window < 0) return fail(QMV_EINVAL, "%s: window must be >= 0", name);
    if (n_heads > 1 && q_stride_head < cache->head_dim)
        return fail(QMV_EINVAL, "%s: the stride per head must be >= head_dim", name);
    const size_t need = qmv_cache_attention_workspace_bytes(cache, n_requests, n_tokens, n_heads, max_q);
    if (workspace_bytes < need)
        return fail(QMV_EINVAL, "%s: the workspace needs %zu bytes, got %zu", name, need, workspace_bytes);
    if (!aligned(q, xe) || !aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(q_begin, 4) || !aligned(sinks, 4) ||
        !aligned(out, 16) || !aligned(workspace, 16))
        return fail(QMV_EALIGN, "%s: a pointer is not aligned to its elements (out and workspace: 16 bytes)", name);
    AttnArgs a{};
    a.k = cache_side(*cache, true);
    a.v = cache_side(*cache, false);
    a.n_pages = cache->n_pages;
    a.page_shift = log2_of(cache->page_size);
    a.H = cache->n_kv_heads;
    a.G = n_heads / cache->n_kv_heads;
    a.g_shift = a.G > 1 ? 32 - __builtin_clz(a.G - 1) : 0;
    a.g_mul = (uint32_t)(((uint64_t(1) << (31 + a.g_shift)) + a.G - 1) / a.G);
    a.R = (int32_t)n_requests;
    a.q = q;
    a.qst = q_stride_token;
    a.qsh = n_heads > 1 ? q_stride_head : 0;
    a.qvec = aligned(q, 16) && (a.qst * xe) % 16 == 0 && (a.qsh * xe) % 16 == 0;
    a.n_tokens = n_tokens;
    a.max_q = max_q;
    a.table = page_table;
    a.max_pages = max_pages;
    a.lens = kv_lens;
    a.q_begin = q_begin;
    a.scale = scale;
    a.window = window > (1 << 30) ? 1 << 30 : window;
    a.sinks = sinks;
    a.out = out;
    a.x_type = x_type;
    a.prefix = static_cast<int64_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + round16((size_t)(n_requests + 2) * 8));
    const hipStream_t st = as_stream(stream);
    a.tile_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + stream_bytes(*cache, n_requests, n_heads, max_q));
    const bool two = x_type != QMV_X_BF16;
    const int splits = tile_splits(*cache, n_tokens, n_heads, max_q, x_type);
    // of many requests some may be short; one that may be long goes the one way
    const bool both = splits > 0 && n_requests > 1;
    a.stream_to = both ? kFewRows : INT32_MAX;
    a.tile_over = both ? kFewRows : 0;
    if (splits > 0) {
        const int32_t e = two ? attn_tile_2(a, cache->head_dim, splits, st) : attn_tile_1(a, cache->head_dim, splits, st);
        if (e != QMV_OK || !both || a.G > kFewRows) return e;
    }
    switch (cache->k_fmt) {
    case QMV_Q8_0: return two ? attn_stream_q8_0_2(a, cache->head_dim, st) : attn_stream_q8_0_1(a, cache->head_dim, st);
    case QMV_Q4_0: return two ? attn_stream_q4_0_2(a, cache->head_dim, st) : attn_stream_q4_0_1(a, cache->head_dim, st);
    default: return two ? attn_stream_q4_1_2(a, cache->head_dim, st) : attn_stream_q4_1_1(a, cache->head_dim, st);
    }
}
