// Host-side interface of the many-token products: the plan that sorts items
// by group and the tiled product that reads it.
#pragma once
#include "qmv_host.h"

namespace qmv {

// A plan in device memory, int32 words:
//   [0..7]   header: kPlanMagic, n_items, n_groups, tile, number of tiles
//   offsets  [n_groups + 2]: the items of group g are order[offsets[g]] up to
//            order[offsets[g + 1]]; group n_groups holds the items whose id
//            is no group
//   tiles    [4 * plan_tile_bound]: group, first place in order, items, 0
//   order    [n_items]: item indices by group, in item order within a group
constexpr int kPlanMagic = 0x716d7667;
constexpr int kPlanHeader = 8;
constexpr int kMaxGroups = 1024;
constexpr int64_t kMaxItems = 1 << 24;

// Tokens of a tile, from the mean items per group: both sides measured, see
// plan_tile in qmv_group.hip.
int plan_tile(int64_t n_items, int n_groups);
// No plan has more tiles: full ones, and a partial one per group with items.
inline int64_t plan_tile_bound(int64_t n_items, int n_groups, int tile) {
    const int64_t part = n_items < n_groups + 1 ? n_items : n_groups + 1;
    return n_items / tile + part;
}
inline int64_t plan_tiles_at(int n_groups) { return (kPlanHeader + n_groups + 2 + 3) / 4 * 4; }
inline int64_t plan_order_at(int64_t n_items, int n_groups) {
    return plan_tiles_at(n_groups) + 4 * plan_tile_bound(n_items, n_groups, plan_tile(n_items, n_groups));
}

// Low-rank adapters added to a product without a plan (rank 0: none): item t
// gains sum_r B[ids[t]][row][r] v[t][r], v summed over its parts.
struct LoraTile {
    const void* B;          // [n_adapters][rows][rank] of b_type
    const int32_t* ids;
    const float* v;         // [parts][n_items][rank]
    int32_t b_type, n_adapters, rank, parts;
    int32_t b16;            // 16-bit B whose rows may be read in 16-byte pieces of eight ranks
};

// One tiled product.  plan == nullptr: one matrix, the items are rows
// 0..n_items-1 of x (top_k = 1) and of y.
struct TileCall {
    const uint8_t* W;
    int64_t estride;      // bytes from one group's matrix to the next
    int64_t rows;         // output rows (with swiglu: half the matrix's rows)
    int64_t cols;
    const int32_t* plan;
    int64_t n_items;
    int n_groups;
    int top_k;
    const void* x;
    int32_t x_type;
    int64_t xs_tok, xs_slot;   // elements
    void* y;
    int32_t y_type;
    int64_t ldy;          // elements from one item's outputs to the next
    bool swiglu;
    LoraTile lora;
};
// Launches it (arguments already checked); one per format.
int32_t tile_q8_0(const TileCall& c, hipStream_t st);
int32_t tile_q4_0(const TileCall& c, hipStream_t st);
int32_t tile_q4_1(const TileCall& c, hipStream_t st);
int32_t tile_q4_k(const TileCall& c, hipStream_t st);
int32_t tile_q6_k(const TileCall& c, hipStream_t st);
int32_t tile_product(qmv_fmt fmt, const TileCall& c, hipStream_t st);

// Weights and bytes of a format's storage unit; false for an unknown format.
bool fmt_unit(qmv_fmt fmt, int* weights, int* bytes);
// Alignment of W, and of the stride from one matrix to the next (matrices of
// 34-, 18- and 210-byte units may start 2 bytes past a word).
inline int fmt_align(qmv_fmt fmt) { return fmt == QMV_Q4_K ? 16 : 4; }
inline int fmt_stride_align(qmv_fmt fmt) { return fmt == QMV_Q4_K ? 16 : (fmt == QMV_Q4_1 ? 4 : 2); }
inline int x_elem(int32_t t) { return t == QMV_X_F32 ? 4 : 2; }
inline bool x_type_ok(int32_t t) { return t == QMV_X_F32 || t == QMV_X_F16 || t == QMV_X_BF16; }

}  // namespace qmv
