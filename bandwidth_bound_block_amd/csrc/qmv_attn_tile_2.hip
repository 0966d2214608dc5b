// The attention kernel for many rows of queries, fp16 or fp32 queries (pairs of pieces).
#include "qmv_attn_tile.h"

namespace qmv {
int32_t attn_tile_2(const AttnArgs& a, int D, int splits, hipStream_t st) {
    return D == 64 ? launch_tile<64, 2>(a, splits, st) : D == 128 ? launch_tile<128, 2>(a, splits, st) : launch_tile<256, 2>(a, splits, st);
}
}  // namespace qmv
