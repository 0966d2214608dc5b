// The attention kernel for many rows of queries, bf16 queries.
#include "qmv_attn_tile.h"

namespace qmv {
int32_t attn_tile_1(const AttnArgs& a, int D, int splits, hipStream_t st) {
    return D == 64 ? launch_tile<64, 1>(a, splits, st) : D == 128 ? launch_tile<128, 1>(a, splits, st) : launch_tile<256, 1>(a, splits, st);
}
}  // namespace qmv
