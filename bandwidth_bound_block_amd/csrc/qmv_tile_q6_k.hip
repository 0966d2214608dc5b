// The many-token tile kernel for Q6_K weights.
#include "qmv_tile.h"

namespace qmv {
int32_t tile_q6_k(const TileCall& c, hipStream_t st) { return launch_tile_x<Q6KTile>(c, st); }
}  // namespace qmv
