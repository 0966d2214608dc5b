// The many-token tile kernel for Q4_K weights.
#include "qmv_tile.h"

namespace qmv {
int32_t tile_q4_k(const TileCall& c, hipStream_t st) { return launch_tile_x<Q4KTile>(c, st); }
}  // namespace qmv
