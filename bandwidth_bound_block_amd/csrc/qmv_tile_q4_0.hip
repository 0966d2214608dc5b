// The many-token tile kernel for Q4_0 weights.
#include "qmv_tile.h"

namespace qmv {
int32_t tile_q4_0(const TileCall& c, hipStream_t st) { return launch_tile_x<Q4_0>(c, st); }
}  // namespace qmv
