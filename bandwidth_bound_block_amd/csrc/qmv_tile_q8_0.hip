// The many-token tile kernel for Q8_0 weights.
#include "qmv_tile.h"

namespace qmv {
int32_t tile_q8_0(const TileCall& c, hipStream_t st) { return launch_tile_x<Q8_0>(c, st); }
}  // namespace qmv
