// The many-token tile kernel for Q4_1 weights.
#include "qmv_tile.h"

namespace qmv {
int32_t tile_q4_1(const TileCall& c, hipStream_t st) { return launch_tile_x<Q4_1>(c, st); }
}  // namespace qmv
