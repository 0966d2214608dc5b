// The streaming attention kernel for Q8_0 keys and bf16 queries.
#include "qmv_attention.h"

namespace qmv {
int32_t attn_stream_q8_0_1(const AttnArgs& a, int D, hipStream_t st) { return launch_stream<QMV_Q8_0, 1>(a, D, st); }
}  // namespace qmv
