// The streaming attention kernel for Q8_0 keys and fp16 or fp32 queries (pairs of pieces).
#include "qmv_attention.h"

namespace qmv {
int32_t attn_stream_q8_0_2(const AttnArgs& a, int D, hipStream_t st) { return launch_stream<QMV_Q8_0, 2>(a, D, st); }
}  // namespace qmv
