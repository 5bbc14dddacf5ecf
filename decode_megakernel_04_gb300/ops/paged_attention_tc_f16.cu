// The tensor-memory attention kernels over f16 caches.
#include "paged_attention_tc.cuh"

namespace mkop {
namespace attn {
const Build* pick_tc_f16(int d, int rows) { return pick_tc<__half>(d, rows); }
}  // namespace attn
}  // namespace mkop
