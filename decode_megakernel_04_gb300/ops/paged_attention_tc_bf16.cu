// The tensor-memory attention kernels over bf16 caches.
#include "paged_attention_tc.cuh"

namespace mkop {
namespace attn {
const Build* pick_tc_bf16(int d, int rows) { return pick_tc<__nv_bfloat16>(d, rows); }
}  // namespace attn
}  // namespace mkop
