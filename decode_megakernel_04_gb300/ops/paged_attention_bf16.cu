// The attention kernels over bf16 caches.
#include "paged_attention.cuh"

namespace mkop {
namespace attn {
const Build* pick_bf16(int dp, int mt, bool longer) { return pick<__nv_bfloat16, false>(dp, mt, longer); }
}  // namespace attn
}  // namespace mkop
