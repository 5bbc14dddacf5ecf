// The attention kernels over f16 caches.
#include "paged_attention.cuh"

namespace mkop {
namespace attn {
const Build* pick_f16(int dp, int mt, bool longer) { return pick<__half, false>(dp, mt, longer); }
}  // namespace attn
}  // namespace mkop
