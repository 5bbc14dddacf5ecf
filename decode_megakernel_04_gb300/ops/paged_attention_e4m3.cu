// The attention kernels over e4m3 caches.
#include "paged_attention.cuh"

namespace mkop {
namespace attn {
const Build* pick_e4m3(int dp, int mt, bool longer) { return pick<__half, true>(dp, mt, longer); }
}  // namespace attn
}  // namespace mkop
