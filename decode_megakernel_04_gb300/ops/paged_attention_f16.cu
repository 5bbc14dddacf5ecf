// The attention kernels over f16 caches.
#include "paged_attention.cuh"

namespace mkop {
namespace attn {
const Build* pick_f16(int dp, int mt) { return pick<__half, false>(dp, mt); }
}  // namespace attn
}  // namespace mkop
