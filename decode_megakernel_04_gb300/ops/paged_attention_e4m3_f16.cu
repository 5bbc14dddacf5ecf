// The attention kernels over e4m3 caches with fp16 queries.
#include "paged_attention.cuh"

namespace mkop {
namespace attn {
const Build* pick_e4m3_f16(int dp, int mt, bool longer) { return pick<__half, true, true>(dp, mt, longer); }
}  // namespace attn
}  // namespace mkop
