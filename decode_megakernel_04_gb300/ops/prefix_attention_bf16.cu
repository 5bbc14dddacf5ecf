// The shared prefix's kernels over bf16 caches.
#include "prefix_attention.cuh"

namespace mkop {
namespace prefix {
cudaError_t launch_prefix_bf16(const PrefixParams& p, int device, cudaStream_t s) { return launch_prefix<__nv_bfloat16, __nv_bfloat16, false>(p, device, s); }
}  // namespace prefix
}  // namespace mkop
