// The shared prefix's kernels over fp16 caches.
#include "prefix_attention.cuh"

namespace mkop {
namespace prefix {
cudaError_t launch_prefix_f16(const PrefixParams& p, int device, cudaStream_t s) { return launch_prefix<__half, __half, false>(p, device, s); }
}  // namespace prefix
}  // namespace mkop
