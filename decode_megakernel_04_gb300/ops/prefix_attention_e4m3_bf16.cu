// The shared prefix's kernels over e4m3 caches with bf16 queries.
#include "prefix_attention.cuh"

namespace mkop {
namespace prefix {
cudaError_t launch_prefix_e4m3_bf16(const PrefixParams& p, int device, cudaStream_t s) { return launch_prefix<__half, __nv_bfloat16, true>(p, device, s); }
}  // namespace prefix
}  // namespace mkop
