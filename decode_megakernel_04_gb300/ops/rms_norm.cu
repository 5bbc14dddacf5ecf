// mk_rms_norm: root-mean-square norm of rows with the residual's addition and, where asked, e4m3 results with scales.
//
// Bound by memory: each value is read once and written once, with about 10 operations in between. A CTA has a row and
// keeps it in registers (8 elements a thread and round, up to 4 rounds), so the norm's second look at it costs nothing: all loads
// are in flight together, one block-wide sum, one look at the registers, stores. A scale's group of at most 256 columns
// lies with neighbouring lanes (shuffles); a scale for the whole row takes a second block-wide step.
#include "mk_ops.cuh"

namespace mkop {
namespace {

constexpr int kMaxThreads = 1024;

// 8 elements as they lie in memory
template <typename T>
struct Eight {
  uint4 u;
  __device__ void load(const void* p, long long i) { u = *reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i); }
  __device__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
  static __device__ void store(void* p, long long i, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(static_cast<T*>(p) + i) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ void load(const void* p, long long i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0], b = q[1];
  }
  __device__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ void store(void* p, long long i, const float (&v)[8]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// The larger of two; NaN if one is.
__device__ inline float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// The sum or the largest of a block's values, for every thread; `red` holds a value for each warp.
template <bool SUM>
__device__ inline float of_block(float x, float* red) {
  auto both = [](float a, float b) { return SUM ? a + b : max_nan(a, b); };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 16; d; d >>= 1) x = both(x, __shfl_xor_sync(~0u, x, d));
  if (lane == 0) red[warp] = x;
  __syncthreads();
  x = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d; d >>= 1) x = both(x, __shfl_xor_sync(~0u, x, d));
  return x;
}

template <typename T, int ROUNDS, bool E4M3>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const __grid_constant__ mk_rms_norm_args a) {
  __shared__ float red[2][kMaxThreads / 32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  float h[ROUNDS][8];
  {
    Eight<T> xs[ROUNDS], rs[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int i = (r * blockDim.x + threadIdx.x) * 8;
      xs[r].zero(), rs[r].zero();
      if (i < a.width) {
        xs[r].load(x, i);
        if (a.residual) rs[r].load(res, i);
      }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      float v[8];
      xs[r].get(h[r]);
      if (a.residual) {
        rs[r].get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[r][k] += v[k];
      }
    }
  }
  float ss = 0;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int i = (r * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += h[r][k] * h[r][k];
    if (a.residual_out && i < a.width) Eight<T>::store(static_cast<T*>(a.residual_out) + row * a.residual_out_stride, i, h[r]);
  }
  ss = of_block<true>(ss, red[0]);
  const float inv = rsqrtf(ss / a.width + a.eps);
  float top = 0;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int i = (r * blockDim.x + threadIdx.x) * 8;
    float g[8];
    if (a.gain && i < a.width) {
      Eight<T> e;
      e.load(a.gain, i);
      e.get(g);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[r][k] *= inv;
      if (a.gain && i < a.width) h[r][k] *= g[k];
    }
    if (!E4M3) {
      if (i < a.width) Eight<T>::store(static_cast<T*>(a.out) + row * a.out_stride, i, h[r]);
    } else if (a.group == a.width) {
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(h[r][k]));
    }
  }
  if (!E4M3) return;
  const float bad = __int_as_float(0x7fffffff);  // NaN
  const bool fine = ss < INFINITY;
  if (a.group == a.width) top = of_block<false>(top, red[1]);
  unsigned char* out = static_cast<unsigned char*>(a.out) + row * a.out_stride;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int i = (r * blockDim.x + threadIdx.x) * 8;
    if (a.group != a.width) {
      top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(h[r][k]));
      for (int d = 1; d < a.group / 8; d <<= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, d));
    }
    float s = top / 448.0f;
    const bool code = fine && s < INFINITY;
    if (!code) s = bad;
    if (i >= a.width) continue;
    if (i % a.group == 0) a.scales[row * a.scales_stride + i / a.group] = s;
    uint2 u = make_uint2(0, 0);
    if (!code) {
      u = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    } else if (s > 0.0f) {
      const Scale by(s);
      u = make_uint2(e4m3x4(h[r], by), e4m3x4(h[r] + 4, by));
    }
    *reinterpret_cast<uint2*>(out + i) = u;
  }
}

template <typename T, bool E4M3>
cudaError_t launch(const mk_rms_norm_args& a, int rounds, int threads, cudaStream_t s) {
  return rounds == 1   ? start(norm_kernel<T, 1, E4M3>, a.rows, threads, 0, s, a)
         : rounds == 2 ? start(norm_kernel<T, 2, E4M3>, a.rows, threads, 0, s, a)
                       : start(norm_kernel<T, 4, E4M3>, a.rows, threads, 0, s, a);
}

}  // namespace
}  // namespace mkop

extern "C" mk_status mk_rms_norm(const mk_rms_norm_args* p, int device, void* stream) {
  using namespace mkop;
  static const char* me = "mk_rms_norm";
  if (!p) return MK_ERR_INVALID_ARG;
  const mk_rms_norm_args& a = *p;
  const bool e4m3 = a.out_dtype == MK_E4M3;
  if (a.rows < 0) return refuse(MK_ERR_INVALID_ARG, me, "%d rows", a.rows);
  if (a.width < 8 || a.width > 32768 || a.width % 8)
    return refuse(MK_ERR_UNSUPPORTED, me, "width %d is not a multiple of 8 in 8..32768", a.width);
  if (a.dtype != MK_BF16 && a.dtype != MK_F16 && a.dtype != MK_F32) return refuse(MK_ERR_UNSUPPORTED, me, "dtype %d", a.dtype);
  if (a.out_dtype != a.dtype && !e4m3) return refuse(MK_ERR_UNSUPPORTED, me, "out dtype %d with dtype %d", a.out_dtype, a.dtype);
  const bool lanes = a.group == 8 || a.group == 16 || a.group == 32 || a.group == 64 || a.group == 128 || a.group == 256;
  if (e4m3 && (a.group < 1 || a.width % a.group || (a.group != a.width && !lanes)))
    return refuse(MK_ERR_UNSUPPORTED, me, "a scale for %d of %d columns", a.group, a.width);
  if (!(a.eps >= 0.0f)) return refuse(MK_ERR_INVALID_ARG, me, "eps %g", a.eps);
  if (mk_status s = check_device(me, device)) return s;
  if (a.rows == 0) return MK_OK;
  if (!a.x || !a.out || (e4m3 && !a.scales)) return refuse(MK_ERR_INVALID_ARG, me, "a required pointer is NULL");
  if (!aligned({a.x, a.residual, a.gain, a.residual_out, a.out}, 16) || !aligned(a.scales, 4))
    return refuse(MK_ERR_INVALID_ARG, me, "a misaligned pointer");
  // the stride of one row is never used
  const int64_t strides[4] = {a.x_stride, a.out_stride, a.residual ? a.residual_stride : a.x_stride,
                              a.residual_out ? a.residual_out_stride : a.x_stride};
  for (int64_t s : strides)
    if (a.rows > 1 && (s % 8 || s < a.width)) return refuse(MK_ERR_INVALID_ARG, me, "a stride is not a multiple of 8 elements, or rows overlap");
  if (a.rows > 1 && e4m3 && a.scales_stride < a.width / a.group) return refuse(MK_ERR_INVALID_ARG, me, "rows of scales overlap");
  // a thread reads its elements before it writes them, so results may lie exactly over an input
  if (a.residual_out && a.residual_out == a.out) return refuse(MK_ERR_INVALID_ARG, me, "out is residual_out");
  const struct { const void* p; int64_t stride; } in[2] = {{a.x, a.x_stride}, {a.residual, a.residual_stride}};
  for (const auto& i : in) {
    if (e4m3 && a.out == i.p) return refuse(MK_ERR_INVALID_ARG, me, "8-bit results over an input");
    if (a.rows > 1 && ((a.out == i.p && a.out_stride != i.stride) || (a.residual_out && a.residual_out == i.p && a.residual_out_stride != i.stride)))
      return refuse(MK_ERR_INVALID_ARG, me, "a result over an input with other strides");
  }
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  const int vectors = a.width / 8;
  // One round is best where an SM has one row (1 x 5120 bf16: 2.0 us in a graph, 2 rounds 2.4, 4 rounds 2.8) and in fp32, where a round
  // is 32 bytes already (4000 x 5120: 50.2 us, 50.9, 56.2; 4 rounds, for rows above 16384, spill 64 to 92 bytes a thread); 16 bits are better with 4
  // (8191 x 6144 to e4m3: 80.6 us, 67.4, 61.1; 512 x 7168 7.5, 7.7, 7.2): an SM has several rows, one's loads run beside another's
  // sums and stores.
  int sms = 0;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);
  int rounds = vectors <= 1024 ? 1 : vectors <= 2048 ? 2 : 4;
  if (a.rows > sms && a.dtype != MK_F32 && vectors >= 64) rounds = vectors >= 128 ? 4 : 2;
  const int threads = (vectors + rounds * 32 - 1) / (rounds * 32) * 32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == MK_BF16  ? e4m3 ? launch<__nv_bfloat16, true>(a, rounds, threads, s) : launch<__nv_bfloat16, false>(a, rounds, threads, s)
                        : a.dtype == MK_F16 ? e4m3 ? launch<__half, true>(a, rounds, threads, s) : launch<__half, false>(a, rounds, threads, s)
                                            : e4m3 ? launch<float, true>(a, rounds, threads, s) : launch<float, false>(a, rounds, threads, s);
  return launched(me, e);
}
