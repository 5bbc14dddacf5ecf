// What the serving operators share: argument errors, the device guard, per-device facts, small device helpers.
#pragma once
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <utility>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mk.h"

namespace mkop {

constexpr int kMaxDevices = 64;

inline mk_status refuse(mk_status s, const char* call, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  fprintf(stderr, "%s: %s\n", call, buf);
  return s;
}

// Makes `device` current and puts the caller's device back.
struct DeviceGuard {
  int prev = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceGuard(int device) {
    err = cudaGetDevice(&prev);
    if (err != cudaSuccess) {
      prev = -1;
    } else if (prev == device) {
      prev = -1;
    } else {
      err = cudaSetDevice(device);
    }
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
};

// SMs of a device (read once per device).
inline cudaError_t sm_count(int device, int* n) {
  static std::atomic<int> known[kMaxDevices];
  *n = known[device].load(std::memory_order_relaxed);
  if (*n) return cudaSuccess;
  const cudaError_t e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) known[device].store(*n, std::memory_order_relaxed);
  return e;
}

// Lets a kernel use up to `bytes` of dynamic shared memory (asked for once per kernel and device).
template <auto Kernel>
inline cudaError_t allow_smem(int device, int bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << device;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned(std::initializer_list<const void*> ps, unsigned n) {
  for (const void* p : ps)
    if (!aligned(p, n)) return false;
  return true;
}

inline mk_status check_device(const char* call, int device) {
  return device < 0 || device >= kMaxDevices ? refuse(MK_ERR_INVALID_ARG, call, "device %d", device) : MK_OK;
}

// What the call returns. An error does not stay behind as the runtime's last one, which a later call would take for its own.
inline mk_status launched(const char* call, cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return refuse(MK_ERR_CUDA, call, "%s", cudaGetErrorString(e));
}

// A plain launch. Its status is that of this launch, not of what an earlier call left behind.
template <typename... Params, typename... Args>
cudaError_t start(void (*kernel)(Params...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// n / d for 0 <= n < 2^31 by a product: with 2^(k-1) < d <= 2^k, mul = floor(2^(31+k) / d) + 1 is off by at most 1 from
// 2^(31+k) / d, so n * mul / 2^(31+k) is off by less than 1 / d.
struct Div {
  uint32_t mul;
  int shift;  // k - 1; -1: d = 1
  __device__ int operator()(int n) const {
    return shift < 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
};
inline Div div_by(int d) {
  int k = 0;
  while ((1ll << k) < d) ++k;
  return {static_cast<uint32_t>((1ull << (31 + k)) / d + 1), k - 1};
}

__device__ inline void flag(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Two fp32 values as a 16-bit pair and back; `lo` is the lower half.
template <typename T>
__device__ inline uint32_t pack2(float lo, float hi);
template <>
__device__ inline uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ inline uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ inline float2 unpack2(uint32_t u);
template <>
__device__ inline float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ inline float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// x / scale for an e4m3 result, by a product and one correction. The product with inv = 1 / scale alone is off by up to 1.5
// steps of fp32, so that a value halfway between two codes could go to either. What it leaves, x - q scale, is exact in one
// fused multiply-add; the corrected sum is off by 2^-46 before its rounding, so a quotient that is an fp32 value, as
// halfway ones are, comes out as that value. Nothing overflows or gets too small for that: a scale outside 2^+-60 is brought there
// with the value (`lift`, a power of two), and quotients past 448, infinite ones among them, are not corrected.
// mk_qk_norm_rope, 8190 tokens of 48 / 8 heads x 128 with an e4m3 append 63 us (the product alone 60, divisions 67); a verify batch of 512 rows 7.5
// (7.0, 8.7).
struct Scale {
  float scale, inv, lift;
  __device__ explicit Scale(float s) {
    lift = fabsf(s) < 0x1p-60f ? 0x1p100f : fabsf(s) > 0x1p60f ? 0x1p-64f : 1.0f;
    scale = s * lift;
    inv = 1.0f / scale;
  }
  __device__ float quotient(float x) const {
    x *= lift;
    const float q = x * inv;
    return fabsf(q) < 512.0f ? fmaf(fmaf(-q, scale, x), inv, q) : q;
  }
};

__device__ inline uint32_t e4m3x4(const float* x, const Scale& s) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(s.quotient(x[1])), "f"(s.quotient(x[0])));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(s.quotient(x[3])), "f"(s.quotient(x[2])));
  return lo | static_cast<uint32_t>(hi) << 16;
}

}  // namespace mkop
