// mk_qk_norm_rope: per-head RMSNorm of queries and keys, rotate-half RoPE and the append to a paged cache.
//
// Bound by memory: each value is read once and written once, with about 10 operations in between. A head is held by
// L = 8, 16 or 32 lanes, 8 elements a lane, so a warp works on 32 / L heads at a time. A lane of the rotated part holds
// the 4 elements 4l.. and their partners 4l + rope_dim / 2.., so that the rotation needs no exchange; the other lanes
// hold 8 elements in a row. The mean square is log2(L) shuffles. A warp loads the heads of kBatch rounds before it
// works on the first (64 bytes a lane in flight); a token's angles are computed once per warp and token and serve
// every head the warp has of it.
//
// Angles: inv_freq / (2 pi) is turned into a 64-bit binary fraction of a turn; position x fraction mod 2^64 is then the
// exact phase whatever the position, and its upper 32 bits (as a signed half-turn count) go to sincospif. An fp32
// product position x inv_freq would be off by 2^-24 of the angle: 0.06 rad at a million positions.
#include "mk_ops.cuh"

namespace mkop {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;  // rounds of 32 / L heads whose loads are in flight together

__device__ inline uint64_t turns_of(double inv_freq) {
  double t = inv_freq * 0.15915494309189533576888;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // a fraction that rounds to one turn saturates, 2^-64 off
}

__device__ inline uint32_t e4m3x4(const float* x, float scale) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] / scale), "f"(x[0] / scale));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] / scale), "f"(x[2] / scale));
  return lo | static_cast<uint32_t>(hi) << 16;
}

struct Work {
  mk_qk_norm_rope_args a;
  int heads;       // rows of work per token: queries, keys, values
  int per_item;    // of them in one item (one warp's turn)
  int parts;       // items per token
};

template <typename T, int L, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) qk_kernel(const __grid_constant__ Work w) {
  const mk_qk_norm_rope_args& a = w.a;
  constexpr int H = 32 / L;  // heads a warp holds at once
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int D = a.head_dim, half = a.rope_dim / 2;
  const bool live = 8 * l < D, turned = 8 * l < a.rope_dim;
  // where this lane's two groups of 4 elements sit in a head
  const int lo = turned ? 4 * l : 8 * l, hi = turned ? 4 * l + half : 8 * l + 4;
  uint64_t turns[4] = {0, 0, 0, 0};
  if (turned && live)
#pragma unroll
    for (int i = 0; i < 4; ++i) turns[i] = turns_of(a.inv_freq[4 * l + i]);

  const long long items = static_cast<long long>(a.n_tokens) * w.parts;
  const long long n_warps = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += n_warps) {
    const int t = static_cast<int>(it / w.parts), part = static_cast<int>(it - static_cast<long long>(t) * w.parts);
    const int r0 = part * w.per_item, r1 = min(w.heads, r0 + w.per_item);
    float c[4], s[4];
    if (turned && live) {
      const int64_t pos = a.positions[t];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t phase = turns[i] * static_cast<uint64_t>(pos);
        const int half_turns = static_cast<int>(phase >> 32);  // units of 2^-31 half turns
        sincospif(static_cast<float>(half_turns) * 4.656612873077392578125e-10f, &s[i], &c[i]);
      }
    }
    long long k_at = -1, v_at = -1;  // the slot's place in the cache
    if (a.k_pages && r1 > a.n_q_heads) {
      const long long slot = a.slots[t];
      if (slot >= static_cast<long long>(a.n_pages) * a.page_size) {
        if (lane == 0) flag(a.status, MK_OP_BAD_PAGE);
      } else if (slot >= 0) {
        const int page = static_cast<int>(slot) / a.page_size, place = static_cast<int>(slot) - page * a.page_size;
        k_at = page * a.k_page_stride[0] + place * a.k_page_stride[2];
        v_at = page * a.v_page_stride[0] + place * a.v_page_stride[2];
      }
    }
    for (int r = r0; r < r1; r += H * kBatch) {
      uint2 in[kBatch][2];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int row = r + j * H + sub;
        in[j][0] = in[j][1] = make_uint2(0, 0);
        if (row >= r1 || !live) continue;
        const T* x;
        if (row < a.n_q_heads) {
          x = static_cast<const T*>(a.q) + t * a.q_stride[0] + row * a.q_stride[1];
        } else if (row < a.n_q_heads + a.n_kv_heads) {
          x = static_cast<const T*>(a.k) + t * a.k_stride[0] + (row - a.n_q_heads) * a.k_stride[1];
        } else {
          if (v_at < 0) continue;
          x = static_cast<const T*>(a.v) + t * a.v_stride[0] + (row - a.n_q_heads - a.n_kv_heads) * a.v_stride[1];
        }
        in[j][0] = *reinterpret_cast<const uint2*>(x + lo);
        in[j][1] = *reinterpret_cast<const uint2*>(x + hi);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int row = r + j * H + sub;
        if (r + j * H >= r1) break;  // the whole warp
        const bool is_q = row < a.n_q_heads, is_v = row >= a.n_q_heads + a.n_kv_heads;
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 p = unpack2<T>(in[j][i].x), q = unpack2<T>(in[j][i].y);
          x[4 * i] = p.x, x[4 * i + 1] = p.y, x[4 * i + 2] = q.x, x[4 * i + 3] = q.y;
        }
        float ss = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
        for (int d = 1; d < L; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
        if (row >= r1 || !live) continue;
        if (!is_v) {
          const T* gain = static_cast<const T*>(is_q ? a.q_gain : a.k_gain);
          if (gain) {
            const float inv = 1.0f / sqrtf(ss / D + a.eps);
            const uint2 g[2] = {*reinterpret_cast<const uint2*>(gain + lo), *reinterpret_cast<const uint2*>(gain + hi)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 p = unpack2<T>(g[i].x), q = unpack2<T>(g[i].y);
              x[4 * i] *= inv * p.x, x[4 * i + 1] *= inv * p.y, x[4 * i + 2] *= inv * q.x, x[4 * i + 3] *= inv * q.y;
            }
          }
          if (turned)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = x[i], v = x[4 + i];
              x[i] = u * c[i] - v * s[i];
              x[4 + i] = v * c[i] + u * s[i];
            }
        }
        const int head = is_q ? row : is_v ? row - a.n_q_heads - a.n_kv_heads : row - a.n_q_heads;
        T* out = is_q ? static_cast<T*>(a.q_out) + t * a.q_out_stride[0] + head * a.q_out_stride[1]
                 : is_v || !a.k_out ? nullptr
                                    : static_cast<T*>(a.k_out) + t * a.k_out_stride[0] + head * a.k_out_stride[1];
        const long long at = is_v ? v_at : k_at;
        const bool store = !is_q && at >= 0;
        const int64_t* ps = is_v ? a.v_page_stride : a.k_page_stride;
        void* pages = is_v ? a.v_pages : a.k_pages;
        if (out || (store && !E4M3)) {
          const uint2 y0 = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
          const uint2 y1 = make_uint2(pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
          if (out) {
            *reinterpret_cast<uint2*>(out + lo) = y0;
            *reinterpret_cast<uint2*>(out + hi) = y1;
          }
          if (store && !E4M3) {
            T* to = static_cast<T*>(pages) + at + head * ps[1];
            *reinterpret_cast<uint2*>(to + lo) = y0;
            *reinterpret_cast<uint2*>(to + hi) = y1;
          }
        }
        if (E4M3 && store) {
          const float scale = (is_v ? a.v_scale : a.k_scale)[head];
          uint8_t* to = static_cast<uint8_t*>(pages) + at + head * ps[1];
          *reinterpret_cast<uint32_t*>(to + lo) = e4m3x4(x, scale);
          *reinterpret_cast<uint32_t*>(to + hi) = e4m3x4(x + 4, scale);
        }
      }
    }
  }
}

template <typename T, int L>
cudaError_t launch(const Work& w, bool e4m3, int grid, cudaStream_t s) {
  if (e4m3) qk_kernel<T, L, true><<<grid, kWarps * 32, 0, s>>>(w);
  else qk_kernel<T, L, false><<<grid, kWarps * 32, 0, s>>>(w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const Work& w, bool e4m3, int lanes, int grid, cudaStream_t s) {
  return lanes == 8 ? launch<T, 8>(w, e4m3, grid, s)
                    : lanes == 16 ? launch<T, 16>(w, e4m3, grid, s) : launch<T, 32>(w, e4m3, grid, s);
}

}  // namespace
}  // namespace mkop

extern "C" mk_status mk_qk_norm_rope(const mk_qk_norm_rope_args* p, int device, void* stream) {
  using namespace mkop;
  static const char* me = "mk_qk_norm_rope";
  if (!p) return MK_ERR_INVALID_ARG;
  Work w;
  w.a = *p;
  const mk_qk_norm_rope_args& a = w.a;
  const bool cache = a.k_pages || a.v_pages, e4m3 = a.cache_dtype == MK_E4M3;
  if (a.n_tokens < 0 || a.n_q_heads < 1 || a.n_kv_heads < 1 || a.n_q_heads > 4096 || a.n_kv_heads > 4096)
    return refuse(MK_ERR_INVALID_ARG, me, "%d tokens, %d / %d heads", a.n_tokens, a.n_q_heads, a.n_kv_heads);
  if (a.head_dim < 16 || a.head_dim > 256 || a.head_dim % 16)
    return refuse(MK_ERR_UNSUPPORTED, me, "head_dim %d is not a multiple of 16 in 16..256", a.head_dim);
  if (a.rope_dim < 0 || a.rope_dim > a.head_dim || a.rope_dim % 8)
    return refuse(MK_ERR_UNSUPPORTED, me, "rope_dim %d is not a multiple of 8 in 0..head_dim", a.rope_dim);
  if (a.dtype != MK_BF16 && a.dtype != MK_F16) return refuse(MK_ERR_UNSUPPORTED, me, "dtype %d", a.dtype);
  if (cache && a.cache_dtype != a.dtype && !e4m3)
    return refuse(MK_ERR_UNSUPPORTED, me, "cache dtype %d with dtype %d", a.cache_dtype, a.dtype);
  if (cache && (!a.k_pages || !a.v_pages || a.n_pages < 1 || a.page_size < 1))
    return refuse(MK_ERR_INVALID_ARG, me, "a cache needs keys and values, pages and a page size");
  if (cache && static_cast<int64_t>(a.n_pages) * a.page_size > INT32_MAX)
    return refuse(MK_ERR_UNSUPPORTED, me, "slots beyond 2^31 - 1");
  if (!(a.eps >= 0.0f)) return refuse(MK_ERR_INVALID_ARG, me, "eps %g", a.eps);
  if (a.n_tokens == 0) return MK_OK;
  if (!a.q || !a.k || !a.q_out || (a.rope_dim && (!a.inv_freq || !a.positions)) || (cache && (!a.v || !a.slots)) ||
      (cache && e4m3 && (!a.k_scale || !a.v_scale)))
    return refuse(MK_ERR_INVALID_ARG, me, "a required pointer is NULL");
  const void* ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out, a.q_gain, a.k_gain, a.k_pages, a.v_pages};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return refuse(MK_ERR_INVALID_ARG, me, "a pointer is not 16-byte aligned");
  for (int i = 0; i < 2; ++i)
    if (a.q_stride[i] % 8 || a.k_stride[i] % 8 || a.q_out_stride[i] % 8 || (cache && a.v_stride[i] % 8) ||
        (a.k_out && a.k_out_stride[i] % 8))
      return refuse(MK_ERR_INVALID_ARG, me, "a stride is not a multiple of 8 elements");
  for (int i = 0; cache && i < 3; ++i)
    if (a.k_page_stride[i] % (e4m3 ? 16 : 8) || a.v_page_stride[i] % (e4m3 ? 16 : 8))
      return refuse(MK_ERR_INVALID_ARG, me, "a cache stride is not a multiple of 16 bytes");
  if (mk_status s = check_device(me, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);

  const int lanes = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 16 : 32, H = 32 / lanes;
  w.heads = a.n_q_heads + a.n_kv_heads * (cache ? 2 : 1);
  // Items: enough to give every SM its warps, and beyond that as many heads each as one token has, so that the
  // angles are computed once.
  const long long room = static_cast<long long>(sms) * 4 * kWarps;
  const int rounds = (w.heads + H * kBatch - 1) / (H * kBatch);
  long long parts = room / a.n_tokens;
  parts = parts < 1 ? 1 : parts > rounds ? rounds : parts;
  w.per_item = static_cast<int>((rounds + parts - 1) / parts) * H * kBatch;
  w.parts = (w.heads + w.per_item - 1) / w.per_item;
  const long long ctas = (static_cast<long long>(a.n_tokens) * w.parts + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(ctas < sms * 4 ? ctas : sms * 4);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(me, a.dtype == MK_BF16 ? launch<__nv_bfloat16>(w, e4m3 && cache, lanes, grid, s)
                                         : launch<__half>(w, e4m3 && cache, lanes, grid, s));
}
