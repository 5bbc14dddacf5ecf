// mk_qk_norm_rope: per-head RMSNorm of queries and keys, rotate-half RoPE and the append to a paged cache.
//
// Bound by memory: each value is read once and written once, with about 10 operations in between. A head is held by
// L = 8, 16 or 32 lanes, 8 elements a lane, so a warp works on 32 / L heads at a time. A lane of the rotated part holds
// the 4 elements 4l.. and their partners 4l + rope_dim / 2.., so that the rotation needs no exchange; the other lanes
// hold 8 elements in a row. The mean square is log2(L) shuffles. A warp loads the heads of kBatch rounds before it
// works on the first, and the next kBatch while it does (128 bytes a lane in flight; 63 us without, 51 with); a token's
// angles are computed once per warp and token and serve every head the warp has of it.
// Measured: 8190 tokens of 48 / 8 heads x 128 with the append, fp16: 51 us, 5.3 TB/s, 79 % of the measured copy rate,
// bound by the instructions issued (66 % of the slots); one token 3.9 us.
//
// Angles: inv_freq / (2 pi) is turned into a 64-bit binary fraction of a turn; position x fraction mod 2^64 is then the
// exact phase whatever the position, and its upper 32 bits (as a signed half-turn count) go to sincospif. An fp32
// product position x inv_freq would be off by 2^-24 of the angle: 0.06 rad at a million positions.
#include <type_traits>

#include "mk_ops.cuh"

namespace mkop {
namespace {

constexpr int kWarps = 8;
constexpr int kCtas = 3;   // on an SM
constexpr int kBatch = 4;  // rounds of 32 / L heads whose loads are in flight together

__device__ inline uint64_t turns_of(double inv_freq) {
  double t = inv_freq * 0.15915494309189533576888;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // a fraction that rounds to one turn saturates, 2^-64 off
}

enum Kind { kQuery, kKey, kValue };

struct Work {
  mk_qk_norm_rope_args a;
  int q_rounds, k_rounds, rounds;  // rounds of kBatch * 32 / L heads of a token: queries, keys, and with the values
  int per_item;                    // rounds of one item (one warp's turn)
  int parts;                       // items per token
  float inv_width;                 // 1 / head_dim
};

template <typename T, int L, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, kCtas) qk_kernel(const __grid_constant__ Work w) {
  const mk_qk_norm_rope_args& a = w.a;
  constexpr int H = 32 / L;  // heads a warp holds at once
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int half = a.rope_dim / 2;
  const bool live = 8 * l < a.head_dim, turned = live && 8 * l < a.rope_dim;
  // where this lane's two groups of 4 elements sit in a head
  const int lo = turned ? 4 * l : 8 * l, hi = turned ? 4 * l + half : 8 * l + 4;
  __shared__ uint64_t turns[128];
  for (int i = threadIdx.x; i < half; i += kWarps * 32) turns[i] = turns_of(a.inv_freq[i]);
  __syncthreads();
  uint2 gains[2][2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const T* gain = static_cast<const T*>(i ? a.k_gain : a.q_gain);
    if (gain && live) gains[i][0] = *reinterpret_cast<const uint2*>(gain + lo), gains[i][1] = *reinterpret_cast<const uint2*>(gain + hi);
  }

  const long long items = static_cast<long long>(a.n_tokens) * w.parts;
  const long long n_warps = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += n_warps) {
    const int t = static_cast<int>(it / w.parts), part = static_cast<int>(it - static_cast<long long>(t) * w.parts);
    const int r0 = part * w.per_item, r1 = min(w.rounds, r0 + w.per_item);
    float c[4] = {1, 1, 1, 1}, s[4] = {0, 0, 0, 0};
    if (turned && r0 < w.q_rounds + w.k_rounds) {
      const int64_t pos = a.positions[t];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t phase = turns[4 * l + i] * static_cast<uint64_t>(pos);
        const int half_turns = static_cast<int>(phase >> 32);  // units of 2^-31 half turns
        sincospif(static_cast<float>(half_turns) * 4.656612873077392578125e-10f, &s[i], &c[i]);
      }
    }
    long long k_at = -1, v_at = -1;  // the slot's place in the cache
    if (a.k_pages && r1 > w.q_rounds) {
      const long long slot = a.slots[t];
      if (slot >= static_cast<long long>(a.n_pages) * a.page_size) {
        if (lane == 0) flag(a.status, MK_OP_BAD_PAGE);
      } else if (slot >= 0) {
        const int page = static_cast<int>(slot) / a.page_size, place = static_cast<int>(slot) - page * a.page_size;
        k_at = page * a.k_page_stride[0] + place * a.k_page_stride[2];
        v_at = page * a.v_page_stride[0] + place * a.v_page_stride[2];
      }
    }
    // A round: kBatch x H heads of one kind. The next round is loaded before the current one is worked on.
    auto load = [&](int r, uint2 (&in)[kBatch][2]) {
      const bool is_q = r < w.q_rounds, is_k = !is_q && r < w.q_rounds + w.k_rounds;
      const int row0 = (is_q ? r : is_k ? r - w.q_rounds : r - w.q_rounds - w.k_rounds) * H * kBatch + sub;
      const int n = is_q ? a.n_q_heads : !is_k && v_at < 0 ? 0 : a.n_kv_heads;
      const int64_t* xs = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
      const T* x = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v) + t * xs[0] + row0 * xs[1];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        in[j][0] = in[j][1] = make_uint2(0, 0);
        if (row0 + j * H < n && live) {
          in[j][0] = *reinterpret_cast<const uint2*>(x + j * H * xs[1] + lo);
          in[j][1] = *reinterpret_cast<const uint2*>(x + j * H * xs[1] + hi);
        }
      }
    };
    // out: q_out or k_out (NULL: none); pages: the cache, at: the token's place in it (< 0: none)
    auto turn_and_store = [&](auto kind_tag, int first, int n, const uint2 (&in)[kBatch][2], T* out, const int64_t* os, void* pages,
                    long long at, const int64_t* ps, const float* scales) {
      constexpr Kind kind = decltype(kind_tag)::value;
      const int row0 = first + sub;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int row = row0 + j * H;
        if (first + j * H >= n) break;  // the whole warp
        float y[8];
        uint2 packed[2] = {in[j][0], in[j][1]};
        if (kind != kValue || E4M3)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 p = unpack2<T>(packed[i].x), q = unpack2<T>(packed[i].y);
            y[4 * i] = p.x, y[4 * i + 1] = p.y, y[4 * i + 2] = q.x, y[4 * i + 3] = q.y;
          }
        if (kind != kValue) {
          if (kind == kQuery ? a.q_gain != nullptr : a.k_gain != nullptr) {
            float ss = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
            for (int d = 1; d < L; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
            const float inv = rsqrtf(ss * w.inv_width + a.eps);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 p = unpack2<T>(gains[kind][i].x), q = unpack2<T>(gains[kind][i].y);
              y[4 * i] *= inv * p.x, y[4 * i + 1] *= inv * p.y, y[4 * i + 2] *= inv * q.x, y[4 * i + 3] *= inv * q.y;
            }
          }
          if (turned)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = y[i], v = y[4 + i];
              y[i] = u * c[i] - v * s[i];
              y[4 + i] = v * c[i] + u * s[i];
            }
          packed[0] = make_uint2(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]));
          packed[1] = make_uint2(pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
        }
        if (row >= n || !live) continue;
        if (kind != kValue && out) {
          T* to = out + t * os[0] + row * os[1];
          *reinterpret_cast<uint2*>(to + lo) = packed[0];
          *reinterpret_cast<uint2*>(to + hi) = packed[1];
        }
        if (kind == kQuery || at < 0) continue;
        if (E4M3) {
          uint8_t* to = static_cast<uint8_t*>(pages) + at + row * ps[1];
          const Scale scale(scales[row]);
          *reinterpret_cast<uint32_t*>(to + lo) = e4m3x4(y, scale);
          *reinterpret_cast<uint32_t*>(to + hi) = e4m3x4(y + 4, scale);
        } else {
          T* to = static_cast<T*>(pages) + at + row * ps[1];
          *reinterpret_cast<uint2*>(to + lo) = packed[0];
          *reinterpret_cast<uint2*>(to + hi) = packed[1];
        }
      }
    };
    uint2 in[kBatch][2], next[kBatch][2];
    load(r0, in);
    for (int r = r0; r < r1; ++r) {
      if (r + 1 < r1) load(r + 1, next);
      if (r < w.q_rounds)
        turn_and_store(std::integral_constant<Kind, kQuery>{}, r * H * kBatch, a.n_q_heads, in, static_cast<T*>(a.q_out), a.q_out_stride,
             nullptr, -1, nullptr, nullptr);
      else if (r < w.q_rounds + w.k_rounds)
        turn_and_store(std::integral_constant<Kind, kKey>{}, (r - w.q_rounds) * H * kBatch, a.n_kv_heads, in, static_cast<T*>(a.k_out),
             a.k_out_stride, a.k_pages, k_at, a.k_page_stride, a.k_scale);
      else if (v_at >= 0)
        turn_and_store(std::integral_constant<Kind, kValue>{}, (r - w.q_rounds - w.k_rounds) * H * kBatch, a.n_kv_heads, in,
             static_cast<T*>(nullptr), nullptr, a.v_pages, v_at, a.v_page_stride, a.v_scale);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) in[j][0] = next[j][0], in[j][1] = next[j][1];
    }
  }
}

template <typename T, int L>
cudaError_t launch(const Work& w, bool e4m3, int grid, cudaStream_t s) {
  return start(e4m3 ? qk_kernel<T, L, true> : qk_kernel<T, L, false>, grid, kWarps * 32, 0, s, w);
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
  if (!aligned({a.q, a.k, a.v, a.q_out, a.k_out, a.q_gain, a.k_gain, a.k_pages, a.v_pages}, 16))
    return refuse(MK_ERR_INVALID_ARG, me, "a pointer is not 16-byte aligned");
  if (!aligned({a.inv_freq, a.slots}, 8) || !aligned({a.positions, a.k_scale, a.v_scale, a.status}, 4))
    return refuse(MK_ERR_INVALID_ARG, me, "a misaligned pointer");
  // the stride of a dimension of one element is never used
  const int tokens_heads[2][2] = {{a.n_tokens, a.n_q_heads}, {a.n_tokens, a.n_kv_heads}};
  for (int i = 0; i < 2; ++i) {
    const bool q = tokens_heads[0][i] > 1, k = tokens_heads[1][i] > 1;
    if ((q && (a.q_stride[i] % 8 || a.q_out_stride[i] % 8)) ||
        (k && (a.k_stride[i] % 8 || (cache && a.v_stride[i] % 8) || (a.k_out && a.k_out_stride[i] % 8))))
      return refuse(MK_ERR_INVALID_ARG, me, "a stride is not a multiple of 8 elements");
  }
  const int page_dims[3] = {a.n_pages, a.n_kv_heads, a.page_size};
  for (int i = 0; cache && i < 3; ++i)
    if (page_dims[i] > 1 && (a.k_page_stride[i] % (e4m3 ? 16 : 8) || a.v_page_stride[i] % (e4m3 ? 16 : 8)))
      return refuse(MK_ERR_INVALID_ARG, me, "a cache stride is not a multiple of 16 bytes");
  if (mk_status s = check_device(me, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);

  const int lanes = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 16 : 32, heads = 32 / lanes * kBatch;
  w.q_rounds = (a.n_q_heads + heads - 1) / heads;
  w.k_rounds = (a.n_kv_heads + heads - 1) / heads;
  w.rounds = w.q_rounds + w.k_rounds * (cache ? 2 : 1);
  w.inv_width = 1.0f / a.head_dim;
  // Items: enough to give every SM its warps, and beyond that as many rounds each as one token has, so that the
  // angles are computed once.
  const long long room = static_cast<long long>(sms) * kCtas * kWarps;
  long long parts = room / a.n_tokens;
  parts = parts < 1 ? 1 : parts > w.rounds ? w.rounds : parts;
  w.per_item = static_cast<int>((w.rounds + parts - 1) / parts);
  w.parts = (w.rounds + w.per_item - 1) / w.per_item;
  const long long ctas = (static_cast<long long>(a.n_tokens) * w.parts + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(ctas < sms * kCtas ? ctas : sms * kCtas);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(me, a.dtype == MK_BF16 ? launch<__nv_bfloat16>(w, e4m3 && cache, lanes, grid, s)
                                         : launch<__half>(w, e4m3 && cache, lanes, grid, s));
}
