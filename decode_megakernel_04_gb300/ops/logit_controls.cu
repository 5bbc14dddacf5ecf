// mk_logit_controls: penalties, biases and masks on logits, and the greedy token of what is left.
//
// Bound by memory: the logits are read once and written once. What a row's history and biases say about a token is
// gathered first, in shared memory: one 32-bit word for each token of the CTA's slice of the vocabulary,
//   bit 31 seen in the history | bits 11..30 times generated | bits 0..10 its last bias entry + 1,
// built with integer atomics (any order gives the same word), so a row's pass over its logits needs no search. A
// cluster of 8 CTAs shares a row, each with an eighth of the vocabulary; it joins the greedy token through
// distributed shared memory, so the call is one launch without a workspace. A slice is at most kSlice tokens (112 KB:
// two CTAs on an SM); a wider vocabulary takes several passes of slices.
#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mkop {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;        // of a row's cluster
constexpr int kSlice = 28640;   // tokens of a CTA's slice at most: (28640 + 8) words, two CTAs on an SM
constexpr int kAhead = 8;       // history tokens a thread loads before it uses the first
constexpr uint32_t kSeen = 0x80000000u;

struct RowControls {
  float repetition, presence, frequency;
  bool has_repetition, has_presence, has_frequency, has_words;
  const float* bias_vals;
};

// Each step rounds on its own, as the definition does.
__device__ inline float control(float z, uint32_t word, bool allowed, const RowControls& c) {
  if (word) {
    const uint32_t times = (word >> 11) & 0xfffffu, entry = word & 0x7ffu;
    if (c.has_repetition && (word >> 11)) z = z > 0 ? __fdiv_rn(z, c.repetition) : __fmul_rn(z, c.repetition);
    if (times) {
      if (c.has_frequency) z = __fsub_rn(z, __fmul_rn(c.frequency, static_cast<float>(times)));
      if (c.has_presence) z = __fsub_rn(z, c.presence);
    }
    if (entry) z = __fadd_rn(z, c.bias_vals[entry - 1]);
  }
  return allowed ? z : -INFINITY;
}

// Larger key = larger value, then lower index (0 stands for no token).
__device__ inline unsigned long long key_of(float z, int index) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.0f));  // -0 counts as 0
  const uint32_t rank = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(rank) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}

__device__ inline unsigned long long larger(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

template <typename T>
__device__ inline float load1(const T* p) {
  return static_cast<float>(*p);
}
__device__ inline float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <typename T>
__device__ inline float4 load4(const T* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = unpack2<T>(u.x), b = unpack2<T>(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logit_kernel(const __grid_constant__ mk_logit_controls_args a, int slice) {
  extern __shared__ __align__(16) uint32_t words[];
  __shared__ unsigned long long best_of[kWarps];
  __shared__ unsigned long long cta_best;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), tid = threadIdx.x;
  const int64_t row = blockIdx.x / kCtas;
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* out = a.out + row * a.out_stride;
  const int32_t* mask = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;
  const int32_t* hist = a.history ? a.history + row * a.history_stride : nullptr;
  const int32_t* ids = a.bias_ids ? a.bias_ids + row * a.bias_stride : nullptr;
  RowControls c;
  c.has_repetition = a.repetition, c.has_presence = a.presence, c.has_frequency = a.frequency;
  c.repetition = a.repetition ? a.repetition[row] : 1.0f;
  c.presence = a.presence ? a.presence[row] : 0.0f;
  c.frequency = a.frequency ? a.frequency[row] : 0.0f;
  c.bias_vals = ids ? a.bias_vals + row * a.bias_stride : nullptr;
  const bool penal = hist && (a.repetition || a.presence || a.frequency);
  c.has_words = penal || ids;
  int total = 0, prompt = 0;
  if (penal) {
    total = a.total_len ? min(max(a.total_len[row], 0), a.max_history) : a.max_history;
    prompt = a.prompt_len ? min(max(a.prompt_len[row], 0), total) : 0;
  }
  // The first `lead` tokens bring the output to a 16-byte boundary; groups of 4 follow, and a tail of fewer than 4.
  // Slices are whole groups, the first with the lead and the last with the tail. Token v of a slice that starts at
  // group boundary g has word v - g + 4, so a group's 4 words are one 16-byte load.
  const int V = a.vocab;
  const int lead = min(V, static_cast<int>((4 - (reinterpret_cast<uintptr_t>(out) >> 2 & 3)) & 3));
  const bool wide = (reinterpret_cast<uintptr_t>(z + lead) & (4 * sizeof(T) - 1)) == 0;
  const int n_words = (V + 31) >> 5;
  // The greedy token so far: this thread meets its tokens in ascending order, so the first of equals stays.
  float best_z = -INFINITY;
  int best_v = -1;
  auto better = [&](float y, int v) {
    if (y > best_z) best_z = y, best_v = v;  // NaN never is
  };

  for (long long g0 = lead + static_cast<long long>(rank) * slice; g0 < V || (g0 == lead && rank == 0);
       g0 += static_cast<long long>(kCtas) * slice) {
    const int g = static_cast<int>(g0);
    const int from = g == lead ? 0 : g, to = min(V, g + slice);
    if (c.has_words) {
      // the logits come into L2 while the words are made
      for (int i = from + tid * (128 / static_cast<int>(sizeof(T))); i < to; i += kThreads * (128 / static_cast<int>(sizeof(T))))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(z + i));
      __syncthreads();
      for (int i = tid; i < (to - g + 4 + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int e = tid; ids && e < a.n_biases; e += kThreads) {
        const int v = ids[e];
        if (v >= from && v < to) atomicMax(&words[v - g + 4], static_cast<uint32_t>(e + 1));
      }
      __syncthreads();
      for (int h0 = tid; h0 < total; h0 += kThreads * kAhead) {
        int seen[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int h = h0 + i * kThreads;
          seen[i] = h < total ? hist[h] : -1;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (seen[i] < from || seen[i] >= to) continue;
          uint32_t* word = &words[seen[i] - g + 4];
          if (h0 + i * kThreads >= prompt) atomicAdd(word, 1u << 11);
          else atomicOr(word, kSeen);
        }
      }
      __syncthreads();
    }
    auto one = [&](int v) {
      const bool ok = !mask || (static_cast<uint32_t>(mask[v >> 5]) >> (v & 31) & 1);
      const float y = control(load1(z + v), c.has_words ? words[v - g + 4] : 0, ok, c);
      out[v] = y;
      better(y, v);
    };
    if (tid < g - from) one(from + tid);
    const int groups = (to - g) >> 2;
#pragma unroll 4
    for (int i = tid; i < groups; i += kThreads) {
      const int v = g + 4 * i;
      float4 y = wide ? load4(z + v) : make_float4(load1(z + v), load1(z + v + 1), load1(z + v + 2), load1(z + v + 3));
      if (c.has_words) {
        const uint4 w = reinterpret_cast<const uint4*>(words)[i + 1];
        if (w.x | w.y | w.z | w.w) {
          y.x = control(y.x, w.x, true, c);
          y.y = control(y.y, w.y, true, c);
          y.z = control(y.z, w.z, true, c);
          y.w = control(y.w, w.w, true, c);
        }
      }
      if (mask) {
        const uint32_t m0 = mask[v >> 5], m1 = mask[min((v >> 5) + 1, n_words - 1)];
        const uint32_t ok = __funnelshift_r(m0, m1, v & 31);
        y.x = ok & 1 ? y.x : -INFINITY;
        y.y = ok & 2 ? y.y : -INFINITY;
        y.z = ok & 4 ? y.z : -INFINITY;
        y.w = ok & 8 ? y.w : -INFINITY;
      }
      *reinterpret_cast<float4*>(out + v) = y;
      better(y.x, v);
      better(y.y, v + 1);
      better(y.z, v + 2);
      better(y.w, v + 3);
    }
    const int rest = g + 4 * groups;
    if (tid < to - rest) one(rest + tid);
  }
  if (!a.token) return;  // the same for every CTA

  unsigned long long best = best_v < 0 ? 0 : key_of(best_z, best_v);
#pragma unroll
  for (int d = 16; d; d >>= 1) best = larger(best, __shfl_xor_sync(~0u, best, d));
  if ((tid & 31) == 0) best_of[tid >> 5] = best;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kWarps; ++i) best = larger(best, best_of[i]);
    cta_best = best;
  }
  cluster.sync();
  if (rank == 0 && tid == 0) {
    for (int i = 1; i < kCtas; ++i) best = larger(best, *cluster.map_shared_rank(&cta_best, i));
    a.token[row] = best ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
  }
  cluster.sync();  // the others' shared memory stays until it has been read
}

template <typename T>
cudaError_t launch(const mk_logit_controls_args& a, int device, cudaStream_t s) {
  int slice = (((a.vocab + kCtas - 1) / kCtas) + 3) & ~3;
  if (slice > kSlice) {
    // equal passes
    const int passes = (slice + kSlice - 1) / kSlice;
    slice = ((slice + passes - 1) / passes + 3) & ~3;
  }
  const bool has_words = a.bias_ids || (a.history && (a.repetition || a.presence || a.frequency));
  const size_t smem = has_words ? sizeof(uint32_t) * (slice + 8) : 0;
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem<logit_kernel<T>>(device, static_cast<int>(sizeof(uint32_t) * (kSlice + 8)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logit_kernel<T>, a, slice);
}

}  // namespace
}  // namespace mkop

extern "C" mk_status mk_logit_controls(const mk_logit_controls_args* p, int device, void* stream) {
  using namespace mkop;
  static const char* me = "mk_logit_controls";
  if (!p) return MK_ERR_INVALID_ARG;
  const mk_logit_controls_args a = *p;
  if (a.rows < 0 || a.rows > 1 << 24 || a.vocab < 1 || a.vocab > 1 << 30)
    return refuse(MK_ERR_INVALID_ARG, me, "rows %d, vocab %d", a.rows, a.vocab);
  if (a.dtype != MK_F32 && a.dtype != MK_BF16 && a.dtype != MK_F16) return refuse(MK_ERR_UNSUPPORTED, me, "dtype %d", a.dtype);
  if (a.max_history < 0 || a.max_history > MK_LOGIT_MAX_HISTORY || a.n_biases < 0 || a.n_biases > MK_LOGIT_MAX_BIASES)
    return refuse(MK_ERR_UNSUPPORTED, me, "max_history %d (at most %d), n_biases %d (at most %d)", a.max_history,
                  MK_LOGIT_MAX_HISTORY, a.n_biases, MK_LOGIT_MAX_BIASES);
  if (a.rows == 0) return MK_OK;
  if (!a.logits || !a.out) return refuse(MK_ERR_INVALID_ARG, me, "a required pointer is NULL");
  if (!a.history && (a.repetition || a.presence || a.frequency))
    return refuse(MK_ERR_INVALID_ARG, me, "penalties without a history");
  if (!a.bias_ids != !a.bias_vals) return refuse(MK_ERR_INVALID_ARG, me, "bias ids and values come together");
  if (a.logits_stride < a.vocab || a.out_stride < a.vocab || (a.history && a.history_stride < a.max_history) ||
      (a.bias_ids && a.bias_stride < a.n_biases) || (a.allowed && a.allowed_stride < (a.vocab + 31) / 32))
    return refuse(MK_ERR_INVALID_ARG, me, "a row stride is shorter than its row");
  if (a.logits == a.out && (a.dtype != MK_F32 || a.logits_stride != a.out_stride))
    return refuse(MK_ERR_INVALID_ARG, me, "out may be logits only in fp32 with one stride");
  if (!aligned(a.logits, a.dtype == MK_F32 ? 4 : 2) || !aligned(a.out, 4) || !aligned(a.allowed, 4))
    return refuse(MK_ERR_INVALID_ARG, me, "a misaligned pointer");
  if (mk_status s = check_device(me, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(me, a.dtype == MK_F32 ? launch<float>(a, device, s)
                      : a.dtype == MK_BF16 ? launch<__nv_bfloat16>(a, device, s) : launch<__half>(a, device, s));
}
