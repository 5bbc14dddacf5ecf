// mk_verify_drafts: drafted tokens against the target's probabilities from given random numbers, and the token after them.
//
// Two kernels. `stats_kernel`: the largest logit of every row, its first place and the sum of exp((z - largest) / T), one
// pass, a row cut into up to 32 parts so that few rows fill the GPU. `draw_kernel`: a cluster for each request joins the
// parts, walks the drafts and runs the race: the token with the largest weight / noise. With given exponential noise the
// race is a draw from the weights, and unlike an inverse distribution function it is no sum over the vocabulary: a token's
// quotient depends on that token alone, in fp32, whatever the order of the work.
// Bound by memory: every logit once, and the drawn row, its draft row and the noise.
#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mkop {
namespace drafts {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kMaxParts = 32;    // of a row: one a lane
constexpr int kMaxRows = 64;     // of a request

struct Part {
  float top, sum;  // the largest logit, the sum of exp2((z - top) * c)
  int at;          // the first place of the largest; -1: none above -infinity
  int pad;
};
struct Work {
  mk_verify_drafts_args a;
  int parts;       // of a row
  Part* part;      // [batch * rows + batch * (rows - 1)][parts]
};

__device__ inline float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A logit as it counts: NaN is -infinity, +infinity the largest finite value (so that differences stay defined).
__device__ inline float logit(float z) { return fminf(fmaxf(z, -INFINITY), 3.402823466e38f); }
template <typename T>
__device__ inline float as_float(T x) { return static_cast<float>(x); }

// log2(e) / T, with T within 2^+-100 so that 0 * c and infinity * c stay defined; 0: greedy
__device__ inline float per_log2(float t) {
  return t > 0.0f ? 1.44269504088896340736f / fminf(fmaxf(t, 0x1p-100f), 0x1p100f) : 0.0f;
}

// An online softmax's state of one thread. `base`: the largest so far, 0 while there is none.
struct State {
  float top = -INFINITY, base = 0, sum = 0;
  int at = -1;
  template <int N>
  __device__ void add(const float (&z)[N], int first, int step, float c) {
    float big = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) big = fmaxf(big, z[i]);
    if (big > top) {
      sum *= exp2_fast((top - big) * c);
      top = base = big;
#pragma unroll
      for (int i = N - 1; i >= 0; --i)
        if (z[i] == big) at = first + i * step;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum += exp2_fast((z[i] - base) * c);
  }
  __device__ void join(float otop, float osum, int oat, float c) {
    const float big = fmaxf(top, otop);
    if (big == -INFINITY) return;
    sum = sum * exp2_fast((top - big) * c) + osum * exp2_fast((otop - big) * c);
    at = otop > top || (otop == top && oat < at) ? oat : at;
    top = base = big;
  }
};

// Part y of row x (target rows, then draft rows).
template <typename T>
__global__ void __launch_bounds__(kThreads) stats_kernel(const __grid_constant__ Work w) {
  __shared__ Part red[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const mk_verify_drafts_args& a = w.a;
  const int row = blockIdx.x / w.parts, part = blockIdx.x - row * w.parts, tid = threadIdx.x;
  const int targets = a.batch * a.rows;
  const bool draft = row >= targets;
  const int b = draft ? (row - targets) / (a.rows - 1) : row / a.rows;
  const T* z = draft ? static_cast<const T*>(a.draft_logits) + (row - targets) * a.draft_stride
                     : static_cast<const T*>(a.logits) + row * a.logits_stride;
  const float c = per_log2(a.temperature ? a.temperature[b] : 1.0f);
  const int i0 = static_cast<int>(static_cast<long long>(a.vocab) * part / w.parts);
  const int i1 = static_cast<int>(static_cast<long long>(a.vocab) * (part + 1) / w.parts);
  State s;
  for (int i = i0 + tid; i < i1; i += kThreads) {
    const float v[1] = {logit(as_float(z[i]))};
    s.add(v, i, 1, c);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float otop = __shfl_xor_sync(~0u, s.top, d), osum = __shfl_xor_sync(~0u, s.sum, d);
    const int oat = __shfl_xor_sync(~0u, s.at, d);
    s.join(otop, osum, oat, c);
  }
  if ((tid & 31) == 0) red[tid >> 5] = {s.top, s.sum, s.at, 0};
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < kThreads / 32; ++k) s.join(red[k].top, red[k].sum, red[k].at, c);
    w.part[static_cast<long long>(row) * w.parts + part] = {s.top, s.sum, s.at, 0};
  }
}

// The better of two tokens of the race: the larger quotient, the lower index on ties; at -1: none.
__device__ inline void better(float& score, int& at, float oscore, int oat) {
  if (oscore > score || (oscore == score && static_cast<unsigned>(oat) < static_cast<unsigned>(at))) score = oscore, at = oat;
}

struct Chosen {
  int row, cut;            // the drawn row of the request; whether a draft was refused there
  float top, sum;          // of that row
  float draft_top, draft_sum;
  int token;               // what needs no race
};

template <typename T>
__global__ void __launch_bounds__(kThreads) draw_kernel(const __grid_constant__ Work w, int ctas) {
  __shared__ Part stats[2 * kMaxRows];
  __shared__ Chosen chosen;
  __shared__ float best_score[kThreads / 32];
  __shared__ int best_at[kThreads / 32];
  __shared__ float mine_score;
  __shared__ int mine_at;
  const mk_verify_drafts_args& a = w.a;
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const float c = per_log2(t);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the rows' statistics ----------------------------------------------------------------------------------------
  const int rows = a.rows, all = a.draft_logits ? 2 * rows - 1 : rows;
  for (int r = warp; r < all; r += kThreads / 32) {
    const long long row = r < rows ? static_cast<long long>(b) * rows + r
                                   : static_cast<long long>(a.batch) * rows + static_cast<long long>(b) * (rows - 1) + r - rows;
    State s;
    if (lane < w.parts) {
      const Part p = w.part[row * w.parts + lane];
      s.top = p.top, s.sum = p.sum, s.at = p.at;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const float otop = __shfl_xor_sync(~0u, s.top, d), osum = __shfl_xor_sync(~0u, s.sum, d);
      const int oat = __shfl_xor_sync(~0u, s.at, d);
      s.join(otop, osum, oat, c);
    }
    if (lane == 0) stats[r] = {s.top, s.sum, s.at, 0};
  }
  __syncthreads();
  const T* z = static_cast<const T*>(a.logits) + static_cast<long long>(b) * rows * a.logits_stride;
  const T* y = static_cast<const T*>(a.draft_logits) + static_cast<long long>(b) * (rows - 1) * a.draft_stride;
  // ---- the drafts, by the first thread of each CTA -------------------------------------------------------------------
  if (tid == 0) {
    const bool says = rank == 0;  // one CTA writes
    int n = a.n_drafts ? a.n_drafts[b] : rows - 1;
    if (n < 0 || n > rows - 1) {
      if (says) flag(a.status, MK_OP_BAD_LENGTH);
      n = min(max(n, 0), rows - 1);
    }
    // log of the probability of a row's token
    auto log_p = [&](const T* row, const Part& s, int x) -> double {
      if (s.at < 0) return -INFINITY;
      if (c == 0.0f) return x == s.at ? 0.0 : -INFINITY;
      return (static_cast<double>(logit(as_float(row[x]))) - s.top) * c * 0.6931471805599453 - log(static_cast<double>(s.sum));
    };
    int r = 0;
    for (; r < n; ++r) {
      const int x = a.tokens[static_cast<long long>(b) * rows + r + 1];
      bool good = false;
      if (x < 0 || x >= a.vocab) {
        if (says) flag(a.status, MK_OP_BAD_TOKEN);
      } else {
        const double lp = log_p(z + r * a.logits_stride, stats[r], x);
        const double q = a.draft_logits ? exp(log_p(y + r * a.draft_stride, stats[rows + r], x)) : 1.0;
        good = a.uniforms[static_cast<long long>(b) * (rows - 1) + r] * q < exp(lp);
        if (good && says && a.logprobs) a.logprobs[static_cast<long long>(b) * rows + r] = static_cast<float>(lp);
      }
      if (!good) break;
    }
    chosen.row = r;
    chosen.cut = r < n;
    chosen.top = stats[r].top;
    chosen.sum = stats[r].sum;
    chosen.token = stats[r].at;
    if (r < n && a.draft_logits) chosen.draft_top = stats[rows + r].top, chosen.draft_sum = stats[rows + r].sum;
    if (says && a.logprobs)
      for (int k = r + 1; k < rows; ++k) a.logprobs[static_cast<long long>(b) * rows + k] = 0.0f;
  }
  __syncthreads();
  const Chosen ch = chosen;
  const T* zr = z + ch.row * a.logits_stride;
  int token = ch.token;
  if (ch.token >= 0 && c != 0.0f) {
    // ---- the race ----------------------------------------------------------------------------------------------------
    const float* noise = a.noise + b * a.noise_stride;
    const T* yr = y + ch.row * a.draft_stride;
    const int out = ch.cut && !a.draft_logits ? a.tokens[static_cast<long long>(b) * rows + ch.row + 1] : -1;  // not drawn
    const bool minus = ch.cut && a.draft_logits && ch.draft_top > -INFINITY;
    const float by = 1.0f / ch.sum, draft_by = minus ? 1.0f / ch.draft_sum : 0.0f;
    const int i0 = static_cast<int>(static_cast<long long>(a.vocab) * rank / ctas);
    const int i1 = static_cast<int>(static_cast<long long>(a.vocab) * (rank + 1) / ctas);
    for (int pass = 0; pass < 2; ++pass) {  // the second one where max(p - q, 0) is 0 everywhere
      float score = 0;
      int at = -1;
      for (int i = i0 + tid; i < i1; i += kThreads) {
        // (rounded products, so that equal probabilities leave 0 and not what a fused difference would)
        float p = __fmul_rn(exp2_fast((logit(as_float(zr[i])) - ch.top) * c), by);
        if (pass == 0 && minus) p -= __fmul_rn(exp2_fast((logit(as_float(yr[i])) - ch.draft_top) * c), draft_by);
        if (pass == 0 && i == out) p = 0.0f;
        const float s = __fdividef(p, noise[i]);
        if (s > score) score = s, at = i;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const float os = __shfl_xor_sync(~0u, score, d);
        const int oa = __shfl_xor_sync(~0u, at, d);
        better(score, at, os, oa);
      }
      if (lane == 0) best_score[warp] = score, best_at[warp] = at;
      __syncthreads();
      if (tid == 0) {
        for (int k = 1; k < kThreads / 32; ++k) better(score, at, best_score[k], best_at[k]);
        mine_score = score, mine_at = at;
      }
      cluster.sync();
      score = 0, at = -1;
      for (int k = 0; k < ctas; ++k) better(score, at, *cluster.map_shared_rank(&mine_score, k), *cluster.map_shared_rank(&mine_at, k));
      token = at;
      cluster.sync();  // the others' results stay until they have been read
      if (token >= 0 || !ch.cut) break;
    }
  }
  if (rank == 0 && tid == 0) {
    a.accept_out[b] = ch.row + 1;
    a.accept_out[a.batch + b] = token;
    a.accept_out[2 * a.batch + b] = (a.positions ? a.positions[b] : 0) + ch.row + 1;
    if (a.logprobs) {
      float lp = -INFINITY;
      if (token >= 0)
        lp = c == 0.0f ? 0.0f
                       : static_cast<float>((static_cast<double>(logit(as_float(zr[token]))) - ch.top) * c * 0.6931471805599453 -
                                            log(static_cast<double>(ch.sum)));
      a.logprobs[static_cast<long long>(b) * rows + ch.row] = lp;
    }
  }
}

const char* const kMe = "mk_verify_drafts";

mk_status check_shape(const mk_verify_drafts_args& a, int device) {
  if (a.batch < 0 || a.rows < 1 || a.rows > kMaxRows || static_cast<int64_t>(a.batch) * a.rows > 1 << 20)
    return refuse(MK_ERR_INVALID_ARG, kMe, "batch %d, rows %d", a.batch, a.rows);
  if (a.vocab < 1 || a.vocab > 1 << 24) return refuse(MK_ERR_INVALID_ARG, kMe, "vocab %d", a.vocab);
  if (a.dtype != MK_BF16 && a.dtype != MK_F16 && a.dtype != MK_F32) return refuse(MK_ERR_UNSUPPORTED, kMe, "dtype %d", a.dtype);
  return check_device(kMe, device);
}

int parts_of(const mk_verify_drafts_args& a) {
  const int parts = (a.vocab + 16383) / 16384;
  return parts > kMaxParts ? kMaxParts : parts;
}
uint64_t workspace_of(const mk_verify_drafts_args& a) {
  return static_cast<uint64_t>(a.batch) * (2 * a.rows - 1) * parts_of(a) * sizeof(Part);
}

mk_status check(const mk_verify_drafts_args& a, int device) {
  if (mk_status s = check_shape(a, device)) return s;
  if (a.batch == 0) return MK_OK;
  if (!a.logits || !a.tokens || !a.noise || !a.accept_out || (a.rows > 1 && !a.uniforms))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a required pointer is NULL");
  const unsigned size = a.dtype == MK_F32 ? 4 : 2;
  if (!aligned({a.logits, a.draft_logits}, size) ||
      !aligned({a.tokens, a.n_drafts, a.positions, a.temperature, a.uniforms, a.noise, a.accept_out, a.logprobs, a.status}, 4) ||
      !aligned(a.workspace, 16))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a misaligned pointer");
  // the stride of one row is never used
  const int64_t targets = static_cast<int64_t>(a.batch) * a.rows, draft_rows = targets - a.batch;
  if ((targets > 1 && a.logits_stride < a.vocab) || (a.draft_logits && draft_rows > 1 && a.draft_stride < a.vocab) ||
      (a.batch > 1 && a.noise_stride < a.vocab))
    return refuse(MK_ERR_INVALID_ARG, kMe, "rows shorter than the vocabulary");
  const uint64_t need = workspace_of(a);
  if (!a.workspace || a.workspace_bytes < 0 || static_cast<uint64_t>(a.workspace_bytes) < need)
    return refuse(MK_ERR_INVALID_ARG, kMe, "workspace of %lld bytes, %llu needed", static_cast<long long>(a.workspace_bytes),
                  static_cast<unsigned long long>(need));
  return MK_OK;
}

template <typename T>
cudaError_t launch(const Work& w, int ctas, cudaStream_t s) {
  const mk_verify_drafts_args& a = w.a;
  const unsigned all = static_cast<unsigned>(a.batch) * (a.draft_logits ? 2 * a.rows - 1 : a.rows);
  if (const cudaError_t e = start(stats_kernel<T>, all * w.parts, kThreads, 0, s, w)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, draw_kernel<T>, w, ctas);
}

}  // namespace
}  // namespace drafts
}  // namespace mkop

extern "C" mk_status mk_verify_drafts_workspace(const mk_verify_drafts_args* p, int device, uint64_t* bytes) {
  using namespace mkop::drafts;
  if (!p || !bytes) return MK_ERR_INVALID_ARG;
  if (mk_status s = check_shape(*p, device)) return s;
  *bytes = workspace_of(*p);
  return MK_OK;
}

extern "C" mk_status mk_verify_drafts_check(const mk_verify_drafts_args* p, int device) {
  return p ? mkop::drafts::check(*p, device) : MK_ERR_INVALID_ARG;
}

extern "C" mk_status mk_verify_drafts(const mk_verify_drafts_args* p, int device, void* stream) {
  using namespace mkop;
  using namespace mkop::drafts;
  if (!p) return MK_ERR_INVALID_ARG;
  if (mk_status s = check(*p, device)) return s;
  if (p->batch == 0) return MK_OK;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(kMe, guard.err);
  Work w;
  w.a = *p;
  if (w.a.rows == 1) w.a.draft_logits = nullptr;
  w.parts = parts_of(w.a);
  w.part = static_cast<Part*>(w.a.workspace);
  const int ctas = 8;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(kMe, p->dtype == MK_BF16 ? launch<__nv_bfloat16>(w, ctas, s)
                       : p->dtype == MK_F16 ? launch<__half>(w, ctas, s) : launch<float>(w, ctas, s));
}
