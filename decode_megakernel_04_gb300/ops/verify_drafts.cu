// mk_verify_drafts: drafted tokens against the target's probabilities from given random numbers, and the token after them.
//
// Two kernels. `stats_kernel`: the largest logit of every row, its first place and the sum of exp((z - largest) / T), one
// pass, a row cut into up to 32 parts so that few rows fill the GPU. `draw_kernel`: up to 64 CTAs for each request. Each joins
// the statistics and walks the drafts (what that reads is small, and asked for before the first kernel has ended), and runs
// the race over its share of the drawn row: the token with the largest weight / noise. The request's last CTA joins the shares.
// With given exponential noise the race is a draw from the weights, and unlike an inverse distribution function it is no sum
// over the vocabulary: a token's quotient depends on that token alone, in fp32, whatever the order of the work.
// Bound by memory: every logit once, and the drawn row, its draft row and the noise. 64 requests of 4 rows of 202048 fp32 logits
// and 3 of the drafts: 92 us, 60 of them for the statistics (6.0 TB/s; rows that n_drafts leaves out are read too); one request of 8 x
// 151936: 18 us, all latencies (the statistics 7, the draw 11: a row's parts, the drafts' probabilities, the race and its join wait for each
// other); 128 rows of 163841 bf16: 48. (Figures of single steps below are with cold caches.)
#include <algorithm>
#include <type_traits>

#include "mk_ops.cuh"

namespace mkop {
namespace drafts {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxParts = 32;    // of a row's statistics: one a lane
constexpr int kMaxShares = 64;   // of a request's race
constexpr int kMaxRows = 64;     // of a request
constexpr int kVectors = 4;      // of 16 bytes that a thread asks for before it uses the first
constexpr int kFlight = 4;       // of a race's elements (rows and noise begin anywhere, so these loads are of one element)

struct Part {
  float top, sum;  // the largest logit, the sum of exp2((z - top) * c)
  int at;          // the first place of the largest; -1: none above -infinity
  int pad;
};
struct Work {
  mk_verify_drafts_args a;
  int parts;       // of a row
  int shares;      // of a race
  Part* part;      // [batch * rows + batch * (rows - 1)][parts]
  float* score;    // [batch][shares] the best quotient of a share and
  int* score_at;   // [batch][shares] its token
  int* ended;      // [batch] shares that are there
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

// log of a token's probability: its logit z of a row with a largest `top` and a `sum`. (The product is rounded once; a
// logarithm in 64 bits takes some thousand cycles, and the 32-bit sum has no more to give.)
__device__ inline float log_p(float z, float top, float sum, float c) {
  return static_cast<float>((static_cast<double>(logit(z)) - top) * c * 0.6931471805599453 - logf(sum));
}

// An online softmax's state of one thread. `base`: the largest so far, 0 while there is none.
struct State {
  float top = -INFINITY, base = 0, sum = 0;
  int at = -1;
  template <int N>
  __device__ void add(const float (&z)[N], int first, float c) {
    float big = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) big = fmaxf(big, z[i]);
    if (big > top) {
      sum *= exp2_fast((top - big) * c);
      top = base = big;
#pragma unroll
      for (int i = N - 1; i >= 0; --i)
        if (z[i] == big) at = first + i;
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

// The logits of 16 bytes
template <typename T>
struct Logits {
  float v[16 / sizeof(T)];
};
template <typename T>
__device__ inline Logits<T> logits_of(const uint4& u) {
  Logits<T> l;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      l.v[i] = logit(__uint_as_float(w[i]));
    } else {
      const float2 f = unpack2<T>(w[i]);
      l.v[2 * i] = logit(f.x), l.v[2 * i + 1] = logit(f.y);
    }
  }
  return l;
}

// Part y of row x (target rows, then draft rows).
template <typename T>
__global__ void __launch_bounds__(kThreads) stats_kernel(const __grid_constant__ Work w) {
  __shared__ Part red[kWarps];
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
  if (!draft && part == 0 && tid == 0 && row == b * a.rows) w.ended[b] = 0;
  State s;
  // elements up to the first on 16 bytes, vectors, elements behind the last whole one
  constexpr int kPer = 16 / sizeof(T);
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z + i0) % 16 / sizeof(T));
  const int v0 = min(i1, i0 + (off ? kPer - off : 0)), nv = (i1 - v0) / kPer;
  auto one = [&](int i) {
    const float v[1] = {logit(as_float(z[i]))};
    s.add(v, i, c);
  };
  if (i0 + tid < v0) one(i0 + tid);
  const uint4* from = reinterpret_cast<const uint4*>(z + v0);
  for (int k = tid; k < nv; k += kVectors * kThreads) {
    uint4 u[kVectors];
#pragma unroll
    for (int x = 0; x < kVectors; ++x)
      if (k + x * kThreads < nv) u[x] = from[k + x * kThreads];
#pragma unroll
    for (int x = 0; x < kVectors; ++x)
      if (k + x * kThreads < nv) s.add(logits_of<T>(u[x]).v, v0 + (k + x * kThreads) * kPer, c);
  }
  if (v0 + nv * kPer + tid < i1) one(v0 + nv * kPer + tid);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float otop = __shfl_xor_sync(~0u, s.top, d), osum = __shfl_xor_sync(~0u, s.sum, d);
    const int oat = __shfl_xor_sync(~0u, s.at, d);
    s.join(otop, osum, oat, c);
  }
  if ((tid & 31) == 0) red[tid >> 5] = {s.top, s.sum, s.at, 0};
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < kWarps; ++k) s.join(red[k].top, red[k].sum, red[k].at, c);
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
__global__ void __launch_bounds__(kThreads, 6) draw_kernel(const __grid_constant__ Work w) {
  __shared__ Part stats[2 * kMaxRows];
  __shared__ Chosen chosen;
  __shared__ float draft_log_p[kMaxRows];
  __shared__ int verdict[kMaxRows];  // 1: taken, 0: refused, -1: no token of the vocabulary
  __shared__ float best_score[kWarps];
  __shared__ int best_at[kWarps];
  __shared__ bool last;
  const mk_verify_drafts_args& a = w.a;
  const int b = blockIdx.x / w.shares, share = blockIdx.x - b * w.shares, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = a.rows, all = a.draft_logits ? 2 * rows - 1 : rows;
  const float c = per_log2(a.temperature ? a.temperature[b] : 1.0f);
  const T* z = static_cast<const T*>(a.logits) + static_cast<long long>(b) * rows * a.logits_stride;
  const T* y = static_cast<const T*>(a.draft_logits) + static_cast<long long>(b) * (rows - 1) * a.draft_stride;
  // ---- what the drafts need of the inputs, before the statistics are there (the first kernel began after whatever wrote the inputs)
  const int asked = a.n_drafts ? a.n_drafts[b] : rows - 1, n = min(max(asked, 0), rows - 1);
  int x = -1;
  float zx = 0, yx = 0, uniform = 0;
  if (tid < n) {
    x = a.tokens[static_cast<long long>(b) * rows + tid + 1];
    uniform = a.uniforms[static_cast<long long>(b) * (rows - 1) + tid];
    if (x >= 0 && x < a.vocab) {
      zx = as_float(z[tid * a.logits_stride + x]);
      if (a.draft_logits) yx = as_float(y[tid * a.draft_stride + x]);
    }
  }
  const float* noise = a.noise + b * a.noise_stride;
  const int i0 = static_cast<int>(static_cast<long long>(a.vocab) * share / w.shares);
  const int i1 = static_cast<int>(static_cast<long long>(a.vocab) * (share + 1) / w.shares);
  // (and the noise on its way: a request alone 21.0 -> 19.3 us)
  if (c != 0.0f)
    for (int i = i0 + tid * 32; i < i1; i += kThreads * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + i));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the rows' statistics ----------------------------------------------------------------------------------------
  for (int r = warp; r < all; r += kWarps) {
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
  // ---- the drafts, each by a thread, up to the first that is refused ---------------------------------------------------
  const bool says = share == 0;  // one CTA writes
  if (tid < n) {
    auto log_of = [&](float logit_x, const Part& s) -> float {
      if (s.at < 0) return -INFINITY;
      if (c == 0.0f) return x == s.at ? 0.0f : -INFINITY;
      return log_p(logit_x, s.top, s.sum, c);
    };
    int good = -1;
    if (x >= 0 && x < a.vocab) {
      const float lp = log_of(zx, stats[tid]), q = a.draft_logits ? expf(log_of(yx, stats[rows + tid])) : 1.0f;
      // (the product in 64 bits: a uniform number below 1 of equal probabilities is below them)
      good = static_cast<double>(uniform) * q < expf(lp);
      draft_log_p[tid] = lp;
    }
    verdict[tid] = good;
  }
  __syncthreads();
  if (tid == 0) {
    if (says && asked != n) flag(a.status, MK_OP_BAD_LENGTH);
    int r = 0;
    for (; r < n && verdict[r] == 1; ++r)
      if (says && a.logprobs) a.logprobs[static_cast<long long>(b) * rows + r] = draft_log_p[r];
    if (says && r < n && verdict[r] < 0) flag(a.status, MK_OP_BAD_TOKEN);
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
  const bool race = ch.token >= 0 && c != 0.0f;
  if (!race && share) return;
  if (race) {
    // ---- the race ----------------------------------------------------------------------------------------------------
    const T* yr = y + ch.row * a.draft_stride;
    const int out = ch.cut && !a.draft_logits ? a.tokens[static_cast<long long>(b) * rows + ch.row + 1] : -1;  // not drawn
    const bool minus = ch.cut && a.draft_logits && ch.draft_top > -INFINITY;
    const float by = 1.0f / ch.sum, draft_by = minus ? 1.0f / ch.draft_sum : 0.0f;
    // A token's weight where a draft was refused, but for `out`; else its probability.
    auto weight = [&](T z_in, T y_in, bool less) -> float {
      // (rounded products, so that equal probabilities leave 0 and not what a fused difference would)
      const float p = __fmul_rn(exp2_fast((logit(as_float(z_in)) - ch.top) * c), by);
      return less ? fmaxf(p - __fmul_rn(exp2_fast((logit(as_float(y_in)) - ch.draft_top) * c), draft_by), 0.0f) : p;
    };
    // The best of tokens from .. to - 1, for every thread. `cut`: of max(p - q, 0), or without `out`.
    auto best = [&](int from, int to, bool cut, float& score, int& at) {
      score = 0, at = -1;
      const bool less = cut && minus;
      const int left_out = cut ? out : -1;
      // Batches that end inside to and are without the token left out have no comparisons of indices, and loads from one address.
      auto batch = [&](int i, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        T p_in[kFlight], q_in[kFlight];
        float e[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int j = kWhole ? i + k * kThreads : min(i + k * kThreads, to - 1);
          p_in[k] = zr[j];
          e[k] = noise[j];
          if (less) q_in[k] = yr[j];
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int j = i + k * kThreads;
          float p = weight(p_in[k], q_in[k], less);
          if (!kWhole && (j >= to || j == left_out)) p = 0.0f;
          const float s = __fdividef(p, e[k] + 0.0f);  // (-0, as -log(1) is, counts as 0; past 2^126 the quotient is 0)
          if (s > score) score = s, at = j;
        }
      };
      for (int first = from; first < to; first += kFlight * kThreads) {
        const int end = first + kFlight * kThreads;
        if (end <= to && (left_out < first || left_out >= end)) batch(first + tid, std::true_type{});
        else batch(first + tid, std::false_type{});
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const float os = __shfl_xor_sync(~0u, score, d);
        const int oa = __shfl_xor_sync(~0u, at, d);
        better(score, at, os, oa);
      }
      if (lane == 0) best_score[warp] = score, best_at[warp] = at;
      __syncthreads();
      for (int k = 0; k < kWarps; ++k) better(score, at, best_score[k], best_at[k]);
      __syncthreads();
    };
    float score;
    best(i0, i1, ch.cut, score, token);
    if (w.shares > 1) {
      const long long place = static_cast<long long>(b) * w.shares;
      if (tid == 0) {
        w.score[place + share] = score, w.score_at[place + share] = token;
        __threadfence();
        last = atomicAdd(&w.ended[b], 1) == w.shares - 1;
        __threadfence();
      }
      __syncthreads();
      if (!last) return;
      // (every warp; a share's place has been written by another CTA of this launch)
      score = 0, token = -1;
      for (int k = lane; k < w.shares; k += 32) better(score, token, __ldcg(&w.score[place + k]), __ldcg(&w.score_at[place + k]));
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const float os = __shfl_xor_sync(~0u, score, d);
        const int oa = __shfl_xor_sync(~0u, token, d);
        better(score, token, os, oa);
      }
    }
    // No token, as max(p - q, 0) is 0 everywhere, as far as fp32 shows it: a draw from p (too seldom to share). Not so where tokens
    // with a weight have noise that does not draw them.
    if (token < 0 && ch.cut) {
      bool barred = false;
      for (int j = tid; j < a.vocab; j += kThreads)
        barred |= j != out && !(noise[j] >= 0.0f && noise[j] <= 0x1p126f) && weight(zr[j], minus ? yr[j] : zr[j], minus) > 0.0f;
      if (!__syncthreads_or(barred)) best(0, a.vocab, false, score, token);
    }
  }
  if (tid == 0) {
    a.accept_out[b] = ch.row + 1;
    a.accept_out[a.batch + b] = token;
    a.accept_out[2 * a.batch + b] = (a.positions ? a.positions[b] : 0) + ch.row + 1;
    if (a.logprobs) {
      float lp = -INFINITY;
      if (token >= 0) lp = c == 0.0f ? 0.0f : log_p(as_float(zr[token]), ch.top, ch.sum, c);
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

// CTAs that an SM holds at once, and SMs that workspaces are made for: their sizes and the checks of arguments need no device. More SMs
// are not made use of by few rows.
constexpr int64_t kStatsCtas = 8, kRaceCtas = 6, kMostSms = 152;

int64_t all_rows(const mk_verify_drafts_args& a) { return static_cast<int64_t>(a.batch) * (2 * a.rows - 1); }
int whole_parts(const mk_verify_drafts_args& a) { return std::min(kMaxParts, (a.vocab + 16383) / 16384); }
// parts of 16384 elements; where that leaves SMs with less than they hold, more and smaller ones (one request of 15 rows: 480 parts
// instead of 150, statistics 12 -> 7 us)
int parts_of(const mk_verify_drafts_args& a, int64_t sms) {
  const int64_t more = std::min<int64_t>({kMaxParts, kStatsCtas * sms / std::max<int64_t>(1, all_rows(a)), (a.vocab + 1023) / 1024});
  return std::max<int64_t>(whole_parts(a), more);
}
// So many shares that the GPU holds all requests' at once (6 CTAs an SM; 4 of them with 8 elements in flight leave more SMs with one
// less than others: 128 rows 58.0 -> 55.6 us), of 1024 tokens at least
int shares_of(const mk_verify_drafts_args& a, int64_t sms) {
  return std::max<int64_t>(1, std::min<int64_t>({kMaxShares, kRaceCtas * sms / std::max(1, a.batch), (a.vocab + 1023) / 1024}));
}
// What any such parts and shares take: never less for more requests, rows or tokens.
uint64_t workspace_of(const mk_verify_drafts_args& a) {
  const int64_t parts = std::max(all_rows(a) * whole_parts(a), std::min(all_rows(a) * kMaxParts, kStatsCtas * kMostSms));
  const int64_t shares = std::max<int64_t>(a.batch, std::min<int64_t>(static_cast<int64_t>(a.batch) * kMaxShares, kRaceCtas * kMostSms));
  return parts * sizeof(Part) + shares * (sizeof(float) + sizeof(int)) + a.batch * sizeof(int);
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
cudaError_t launch(const Work& w, cudaStream_t s) {
  const mk_verify_drafts_args& a = w.a;
  const unsigned all = static_cast<unsigned>(a.batch) * (a.draft_logits ? 2 * a.rows - 1 : a.rows);
  if (const cudaError_t e = start(stats_kernel<T>, all * w.parts, kThreads, 0, s, w)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.batch * w.shares);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, draw_kernel<T>, w);
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
  int sms = 0;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(kMe, e);
  w.parts = parts_of(w.a, std::min<int64_t>(sms, kMostSms));
  w.shares = shares_of(w.a, std::min<int64_t>(sms, kMostSms));
  w.part = static_cast<Part*>(w.a.workspace);
  w.score = reinterpret_cast<float*>(w.part + static_cast<int64_t>(p->batch) * (2 * p->rows - 1) * w.parts);
  w.score_at = reinterpret_cast<int*>(w.score + static_cast<int64_t>(p->batch) * w.shares);
  w.ended = w.score_at + static_cast<int64_t>(p->batch) * w.shares;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(kMe, p->dtype == MK_BF16 ? launch<__nv_bfloat16>(w, s) : p->dtype == MK_F16 ? launch<__half>(w, s) : launch<float>(w, s));
}
