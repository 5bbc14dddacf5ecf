// mk_logit_controls: penalties, biases and masks on logits, and the greedy token of what is left.
//
// Bound by memory: the logits are read once and written once. What a row's history and biases say about a token is one
// 32-bit word
//   bit 31 seen in the history | bits 11..30 times generated | bits 0..10 its last bias entry + 1
// built in shared memory with integer atomics (any order gives the same word). The pass over the logits only masks; the
// tokens with a word are few and are computed on their own. (Computed inside the pass they cost every warp the whole
// branch: 128 neighbours nearly always hold one.)
// Two forms:
// - Few rows (or a history too long for the other): a cluster of 8 CTAs shares a row, each with an eighth of the
//   vocabulary, one word for each of its tokens, and joins the greedy token through distributed shared memory: one launch.
//   Every CTA reads the whole history.
// - Many rows: that would read histories as often as logits (64 rows with 4 to 8 thousand tokens of history: 82 us against
//   17 for the pass alone). So a plain pass masks and leaves each chunk's largest logit, and a second kernel, one CTA or
//   more a row, gathers the words in a hash table, computes the named tokens, and joins the largest: a chunk whose largest is a
//   named token is looked through again without these. (The other order, words sorted by chunk first and computed in
//   the pass, was slower: 48 against 39 us for these rows, 77 against 70 for 256 rows of 163841 bf16 logits.)
#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mkop {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;        // of a row's cluster
constexpr int kThreads = 1024;  // of the cluster form and of the other's second kernel
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 24576;   // tokens a CTA of the cluster form has words for at a time
constexpr int kPassThreads = 256;
constexpr int kBatch = 4;       // 16-byte groups of logits a thread loads before it stores the first
constexpr int kAhead = 8;       // history tokens a thread loads before it uses the first
constexpr int kPlaces = 16384;  // of the hash table at most
constexpr int kChunkBits = 12;  // of the pass: 2^12 fp32 logits, 2^13 of 16 bits
static_assert(kPassThreads * kBatch * 4 == 1 << kChunkBits, "a chunk is a batch of every thread");
constexpr uint32_t kSeen = 0x80000000u;

struct RowControls {
  float repetition, presence, frequency;
  bool has_repetition, has_presence, has_frequency;
  const float* bias_vals;
};

// Each step rounds on its own, as the definition does.
__device__ inline float control(float z, uint32_t word, const RowControls& c) {
  const uint32_t times = (word >> 11) & 0xfffffu, entry = word & 0x7ffu;
  if (c.has_repetition && (word >> 11)) z = z > 0 ? __fdiv_rn(z, c.repetition) : __fmul_rn(z, c.repetition);
  if (times) {
    if (c.has_frequency) z = __fsub_rn(z, __fmul_rn(c.frequency, static_cast<float>(times)));
    if (c.has_presence) z = __fsub_rn(z, c.presence);
  }
  if (entry) z = __fadd_rn(z, c.bias_vals[entry - 1]);
  return z;
}

// Larger key = larger value, then lower index (0 stands for no token).
__device__ inline unsigned long long key_of(float z, int index) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.0f));  // -0 counts as 0
  const uint32_t rank = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(rank) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}

__device__ inline int token_of(unsigned long long key) {
  return key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
}

__device__ inline unsigned long long larger(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

// 16 bytes of logits as floats
__device__ inline void unpack(const uint4& u, float (&y)[4], const float*) {
  y[0] = __uint_as_float(u.x), y[1] = __uint_as_float(u.y), y[2] = __uint_as_float(u.z), y[3] = __uint_as_float(u.w);
}
template <typename T>
__device__ inline void unpack(const uint4& u, float (&y)[8], const T*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<T>(w[i]);
    y[2 * i] = p.x, y[2 * i + 1] = p.y;
  }
}

// The largest of the block's keys, for every thread.
template <int kWarps>
__device__ inline unsigned long long block_largest(unsigned long long key) {
  __shared__ unsigned long long of_warp[kWarps];
#pragma unroll
  for (int d = 16; d; d >>= 1) key = larger(key, __shfl_xor_sync(~0u, key, d));
  __syncthreads();  // the last call's keys have been read
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = key;
  __syncthreads();
  key = of_warp[threadIdx.x % kWarps];
#pragma unroll
  for (int d = kWarps / 2; d; d >>= 1) key = larger(key, __shfl_xor_sync(~0u, key, d));
  return key;
}

template <typename T>
__device__ inline RowControls controls_of(const mk_logit_controls_args& a, int64_t row) {
  RowControls c;
  c.has_repetition = a.repetition, c.has_presence = a.presence, c.has_frequency = a.frequency;
  c.repetition = a.repetition ? a.repetition[row] : 1.0f;
  c.presence = a.presence ? a.presence[row] : 0.0f;
  c.frequency = a.frequency ? a.frequency[row] : 0.0f;
  c.bias_vals = a.bias_ids ? a.bias_vals + row * a.bias_stride : nullptr;
  return c;
}

// The first `lead` tokens bring the output, and the logits where both can be, to a 16-byte boundary.
template <typename T>
__device__ inline int lead_of(const T* z, const float* out, int vocab) {
  int lead = static_cast<int>((4 - (reinterpret_cast<uintptr_t>(out) >> 2 & 3)) & 3);
  if (sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(z + lead) & 15) == 8) lead += 4;
  return min(vocab, lead);
}

__device__ inline bool bit_set(const int32_t* mask, int v) {
  return !mask || (static_cast<uint32_t>(mask[v >> 5]) >> (v & 31) & 1);
}

// The plain pass over tokens [from, to) with whole groups from g on, by the block's kN threads: masks, stores, and calls
// better(value, token) in ascending order with word(v) = 0 tokens' values, -infinity for the others.
template <int kN, typename T, typename Word, typename Better>
__device__ inline void mask_pass(const T* z, float* out, const int32_t* mask, int from, int g, int to, Word&& word, Better&& better) {
  constexpr int U = 16 / sizeof(T);  // logits of a group
  const int tid = threadIdx.x;
  auto one = [&](int v) {
    const float y = bit_set(mask, v) ? static_cast<float>(z[v]) : -INFINITY;
    out[v] = y;
    better(word(v) ? -INFINITY : y, v);
  };
  if (tid < g - from) one(from + tid);
  // Groups of U, kBatch of them loaded before the first is stored: out may be the logits, so the compiler does not move a
  // load over a store.
  const int groups = (reinterpret_cast<uintptr_t>(z + g) & 15) == 0 ? (to - g) / U : 0;
  const bool split = mask && (g & (U - 1));  // groups whose bits may lie in two words
  for (int i0 = tid; i0 < groups; i0 += kN * kBatch) {
    uint4 x[kBatch];
    uint32_t m0[kBatch], m1[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kN, v = g + U * i;
      if (i >= groups) continue;
      x[k] = *reinterpret_cast<const uint4*>(z + v);
      if (mask) m0[k] = mask[v >> 5];
      if (split) m1[k] = mask[(v + U - 1) >> 5];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kN, v = g + U * i;
      if (i >= groups) continue;
      float y[U];
      unpack(x[k], y, z);
      if (mask) {
        const uint32_t ok = __funnelshift_r(m0[k], split ? m1[k] : 0, v & 31);
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = ok >> u & 1 ? y[u] : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < U; u += 4) *reinterpret_cast<float4*>(out + v + u) = make_float4(y[u], y[u + 1], y[u + 2], y[u + 3]);
#pragma unroll
      for (int u = 0; u < U; ++u) better(word(v + u) ? -INFINITY : y[u], v + u);
    }
  }
  for (int v = g + U * groups + tid; v < to; v += kN) one(v);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    cluster_kernel(const __grid_constant__ mk_logit_controls_args a, int part, int slice) {
  extern __shared__ __align__(16) uint32_t words[];  // [slice + 8]
  __shared__ unsigned long long cta_best;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / kCtas;
  const int rank = blockIdx.x % kCtas;
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* out = a.out + row * a.out_stride;
  const int32_t* mask = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;
  const bool penal = a.history && (a.repetition || a.presence || a.frequency);
  const bool named = penal || a.bias_ids;
  const int32_t* hist = penal ? a.history + row * a.history_stride : nullptr;
  const int32_t* ids = a.bias_ids ? a.bias_ids + row * a.bias_stride : nullptr;
  int total = 0, prompt = 0;
  if (penal) {
    total = a.total_len ? min(max(a.total_len[row], 0), a.max_history) : a.max_history;
    prompt = a.prompt_len ? min(max(a.prompt_len[row], 0), total) : 0;
  }
  // Parts and slices are whole groups, the first with the lead and the last with the tail. Token v of a slice that starts
  // at group boundary g has word v - g + 8.
  const int V = a.vocab, lead = lead_of(z, out, V);
  const int begin = static_cast<int>(min(static_cast<long long>(V), lead + static_cast<long long>(rank) * part));
  const int end = static_cast<int>(min(static_cast<long long>(V), static_cast<long long>(begin) + part));
  // The greedy token so far: this thread meets its tokens in ascending order, so the first of equals stays.
  float best_z = -INFINITY;
  int best_v = -1;
  auto better = [&](float y, int v) {
    if (y > best_z) best_z = y, best_v = v;  // NaN never is
  };

  for (int g = begin; g < end || (g == begin && rank == 0); g += slice) {
    const int from = rank == 0 && g == begin ? 0 : g, to = min(end, g + slice);
    uint32_t* word = words + 8 - g;  // word[v]
    if (named) {
      __syncthreads();  // the last slice's words have been taken
      for (int i = tid; i < (to - g + 8 + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      if (ids) {
        for (int e = tid; e < a.n_biases; e += kThreads) {
          const int v = ids[e];
          if (v >= from && v < to) atomicMax(word + v, static_cast<uint32_t>(e + 1));
        }
        __syncthreads();
      }
      for (int h0 = tid; h0 < total; h0 += kThreads * kAhead) {
        int v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = h0 + i * kThreads < total ? hist[h0 + i * kThreads] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (v[i] < from || v[i] >= to) continue;
          if (h0 + i * kThreads >= prompt) atomicAdd(word + v[i], 1u << 11);
          else atomicOr(word + v[i], kSeen);
        }
      }
      __syncthreads();
    }
    mask_pass<kThreads>(z, out, mask, from, g, to, [&](int v) { return named ? word[v] : 0; }, better);
    if (!named) continue;
    __syncthreads();  // the slice is written; out may be the logits, where a masked one is -infinity by now
    const RowControls c = controls_of<T>(a, row);
    // tokens v[i] >= 0 of the slice, their loads together
    auto touch = [&](int (&v)[kAhead]) {
      uint32_t w[kAhead];
      float y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        w[i] = v[i] >= from && v[i] < to ? atomicExch(word + v[i], 0u) : 0;
        if (w[i]) y[i] = static_cast<float>(z[v[i]]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (!w[i] || !bit_set(mask, v[i])) continue;
        y[i] = control(y[i], w[i], c);
        out[v[i]] = y[i];
        if (y[i] > best_z || (y[i] == best_z && v[i] < best_v)) best_z = y[i], best_v = v[i];
      }
    };
    for (int n = 0; n < 2; ++n) {  // the biases, then the history
      const int32_t* list = n ? hist : ids;
      const int length = n ? total : ids ? a.n_biases : 0;
#pragma unroll 1
      for (int h0 = tid; h0 < length; h0 += kThreads * kAhead) {
        int v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = h0 + i * kThreads < length ? list[h0 + i * kThreads] : -1;
        touch(v);
      }
    }
  }

  const unsigned long long best = block_largest<kWarps>(best_v < 0 ? 0 : key_of(best_z, best_v));
  if (tid == 0) cta_best = best;
  cluster.sync();
  if (rank == 0 && tid < 32 && a.token) {
    unsigned long long all = tid < kCtas ? *cluster.map_shared_rank(&cta_best, tid) : 0;
#pragma unroll
    for (int d = 16; d; d >>= 1) all = larger(all, __shfl_xor_sync(~0u, all, d));
    if (tid == 0) a.token[row] = token_of(all);
  }
  cluster.sync();  // the others' shared memory stays until it has been read
}

// ---- many rows: the plain pass ----------------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kPassThreads, 6)
    pass_kernel(const __grid_constant__ mk_logit_controls_args a, int chunk_bits, int chunks, unsigned long long* largest) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.x / chunks;
  const int n = blockIdx.x - static_cast<int>(row) * chunks;
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* out = a.out + row * a.out_stride;
  const int lead = lead_of(z, out, a.vocab);
  const int g = min(a.vocab, lead + (n << chunk_bits)), to = min(a.vocab, g + (1 << chunk_bits));
  float best_z = -INFINITY;
  int best_v = -1;
  mask_pass<kPassThreads>(z, out, a.allowed ? a.allowed + row * a.allowed_stride : nullptr, n ? g : 0, g, to,
                          [](int) { return 0u; }, [&](float y, int v) {
                            if (y > best_z) best_z = y, best_v = v;
                          });
  if (!a.token) return;
  const unsigned long long best = block_largest<kPassThreads / 32>(best_v < 0 ? 0 : key_of(best_z, best_v));
  if (threadIdx.x == 0) largest[blockIdx.x] = best;
}

// ---- many rows: the named tokens and the join -----------------------------------------------------------------------
// Open addressing over the token, filled to three quarters at most.
struct Table {
  int* tokens;
  uint32_t* words;
  int mask;
  static __device__ uint32_t hash(int v) { return static_cast<uint32_t>(v) * 2654435769u; }
  __device__ int first(int v) const { return static_cast<int>(hash(v) >> 8) & mask; }
  __device__ uint32_t* word_of(int v) {
    for (int i = first(v);; i = (i + 1) & mask) {
      int old = *reinterpret_cast<volatile int*>(tokens + i);
      if (old == -1) old = atomicCAS(tokens + i, -1, v);
      if (old == -1 || old == v) return words + i;
    }
  }
  __device__ bool has(int v) const {
    for (int i = first(v);; i = (i + 1) & mask) {
      if (tokens[i] == v) return true;
      if (tokens[i] == -1) return false;
    }
  }
};

// A cluster of `split` CTAs (1, 2 or 4) has a row, each the tokens whose hash says so.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) named_kernel(const __grid_constant__ mk_logit_controls_args a, int split, int places,
                                                           int chunk_bits, int chunks, const unsigned long long* largest) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ unsigned long long cta_best;
  cg::cluster_group cluster = cg::this_cluster();
  Table table{reinterpret_cast<int*>(smem), smem + places, places - 1};
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / split;
  const uint32_t rank = blockIdx.x % split;
  auto owner = [&](int v) { return Table::hash(v) >> 30 & (split - 1); };
  const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
  float* out = a.out + row * a.out_stride;
  const int32_t* mask = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;
  const int32_t* ids = a.bias_ids ? a.bias_ids + row * a.bias_stride : nullptr;
  const int V = a.vocab;
  if (places) {
    for (int i = tid; i < places / 4; i += kThreads) {  // places is a multiple of 256
      reinterpret_cast<int4*>(table.tokens)[i] = make_int4(-1, -1, -1, -1);
      reinterpret_cast<uint4*>(table.words)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int e = tid; ids && e < a.n_biases; e += kThreads) {
      const int v = ids[e];
      if (v >= 0 && v < V && owner(v) == rank) atomicMax(table.word_of(v), static_cast<uint32_t>(e + 1));
    }
    __syncthreads();
    if (a.history && (a.repetition || a.presence || a.frequency)) {
      const int32_t* hist = a.history + row * a.history_stride;
      const int total = a.total_len ? min(max(a.total_len[row], 0), a.max_history) : a.max_history;
      const int prompt = a.prompt_len ? min(max(a.prompt_len[row], 0), total) : 0;
      for (int h0 = tid; h0 < total; h0 += kThreads * kAhead) {
        int v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = h0 + i * kThreads < total ? hist[h0 + i * kThreads] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (v[i] < 0 || v[i] >= V || owner(v[i]) != rank) continue;
          uint32_t* word = table.word_of(v[i]);
          if (h0 + i * kThreads >= prompt) atomicAdd(word, 1u << 11);
          else atomicOr(word, kSeen);
        }
      }
      __syncthreads();
    }
  }
  const RowControls c = controls_of<T>(a, row);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pass is over and its values are there
  float best_z = -INFINITY;
  int best_v = -1;
  for (int i0 = tid; i0 < places; i0 += kThreads * kAhead) {
    int v[kAhead];
    float y[kAhead];
    bool ok[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {  // out may be the logits, where a masked one is -infinity by now
      v[i] = i0 + i * kThreads < places ? table.tokens[i0 + i * kThreads] : -1;
      ok[i] = v[i] >= 0;
      if (!ok[i]) continue;
      y[i] = static_cast<float>(z[v[i]]);
      ok[i] = bit_set(mask, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!ok[i]) continue;
      y[i] = control(y[i], table.words[i0 + i * kThreads], c);
      out[v[i]] = y[i];
      if (y[i] > best_z || (y[i] == best_z && v[i] < best_v)) best_z = y[i], best_v = v[i];
    }
  }
  if (!a.token) return;
  unsigned long long named = block_largest<kWarps>(best_v < 0 ? 0 : key_of(best_z, best_v));
  if (tid == 0) cta_best = named;
  if (split > 1) {
    cluster.sync();
    if (rank) {
      cluster.sync();  // this CTA's table stays until it has been read
      return;
    }
    for (int r = 1; r < split; ++r) named = larger(named, *cluster.map_shared_rank(&cta_best, r));
  }
  auto is_named = [&](int v) {
    if (!places) return false;
    const Table of{split > 1 ? cluster.map_shared_rank(table.tokens, owner(v)) : table.tokens, nullptr, table.mask};
    return of.has(v);
  };
  // The largest of the chunks' largest that is not a named token. A chunk is looked through again at most once.
  const int lead = lead_of(z, out, V);
  unsigned long long best = 0;
  for (int n0 = 0; n0 < chunks; n0 += kThreads) {
    unsigned long long mine = n0 + tid < chunks ? largest[row * chunks + n0 + tid] : 0;
    for (;;) {
      const unsigned long long top = block_largest<kWarps>(mine);
      if (top <= larger(best, named)) break;
      const int v = token_of(top);
      if (!is_named(v)) {
        best = top;
        break;
      }
      const int n = max(v - lead, 0) >> chunk_bits, from = n ? lead + (n << chunk_bits) : 0;
      const int to = min(V, lead + ((n + 1) << chunk_bits));
      best_z = -INFINITY, best_v = -1;
      for (int u0 = from + tid; u0 < to; u0 += kThreads * kAhead) {
        float y[kAhead];
        bool ok[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int u = min(u0 + i * kThreads, to - 1);
          y[i] = static_cast<float>(z[u]);
          ok[i] = bit_set(mask, u) && u0 + i * kThreads < to;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int u = u0 + i * kThreads;
          if (ok[i] && y[i] > best_z && !is_named(u)) best_z = y[i], best_v = u;
        }
      }
      const unsigned long long again = block_largest<kWarps>(best_v < 0 ? 0 : key_of(best_z, best_v));
      if (n0 + tid == n) mine = again;
    }
  }
  if (tid == 0) a.token[row] = token_of(larger(best, named));
  if (split > 1) cluster.sync();
}

// ---- host -------------------------------------------------------------------------------------------------------------
struct Plan {
  bool clusters;
  int split, places, chunk_bits, chunks;
  size_t bytes;
};

Plan plan(const mk_logit_controls_args& a, int sms) {
  const bool penal = a.history && (a.repetition || a.presence || a.frequency);
  const int entries = (penal ? a.max_history : 0) + (a.bias_ids ? a.n_biases : 0);
  Plan p{};
  p.clusters = a.rows * static_cast<int64_t>(kCtas) <= sms || entries > kPlaces / 4 * 3;
  if (p.clusters) return p;
  if (entries)
    for (p.places = 256; p.places / 4 * 3 < entries;) p.places *= 2;
  // CTAs of a row's named tokens, while every cluster has SMs: 64 rows of 151936 fp32 logits, 8192 tokens of history 37.9 us with
  // one, 32.7 with two; 2048: 24.6, 23.8; 256: 20.4, 20.9; 32 rows, 8192: 30.5, 24.9, 23.3 with four; 100 rows, 4096: 34.6, 43.7.
  p.split = entries <= 1024 || a.rows * 2 > sms ? 1 : a.rows * 4 > sms ? 2 : 4;
  p.chunk_bits = a.dtype == MK_F32 ? kChunkBits : kChunkBits + 1;
  p.chunks = (a.vocab + (1 << p.chunk_bits) - 1) >> p.chunk_bits;
  p.bytes = sizeof(unsigned long long) * p.chunks * a.rows;
  return p;
}

template <typename T>
cudaError_t launch_clusters(const mk_logit_controls_args& a, int device, cudaStream_t s) {
  const bool named = a.bias_ids || (a.history && (a.repetition || a.presence || a.frequency));
  // a part is an eighth of the row in whole groups, in equal slices (without words: one)
  const int share = (a.vocab + kCtas - 1) / kCtas, slices = named ? (share + kSlice - 1) / kSlice : 1;
  const int slice = ((share + slices - 1) / slices + 31) & ~31, part = slice * slices;
  const cudaError_t e = allow_smem<cluster_kernel<T>>(device, sizeof(uint32_t) * (kSlice + 32 + 8));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = named ? sizeof(uint32_t) * (slice + 8) : 0;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cluster_kernel<T>, a, part, slice);
}

template <typename T>
cudaError_t launch_pass(const mk_logit_controls_args& a, const Plan& p, int device, cudaStream_t s) {
  unsigned long long* largest = static_cast<unsigned long long*>(a.workspace);
  cudaError_t e = start(pass_kernel<T>, static_cast<unsigned>(a.rows) * p.chunks, kPassThreads, 0, s, a, p.chunk_bits, p.chunks, largest);
  if (e != cudaSuccess || (!p.places && !a.token)) return e;
  if ((e = allow_smem<named_kernel<T>>(device, 8 * kPlaces)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * p.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 8 * static_cast<size_t>(p.places);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, named_kernel<T>, a, p.split, p.places, p.chunk_bits, p.chunks, static_cast<const unsigned long long*>(largest));
}

mk_status check_shape(const mk_logit_controls_args& a, const char* me, int device) {
  if (a.rows < 0 || a.rows > 1 << 20 || a.vocab < 1 || a.vocab > 1 << 24)
    return refuse(MK_ERR_INVALID_ARG, me, "rows %d, vocab %d", a.rows, a.vocab);
  if (a.dtype != MK_F32 && a.dtype != MK_BF16 && a.dtype != MK_F16) return refuse(MK_ERR_UNSUPPORTED, me, "dtype %d", a.dtype);
  if (a.max_history < 0 || a.max_history > MK_LOGIT_MAX_HISTORY || a.n_biases < 0 || a.n_biases > MK_LOGIT_MAX_BIASES)
    return refuse(MK_ERR_UNSUPPORTED, me, "max_history %d (at most %d), n_biases %d (at most %d)", a.max_history,
                  MK_LOGIT_MAX_HISTORY, a.n_biases, MK_LOGIT_MAX_BIASES);
  if (static_cast<int64_t>(a.rows) * ((a.vocab + 4095) / 4096) > INT32_MAX)
    return refuse(MK_ERR_UNSUPPORTED, me, "%d rows of %d logits", a.rows, a.vocab);
  return check_device(me, device);
}

// Everything that a call of at least one row can be refused for before the device is touched.
mk_status check(const mk_logit_controls_args& a, const char* me, int device) {
  if (mk_status s = check_shape(a, me, device)) return s;
  if (a.rows == 0) return MK_OK;
  if (!a.logits || !a.out) return refuse(MK_ERR_INVALID_ARG, me, "a required pointer is NULL");
  if (!a.history && a.max_history > 0 && (a.repetition || a.presence || a.frequency))
    return refuse(MK_ERR_INVALID_ARG, me, "penalties without a history");
  if (!a.bias_ids != !a.bias_vals) return refuse(MK_ERR_INVALID_ARG, me, "bias ids and values come together");
  if (a.logits_stride < a.vocab || a.out_stride < a.vocab || (a.history && a.history_stride < a.max_history) ||
      (a.bias_ids && a.bias_stride < a.n_biases) || (a.allowed && a.allowed_stride < (a.vocab + 31) / 32))
    return refuse(MK_ERR_INVALID_ARG, me, "a row stride is shorter than its row");
  if (a.logits == a.out && (a.dtype != MK_F32 || a.logits_stride != a.out_stride))
    return refuse(MK_ERR_INVALID_ARG, me, "out may be logits only in fp32 with one stride");
  if (!aligned(a.logits, a.dtype == MK_F32 ? 4 : 2) || 
      !aligned({a.out, a.token, a.history, a.prompt_len, a.total_len, a.repetition, a.presence, a.frequency, a.bias_ids, a.bias_vals,
                a.allowed}, 4))
    return refuse(MK_ERR_INVALID_ARG, me, "a misaligned pointer");
  return MK_OK;
}

// The plan on the current device `device`, and whether the workspace holds what it needs.
mk_status plan_within(const mk_logit_controls_args& a, const char* me, int device, Plan* p) {
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);
  *p = plan(a, sms);
  if (p->bytes && (!a.workspace || !aligned(a.workspace, 8) || a.workspace_bytes < static_cast<int64_t>(p->bytes)))
    return refuse(MK_ERR_INVALID_ARG, me, "workspace of %lld bytes, %zu needed", static_cast<long long>(a.workspace_bytes), p->bytes);
  return MK_OK;
}

}  // namespace
}  // namespace mkop

extern "C" mk_status mk_logit_controls_check(const mk_logit_controls_args* args, int device) {
  using namespace mkop;
  static const char* me = "mk_logit_controls_check";
  if (!args) return MK_ERR_INVALID_ARG;
  if (mk_status s = check(*args, me, device)) return s;
  if (args->rows == 0) return MK_OK;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  Plan p;
  return plan_within(*args, me, device, &p);
}

extern "C" mk_status mk_logit_controls(const mk_logit_controls_args* args, int device, void* stream) {
  using namespace mkop;
  static const char* me = "mk_logit_controls";
  if (!args) return MK_ERR_INVALID_ARG;
  const mk_logit_controls_args a = *args;
  if (mk_status s = check(a, me, device)) return s;
  if (a.rows == 0) return MK_OK;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  Plan p;
  if (mk_status s = plan_within(a, me, device, &p)) return s;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.clusters)
    return launched(me, a.dtype == MK_F32 ? launch_clusters<float>(a, device, s)
                        : a.dtype == MK_BF16 ? launch_clusters<__nv_bfloat16>(a, device, s)
                                             : launch_clusters<__half>(a, device, s));
  return launched(me, a.dtype == MK_F32 ? launch_pass<float>(a, p, device, s)
                      : a.dtype == MK_BF16 ? launch_pass<__nv_bfloat16>(a, p, device, s)
                                           : launch_pass<__half>(a, p, device, s));
}

extern "C" mk_status mk_logit_controls_workspace(const mk_logit_controls_args* p, int device, uint64_t* bytes) {
  using namespace mkop;
  static const char* me = "mk_logit_controls_workspace";
  if (!p || !bytes) return MK_ERR_INVALID_ARG;
  if (mk_status s = check_shape(*p, me, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);
  *bytes = p->rows ? plan(*p, sms).bytes : 0;
  return MK_OK;
}
