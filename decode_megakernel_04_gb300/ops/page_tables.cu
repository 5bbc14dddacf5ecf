// mk_page_tables: the page table rows and the slot map of one step from the requests' lengths.
//
// Three prefix sums over the requests (new tokens, pages taken, pages returned) place everything; after them each
// token, each taken page and each returned page is computed on its own. One cluster of up to 8 CTAs runs the whole
// call: every CTA repeats the sums (a few thousand integers), the CTAs share the tokens, and the one value that is
// read by all and written by one (the ring's state, lens over held) is written behind a cluster barrier, so the
// call is one launch that needs no workspace and may update its state in place. Pages are taken from the front of the
// free run and returned behind its end; with n_free + returned <= ring_size (checked) the two never touch one
// entry, so they need no order between them.
#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mkop {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = MK_PAGE_TABLES_MAX_BATCH;
constexpr int kPer = kMaxBatch / kThreads;  // requests per thread
constexpr int kRun = 8;  // neighbouring tokens of one thread, where there are many
static_assert(kMaxBatch % kThreads == 0, "whole requests per thread");

struct Sums {
  long long tokens, taken, returned;
};

__device__ inline Sums add(const Sums& a, const Sums& b) {
  return {a.tokens + b.tokens, a.taken + b.taken, a.returned + b.returned};
}

// The last index i in [0, n) with at[i] <= x (at[0] = 0, ascending; equal entries: the last of them).
__device__ inline int owner_of(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(const __grid_constant__ mk_page_tables_args a) {
  extern __shared__ int sm[];
  const int B = a.batch, P = a.page_size;
  int* tok0 = sm;                // [B] first token of each request
  int* take0 = sm + B;           // [B] first taken page
  int* back0 = sm + 2 * B;       // [B] first returned page
  int* have = sm + 3 * B;        // [B] pages the row holds before the call
  int* first = sm + 4 * B;       // [B] position of the first new token
  __shared__ Sums warp_sum[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster.block_rank(), n_ctas = cluster.num_blocks();
  const int head = a.ring_state[0], n_free = a.ring_state[1];

  const int per = (B + kThreads - 1) / kThreads;
  Sums mine[kPer];
  Sums sum{0, 0, 0};
  const long long most = static_cast<long long>(a.max_pages) * P;
  bool bad = head < 0 || head >= a.ring_size || n_free < 0 || n_free > a.ring_size;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    mine[i] = sum;
    if (i >= per || b >= B) continue;
    const int held = a.held[b], start = a.start[b], count = a.count[b];
    const long long len = static_cast<long long>(start) + count;
    if (held < 0 || held > most || start < 0 || start > held || count < 0 || len > most) {
      bad = true;
      continue;
    }
    const int h = static_cast<int>((held + static_cast<long long>(P) - 1) / P), n = static_cast<int>((len + P - 1) / P);
    have[b] = h;
    first[b] = start;
    sum = add(sum, {count, n > h ? n - h : 0, n < h ? h - n : 0});
  }
  // exclusive sums over the block
  Sums incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o{__shfl_up_sync(~0u, incl.tokens, d), __shfl_up_sync(~0u, incl.taken, d),
                 __shfl_up_sync(~0u, incl.returned, d)};
    if (lane >= d) incl = add(incl, o);
  }
  if (lane == 31) warp_sum[warp] = incl;
  bad = __syncthreads_or(bad);
  Sums base{incl.tokens - sum.tokens, incl.taken - sum.taken, incl.returned - sum.returned}, total{0, 0, 0};
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base = add(base, warp_sum[w]);
    total = add(total, warp_sum[w]);
  }
  int why = 0;
  if (bad) {
    why = MK_OP_BAD_LENGTH;
  } else {
    if (total.taken > n_free) why |= MK_OP_NO_PAGES;
    if (total.tokens > a.n_tokens) why |= MK_OP_NO_ROOM;
    if (n_free + total.returned > a.ring_size) why |= MK_OP_BAD_LENGTH;
  }

  const int step = n_ctas * kThreads, id = rank * kThreads + tid;
  if (why) {  // the same decision in every CTA
    for (int t = id; t < a.n_tokens; t += step) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = 0;
      if (a.owners) a.owners[t] = -1;
    }
    cluster.sync();
    if (rank == 0) {
      if (tid == 0) {
        flag(a.status, why);
        a.ring_state_out[0] = head;
        a.ring_state_out[1] = n_free;
      }
      for (int b = tid; b < B; b += kThreads)
        if (a.lens) a.lens[b] = a.held[b];
      if (a.starts)
        for (int b = tid; b <= B; b += kThreads) a.starts[b] = 0;
    }
    return;
  }

  // every sum fits 32 bits now: tokens <= n_tokens, taken and returned <= ring_size
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= B) continue;
    const Sums at = add(base, mine[i]);
    tok0[b] = static_cast<int>(at.tokens);
    take0[b] = static_cast<int>(at.taken);
    back0[b] = static_cast<int>(at.returned);
  }
  __syncthreads();
  const int n_tok = static_cast<int>(total.tokens), n_take = static_cast<int>(total.taken);
  const int n_back = static_cast<int>(total.returned);
  const unsigned size = a.ring_size;
  const bool whole = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.owners)) & 15) == 0;

  int flags = 0;
  auto page_of = [&](int b, int k) {
    const int h = have[b];
    return k < h ? a.table[b * a.table_stride + k] : a.ring[(static_cast<unsigned>(head) + take0[b] + (k - h)) % size];
  };
  auto put = [&](int t, long long slot, int pos, int b) {
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
    if (a.owners) a.owners[t] = b;
  };
  if (a.n_tokens <= kRun * step) {
    for (int t = id; t < a.n_tokens; t += step) {
      long long slot = -1;
      int pos = 0, b = -1;
      if (t < n_tok) {
        b = owner_of(tok0, B, t);
        pos = first[b] + t - tok0[b];
        const int k = pos / P, page = page_of(b, k);
        if (page >= 0 && page < a.n_pages) slot = static_cast<long long>(page) * P + (pos - k * P);
        else flags |= MK_OP_BAD_PAGE;
      }
      put(t, slot, pos, b);
    }
  } else {
    // Many tokens: a thread takes kRun neighbours, which mostly share a request and a page: one search and one or two
    // page lookups for all of them, and whole 32-byte sectors of each output.
    for (long long u = id; u * kRun < a.n_tokens; u += step) {
      const int t0 = static_cast<int>(u) * kRun;
      int b = -1, end = 0, pos = 0, at = P;  // end: first token of the next request; at: place on the page
      long long base = -1;
      long long slot[kRun];
      int where[kRun], who[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int t = t0 + i;
        slot[i] = -1, where[i] = 0, who[i] = -1;
        if (i >= n_tok - t0) continue;
        ++pos;
        if (b < 0 || t >= end) {
          b = owner_of(tok0, B, t);
          end = b + 1 < B ? tok0[b + 1] : n_tok;
          pos = first[b] + t - tok0[b];
          at = P;
        }
        if (at >= P) {
          const int k = pos / P, page = page_of(b, k);
          at = pos - k * P;
          const bool ok = page >= 0 && page < a.n_pages;
          base = ok ? static_cast<long long>(page) * P : -1;
          if (!ok) flags |= MK_OP_BAD_PAGE;
        }
        slot[i] = base < 0 ? -1 : base + at;
        where[i] = pos, who[i] = b;
        ++at;
      }
      if (whole && a.n_tokens - t0 >= kRun) {
#pragma unroll
        for (int i = 0; i < kRun; i += 2) *reinterpret_cast<longlong2*>(a.slots + t0 + i) = make_longlong2(slot[i], slot[i + 1]);
#pragma unroll
        for (int i = 0; i < kRun; i += 4) {
          if (a.positions) *reinterpret_cast<int4*>(a.positions + t0 + i) = make_int4(where[i], where[i + 1], where[i + 2], where[i + 3]);
          if (a.owners) *reinterpret_cast<int4*>(a.owners + t0 + i) = make_int4(who[i], who[i + 1], who[i + 2], who[i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (i < a.n_tokens - t0) put(t0 + i, slot[i], where[i], who[i]);
      }
    }
  }
  for (int j = id; j < n_take; j += step) {
    const int b = owner_of(take0, B, j);
    a.table[b * a.table_stride + have[b] + (j - take0[b])] = a.ring[(static_cast<unsigned>(head) + j) % size];
  }
  for (int j = id; j < n_back; j += step) {
    const int b = owner_of(back0, B, j);
    // the row keeps as many pages as it held less those it returns
    const int gone = (b + 1 < B ? back0[b + 1] : n_back) - back0[b];
    a.ring[(static_cast<unsigned>(head) + n_free + j) % size] =
        a.table[b * a.table_stride + have[b] - gone + (j - back0[b])];
  }
  if (flags) flag(a.status, flags);
  cluster.sync();  // every CTA has read the lengths and the ring's state
  if (rank == 0) {
    if (tid == 0) {
      a.ring_state_out[0] = static_cast<int>((static_cast<unsigned>(head) + n_take) % size);
      a.ring_state_out[1] = n_free - n_take + n_back;
      if (a.starts) a.starts[B] = n_tok;
    }
    for (int b = tid; b < B; b += kThreads) {
      if (a.lens) a.lens[b] = first[b] + (b + 1 < B ? tok0[b + 1] : n_tok) - tok0[b];
      if (a.starts) a.starts[b] = tok0[b];
    }
  }
}

}  // namespace
}  // namespace mkop

extern "C" mk_status mk_page_tables(const mk_page_tables_args* p, int device, void* stream) {
  using namespace mkop;
  static const char* me = "mk_page_tables";
  if (!p) return MK_ERR_INVALID_ARG;
  const mk_page_tables_args a = *p;
  if (!a.table || !a.held || !a.start || !a.count || !a.ring || !a.ring_state || !a.ring_state_out ||
      (!a.slots && a.n_tokens > 0))
    return refuse(MK_ERR_INVALID_ARG, me, "a required pointer is NULL");
  if (a.batch < 1 || a.batch > MK_PAGE_TABLES_MAX_BATCH)
    return refuse(MK_ERR_INVALID_ARG, me, "batch %d outside 1..%d", a.batch, MK_PAGE_TABLES_MAX_BATCH);
  if (a.max_pages < 1 || a.page_size < 1 || a.n_pages < 1 || a.n_tokens < 0)
    return refuse(MK_ERR_INVALID_ARG, me, "max_pages %d, page_size %d, n_pages %d, n_tokens %d", a.max_pages,
                  a.page_size, a.n_pages, a.n_tokens);
  if (a.table_stride < a.max_pages) return refuse(MK_ERR_INVALID_ARG, me, "table rows shorter than max_pages");
  if (static_cast<int64_t>(a.max_pages) * a.page_size > INT32_MAX ||
      static_cast<int64_t>(a.n_pages) * a.page_size > INT32_MAX)
    return refuse(MK_ERR_UNSUPPORTED, me, "positions or slots beyond 2^31 - 1");
  if (a.ring_size < a.n_pages) return refuse(MK_ERR_INVALID_ARG, me, "ring of %d for %d pages", a.ring_size, a.n_pages);
  if (mk_status s = check_device(me, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(me, guard.err);
  // 5 ints per request: beyond 2,457 requests more than the 48 KB a kernel has unasked
  const size_t smem = sizeof(int) * 5 * a.batch;
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem<page_tables_kernel>(device, static_cast<int>(sizeof(int) * 5 * kMaxBatch));
    if (e != cudaSuccess) return launched(me, e);
  }
  const int ctas = a.n_tokens <= 4 * kThreads ? 1 : 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launched(me, cudaLaunchKernelEx(&cfg, page_tables_kernel, a));
}
