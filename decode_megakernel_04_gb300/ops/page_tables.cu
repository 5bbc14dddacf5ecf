// mk_page_tables: the page table rows and the slot map of one step from the requests' lengths.
//
// Three prefix sums over the requests (new tokens, pages taken, pages returned) place everything; after them each
// token, each taken page and each returned page is computed on its own, so any number of CTAs share the work and each
// repeats the sums (a few thousand integers). Pages are taken from the front of the free run and returned behind its
// end; with n_free + returned <= ring_size (checked) the two never touch one entry, so they need no order between
// them. What is read by all and may be written in place (the ring's state, lens over the lengths) is the one hazard:
// a call of one CTA writes it behind a barrier, a larger one in place takes a second launch for it.
// Bound by latency: one token of one request 3.8 us on the GPU, 256 requests with 197 thousand tokens 6.1 us (their 2 MB
// at the copy rate: 0.3), of which the sums and the binary searches' dependent loads are most; 25 us with one CTA.
#include "mk_ops.cuh"

namespace mkop {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = MK_PAGE_TABLES_MAX_BATCH;
constexpr int kPer = kMaxBatch / kThreads;  // requests per thread
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

// tokens: write slots, pages and ring entries; state: block 0 also writes the ring's state, lens and starts.
__global__ void __launch_bounds__(kThreads) page_tables_kernel(const __grid_constant__ mk_page_tables_args a, bool tokens,
                                                              bool state) {
  extern __shared__ int sm[];
  const int B = a.batch, P = a.page_size;
  int* tok0 = sm;                // [B] first token of each request
  int* take0 = sm + B;           // [B] first taken page
  int* back0 = sm + 2 * B;       // [B] first returned page
  int* have = sm + 3 * B;        // [B] pages the row holds before the call
  int* first = sm + 4 * B;       // [B] position of the first new token
  __shared__ Sums warp_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

  const int step = gridDim.x * kThreads, id = blockIdx.x * kThreads + tid;
  state = state && blockIdx.x == 0;
  if (why) {  // the same decision in every CTA
    for (unsigned t = id; tokens && t < static_cast<unsigned>(a.n_tokens); t += step) {  // (t + step passes 2^31)
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = 0;
      if (a.owners) a.owners[t] = -1;
    }
    __syncthreads();
    if (state) {
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
  if (tokens) {
    int flags = 0;
    for (unsigned t = id; t < static_cast<unsigned>(a.n_tokens); t += step) {
      long long slot = -1;
      int pos = 0, b = -1;
      if (t < static_cast<unsigned>(n_tok)) {
        b = owner_of(tok0, B, t);
        pos = first[b] + (static_cast<int>(t) - tok0[b]);
        const int k = pos / P, h = have[b];
        const int page = k < h ? a.table[b * a.table_stride + k]
                               : a.ring[(static_cast<unsigned>(head) + take0[b] + (k - h)) % size];
        if (page >= 0 && page < a.n_pages) slot = static_cast<long long>(page) * P + (pos - k * P);
        else flags |= MK_OP_BAD_PAGE;
      }
      a.slots[t] = slot;
      if (a.positions) a.positions[t] = pos;
      if (a.owners) a.owners[t] = b;
    }
    for (unsigned j = id; j < static_cast<unsigned>(n_take); j += step) {
      const int b = owner_of(take0, B, j);
      a.table[b * a.table_stride + have[b] + (static_cast<int>(j) - take0[b])] = a.ring[(head + j) % size];
    }
    for (unsigned j = id; j < static_cast<unsigned>(n_back); j += step) {
      const int b = owner_of(back0, B, j);
      // the row keeps as many pages as it held less those it returns
      const int gone = (b + 1 < B ? back0[b + 1] : n_back) - back0[b];
      a.ring[(static_cast<unsigned>(head) + n_free + j) % size] =
          a.table[b * a.table_stride + have[b] - gone + (static_cast<int>(j) - back0[b])];
    }
    if (flags) flag(a.status, flags);
  }
  __syncthreads();  // this CTA has read the lengths and the ring's state
  if (state) {
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

// Whether the n elements at p lie (partly) within the m at q.
bool overlap(const int32_t* p, int n, const int32_t* q, int m) { return p && p < q + m && q < p + n; }

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
  if (!aligned({a.table, a.held, a.start, a.count, a.ring, a.ring_state, a.ring_state_out, a.positions, a.owners, a.starts,
                a.lens, a.status}, 4) || !aligned(a.slots, 8))
    return refuse(MK_ERR_INVALID_ARG, me, "a misaligned pointer");
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
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(me, e);
  // One CTA up to 1024 places (two tokens a thread): a second CTA would gain less than the second launch in place costs.
  const int want = a.n_tokens <= 2 * kThreads ? 1 : a.n_tokens / kThreads + 1;
  const int ctas = want < 2 * sms ? want : 2 * sms;
  bool in_place = overlap(a.ring_state_out, 2, a.ring_state, 2);
  for (const int32_t* in : {a.held, a.start, a.count}) {
    in_place |= overlap(a.lens, a.batch, in, a.batch) || overlap(a.starts, a.batch + 1, in, a.batch) ||
                overlap(a.ring_state_out, 2, in, a.batch);
  }
  in_place |= overlap(a.lens, a.batch, a.ring_state, 2) || overlap(a.starts, a.batch + 1, a.ring_state, 2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool split = in_place && ctas > 1;
  cudaError_t e = start(page_tables_kernel, ctas, kThreads, smem, s, a, true, !split);
  if (e == cudaSuccess && split) e = start(page_tables_kernel, 1, kThreads, smem, s, a, false, true);
  return launched(me, e);
}
