// The attention kernel of mk_paged_attention for long calls over 16-bit caches 128 or 256 wide: the 5th-generation
// tensor cores with accumulators in tensor memory.
//
// Work, workspace and join are those of paged_attention.cuh's line of tiles; a tile is 128 keys and one CTA has an SM.
// With mma.sync every warp loads fragments, rescales and moves its sums itself: 4800 warp instructions for 64 keys
// of 48 rows, which bound it (IPC 1.3, 31 % of the tensor pipe; 107 us for 8 requests of 8192 positions and 8 rows of
// 48 / 8 heads x 128, against 67 us here; 64 requests of 1 to 8192 positions, one row: 209 and 177 us, 91 % of the measured
// copy rate). Here one thread issues the products of whole tiles
// from shared memory and the softmax has one thread per key:
//   scores  S [128 keys x R rows] = K Q^T         A = the tile's keys (K-major), B = the query rows
//   sums    O [128 of D x 2 R] += V^T [P hi, P lo]  A = the tile's values as they lie (M-major), B = the probabilities
// R = 8, 16, 32, 48 or 64 rows. Probabilities are 16-bit pairs hi + lo, side by side in one product (an instruction takes
// about 50 cycles whatever its width, so two narrow ones cost twice); the halves are added at the end (kLowScale).
// Roles: warps 0-7 softmax (a thread is a key of the scores and one of the D of the sums; warps 0-3 have the first half
// of the rows, 4-7 the second), warp 8 one thread that issues, warps 9-11 load keys and 12-14 values (cp.async, page by
// page) into a ring of 32 KB slots, 128 keys x 128 wide each. The scores of the next tile are computed while this one's
// probabilities are made (two score buffers).
// The running maximum is the same for all threads of a row and grows only when a score passes it by kGrow (in the
// exponent's units): then the sums are rescaled in tensor memory; else nothing is exchanged but two votes per tile.
// Code that runs once per request is kept short: it comes from memory every time (an unrolled end of a request took
// 11 us).
// Every wait has a limit (2 s), after which the CTA gives up, drains and frees what it holds and MK_OP_TIMEOUT is set.
#pragma once
#include "paged_attention.cuh"

namespace mkop {
namespace attn {

// ---- PTX ----------------------------------------------------------------------------------------------------------
__device__ inline void bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ inline void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ inline bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
  return ok != 0;
}
// Arrives when this thread's copies so far have landed. Their writes are ordinary ones: who hands them to the tensor
// cores waits on the barrier and then fences the proxies.
__device__ inline void cp_arrive(uint64_t* b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
// Waits for the phase of that parity; false after the time limit or when another thread of the CTA gave up.
__device__ inline bool bar_wait(uint64_t* b, uint32_t parity, volatile int* dead) {
  unsigned long long t0 = 0;
  for (uint32_t n = 1; !bar_try(b, parity); ++n) {
    if (n & 63) continue;
    if (*dead) return false;
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (!t0) t0 = t;
    else if (t - t0 > kWaitLimitNs) {
      *dead = 1;
      return false;
    }
  }
  return true;
}
// Barrier `id` of `n` threads; whether any of them says so.
__device__ inline bool any_of(int id, int n, bool mine) {
  uint32_t r;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\nbarrier.cta.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}"
               : "=r"(r) : "r"(id), "r"(n), "r"(static_cast<uint32_t>(mine)) : "memory");
  return r != 0;
}
__device__ inline void named_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ inline void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ inline void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ inline void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ inline void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
// N consecutive fp32 columns of this warp's 32 lanes. Load and wait are one statement: before the wait the registers do
// not hold the values.
__device__ inline void tc_ld(float (&v)[4], uint32_t addr) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3])
               : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tc_ld(float (&v)[8], uint32_t addr) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7])
               : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tc_ld(float (&v)[16], uint32_t addr) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
                 "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]),
                 "=&r"(r[15])
               : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tc_ld(float (&v)[24], uint32_t addr) {
  uint32_t r[24];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%24];\n"
               "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%25];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
                 "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]),
                 "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]),
                 "=&r"(r[22]), "=&r"(r[23])
               : "r"(addr), "r"(addr + 16) : "memory");
#pragma unroll
  for (int i = 0; i < 24; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tc_ld(float (&v)[32], uint32_t addr) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
               "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
                 "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]),
                 "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]),
                 "=&r"(r[22]), "=&r"(r[23]), "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]),
                 "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31])
               : "r"(addr), "r"(addr + 16) : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ inline void tc_st(uint32_t addr, const float (&v)[4]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};\n"
               "tcgen05.wait::st.sync.aligned;" ::
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(addr) : "memory");
}
__device__ inline void tc_st(uint32_t addr, const float (&v)[8]) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n"
               "tcgen05.wait::st.sync.aligned;" ::
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr) : "memory");
}
__device__ inline void tc_st(uint32_t addr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n"
               "tcgen05.wait::st.sync.aligned;" ::
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                   "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}
__device__ inline void tc_st(uint32_t addr, const float (&v)[24]) {
  uint32_t r[24];
#pragma unroll
  for (int i = 0; i < 24; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%24], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n"
               "tcgen05.st.sync.aligned.32x32b.x8.b32 [%25], {%16,%17,%18,%19,%20,%21,%22,%23};\n"
               "tcgen05.wait::st.sync.aligned;" ::
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                   "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                   "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(addr),
                   "r"(addr + 16) : "memory");
}
__device__ inline void tc_st(uint32_t addr, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n"
               "tcgen05.st.sync.aligned.32x32b.x16.b32 [%33], {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n"
               "tcgen05.wait::st.sync.aligned;" ::
                   "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                   "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                   "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                   "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr),
                   "r"(addr + 16) : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle: 8-row groups (of 128-byte rows) 1024 bytes apart; `lead` bytes
// between 64-element pieces of an M- or N-major operand's rows (not used by a K-major one).
__device__ inline uint64_t tc_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: fp32 sums, 16-bit operands, M = 128; `major`: both operands M- / N-major
template <typename T>
__device__ constexpr uint32_t tc_idesc(int n, bool major) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (major ? 3u << 15 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}
// the largest of a warp's values; NaN counts as -infinity
__device__ inline float warp_largest(float x) {
  int i = __float_as_int(x == x ? x : -INFINITY);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(~0u, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// ---- shape ----------------------------------------------------------------------------------------------------------
// R: query rows of a block that the softmax works on (8, 16, 32, 48 or 64); products have N >= 16.
template <int D, int R>
struct TcShape {
  static constexpr int N = R < 16 ? 16 : R;   // columns of the scores
  static constexpr int kPairs = 2 * R;        // columns of the sums
  static constexpr int kTmem = 128 + 128 * (D / 128) <= 256 ? 256 : 512;  // two score buffers, then the sums
  static constexpr int kTile = 128, kThreads = 480, kSoftmax = 256, kLoaders = 96;
  static constexpr int kHalves = D / 128;              // 128-wide pieces of a key or a value
  static constexpr int kSlot = 128 * 128 * 2, kP = 128 * 128, kQ = N * D * 2;
  static constexpr int kStats = 16 * 64 * 4 + 16 * 64 * 4 + 2 * 2 * 128 * 8 + 512;
  static constexpr int kLimit = 227 * 1024 - 1024;     // less what aligning to 1024 bytes may take
  static constexpr int kQs = 4 * kSlot + 2 * kP + 2 * kQ + kStats <= kLimit ? 2 : 1;
  static constexpr int kSlots = 5 * kSlot + 2 * kP + kQs * kQ + kStats <= kLimit ? 5 : 4;
  // probabilities [2][128 keys][64 columns], column c of the 2 R in piece c / 64; scratch at the end of a request
  static constexpr int kOffP = kSlots * kSlot;
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffTail = kOffQ + kQs * kQ;    // float [16][64]: scores of keys not all rows see
  static constexpr int kOffStat = kOffTail + 16 * 64 * 4;
  static constexpr int kOffAddr = kOffStat + 16 * 64 * 4;  // address [2][2][128]
  static constexpr int kOffBar = kOffAddr + 2 * 2 * 128 * 8;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};
constexpr float kNoBase = -3.402823466e38f;  // the lowest finite value: what a row's base begins with
// fp16 has few exponents, and many weak keys behind one strong key of a small value make the whole result. So fp16
// probabilities are taken against a base 7 under the maximum (up to 2^15 before the sums are rescaled) and the lower half
// of a pair is 2^11 times what is left: off by 2^-22, or by 2^-43 of the largest.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
template <typename T>
constexpr float kLowScale = std::is_same<T, __half>::value ? 2048.0f : 1.0f;
constexpr float kGrow = 8.0f;  // a score above the maximum by this (in the exponent's units) moves the base
constexpr int kTcMaxRows = 16;   // query rows of a request (of its block of new tokens)

struct TcBars {
  uint64_t full[5], empty[5], q_full[2], q_empty[2], s_full[2], s_empty[2], p_full, p_empty, drained;
  uint32_t tmem;
  int dead;
};

// A role's place in the CTA's tiles.
struct Walk {
  const mk_paged_attention_args& a;
  const Params& p;
  int b, head, block, tile, n, len, next_len, first_tile;
  int done, count, items;
  __device__ int length(int i) const { return min(max(a.lens[i], 0), p.max_len); }
  __device__ static int tiles_of(int len) { return max(1, (len + 127) >> 7); }
  __device__ Walk(const Params& pp, int b0, long long rem, int cnt) : a(pp.a), p(pp) {
    b = b0;
    len = length(b);
    n = tiles_of(len);
    const int hm = static_cast<int>(rem / n);
    tile = static_cast<int>(rem - static_cast<long long>(hm) * n);
    head = hm / p.blocks;
    block = hm - head * p.blocks;
    next_len = b + 1 < a.batch ? length(b + 1) : 0;
    first_tile = tile;
    done = 0, count = cnt, items = 0;
  }
  __device__ bool first() const { return done == 0 || tile == 0; }
  __device__ bool last() const { return done == count - 1 || tile == n - 1; }
  __device__ void next() {
    if (last()) ++items;
    ++done;
    if (++tile == n) {
      tile = 0;
      if (++block == p.blocks) {
        block = 0;
        if (++head == a.n_kv_heads) {
          head = 0;
          ++b;
          len = next_len;
          n = tiles_of(len);
          next_len = b + 1 < a.batch ? length(b + 1) : 0;
        }
      }
      first_tile = 0;
    }
  }
  __device__ int all_see() const { return len - (a.rows - 1); }  // keys before it are seen by every row
};

template <typename T, int D, int R>
__global__ void __launch_bounds__(TcShape<D, R>::kThreads, 1) tc_kernel(const __grid_constant__ Params p) {
  using S = TcShape<D, R>;
  constexpr int N = S::N;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t s0 = smem_u32(smem);
  const mk_paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  TcBars& bars = *reinterpret_cast<TcBars*>(smem + S::kOffBar);
  volatile int* dead = &bars.dead;
  __shared__ long long warp_tiles[S::kThreads / 32];
  __shared__ long long at_rem;
  __shared__ int at_b;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's piece of the line (as in attention_kernel) --------------------------------------------------------
  const int hm_n = a.n_kv_heads * p.blocks;
  long long total;
  int count;
  {
    auto length = [&](int b) { return min(max(a.lens[b], 0), p.max_len); };
    const int per = (a.batch + S::kThreads - 1) / S::kThreads;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      if (blockIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > p.max_len)) flag(a.status, MK_OP_BAD_LENGTH);
      mine += Walk::tiles_of(length(b));
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    total = 0;
    for (int w = 0; w < S::kThreads / 32; ++w) {
      if (w < warp) before += warp_tiles[w];
      total += warp_tiles[w];
    }
    total *= hm_n;
    const long long worth = (total + kMinTiles - 1) / kMinTiles;
    const int used = worth < p.ctas ? static_cast<int>(worth) : p.ctas;
    const long long begin = piece_begin(blockIdx.x, total, used);
    if (static_cast<int>(blockIdx.x) < used && before * hm_n <= begin && begin < (before + mine) * hm_n) {
      for (int b = b0; b < b1; ++b) {
        const int n = Walk::tiles_of(length(b));
        if (begin < (before + n) * hm_n) {
          at_b = b;
          at_rem = begin - before * hm_n;
          break;
        }
        before += n;
      }
    }
    if (tid == 0) {
      for (int i = 0; i < 5; ++i) bar_init(&bars.full[i], S::kLoaders), bar_init(&bars.empty[i], 1);
      for (int i = 0; i < 2; ++i) {
        bar_init(&bars.q_full[i], S::kLoaders), bar_init(&bars.q_empty[i], 1);
        bar_init(&bars.s_full[i], 1), bar_init(&bars.s_empty[i], S::kSoftmax);
      }
      bar_init(&bars.p_full, S::kSoftmax), bar_init(&bars.p_empty, 1), bar_init(&bars.drained, 1);
      bars.dead = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (static_cast<int>(blockIdx.x) >= used) {
      if (tid == 0) p.piece[blockIdx.x].used = used;
      return;
    }
    count = static_cast<int>(piece_begin(blockIdx.x + 1, total, used) - begin);
    if (tid == 0) {
      const Walk w(p, at_b, at_rem, count);
      Piece& pc = p.piece[blockIdx.x];
      pc.total = total;
      pc.item0 = begin - w.tile;
      pc.item1 = pc.item0 + w.n;
      pc.used = used;
      pc.b = w.b;
      pc.hm = w.head * p.blocks + w.block;
    }
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)), "r"(S::kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = bars.tmem;
  auto scores_at = [&](int j) { return tmem + static_cast<uint32_t>(j & 1) * 64; };
  auto sums_at = [&](int h) { return tmem + 128 + h * 128; };
  Walk w(p, at_b, at_rem, count);

  if (warp >= 9) {
    // ---- loaders --------------------------------------------------------------------------------------------------
    const bool value = warp >= 12;  // warps 9-11 load keys (and query rows), 12-14 values
    const int t = tid - (value ? 384 : 288), barrier = value ? 3 : 2;
    const unsigned char** addr = reinterpret_cast<const unsigned char**>(smem + S::kOffAddr) + (value ? 256 : 0);  // [2 tiles][128]
    // The pages of this thread's keys (t, and t + 96 where that is one of the tile's) are loaded a tile before their
    // addresses are made, and these a tile before the copies.
    auto look_up = [&](int key) -> int {
      key += w.tile * 128;
      return w.done < count && key < w.len ? a.table[w.b * a.table_stride + p.page(key)] : -1;
    };
    auto make_address = [&](const unsigned char** at, int page, int i) {  // of tile w's key i
      const unsigned char* from = kZeros;
      const int key = w.tile * 128 + i;
      if (w.done < count && key < w.len) {
        if (page < 0 || page >= a.n_pages)
          flag(a.status, MK_OP_BAD_PAGE);
        else if (!value || a.rows == 1 || key < w.all_see())
          // (values that not all rows see are left out of the product: see the softmax's end of a part)
          from = value ? row_at(a.v_pages, p.v_step, page, w.head, key - p.page(key) * a.page_size)
                       : row_at(a.k_pages, p.k_step, page, w.head, key - p.page(key) * a.page_size);
      }
      at[i] = from;
    };
    const bool two = t < 128 - S::kLoaders;
    struct Item {  // what the copies of a tile need besides addresses
      int b, head, block, items;
      bool first;
    };
    auto item_of = [&]() -> Item { return {w.b, w.head, w.block, w.items, w.first()}; };
    bool ok = true;
    auto wait_free = [&](uint64_t* bar, uint32_t parity) { ok = bar_wait(bar, parity, dead) && ok; };
    make_address(addr, look_up(t), t);
    if (two) make_address(addr, look_up(t + S::kLoaders), t + S::kLoaders);
    Item now = item_of();
    w.next();
    int page = look_up(t), page2 = two ? look_up(t + S::kLoaders) : -1;  // of tile w, one ahead of `now`
    for (int j = 0; j < count; ++j) {
      const unsigned char** at = addr + (j & 1) * 128;
      if (any_of(barrier, S::kLoaders, !ok)) break;
      if (!value && now.first) {
        const int q = now.items % S::kQs;
        const int turn = now.items / S::kQs;
        if (turn) wait_free(&bars.q_empty[q], (turn - 1) & 1);
        const uint32_t to = s0 + S::kOffQ + q * S::kQ;
        const unsigned char* from = static_cast<const unsigned char*>(a.q);
        for (int i = t; i < N * (D / 8); i += S::kLoaders) {
          const int row = i / (D / 8), chunk = i % (D / 8), mrow = now.block * R + row;
          const bool in = row < R && mrow < p.n_rows;
          const int r = p.group_div(mrow), h = now.head * p.group + mrow - r * p.group;
          const long long off = in ? now.b * a.q_stride[0] + r * a.q_stride[1] + h * a.q_stride[2] + chunk * 8 : 0;
          cp16(to + (chunk / 8) * (N * 128) + row * 128 + (((chunk % 8) ^ (row & 7)) << 4), from + off * 2, in);
        }
        cp_arrive(&bars.q_full[q]);
      }
#pragma unroll 1
      for (int h = 0; h < S::kHalves; ++h) {
        const uint32_t group = (static_cast<uint32_t>(j) * 2 + (value ? 1 : 0)) * S::kHalves + h;
        const int slot = group % S::kSlots, turn = group / S::kSlots;
        if (turn) wait_free(&bars.empty[slot], (turn - 1) & 1);
        const int chunk = t & 15, row0 = t >> 4;
        const uint32_t to = s0 + slot * S::kSlot + (chunk >> 3) * 16384;
        const unsigned char* const* from = at + row0;
        const int column = h * 256 + chunk * 16;
#pragma unroll
        for (int i = 0; i < (128 * 16 + S::kLoaders - 1) / S::kLoaders; ++i) {
          const int row = row0 + S::kLoaders / 16 * i;
          if (row >= 128) break;
          cp16(to + row * 128 + (((chunk ^ row) & 7) << 4), from[S::kLoaders / 16 * i] + column);
        }
        cp_arrive(&bars.full[slot]);
        if (h == 0) {  // the next tile's addresses, while copies are in flight
          make_address(addr + (~j & 1) * 128, page, t);
          if (two) make_address(addr + (~j & 1) * 128, page2, t + S::kLoaders);
          now = item_of();
          w.next();
          page = look_up(t);
          if (two) page2 = look_up(t + S::kLoaders);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 8) {
    // ---- the thread that issues the products -------------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t kScores = tc_idesc<T>(N, false), kSums = tc_idesc<T>(S::kPairs, true);
      bool ok = true;
      auto scores = [&](int j) {
        const int q = w.items % S::kQs;
        if (w.first()) ok = ok && bar_wait(&bars.q_full[q], (w.items / S::kQs) & 1, dead);
        if (j >= 2) ok = ok && bar_wait(&bars.s_empty[j & 1], static_cast<uint32_t>((j >> 1) - 1) & 1, dead);
        const uint32_t qa = s0 + S::kOffQ + q * S::kQ;
        for (int h = 0; h < S::kHalves && ok; ++h) {
          const uint32_t g = static_cast<uint32_t>(j) * 2 * S::kHalves + h, slot = g % S::kSlots;
          ok = bar_wait(&bars.full[slot], (g / S::kSlots) & 1, dead);
          if (!ok) break;
          proxy_fence();
          tc_after();
          // a step along a descriptor's address is 1 / 16 of the bytes
          const uint64_t kd = tc_desc(s0 + slot * S::kSlot, 16), qd = tc_desc(qa + 2 * h * (N * 128), 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma(scores_at(j), kd + ((k >> 2) * 16384 + (k & 3) * 32) / 16, qd + ((k >> 2) * (N * 128) + (k & 3) * 32) / 16,
                   kScores, h > 0 || k > 0);
          tc_commit(&bars.empty[slot]);
        }
        if (!ok) return;
        if (w.last()) tc_commit(&bars.q_empty[q]);
        tc_commit(&bars.s_full[j & 1]);
      };
      scores(0);
      for (int j = 0; j < count && ok; ++j) {
        const bool fresh = w.first();
        w.next();
        if (j + 1 < count) scores(j + 1);
        if (!ok || !(ok = bar_wait(&bars.p_full, j & 1, dead))) break;
        for (int h = 0; h < S::kHalves; ++h) {
          const uint32_t g = static_cast<uint32_t>(j) * 2 * S::kHalves + S::kHalves + h, slot = g % S::kSlots;
          ok = bar_wait(&bars.full[slot], (g / S::kSlots) & 1, dead);
          if (!ok) break;
          proxy_fence();
          tc_after();
          const uint64_t vd = tc_desc(s0 + slot * S::kSlot, 16384), pd = tc_desc(s0 + S::kOffP, 16384);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma(sums_at(h), vd + k * 2048 / 16, pd + k * 2048 / 16, kSums, !fresh || k > 0);
          tc_commit(&bars.empty[slot]);
        }
        if (ok) tc_commit(&bars.p_empty);
      }
      // every product has ended before the tensor memory is freed, also when the CTA gave up
      tc_commit(&bars.drained);
      int alive = 0;
      bar_wait(&bars.drained, 0, &alive);
    }
    __syncwarp();
  } else {
    // ---- softmax --------------------------------------------------------------------------------------------------
    constexpr int RH = R / 2;                       // rows of this thread: r0 .. r0 + RH - 1
    const int part = warp >> 2, r0 = part * RH, t = tid & 127, wq = warp & 3;
    float* tail = reinterpret_cast<float*>(smem + S::kOffTail);
    float* stat = reinterpret_cast<float*>(smem + S::kOffStat);
    float *warp_max = stat, *base_of = stat + 256, *shrink = stat + 320, *sum_of = stat + 384;
    int* back = reinterpret_cast<int*>(stat + 448);  // keys at the end that a row does not see
    unsigned char** out_of = reinterpret_cast<unsigned char**>(stat + 512);        // [64]: where a row's result begins
    const T** late_at = reinterpret_cast<const T**>(stat + 640);                   // [16]: values not all rows see
    float* scratch = reinterpret_cast<float*>(smem + S::kOffP);                    // 32 KB, free at a request's end
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;  // this warp's 32 of the tensor memory's lanes
    float l[RH];
    bool ok = true;
    int first_tile = 0;
    for (int j = 0; j < count; ++j) {
      const bool first = w.first(), last = w.last();
      const int rows = min(R, p.n_rows - w.block * R), all_see = w.all_see();
      if (first) {
        first_tile = w.tile;
#pragma unroll
        for (int r = 0; r < RH; ++r) l[r] = 0;
        if (tid < R) back[tid] = a.rows - 1 - p.group_div(min(w.block * R + tid, p.n_rows - 1));
      }
      ok = bar_wait(&bars.s_full[j & 1], static_cast<uint32_t>(j >> 1) & 1, dead) && ok;
      if (any_of(1, S::kSoftmax, !ok)) break;
      tc_after();
      float s[RH];
      tc_ld(s, scores_at(j) + lanes + r0);
      tc_before();
      bar_arrive(&bars.s_empty[j & 1]);
#pragma unroll
      for (int r = 0; r < RH; ++r) s[r] *= p.scale_log2;
      const int key = w.tile * 128 + t;
      if (w.tile * 128 + 128 > all_see) {
        const bool late = a.rows > 1 && key >= all_see && key < w.len;
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          if (key >= w.len - back[r0 + r]) s[r] = -INFINITY;
          if (late) tail[(key - all_see) * 64 + r0 + r] = s[r];
        }
      }
      // The base is subtracted once it is known to stay: added back it would not give the score again (base kNoBase).
      float big = -INFINITY;
      if (!first) {
#pragma unroll
        for (int r = 0; r < RH; r += 4) {
          const float4 base = *reinterpret_cast<const float4*>(base_of + r0 + r);
          big = fmaxf(big, fmaxf(fmaxf(s[r] - base.x, s[r + 1] - base.y), fmaxf(s[r + 2] - base.z, s[r + 3] - base.w)));
        }
      }
      bool waited = false;
      if (any_of(1, S::kSoftmax, first || big > kLift<T> + kGrow)) {
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          const float x = warp_largest(s[r]);
          if (lane == 0) warp_max[wq * 64 + r0 + r] = x;
        }
        named_sync(1, S::kSoftmax);
        if (tid < R) {
          const float old = first ? kNoBase : base_of[tid];
          const float top = fmaxf(fmaxf(warp_max[tid], warp_max[64 + tid]), fmaxf(warp_max[128 + tid], warp_max[192 + tid]));
          const float base = fmaxf(kLift<T> ? __fadd_ru(top, -kLift<T>) : top, old);  // upwards: the lift is no more than that
          base_of[tid] = base;
          shrink[tid] = exp2_fast(old - base);
        }
        named_sync(1, S::kSoftmax);
        if (!first) {
          ok = bar_wait(&bars.p_empty, static_cast<uint32_t>(j - 1) & 1, dead) && ok;  // the last tile's sums are complete
          waited = true;
          tc_after();
#pragma unroll
          for (int r = 0; r < RH; ++r) l[r] *= shrink[r0 + r];
#pragma unroll 1
          for (int c = 0; c < 2 * S::kHalves; ++c) {  // hi and lo of each piece of D
            const uint32_t at = sums_at(c >> 1) + lanes + (c & 1) * R + r0;
            float v[RH];
            tc_ld(v, at);
#pragma unroll
            for (int r = 0; r < RH; ++r) v[r] *= shrink[r0 + r];
            tc_st(at, v);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RH; r += 4) {
        const float4 base = *reinterpret_cast<const float4*>(base_of + r0 + r);
        s[r] -= base.x, s[r + 1] -= base.y, s[r + 2] -= base.z, s[r + 3] -= base.w;
      }
      if (j > 0 && !waited) ok = bar_wait(&bars.p_empty, static_cast<uint32_t>(j - 1) & 1, dead) && ok;  // the buffer is free
      unsigned char* to = smem + S::kOffP + t * 128;
      auto column = [&](int c) {  // of a row of probabilities: 16-byte piece c / 8, its place swizzled by the key
        return to + (c >> 6) * S::kP + ((((c >> 3) & 7) ^ (t & 7)) << 4) + (c & 7) * 2;
      };
      constexpr int kAtOnce = RH % 8 ? 4 : 8;  // rows of one store
#pragma unroll
      for (int c = 0; c < RH; c += kAtOnce) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < kAtOnce / 2; ++i) {
          const int r = c + 2 * i;
          const float x = exp2_fast(s[r]), y = exp2_fast(s[r + 1]);
          l[r] += x, l[r + 1] += y;
          hi[i] = pack2<T>(x, y);
          const float2 u = unpack2<T>(hi[i]);
          lo[i] = pack2<T>((x - u.x) * kLowScale<T>, (y - u.y) * kLowScale<T>);
        }
        if (kAtOnce == 8) {
          *reinterpret_cast<uint4*>(column(r0 + c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(column(R + r0 + c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          *reinterpret_cast<uint2*>(column(r0 + c)) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(column(R + r0 + c)) = make_uint2(lo[0], lo[1]);
        }
      }
      proxy_fence();
      tc_before();
      bar_arrive(&bars.p_full);

      if (last) {  // the end of this CTA's part of the request
        const bool whole = first_tile == 0 && w.tile == w.n - 1;
        const long long slot = 2ll * blockIdx.x + (j == w.tile - first_tile ? 0 : 1);
        // This part's keys that not all rows see: their probabilities into the place of their scores (-1: hidden from the
        // row, whose sum its value must not touch even times 0), and where their values are.
        const int late0 = a.rows > 1 ? max(max(all_see, 0), first_tile * 128) : 0;
        const int late_n = a.rows > 1 ? max(min(w.len, w.tile * 128 + 128) - late0, 0) : 0;
        float* late = tail + (late0 - all_see) * 64;
        named_sync(1, S::kSoftmax);  // the scores of these keys are written
#pragma unroll 1
        for (int i = tid; i < late_n * 64; i += S::kSoftmax) {
          const int r = i & 63;
          if (r < R) late[i] = late0 + (i >> 6) < w.len - back[r] ? exp2_fast(late[i] - base_of[r]) : -1.0f;
        }
        if (tid < late_n) {
          const int page = a.table[w.b * a.table_stride + p.page(late0 + tid)];
          late_at[tid] = page < 0 || page >= a.n_pages
                             ? nullptr
                             : static_cast<const T*>(a.v_pages) + page * a.v_page_stride[0] + w.head * a.v_page_stride[1] +
                                   (late0 + tid - p.page(late0 + tid) * a.page_size) * a.v_page_stride[2];
        }
        ok = bar_wait(&bars.p_empty, static_cast<uint32_t>(j) & 1, dead) && ok;  // the sums are complete, the scratch is free
#pragma unroll
        for (int r = 0; r < RH; ++r) scratch[(r0 + r) * 128 + t] = l[r];
        named_sync(1, S::kSoftmax);
        tc_after();
#pragma unroll 1
        for (int r = warp; r < R; r += 8) {  // a row's sum of exponentials
          const float4 v = *reinterpret_cast<const float4*>(scratch + r * 128 + lane * 4);
          float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
          for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
          if (lane == 0 && r < rows) {
            const int mrow = w.block * R + r, q = p.group_div(mrow), h = w.head * p.group + mrow - q * p.group;
            if (whole) {
              out_of[r] = reinterpret_cast<unsigned char*>(static_cast<T*>(a.out) + w.b * a.out_stride[0] + q * a.out_stride[1] + h * a.out_stride[2]);
              sum_of[r] = sum == 0.0f ? 0.0f : 1.0f / sum;
              if (a.lse)
                a.lse[(static_cast<long long>(w.b) * a.rows + q) * a.n_q_heads + h] =
                    sum == 0.0f ? -INFINITY : (base_of[r] + log2f(sum)) * 0.693147180559945309f;
            } else {
              out_of[r] = reinterpret_cast<unsigned char*>(p.part + (slot * R + r) * D);
              p.part_ml[slot * R + r] = make_float2(sum == 0.0f ? -INFINITY : base_of[r], sum);
            }
          }
        }
        named_sync(1, S::kSoftmax);
#pragma unroll 1
        for (int h = 0; h < S::kHalves; ++h) {
          float v[RH], u[RH];
          tc_ld(v, sums_at(h) + lanes + r0);
          tc_ld(u, sums_at(h) + lanes + R + r0);
#pragma unroll
          for (int r = 0; r < RH; ++r) v[r] += u[r] * (1.0f / kLowScale<T>);
#pragma unroll 2
          for (int x = 0; x < late_n; ++x) {
            const float value = late_at[x] ? static_cast<float>(late_at[x][h * 128 + t]) : 0.0f;
#pragma unroll
            for (int r = 0; r < RH; r += 4) {
              const float4 f = *reinterpret_cast<const float4*>(late + x * 64 + r0 + r);
              if (!(f.x < 0.0f)) v[r] += f.x * value;
              if (!(f.y < 0.0f)) v[r + 1] += f.y * value;
              if (!(f.z < 0.0f)) v[r + 2] += f.z * value;
              if (!(f.w < 0.0f)) v[r + 3] += f.w * value;
            }
          }
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            if (r0 + r >= rows) break;
            if (whole) reinterpret_cast<T*>(out_of[r0 + r])[h * 128 + t] = static_cast<T>(v[r] * sum_of[r0 + r]);
            else reinterpret_cast<float*>(out_of[r0 + r])[h * 128 + t] = v[r];
          }
        }
        tc_before();                 // the next part's first product comes after its first p_full
        named_sync(1, S::kSoftmax);  // every thread is done with what the next part writes
      }
      w.next();
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem) : "memory");
  if (tid == 0 && *dead) flag(a.status, MK_OP_TIMEOUT);
}

template <typename T, int D, int R>
struct TcMake {
  using S = TcShape<D, R>;
  static constexpr auto kKernel = tc_kernel<T, D, R>;
  static cudaError_t occupancy(int device, int* n) {
    *n = 1;  // more than half of an SM's shared memory
    return allow_smem<kKernel>(device, S::kSmem);
  }
  static cudaError_t launch(const Params& p, cudaStream_t s) {
    return start(kKernel, p.ctas, S::kThreads, S::kSmem, s, p);
  }
  static constexpr Build build() { return {R, S::kTile, occupancy, nullptr, launch}; }
};

// rows: of a block, at most 64
template <typename T>
inline const Build* pick_tc(int d, int rows) {
  static constexpr Build all[2][5] = {{TcMake<T, 128, 8>::build(), TcMake<T, 128, 16>::build(), TcMake<T, 128, 32>::build(),
                                       TcMake<T, 128, 48>::build(), TcMake<T, 128, 64>::build()},
                                      {TcMake<T, 256, 8>::build(), TcMake<T, 256, 16>::build(), TcMake<T, 256, 32>::build(),
                                       TcMake<T, 256, 48>::build(), TcMake<T, 256, 64>::build()}};
  return &all[d == 256][rows <= 8 ? 0 : (rows + 15) / 16];
}

const Build* pick_tc_bf16(int d, int rows);
const Build* pick_tc_f16(int d, int rows);

}  // namespace attn
}  // namespace mkop
