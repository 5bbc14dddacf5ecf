// The attention kernel of mk_paged_attention for small calls, e4m3 caches and every width (paged_attention_tc.cuh has the
// one for long calls over 16-bit caches 128 and 256 wide, paged_attention.cu the entry point and the join).
//
// What it computes: for each request b and kv head, the rows (query row r, query head of the group) against the keys
// of the request's pages: an online softmax in log2 units, one pass over keys and values.
//
// What bounds it: each cached byte is read once and meets rows x group query rows, 2 x rows x group flops a byte at 16
// bits (6 to 96 for the models here) where the tensor cores' bound begins at 284. So the design keeps bytes in flight:
// - Work: a tile is kTile keys of one (request, kv head, block of 16 MT rows). Small calls: a cluster of up to 16 CTAs
//   shares the tiles of one and joins through distributed shared memory, or one CTA has it alone. Else all tiles of the
//   call, request after request, are one line that is cut into equal pieces, one per resident CTA. A piece may begin and
//   end inside a request; ragged lengths balance by themselves and nothing depends on the host knowing the lengths. A
//   part of a request that a CTA did not cover alone goes to the workspace (at most two per CTA: its first and its last)
//   and is joined by the second kernel.
// - Loads: cp.async in a ring of kStages tiles that runs on across requests, so the next request's keys (and its query
//   rows, in a ring of their own) are in flight while the current one is finished. Page ids are looked up one tile
//   further ahead; a key's address is made once, by one thread. Two stages and more CTAs on an SM measured faster
//   than three (48 rows x 128: 107 against 129 us), keys times values of 128 keys faster than 64 for e4m3 (248, 266).
// - Products: mma.sync m16n8k16, a warp to 16 query rows x (kTile / WK) keys: scores, probabilities and sums stay in
//   its registers (the score accumulators are the probability operand), so a tile needs one barrier. The WK warps that
//   share rows are joined in shared memory when a request ends.
// - 16-bit caches: probabilities enter the product as a pair hi + lo of 16-bit values (16 mantissa bits): rounded to one they
//   would cost as much accuracy as the final rounding; the second product costs 5 % of the time. e4m3 caches: keys and
//   values become fp16 (exact) and the queries fp16 scaled per row by a power of two (bf16 mantissas fit; what falls under
//   2^-24 of a row's largest is rounded); probabilities are one fp16 (2^-11), an eighth of a bf16 result's rounding, for bf16
//   queries, and a pair for fp16 ones (64 requests of 1 to 16384 positions 246 us, with one 235, while an fp16 result then is as far
//   off again as its own rounding; 8 requests x 8 rows of 8192 85, 76).
//   fp16 has few exponents, and many weak keys behind one strong key of a small value make the whole result: so fp16
//   probabilities are taken against a base 15 under the running maximum (2^15 at it): off by 2^-11 (a pair: 2^-22) or by 2^-40
//   of the largest. The sums are against the same base, which is what parts are joined by.
// What bounds it now: warps x instructions in flight (IPC 1.8 of 4 at 8 warps on an SM); 64 requests of 1 to 16384
// positions, 48 / 8 heads x 128, e4m3: 229 us, 70 % of the measured copy rate.
#pragma once
#include <type_traits>

#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace mkop {
namespace attn {

namespace cg = cooperative_groups;

constexpr int kMaxCtas = 2048;   // pieces a call is cut into at most
constexpr int kMinTiles = 2;     // tiles of a piece at least: less is not worth joining

struct Params {
  mk_paged_attention_args a;
  Div page, group_div;
  int group;        // query heads per kv head
  int n_rows;       // query rows of a (request, kv head): rows * group
  int blocks;       // blocks of 16 MT rows
  int max_len;      // max_pages * page_size
  int ctas;         // grid of the attention kernel
  int parts;        // > 0: clusters of `parts` CTAs share a (request, kv head, row block); 0: pieces of the line
  float scale_log2; // scale * log2(e)
  uint32_t k_step[3], v_step[3];  // the caches' strides (page, head, place) in units of 16 bytes
  float* part;      // [2 ctas][16 MT][DP] sums of a part
  float2* part_ml;  // [2 ctas][16 MT] its maximum (log2 units) and sum
  struct Piece* piece;  // [ctas]
};

// Where a CTA's piece of the line of tiles begins (written by every CTA for the join).
struct Piece {
  long long total;         // tiles in all
  long long item0, item1;  // the line's range of the (request, kv head, row block) the piece begins in
  int used;                // CTAs that have a piece
  int b, hm;               // request, kv head * blocks + block
  int pad;
};

__host__ __device__ inline long long piece_begin(long long c, long long total, int used) { return c * total / used; }

// Rows that are not there (behind a request's length, of a page that does not exist, columns that pad a head) are copied
// from here: an address instead of a size that every copy would have to select.
static __device__ __align__(16) const unsigned char kZeros[512] = {};

// Where key or value `place` of a page and head begins.
__device__ inline const unsigned char* row_at(const void* cache, const uint32_t (&step)[3], int page, int head, int place) {
  const uint64_t units = static_cast<uint64_t>(static_cast<uint32_t>(page)) * step[0] +
                         static_cast<uint64_t>(static_cast<uint32_t>(head)) * step[1] +
                         static_cast<uint64_t>(static_cast<uint32_t>(place)) * step[2];
  return static_cast<const unsigned char*>(cache) + units * 16;
}

// ---- PTX ----------------------------------------------------------------------------------------------------------
__device__ inline uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes, zeros when !valid (nothing is read then)
__device__ inline void cp16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ inline void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ inline void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ inline void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ inline void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ inline void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ inline void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ inline void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 codes as two fp16 pairs; exact
__device__ inline void e4m3_to_f16(uint32_t (&r)[2], uint32_t codes) {
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}"
      : "=r"(r[0]), "=r"(r[1]) : "r"(codes));
}
__device__ inline float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- the shape of one build -----------------------------------------------------------------------------------------
template <typename T, int DP, int MT, bool E4M3, bool LONG>
struct Shape {
  static constexpr int WM = MT, WK = MT == 1 ? 4 : 2, kWarps = WM * WK, kThreads = 32 * kWarps;
  static constexpr int kRows = 16 * MT;
  static constexpr int kElt = E4M3 ? 1 : 2;
  // fp16 probabilities are 2^15 at the largest score, so that what falls under fp16's range is 2^-40 of it, not 2^-25
  static constexpr float kLift = std::is_same<T, __half>::value ? 15.0f : 0.0f;
  static constexpr int kRowBytes = DP * kElt;         // of a key in shared memory
  static constexpr int kChunks = kRowBytes / 16;
  // 16 to 32 KB of keys and values a tile (64 KB at 256 wide and 16 rows, where four warps take 16 keys each)
  static constexpr int kTile = E4M3 ? (DP == 64 ? 128 : DP == 128 && MT == 1 ? 128 : 64) : (DP == 256 && MT > 1 ? 32 : DP == 64 && LONG ? 128 : 64);
  static constexpr int kWarpKeys = kTile / WK;
  static constexpr int kBlock = kWarpKeys < 32 ? kWarpKeys : 32;  // keys of one softmax step
  static constexpr int kStages = MT > 2 && (DP == 256 || E4M3) ? 3 : 2;
  static constexpr int kKeyBytes = kTile * kRowBytes;  // of a tile's keys (as many of values)
  static constexpr int kStageBytes = 2 * kKeyBytes;
  static constexpr int kQBytes = kRows * DP * 2;
  static constexpr int kRing = kStages + 1;            // tiles whose page offsets and descriptions are held
  // joining the WK warps: a tile's buffer holds kJoin columns of all their sums
  static constexpr int kJoin = kStageBytes >= WK * kRows * 64 * 4 ? 64 : 32;
  static constexpr int kOffKV = 0;
  static constexpr int kOffQ = kStages * kStageBytes;
  static constexpr int kOffAddr = kOffQ + kStages * kQBytes;           // address [kRing][2][kTile]
  static constexpr int kOffMeta = kOffAddr + kRing * 2 * kTile * 8;    // Tile [kRing]
  static constexpr int kOffMl = kOffMeta + kRing * 48;                 // float2 [WK][kRows]
  static constexpr int kSmem = kOffMl + WK * kRows * 8;
  static constexpr int kFit = 227 * 1024 / (kSmem + 1024) < 1 ? 1 : 227 * 1024 / (kSmem + 1024);
  // CTAs on an SM: what shared memory allows, with at least 168 registers a thread (128 at 64 wide)
  static constexpr int kRegFit = 65536 / (kThreads * (DP == 64 ? 128 : DP == 128 ? 168 : 255));
  static constexpr int kCtas = kFit < kRegFit ? kFit : kRegFit < 1 ? 1 : kRegFit;
  static_assert(kWarpKeys % 16 == 0, "a warp's keys are whole k16 steps");
  static_assert(kStageBytes >= WK * kRows * kJoin * 4, "the join fits a stage");
  static_assert(kStages * kStageBytes >= kRows * DP * 4 + WK * kRows * kJoin * 4, "the cluster's join fits the ring");
  static_assert(kTile <= kThreads, "one thread looks up one key's page");
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

struct Tile {
  int b, head, block, len; // request, kv head, row block, the request's length
  int key0;                // first key
  int first, last;         // of the CTA's part of this request
  int whole;               // the part is the whole request
  int slot;                // else: which of the CTA's two places in the workspace (0: the piece begins with it)
  int q;                   // place in the ring of query rows
  int pad[2];
};
static_assert(sizeof(Tile) == 48, "three 16-byte words");

template <int kChunks>
__device__ inline uint32_t place(int row, int chunk) {  // byte offset of a 16-byte piece, conflict-free for ldmatrix
  if (kChunks >= 8) return row * (kChunks * 16) + ((chunk ^ (row & 7)) << 4);
  return row * (kChunks * 16) + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// PAIRS: probabilities as hi + lo (over e4m3 caches with fp16 queries and not with bf16 ones)
template <typename T, int DP, int MT, bool E4M3, bool LONG, bool PAIRS>
__global__ void __launch_bounds__(Shape<T, DP, MT, E4M3, LONG>::kThreads, Shape<T, DP, MT, E4M3, LONG>::kCtas)
    attention_kernel(const __grid_constant__ Params p) {
  using S = Shape<T, DP, MT, E4M3, LONG>;
  using Out = std::conditional_t<E4M3 && !PAIRS, __nv_bfloat16, T>;  // of the queries and the results
  extern __shared__ __align__(128) unsigned char smem[];
  const mk_paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % S::WM, wk = warp / S::WM;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t s0 = smem_u32(smem);
  const unsigned char** addr = reinterpret_cast<const unsigned char**>(smem + S::kOffAddr);
  Tile* meta = reinterpret_cast<Tile*>(smem + S::kOffMeta);
  float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);
  __shared__ long long warp_tiles[S::kWarps];
  __shared__ long long at_rem;
  __shared__ int at_b;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's tiles -------------------------------------------------------------------------------------------
  const int hm_n = a.n_kv_heads * p.blocks;
  auto length = [&](int b) { return min(max(a.lens[b], 0), p.max_len); };
  auto tiles_of = [&](int len) { return max(1, (len + S::kTile - 1) / S::kTile); };  // an empty request has one to write its zeros
  // c_*: the load side's place in the line, the next tile to describe
  int c_b, c_hm, c_tile, c_len, c_n, c_next_len = 0;
  long long count;
  if (p.parts) {
    const int item = blockIdx.x / p.parts, rank = blockIdx.x - item * p.parts;
    c_b = item / hm_n;
    c_hm = item - c_b * hm_n;
    if (rank == 0 && c_hm == 0 && tid == 0 && (a.lens[c_b] < 0 || a.lens[c_b] > p.max_len)) flag(a.status, MK_OP_BAD_LENGTH);
    c_len = length(c_b);
    c_n = tiles_of(c_len);
    c_tile = static_cast<int>(static_cast<long long>(rank) * c_n / p.parts);
    count = static_cast<int>(static_cast<long long>(rank + 1) * c_n / p.parts) - c_tile;
  } else {
    const int per = (a.batch + S::kThreads - 1) / S::kThreads;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      if (blockIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > p.max_len)) flag(a.status, MK_OP_BAD_LENGTH);
      mine += tiles_of(length(b));
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < S::kWarps; ++w) {
      if (w < warp) before += warp_tiles[w];
      total += warp_tiles[w];
    }
    total *= hm_n;
    const long long worth = (total + kMinTiles - 1) / kMinTiles;
    const int used = worth < p.ctas ? static_cast<int>(worth) : p.ctas;
    const long long begin = piece_begin(blockIdx.x, total, used);
    if (static_cast<int>(blockIdx.x) < used && before * hm_n <= begin && begin < (before + mine) * hm_n) {
      for (int b = b0; b < b1; ++b) {
        const int n = tiles_of(length(b));
        if (begin < (before + n) * hm_n) {
          at_b = b;
          at_rem = begin - before * hm_n;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    if (static_cast<int>(blockIdx.x) >= used) {
      if (tid == 0) p.piece[blockIdx.x].used = used;
      return;
    }
    count = piece_begin(blockIdx.x + 1, total, used) - begin;
    c_b = at_b;
    c_len = length(c_b);
    c_n = tiles_of(c_len);
    c_hm = static_cast<int>(at_rem / c_n);
    c_tile = static_cast<int>(at_rem % c_n);
    c_next_len = c_b + 1 < a.batch ? length(c_b + 1) : 0;
    if (tid == 0) {
      Piece& pc = p.piece[blockIdx.x];
      pc.total = total;
      pc.item0 = begin - c_tile;
      pc.item1 = pc.item0 + c_n;
      pc.used = used;
      pc.b = c_b;
      pc.hm = c_hm;
    }
  }
  int c_head = c_hm / p.blocks, c_block = c_hm - c_head * p.blocks;
  int c_first_tile = c_tile, c_items = 0;
  long long c_done = 0;

  // A tile is described in two halves with a tile's products between them, so that the page id's load is not waited for.
  auto look_up = [&]() -> int {  // the page of this thread's key, -1: no key
    if (c_done >= count || tid >= S::kTile) return -1;
    const int key = c_tile * S::kTile + tid;
    if (key >= c_len) return -1;
    const int page = a.table[c_b * a.table_stride + p.page(key)];
    return page >= 0 && page < a.n_pages ? page : -2;
  };
  auto describe = [&](int page, int ring) {
    if (c_done >= count) return;
    if (tid < S::kTile) {
      const unsigned char *k = kZeros, *v = kZeros;
      if (page >= 0) {
        const int key = c_tile * S::kTile + tid, at = key - p.page(key) * a.page_size;
        k = row_at(a.k_pages, p.k_step, page, c_head, at);
        v = row_at(a.v_pages, p.v_step, page, c_head, at);
      } else if (page == -2) {
        flag(a.status, MK_OP_BAD_PAGE);
      }
      addr[(ring * 2) * S::kTile + tid] = k;
      addr[(ring * 2 + 1) * S::kTile + tid] = v;
    }
    const bool first = c_done == 0 || c_tile == 0;
    if (first) c_first_tile = c_tile;
    const bool last = c_done == count - 1 || c_tile == c_n - 1;
    if (tid == 0) {
      Tile& m = meta[ring];
      m.b = c_b, m.head = c_head, m.block = c_block, m.len = c_len, m.key0 = c_tile * S::kTile;
      m.first = first, m.last = last, m.whole = c_first_tile == 0 && c_tile == c_n - 1;
      m.slot = c_done == c_tile - c_first_tile ? 0 : 1;
      m.q = c_items % S::kStages;
    }
    if (last) ++c_items;
    ++c_done;
    if (++c_tile == c_n) {
      c_tile = 0;
      if (++c_block == p.blocks) {
        c_block = 0;
        if (++c_head == a.n_kv_heads) {
          c_head = 0;
          ++c_b;
          c_len = c_next_len;
          c_n = tiles_of(c_len);
          c_next_len = c_b + 1 < a.batch ? length(c_b + 1) : 0;
        }
      }
    }
  };
  // A loading thread has one 16-byte column and every kLoadRows-th key.
  constexpr int kLoaders = S::kThreads & (S::kThreads - 1) ? 128 : S::kThreads;
  constexpr int kLoadRows = kLoaders / S::kChunks;
  static_assert(S::kTile % kLoadRows == 0, "whole rounds");
  // The first tile of a piece may be all there is (a short request), so only its keys that the products read (whole 32) are
  // copied: 129 to 200 requests of a few keys 1.5 to 3.5 times faster. In the loop the second copy of the code costs 2 %.
  auto load = [&](auto begins, int stage, int ring) {
    const Tile m = meta[ring];
    const uint32_t kd = s0 + S::kOffKV + stage * S::kStageBytes, vd = kd + S::kKeyBytes;
    if (kLoaders == S::kThreads || tid < kLoaders) {
      const int chunk = tid % S::kChunks, row0 = tid / S::kChunks;
      const bool in = chunk * 16 < a.head_dim * S::kElt;
      const unsigned char* const* at = addr + (ring * 2) * S::kTile + row0;
      auto round = [&](int i) {
        const uint32_t to = place<S::kChunks>(row0 + i * kLoadRows, chunk);
        const unsigned char *k = at[i * kLoadRows], *v = at[S::kTile + i * kLoadRows];
        cp16(kd + to, in ? k + chunk * 16 : kZeros);
        cp16(vd + to, in ? v + chunk * 16 : kZeros);
      };
      const int rows = (m.len - m.key0 + 31) & ~31;
      if (!decltype(begins)::value || rows >= S::kTile) {
#pragma unroll 8
        for (int i = 0; i < S::kTile / kLoadRows; ++i) round(i);
      } else {
#pragma unroll 1
        for (int i = 0; i * kLoadRows < rows; ++i) round(i);
      }
    }
    if (m.first) {
      const uint32_t qd = s0 + S::kOffQ + m.q * S::kQBytes;
      const unsigned char* q = static_cast<const unsigned char*>(a.q);
      for (int i = tid; i < S::kRows * (DP / 8); i += S::kThreads) {
        const int row = i / (DP / 8), chunk = i % (DP / 8), mrow = m.block * S::kRows + row;
        const bool in = mrow < p.n_rows && chunk * 8 < a.head_dim;
        const int r = p.group_div(mrow), h = m.head * p.group + mrow - r * p.group;
        const long long off = in ? m.b * a.q_stride[0] + r * a.q_stride[1] + h * a.q_stride[2] + chunk * 8 : 0;
        cp16(qd + place<DP / 8>(row, chunk), q + off * 2, in);
      }
    }
  };

  // ---- pipeline start: tiles 0 .. kStages - 1 described, all but the last of them loading -----------------------------
#pragma unroll 1
  for (int i = 0; i < S::kStages; ++i) describe(look_up(), i);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) {
    if (i < count) load(std::bool_constant<!LONG>{}, i, i);
    cp_commit();
  }

  float o[DP / 8][4];
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0, 0};  // the base (largest score - kLift) and the sum against it
  uint32_t qf[DP / 16][4];
  float row_scale[2];
  int limit[2];
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0;

  // Joins the warps that share rows: their sums, kJoin columns at a time, through `buf` ([WK][kRows][kJoin]);
  // sink(row, first of 4 columns, sums, largest maximum, sum of exponentials) gets every row below `rows`.
  auto join_warps = [&](float* buf, int rows, auto&& sink) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l_run[h] += __shfl_xor_sync(~0u, l_run[h], 1);
      l_run[h] += __shfl_xor_sync(~0u, l_run[h], 2);
      if (t4 == 0) ml[wk * S::kRows + wm * 16 + g + 8 * h] = make_float2(m_run[h], l_run[h]);
    }
#pragma unroll
    for (int c = 0; c < DP / S::kJoin; ++c) {
      __syncthreads();  // what buf held (c = 0) or the last columns have been read by every warp
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = wm * 16 + g + 8 * h;
        float* to = buf + (wk * S::kRows + row) * S::kJoin;
        const int turn = (row & 3) * 8;  // spreads the rows over the banks
#pragma unroll
        for (int i = 0; i < S::kJoin / 16; ++i) {
          const int n = c * (S::kJoin / 8) + 2 * i;
          if (!E4M3) {
            *reinterpret_cast<float2*>(to + ((16 * i + 2 * t4) ^ turn)) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
            *reinterpret_cast<float2*>(to + ((16 * i + 8 + 2 * t4) ^ turn)) = make_float2(o[n + 1][2 * h], o[n + 1][2 * h + 1]);
          } else {
            *reinterpret_cast<float4*>(to + ((16 * i + 4 * t4) ^ turn)) =
                make_float4(o[n][2 * h], o[n + 1][2 * h], o[n][2 * h + 1], o[n + 1][2 * h + 1]);
          }
        }
      }
      __syncthreads();
      for (int i = tid; i < rows * (S::kJoin / 4); i += S::kThreads) {
        const int row = i / (S::kJoin / 4), col = (i % (S::kJoin / 4)) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < S::WK; ++w) top = fmaxf(top, ml[w * S::kRows + row].x);
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0;
        float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < S::WK; ++w) {
          const float2 s = ml[w * S::kRows + row];
          const float f = exp2_fast(s.x - base);
          const float4 x = *reinterpret_cast<const float4*>(buf + (w * S::kRows + row) * S::kJoin + (col ^ ((row & 3) * 8)));
          sum += f * s.y;
          y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
        }
        sink(row, c * S::kJoin + col, y, top, sum);
      }
    }
  };
  // 4 columns of a finished row
  auto finish = [&](int b, int head, int block, int row, int d, float4 y, float top, float sum) {
    if (d >= a.head_dim) return;
    const int mrow = block * S::kRows + row, r = p.group_div(mrow), h = head * p.group + mrow - r * p.group;
    const float f = sum == 0.0f ? 0.0f : (E4M3 ? a.v_scale[head] : 1.0f) / sum;
    const uint2 u = make_uint2(pack2<Out>(y.x * f, y.y * f), pack2<Out>(y.z * f, y.w * f));
    uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_stride[0] + r * a.out_stride[1] + h * a.out_stride[2] + d;
    *reinterpret_cast<uint2*>(out) = u;
    if (d == 0 && a.lse)
      a.lse[(static_cast<long long>(b) * a.rows + r) * a.n_q_heads + h] =
          sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
  };

  int stage = 0, ring = 0;
#pragma unroll 1
  for (long long j = 0; j < count; ++j) {
    cp_wait<S::kStages - 2>();
    __syncthreads();  // tile j is there for every warp; tile j - 1's buffer and description are free
    {
      const int ahead = S::kStages - 1;
      if (j + ahead < count) load(std::false_type{}, (stage + ahead) % S::kStages, (ring + ahead) % S::kRing);
      cp_commit();
    }
    const int next = look_up();
    const Tile m = meta[ring];
    if (m.first) {
      const uint32_t qd = s0 + S::kOffQ + m.q * S::kQBytes;
      if (!E4M3) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          ldsm4(qf[k], qd + place<DP / 8>(wm * 16 + (lane & 15), 2 * k + (lane >> 4)));
        row_scale[0] = row_scale[1] = p.scale_log2;
      } else {
        // Key fragments hold 4 neighbouring elements a lane (one byte each), so the k order within 16 is that of
        // the lanes' quadruples; the query fragments follow it.
        const float ks = p.scale_log2 * a.k_scale[m.head];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = wm * 16 + g + 8 * h;
          const unsigned char* q = smem + S::kOffQ + m.q * S::kQBytes;
          auto piece = [&](int k) {
            return *reinterpret_cast<const uint2*>(q + place<DP / 8>(row, 2 * k + (t4 >> 1)) + (t4 & 1) * 8);
          };
          float big = 0;
          for (int k = 0; k < DP / 16; ++k) {
            const uint2 u = piece(k);
            const float2 x = unpack2<Out>(u.x);
            const float2 y = unpack2<Out>(u.y);
            big = fmaxf(big, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
          }
          big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
          big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
          // 2^e with big / 2^e in [1, 2); 1 for a row of zeros or with an infinity
          const int e = big > 0 && big < INFINITY ? min(max(ilogbf(big), -120), 120) : 0;
          const float down = __uint_as_float((127 - e) << 23);
          row_scale[h] = ks * __uint_as_float((127 + e) << 23);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint2 u = piece(k);
            const float2 x = unpack2<Out>(u.x);
            const float2 y = unpack2<Out>(u.y);
            qf[k][h] = pack2<__half>(x.x * down, x.y * down);
            qf[k][2 + h] = pack2<__half>(y.x * down, y.y * down);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0;
      m_run[0] = m_run[1] = -INFINITY;
      l_run[0] = l_run[1] = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int mrow = m.block * S::kRows + wm * 16 + g + 8 * h;
        limit[h] = mrow < p.n_rows ? m.len - (a.rows - 1 - p.group_div(mrow)) : 0;
      }
    }

    // ---- products of tile j ------------------------------------------------------------------------------------------
    const uint32_t kd = s0 + S::kOffKV + stage * S::kStageBytes, vd = kd + S::kKeyBytes;
    const int all_see = m.len - (a.rows - 1);  // keys before it are seen by every row
#pragma unroll 1
    for (int kb = wk * S::kWarpKeys; kb < (wk + 1) * S::kWarpKeys; kb += S::kBlock) {
      const int key = m.key0 + kb;
      if (key >= m.len) break;
      float s[S::kBlock / 8][4];
#pragma unroll
      for (int n = 0; n < S::kBlock / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0;
      if (!E4M3) {
#pragma unroll
        for (int k = 0; k < DP / 32; ++k)
#pragma unroll
          for (int n = 0; n < S::kBlock / 8; ++n) {
            uint32_t f[4];
            ldsm4(f, kd + place<S::kChunks>(kb + 8 * n + (lane & 7), 4 * k + (lane >> 3)));
            mma<T>(s[n], qf[2 * k], f[0], f[1]);
            mma<T>(s[n], qf[2 * k + 1], f[2], f[3]);
          }
      } else {
#pragma unroll
        for (int k = 0; k < DP / 64; ++k)
#pragma unroll
          for (int n = 0; n < S::kBlock / 8; ++n) {
            uint32_t f[4];
            ldsm4(f, kd + place<S::kChunks>(kb + 8 * n + (lane & 7), 4 * k + (lane >> 3)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b[2];
              e4m3_to_f16(b, f[i]);
              mma<T>(s[n], qf[4 * k + i], b[0], b[1]);
            }
          }
      }
      const bool ragged = key + S::kBlock > all_see;
#pragma unroll
      for (int n = 0; n < S::kBlock / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] *= row_scale[i >> 1];
      if (ragged)
#pragma unroll
        for (int n = 0; n < S::kBlock / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + 8 * n + 2 * t4 + (i & 1) >= limit[i >> 1]) s[n][i] = -INFINITY;
      float top[2] = {S::kLift ? -INFINITY : m_run[0], S::kLift ? -INFINITY : m_run[1]};
#pragma unroll
      for (int n = 0; n < S::kBlock / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
      float base[2];
      bool grew = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(~0u, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(~0u, top[h], 2));
        if (S::kLift) top[h] = fmaxf(m_run[h], __fadd_ru(top[h], -S::kLift));  // upwards: no more than 2^kLift
        base[h] = top[h] == -INFINITY ? 0.0f : top[h];
        grew |= top[h] > m_run[h];
      }
      if (__any_sync(~0u, grew)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = exp2_fast(m_run[h] - base[h]);  // 0 before the first key
          l_run[h] *= f;
          m_run[h] = top[h];
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) o[i][2 * h] *= f, o[i][2 * h + 1] *= f;
        }
      }
#pragma unroll
      for (int n = 0; n < S::kBlock / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[n][i] = exp2_fast(s[n][i] - base[i >> 1]);
          l_run[i >> 1] += s[n][i];
        }
      // o += p v. Keys that some rows see and others do not (at most rows - 1): a hidden value must not reach a row
      // even times 0 (it may be NaN), so they leave the product (Mixed) and are added one by one below.
      auto add_values = [&](auto mixed_tag) {
        constexpr bool kMixed = decltype(mixed_tag)::value;
#pragma unroll
        for (int q = 0; q < S::kBlock / 16; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = s[2 * q + (i >> 1)][2 * (i & 1)], y = s[2 * q + (i >> 1)][2 * (i & 1) + 1];
            hi[i] = pack2<T>(x, y);
            if (PAIRS) {
              const float2 r = unpack2<T>(hi[i]);
              lo[i] = pack2<T>(x - r.x, y - r.y);
            }
          }
          uint32_t keep[2] = {~0u, ~0u};
          if (kMixed)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int k0 = key + 16 * q + 8 * i + 2 * t4;
              keep[i] = (k0 < all_see ? 0xffffu : 0) | (k0 + 1 < all_see ? 0xffff0000u : 0);
            }
          const int vrow = kb + 16 * q + (lane & 7) + ((lane >> 3) & 1) * 8;
          if (!E4M3) {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
              uint32_t f[4];
              ldsm4t(f, vd + place<S::kChunks>(vrow, 2 * d + (lane >> 4)));
              if (kMixed) f[0] &= keep[0], f[1] &= keep[1], f[2] &= keep[0], f[3] &= keep[1];
              mma<T>(o[2 * d], hi, f[0], f[1]);
              mma<T>(o[2 * d + 1], hi, f[2], f[3]);
              mma<T>(o[2 * d], lo, f[0], f[1]);
              mma<T>(o[2 * d + 1], lo, f[2], f[3]);
            }
          } else {
            // transposed pairs of bytes: even elements of 16 make one n8 tile, odd ones the next
#pragma unroll
            for (int d = 0; d < DP / 32; ++d) {
              uint32_t f[4];
              ldsm4t(f, vd + place<S::kChunks>(vrow, 2 * d + (lane >> 4)));
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t u[2], v[2];
                e4m3_to_f16(u, __byte_perm(f[2 * i], 0, 0x3120));
                e4m3_to_f16(v, __byte_perm(f[2 * i + 1], 0, 0x3120));
                if (kMixed) u[0] &= keep[0], u[1] &= keep[0], v[0] &= keep[1], v[1] &= keep[1];
                mma<T>(o[4 * d + 2 * i], hi, u[0], v[0]);
                mma<T>(o[4 * d + 2 * i + 1], hi, u[1], v[1]);
                if (PAIRS) {
                  mma<T>(o[4 * d + 2 * i], lo, u[0], v[0]);
                  mma<T>(o[4 * d + 2 * i + 1], lo, u[1], v[1]);
                }
              }
            }
          }
        }
      };
      if (!ragged || a.rows == 1) {
        add_values(std::false_type{});
      } else {
        add_values(std::true_type{});
#pragma unroll 1
        for (int x = max(0, all_see - key); x < S::kBlock && key + x < m.len; ++x) {
          // the probability of key x sits with lane (x % 8) / 2 of each row's quad
          float pr[2] = {0, 0};
#pragma unroll
          for (int n = 0; n < S::kBlock / 8; ++n)
            if (n == x >> 3) {
              pr[0] = x & 1 ? s[n][1] : s[n][0];
              pr[1] = x & 1 ? s[n][3] : s[n][2];
            }
          const int src = (lane & ~3) | ((x & 7) >> 1);
          pr[0] = __shfl_sync(~0u, pr[0], src);
          pr[1] = __shfl_sync(~0u, pr[1], src);
          const bool see[2] = {key + x < limit[0], key + x < limit[1]};
          const unsigned char* row = smem + S::kOffKV + stage * S::kStageBytes + S::kKeyBytes;
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            float2 v;
            if (!E4M3) {
              const int d = 8 * i + 2 * t4;
              v = unpack2<T>(*reinterpret_cast<const uint32_t*>(row + place<S::kChunks>(kb + x, d / 8) + (d % 8) * 2));
            } else {
              const int d = 16 * (i >> 1) + 4 * t4;  // this tile's elements: d + (i & 1), d + 2 + (i & 1)
              const uint32_t u = *reinterpret_cast<const uint32_t*>(row + place<S::kChunks>(kb + x, d / 16) + d % 16);
              uint32_t pair[2];
              e4m3_to_f16(pair, __byte_perm(u, 0, 0x3120));
              v = unpack2<__half>(pair[i & 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (see[h]) o[i][2 * h] += pr[h] * v.x, o[i][2 * h + 1] += pr[h] * v.y;
          }
        }
      }
    }

    if (m.last && p.parts <= 1) {  // the end of this CTA's part of the request
      const long long slot = 2ll * blockIdx.x + m.slot;
      join_warps(reinterpret_cast<float*>(smem + S::kOffKV + stage * S::kStageBytes),
                 min(S::kRows, p.n_rows - m.block * S::kRows), [&](int row, int d, float4 y, float top, float sum) {
                   if (m.whole) {
                     finish(m.b, m.head, m.block, row, d, y, top, sum);
                   } else {
                     *reinterpret_cast<float4*>(p.part + (slot * S::kRows + row) * DP + d) = y;
                     if (d == 0) p.part_ml[slot * S::kRows + row] = make_float2(top, sum);
                   }
                 });
    }
    describe(next, (ring + S::kStages) % S::kRing);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    ring = ring + 1 == S::kRing ? 0 : ring + 1;
  }
  cp_wait<0>();
  if (p.parts <= 1) return;

  // ---- a cluster's join: each CTA's rows in its own shared memory, then each CTA sums its share of the columns ------------
  cg::cluster_group cluster = cg::this_cluster();
  const int item = blockIdx.x / p.parts, rank = blockIdx.x - item * p.parts;
  const int b = item / hm_n, hm = item - b * hm_n, head = hm / p.blocks, block = hm - head * p.blocks;
  const int rows = min(S::kRows, p.n_rows - block * S::kRows);
  float* mine = reinterpret_cast<float*>(smem + S::kOffKV);           // [kRows][DP]
  float2* mine_ml = reinterpret_cast<float2*>(smem + S::kOffQ);       // [kRows]
  join_warps(reinterpret_cast<float*>(smem + S::kOffKV + S::kRows * DP * 4), rows,
             [&](int row, int d, float4 y, float top, float sum) {
               *reinterpret_cast<float4*>(mine + row * DP + d) = y;
               if (d == 0) mine_ml[row] = make_float2(top, sum);
             });
  cluster.sync();
  for (int i = tid * p.parts + rank; i < rows * (DP / 4); i += S::kThreads * p.parts) {
    const int row = i / (DP / 4), d = (i % (DP / 4)) * 4;
    float top = -INFINITY;
    for (int c = 0; c < p.parts; ++c) top = fmaxf(top, cluster.map_shared_rank(mine_ml, c)[row].x);
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0;
    float4 y = make_float4(0, 0, 0, 0);
    for (int c = 0; c < p.parts; ++c) {
      const float2 s = cluster.map_shared_rank(mine_ml, c)[row];
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(mine, c) + row * DP + d);
      const float f = exp2_fast(s.x - base);
      sum += f * s.y;
      y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
    }
    finish(b, head, block, row, d, y, top, sum);
  }
  cluster.sync();  // the others' shared memory stays until it has been read
}

// One build's launch facts, filled by the three translation units that hold the kernels.
struct Build {
  int rows, tile;
  cudaError_t (*occupancy)(int device, int* ctas_per_sm);
  cudaError_t (*clusters)(int device, int parts, int* resident);
  cudaError_t (*launch)(const Params& p, cudaStream_t s);
};

template <typename T, int DP, int MT, bool E4M3, bool LONG = false, bool PAIRS = !E4M3>
struct Make {
  using S = Shape<T, DP, MT, E4M3, LONG>;
  static constexpr auto kKernel = attention_kernel<T, DP, MT, E4M3, LONG, PAIRS>;
  static cudaError_t occupancy(int device, int* n) {
    static std::atomic<int> known[kMaxDevices];
    *n = known[device].load(std::memory_order_relaxed);
    if (*n) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kKernel, S::kThreads, S::kSmem);
    if (e == cudaSuccess && *n < 1) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) known[device].store(*n, std::memory_order_relaxed);
    return e;
  }
  static cudaLaunchConfig_t config(int ctas, int parts, cudaLaunchAttribute* at, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    if (parts) {
      at->id = cudaLaunchAttributeClusterDimension;
      at->val.clusterDim.x = parts;
      at->val.clusterDim.y = at->val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
    }
    return cfg;
  }
  // clusters of 2, 4, 8 or 16 CTAs the device holds at once (0: none); occupancy() has run
  static cudaError_t clusters(int device, int parts, int* n) {
    static std::atomic<int> known[kMaxDevices][17];
    const int k = known[device][parts].load(std::memory_order_relaxed);
    *n = k - 1;
    if (k) return cudaSuccess;
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t cfg = config(parts, parts, at, nullptr);
    if (cudaOccupancyMaxActiveClusters(n, kKernel, &cfg) != cudaSuccess) {
      cudaGetLastError();  // a size the device does not have
      *n = 0;
    }
    known[device][parts].store(*n + 1, std::memory_order_relaxed);
    return cudaSuccess;
  }
  static cudaError_t launch(const Params& p, cudaStream_t s) {
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t cfg = config(p.ctas, p.parts, at, s);
    return cudaLaunchKernelEx(&cfg, kKernel, p);
  }
  static constexpr Build build() { return {S::kRows, S::kTile, occupancy, clusters, launch}; }
};

// longer: the call's tiles are one line. 16-bit caches 64 wide then have tiles of 128 keys up to 32 rows (64 requests of 1 to
// 16384 positions, 32 / 8 heads: 212 us against 242 with 64 keys; 64 / 2 heads: 265, 336), of 64 with more (48 rows: 367
// against 442, fewer CTAs on an SM); a cluster wants more tiles to share (129 requests of up to 700: 8.7 against 10.4).
template <typename T, bool E4M3, bool PAIRS = !E4M3>
inline const Build* pick(int dp, int mt, bool longer) {
  if constexpr (!E4M3) {
    static constexpr Build narrow[2] = {Make<T, 64, 1, false, true>::build(), Make<T, 64, 2, false, true>::build()};
    if (longer && dp == 64 && mt <= 2) return &narrow[mt - 1];
  }
  static constexpr Build all[3][4] = {
      {Make<T, 64, 1, E4M3, false, PAIRS>::build(), Make<T, 64, 2, E4M3, false, PAIRS>::build(),
       Make<T, 64, 3, E4M3, false, PAIRS>::build(), Make<T, 64, 4, E4M3, false, PAIRS>::build()},
      {Make<T, 128, 1, E4M3, false, PAIRS>::build(), Make<T, 128, 2, E4M3, false, PAIRS>::build(),
       Make<T, 128, 3, E4M3, false, PAIRS>::build(), Make<T, 128, 4, E4M3, false, PAIRS>::build()},
      {Make<T, 256, 1, E4M3, false, PAIRS>::build(), Make<T, 256, 2, E4M3, false, PAIRS>::build(),
       Make<T, 256, 3, E4M3, false, PAIRS>::build(), Make<T, 256, 4, E4M3, false, PAIRS>::build()}};
  return &all[dp == 64 ? 0 : dp == 128 ? 1 : 2][mt - 1];
}

// mk_paged_attention's host-side refusals, in the name of `me`: of the shape, and all short of the workspace's.
mk_status check_shape(const char* me, const mk_paged_attention_args& a, int device);
mk_status check(const char* me, const mk_paged_attention_args& a, int device);

// The caches' strides (page, head, place) in units of 16 bytes; those of a dimension of one element are never used and 0 here.
inline void cache_steps(int cache_dtype, int n_pages, int n_kv_heads, int page_size, const int64_t* k, const int64_t* v,
                        uint32_t (&k_step)[3], uint32_t (&v_step)[3]) {
  const int dims[3] = {n_pages, n_kv_heads, page_size}, unit = cache_dtype == MK_E4M3 ? 16 : 8;
  for (int i = 0; i < 3; ++i) {
    k_step[i] = dims[i] > 1 ? static_cast<uint32_t>(k[i] / unit) : 0;
    v_step[i] = dims[i] > 1 ? static_cast<uint32_t>(v[i] / unit) : 0;
  }
}

const Build* pick_bf16(int dp, int mt, bool longer);
const Build* pick_f16(int dp, int mt, bool longer);
const Build* pick_e4m3_bf16(int dp, int mt, bool longer);
const Build* pick_e4m3_f16(int dp, int mt, bool longer);

}  // namespace attn
}  // namespace mkop
