// The kernel of mk_prefix_attention, on the 5th-generation tensor cores with accumulators in tensor memory
// (prefix_attention.cu: arguments and the join).
//
// For a kv head, every query row of every request meets the same keys of the prefix, and the rows of one request its own keys:
// scores S = Q K^T of [128 rows x 128 keys], an online softmax, sums O += P V. At rows x 2 flops a cached byte (16 bits) this
// is bound by the tensor cores from about 280 rows on, by memory below.
// - Work: 128 query rows of a kv head are a row tile. Three lines of key tiles, each cut into equal pieces, one piece a CTA:
//   pairs of row tiles over the prefix (a tile of keys and values is read once for 256 rows), single row tiles over the prefix
//   (an odd one; all of them 256 wide, where the tensor memory holds one), and row tiles of one request (of up to 8 of its
//   new rows) over its own keys. CTAs are dealt to the lines in proportion to their products, by a rule on the lengths alone.
//   Where a CTA has one row tile, even and odd key tiles go to two sets of sums, so that there are two streams of work
//   in any case (one 256 wide).
// - Units: the product of one row tile and one key tile, in turn on two score buffers. One warp issues S(0), S(1), then
//   for each unit u: O += P(u) V and S(u + 2): while one stream's softmax runs, the tensor cores work on the other.
// - Softmax: a thread has a row (128 threads a stream), so nothing is exchanged; its 128 scores are in registers at once.
//   Probabilities go back to tensor memory over the first half of the scores' columns as the product's operand (16 bits).
//   They are taken against a base that moves only when a score passes it by kPrefixGrow: else sums stay as they are.
// - Loads: warps 9-11 copy keys, 12-14 values (cp.async, row by row through the page table) into a ring of slots; codes of e4m3
//   caches pass through registers and become fp16 there. Queries are stored by the softmax threads; those of the next item
//   while the last product of this one runs.
// - Keys that not every row of a request's tile sees (at most 7): their values stay out of the product (they may hold
//   anything, NaN too) and are added one by one at the item's end, by the rows that see them.
// Probabilities are one 16-bit number (a pair hi + lo would be half as much work again for the tensor cores). bf16: 2^-8 of each
// at most; fp16: 2^-11, against a base 14 under the maximum, so that what falls under its range is 2^-39 of the largest. Sums of
// probabilities are those of the unrounded ones.
// Every wait has a limit (2 s), after which the CTA gives up, drains and frees what it holds and MK_OP_TIMEOUT is set.
#pragma once
#include "paged_attention_tc.cuh"

namespace mkop {
namespace prefix {

using namespace attn;

constexpr int kPrefixTile = 128;      // keys
constexpr int kTileRows = 128;        // query rows of a row tile
constexpr int kGroupRows = 8;         // new rows of a request that share an item over its own keys
constexpr int kMinPiece = 1;          // key tiles of a piece at least
enum { kPairs, kSingles, kOwn };      // the lines

// What the first CTA writes for the join. Piece c's part of item i of a line goes to place c + i (after `place0`): along the line
// either grows by one from part to part.
struct Head {
  long long total[3];  // key tiles of a line
  int used[3];         // its pieces
  int tiles;           // key tiles of the prefix
  __device__ static int piece_of(long long x, long long total, int used) {  // the last piece that begins at or before tile x
    if (total <= 0xffffffffu / static_cast<unsigned>(used))
      return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(used) - 1) / static_cast<uint32_t>(total));
    return static_cast<int>(((x + 1) * used - 1) / total);
  }
};

struct PrefixParams {
  mk_prefix_attention_args a;
  Div page, group_div, row_div, q_head_div;
  int group;          // query heads per kv head
  int n_rows;         // query rows of a kv head: batch * rows * group
  int max_prefix, max_own;
  int dp;             // 64, 128 or 256
  int streams;        // sums a place holds (1 at 256 wide, else 2)
  int blocks[3];      // pairs and single row tiles of a kv head; row tiles of a request's row group
  int groups;         // row groups of a request
  int own_rows;       // rows of a place over own keys
  int ctas;
  float scale_log2;   // |scale| * log2(e)
  uint32_t flip;      // sign bits of two 16-bit values where the scale is negative: queries change their sign instead
  uint32_t k_step[3], v_step[3];  // the caches' strides (page, head, place) in units of 16 bytes
  float* part;        // [places][streams][128][dp] sums of a part over the prefix
  float2* part_ml;    // [places][streams][128] its base (log2 units) and sum of probabilities; sum 0: an empty part, sums not written
  float* own;         // [places][streams][own_rows][dp] and
  float2* own_ml;     // [places][streams][own_rows] over own keys
  Head* head;
  long long* cum;     // [batch * groups + 1] key tiles of the row groups so far (of one row tile)
  __device__ int first_single() const { return blocks[kPairs] * 2 * kTileRows; }
  __device__ int rows_of(int group_index) const { return min(kGroupRows, a.rows - group_index * kGroupRows); }
  // Own keys of a row group: those its last row sees.
  __device__ int own_len(int bg) const {
    const int b = bg / groups, g = bg - b * groups;
    return max(0, min(max(a.lens[b], 0), max_own) - (a.rows - g * kGroupRows - rows_of(g)));
  }
  __device__ static int tiles_of(int len) { return (len + kPrefixTile - 1) >> 7; }
};

// A role's place in its CTA's piece of a line.
struct PrefixWalk {
  const PrefixParams& p;
  int line, per;          // per: items of a row group
  long long item;         // of the line
  int bg, hm, len, n, tile;  // own: row group, item in it; keys and key tiles of the item, the current one
  long long done, count;
  __device__ bool ends() const { return done >= count; }
  // key tiles of the item from here on, in this piece
  __device__ long long left() const { return min(static_cast<long long>(n - tile), count - done); }
  __device__ void next_item() {
    ++item;
    tile = 0;
    if (line != kOwn) {
      hm = static_cast<int>(item);
    } else if (++hm == per && !ends()) {  // (there is another group with keys, then)
      hm = 0;
      item -= per;
      do {  // (groups without keys have no tiles, but items)
        item += per;
        len = p.own_len(++bg);
        n = PrefixParams::tiles_of(len);
      } while (n == 0);
    }
  }
  __device__ void next() {
    ++done;
    if (++tile == n) next_item();
  }
  __device__ void skip() {
    done += left();
    next_item();
  }
  __device__ int kv_head() const { return hm / p.blocks[line]; }
  __device__ int block() const { return hm - kv_head() * p.blocks[line]; }
  __device__ int request() const { return bg / p.groups; }
  __device__ int group_rows() const { return p.rows_of(bg - request() * p.groups); }
  __device__ int all_see() const { return line == kOwn ? len - (group_rows() - 1) : len; }  // keys before it are seen by every row
};

// Registers of a thread: 256 threads each of 512 launched with 128 (e4m3 loaders hold codes in registers)
template <bool E4M3>
constexpr int kSoftmaxRegs = E4M3 ? 176 : 192;
template <bool E4M3>
constexpr int kOtherRegs = E4M3 ? 72 : 56;

template <int D>
struct PrefixShape {
  static constexpr int kThreads = 512, kLoaders = 96, kStreamThreads = 128;
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kHalves = D == 256 ? 2 : 1;          // slots of a tile's keys
  static constexpr int kWide = D == 256 ? 128 : D;          // columns of a slot
  static constexpr int kSlot = kPrefixTile * kWide * 2;
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kQ = kTileRows * D * 2;              // a stream's queries
  static constexpr int kOffQ = kSlots * kSlot;
  static constexpr int kOffAddr = kOffQ + kStreams * kQ;    // address [2 roles][2 tiles][128]
  // of keys that not all rows see: scores, float [2 streams][8][128]; values as they are in the cache, [streams][2 turns][8][D]
  static constexpr int kOffLate = kOffAddr + 2 * 2 * 128 * 8;
  static constexpr int kOffLateV = kOffLate + 2 * kGroupRows * 128 * 4;
  static constexpr int kOffBar = kOffLateV + kStreams * 2 * kGroupRows * D * 2;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

template <typename T>
constexpr float kPrefixLift = std::is_same<T, __half>::value ? 14.0f : 0.0f;  // the base is this much under the maximum
template <typename T>
constexpr float kPrefixGrow = std::is_same<T, __half>::value ? 1.0f : 8.0f;   // and moves when a score passes that by this

struct PrefixBars {
  uint64_t full[8], empty[8], q_full[2], s_full[2], p_full[2], pv_done[2], late_full[2], drained;
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(PrefixBars) <= 512, "");

// D[tmem] (+)= A[tmem] B: A is 16-bit pairs, a lane a row
__device__ inline void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
// One lane of a converged warp, the same each time.
__device__ inline bool elected() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// A value that all lanes have, as the warp's one value.
__device__ inline uint32_t of_warp(uint32_t x) { return __reduce_max_sync(~0u, x); }
// 64 consecutive fp32 columns of this warp's 32 lanes into v[at ..]. Load and wait are one statement: before the wait the
// registers do not hold the values.
__device__ inline void tc_ld64(float (&v)[128], int at, uint32_t addr) {
  uint32_t r[64];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
               "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,"
               "%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
                 "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
                 "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
                 "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
                 "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]),
                 "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]),
                 "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]), "=&r"(r[54]), "=&r"(r[55]),
                 "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]), "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63])
               : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[at + i] = __uint_as_float(r[i]);
}
// One column.
__device__ inline void tc_ld1(float& v, uint32_t addr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n"
               "tcgen05.wait::ld.sync.aligned;" : "=&r"(r) : "r"(addr) : "memory");
  v = __uint_as_float(r);
}
// 16 consecutive columns of this warp's lanes from packed values (tcgen05.wait::st follows separately)
__device__ inline void tc_st_packed(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}
// Two fp32 operations in one instruction
__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 x, y, z, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 w, x, y, z;\nmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ inline float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, w;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 w, x, y;\nmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ inline float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ inline void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Instruction descriptor: fp32 sums, 16-bit operands, M = 128; `turned`: B is N-major
template <typename T>
__device__ constexpr uint32_t prefix_idesc(int n, bool turned) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (turned ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

// T: the products' type; QT: the queries'; E4M3: the cache holds codes (T is __half then)
template <typename T, typename QT, int D, bool E4M3>
__global__ void __launch_bounds__(PrefixShape<D>::kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
  using S = PrefixShape<D>;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t s0 = smem_u32(smem);
  const mk_prefix_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = of_warp(tid >> 5);
  PrefixBars& bars = *reinterpret_cast<PrefixBars*>(smem + S::kOffBar);
  volatile int* dead = &bars.dead;
  __shared__ long long warp_tiles[S::kThreads / 32];
  __shared__ long long at_rem;
  __shared__ int at_bg;

  // ---- the lines, and this CTA's piece of one -------------------------------------------------------------------------
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Head hd;
  int line, c = blockIdx.x;
  long long begin;
  const int n_groups = a.batch * p.groups, per = a.n_kv_heads * p.blocks[kOwn];
  const int prefix_len = min(max(a.prefix_len[0], 0), p.max_prefix);
  {
    const int each = (n_groups + S::kThreads - 1) / S::kThreads;
    const int g0 = min(n_groups, tid * each), g1 = min(n_groups, g0 + each);
    long long mine = 0;
    for (int g = g0; g < g1; ++g) mine += PrefixParams::tiles_of(p.own_len(g));
    long long before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, before, d);
      if (lane >= d) before += o;
    }
    if (lane == 31) warp_tiles[warp] = before;
    __syncthreads();
    before -= mine;
    long long own = 0;
    for (int w = 0; w < S::kThreads / 32; ++w) {
      if (w < warp) before += warp_tiles[w];
      own += warp_tiles[w];
    }
    hd.tiles = PrefixParams::tiles_of(prefix_len);
    hd.total[kPairs] = static_cast<long long>(a.n_kv_heads) * p.blocks[kPairs] * hd.tiles;
    hd.total[kSingles] = static_cast<long long>(a.n_kv_heads) * p.blocks[kSingles] * hd.tiles;
    hd.total[kOwn] = own * per;
    // A line's CTAs: in proportion to its products, one at least. (An item over own keys counts as a tile more: it is short.)
    const int ctas = gridDim.x;
    const long long cost[3] = {2 * hd.total[kPairs], hd.total[kSingles],
                               hd.total[kOwn] ? hd.total[kOwn] + static_cast<long long>(n_groups) * per : 0};
    const long long sum = cost[0] + cost[1] + cost[2];
    int n0 = cost[0] ? max(1, static_cast<int>(cost[0] * ctas / sum)) : 0, n1 = cost[1] ? max(1, static_cast<int>(cost[1] * ctas / sum)) : 0;
    const int most = ctas - (cost[2] ? 1 : 0);
    if (n0 + n1 > most) (n0 > n1 ? n0 : n1) -= n0 + n1 - most;
    if (!cost[2]) (cost[1] ? n1 : n0) += most - n0 - n1;
    const int got[3] = {n0, n1, ctas - n0 - n1};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long worth = (hd.total[i] + kMinPiece - 1) / kMinPiece;
      hd.used[i] = static_cast<int>(worth < got[i] ? worth : got[i]);
    }
    line = c < n0 ? kPairs : c < n0 + n1 ? kSingles : kOwn;
    c -= line == kPairs ? 0 : line == kSingles ? n0 : n0 + n1;
    begin = hd.used[line] ? piece_begin(c, hd.total[line], hd.used[line]) : 0;
    if (blockIdx.x == 0) {
      if (tid == 0) {
        *p.head = hd;
        p.cum[n_groups] = own;
        if (prefix_len != a.prefix_len[0]) flag(a.status, MK_OP_BAD_LENGTH);
      }
      long long at = before;
      for (int g = g0; g < g1; ++g) {
        p.cum[g] = at;
        at += PrefixParams::tiles_of(p.own_len(g));
        const int b = g / p.groups;
        if (a.lens[b] < 0 || a.lens[b] > p.max_own) flag(a.status, MK_OP_BAD_LENGTH);
      }
    }
    if (line == kOwn && c < hd.used[kOwn] && before * per <= begin && begin < (before + mine) * per) {
      for (int g = g0; g < g1; ++g) {
        const int n = PrefixParams::tiles_of(p.own_len(g));
        if (begin < (before + n) * per) {
          at_bg = g;
          at_rem = begin - before * per;
          break;
        }
        before += n;
      }
    }
  }
  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) bar_init(&bars.full[i], S::kLoaders), bar_init(&bars.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.q_full[i], S::kStreamThreads), bar_init(&bars.s_full[i], 1);
      bar_init(&bars.p_full[i], S::kStreamThreads), bar_init(&bars.pv_done[i], 1);
      bar_init(&bars.late_full[i], S::kStreamThreads);
    }
    bar_init(&bars.drained, 1);
    bars.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (c >= hd.used[line]) return;
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = bars.tmem;
  const bool pair = line == kPairs;
  const long long count = piece_begin(c + 1, hd.total[line], hd.used[line]) - begin;  // key tiles of this piece
  auto walk = [&]() -> PrefixWalk {
    PrefixWalk w{p, line, per, 0, 0, 0, prefix_len, hd.tiles, 0, 0, count};
    if (line == kOwn) {
      w.bg = at_bg;
      w.len = p.own_len(w.bg);
      w.n = PrefixParams::tiles_of(w.len);
      w.hm = static_cast<int>(at_rem / w.n);
      w.tile = static_cast<int>(at_rem - static_cast<long long>(w.hm) * w.n);
      w.item = static_cast<long long>(w.bg) * per + w.hm;
    } else {
      w.item = begin / hd.tiles;
      w.tile = static_cast<int>(begin - w.item * hd.tiles);
      w.hm = static_cast<int>(w.item);
    }
    return w;
  };

  // (256 x (192 + 56) or 256 x (176 + 72) registers: 63488 of the 65536 of 512 x 128)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<E4M3>));
    if (warp >= 9 && warp < 15) {
      // ---- loaders ------------------------------------------------------------------------------------------------
      const bool value = warp >= 12;
      const int t = tid - (value ? 384 : 288), barrier = value ? 3 : 2;
      const unsigned char** addr = reinterpret_cast<const unsigned char**>(smem + S::kOffAddr) + (value ? 256 : 0);
      PrefixWalk w = walk();  // at the next tile that gets addresses
      auto look_up = [&](int key) -> int {
        key += w.tile * kPrefixTile;
        if (w.ends() || key >= w.len) return -1;
        return line == kOwn ? a.table[w.request() * a.table_stride + p.page(key)] : a.prefix_table[p.page(key)];
      };
      auto make_address = [&](const unsigned char** at, int page, int i) {
        const unsigned char* from = kZeros;
        const int key = w.tile * kPrefixTile + i;
        if (!w.ends() && key < w.len) {
          if (page < 0 || page >= a.n_pages) {
            flag(a.status, MK_OP_BAD_PAGE);
          } else if (!value || key < w.all_see()) {
            const int place = key - p.page(key) * a.page_size, head = w.kv_head();
            from = value ? row_at(a.v_pages, p.v_step, page, head, place) : row_at(a.k_pages, p.k_step, page, head, place);
          }
        }
        at[i] = from;
      };
      const bool two = t < 128 - S::kLoaders;
      bool ok = true;
      make_address(addr, look_up(t), t);
      if (two) make_address(addr, look_up(t + S::kLoaders), t + S::kLoaders);
      w.next();
      int page = look_up(t), page2 = two ? look_up(t + S::kLoaders) : -1;
      constexpr int kSrc = E4M3 ? S::kWide / 16 : S::kWide / 8;  // 16-byte pieces of a slot's row in the cache
      constexpr int kStep = S::kLoaders / kSrc, kTurns = (kPrefixTile + kStep - 1) / kStep;
      const int chunk = t % kSrc, row0 = t / kSrc;
      for (long long j = 0; j < count; ++j) {
        const unsigned char** at = addr + (j & 1) * 128;
        if (any_of(barrier, S::kLoaders, !ok)) break;
#pragma unroll 1
        for (int h = 0; h < S::kHalves; ++h) {
          const uint32_t g = (static_cast<uint32_t>(j) * 2 + (value ? 1 : 0)) * S::kHalves + h;
          const int slot = g % S::kSlots, turn = (g / S::kSlots) & 1;
          const bool waits = j >= S::kSlots / (2 * S::kHalves);         // the slot has been used before
          const int column = h * S::kWide * (E4M3 ? 1 : 2) + chunk * 16;  // bytes
          const bool in = column < a.head_dim * (E4M3 ? 1 : 2);         // columns behind the head are not read, or not used
          const unsigned char* const* from = at + row0;
          if (!E4M3) {
            if (waits) ok = bar_wait(&bars.empty[slot], turn ^ 1, dead) && ok;
            const uint32_t to = s0 + slot * S::kSlot + (chunk >> 3) * (kPrefixTile * 128);
            if (in)
#pragma unroll
              for (int i = 0; i < kTurns; ++i) {
                const int row = row0 + kStep * i;
                if (row >= kPrefixTile) break;
                cp16(to + row * 128 + (((chunk ^ row) & 7) << 4), from[kStep * i] + column);
              }
            cp_arrive(&bars.full[slot]);
          } else {
            constexpr int kAhead = kTurns < 6 ? kTurns : 6;  // loads in flight
            uint4 u[kAhead];
            auto fetch = [&](int i) {
              if (row0 + kStep * i < kPrefixTile)
                u[i % kAhead] = in ? *reinterpret_cast<const uint4*>(from[kStep * i] + column) : make_uint4(0, 0, 0, 0);
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i);
            if (waits) ok = bar_wait(&bars.empty[slot], turn ^ 1, dead) && ok;
            // codes 16 chunk .. become pieces 2 chunk and 2 chunk + 1
            unsigned char* to = smem + slot * S::kSlot + (chunk >> 2) * (kPrefixTile * 128);
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
              const int row = row0 + kStep * i;
              if (row >= kPrefixTile) break;
              const uint4 x = u[i % kAhead];
              if (i + kAhead < kTurns) fetch(i + kAhead);
              const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t lo[2], hi[2];
                e4m3_to_f16(lo, v[2 * k]);
                e4m3_to_f16(hi, v[2 * k + 1]);
                *reinterpret_cast<uint4*>(to + row * 128 + ((((2 * chunk + k) ^ row) & 7) << 4)) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
              }
            }
            proxy_fence();
            bar_arrive(&bars.full[slot]);
          }
          if (h == 0) {  // the next tile's addresses, while copies are in flight
            make_address(addr + (~j & 1) * 128, page, t);
            if (two) make_address(addr + (~j & 1) * 128, page2, t + S::kLoaders);
            if (!w.ends()) w.next();
            page = look_up(t);
            if (two) page2 = look_up(t + S::kLoaders);
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 8) {
      // ---- the warp that issues the products ----------------------------------------------------------------------------
      // All lanes walk and wait together, on values that are the warp's; one issues. (Under a branch of one lane, on values of
      // that lane, a product took 130 cycles to issue.)
      constexpr uint32_t kScores = prefix_idesc<T>(kPrefixTile, false), kSums = prefix_idesc<T>(S::kWide, true);
      const int steps = a.head_dim / 16;
      const uint32_t tm = of_warp(tmem), base_q = of_warp(s0 + S::kOffQ), base_kv = of_warp(s0);
      const long long units = pair ? 2 * count : count;
      PrefixWalk ws = walk(), wp = walk();  // at the key tile of the next scores, of the next sums
      long long q_item0 = -1, q_item1 = -1, o_item0 = -1, o_item1 = -1;  // of either stream
      uint32_t q_turn0 = 0, q_turn1 = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (__all_sync(~0u, bar_try(bar, parity))) return true;
        return __all_sync(~0u, bar_wait(bar, parity, dead));
      };
      auto stream_of = [&](long long u) { return S::kStreams == 2 ? static_cast<int>(u) & 1 : 0; };
      // Waits for what the scores of unit u need.
      auto ready = [&](long long u) {
        const int st = stream_of(u);
        if (ws.item != (st ? q_item1 : q_item0)) {
          (st ? q_item1 : q_item0) = ws.item;
          ok = ok && wait(&bars.q_full[st], (st ? q_turn1 : q_turn0) & 1);
          ++(st ? q_turn1 : q_turn0);
        }
        if (pair && (u & 1)) return;  // the keys are those of unit u - 1
        const uint32_t j = static_cast<uint32_t>(pair ? u >> 1 : u);
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h) {
          const uint32_t g = j * 2 * S::kHalves + h;
          ok = ok && wait(&bars.full[g % S::kSlots], (g / S::kSlots) & 1);
        }
      };
      // By one lane, after ready().
      auto scores = [&](long long u) {
        const uint32_t j = static_cast<uint32_t>(pair ? u >> 1 : u), b = static_cast<uint32_t>(u) & 1;
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h) {
          const uint32_t slot = (j * 2 * S::kHalves + h) % S::kSlots;
          const uint64_t kd = tc_desc(base_kv + slot * S::kSlot, 16);
          const uint64_t qd = tc_desc(base_q + stream_of(u) * S::kQ + 2 * h * (kTileRows * 128), 16);
#pragma unroll
          for (int k = 0; k < S::kWide / 16; ++k)
            if (h * 8 + k < steps)
              tc_mma(tm + b * 128, qd + ((k >> 2) * (kTileRows * 128) + (k & 3) * 32) / 16,
                     kd + ((k >> 2) * (kPrefixTile * 128) + (k & 3) * 32) / 16, kScores, h > 0 || k > 0);
          if (!pair || b) tc_commit(&bars.empty[slot]);
        }
        tc_commit(&bars.s_full[b]);
      };
      auto after_scores = [&](long long u) {
        if ((!pair || (u & 1)) && !ws.ends()) ws.next();
      };
      for (int u = 0; u < 2 && u < units && ok; ++u) {
        ready(u);
        proxy_fence();
        tc_after();
        if (ok && elected()) scores(u);
        __syncwarp();
        after_scores(u);
      }
      for (long long u = 0; u < units && ok; ++u) {
        const int st = stream_of(u);
        const uint32_t j = static_cast<uint32_t>(pair ? u >> 1 : u), b = static_cast<uint32_t>(u) & 1;
        const bool fresh = wp.item != (st ? o_item1 : o_item0), more = u + 2 < units;
        (st ? o_item1 : o_item0) = wp.item;
        // The next scores' keys are waited for before these sums are issued, so that both run without a pause; not so
        // the first of another item, whose queries come after this unit's probabilities.
        const bool same = more && ws.item == (st ? q_item1 : q_item0);
        if (same) ready(u + 2);
        ok = ok && wait(&bars.p_full[b], static_cast<uint32_t>(u >> 1) & 1);
        if (!pair || !b) {
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h) {
            const uint32_t g = j * 2 * S::kHalves + S::kHalves + h;
            ok = ok && wait(&bars.full[g % S::kSlots], (g / S::kSlots) & 1);
          }
          proxy_fence();  // of these values, and of the keys that ready() waited for
        }
        if (!ok) break;
        tc_after();
        if (elected()) {
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h) {
            const uint32_t slot = (j * 2 * S::kHalves + S::kHalves + h) % S::kSlots;
            const uint64_t vd = tc_desc(base_kv + slot * S::kSlot, kPrefixTile * 128);
#pragma unroll
            for (int k = 0; k < kPrefixTile / 16; ++k)
              tc_mma_ts(tm + 256 + st * D + h * 128, tm + b * 128 + k * 8, vd + k * 2048 / 16, kSums, !fresh || k > 0);
            if (!pair || b) tc_commit(&bars.empty[slot]);
          }
          tc_commit(&bars.pv_done[b]);
          // (the scores of u + 2 go where the probabilities of u were: the products run in the order of their issue)
          if (same) scores(u + 2);
        }
        __syncwarp();
        if (more && !same) {
          ready(u + 2);
          proxy_fence();
          tc_after();
          if (ok && elected()) scores(u + 2);
          __syncwarp();
        }
        if (more) after_scores(u + 2);
        if ((!pair || b) && !wp.ends()) wp.next();
      }
      // every product has ended before the tensor memory is freed, also when the CTA gave up
      if (elected()) tc_commit(&bars.drained);
      int alive = 0;
      bar_wait(&bars.drained, 0, &alive);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<E4M3>));
    if (warp < 4 * S::kStreams) {
      // ---- softmax: a thread has a row of the stream's row tile -------------------------------------------------------
      const int st = warp >> 2, row = tid & 127;
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
      const uint32_t sums_at = tmem + lanes + 256 + static_cast<uint32_t>(st) * D;
      float* late = reinterpret_cast<float*>(smem + S::kOffLate) + st * kGroupRows * 128 + row;  // [8][128]
      float cs = fmaxf(p.scale_log2, 1.17549435e-38f);  // (a score of -infinity stays one where the scale is 0)
      float next_cs = cs;                               // of the queries loaded last
      // A warp's 32 rows of an item's queries into shared memory: a lane makes the address of its own row, D / 8 lanes copy one.
      auto load_queries = [&](const PrefixWalk& w) {
        const int head = w.kv_head();
        const float ks = E4M3 ? a.k_scale[head] : 1.0f;
        const uint32_t flip = p.flip ^ (ks < 0.0f ? 0x80008000u : 0u);
        long long mine = -1;
        if (line == kOwn) {
          const int m = w.block() * kTileRows + row, q = p.group_div(m), b = w.request();
          if (q < w.group_rows())
            mine = b * a.q_stride[0] + ((w.bg - b * p.groups) * kGroupRows + q) * a.q_stride[1] + (head * p.group + m - q * p.group) * a.q_stride[2];
        } else {
          const int m = pair ? (2 * w.block() + st) * kTileRows + row : p.first_single() + w.block() * kTileRows + row;
          if (m < p.n_rows) {
            const int br = p.group_div(m), h = head * p.group + m - br * p.group, b = p.row_div(br), qr = br - b * a.rows;
            mine = b * a.q_stride[0] + qr * a.q_stride[1] + h * a.q_stride[2];
          }
        }
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 8;
        const int chunk = lane % kLanes, sub = lane / kLanes;
        const bool in = chunk * 8 < a.head_dim;
        unsigned char* to = smem + S::kOffQ + st * S::kQ + (chunk >> 3) * (kTileRows * 128);
#pragma unroll 1
        for (int i0 = 0; i0 < kLanes; i0 += kBatch) {
          uint4 u[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const long long off = __shfl_sync(~0u, mine, (i0 + i) * kRows + sub);
            u[i] = make_uint4(0, 0, 0, 0);
            if (in && off != -1) u[i] = *reinterpret_cast<const uint4*>(static_cast<const QT*>(a.q) + off + chunk * 8);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = (row & ~31) + (i0 + i) * kRows + sub;
            uint4 x = u[i];
            x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
            if (E4M3) {
              // fp16 against a power of two near the row's largest (bf16 mantissas fit); the scores take it back
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              float big = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2<QT>(w[k]);
                big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
#pragma unroll
              for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
              const int e = big > 0 && big < INFINITY ? min(max(ilogbf(big), -120), 120) : 0;
              const float down = __uint_as_float((127 - e) << 23);
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = unpack2<QT>(w[k]);
                v[k] = pack2<__half>(f.x * down, f.y * down);
              }
              x = make_uint4(v[0], v[1], v[2], v[3]);
              const float up = __shfl_sync(~0u, __uint_as_float((127 + e) << 23), (lane % kRows) * kLanes);
              if (lane / kRows == i0 + i) next_cs = fmaxf(p.scale_log2 * fabsf(ks), 1.17549435e-38f) * up;
            }
            *reinterpret_cast<uint4*>(to + r * 128 + (((chunk ^ r) & 7) << 4)) = x;
          }
        }
        proxy_fence();
        bar_arrive(&bars.q_full[st]);
      };
      // the first key tile of this stream in the piece's tiles j0 .. j1 - 1 of an item
      auto first_of = [&](long long j0) { return pair || S::kStreams == 1 ? j0 : j0 + ((j0 ^ st) & 1); };
      bool ok = true;
      uint32_t late_turn = 0;
      const int rows = line == kOwn ? p.own_rows : kTileRows;  // of a place
      auto row_of = [&](const PrefixWalk& w) -> long long {    // this row's place among the parts
        long long place = c + w.item;
        if (line == kSingles) place += hd.used[kPairs] + static_cast<long long>(a.n_kv_heads) * p.blocks[kPairs];
        return (place * S::kStreams + st) * rows + row;
      };
      // w: the next item with key tiles for this stream. Those before it get an empty part.
      PrefixWalk w = walk();
      auto seek = [&]() {
        for (; !w.ends() && first_of(w.done) >= w.done + w.left(); w.skip())
          if (row < rows) (line == kOwn ? p.own_ml : p.part_ml)[row_of(w)] = make_float2(-INFINITY, 0.0f);
      };
      seek();
      if (!w.ends()) load_queries(w);
      while (ok && !w.ends()) {
        const long long j0 = w.done, j1 = j0 + w.left(), at_row = row_of(w);
        float2* ml = (line == kOwn ? p.own_ml : p.part_ml) + at_row;
        long long j = first_of(j0);
        cs = next_cs;
        const int first_tile = w.tile;
        // keys that this row sees: those before `limit`
        int limit = w.len;
        if (line == kOwn) limit -= max(0, w.group_rows() - 1 - p.group_div(w.block() * kTileRows + row));
        const int all_see = w.all_see(), len = w.len;
        uint32_t late_keys = 0;  // of this part: bit i is key all_see + i
        float base = kNoBase, l = 0;  // (the first unit sets the base)
        bool first = true;
        long long u = 0;
        for (; ok && j < j1; j += pair ? 1 : S::kStreams) {
          u = pair ? 2 * j + st : j;
          ok = __all_sync(~0u, bar_wait(&bars.s_full[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead));
          if (!ok) break;
          tc_after();
          const int key0 = (first_tile + static_cast<int>(j - j0)) * kPrefixTile;
          const uint32_t at = tmem + lanes + static_cast<uint32_t>(u & 1) * 128;
          float s[128];
          tc_ld64(s, 0, at);
          tc_ld64(s, 64, at + 64);
          if (key0 + kPrefixTile > all_see) {
            const int valid = limit - key0;
#pragma unroll
            for (int x = 0; x < 128; ++x)
              if (x >= valid) s[x] = -INFINITY;
            const int lo = all_see - key0;
#pragma unroll 1
            for (int x = max(lo, 0); x < min(len - key0, 128); ++x) {
              float y;
              tc_ld1(y, at + x);
              late[(x - lo) * 128] = x < valid ? y * cs : -INFINITY;
              late_keys |= 1u << (x - lo);
            }
          }
          float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int x = 4; x < 124; x += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) tops[k] = max3(tops[k], s[x + k], s[x + 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], s[124 + k]);
          const float top = fmaxf(__fadd_ru(fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * cs, -kPrefixLift<T>), kNoBase);
          const bool grew = first || top > base + kPrefixGrow<T>;
          if (__any_sync(~0u, grew)) {
            // the base moves: what there is so far follows it
            const float moved = grew ? top : base, shrink = exp2_fast(base - moved);
            base = moved;
            l *= shrink;
            if (!first) {
              // (64 and 128 wide this stream's last product came before these scores)
              if (S::kStreams == 1) ok = __all_sync(~0u, bar_wait(&bars.pv_done[(u - 1) & 1], static_cast<uint32_t>((u - 1) >> 1) & 1, dead));
              tc_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                float v[32];
                tc_ld(v, sums_at + d);
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] *= shrink;
                tc_st(sums_at + d, v);
              }
            }
          }
          first = false;
          float2 sums[2] = {make_float2(0, 0), make_float2(0, 0)};
          const float2 by = make_float2(cs, cs), less = make_float2(-base, -base);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t packed[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float2 e = fma2(make_float2(s[32 * k + 2 * x], s[32 * k + 2 * x + 1]), by, less);
              e.x = exp2_fast(e.x), e.y = exp2_fast(e.y);
              sums[x & 1] = add2(sums[x & 1], e);
              packed[x] = pack2<T>(e.x, e.y);
            }
            tc_st_packed(at + 16 * k, packed);  // (over scores that have been read)
          }
          sums[0] = add2(sums[0], sums[1]);
          l += sums[0].x + sums[0].y;
          tc_wait_st();
          tc_before();
          bar_arrive(&bars.p_full[u & 1]);
        }
        if (!ok) break;
        // Values of the part's keys that not all rows see, into shared memory (two turns: a warp may be an item behind).
        constexpr int kBytes = E4M3 ? 1 : 2;
        const unsigned char* late_v = smem + S::kOffLateV + (st * 2 + (late_turn & 1)) * (kGroupRows * D * 2);
        if (late_keys) {
          const int pieces = a.head_dim * kBytes / 16;
          for (int i = row; i < kGroupRows * pieces; i += S::kStreamThreads) {
            const int x = i / pieces, at = (i - x * pieces) * 16;
            if (!(late_keys >> x & 1)) continue;
            const int key = all_see + x, page = a.table[w.request() * a.table_stride + p.page(key)];
            const unsigned char* from = kZeros;
            if (page >= 0 && page < a.n_pages) from = row_at(a.v_pages, p.v_step, page, w.kv_head(), key - p.page(key) * a.page_size);
            cp16(s0 + static_cast<uint32_t>(late_v - smem) + x * D * 2 + at, from + at);
          }
          cp_arrive(&bars.late_full[st]);
        }
        // the next item's queries, whose place the last scores have left
        w.skip();
        seek();
        if (!w.ends()) load_queries(w);
        if (late_keys) {
          ok = __all_sync(~0u, bar_wait(&bars.late_full[st], late_turn & 1, dead));
          ++late_turn;
        }
        ok = __all_sync(~0u, bar_wait(&bars.pv_done[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead)) && ok;
        tc_after();
        float* out = (line == kOwn ? p.own : p.part) + at_row * D;
        const bool write = row < rows;
#pragma unroll 1
        for (int d = 0; d < a.head_dim; d += 32) {
          float v[32];
          tc_ld(v, sums_at + d);
#pragma unroll 1
          for (uint32_t left = late_keys; left; left &= left - 1) {
            const int x = __ffs(left) - 1;
            if (all_see + x >= limit) continue;
            const float f = exp2_fast(late[x * 128] - base);
            const unsigned char* from = late_v + x * D * 2 + d * kBytes;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              if (d + k >= a.head_dim) break;
              uint32_t q[4];  // eight 16-bit values
              if (E4M3) {
                const uint2 codes = *reinterpret_cast<const uint2*>(from + k);
                uint32_t lo[2], hi[2];
                e4m3_to_f16(lo, codes.x);
                e4m3_to_f16(hi, codes.y);
                q[0] = lo[0], q[1] = lo[1], q[2] = hi[0], q[3] = hi[1];
              } else {
                const uint4 y = *reinterpret_cast<const uint4*>(from + k * 2);
                q[0] = y.x, q[1] = y.y, q[2] = y.z, q[3] = y.w;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 y = unpack2<T>(q[i]);
                v[k + 2 * i] += f * y.x, v[k + 2 * i + 1] += f * y.y;
              }
            }
          }
          if (write)
#pragma unroll
            for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(out + d + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
        }
        if (write) *ml = make_float2(l == 0.0f ? -INFINITY : base, l);
        tc_before();
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (tid == 0 && *dead) flag(a.status, MK_OP_TIMEOUT);
}

template <typename T, typename QT, int D, bool E4M3>
cudaError_t launch_prefix(const PrefixParams& p, int device, cudaStream_t s) {
  constexpr auto kernel = prefix_kernel<T, QT, D, E4M3>;
  if (const cudaError_t e = allow_smem<kernel>(device, PrefixShape<D>::kSmem)) return e;
  // setmaxnreg hands out what the block was launched with; a build with less would wait for ever
  static const int regs = [] {
    cudaFuncAttributes f{};
    return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs * PrefixShape<D>::kThreads < 256 * (kSoftmaxRegs<E4M3> + kOtherRegs<E4M3>)) return cudaErrorInvalidConfiguration;
  return start(kernel, p.ctas, PrefixShape<D>::kThreads, PrefixShape<D>::kSmem, s, p);
}
template <typename T, typename QT, bool E4M3>
cudaError_t launch_prefix(const PrefixParams& p, int device, cudaStream_t s) {
  return p.dp == 64 ? launch_prefix<T, QT, 64, E4M3>(p, device, s)
         : p.dp == 128 ? launch_prefix<T, QT, 128, E4M3>(p, device, s)
                       : launch_prefix<T, QT, 256, E4M3>(p, device, s);
}
cudaError_t launch_prefix_bf16(const PrefixParams& p, int device, cudaStream_t s);
cudaError_t launch_prefix_f16(const PrefixParams& p, int device, cudaStream_t s);
cudaError_t launch_prefix_e4m3_bf16(const PrefixParams& p, int device, cudaStream_t s);
cudaError_t launch_prefix_e4m3_f16(const PrefixParams& p, int device, cudaStream_t s);

}  // namespace prefix
}  // namespace mkop
