// The kernel of mk_prefix_attention, on the 5th-generation tensor cores with accumulators in tensor memory
// (prefix_attention.cu: arguments and the join).
//
// For a kv head, every query row of every request meets the same keys of the prefix, and the rows of one request its own keys:
// scores S = Q K^T of [128 rows x 128 keys], an online softmax, sums O += P V. At rows x 2 flops a cached byte (16 bits) this
// is bound by the tensor cores from about 280 rows on, by memory below.
// - Work: 128 query rows of a kv head are a row tile. Three lines of key tiles, each cut into equal pieces, one piece a CTA:
//   pairs of row tiles over the prefix (a tile of keys and values is read once for 256 rows), single row tiles over the prefix
//   (an odd one; all of them 256 wide, where the tensor memory holds one), and row tiles of one request (of up to 8 of its
//   new rows) over its own keys. CTAs are dealt to the lines by what their tiles take, a rule on the lengths alone; an item over
//   own keys counts as four tiles more (with CTAs dealt and cut by tiles alone, 64 requests behind 32768 positions took 128 us
//   instead of 117: those with many short requests ended last).
//   Where a CTA has one row tile, even and odd key tiles go to two sets of sums, so that there are two streams of work
//   in any case (one 256 wide).
// - Units: the product of one row tile and one key tile. A warp for each stream issues S of its first unit, then for each
//   unit O += P V and S of the next: while one stream's softmax runs, the tensor cores work on the other. (256 wide: one
//   stream with two score buffers, S two units ahead.)
// - Softmax: a thread has a row (128 threads a stream), so nothing is exchanged; its 128 scores are in registers at once.
//   Probabilities go back to tensor memory over the first half of the scores' columns as the product's operand (16 bits).
//   They are taken against a base that moves only when a score passes it by kPrefixGrow: else sums stay as they are.
// - Loads: warps for keys and for values copy boxes of a page's rows (TMA, through the page table) into a ring of slots
//   each; a copy takes its warp 140 cycles, so the two 64-column pieces of a tile have a warp each. A box has as many rows as the largest
//   power of two that divides the page size: 8 and more copy a tile of 16 or fewer boxes while another is worked on, but
//   pages of one position (or of an odd number) take 128 boxes a tile, 18 thousand cycles (32 x 8 rows behind 8191 in pages of 8 and more 87
//   to 89 us, 4: 97, 2: 136, 1: 220, 25: 209). Over own keys few query rows
//   leave room for a third tile, which memory's latency under load asks for. (Prefetches into L2 by warps of their own
//   made it slower, 169 us against 127 for the 64 requests below.) Codes of e4m3 caches land in the half of their slot where two
//   warps each make fp16 of them in place (through stages of 64 rows of their own, half as many bytes were on their way: 65536
//   positions 175 us instead of 154). Queries are stored by the softmax threads, an item ahead where there is room for two.
// - Keys that not every row of a request's tile sees (at most 7) have probability 0 in the others. Should their values hold an
//   infinity or NaN (0 times that is NaN), they are left out of the product and added one by one by the rows that see them.
// Probabilities are one 16-bit number (a pair hi + lo would be half as much work again for the tensor cores). bf16: 2^-8 of each
// at most; fp16: 2^-11, against a base 14 under the maximum, so that what falls under its range is 2^-39 of the largest. Sums of
// probabilities are those of the unrounded ones.
// Measured: 64 requests behind 32768 positions with own ones of up to 2000 (48/8 heads of 128, bf16) 112 us, 32 x 8 rows behind
// 8191 90 us (610 TFLOP/s), 64 requests behind 65536 in e4m3 155 us (670 TFLOP/s), 4 samples of 4096 positions 256 wide 25 us. A pair's
// tile takes about 3500 cycles, 2048 of them the tensor cores' (75 % of the rate measured for large products); its chain of products, scores out
// of tensor memory, softmax and probabilities back takes 400 less with almost all products left out and 200 less without exponentials.
// Further from their bounds are single row tiles (71 to 75 % of a pair's time for half of its work), the steps between own items, and what is
// outside of the tiles: 32 x 8 rows are 51 us of tiles and items, 21 of starting, ending and uneven pieces, 15 of the join.
// Every wait has a limit (2 s), after which the CTA gives up, drains and frees what it holds and MK_OP_TIMEOUT is set.
#pragma once
#include <cuda.h>

#include "paged_attention_tc.cuh"

namespace mkop {
namespace prefix {

using namespace attn;

// a * b / c, in 32 bits where that holds the product (a division in 64 bits takes some hundred cycles)
__device__ inline long long scaled(long long a, long long b, long long c) {
  const unsigned long long ab = static_cast<unsigned long long>(a) * b;
  return (ab | c) >> 32 ? static_cast<long long>(ab / c) : static_cast<uint32_t>(ab) / static_cast<uint32_t>(c);
}

constexpr int kPrefixTile = 128;      // keys
constexpr int kTileRows = 128;        // query rows of a row tile
constexpr int kGroupRows = 8;         // new rows of a request that share an item over its own keys
constexpr int kItemTiles = 4;         // what an item over own keys takes besides its tiles, in tiles
enum { kPairs, kSingles, kOwn };      // the lines
// What a tile of a line takes of a CTA, in parts of 24 of a pair's (64 and 256 wide are dealt by the same numbers, without measurements of their
// own): as measured 128 wide, where a pair's tile takes 1.8 to 2.1 us, a single
// one 1.3 to 1.4, one of an item (with its share of the four for the item) 1.0 to 1.2. 64 requests behind 32768 positions and 32 x 8 rows
// behind 8191 take 113 and 91 us; with 24 / 18 / 18 122 and 90, with two tiles an item and 24 / 18 / 18 116 and 95, with 24 / 24 / 24 136
// and 95; e4m3 behind 65536 155, with 24 / 16 / 20 161.
template <bool E4M3>
constexpr int kLineCost[3] = {24, E4M3 ? 17 : 18, E4M3 ? 16 : 14};

// What the first CTA writes for the join. Piece c's part of item i of a line goes to place c + i (after `place0`): along the line
// either grows by one from part to part.
struct Head {
  long long total[3];  // key tiles of a line; over own keys with kItemTiles before each item's
  int used[3];         // its pieces
  int tiles;           // key tiles of the prefix
  __device__ static int piece_of(long long x, long long total, int used) {  // the last piece that begins at or before tile x
    const unsigned long long n = static_cast<unsigned long long>(x + 1) * used - 1;
    return static_cast<int>((n | total) >> 32 ? n / total : static_cast<uint32_t>(n) / static_cast<uint32_t>(total));
  }
};

struct PrefixParams {
  mk_prefix_attention_args a;
  Div page, group_div, row_div, q_head_div, block_div[3], groups_div;
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
  float* part;        // [places][streams][128][dp] sums of a part over the prefix (on 32 bytes, as `own`)
  float2* part_ml;    // [places][streams][128] its base (log2 units) and sum of probabilities; sum 0: an empty part, sums not written
  float* own;         // [places][streams][own_rows][dp] and
  float2* own_ml;     // [places][streams][own_rows] over own keys
  Head* head;
  long long* cum;     // [batch * groups + 1] as total[kOwn], of the row groups so far (of one row tile)
  int box;            // rows of a copied box: the largest power of two that divides the page size, up to a tile
  CUtensorMap keys, values;  // [n_pages][n_kv_heads][page_size][head_dim]
  __device__ int first_single() const { return blocks[kPairs] * 2 * kTileRows; }
  __device__ int rows_of(int group_index) const { return min(kGroupRows, a.rows - group_index * kGroupRows); }
  // Own keys of a row group: those its last row sees.
  __device__ int own_len(int bg) const {
    const int b = groups_div(bg), g = bg - b * groups;
    return max(0, min(max(a.lens[b], 0), max_own) - (a.rows - g * kGroupRows - rows_of(g)));
  }
  __device__ static int tiles_of(int len) { return (len + kPrefixTile - 1) >> 7; }
  __device__ static int with_item(int n) { return n ? n + kItemTiles : 0; }
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
  __device__ int kv_head() const { return p.block_div[line](hm); }
  __device__ int block() const { return hm - kv_head() * p.blocks[line]; }
  __device__ int request() const { return p.groups_div(bg); }
  __device__ int group_rows() const { return p.rows_of(bg - request() * p.groups); }
  __device__ int all_see() const { return line == kOwn ? len - (group_rows() - 1) : len; }  // keys before it are seen by every row
};

template <int D, bool E4M3>
struct PrefixShape {
  static constexpr int kThreads = 512, kStreamThreads = 128;
  // Registers of a thread after the launch's 128: the softmax's 256 threads and the others
  static constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= 65536 / kThreads / 8 * 8 * kThreads, "of those launched with");
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kHalves = D == 256 ? 2 : 1;          // slots of a tile's keys
  static constexpr int kWide = D == 256 ? 128 : D;          // columns of a slot
  static constexpr int kPieces = kWide / 64;                // of 64 columns: [128 rows][128 bytes] each
  static constexpr int kSlot = kPrefixTile * kWide * 2;
  static constexpr int kKeySlots = E4M3 ? 3 : D == 64 ? 4 : 2, kValueSlots = D != 64 ? 2 : E4M3 ? 3 : 4;
  static constexpr int kConverters = 64;                    // threads, of keys and of values
  // Codes of a tile arrive in the second half of their slot, where their row of fp16 values goes; 64 wide, in places of their own.
  static constexpr bool kInPlace = E4M3 && kWide == 128;
  static constexpr int kCodes = kPrefixTile * 128;          // rows of 128 bytes (zeros behind a head's columns)
  static constexpr int kQ = kTileRows * D * 2;              // a stream's queries
  // Queries, keys' slots, values' slots. 128 wide, 16 bits, items of up to 64 or 32 rows: 5 or 6 slots and queries twice. (Lines over the
  // prefix leave the seventh 32 KB empty.)
  static constexpr bool kFewRows = D == 128 && !E4M3;
  static constexpr int kOffCodes = kFewRows ? 7 * kSlot : (kKeySlots + kValueSlots) * kSlot + kStreams * kQ;  // [keys, values][slots]
  static constexpr int kOffBar = kOffCodes + (E4M3 && !kInPlace ? (kKeySlots + kValueSlots) * kCodes : 0);
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// What scores are taken times. A score of -infinity stays one where the scale is 0; NaN stays NaN.
__device__ inline float score_scale(float x) { return x < 1.17549435e-38f ? 1.17549435e-38f : x; }

template <typename T>
constexpr float kPrefixLift = std::is_same<T, __half>::value ? 14.0f : 0.0f;  // the base is this much under the maximum
template <typename T>
constexpr float kPrefixGrow = std::is_same<T, __half>::value ? 1.0f : 8.0f;   // and moves when a score passes that by this

// A place in a ring of slots and its barriers. There are as many barriers as slots, or twice as many where that is an odd number: two
// streams use tiles in turn, and a stream that waits for every other turn of a barrier could not tell the one it waits
// for from the one before the last.
struct Ring {
  uint32_t slots, bars, slot, bar, phase;
  __device__ explicit Ring(uint32_t n) : slots(n), bars(n & 1 ? 2 * n : n), slot(0), bar(0), phase(0) {}
  __device__ void next() {
    if (++slot == slots) slot = 0;
    if (++bar == bars) bar = 0, phase ^= 1;
  }
};

struct PrefixBars {
  uint64_t key_full[6], key_empty[6], value_full[6], value_empty[6], codes_full[12];
  uint64_t q_full[4], s_full[2], p_full[2], pv_done[2], issued[2], tail[2], drained;
  uint32_t tmem;
  int dead;
  alignas(4) uint8_t slow[16][4];  // of key tile j % 16, if not all rows see all of it: whether values are left out of a part of the product
  uint8_t since[16];  // of key tile j % 16: how many of its item's tiles come before it in this piece (2: two and more)
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
__device__ inline void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
// One box into shared memory; what lies outside of the tensor is written as zeros.
__device__ inline void copy_box(uint32_t to, const CUtensorMap* map, int column, int place, int head, int page, uint64_t* bar, uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], "
               "[%6], %7;" ::"r"(to), "l"(map), "r"(column), "r"(place), "r"(head), "r"(page), "r"(smem_u32(bar)), "l"(policy) : "memory");
}
// 64 consecutive fp32 columns of this warp's 32 lanes into v[at ..], and a lane's largest. Load and wait are one statement: before
// the wait the registers do not hold the values.
__device__ inline float tc_ld64_max(float (&v)[128], int at, uint32_t addr) {
  uint32_t r[64];
  float largest;
  asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
               "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,"
               "%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, %64, [%65];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
                 "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
                 "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
                 "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
                 "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]),
                 "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]),
                 "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]), "=&r"(r[54]), "=&r"(r[55]),
                 "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]), "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63]),
                 "=&f"(largest)
               : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[at + i] = __uint_as_float(r[i]);
  return largest;
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
// Whether one of a pair of 16-bit values is an infinity or NaN
template <typename T>
__device__ inline bool not_finite(uint32_t pair) {
  constexpr uint32_t kMask = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (pair & kMask) == kMask || (pair >> 16 & kMask) == kMask;
}
// Instruction descriptor: fp32 sums, 16-bit operands, M = 128; `turned`: B is N-major
template <typename T>
__device__ constexpr uint32_t prefix_idesc(int n, bool turned) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (turned ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

// Element d of a cached row.
template <typename T, bool E4M3>
__device__ inline float cached(const unsigned char* row, int d) {
  if (!E4M3) return static_cast<float>(reinterpret_cast<const T*>(row)[d]);
  uint32_t f[2];
  e4m3_to_f16(f, row[d]);
  return unpack2<__half>(f[0]).x;
}

// T: the products' type; QT: the queries'; E4M3: the cache holds codes (T is __half then)
template <typename T, typename QT, int D, bool E4M3>
__global__ void __launch_bounds__(PrefixShape<D, E4M3>::kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
  using S = PrefixShape<D, E4M3>;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  const uint32_t s0 = smem_u32(smem);
  const mk_prefix_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = of_warp(tid >> 5);
  PrefixBars& bars = *reinterpret_cast<PrefixBars*>(smem + S::kOffBar);
  volatile int* dead = &bars.dead;
  __shared__ long long warp_tiles[2][S::kThreads / 32];
  __shared__ struct {
    long long tiles[2];  // over own keys: this piece's tiles among all, its first and behind its last
    int bg, hm, tile;    // and where the first is
  } ends;

  // ---- the lines, and this CTA's piece of one -------------------------------------------------------------------------
  Head hd;
  int line, c = blockIdx.x;
  long long begin;
  const int n_groups = a.batch * p.groups, per = a.n_kv_heads * p.blocks[kOwn];
  const int prefix_len = min(max(a.prefix_len[0], 0), p.max_prefix);
  {
    const int each = (n_groups + S::kThreads - 1) / S::kThreads;
    const int g0 = min(n_groups, tid * each), g1 = min(n_groups, g0 + each);
    // [0] tiles, [1] with what the items take
    long long mine[2] = {}, before[2], own[2] = {};
    for (int g = g0; g < g1; ++g) {
      const int n = PrefixParams::tiles_of(p.own_len(g));
      mine[0] += n, mine[1] += PrefixParams::with_item(n);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      before[i] = mine[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, before[i], d);
        if (lane >= d) before[i] += o;
      }
      if (lane == 31) warp_tiles[i][warp] = before[i];
      before[i] -= mine[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      for (int w = 0; w < S::kThreads / 32; ++w) {
        if (w < warp) before[i] += warp_tiles[i][w];
        own[i] += warp_tiles[i][w];
      }
    hd.tiles = PrefixParams::tiles_of(prefix_len);
    hd.total[kPairs] = static_cast<long long>(a.n_kv_heads) * p.blocks[kPairs] * hd.tiles;
    hd.total[kSingles] = static_cast<long long>(a.n_kv_heads) * p.blocks[kSingles] * hd.tiles;
    hd.total[kOwn] = own[1] * per;
    // A line's CTAs: in proportion to what its tiles take, one at least.
    const int ctas = gridDim.x;
    const long long cost[3] = {kLineCost<E4M3>[0] * hd.total[0], kLineCost<E4M3>[1] * hd.total[1], kLineCost<E4M3>[2] * hd.total[2]};
    const long long sum = cost[0] + cost[1] + cost[2];
    int n0 = cost[0] ? max(1, static_cast<int>(scaled(cost[0], ctas, sum))) : 0;
    int n1 = cost[1] ? max(1, static_cast<int>(scaled(cost[1], ctas, sum))) : 0;
    const int most = ctas - (cost[2] ? 1 : 0);
    if (n0 + n1 > most) (n0 > n1 ? n0 : n1) -= n0 + n1 - most;
    if (!cost[2]) (cost[1] ? n1 : n0) += most - n0 - n1;
    const int got[3] = {n0, n1, ctas - n0 - n1};
#pragma unroll
    for (int i = 0; i < 3; ++i) hd.used[i] = static_cast<int>(hd.total[i] < got[i] ? hd.total[i] : got[i]);
    line = c < n0 ? kPairs : c < n0 + n1 ? kSingles : kOwn;
    c -= line == kPairs ? 0 : line == kSingles ? n0 : n0 + n1;
    begin = hd.used[line] ? scaled(c, hd.total[line], hd.used[line]) : 0;  // (as piece_of() has it)
    if (blockIdx.x == 0) {
      if (tid == 0) {
        *p.head = hd;
        p.cum[n_groups] = own[1];
        if (prefix_len != a.prefix_len[0]) flag(a.status, MK_OP_BAD_LENGTH);
      }
      long long at = before[1];
      for (int g = g0; g < g1; ++g) {
        p.cum[g] = at;
        at += PrefixParams::with_item(PrefixParams::tiles_of(p.own_len(g)));
        const int b = p.groups_div(g);
        if (a.lens[b] < 0 || a.lens[b] > p.max_own) flag(a.status, MK_OP_BAD_LENGTH);
      }
    }
    if (line == kOwn && c < hd.used[kOwn]) {
      // the first tile at or behind where the piece begins, and that where the next does
      const long long to = scaled(c + 1, hd.total[kOwn], hd.used[kOwn]);
      if (tid == 0 && to == hd.total[kOwn]) ends.tiles[1] = own[0] * per;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const long long x = e ? to : begin;
        if (x < before[1] * per || x >= (before[1] + mine[1]) * per) continue;
        long long tiles = before[0], at = before[1];
        for (int g = g0; g < g1; ++g) {
          const int n = PrefixParams::tiles_of(p.own_len(g)), all = PrefixParams::with_item(n);
          if (x < (at + all) * per) {
            const int hm = static_cast<int>(scaled(x - at * per, 1, all));
            const int tile = max(0, static_cast<int>(x - at * per - static_cast<long long>(hm) * all) - kItemTiles);
            ends.tiles[e] = tiles * per + static_cast<long long>(hm) * n + tile;
            if (!e) ends.bg = g, ends.hm = hm, ends.tile = tile;
            break;
          }
          tiles += n, at += all;
        }
      }
    }
  }
  if (c >= hd.used[line]) return;
  if (line == kOwn) {
    __syncthreads();
    if (ends.tiles[0] == ends.tiles[1]) return;  // (a piece of nothing but what an item takes besides its tiles)
  }
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      bar_init(&bars.key_full[i], E4M3 ? S::kConverters : S::kPieces), bar_init(&bars.key_empty[i], line == kPairs ? 2 : 1);
      bar_init(&bars.value_full[i], E4M3 ? S::kConverters : S::kPieces), bar_init(&bars.value_empty[i], line == kPairs ? 2 : 1);
    }
    for (int i = 0; i < 12; ++i) bar_init(&bars.codes_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.q_full[i], S::kStreamThreads), bar_init(&bars.q_full[2 + i], S::kStreamThreads), bar_init(&bars.s_full[i], 1);
      bar_init(&bars.p_full[i], S::kStreamThreads), bar_init(&bars.pv_done[i], 1), bar_init(&bars.issued[i], 1);
      bar_init(&bars.tail[i], E4M3 ? 2 : 1);
    }
    bar_init(&bars.drained, S::kStreams);
    bars.dead = 0;
    for (auto& x : bars.slow) *reinterpret_cast<uint32_t*>(x) = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = bars.tmem;
  const bool pair = line == kPairs;
  // how shared memory is dealt
  const int few = S::kFewRows && line == kOwn ? p.own_rows <= 32 ? 32 : p.own_rows <= 64 ? 64 : 0 : 0;
  const int q_rows = few ? few : kTileRows, key_slots = few ? 3 : S::kKeySlots, value_slots = few == 32 ? 3 : S::kValueSlots;
  // A stream's queries: [q_turns][columns / 64][q_rows][128 bytes]. They come first: a product reads 128 rows of a piece, and what it reads
  // behind fewer (rows that nothing is done with) has to be the CTA's memory, here slots.
  const uint32_t q_turns = few ? 2 : 1, q_bytes = q_rows * D * 2, at_q = s0, at_k = s0 + S::kStreams * q_turns * q_bytes;
  const uint32_t at_v = at_k + key_slots * S::kSlot;
  // key tiles of this piece
  const long long count = line == kOwn ? ends.tiles[1] - ends.tiles[0] : scaled(c + 1, hd.total[line], hd.used[line]) - begin;
  auto walk = [&]() -> PrefixWalk {
    PrefixWalk w{p, line, per, 0, 0, 0, prefix_len, hd.tiles, 0, 0, count};
    if (line == kOwn) {
      w.bg = ends.bg;
      w.len = p.own_len(w.bg);
      w.n = PrefixParams::tiles_of(w.len);
      w.hm = ends.hm;
      w.tile = ends.tile;
      w.item = static_cast<long long>(w.bg) * per + w.hm;
    } else {
      w.item = scaled(begin, 1, hd.tiles);
      w.tile = static_cast<int>(begin - w.item * hd.tiles);
      w.hm = static_cast<int>(w.item);
    }
    return w;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
    constexpr int kSecondIssuer = E4M3 ? 15 : 11;
    const bool loader = E4M3 ? warp == 9 || warp == 10 : warp == 9 || warp == 12 || (S::kPieces == 2 && (warp == 10 || warp == 13));
    if (loader) {
      // ---- loaders: keys, values --------------------------------------------------------------------------------------
      const bool value = E4M3 ? warp == 10 : warp >= 12;
      const int piece = E4M3 ? 0 : warp - (value ? 12 : 9);  // 64 columns of a slot's
      uint64_t* full = E4M3 ? bars.codes_full + 6 * value : value ? bars.value_full : bars.key_full;
      uint64_t* empty = value ? bars.value_empty : bars.key_empty;
      Ring ring(value ? value_slots : key_slots), freed = ring;
      // a slot, or its codes
      const uint32_t base = E4M3 && !S::kInPlace ? s0 + S::kOffCodes + value * S::kKeySlots * S::kCodes
                                                 : (value ? at_v : at_k) + (E4M3 ? S::kSlot / 2 : 0);
      constexpr uint32_t kBytes = E4M3 && !S::kInPlace ? S::kCodes : S::kSlot;
      const CUtensorMap* map = value ? &p.values : &p.keys;
      const int box = of_warp(p.box);
      // Own keys are read once: the prefix keeps its place in L2 (64 requests behind 32768 positions 120.6 -> 118.2 us, 32 x 8 rows 95.5 ->
      // 93.0).
      uint64_t policy;
      if (line == kOwn) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      PrefixWalk w = walk();
      long long since = 0;
      uint32_t turn = 0, tails = 0;
      bool ok = true;
      // The pages of 32 boxes of walk w's tile, one a lane, looked up a tile ahead. (A copy of many lanes is issued as one each, 140
      // cycles; by one lane with operands handed over it took 440.)
      auto pages_from = [&](int first) -> int {
        const int at = (first + lane) * box, key = w.tile * kPrefixTile + at;
        if (at >= kPrefixTile || key >= w.len) return -1;
        return line == kOwn ? a.table[w.request() * a.table_stride + p.page(key)] : a.prefix_table[p.page(key)];
      };
      int page = pages_from(0), held = 0;
      for (long long j = 0; ok && j < count; ++j) {
        const int key0 = of_warp(w.tile * kPrefixTile), head = of_warp(w.kv_head()), len = of_warp(w.len), all_see = w.all_see();
        const bool tail = !E4M3 && value && key0 + kPrefixTile > all_see;
        const long long item = w.item;
#pragma unroll 1
        for (int h = 0; ok && h < S::kHalves; ++h) {
          if (turn >= ring.slots) {
            ok = __all_sync(~0u, bar_wait(&empty[freed.bar], freed.phase, dead));
            freed.next();
          }
          if (!ok) break;
          ++turn;
          const int end = min(len - key0, kPrefixTile);  // rows with keys
          uint64_t* bar = tail ? &bars.tail[piece] : &full[ring.bar];
          if (lane == 0) {
            if (!E4M3 && !value && piece == 0) bars.since[j & 15] = static_cast<uint8_t>(since);
            bar_expect(bar, max((end + box - 1) / box, 0) * box * 128);
          }
          __syncwarp();
          const uint32_t to = base + ring.slot * kBytes + piece * (kPrefixTile * 128);
#pragma unroll 1
          for (int i = 0; i * box < end; i += 32) {
            if (held != i) held = i, page = pages_from(i);
            const int row = (i + lane) * box, key = key0 + row;
            if (row >= end) continue;
            int id = page;
            if (id < 0 || id >= a.n_pages) {
              flag(a.status, MK_OP_BAD_PAGE);
              id = a.n_pages;  // outside of the tensor: zeros
            }
            copy_box(to + row * 128, map, h * S::kWide + piece * 64, key - p.page(key) * a.page_size, head, id, bar, policy);
          }
          __syncwarp();
          if (tail) {
            // Rows that are not there have to be zeros (0 times what they hold may be NaN), and so those that not every row sees,
            // if they hold such values.
            ok = __all_sync(~0u, bar_wait(bar, tails++ & 1, dead));
            uint4* at = reinterpret_cast<uint4*>(smem + (to - s0));  // 8 a row
            bool bad = false;
#pragma unroll 1
            for (int i = max(all_see - key0, 0) * 8 + lane; i < end * 8; i += 32) {
              const uint4 x = at[i];
              bad |= not_finite<T>(x.x) || not_finite<T>(x.y) || not_finite<T>(x.z) || not_finite<T>(x.w);
            }
            bad = __any_sync(~0u, bad);
            if (lane == 0) bars.slow[j & 15][h * 2 + piece] = bad;
#pragma unroll 1
            for (int i = (bad ? max(all_see - key0, 0) : end) * 8 + lane; i < kPrefixTile * 8; i += 32) at[i] = make_uint4(0, 0, 0, 0);
            proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(&full[ring.bar]);
          }
          ring.next();
        }
        w.next();
        since = w.item != item ? 0 : min(since + 1, 2ll);
        if (!w.ends()) page = pages_from(0), held = 0;
      }
      // What has been asked for lands before the CTA's memory goes: the last turns, from the oldest one on.
      int alive = 0;
      for (uint32_t i = 0; i < min(turn, ring.slots); ++i, freed.next()) bar_wait(&full[freed.bar], freed.phase, &alive);
    } else if (E4M3 && warp >= 11 && warp < 15) {
      // ---- converters: a tile's codes become its slot's fp16 values -------------------------------------------------------
      const bool value = warp >= 13;
      const int t = tid - (value ? 416 : 352);
      Ring ring(value ? value_slots : key_slots);
      uint64_t* full = value ? bars.value_full : bars.key_full;
      PrefixWalk w = walk();
      long long since = 0;
      bool ok = true;
      uint32_t tails = 0;
      // Four lanes have a row: each 16 of its first 64 codes and, 128 wide, 16 of its second. In place a row's codes lie where its
      // second 64 values go, so they are all read before any is written.
      constexpr int kLanes = 4, kStep = S::kConverters / kLanes, kSets = S::kWide / 64;
      const int chunk = t % kLanes, row0 = t / kLanes;
      for (long long j = 0; ok && j < count; ++j) {
        const int key0 = w.tile * kPrefixTile;
        const int all_see = w.all_see() - key0, end = w.len - key0;
#pragma unroll 1
        for (int h = 0; ok && h < S::kHalves; ++h) {
          unsigned char* slot = smem + ((value ? at_v : at_k) - s0) + ring.slot * S::kSlot;
          const unsigned char* codes = S::kInPlace ? slot + S::kSlot / 2
                                                   : smem + S::kOffCodes + (value * S::kKeySlots + ring.slot) * S::kCodes;
          ok = __all_sync(~0u, bar_wait(&bars.codes_full[6 * value + ring.bar], ring.phase, dead));
          if (!ok) break;
          int live = value ? end : kPrefixTile;  // rows from there on are zeros (see the loaders; each warp looks at all of them)
          if (value && all_see < end && all_see < kPrefixTile) {
            const int first = max(all_see, 0), last = min(end, kPrefixTile);
            bool bad = false;
            for (int i = first * 32 + lane; i < last * 32; i += 32) {  // four codes
              const uint32_t x = *reinterpret_cast<const uint32_t*>(codes + i * 4);
#pragma unroll
              for (int k = 0; k < 32; k += 8) bad |= (x >> k & 0x7f) == 0x7f && (i & 31) * 4 + k / 8 < a.head_dim - h * S::kWide;
            }
            bad = __any_sync(~0u, bad);
            if (bad) live = all_see;
            if (t == 0) bars.slow[j & 15][h * 2] = bars.slow[j & 15][h * 2 + 1] = bad;
            // both warps have looked before either's rows change
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.tail[0]);
            ok = __all_sync(~0u, bar_wait(&bars.tail[0], tails++ & 1, dead));
            if (!ok) break;
          }
#pragma unroll 2
          for (int i = 0; i < kPrefixTile / kStep; ++i) {
            const int row = row0 + i * kStep;
            uint4 x[kSets];
            // (of odd rows the second 64 codes first: so 8 lanes have 32 banks)
            const int turned = kSets == 2 ? row & 1 : 0;
#pragma unroll
            for (int k = 0; k < kSets; ++k) {
              x[k] = *reinterpret_cast<const uint4*>(codes + row * 128 + (k ^ turned) * 64 + chunk * 16);
              if (row >= live) x[k] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kSets; ++k) {
              const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
              unsigned char* to = slot + (k ^ turned) * (kPrefixTile * 128) + row * 128;
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint32_t lo[2], hi[2];
                e4m3_to_f16(lo, v[2 * g]);
                e4m3_to_f16(hi, v[2 * g + 1]);
                *reinterpret_cast<uint4*>(to + (((2 * chunk + g) ^ row) & 7) * 16) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
              }
            }
          }
          if (!value && h == 0 && t == 0) bars.since[j & 15] = static_cast<uint8_t>(since);
          proxy_fence();
          bar_arrive(&full[ring.bar]);
          ring.next();
        }
        const long long item = w.item;
        w.next();
        since = w.item != item ? 0 : min(since + 1, 2ll);
      }
    } else if (warp == 8 || (S::kStreams == 2 && warp == kSecondIssuer)) {
      // ---- the warps that issue the products, one for each stream ---------------------------------------------------------
      // All lanes walk and wait together, on values that are the warp's; one issues. (Under a branch of one lane, on values of
      // that lane, a product took 130 cycles to issue; one warp for both streams left the tensor cores idle for 700 cycles of
      // 1850 while it waited and looked for the next unit.)
      constexpr uint32_t kScores = prefix_idesc<T>(kPrefixTile, false), kSums = prefix_idesc<T>(S::kWide, true);
      constexpr bool kOneStream = S::kStreams == 1;
      constexpr uint32_t kAhead = kOneStream ? 2 : 1;  // score buffers of a stream
      const uint32_t st = warp == 8 ? 0 : 1;
      const int steps = a.head_dim / 16;
      const uint32_t tm = of_warp(tmem), base_q = of_warp(at_q + st * q_turns * q_bytes), base_k = of_warp(at_k), base_v = of_warp(at_v);
      const uint32_t q_piece = of_warp(q_rows * 128);
      const long long units = pair || kOneStream ? count : (count + 1 - st) / 2;
      // this stream's next tile of keys and of values; single tiles go to two streams in turn
      Ring keys(of_warp(key_slots)), values(of_warp(value_slots));
      const bool every = pair || kOneStream;
      uint32_t key_tile = st;  // (where since[] has the next tile of keys)
      if (every) key_tile = 0;
      else if (st) keys.next(), values.next();
      uint32_t q_turn = 0;  // items so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!__all_sync(~0u, bar_try(bar, parity))) ok = __all_sync(~0u, ok && bar_wait(bar, parity, dead));
      };
      // (numbers of units wrap: parities are all that is used of them)
      auto buffer_of = [&](uint32_t i) { return kOneStream ? i & 1 : st; };
      auto turn_of = [&](uint32_t i) { return kOneStream ? i >> 1 & 1 : i & 1; };  // its parity
      // Waits for the next tile of keys. Returns whether its unit is the stream's first of an item: the tile is the item's first, or,
      // of single tiles in two streams, the second.
      auto keys_there = [&]() -> bool {
        wait(&bars.key_full[keys.bar], keys.phase);
        if (S::kHalves == 2) {
          Ring second = keys;
          second.next();
          wait(&bars.key_full[second.bar], second.phase);
        }
        return of_warp(bars.since[key_tile & 15]) < (every ? 1 : 2);
      };
      auto queries = [&]() {
        const uint32_t buffer = q_turns == 2 ? q_turn & 1 : 0;
        wait(&bars.q_full[st * 2 + buffer], (q_turns == 2 ? q_turn >> 1 : q_turn) & 1);
        ++q_turn;
        if (!E4M3) proxy_fence();  // (their copies' writes are ordinary ones)
      };
      auto next_keys = [&]() {
        for (int h = 0; h < S::kHalves; ++h) keys.next();
        ++key_tile;
        if (!every) keys.next(), ++key_tile;
      };
      // By one lane: a unit's scores from the next tile of keys.
      auto scores = [&](uint32_t i) {
        Ring r = keys;
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h, r.next()) {
          const uint64_t kd = tc_desc(base_k + r.slot * S::kSlot, 16);
          const uint64_t qd = tc_desc(base_q + (q_turns == 2 && !(q_turn & 1) ? q_bytes : 0) + 2 * h * q_piece, 16);
#pragma unroll
          for (int k = 0; k < S::kWide / 16; ++k)
            if (h * 8 + k < steps)
              tc_mma(tm + buffer_of(i) * 128, qd + ((k >> 2) * q_piece + (k & 3) * 32) / 16,
                     kd + ((k >> 2) * (kPrefixTile * 128) + (k & 3) * 32) / 16, kScores, h > 0 || k > 0);
          tc_commit(&bars.key_empty[r.bar]);
        }
        tc_commit(&bars.s_full[buffer_of(i)]);
      };
      uint32_t firsts = 0;  // bit i % 2: unit i is the first of an item
      for (uint32_t i = 0; i < kAhead && i < units && ok; ++i) {
        if (keys_there()) {
          firsts |= 1u << i;
          queries();
        }
        tc_after();
        if (ok && elected()) scores(i);
        __syncwarp();
        next_keys();
      }
      long long left = units;
      for (uint32_t i = 0; left > 0 && ok; ++i, --left) {
        const bool fresh = firsts >> (i & 1) & 1, more = left > kAhead;
        // The next scores' keys are waited for before these sums are issued, so that both run without a pause; not so
        // the first of another item, whose queries come after this unit's probabilities.
        bool same = more;
        if (more) {
          same = !keys_there();
          const uint32_t bit = 1u << ((i + kAhead) & 1);
          firsts = same ? firsts & ~bit : firsts | bit;
        }
        {
          Ring r = values;
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h, r.next()) wait(&bars.value_full[r.bar], r.phase);
        }
        wait(&bars.p_full[buffer_of(i)], turn_of(i));
        // The streams take turns, so that one's softmax runs while the other's products do (both at once is as stable a state, and a
        // third slower: the products of both, then the softmax of both).
        if (!kOneStream && (st || i)) wait(&bars.issued[st ^ 1], (st ? i : i - 1) & 1);
        if (!ok) break;
        tc_after();
        if (elected()) {
          Ring r = values;
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h, r.next()) {
            const uint64_t vd = tc_desc(base_v + r.slot * S::kSlot, kPrefixTile * 128);
#pragma unroll
            for (int k = 0; k < kPrefixTile / 16; ++k)
              tc_mma_ts(tm + 256 + st * D + h * 128, tm + buffer_of(i) * 128 + k * 8, vd + k * 2048 / 16, kSums, !fresh || k > 0);
            tc_commit(&bars.value_empty[r.bar]);
          }
          tc_commit(&bars.pv_done[buffer_of(i)]);
          // (these scores go where the probabilities were: the products run in the order of their issue)
          if (same) scores(i + kAhead);
          if (!kOneStream) bar_arrive(&bars.issued[st]);
        }
        __syncwarp();
        if (more && !same) {
          queries();
          tc_after();
          if (ok && elected()) scores(i + kAhead);
          __syncwarp();
        }
        if (more) next_keys();
        for (int h = 0; h < S::kHalves; ++h) values.next();
        if (!every) values.next();
      }
      // every product has ended before the tensor memory is freed, also when the CTA gave up
      if (elected()) tc_commit(&bars.drained);
      int alive = 0;
      bar_wait(&bars.drained, 0, &alive);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    if (warp < 4 * S::kStreams) {
      // ---- softmax: a thread has a row of the stream's row tile -------------------------------------------------------
      const int st = warp >> 2, row = tid & 127;
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
      const uint32_t sums_at = tmem + lanes + 256 + static_cast<uint32_t>(st) * D;
      float cs = score_scale(p.scale_log2);
      float next_cs = cs;  // of the queries loaded last
      // Where this thread's row of an item's queries is, in elements; -1: the item has fewer rows.
      auto query_at = [&](const PrefixWalk& w) -> long long {
        const int head = w.kv_head();
        if (line == kOwn) {
          const int m = w.block() * kTileRows + row, q = p.group_div(m), b = w.request();
          if (q >= w.group_rows()) return -1;
          return b * a.q_stride[0] + ((w.bg - b * p.groups) * kGroupRows + q) * a.q_stride[1] + (head * p.group + m - q * p.group) * a.q_stride[2];
        }
        const int m = pair ? (2 * w.block() + st) * kTileRows + row : p.first_single() + w.block() * kTileRows + row;
        if (m >= p.n_rows) return -1;
        const int br = p.group_div(m), h = head * p.group + m - br * p.group, b = p.row_div(br), qr = br - b * a.rows;
        return b * a.q_stride[0] + qr * a.q_stride[1] + h * a.q_stride[2];
      };
      // A warp's 32 rows of an item's queries on their way into shared memory: a lane makes the address of its own row, D / 8 lanes
      // copy one.
      uint32_t q_turn = 0;
      auto load_queries = [&](const PrefixWalk& w) {
        const long long mine = query_at(w);
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 4;
        const int chunk = lane % kLanes, sub = lane / kLanes;
        const bool in = chunk * 8 < a.head_dim;
        const uint32_t buffer = q_turns == 2 ? q_turn & 1 : 0;
        const uint32_t to = at_q + (st * q_turns + buffer) * q_bytes + (chunk >> 3) * 128 * q_rows;
        uint64_t* bar = &bars.q_full[st * 2 + buffer];
        ++q_turn;
        const QT* q = static_cast<const QT*>(a.q);
        if (!E4M3) {
          // (rows that are not there are not written: nothing is done with what the products make of them)
          const int n = __popc(__ballot_sync(~0u, mine != -1));
#pragma unroll 2
            for (int i = 0; i * kRows < n; ++i) {
              const long long off = __shfl_sync(~0u, mine, i * kRows + sub);
              const int r = (row & ~31) + i * kRows + sub;
              cp16(to + r * 128 + (((chunk ^ r) & 7) << 4), off == -1 || !in ? q : q + off + chunk * 8, off != -1 && in);
            }
          cp_arrive(bar);
          return;
        }
        const float ks = a.k_scale[w.kv_head()];
        const uint32_t flip = p.flip ^ (ks < 0.0f ? 0x80008000u : 0u);
        const int n = __popc(__ballot_sync(~0u, mine != -1));
#pragma unroll 1
        for (int i0 = 0; i0 * kRows < n; i0 += kBatch) {
          uint4 u[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const long long off = __shfl_sync(~0u, mine, (i0 + i) * kRows + sub);
            u[i] = make_uint4(0, 0, 0, 0);
            if (in && off != -1) u[i] = *reinterpret_cast<const uint4*>(q + off + chunk * 8);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            // fp16 against a power of two near the row's largest (bf16 mantissas fit); the scores take it back
            const int r = (row & ~31) + (i0 + i) * kRows + sub;
            const uint32_t w4[4] = {u[i].x ^ flip, u[i].y ^ flip, u[i].z ^ flip, u[i].w ^ flip};
            float big = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = unpack2<QT>(w4[k]);
              big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
            // 2^e <= big < 2^(e + 1), within 2^+-120; 1 for a row of zeros or with an infinity
            const int e = big > 0 && big < INFINITY ? min(max((__float_as_int(big) >> 23) - 127, -120), 120) : 0;
            const float down = __uint_as_float((127 - e) << 23);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = unpack2<QT>(w4[k]);
              v[k] = pack2<__half>(f.x * down, f.y * down);
            }
            const float up = __shfl_sync(~0u, __uint_as_float((127 + e) << 23), (lane % kRows) * kLanes);
            if (lane / kRows == i0 + i) next_cs = score_scale(p.scale_log2 * fabsf(ks)) * up;
            *reinterpret_cast<uint4*>(smem + (to - s0) + r * 128 + (((chunk ^ r) & 7) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        proxy_fence();
        bar_arrive(bar);
      };
      // the first key tile of this stream in the piece's tiles j0 .. j1 - 1 of an item
      auto first_of = [&](long long j0) { return pair || S::kStreams == 1 ? j0 : j0 + ((j0 ^ st) & 1); };
      bool ok = true;
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
        const PrefixWalk item = w;
        const long long j0 = w.done, j1 = j0 + w.left(), at_row = row_of(w);
        float2* ml = (line == kOwn ? p.own_ml : p.part_ml) + at_row;
        cs = next_cs;
        const int first_tile = w.tile;
        // keys that this row sees: those before `limit`
        int limit = w.len;
        if (line == kOwn) limit -= max(0, w.group_rows() - 1 - p.group_div(w.block() * kTileRows + row));
        const int all_see = w.all_see();
        float base = kNoBase, l = 0;  // (the first unit sets the base)
        bool first = true;
        const bool idle = (row & ~31) >= rows;  // none of this warp's rows is one: its scores are not looked at
        long long u = 0;
        const int every = pair ? 1 : S::kStreams;
        for (long long j = first_of(j0); ok && j < j1; j += every) {
          u = pair ? 2 * j + st : j;
          ok = __all_sync(~0u, bar_wait(&bars.s_full[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead));
          if (!ok) break;
          const int key0 = (first_tile + static_cast<int>(j - j0)) * kPrefixTile;
          if (!idle) {
          tc_after();
          const uint32_t at = tmem + lanes + static_cast<uint32_t>(u & 1) * 128;
          float s[128];
          float largest = tc_ld64_max(s, 0, at);
          largest = fmaxf(largest, tc_ld64_max(s, 64, at + 64));
          const bool hidden = key0 + kPrefixTile > all_see, flip = !E4M3 && p.flip;  // (flip: a negative scale)
          if (hidden || flip) {
            if (flip)
#pragma unroll
              for (int x = 0; x < 128; ++x) s[x] = -s[x];
            if (hidden) {
              const int valid = limit - key0;
#pragma unroll
              for (int x = 0; x < 128; ++x)
                if (x >= valid) s[x] = -INFINITY;
            }
            float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < 124; x += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) tops[k] = max3(tops[k], s[x + k], s[x + 4 + k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], s[124 + k]);
            largest = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
          }
          const float top = fmaxf(__fadd_ru(largest * cs, -kPrefixLift<T>), kNoBase);
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
          }
          bar_arrive(&bars.p_full[u & 1]);
          // The next item's queries: as soon as there is room for them. With two buffers that is at the item's start, but its
          // first probabilities go before.
          if (q_turns == 2 ? j == first_of(j0) : j + every >= j1) {
            w.skip();
            seek();
            if (!w.ends()) load_queries(w);
          }
        }
        if (!ok) break;
        ok = __all_sync(~0u, bar_wait(&bars.pv_done[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead));
        tc_after();
        float* out = (line == kOwn ? p.own : p.part) + at_row * D;
        const bool write = row < rows;
        // keys that not all rows see and whose values were left out: their probabilities once more
        bool slow = false;
        float late[kGroupRows];
        auto left_out_of = [&](int key) -> const uint8_t* { return bars.slow[(j0 + (key >> 7) - first_tile) & 15]; };
        auto any_left_out = [&](int key) -> bool {  // of the key's tile, where that is one of this stream's
          const long long j = j0 + (key >> 7) - first_tile;
          return j >= j0 && j < j1 && (S::kStreams == 1 || (j & 1) == st) && *reinterpret_cast<const uint32_t*>(left_out_of(key));
        };
        if (all_see < item.len && (any_left_out(max(all_see, 0)) || any_left_out(item.len - 1))) {
          for (int x = 0; x < kGroupRows; ++x) {
            const int key = all_see + x;
            late[x] = -1.0f;
            if (key < 0 || key >= item.len || !any_left_out(key)) continue;
            slow = true;
            const long long at = query_at(item);
            if (at == -1 || key >= limit) continue;
            const int page = a.table[item.request() * a.table_stride + p.page(key)];
            if (page < 0 || page >= a.n_pages) continue;
            const unsigned char* k = row_at(a.k_pages, p.k_step, page, item.kv_head(), key - p.page(key) * a.page_size);
            float t = 0;
            for (int d = 0; d < a.head_dim; ++d) t += static_cast<float>(static_cast<const QT*>(a.q)[at + d]) * cached<T, E4M3>(k, d);
            if (E4M3) t *= a.k_scale[item.kv_head()];
            late[x] = exp2_fast(t * a.scale * 1.44269504088896340736f - base);
          }
        }
#pragma unroll 1
        for (int d = 0; d < a.head_dim && !idle; d += 32) {
          float v[32];
          tc_ld(v, sums_at + d);
          if (slow)
            for (int x = 0; x < kGroupRows; ++x) {
              if (late[x] == -1.0f) continue;
              const int key = all_see + x;
              if (!left_out_of(key)[E4M3 ? (d >> 7) * 2 + (key >> 6 & 1) : d >> 6]) continue;
              const int page = a.table[item.request() * a.table_stride + p.page(key)];
              const unsigned char* from = row_at(a.v_pages, p.v_step, page, item.kv_head(), key - p.page(key) * a.page_size);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (d + i < a.head_dim) v[i] += late[x] * cached<T, E4M3>(from, d + i);
            }
          if (write)
#pragma unroll
            for (int x = 0; x < 32; x += 8)
              asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + d + x), "f"(v[x]), "f"(v[x + 1]),
                           "f"(v[x + 2]), "f"(v[x + 3]), "f"(v[x + 4]), "f"(v[x + 5]), "f"(v[x + 6]), "f"(v[x + 7]) : "memory");
        }
        // (a row that sees none of the item's keys has no part, whatever its scale)
        const bool none = l == 0.0f || limit <= 0;
        if (write) *ml = make_float2(none ? -INFINITY : base, none ? 0.0f : l);
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

// The cache as the copies see it: boxes of `rows` places and 128 bytes of a head (copies begin on 128 bytes of shared memory).
cudaError_t map_cache(CUtensorMap* map, const void* pages, const mk_prefix_attention_args& a, const int64_t* strides, int rows, bool e4m3);

template <typename T, typename QT, int D, bool E4M3>
cudaError_t launch_prefix(const PrefixParams& p, int device, cudaStream_t s) {
  constexpr auto kernel = prefix_kernel<T, QT, D, E4M3>;
  using S = PrefixShape<D, E4M3>;
  if (const cudaError_t e = allow_smem<kernel>(device, S::kSmem)) return e;
  // setmaxnreg hands out what the block was launched with; a build with less would wait for ever
  static std::atomic<int> known{0};
  int regs = known.load(std::memory_order_relaxed);
  if (!regs) {
    cudaFuncAttributes f{};
    if (const cudaError_t e = cudaFuncGetAttributes(&f, kernel)) return e;
    known.store(regs = f.numRegs, std::memory_order_relaxed);
  }
  if (regs * S::kThreads < 256 * S::kSoftmaxRegs + (S::kThreads - 256) * S::kOtherRegs) return cudaErrorInvalidConfiguration;
  PrefixParams q = p;
  const mk_prefix_attention_args& a = p.a;
  q.box = a.page_size & -a.page_size;
  if (q.box > kPrefixTile) q.box = kPrefixTile;
  const int64_t *ks = a.k_page_stride, *vs = a.v_page_stride;
  cudaError_t e = map_cache(&q.keys, a.k_pages, a, ks, q.box, E4M3);
  if (e == cudaSuccess) e = map_cache(&q.values, a.v_pages, a, vs, q.box, E4M3);
  return e == cudaSuccess ? start(kernel, p.ctas, S::kThreads, S::kSmem, s, q) : e;
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
