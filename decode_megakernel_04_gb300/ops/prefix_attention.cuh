// The kernel of mk_prefix_attention for the shared prefix, on the 5th-generation tensor cores with accumulators in tensor
// memory (prefix_attention.cu: arguments, the own positions, the join).
//
// For a kv head, every query row of every request meets the same keys: scores S = Q K^T of [128 rows x 128 keys], an online
// softmax, sums O += P V. At rows x 2 flops a cached byte (16 bits) this is bound by the tensor cores from about 280 rows on,
// by memory below.
// - Work: 128 query rows of a kv head are a row tile. Two row tiles share each tile of keys where there are two (a pair:
//   keys and values are read from L2 once for 256 rows); an odd one is left alone, and then even and odd key tiles go to
//   two sets of sums (so that there are two streams in either case; 256 wide the tensor memory holds one). The
//   (kv head, row block) items' key tiles are one line, cut into equal pieces, one for each CTA; pairs and single tiles are two
//   lines with CTAs in proportion to their products.
// - Units: the product of one row tile and one key tile, in turn on two score buffers. One thread issues S(0), S(1), then
//   for each unit u: O += P(u) V and S(u + 2): while one stream's softmax runs, the tensor cores work on the other.
// - Softmax: a thread has a row (128 threads a stream), so nothing is exchanged. The row's scores come from tensor memory 32 columns at
//   a time; probabilities go back over the first half of the scores' columns as the product's operand (16 bits).
//   They are taken against a base that moves only when a score passes it by kGrow: else sums stay as they are.
// - Loads: warps 9-11 copy keys, 12-14 values (cp.async, row by row through the page table) into a ring of slots; codes of e4m3
//   caches pass through registers and become fp16 there. Queries are stored by the softmax threads; those of the next item
//   while the last product of this one runs.
// Probabilities are one 16-bit number: a pair hi + lo as over own positions would be half as much work again for the tensor cores.
// bf16: 2^-8 of each at most; fp16: 2^-11, against a base 14 under the maximum, so that what falls under its range is 2^-39 of
// the largest. Sums of probabilities are those of the unrounded ones.
// Every wait has a limit (2 s), after which the CTA gives up, drains and frees what it holds and MK_OP_TIMEOUT is set.
#pragma once
#include "paged_attention_tc.cuh"

namespace mkop {
namespace prefix {

using namespace attn;

constexpr int kPrefixTile = 128;      // keys
constexpr int kTileRows = 128;        // query rows of a row tile
constexpr int kMinPiece = 1;          // key tiles of a piece at least

// One line of key tiles: `items` (kv head, row block) one after the other, cut among `ctas`. Piece c's part of item i goes to
// place c + i: along the line either grows by one from part to part.
struct Lane {
  int ctas;         // 0: no such items
  int blocks;       // row blocks of a kv head
  int first_row;    // of the first block
  int rows;         // of a block
  int place0;       // of its places among all
};

struct PrefixParams {
  mk_prefix_attention_args a;
  Div page, group_div, row_div;
  int group;          // query heads per kv head
  int n_rows;         // query rows of a kv head: batch * rows * group
  int max_len;
  int dp;             // 64, 128 or 256
  int streams;        // sums a place holds (1 at 256 wide, else 2)
  Lane lane[2];       // pairs of row tiles; single ones
  float scale_log2;   // |scale| * log2(e)
  uint32_t flip;      // sign bits of two 16-bit values where the scale is negative: queries change their sign instead
  uint32_t k_step[3], v_step[3];  // the caches' strides (page, head, place) in units of 16 bytes
  float* part;        // [places][streams][128][dp] sums of a part
  float2* part_ml;    // [places][streams][128] its base (log2 units) and sum of probabilities; sum 0: an empty part, sums not written
  float* raw;         // [batch][rows][n_q_heads][dp] results over the own positions
  float* raw_lse;     // [batch][rows][n_q_heads] their log-sums, log2 units
};

struct Line {
  int len, tiles, used;
  long long total;
  __device__ Line(const PrefixParams& p, const Lane& l) {
    len = min(max(p.a.prefix_len[0], 0), p.max_len);
    tiles = (len + kPrefixTile - 1) / kPrefixTile;
    total = static_cast<long long>(p.a.n_kv_heads) * l.blocks * tiles;
    const long long worth = (total + kMinPiece - 1) / kMinPiece;
    used = static_cast<int>(worth < l.ctas ? worth : l.ctas);
  }
  // the last piece that begins at or before tile x
  __device__ int piece_of(long long x) const { return static_cast<int>(((x + 1) * used - 1) / total); }
};

constexpr int kSoftmaxRegs = 160, kOtherRegs = 88;

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
  static constexpr int kOffScale = kOffAddr + 2 * 2 * 128 * 8;  // float [2][128]
  static constexpr int kOffBar = kOffScale + 2 * 128 * 4;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

template <typename T>
constexpr float kPrefixLift = std::is_same<T, __half>::value ? 14.0f : 0.0f;  // the base is this much under the maximum
template <typename T>
constexpr float kPrefixGrow = std::is_same<T, __half>::value ? 1.0f : 8.0f;   // and moves when a score passes that by this

struct PrefixBars {
  uint64_t full[8], empty[8], q_full[2], s_full[2], p_full[2], pv_done[2], drained;
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(PrefixBars) <= 512, "");

// D[tmem] (+)= A[tmem] B: A is 16-bit pairs, a lane a row
__device__ inline void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
// 16 consecutive columns of this warp's lanes from packed values (tcgen05.wait::st follows separately)
__device__ inline void tc_st_packed(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
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
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  PrefixBars& bars = *reinterpret_cast<PrefixBars*>(smem + S::kOffBar);
  volatile int* dead = &bars.dead;

  // ---- this CTA's piece of a line -----------------------------------------------------------------------------------
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool single = static_cast<int>(blockIdx.x) >= p.lane[0].ctas;
  const bool pair = S::kStreams == 2 && !single;
  const Lane& ln = p.lane[single];
  const int c = blockIdx.x - (single ? p.lane[0].ctas : 0);
  const Line line(p, ln);
  if (blockIdx.x == 0 && tid == 0 && line.len != a.prefix_len[0]) flag(a.status, MK_OP_BAD_LENGTH);
  if (c >= line.used) {
    // the join follows this kernel and has to follow what came before it
    if (tid == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const long long begin = piece_begin(c, line.total, line.used);
  const int count = static_cast<int>(piece_begin(c + 1, line.total, line.used) - begin);  // key tiles of this piece
  const int item0 = static_cast<int>(begin / line.tiles), tile0 = static_cast<int>(begin - static_cast<long long>(item0) * line.tiles);
  const int units = pair ? 2 * count : count;

  if (tid == 0) {
    for (int i = 0; i < S::kSlots; ++i) bar_init(&bars.full[i], S::kLoaders), bar_init(&bars.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.q_full[i], S::kStreamThreads), bar_init(&bars.s_full[i], 1);
      bar_init(&bars.p_full[i], S::kStreamThreads), bar_init(&bars.pv_done[i], 1);
    }
    bar_init(&bars.drained, 1);
    bars.dead = 0;
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
  auto scores_at = [&](int u) { return tmem + static_cast<uint32_t>(u & 1) * 128; };
  auto sums_at = [&](int stream) { return tmem + 256 + static_cast<uint32_t>(stream) * D; };

  // 512 threads x 128 registers: 256 x 160 for the softmax, 256 x 88 for the rest (63488 of 65536)
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp >= 9 && warp < 15) {
    // ---- loaders --------------------------------------------------------------------------------------------------
    const bool value = warp >= 12;
    const int t = tid - (value ? 384 : 288), barrier = value ? 3 : 2;
    const unsigned char** addr = reinterpret_cast<const unsigned char**>(smem + S::kOffAddr) + (value ? 256 : 0);
    int item = item0, tile = tile0;  // of the next tile that gets addresses
    int made = 0;                    // tiles that have them
    auto look_up = [&](int key) -> int {
      key += tile * kPrefixTile;
      return made < count && key < line.len ? a.prefix_table[p.page(key)] : -1;
    };
    auto make_address = [&](const unsigned char** at, int page, int i) {
      const unsigned char* from = kZeros;
      const int key = tile * kPrefixTile + i;
      if (made < count && key < line.len) {
        if (page < 0 || page >= a.n_pages) {
          flag(a.status, MK_OP_BAD_PAGE);
        } else {
          const int place = key - p.page(key) * a.page_size, head = item / ln.blocks;
          from = value ? row_at(a.v_pages, p.v_step, page, head, place) : row_at(a.k_pages, p.k_step, page, head, place);
        }
      }
      at[i] = from;
    };
    auto next = [&]() {
      ++made;
      if (++tile == line.tiles) tile = 0, ++item;
    };
    const bool two = t < 128 - S::kLoaders;
    bool ok = true;
    make_address(addr, look_up(t), t);
    if (two) make_address(addr, look_up(t + S::kLoaders), t + S::kLoaders);
    next();
    int page = look_up(t), page2 = two ? look_up(t + S::kLoaders) : -1;
    constexpr int kSrc = E4M3 ? S::kWide / 16 : S::kWide / 8;  // 16-byte pieces of a slot's row in the cache
    constexpr int kStep = S::kLoaders / kSrc, kTurns = (kPrefixTile + kStep - 1) / kStep;
    const int chunk = t % kSrc, row0 = t / kSrc;
    for (int j = 0; j < count; ++j) {
      const unsigned char** at = addr + (j & 1) * 128;
      if (any_of(barrier, S::kLoaders, !ok)) break;
#pragma unroll 1
      for (int h = 0; h < S::kHalves; ++h) {
        const uint32_t g = (static_cast<uint32_t>(j) * 2 + (value ? 1 : 0)) * S::kHalves + h;
        const int slot = g % S::kSlots, turn = g / S::kSlots;
        const int column = h * S::kWide * (E4M3 ? 1 : 2) + chunk * 16;  // bytes
        const bool in = column < a.head_dim * (E4M3 ? 1 : 2);         // columns behind the head are not read, or not used
        const unsigned char* const* from = at + row0;
        if (!E4M3) {
          if (turn) ok = bar_wait(&bars.empty[slot], (turn - 1) & 1, dead) && ok;
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
          uint4 u[kTurns];
#pragma unroll
          for (int i = 0; i < kTurns; ++i)
            if (row0 + kStep * i < kPrefixTile) {
              const unsigned char* f = from[kStep * i];
              u[i] = in ? *reinterpret_cast<const uint4*>(f + column) : make_uint4(0, 0, 0, 0);
            }
          if (turn) ok = bar_wait(&bars.empty[slot], (turn - 1) & 1, dead) && ok;
          // codes 16 chunk .. become pieces 2 chunk and 2 chunk + 1
          unsigned char* to = smem + slot * S::kSlot + (chunk >> 2) * (kPrefixTile * 128);
#pragma unroll
          for (int i = 0; i < kTurns; ++i) {
            const int row = row0 + kStep * i;
            if (row >= kPrefixTile) break;
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t lo[2], hi[2];
              e4m3_to_f16(lo, w[2 * k]);
              e4m3_to_f16(hi, w[2 * k + 1]);
              *reinterpret_cast<uint4*>(to + row * 128 + ((((2 * chunk + k) ^ row) & 7) << 4)) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
            }
          }
          proxy_fence();
          bar_arrive(&bars.full[slot]);
        }
        if (h == 0) {  // the next tile's addresses, while copies are in flight
          make_address(addr + (~j & 1) * 128, page, t);
          if (two) make_address(addr + (~j & 1) * 128, page2, t + S::kLoaders);
          next();
          page = look_up(t);
          if (two) page2 = look_up(t + S::kLoaders);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 8) {
    // ---- the thread that issues the products ---------------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t kScores = prefix_idesc<T>(kPrefixTile, false), kSums = prefix_idesc<T>(S::kWide, true);
      const int steps = a.head_dim / 16;
      int q_item0 = -1, q_item1 = -1, q_turn0 = 0, q_turn1 = 0, o_item0 = -1, o_item1 = -1;  // of either stream
      bool ok = true;
      auto tile_of = [&](int u) { return pair ? u >> 1 : u; };
      auto stream_of = [&](int u) { return S::kStreams == 2 ? u & 1 : 0; };
      auto scores = [&](int u) {
        const int j = tile_of(u), st = stream_of(u), item = (tile0 + j) / line.tiles;
        if (item != (st ? q_item1 : q_item0)) {
          (st ? q_item1 : q_item0) = item;
          ok = ok && bar_wait(&bars.q_full[st], (st ? q_turn1 : q_turn0) & 1, dead);
          ++(st ? q_turn1 : q_turn0);
          proxy_fence();
        }
        const uint32_t qa = s0 + S::kOffQ + st * S::kQ;
        for (int h = 0; h < S::kHalves && ok; ++h) {
          const uint32_t g = static_cast<uint32_t>(j) * 2 * S::kHalves + h, slot = g % S::kSlots;
          ok = bar_wait(&bars.full[slot], (g / S::kSlots) & 1, dead);
          if (!ok) break;
          proxy_fence();
          tc_after();
          const uint64_t kd = tc_desc(s0 + slot * S::kSlot, 16), qd = tc_desc(qa + 2 * h * (kTileRows * 128), 16);
#pragma unroll
          for (int k = 0; k < S::kWide / 16; ++k)
            if (h * 8 + k < steps)
              tc_mma(scores_at(u), qd + ((k >> 2) * (kTileRows * 128) + (k & 3) * 32) / 16,
                     kd + ((k >> 2) * (kPrefixTile * 128) + (k & 3) * 32) / 16, kScores, h > 0 || k > 0);
          if (!pair || (u & 1)) tc_commit(&bars.empty[slot]);
        }
        if (ok) tc_commit(&bars.s_full[u & 1]);
      };
      scores(0);
      if (units > 1 && ok) scores(1);
      for (int u = 0; u < units && ok; ++u) {
        const int j = tile_of(u), st = stream_of(u), item = (tile0 + j) / line.tiles;
        const bool fresh = item != (st ? o_item1 : o_item0);
        (st ? o_item1 : o_item0) = item;
        if (!(ok = bar_wait(&bars.p_full[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead))) break;
        for (int h = 0; h < S::kHalves; ++h) {
          const uint32_t g = static_cast<uint32_t>(j) * 2 * S::kHalves + S::kHalves + h, slot = g % S::kSlots;
          ok = bar_wait(&bars.full[slot], (g / S::kSlots) & 1, dead);
          if (!ok) break;
          proxy_fence();
          tc_after();
          const uint64_t vd = tc_desc(s0 + slot * S::kSlot, kPrefixTile * 128);
#pragma unroll
          for (int k = 0; k < kPrefixTile / 16; ++k)
            tc_mma_ts(sums_at(st) + h * 128, scores_at(u) + k * 8, vd + k * 2048 / 16, kSums, !fresh || k > 0);
          if (!pair || (u & 1)) tc_commit(&bars.empty[slot]);
        }
        if (!ok) break;
        tc_commit(&bars.pv_done[u & 1]);
        // (the scores of u + 2 go where the probabilities of u were: the products run in the order of their issue)
        if (u + 2 < units) scores(u + 2);
      }
      // every product has ended before the tensor memory is freed, also when the CTA gave up
      tc_commit(&bars.drained);
      int alive = 0;
      bar_wait(&bars.drained, 0, &alive);
    }
    __syncwarp();
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  if (warp < 4 * S::kStreams) {
    // ---- softmax: a thread has a row of the stream's row tile ---------------------------------------------------------
    const int st = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    float* row_scale = reinterpret_cast<float*>(smem + S::kOffScale) + st * 128;
    float cs = fmaxf(p.scale_log2, 1.17549435e-38f);  // (a score of -infinity stays one where the scale is 0)
    // Queries of an item's row tile into shared memory; D / 8 lanes have a row.
    auto load_queries = [&](int item) {
      const int head = item / ln.blocks, block = item - head * ln.blocks;
      const float ks = E4M3 ? a.k_scale[head] : 1.0f;
      const uint32_t flip = p.flip ^ (ks < 0.0f ? 0x80008000u : 0u);
      const int m0 = ln.first_row + block * ln.rows + (pair ? st * kTileRows : 0);
      constexpr int kLanes = D / 8, kRows = S::kStreamThreads / kLanes;
      const int chunk = row % kLanes, r0 = row / kLanes;
      unsigned char* to = smem + S::kOffQ + st * S::kQ + (chunk >> 3) * (kTileRows * 128);
      const bool in = chunk * 8 < a.head_dim;
#pragma unroll 4
      for (int i = 0; i < kTileRows / kRows; ++i) {
        const int r = r0 + i * kRows, m = m0 + r;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (in && m < p.n_rows) {
          const int br = p.group_div(m), h = head * p.group + m - br * p.group, b = p.row_div(br), qr = br - b * a.rows;
          u = *reinterpret_cast<const uint4*>(static_cast<const QT*>(a.q) + b * a.q_stride[0] + qr * a.q_stride[1] + h * a.q_stride[2] + chunk * 8);
        }
        u.x ^= flip, u.y ^= flip, u.z ^= flip, u.w ^= flip;
        if (E4M3) {
          // fp16 against a power of two near the row's largest (bf16 mantissas fit); the scores take it back
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
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
          u = make_uint4(v[0], v[1], v[2], v[3]);
          if (chunk == 0) row_scale[r] = fmaxf(p.scale_log2 * fabsf(ks), 1.17549435e-38f) * __uint_as_float((127 + e) << 23);
        }
        *reinterpret_cast<uint4*>(to + r * 128 + (((chunk ^ r) & 7) << 4)) = u;
      }
      proxy_fence();
      bar_arrive(&bars.q_full[st]);
    };
    // the first unit of this stream at or after key tile j of the piece
    auto first_unit = [&](int j) { return pair ? 2 * j + st : S::kStreams == 2 ? j + ((j ^ st) & 1) : j; };
    const int last_item = (tile0 + count - 1) / line.tiles;  // counted from item0
    auto end_of = [&](int i) { return min(count, (i + 1) * line.tiles - tile0); };  // its end, in key tiles of the piece
    auto begin_of = [&](int i) { return max(0, i * line.tiles - tile0); };
    auto has_units = [&](int i) { return (pair ? first_unit(begin_of(i)) >> 1 : first_unit(begin_of(i))) < end_of(i); };
    bool ok = true, loaded = false;
    // (no warp leaves this loop early: the named barriers wait without a limit, so each has to reach all of them)
    for (int i = 0; i <= last_item; ++i) {
      const long long place = (ln.place0 + static_cast<long long>(c) + item0 + i) * S::kStreams + st;
      if (!has_units(i)) {
        p.part_ml[place * kTileRows + row] = make_float2(-INFINITY, 0.0f);
        continue;
      }
      if (!loaded) load_queries(item0 + i);
      if (E4M3) {
        ok = !any_of(4 + st, S::kStreamThreads, !ok);  // every row's scale is there
        cs = row_scale[row];
        named_sync(4 + st, S::kStreamThreads);         // and has been read before the next item's are written
      }
      const int u0 = first_unit(begin_of(i)), u1 = pair ? 2 * end_of(i) : end_of(i);
      constexpr int kUnits = S::kStreams;  // from one unit of a stream to the next
      float base = kNoBase, l = 0;  // (the first unit sets the base)
      int u = u0;
      for (; ok && u < u1; u += kUnits) {
        ok = __all_sync(~0u, bar_wait(&bars.s_full[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead));
        if (!ok) break;
        tc_after();
        const int tile = (tile0 + (pair ? u >> 1 : u)) % line.tiles;
        const int valid = line.len - tile * kPrefixTile;  // keys of this tile, where under 128
        const uint32_t at = scores_at(u) + lanes;
        auto chunk_of = [&](int k, float (&s)[32]) {
          tc_ld(s, at + 32 * k);
          if (valid < kPrefixTile)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (32 * k + x >= valid) s[x] = -INFINITY;
        };
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float s[32];
          chunk_of(k, s);
#pragma unroll
          for (int x = 0; x < 32; ++x) tops[x & 3] = fmaxf(tops[x & 3], s[x]);
        }
        const float top = fmaxf(__fadd_ru(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * cs, -kPrefixLift<T>), kNoBase);
        const bool first = u == u0;
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
              tc_ld(v, sums_at(st) + lanes + d);
#pragma unroll
              for (int x = 0; x < 32; ++x) v[x] *= shrink;
              tc_st(sums_at(st) + lanes + d, v);
            }
          }
        }
        float sums[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float s[32];
          uint32_t packed[16];
          chunk_of(k, s);
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float e = exp2_fast(fmaf(s[x], cs, -base)), f = exp2_fast(fmaf(s[x + 1], cs, -base));
            sums[x & 2] += e, sums[(x & 2) + 1] += f;
            packed[x / 2] = pack2<T>(e, f);
          }
          tc_st_packed(at + 16 * k, packed);  // (over scores that have been read)
        }
        l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
        tc_wait_st();
        tc_before();
        bar_arrive(&bars.p_full[u & 1]);
      }
      loaded = false;
      if (!ok) continue;
      // the next item's queries, whose place the last scores have left
      for (int n = i + 1; n <= last_item && !loaded; ++n)
        if (has_units(n)) {
          load_queries(item0 + n);
          loaded = true;
        }
      u -= kUnits;
      ok = __all_sync(~0u, bar_wait(&bars.pv_done[u & 1], static_cast<uint32_t>(u >> 1) & 1, dead));
      tc_after();
      float* out = p.part + (place * kTileRows + row) * D;
#pragma unroll 1
      for (int d = 0; d < a.head_dim; d += 32) {
        float v[32];
        tc_ld(v, sums_at(st) + lanes + d);
#pragma unroll
        for (int x = 0; x < 32; x += 4) *reinterpret_cast<float4*>(out + d + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
      }
      p.part_ml[place * kTileRows + row] = make_float2(l == 0.0f ? -INFINITY : base, l);
      tc_before();
    }
  }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (tid == 0) {
    if (*dead) flag(a.status, MK_OP_TIMEOUT);
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
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
  if (regs * PrefixShape<D>::kThreads < 256 * (kSoftmaxRegs + kOtherRegs)) return cudaErrorInvalidConfiguration;
  // It does not read what the own positions' kernels write, so it may start while they run.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.lane[0].ctas + p.lane[1].ctas);
  cfg.blockDim = dim3(PrefixShape<D>::kThreads);
  cfg.dynamicSmemBytes = PrefixShape<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
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
