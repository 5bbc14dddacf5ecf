// mk_prefix_attention: attention of a batch over a prefix that its requests share and over each request's own positions.
//
// softmax over both parts is joined from parts: own positions by mk_paged_attention (results and their log-sums in fp32),
// the prefix once for all query rows of a kv head, cut along its keys, and a last kernel that weights the parts of a row.
#include <cuda_fp8.h>

#include "paged_attention.cuh"

namespace mkop {
namespace prefix {
namespace {

using attn::piece_begin;
using attn::row_at;

constexpr int kMinTiles = 2;   // of a piece at least
constexpr int kJoinWarps = 8;

struct Params {
  mk_prefix_attention_args a;
  Div page, group_div;
  int group;          // query heads per kv head
  int n_rows;         // query rows of a kv head: batch * rows * group
  int blocks;         // of block_rows query rows
  int block_rows;
  int tile;           // keys
  int ctas;           // pieces that the line is cut into at most
  int max_len;
  int dp;             // 64, 128 or 256
  float scale_log2;
  uint32_t k_step[3], v_step[3];  // the caches' strides (page, head, place) in units of 16 bytes
  float* part;        // [ctas + kv heads * blocks][block_rows][dp] sums of a part
  float2* part_ml;    // [..][block_rows] its base (log2 units) and sum
  float* raw;         // [batch][rows][n_q_heads][dp] results over the own positions
  float* raw_lse;     // [batch][rows][n_q_heads] their log-sums, log2 units
};

// The prefix as a line of tiles, one (kv head, row block) after the other, cut into `used` pieces. Piece c's part of item i
// goes to slot c + i: along the line either grows by one from part to part.
struct Line {
  int len, tiles, used;
  long long total;
  __device__ explicit Line(const Params& p) {
    len = min(max(p.a.prefix_len[0], 0), p.max_len);
    tiles = (len + p.tile - 1) / p.tile;
    total = static_cast<long long>(p.a.n_kv_heads) * p.blocks * tiles;
    const long long worth = (total + kMinTiles - 1) / kMinTiles;
    used = static_cast<int>(worth < p.ctas ? worth : p.ctas);
  }
  // the last piece that begins at or before tile x
  __device__ int piece_of(long long x) const { return static_cast<int>(((x + 1) * used - 1) / total); }
};

constexpr int kRows = 16, kTile = 32, kThreads = 128;

template <typename T>
__device__ inline float element(const unsigned char* row, int i) { return static_cast<float>(reinterpret_cast<const T*>(row)[i]); }

// One CTA per piece. A thread has one of 16 rows and every eighth key and column.
template <typename T, typename Cache, int DP>
__global__ void __launch_bounds__(kThreads) prefix_kernel(const __grid_constant__ Params p) {
  extern __shared__ float smem[];
  float* q = smem;                         // [16][DP + 1]
  float* kv = q + kRows * (DP + 1);        // [32][DP + 1]
  float* prob = kv + kTile * (DP + 1);     // [16][32]
  const mk_prefix_attention_args& a = p.a;
  const int tid = threadIdx.x, row = tid >> 3, sub = tid & 7;
  const Line line(p);
  if (blockIdx.x == 0 && tid == 0 && line.len != a.prefix_len[0]) flag(a.status, MK_OP_BAD_LENGTH);
  const int c = blockIdx.x;
  if (c >= line.used) return;
  const long long end = piece_begin(c + 1, line.total, line.used);
  for (long long x = piece_begin(c, line.total, line.used); x < end;) {
    const int item = static_cast<int>(x / line.tiles), t0 = static_cast<int>(x - static_cast<long long>(item) * line.tiles);
    const int t1 = static_cast<int>(min(static_cast<long long>(line.tiles), t0 + end - x));
    const int head = item / p.blocks, block = item - head * p.blocks;
    __syncthreads();
    for (int i = tid; i < kRows * DP; i += kThreads) {
      const int r = i / DP, d = i % DP, m = block * kRows + r;
      float v = 0;
      if (m < p.n_rows && d < a.head_dim) {
        const int br = p.group_div(m), h = head * p.group + m - br * p.group, b = br / a.rows, qr = br - b * a.rows;
        v = static_cast<float>(static_cast<const T*>(a.q)[b * a.q_stride[0] + qr * a.q_stride[1] + h * a.q_stride[2] + d]);
      }
      q[r * (DP + 1) + d] = v;
    }
    float o[DP / 8], base = -INFINITY, sum = 0;
    for (int i = 0; i < DP / 8; ++i) o[i] = 0;
    const float scale = p.scale_log2 * (sizeof(Cache) == 1 ? a.k_scale[head] : 1.0f);
    auto load = [&](const void* cache, const uint32_t (&step)[3], int key0) {
      __syncthreads();
      for (int i = tid; i < kTile * DP; i += kThreads) {
        const int k = i / DP, d = i % DP, key = key0 + k;
        float v = 0;
        if (key < line.len && d < a.head_dim) {
          const int pg = p.page(key), page = a.prefix_table[pg];
          if (page >= 0 && page < a.n_pages) v = element<Cache>(row_at(cache, step, page, head, key - pg * a.page_size), d);
          else flag(a.status, MK_OP_BAD_PAGE);
        }
        kv[k * (DP + 1) + d] = v;
      }
      __syncthreads();
    };
    for (int t = t0; t < t1; ++t) {
      const int key0 = t * kTile;
      load(a.k_pages, p.k_step, key0);
      float s[4], top = base;
      for (int j = 0; j < 4; ++j) {
        const int k = sub + 8 * j;
        float x = 0;
        for (int d = 0; d < DP; ++d) x += q[row * (DP + 1) + d] * kv[k * (DP + 1) + d];
        s[j] = key0 + k < line.len ? x * scale : -INFINITY;
        top = fmaxf(top, s[j]);
      }
      for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      const float safe = top == -INFINITY ? 0.0f : top, shrink = exp2f(base - safe);
      base = top;
      sum *= shrink;
      for (int i = 0; i < DP / 8; ++i) o[i] *= shrink;
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[j] - safe);
        sum += e;
        prob[row * kTile + sub + 8 * j] = e;
      }
      load(a.v_pages, p.v_step, key0);
      for (int k = 0; k < kTile; ++k) {
        const float e = prob[row * kTile + k];
        for (int i = 0; i < DP / 8; ++i) o[i] += e * kv[k * (DP + 1) + sub + 8 * i];
      }
    }
    for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
    const long long at = static_cast<long long>(c + item) * kRows + row;
    for (int i = 0; i < DP / 8; ++i) p.part[at * DP + sub + 8 * i] = o[i];
    if (sub == 0) p.part_ml[at] = make_float2(base, sum);
    x += t1 - t0;
  }
}

// A warp for each row of out: the parts of the prefix and the result over the own positions, weighted by exp2(base - largest base).
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p) {
  const mk_prefix_attention_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.batch) * a.rows * a.n_q_heads) return;
  const int br = static_cast<int>(row / a.n_q_heads), h = static_cast<int>(row - static_cast<long long>(br) * a.n_q_heads);
  const int head = h / p.group, m = br * p.group + h - head * p.group, block = m / p.block_rows;
  const int b = br / a.rows, r = br - b * a.rows;
  const Line line(p);
  const long long item = static_cast<long long>(head) * p.blocks + block;
  int c0 = 0, n = 0;
  if (line.total) {
    c0 = line.piece_of(item * line.tiles);
    n = line.piece_of((item + 1) * line.tiles - 1) - c0 + 1;
  }
  auto at = [&](int k) { return (c0 + k + item) * p.block_rows + m - block * p.block_rows; };
  const float own = p.raw_lse[row];
  float top = own;
  for (int k = lane; k < n; k += 32) top = fmaxf(top, p.part_ml[at(k)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0;
  for (int k = lane; k < n; k += 32) {
    const float2 s = p.part_ml[at(k)];
    sum += attn::exp2_fast(s.x - base) * s.y;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  const float f_own = attn::exp2_fast(own - base);
  sum += f_own;
  const float scale = sum == 0.0f ? 0.0f : 1.0f / sum, vs = a.cache_dtype == MK_E4M3 ? a.v_scale[head] : 1.0f;
  T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + r * a.out_stride[1] + h * a.out_stride[2];
  for (int d = lane * 4; d < a.head_dim; d += 128) {
    float4 y = make_float4(0, 0, 0, 0);
    for (int k = 0; k < n; ++k) {
      const float f = attn::exp2_fast(p.part_ml[at(k)].x - base);
      const float4 x = *reinterpret_cast<const float4*>(p.part + at(k) * p.dp + d);
      y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
    }
    const float4 x = *reinterpret_cast<const float4*>(p.raw + row * p.dp + d);
    y.x = y.x * vs + f_own * x.x, y.y = y.y * vs + f_own * x.y, y.z = y.z * vs + f_own * x.z, y.w = y.w * vs + f_own * x.w;
    *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(y.x * scale, y.y * scale), pack2<T>(y.z * scale, y.w * scale));
  }
  if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

const char* const kMe = "mk_prefix_attention";

// What mk_paged_attention is asked for the own positions.
mk_paged_attention_args own_call(const mk_prefix_attention_args& a) {
  mk_paged_attention_args o{};
  o.q = a.q, o.k_pages = a.k_pages, o.v_pages = a.v_pages, o.table = a.table, o.lens = a.lens, o.k_scale = a.k_scale;
  o.v_scale = a.v_scale, o.out = a.out, o.status = a.status, o.table_stride = a.table_stride;
  for (int i = 0; i < 3; ++i) {
    o.q_stride[i] = a.q_stride[i], o.out_stride[i] = a.out_stride[i];
    o.k_page_stride[i] = a.k_page_stride[i], o.v_page_stride[i] = a.v_page_stride[i];
  }
  o.batch = a.batch, o.rows = a.rows, o.n_q_heads = a.n_q_heads, o.n_kv_heads = a.n_kv_heads, o.head_dim = a.head_dim;
  o.n_pages = a.n_pages, o.page_size = a.page_size, o.max_pages = a.max_pages, o.dtype = a.dtype, o.cache_dtype = a.cache_dtype;
  o.scale = a.scale;
  return o;
}

// What follows from the shape fields alone.
struct Plan {
  int group, n_rows, blocks, block_rows, tile, ctas, dp;
  uint64_t ml_at, raw_at, lse_at, own_at, bytes;
};

mk_status check_shape(const mk_prefix_attention_args& a, int device) {
  if (a.batch < 0 || a.max_prefix_pages < 1)
    return refuse(MK_ERR_INVALID_ARG, kMe, "batch %d, max_prefix_pages %d", a.batch, a.max_prefix_pages);
  if (mk_status s = attn::check_shape(kMe, own_call(a), device)) return s;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * a.rows * (a.n_q_heads / a.n_kv_heads);
  if (n_rows > 1 << 24) return refuse(MK_ERR_UNSUPPORTED, kMe, "%lld query rows of a kv head", static_cast<long long>(n_rows));
  return MK_OK;
}

// check_shape() has passed
mk_status plan(const mk_prefix_attention_args& a, int device, Plan* out) {
  Plan& pl = *out;
  uint64_t own = 0;
  if (mk_status s = attn::workspace_of(kMe, own_call(a), device, &own)) return s;
  pl.group = a.n_q_heads / a.n_kv_heads;
  pl.n_rows = a.batch * a.rows * pl.group;
  pl.dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
  pl.block_rows = kRows;
  pl.tile = kTile;
  pl.blocks = (pl.n_rows + kRows - 1) / kRows;
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(kMe, e);
  pl.ctas = 4 * sms;
  const uint64_t slots = pl.ctas + static_cast<uint64_t>(a.n_kv_heads) * pl.blocks, results = static_cast<uint64_t>(pl.n_rows) * a.n_kv_heads;
  auto whole = [](uint64_t n) { return (n + 255) / 256 * 256; };
  pl.ml_at = whole(slots * pl.block_rows * pl.dp * sizeof(float));
  pl.raw_at = pl.ml_at + whole(slots * pl.block_rows * sizeof(float2));
  pl.lse_at = pl.raw_at + whole(results * pl.dp * sizeof(float));
  pl.own_at = pl.lse_at + whole(results * sizeof(float));
  pl.bytes = pl.own_at + own;
  return MK_OK;
}

template <typename T, typename Cache, int DP>
cudaError_t launch(const Params& p, int device, cudaStream_t s) {
  constexpr int kSmem = (kRows * (DP + 1) + kTile * (DP + 1) + kRows * kTile) * 4;
  if (const cudaError_t e = allow_smem<prefix_kernel<T, Cache, DP>>(device, kSmem)) return e;
  return start(prefix_kernel<T, Cache, DP>, p.ctas, kThreads, kSmem, s, p);
}
template <typename T, typename Cache>
cudaError_t launch(const Params& p, int device, cudaStream_t s) {
  return p.dp == 64 ? launch<T, Cache, 64>(p, device, s) : p.dp == 128 ? launch<T, Cache, 128>(p, device, s)
                                                                       : launch<T, Cache, 256>(p, device, s);
}

}  // namespace
}  // namespace prefix
}  // namespace mkop

extern "C" mk_status mk_prefix_attention_workspace(const mk_prefix_attention_args* p, int device, uint64_t* bytes) {
  using namespace mkop::prefix;
  if (!p || !bytes) return MK_ERR_INVALID_ARG;
  if (mk_status s = check_shape(*p, device)) return s;
  Plan pl;
  if (mk_status s = plan(*p, device, &pl)) return s;
  *bytes = pl.bytes;
  return MK_OK;
}

extern "C" mk_status mk_prefix_attention(const mk_prefix_attention_args* args, int device, void* stream) {
  using namespace mkop;
  using namespace mkop::prefix;
  if (!args) return MK_ERR_INVALID_ARG;
  Params p{};
  p.a = *args;
  const mk_prefix_attention_args& a = p.a;
  if (mk_status s = check_shape(a, device)) return s;
  mk_paged_attention_args own = own_call(a);
  if (mk_status s = attn::check(kMe, own, device)) return s;
  if (static_cast<int64_t>(a.max_prefix_pages) * a.page_size > INT32_MAX - 1024)
    return refuse(MK_ERR_UNSUPPORTED, kMe, "positions beyond 2^31 - 1024");
  if (a.batch == 0) return MK_OK;
  if (!a.prefix_table || !a.prefix_len) return refuse(MK_ERR_INVALID_ARG, kMe, "a required pointer is NULL");
  if (!aligned({a.prefix_table, a.prefix_len, a.lse}, 4) || !aligned(a.workspace, 16))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a misaligned pointer");
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(kMe, guard.err);
  Plan pl;
  if (mk_status s = plan(a, device, &pl)) return s;
  if (!a.workspace || a.workspace_bytes < 0 || static_cast<uint64_t>(a.workspace_bytes) < pl.bytes)
    return refuse(MK_ERR_INVALID_ARG, kMe, "workspace of %lld bytes, %llu needed", static_cast<long long>(a.workspace_bytes),
                  static_cast<unsigned long long>(pl.bytes));
  char* ws = static_cast<char*>(a.workspace);
  p.page = div_by(a.page_size);
  p.group_div = div_by(pl.group);
  p.group = pl.group;
  p.n_rows = pl.n_rows;
  p.blocks = pl.blocks;
  p.block_rows = pl.block_rows;
  p.tile = pl.tile;
  p.ctas = pl.ctas;
  p.max_len = a.max_prefix_pages * a.page_size;
  p.dp = pl.dp;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  attn::cache_steps(a.cache_dtype, a.n_pages, a.n_kv_heads, a.page_size, a.k_page_stride, a.v_page_stride, p.k_step, p.v_step);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_at);
  p.raw = reinterpret_cast<float*>(ws + pl.raw_at);
  p.raw_lse = reinterpret_cast<float*>(ws + pl.lse_at);
  own.workspace = ws + pl.own_at;
  own.workspace_bytes = a.workspace_bytes - static_cast<int64_t>(pl.own_at);
  if (mk_status s = attn::attend(kMe, own, p.raw, p.raw_lse, device, stream)) return s;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MK_BF16, e4m3 = a.cache_dtype == MK_E4M3;
  cudaError_t e = bf ? e4m3 ? launch<__nv_bfloat16, __nv_fp8_e4m3>(p, device, s) : launch<__nv_bfloat16, __nv_bfloat16>(p, device, s)
                     : e4m3 ? launch<__half, __nv_fp8_e4m3>(p, device, s) : launch<__half, __half>(p, device, s);
  const long long results = static_cast<long long>(p.n_rows) * a.n_kv_heads;
  const unsigned grid = static_cast<unsigned>((results + kJoinWarps - 1) / kJoinWarps);
  if (e == cudaSuccess)
    e = bf ? start(join_kernel<__nv_bfloat16>, grid, kJoinWarps * 32, 0, s, p) : start(join_kernel<__half>, grid, kJoinWarps * 32, 0, s, p);
  return launched(kMe, e);
}
