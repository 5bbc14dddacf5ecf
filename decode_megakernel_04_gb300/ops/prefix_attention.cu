// mk_prefix_attention: attention of a batch over a prefix that its requests share and over each request's own positions: the
// arguments, and the second kernel, which joins a row's parts (prefix_attention.cuh has the first).
#include "prefix_attention.cuh"

namespace mkop {
namespace prefix {
namespace {

constexpr int kJoinWarps = 8;

// W warps for each row of out: its parts over the prefix and over its own keys, weighted by exp2(base - largest base). (Launched
// early, to wait for the first kernel's end by itself, it cost that kernel a microsecond: 13.5 us instead of 12.3 for a short call.)
template <typename T, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ float4 part_sums[kJoinWarps][32];
  const mk_prefix_attention_args& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  const int row = blockIdx.x * (kJoinWarps / W) + warp / W;
  const int br = p.q_head_div(row), h = row - br * a.n_q_heads, head = p.group_div(h), m = br * p.group + h - head * p.group;
  const int b = p.row_div(br), r = br - b * a.rows;
  if (br >= a.batch * a.rows) return;  // (W = 8: the whole CTA)
  const Head& hd = *p.head;
  // Parts 0 .. n0 - 1 are over the prefix, n0 .. n - 1 over own keys. Part k of either is place0 + k / subs, stream k % subs (of a
  // pair: its own stream).
  const int pairs = p.blocks[kPairs], line = pairs && m < p.first_single() ? kPairs : kSingles;
  const int in_line = line == kPairs ? m : m - p.first_single(), per_block = line == kPairs ? 2 * kTileRows : kTileRows;
  const int block = in_line / per_block, in_block = in_line - block * per_block;
  const int subs = line == kSingles ? p.streams : 1, own_subs = p.streams;
  const long long item = static_cast<long long>(head) * p.blocks[line] + block;
  long long place0 = item, own0 = 0;
  int n0 = 0, n1 = 0;
  if (hd.total[line]) {
    const int c0 = Head::piece_of(item * hd.tiles, hd.total[line], hd.used[line]);
    n0 = (Head::piece_of((item + 1) * hd.tiles - 1, hd.total[line], hd.used[line]) - c0 + 1) * subs;
    place0 += c0 + (line == kSingles ? hd.used[kPairs] + static_cast<long long>(a.n_kv_heads) * pairs : 0);
  }
  const int group = r / kGroupRows, bg = b * p.groups + group, own_m = (r - group * kGroupRows) * p.group + h - head * p.group;
  const int own_row = own_m % kTileRows;
  const long long cum = p.cum[bg], own_n = p.cum[bg + 1] - cum;
  if (own_n) {
    const int per = a.n_kv_heads * p.blocks[kOwn], hm = head * p.blocks[kOwn] + own_m / kTileRows;
    const long long x = cum * per + hm * own_n;
    const int c0 = Head::piece_of(x + kItemTiles, hd.total[kOwn], hd.used[kOwn]);
    n1 = (Head::piece_of(x + own_n - 1, hd.total[kOwn], hd.used[kOwn]) - c0 + 1) * own_subs;
    own0 = c0 + static_cast<long long>(bg) * per + hm;
  }
  const int n = n0 + n1;
  // the index of a part's row, and whether it is over own keys
  auto at = [&](int k) -> long long {
    if (k >= n0) return (own0 * own_subs + (k - n0)) * p.own_rows + own_row;
    return (subs == p.streams ? place0 * p.streams + k : (place0 + k) * p.streams + in_block / kTileRows) * kTileRows + in_block % kTileRows;
  };
  auto ml_of = [&](int k) { return (k < n0 ? p.part_ml : p.own_ml)[at(k)]; };
  // A lane has a part: its base, its sum, where its row is. (Up to 32 are kept; more are read again.)
  float2 mine = lane < n ? ml_of(lane) : make_float2(-INFINITY, 0.0f);
  const float* from = lane < n ? (lane < n0 ? p.part : p.own) + at(lane) * p.dp : p.part;
  float top = mine.x;
  for (int k = lane + 32; k < n; k += 32) top = fmaxf(top, ml_of(k).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  const float base = top == -INFINITY ? 0.0f : top;
  const float vs = a.cache_dtype == MK_E4M3 ? a.v_scale[head] : 1.0f;
  T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + r * a.out_stride[1] + h * a.out_stride[2];
  float sum = 0;
#pragma unroll 1
  for (int d0 = 0; d0 < a.head_dim; d0 += 128) {
    const int d = min(d0 + lane * 4, p.dp - 4);  // (64 wide: half of the lanes repeat the last columns)
    float4 y = make_float4(0, 0, 0, 0);
    sum = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 32) {
      if (n > 32) {
        const int k = k0 + lane;
        mine = k < n ? ml_of(k) : make_float2(-INFINITY, 0.0f);
        from = k < n ? (k < n0 ? p.part : p.own) + at(k) * p.dp : p.part;
      }
      const float weight = exp2_fast(mine.x - base);
      sum += weight * mine.y;
      // (an empty part has no sums: its weight is 0 and its row is not read)
      const unsigned there = __ballot_sync(~0u, !(mine.y == 0.0f));
      constexpr int kFlight = 6;
#pragma unroll 1
      for (int k1 = w; k1 < min(32, n - k0); k1 += W * kFlight) {
        float4 x[kFlight];
        float f[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int k = min(k1 + i * W, 31);
          f[i] = __shfl_sync(~0u, weight, k);
          const float* x_at = reinterpret_cast<const float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(from), k));
          x[i] = make_float4(0, 0, 0, 0);
          if (k1 + i * W < 32 && there >> k & 1) x[i] = *reinterpret_cast<const float4*>(x_at + d);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) y.x += f[i] * x[i].x, y.y += f[i] * x[i].y, y.z += f[i] * x[i].z, y.w += f[i] * x[i].w;
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if (W > 1) {
      __syncthreads();
      part_sums[warp][lane] = y;
      __syncthreads();
      if (w == 0)
        for (int k = 1; k < W; ++k) {
          const float4 x = part_sums[warp + k][lane];
          y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
        }
    }
    if (w == 0) {
      const float scale = sum == 0.0f ? 0.0f : vs / sum;
      y.x *= scale, y.y *= scale, y.z *= scale, y.w *= scale;
      if (d0 + lane * 4 < a.head_dim) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
    }
  }
  if (w == 0 && lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

const char* const kMe = "mk_prefix_attention";

// The same call of mk_paged_attention over own positions alone: most refusals are its.
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
  int group, n_rows, dp, streams, blocks[3], groups, own_rows, ctas;
  uint64_t ml_at, own_at, own_ml_at, head_at, cum_at, bytes;
};

mk_status check_shape(const mk_prefix_attention_args& a, int device) {
  if (a.batch < 0 || a.max_prefix_pages < 1)
    return refuse(MK_ERR_INVALID_ARG, kMe, "batch %d, max_prefix_pages %d", a.batch, a.max_prefix_pages);
  if (mk_status s = attn::check_shape(kMe, own_call(a), device)) return s;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * a.rows * (a.n_q_heads / a.n_kv_heads);
  if (n_rows * a.n_kv_heads > INT32_MAX - 64) return refuse(MK_ERR_UNSUPPORTED, kMe, "2^31 rows and more");
  if (n_rows > 1 << 24) return refuse(MK_ERR_UNSUPPORTED, kMe, "%lld query rows of a kv head", static_cast<long long>(n_rows));
  return MK_OK;
}

// check_shape() has passed
mk_status plan(const mk_prefix_attention_args& a, int device, Plan* out) {
  Plan& pl = *out;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(kMe, guard.err);
  if (const cudaError_t e = sm_count(device, &pl.ctas)) return launched(kMe, e);
  pl.group = a.n_q_heads / a.n_kv_heads;
  pl.n_rows = a.batch * a.rows * pl.group;
  pl.dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
  pl.streams = pl.dp == 256 ? 1 : 2;
  const int tiles = (pl.n_rows + kTileRows - 1) / kTileRows, own = (a.rows < kGroupRows ? a.rows : kGroupRows) * pl.group;
  pl.blocks[kPairs] = pl.streams == 2 ? tiles / 2 : 0;
  pl.blocks[kSingles] = tiles - 2 * pl.blocks[kPairs];
  pl.blocks[kOwn] = (own + kTileRows - 1) / kTileRows;
  pl.groups = (a.rows + kGroupRows - 1) / kGroupRows;
  pl.own_rows = own < kTileRows ? own : kTileRows;
  const uint64_t kv = a.n_kv_heads, groups = static_cast<uint64_t>(a.batch) * pl.groups;
  const uint64_t rows = (pl.ctas + kv * (pl.blocks[kPairs] + pl.blocks[kSingles])) * pl.streams * kTileRows;
  const uint64_t own_rows = (pl.ctas + groups * kv * pl.blocks[kOwn]) * pl.streams * pl.own_rows;
  auto whole = [](uint64_t n) { return (n + 255) / 256 * 256; };
  pl.ml_at = whole(rows * pl.dp * sizeof(float));
  pl.own_at = pl.ml_at + whole(rows * sizeof(float2));
  pl.own_ml_at = pl.own_at + whole(own_rows * pl.dp * sizeof(float));
  pl.head_at = pl.own_ml_at + whole(own_rows * sizeof(float2));
  pl.cum_at = pl.head_at + whole(sizeof(Head));
  // the first kernel stores sums by 32 bytes: places begin at the workspace's first 32-byte boundary
  pl.bytes = pl.cum_at + whole((groups + 1) * sizeof(long long)) + 16;
  return MK_OK;
}

template <typename T, int W>
cudaError_t join(const PrefixParams& p, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.n_rows) * p.a.n_kv_heads;
  return start(join_kernel<T, W>, static_cast<unsigned>((rows * W + kJoinWarps - 1) / kJoinWarps), kJoinWarps * 32, 0, s, p);
}
template <typename T>
cudaError_t join(const PrefixParams& p, cudaStream_t s) {
  // Few rows of many parts: 8 warps each.
  const long long rows = static_cast<long long>(p.n_rows) * p.a.n_kv_heads;
  return rows * 8 <= 16 * p.ctas * kJoinWarps ? join<T, 8>(p, s) : join<T, 1>(p, s);
}

}  // namespace

cudaError_t map_cache(CUtensorMap* map, const void* pages, const mk_prefix_attention_args& a, const int64_t* strides, int rows, bool e4m3) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  const int size = e4m3 ? 1 : 2;
  const int order[3] = {2, 1, 0};  // place, head, page
  const int counts[3] = {a.n_pages, a.n_kv_heads, a.page_size};
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim)}, steps[3];
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = counts[order[i]];
    // (a dimension of one element has no stride, but one is asked for)
    steps[i] = counts[order[i]] > 1 ? strides[order[i]] * size : 16;
  }
  const cuuint32_t box[4] = {e4m3 ? 128u : 64u, static_cast<cuuint32_t>(rows), 1, 1}, ones[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(pages), dims,
                            steps, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

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
  PrefixParams p{};
  p.a = *args;
  const mk_prefix_attention_args& a = p.a;
  if (mk_status s = check_shape(a, device)) return s;
  if (mk_status s = attn::check(kMe, own_call(a), device)) return s;
  const int counts[3] = {a.n_pages, a.n_kv_heads, a.page_size};
  for (int i = 0; i < 3; ++i)
    if (counts[i] > 1 && (a.k_page_stride[i] == 0 || a.v_page_stride[i] == 0))  // (not as a copied box's tensor)
      return refuse(MK_ERR_UNSUPPORTED, kMe, "a cache stride of 0");
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
  char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(a.workspace) + 31) & ~uintptr_t{31});
  p.page = div_by(a.page_size);
  p.group_div = div_by(pl.group);
  p.group = pl.group;
  p.n_rows = pl.n_rows;
  p.row_div = div_by(a.rows);
  p.q_head_div = div_by(a.n_q_heads);
  p.max_prefix = a.max_prefix_pages * a.page_size;
  p.max_own = a.max_pages * a.page_size;
  p.dp = pl.dp;
  p.streams = pl.streams;
  for (int i = 0; i < 3; ++i) {
    p.blocks[i] = pl.blocks[i];
    p.block_div[i] = div_by(pl.blocks[i] ? pl.blocks[i] : 1);
  }
  p.groups = pl.groups;
  p.groups_div = div_by(pl.groups);
  p.own_rows = pl.own_rows;
  p.ctas = pl.ctas;
  p.scale_log2 = fabsf(a.scale) * 1.44269504088896340736f;
  p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
  cache_steps(a.cache_dtype, a.n_pages, a.n_kv_heads, a.page_size, a.k_page_stride, a.v_page_stride, p.k_step, p.v_step);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_at);
  p.own = reinterpret_cast<float*>(ws + pl.own_at);
  p.own_ml = reinterpret_cast<float2*>(ws + pl.own_ml_at);
  p.head = reinterpret_cast<Head*>(ws + pl.head_at);
  p.cum = reinterpret_cast<long long*>(ws + pl.cum_at);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MK_BF16, e4m3 = a.cache_dtype == MK_E4M3;
  cudaError_t e = e4m3 ? bf ? launch_prefix_e4m3_bf16(p, device, s) : launch_prefix_e4m3_f16(p, device, s)
                       : bf ? launch_prefix_bf16(p, device, s) : launch_prefix_f16(p, device, s);
  if (e == cudaSuccess) e = bf ? join<__nv_bfloat16>(p, s) : join<__half>(p, s);
  return launched(kMe, e);
}
