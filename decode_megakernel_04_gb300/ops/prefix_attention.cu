// mk_prefix_attention: attention of a batch over a prefix that its requests share and over each request's own positions.
//
// One softmax over both, joined from parts: own positions by mk_paged_attention (results and their log-sums in fp32), the
// prefix once for all query rows of a kv head (prefix_attention.cuh), cut along its keys, and a last kernel that weights the
// parts of a row.
#include "prefix_attention.cuh"

namespace mkop {
namespace prefix {
namespace {

constexpr int kJoinWarps = 8;

// W warps for each row of out: the parts of the prefix and the result over the own positions, weighted by exp2(base - largest
// base). Launched so that it may start while the prefix's kernel runs; it waits for that kernel's end, which waits for what
// came before it.
template <typename T, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ float4 part_sums[kJoinWarps][32];
  __shared__ float part_sum[kJoinWarps];
  const mk_prefix_attention_args& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  const long long row = static_cast<long long>(blockIdx.x) * (kJoinWarps / W) + warp / W;
  const bool there = row < static_cast<long long>(a.batch) * a.rows * a.n_q_heads;  // (W = 8: the whole CTA)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!there) return;
  const int br = static_cast<int>(row / a.n_q_heads), h = static_cast<int>(row - static_cast<long long>(br) * a.n_q_heads);
  const int head = h / p.group, m = br * p.group + h - head * p.group;
  const int b = br / a.rows, r = br - b * a.rows;
  // the places of this row's sums: part k is place0 + k / subs, stream k % subs (or the row tile's own)
  const int which = p.lane[1].blocks && m >= p.lane[1].first_row;
  const Lane& ln = p.lane[which];
  const int block = (m - ln.first_row) / ln.rows, in_block = m - ln.first_row - block * ln.rows;
  const int subs = which ? p.streams : 1, stream = in_block / kTileRows, tile_row = in_block % kTileRows;
  const Line line(p, ln);
  const long long item = static_cast<long long>(head) * ln.blocks + block;
  long long place0 = 0;
  int n = 0;
  if (line.total) {
    const int c0 = line.piece_of(item * line.tiles);
    n = (line.piece_of((item + 1) * line.tiles - 1) - c0 + 1) * subs;
    place0 = ln.place0 + c0 + item;
  }
  auto at = [&](int k) {
    return ((place0 + (subs == 2 ? k >> 1 : k)) * p.streams + (subs == 2 ? k & 1 : stream)) * kTileRows + tile_row;
  };
  const float own = p.raw_lse[row];
  float top = own;
  for (int k = lane; k < n; k += 32) top = fmaxf(top, p.part_ml[at(k)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  const float base = top == -INFINITY ? 0.0f : top;
  const float f_own = exp2_fast(own - base), vs = a.cache_dtype == MK_E4M3 ? a.v_scale[head] : 1.0f;
  T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + r * a.out_stride[1] + h * a.out_stride[2];
  float sum = 0;
#pragma unroll 1
  for (int d0 = 0; d0 < a.head_dim; d0 += 128) {
    const int d = min(d0 + lane * 4, p.dp - 4);  // (64 wide: half of the lanes repeat the last columns)
    float4 y = make_float4(0, 0, 0, 0);
    sum = 0;
#pragma unroll 4
    for (int k = w; k < n; k += W) {
      const float2 ml = p.part_ml[at(k)];
      const float f = exp2_fast(ml.x - base);
      sum += f * ml.y;
      if (ml.y == 0.0f) continue;  // an empty part has no sums
      const float4 x = *reinterpret_cast<const float4*>(p.part + at(k) * p.dp + d);
      y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
    }
    if (W > 1) {
      __syncthreads();
      part_sums[warp][lane] = y;
      if (lane == 0) part_sum[warp] = sum;
      __syncthreads();
      if (w == 0)
        for (int k = 1; k < W; ++k) {
          const float4 x = part_sums[warp + k][lane];
          y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
          sum += part_sum[warp + k];
        }
    }
    if (w == 0) {
      sum += f_own;
      const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
      float4 x = make_float4(0, 0, 0, 0);
      if (f_own != 0.0f && d < a.head_dim) x = *reinterpret_cast<const float4*>(p.raw + row * p.dp + d);
      y.x = (y.x * vs + f_own * x.x) * scale, y.y = (y.y * vs + f_own * x.y) * scale;
      y.z = (y.z * vs + f_own * x.z) * scale, y.w = (y.w * vs + f_own * x.w) * scale;
      if (d0 + lane * 4 < a.head_dim) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
    }
  }
  if (w == 0 && lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
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
  int group, n_rows, dp, streams;
  Lane lane[2];
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
  pl.streams = pl.dp == 256 ? 1 : 2;
  int sms;
  if (const cudaError_t e = sm_count(device, &sms)) return launched(kMe, e);
  // Pairs of row tiles and single ones, their CTAs in proportion to their products.
  const int tiles = (pl.n_rows + kTileRows - 1) / kTileRows, pairs = pl.streams == 2 ? tiles / 2 : 0, singles = tiles - 2 * pairs;
  int ctas = pairs == 0 ? 0 : singles == 0 ? sms : (sms * 2 * pairs + pairs) / (2 * pairs + singles);
  if (pairs && singles && ctas > sms - 1) ctas = sms - 1;
  pl.lane[0] = {ctas, pairs, 0, 2 * kTileRows, 0};
  pl.lane[1] = {singles ? sms - ctas : 0, singles, 2 * pairs * kTileRows, kTileRows, ctas + a.n_kv_heads * pairs};
  const uint64_t places = sms + static_cast<uint64_t>(a.n_kv_heads) * (pairs + singles), results = static_cast<uint64_t>(pl.n_rows) * a.n_kv_heads;
  auto whole = [](uint64_t n) { return (n + 255) / 256 * 256; };
  const uint64_t rows = places * pl.streams * kTileRows;
  pl.ml_at = whole(rows * pl.dp * sizeof(float));
  pl.raw_at = pl.ml_at + whole(rows * sizeof(float2));
  pl.lse_at = pl.raw_at + whole(results * pl.dp * sizeof(float));
  pl.own_at = pl.lse_at + whole(results * sizeof(float));
  pl.bytes = pl.own_at + own;
  return MK_OK;
}

template <typename T, int W>
cudaError_t join(const PrefixParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  const long long rows = static_cast<long long>(p.n_rows) * p.a.n_kv_heads;
  cfg.gridDim = dim3(static_cast<unsigned>((rows * W + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, W>, p);
}
template <typename T>
cudaError_t join(const PrefixParams& p, cudaStream_t s) {
  // a row has about this many parts at most
  const int parts = (p.lane[0].ctas + p.lane[1].ctas) * p.streams / (p.a.n_kv_heads * (p.lane[0].blocks + p.lane[1].blocks)) + 1;
  return parts > 8 ? join<T, 8>(p, s) : join<T, 1>(p, s);
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
  PrefixParams p{};
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
  p.row_div = div_by(a.rows);
  p.streams = pl.streams;
  p.lane[0] = pl.lane[0];
  p.lane[1] = pl.lane[1];
  p.max_len = a.max_prefix_pages * a.page_size;
  p.dp = pl.dp;
  p.scale_log2 = fabsf(a.scale) * 1.44269504088896340736f;
  p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
  cache_steps(a.cache_dtype, a.n_pages, a.n_kv_heads, a.page_size, a.k_page_stride, a.v_page_stride, p.k_step, p.v_step);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_at);
  p.raw = reinterpret_cast<float*>(ws + pl.raw_at);
  p.raw_lse = reinterpret_cast<float*>(ws + pl.lse_at);
  own.workspace = ws + pl.own_at;
  own.workspace_bytes = a.workspace_bytes - static_cast<int64_t>(pl.own_at);
  if (mk_status s = attend(kMe, own, p.raw, p.raw_lse, device, stream)) return s;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MK_BF16, e4m3 = a.cache_dtype == MK_E4M3;
  cudaError_t e = e4m3 ? bf ? launch_prefix_e4m3_bf16(p, device, s) : launch_prefix_e4m3_f16(p, device, s)
                       : bf ? launch_prefix_bf16(p, device, s) : launch_prefix_f16(p, device, s);
  if (e == cudaSuccess) e = bf ? join<__nv_bfloat16>(p, s) : join<__half>(p, s);
  return launched(kMe, e);
}
