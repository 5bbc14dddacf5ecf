// mk_paged_attention: arguments, the choice of a build, and the second kernel, which joins the parts of requests that
// were cut (paged_attention.cuh has the attention kernel).
#include "paged_attention_tc.cuh"

namespace mkop {
namespace attn {
namespace {

constexpr int kJoinWarps = 8;

// Block (x, y): the request cut at the beginning of piece x + 1, if that is the first cut in it; rows y, y + gridDim.y, ...
// A row's parts are weighted by exp2(maximum - largest maximum). Up to 16 parts: a warp has a row; more: the warps take
// the parts of one row in turn and are summed in a fixed order. Launched so that it may start while the attention kernel
// runs; it waits for that kernel's end before it reads anything (a plain second launch: 1 us more on the GPU).
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p, int dp, int rows_of_block,
                                                             bool scaled) {
  __shared__ float weight[kMaxCtas];
  __shared__ __align__(16) float sums[kJoinWarps][256];
  __shared__ float red[2][kJoinWarps];
  const mk_paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x + 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Piece pc = p.piece[c];
  if (c >= pc.used) return;
  const long long begin = piece_begin(c, pc.total, pc.used), prev = piece_begin(c - 1, pc.total, pc.used);
  if (begin == pc.item0 || prev > pc.item0) return;  // cut between requests, or not the first cut of this one
  // the last piece that begins inside the request: q * total / used < item1
  const int last = static_cast<int>((pc.item1 * pc.used - 1) / pc.total);
  const int n = last - (c - 1) + 1;
  const long long slot0 = 2ll * (c - 1) + (prev == pc.item0 ? 0 : 1);
  auto slot = [&](int k) { return k == 0 ? slot0 : 2ll * (c - 1 + k); };
  const int head = pc.hm / p.blocks, block = pc.hm - head * p.blocks;
  const int rows = min(rows_of_block, p.n_rows - block * rows_of_block);
  if (n <= 16) {
    for (int row = blockIdx.y * kJoinWarps + warp; row < rows; row += gridDim.y * kJoinWarps) {
      const float2 mine = lane < n ? p.part_ml[slot(lane) * rows_of_block + row] : make_float2(-INFINITY, 0.0f);
      float top = mine.x;
#pragma unroll
      for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      top = __shfl_sync(~0u, top, 0);
      const float f = exp2_fast(mine.x - (top == -INFINITY ? 0.0f : top));
      float sum = f * mine.y;
#pragma unroll
      for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      sum = __shfl_sync(~0u, sum, 0);
      const int mrow = block * rows_of_block + row, r = p.group_div(mrow), h = head * p.group + mrow - r * p.group;
      const float scale = sum == 0.0f ? 0.0f : (scaled ? a.v_scale[head] : 1.0f) / sum;
      uint16_t* out = static_cast<uint16_t*>(a.out) + pc.b * a.out_stride[0] + r * a.out_stride[1] + h * a.out_stride[2];
      for (int d0 = 0; d0 < dp; d0 += 128) {
        const int d = min(d0 + lane * 4, dp - 4);  // (64 wide: half of the lanes repeat the last columns)
        float4 y = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(p.part + (slot(k) * rows_of_block + row) * dp + d);
          const float g = __shfl_sync(~0u, f, k);
          y.x += g * x.x, y.y += g * x.y, y.z += g * x.z, y.w += g * x.w;
        }
        if (d < a.head_dim)
          *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(y.x * scale, y.y * scale), pack2<T>(y.z * scale, y.w * scale));
      }
      if (lane == 0 && a.lse)
        a.lse[(static_cast<long long>(pc.b) * a.rows + r) * a.n_q_heads + h] =
            sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    float top = -INFINITY;
    for (int k = tid; k < n; k += kJoinWarps * 32) top = fmaxf(top, p.part_ml[slot(k) * rows_of_block + row].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red[0][w]);
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0;
    for (int k = tid; k < n; k += kJoinWarps * 32) {
      const float2 s = p.part_ml[slot(k) * rows_of_block + row];
      const float f = exp2_fast(s.x - base);
      weight[k] = f;
      sum += f * s.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < kJoinWarps; ++w) sum += red[1][w];
    for (int d = lane * 4; d < dp; d += 128) {
      float4 y = make_float4(0, 0, 0, 0);
#pragma unroll 4
      for (int k = warp; k < n; k += kJoinWarps) {
        const float4 x = *reinterpret_cast<const float4*>(p.part + (slot(k) * rows_of_block + row) * dp + d);
        const float f = weight[k];
        y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
      }
      *reinterpret_cast<float4*>(&sums[warp][d]) = y;
    }
    __syncthreads();
    const int mrow = block * rows_of_block + row, r = mrow / p.group, h = head * p.group + mrow - r * p.group;
    const float f = sum == 0.0f ? 0.0f : (scaled ? a.v_scale[head] : 1.0f) / sum;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + pc.b * a.out_stride[0] +
                                                r * a.out_stride[1] + h * a.out_stride[2]);
    for (int d = 2 * tid; d < a.head_dim; d += 2 * kJoinWarps * 32) {
      float x = 0, y = 0;
      for (int w = 0; w < kJoinWarps; ++w) x += sums[w][d], y += sums[w][d + 1];
      out[d / 2] = pack2<T>(x * f, y * f);
    }
    if (tid == 0 && a.lse)
      a.lse[(static_cast<long long>(pc.b) * a.rows + r) * a.n_q_heads + h] =
          sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
    __syncthreads();
  }
}

const char* const kMe = "mk_paged_attention";

// What follows from the shape fields alone: the build, the grid, the workspace.
struct Plan {
  const Build* build;
  int dp, group, n_rows, blocks, ctas, parts;
  size_t piece_at, ml_at;
  size_t bytes;   // what this call uses
  size_t offer;   // what mk_paged_attention_workspace says: `bytes` or more, so that the largest call's fits smaller ones
};

// The line's grid and workspace with a build.
size_t lay_out(Plan& pl, const Build* build, int sms, int per_sm) {
  pl.build = build;
  pl.ctas = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
  const size_t slots = 2 * static_cast<size_t>(pl.ctas);
  pl.ml_at = slots * build->rows * pl.dp * sizeof(float);
  pl.piece_at = pl.ml_at + slots * build->rows * sizeof(float2);
  return pl.piece_at + pl.ctas * sizeof(Piece);
}

// Small calls: a cluster of up to 16 CTAs, all resident, per (request, kv head, row block) splits its keys evenly and
// joins through distributed shared memory; where there are too many for two CTAs each, one CTA has it alone. No workspace,
// no second launch, no sums over the batch first. It does not balance ragged requests against each other, so it is for
// calls whose CTAs have at most this much to read each, twice that where they are more than fit at once.
// Measured both ways (GPU us, and the host's per call), 128 wide, bf16. One request, 48 / 8 heads: 4096 positions 10.9 (10)
// as clusters, 15.0 (21) as pieces of the line; 8192 (256 KB a CTA) 18.0 and 18; 16384 (512 KB) 30 and 22. One CTA each, 32
// / 8 heads, 60 requests of 10 to 256 positions 18 and 36, to 700 (352 KB) 31 and 49, to 1500 (768 KB) 53 and 62; 150 of
// these 103 and 133; 60 of 8 rows to 700 57 and 102; 256 wide to 700 (704 KB) 42 and 40.
constexpr size_t kClusterBytes = 384 * 1024;

mk_status check_shape(const mk_paged_attention_args& a, int device) {
  if (a.rows < 1 || a.rows > 4096 || a.n_q_heads < 1 || a.n_q_heads > 4096 || a.n_kv_heads < 1 || a.n_q_heads % a.n_kv_heads)
    return refuse(MK_ERR_INVALID_ARG, kMe, "rows %d, heads %d / %d", a.rows, a.n_q_heads, a.n_kv_heads);
  if (a.head_dim < 16 || a.head_dim > 256 || a.head_dim % 16)
    return refuse(MK_ERR_UNSUPPORTED, kMe, "head_dim %d is not a multiple of 16 in 16..256", a.head_dim);
  if (a.dtype != MK_BF16 && a.dtype != MK_F16) return refuse(MK_ERR_UNSUPPORTED, kMe, "dtype %d", a.dtype);
  if (a.cache_dtype != a.dtype && a.cache_dtype != MK_E4M3)
    return refuse(MK_ERR_UNSUPPORTED, kMe, "cache dtype %d with dtype %d", a.cache_dtype, a.dtype);
  return check_device(kMe, device);
}

cudaError_t plan(const mk_paged_attention_args& a, int device, Plan* out) {
  Plan& pl = *out;
  pl.group = a.n_q_heads / a.n_kv_heads;
  pl.n_rows = a.rows * pl.group;
  pl.dp = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
  // Row blocks of up to 64 rows, as equal as whole 16-row tiles allow (80 rows: 48 + 32, not 64 + 16).
  const int tiles = (pl.n_rows + 15) / 16;
  pl.blocks = (tiles + 3) / 4;
  const int mt = (tiles + pl.blocks - 1) / pl.blocks;
  auto pick = [&](bool longer) {
    const bool bf = a.dtype == MK_BF16;
    if (a.cache_dtype == MK_E4M3) return bf ? pick_e4m3_bf16(pl.dp, mt, longer) : pick_e4m3_f16(pl.dp, mt, longer);
    return bf ? pick_bf16(pl.dp, mt, longer) : pick_f16(pl.dp, mt, longer);
  };
  pl.build = pick(false);
  int sms, per_sm;
  cudaError_t e = sm_count(device, &sms);
  if (e == cudaSuccess) e = pl.build->occupancy(device, &per_sm);
  if (e != cudaSuccess) return e;
  pl.ctas = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
  pl.parts = 0;
  pl.ml_at = pl.piece_at = pl.bytes = pl.offer = 0;
  const int64_t items = static_cast<int64_t>(a.batch) * a.n_kv_heads * pl.blocks;
  const int64_t key_tiles = (static_cast<int64_t>(a.max_pages) * a.page_size + pl.build->tile - 1) / pl.build->tile;
  const size_t tile_bytes = 2 * static_cast<size_t>(pl.build->tile) * pl.dp * (a.cache_dtype == MK_E4M3 ? 1 : 2);
  int parts = 1, resident = 0;
  if (key_tiles > kMinTiles)
    for (parts = 16; parts > 1; parts /= 2) {
      if (parts > key_tiles || items * parts > pl.ctas) continue;
      if ((e = pl.build->clusters(device, parts, &resident)) != cudaSuccess) return e;
      if (items <= resident) break;
    }
  const size_t each = static_cast<size_t>((key_tiles + parts - 1) / parts) * tile_bytes;  // a CTA's keys and values
  const size_t most = parts == 1 && items >= pl.ctas ? 2 * kClusterBytes : kClusterBytes;
  const bool small = items * parts < 1 << 24 && each <= most;
  if (!small || each > kClusterBytes) {  // the line, or a batch that would be one with fewer requests
    Plan line = pl;
    const Build* build = pick(true);
    if ((e = build->occupancy(device, &per_sm)) != cudaSuccess) return e;
    pl.offer = line.bytes = lay_out(line, build, sms, per_sm);
    if (a.cache_dtype != MK_E4M3 && (a.head_dim == 128 || a.head_dim == 256) && a.rows <= kTcMaxRows) {
      const int block_rows = pl.blocks == 1 ? pl.n_rows : 16 * mt;
      build = a.dtype == MK_BF16 ? pick_tc_bf16(pl.dp, block_rows) : pick_tc_f16(pl.dp, block_rows);
      if ((e = build->occupancy(device, &per_sm)) != cudaSuccess) return e;
      Plan tc = pl;
      tc.bytes = lay_out(tc, build, sms, per_sm);
      pl.offer = tc.bytes > line.bytes ? tc.bytes : line.bytes;
      // (its CTAs count their tiles in 32 bits)
      if (items * ((static_cast<int64_t>(a.max_pages) * a.page_size >> 7) + 1) < INT32_MAX) line = tc;
    }
    if (!small) {
      line.offer = pl.offer;
      pl = line;
      return cudaSuccess;
    }
  }
  pl.parts = parts;
  pl.ctas = static_cast<int>(items) * parts;
  return cudaSuccess;
}

template <typename T>
cudaError_t join(const Params& p, const Plan& pl, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  // a few rows each, so that the blocks without a cut to join stay few
  const int rows = p.n_rows < pl.build->rows ? p.n_rows : pl.build->rows;
  const int y = 1216 / pl.ctas < 1 ? 1 : 1216 / pl.ctas > rows ? rows : 1216 / pl.ctas;
  cfg.gridDim = dim3(pl.ctas - 1, y);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T>, p, pl.dp, pl.build->rows, p.a.cache_dtype == MK_E4M3);
}

}  // namespace
}  // namespace attn
}  // namespace mkop

extern "C" mk_status mk_paged_attention_workspace(const mk_paged_attention_args* p, int device, uint64_t* bytes) {
  using namespace mkop;
  using namespace mkop::attn;
  if (!p || !bytes) return MK_ERR_INVALID_ARG;
  if (mk_status s = check_shape(*p, device)) return s;
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(kMe, guard.err);
  Plan pl;
  if (const cudaError_t e = plan(*p, device, &pl)) return launched(kMe, e);
  *bytes = pl.offer;
  return MK_OK;
}

extern "C" mk_status mk_paged_attention(const mk_paged_attention_args* args, int device, void* stream) {
  using namespace mkop;
  using namespace mkop::attn;
  if (!args) return MK_ERR_INVALID_ARG;
  Params p{};
  p.a = *args;
  const mk_paged_attention_args& a = p.a;
  const bool e4m3 = a.cache_dtype == MK_E4M3;
  if (a.batch < 0 || a.batch > 1 << 24 || a.n_pages < 1 || a.page_size < 1 || a.max_pages < 1)
    return refuse(MK_ERR_INVALID_ARG, kMe, "batch %d, n_pages %d, page_size %d, max_pages %d", a.batch, a.n_pages,
                  a.page_size, a.max_pages);
  // a tile may end past max_len, so that leaves room below 2^31
  if (static_cast<int64_t>(a.max_pages) * a.page_size > INT32_MAX - 1024)
    return refuse(MK_ERR_UNSUPPORTED, kMe, "positions beyond 2^31 - 1024");
  if (mk_status s = check_shape(a, device)) return s;
  if (a.batch == 0) return MK_OK;
  if (!a.q || !a.k_pages || !a.v_pages || !a.table || !a.lens || !a.out || (e4m3 && (!a.k_scale || !a.v_scale)))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a required pointer is NULL");
  if (a.table_stride < a.max_pages) return refuse(MK_ERR_INVALID_ARG, kMe, "table rows shorter than max_pages");
  if (!aligned({a.q, a.k_pages, a.v_pages, a.out, a.workspace}, 16))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a pointer is not 16-byte aligned");
  if (!aligned({a.table, a.lens, a.k_scale, a.v_scale, a.lse, a.status}, 4))
    return refuse(MK_ERR_INVALID_ARG, kMe, "a misaligned pointer");
  // the stride of a dimension of one element is never used
  const int q_size[3] = {a.batch, a.rows, a.n_q_heads}, page_dims[3] = {a.n_pages, a.n_kv_heads, a.page_size};
  for (int i = 0; i < 3; ++i) {
    if (q_size[i] > 1 && (a.q_stride[i] % 8 || a.out_stride[i] % 8))
      return refuse(MK_ERR_INVALID_ARG, kMe, "a stride is not a multiple of 8 elements");
    if (page_dims[i] > 1 && (a.k_page_stride[i] % (e4m3 ? 16 : 8) || a.v_page_stride[i] % (e4m3 ? 16 : 8)))
      return refuse(MK_ERR_INVALID_ARG, kMe, "a cache stride is not a multiple of 16 bytes");
    const int64_t k = page_dims[i] > 1 ? a.k_page_stride[i] : 0, v = page_dims[i] > 1 ? a.v_page_stride[i] : 0;
    const int64_t unit = e4m3 ? 16 : 8;  // elements of 16 bytes
    if (k < 0 || k / unit > UINT32_MAX || v < 0 || v / unit > UINT32_MAX)
      return refuse(MK_ERR_UNSUPPORTED, kMe, "a cache stride is negative or 64 GB and more");
    p.k_step[i] = static_cast<uint32_t>(k / unit);
    p.v_step[i] = static_cast<uint32_t>(v / unit);
  }
  DeviceGuard guard(device);
  if (guard.err != cudaSuccess) return launched(kMe, guard.err);
  Plan pl;
  if (const cudaError_t e = plan(a, device, &pl)) return launched(kMe, e);
  if (pl.bytes && (!a.workspace || a.workspace_bytes < static_cast<int64_t>(pl.bytes)))
    return refuse(MK_ERR_INVALID_ARG, kMe, "workspace of %lld bytes, %zu needed", static_cast<long long>(a.workspace_bytes), pl.bytes);
  char* ws = static_cast<char*>(a.workspace);
  p.page = div_by(a.page_size);
  p.group_div = div_by(pl.group);
  p.group = pl.group;
  p.parts = pl.parts;
  p.n_rows = pl.n_rows;
  p.blocks = pl.blocks;
  p.max_len = a.max_pages * a.page_size;
  p.ctas = pl.ctas;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml_at);
  p.piece = reinterpret_cast<Piece*>(ws + pl.piece_at);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = pl.build->launch(p, s);
  if (e == cudaSuccess && !pl.parts && pl.ctas > 1) e = a.dtype == MK_BF16 ? join<__nv_bfloat16>(p, pl, s) : join<__half>(p, pl, s);
  return launched(kMe, e);
}
