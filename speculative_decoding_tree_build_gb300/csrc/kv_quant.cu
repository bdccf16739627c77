// tv_kv_quant_append and tv_kv_quant_read: rows written into the 8-bit paged
// KV cache and read back into bf16 pools.
//
// A row (one head's D values of one token) is quantised on its own: largest
// magnitude, scale, codes (tv_kv8.cuh). Both calls are bound by memory: the
// append reads 2 D bytes a row and writes D + 4, the read the other way round.
// A row is held by D / 8 neighbouring lanes, 16 bytes of bf16 each; its
// largest magnitude takes log2(D / 8) shuffles of an integer maximum.
#include "tv_kv8.cuh"

namespace tv {

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;       // rows of k_new / v_new per CTA

struct AppendParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  long long kv_ld;
  const int32_t* cu_rows;
  const int32_t* start_len;
  const int32_t* block_table;
  const int32_t* n_blocks;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  int32_t* status;
  int batch, rows, hkv, max_blocks, num_blocks;
};

// The request that owns row t: the largest b with cu[b] <= t (requests without
// rows are passed over), -1 when t is outside [cu[0], cu[batch]).
__device__ __forceinline__ int request_of_row(const int32_t* cu, int batch, int t) {
  if (t < cu[0] || t >= cu[batch]) return -1;
  int lo = 0, hi = batch;              // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <int kFmt, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_quant_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;        // lanes that hold one row
  __shared__ int s_cu[kKvMaxBatch + 1];
  __shared__ int s_req[kAppendRows], s_slot[kAppendRows], s_blk[kAppendRows], s_bad[kAppendRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * kAppendRows;
  const int nrows = min(kAppendRows, p.rows - t0);
  for (int i = threadIdx.x; i <= p.batch; i += blockDim.x) s_cu[i] = p.cu_rows[i];
  __syncthreads();
  if (threadIdx.x < kAppendRows) {
    const int r = threadIdx.x;
    const int b = r < nrows ? request_of_row(s_cu, p.batch, t0 + r) : -1;
    s_req[r] = b;
    s_bad[r] = 0;
    s_blk[r] = -1;
    if (b >= 0) {
      const int start = p.start_len[b];
      const long long slot = static_cast<long long>(start) + (t0 + r - s_cu[b]);
      if (p.status[b] != 0) {
        s_bad[r] = -1;                                       // skipped, nothing to report
      } else if (start < 0 || s_cu[b] < 0 || s_cu[b + 1] > p.rows || slot > 0x7fffffffll) {
        s_bad[r] = TV_ST_BAD_SIZE;
      }
      s_slot[r] = static_cast<int>(slot);
    }
  }
  __syncthreads();
  // every block of a request's written slots has to be held and in range
  for (int r = 0; r < nrows; ++r) {
    const int b = s_req[r];
    if (b < 0 || s_bad[r] != 0) continue;
    if (r > 0 && s_req[r - 1] == b) continue;
    const long long first = p.start_len[b];
    const long long last = first + (s_cu[b + 1] - s_cu[b]) - 1;
    const int held = min(p.n_blocks[b], p.max_blocks);
    int bad = last / TV_BLOCK_SIZE >= held ? 1 : 0;
    if (!bad) {
      const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
      for (int e = static_cast<int>(first / TV_BLOCK_SIZE) + threadIdx.x; e <= last / TV_BLOCK_SIZE; e += blockDim.x) {
        const int blk = row[e];
        bad |= (blk < 0 || blk >= p.num_blocks) ? 1 : 0;
      }
    }
    if (bad) s_bad[r] = TV_ST_BAD_BLOCK;
  }
  __syncthreads();
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x, b = s_req[r];
    if (b >= 0) {
      int head = r;                                          // the run's first row holds the verdict
      while (head > 0 && s_req[head - 1] == b) --head;
      const int bad = s_bad[head];
      if (bad > 0 && head == r) atomicOr(p.status + b, bad);
      if (bad == 0) s_blk[r] = p.block_table[static_cast<size_t>(b) * p.max_blocks + s_slot[r] / TV_BLOCK_SIZE];
    }
  }
  __syncthreads();
  const int per_row = 2 * p.hkv;                             // K heads, then V heads
  const int lane = threadIdx.x % kLanes;
  const int total = nrows * per_row;
  // whole groups of kLanes threads take an item, so the shuffles have all of their lanes
  for (int it = threadIdx.x / kLanes; it < (total + 32 / kLanes - 1) / (32 / kLanes) * (32 / kLanes);
       it += blockDim.x / kLanes) {
    const bool live = it < total;
    const int r = live ? it / per_row : 0, kvh = live ? it % per_row : 0;
    const bool isv = kvh >= p.hkv;
    const int h = isv ? kvh - p.hkv : kvh;
    const int blk = live ? s_blk[r] : -1;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (blk >= 0)
      x = *reinterpret_cast<const uint4*>((isv ? p.v_new : p.k_new) + (t0 + r) * p.kv_ld +
                                          static_cast<long long>(h) * D + lane * 8);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
    if (blk < 0) continue;
    const KvRowScale sc = kv_row_scale<kFmt>(top);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = kv_encode2<kFmt>(bf16_lo(w[e]), bf16_hi(w[e]), sc);
    const size_t row = (static_cast<size_t>(blk) * p.hkv + h) * TV_BLOCK_SIZE + s_slot[r] % TV_BLOCK_SIZE;
    *reinterpret_cast<uint2*>((isv ? p.v_cache : p.k_cache) + row * D + lane * 8) =
        make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    if (lane == 0) (isv ? p.v_scale : p.k_scale)[row] = sc.scale;
  }
}

// ------------------------------------------------------------------ read back

constexpr int kReadThreads = 256;

struct ReadParams {
  const int32_t* first;
  const int32_t* last;
  const int32_t* block_table;
  const int32_t* n_blocks;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* out_table;
  const int32_t* out_n_blocks;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* status;
  int batch, hkv, max_blocks, num_blocks, out_max_blocks, out_num_blocks;
};

template <int kFmt, int D>
__global__ void __launch_bounds__(kReadThreads) kv_quant_read_kernel(const __grid_constant__ ReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.y;
  const int st = p.status[b];
  const int first = p.first ? p.first[b] : 0, last = p.last[b];
  if (st != 0) return;
  if (first < 0 || last < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status + b, TV_ST_BAD_SIZE);
    return;
  }
  if (last <= first) return;
  const int page0 = first / TV_BLOCK_SIZE, page1 = (last - 1) / TV_BLOCK_SIZE;
  if (static_cast<long long>(page0) + blockIdx.x > page1 && blockIdx.x != 0) return;
  const int32_t* from = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const int32_t* to = p.out_table + static_cast<size_t>(b) * p.out_max_blocks;
  int bad = page1 >= min(p.n_blocks[b], p.max_blocks) || page1 >= min(p.out_n_blocks[b], p.out_max_blocks);
  if (!bad) {
    for (int e = page0 + threadIdx.x; e <= page1; e += blockDim.x) {
      const int s = from[e], d = to[e];
      bad |= s < 0 || s >= p.num_blocks || d < 0 || d >= p.out_num_blocks;
    }
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status + b, TV_ST_BAD_BLOCK);
    return;
  }
  constexpr int kVecs = TV_BLOCK_SIZE * D / 16;              // 16-byte vectors of codes of a page's head
  for (int page = page0 + blockIdx.x; page <= page1; page += gridDim.x) {
    const size_t sblk = from[page], dblk = to[page];
    for (int i = threadIdx.x; i < 2 * p.hkv * kVecs; i += blockDim.x) {
      const bool isv = i >= p.hkv * kVecs;
      const int e = isv ? i - p.hkv * kVecs : i;
      const int h = e / kVecs, row = e % kVecs / (D / 16), vec = e % (D / 16);
      const int slot = page * TV_BLOCK_SIZE + row;
      if (slot < first || slot >= last) continue;
      const size_t srow = (sblk * p.hkv + h) * TV_BLOCK_SIZE + row;
      const uint4 c = *reinterpret_cast<const uint4*>((isv ? p.v_cache : p.k_cache) + srow * D + vec * 16);
      const float sc = (isv ? p.v_scale : p.k_scale)[srow];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = kv_decode2<kFmt>(w[j] & 0xffffu), hi = kv_decode2<kFmt>(w[j] >> 16);
        o[2 * j] = pack_bf16x2(lo.x * sc, lo.y * sc);
        o[2 * j + 1] = pack_bf16x2(hi.x * sc, hi.y * sc);
      }
      uint4* dst = reinterpret_cast<uint4*>((isv ? p.v_out : p.k_out) +
                                            ((dblk * p.hkv + h) * TV_BLOCK_SIZE + row) * D + vec * 16);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

static int check_kv_format(int fmt) {
  return fmt == TV_KV_E4M3 || fmt == TV_KV_INT8 ? TV_OK : TV_ERR_BAD_GEOMETRY;
}

}  // namespace tv

extern "C" int tv_kv_quant_append(const tv_geom* geom, int32_t kv_format, int32_t batch,
                                  int32_t rows, const void* k_new, const void* v_new,
                                  int64_t kv_ld, const int32_t* cu_rows, const int32_t* start_len,
                                  const int32_t* block_table, const int32_t* n_blocks,
                                  int32_t max_blocks_per_req, void* k_cache, void* v_cache,
                                  float* k_scale, float* v_scale, int32_t num_blocks,
                                  int32_t* status, void* stream) {
  int rc = tv::check_geom(geom);
  if (rc != TV_OK) return rc;
  rc = tv::check_kv_format(kv_format);
  if (rc != TV_OK) return rc;
  if (batch < 0 || batch > tv::kKvMaxBatch || rows < 0 || max_blocks_per_req < 1 || num_blocks < 1 ||
      kv_ld < static_cast<long long>(geom->num_kv_heads) * geom->head_dim)
    return TV_ERR_BAD_SIZE;
  if (batch == 0 || rows == 0) return TV_OK;
  if (!k_new || !v_new || !cu_rows || !start_len || !block_table || !n_blocks || !k_cache ||
      !v_cache || !k_scale || !v_scale || !status)
    return TV_ERR_NULL_POINTER;
  if (!tv::aligned(k_new, 16) || !tv::aligned(v_new, 16) || kv_ld % 8 != 0 ||
      !tv::aligned(k_cache, 16) || !tv::aligned(v_cache, 16) || !tv::aligned(k_scale, 4) ||
      !tv::aligned(v_scale, 4))
    return TV_ERR_MISALIGNED;
  tv::AppendParams p = {};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.kv_ld = kv_ld;
  p.cu_rows = cu_rows; p.start_len = start_len; p.block_table = block_table; p.n_blocks = n_blocks;
  p.k_cache = static_cast<uint8_t*>(k_cache); p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale; p.status = status;
  p.batch = batch; p.rows = rows; p.hkv = geom->num_kv_heads; p.max_blocks = max_blocks_per_req;
  p.num_blocks = num_blocks;
  auto* kernel = kv_format == TV_KV_E4M3
      ? (geom->head_dim == 64 ? tv::kv_quant_append_kernel<TV_KV_E4M3, 64> : tv::kv_quant_append_kernel<TV_KV_E4M3, 128>)
      : (geom->head_dim == 64 ? tv::kv_quant_append_kernel<TV_KV_INT8, 64> : tv::kv_quant_append_kernel<TV_KV_INT8, 128>);
  const dim3 grid((rows + tv::kAppendRows - 1) / tv::kAppendRows);
  const cudaError_t err = tv::launch_pdl(kernel, grid, dim3(tv::kAppendThreads), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

extern "C" int tv_kv_quant_read(const tv_geom* geom, int32_t kv_format, int32_t batch,
                                const int32_t* first, const int32_t* last,
                                const int32_t* block_table, const int32_t* n_blocks,
                                int32_t max_blocks_per_req, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                int32_t num_blocks, const int32_t* out_block_table,
                                const int32_t* out_n_blocks, int32_t out_max_blocks_per_req,
                                void* k_out, void* v_out, int32_t out_num_blocks, int32_t* status,
                                void* stream) {
  int rc = tv::check_geom(geom);
  if (rc != TV_OK) return rc;
  rc = tv::check_kv_format(kv_format);
  if (rc != TV_OK) return rc;
  if (batch < 0 || batch > tv::kKvMaxBatch || max_blocks_per_req < 1 || num_blocks < 1 ||
      out_max_blocks_per_req < 1 || out_num_blocks < 1)
    return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!last || !block_table || !n_blocks || !k_cache || !v_cache || !k_scale || !v_scale ||
      !out_block_table || !out_n_blocks || !k_out || !v_out || !status)
    return TV_ERR_NULL_POINTER;
  if (!tv::aligned(k_cache, 16) || !tv::aligned(v_cache, 16) || !tv::aligned(k_out, 16) ||
      !tv::aligned(v_out, 16) || !tv::aligned(k_scale, 4) || !tv::aligned(v_scale, 4))
    return TV_ERR_MISALIGNED;
  tv::ReadParams p = {};
  p.first = first; p.last = last; p.block_table = block_table; p.n_blocks = n_blocks;
  p.k_cache = static_cast<const uint8_t*>(k_cache); p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale;
  p.out_table = out_block_table; p.out_n_blocks = out_n_blocks;
  p.k_out = static_cast<__nv_bfloat16*>(k_out); p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.status = status;
  p.batch = batch; p.hkv = geom->num_kv_heads; p.max_blocks = max_blocks_per_req; p.num_blocks = num_blocks;
  p.out_max_blocks = out_max_blocks_per_req; p.out_num_blocks = out_num_blocks;
  auto* kernel = kv_format == TV_KV_E4M3
      ? (geom->head_dim == 64 ? tv::kv_quant_read_kernel<TV_KV_E4M3, 64> : tv::kv_quant_read_kernel<TV_KV_E4M3, 128>)
      : (geom->head_dim == 64 ? tv::kv_quant_read_kernel<TV_KV_INT8, 64> : tv::kv_quant_read_kernel<TV_KV_INT8, 128>);
  const int pages = max_blocks_per_req < out_max_blocks_per_req ? max_blocks_per_req : out_max_blocks_per_req;
  const dim3 grid(pages < 256 ? pages : 256, batch);
  const cudaError_t err = tv::launch_pdl(kernel, grid, dim3(tv::kReadThreads), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
