// tv_kv_quant_append and tv_kv_quant_read: rows written into the 8-bit paged
// KV cache and read back into bf16 pools.
//
// A row (one head's D values of one token) is quantised on its own: largest
// magnitude, scale, codes (tv_kv8.cuh). Both calls are bound by memory: the
// append reads 2 D bytes a row and writes D + 4, the read the other way round.
// A row is held by D / 8 neighbouring lanes, 16 bytes of bf16 each; its
// largest magnitude takes log2(D / 8) shuffles of a paired integer maximum.
// The append's rows are loaded before their slots are known, so the chain of
// small loads (offsets, lengths, block ids) overlaps the one large one.
#include "tv_kv8.cuh"
#include "tv_share.cuh"

namespace tv {

constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 4;      // rows whose loads a thread has in flight
constexpr int kAppendMaxRows = 64;   // rows of k_new / v_new per CTA at most

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
  int batch, rows, hkv, max_blocks, num_blocks, cta_rows;
  int cta_heads;                     // of the 2 hkv heads of a row (K's, then V's), taken at a time
  int slots;                         // rows taken at a time
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
  extern __shared__ int s_cu[];        // [batch + 1]
  __shared__ int s_req[kAppendMaxRows], s_slot[kAppendMaxRows], s_blk[kAppendMaxRows], s_bad[kAppendMaxRows];
  __shared__ int s_first[kAppendMaxRows], s_pages[kAppendMaxRows];     // of a run's request: its span
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * p.cta_rows;
  const int nrows = min(p.cta_rows, p.rows - t0);
  // kLanes threads keep one head and step through the CTA's rows
  const int part = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int slot0 = part / p.cta_heads, head = blockIdx.y * p.cta_heads + part - slot0 * p.cta_heads;
  const bool mine = slot0 < p.slots && head < 2 * p.hkv;
  const bool isv = head >= p.hkv;
  const int h = isv ? head - p.hkv : head;
  const __nv_bfloat16* src = (isv ? p.v_new : p.k_new) + static_cast<long long>(h) * D + lane * 8;
  uint4 x[kAppendBatch];
  auto load = [&](int r0) {
#pragma unroll
    for (int e = 0; e < kAppendBatch; ++e) {
      const int r = r0 + e * p.slots;
      x[e] = mine && r < nrows ? *reinterpret_cast<const uint4*>(src + (t0 + r) * p.kv_ld) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(slot0);                         // on their way while the rows' slots are found

  for (int i = threadIdx.x; i <= p.batch; i += kAppendThreads) s_cu[i] = p.cu_rows[i];
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0) {    // requests whose rows lie past the array, in part or altogether
    for (int b = threadIdx.x; b < p.batch; b += kAppendThreads)
      if (s_cu[b + 1] > p.rows && s_cu[b + 1] > s_cu[b] && p.status[b] == 0) atomicOr(p.status + b, TV_ST_BAD_SIZE);
  }
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x, t = t0 + r;
    const int b = request_of_row(s_cu, p.batch, t);
    int bad = -1, blk = -1;            // -1: not this call's to write, nothing to report
    s_req[r] = b;
    s_pages[r] = 0;
    if (b >= 0) {
      const int st = p.status[b], start = p.start_len[b], held = min(p.n_blocks[b], p.max_blocks);
      const long long slot = static_cast<long long>(start) + (t - s_cu[b]);
      const long long end = static_cast<long long>(start) + (s_cu[b + 1] - s_cu[b]);
      if (st == 0) {
        bad = 0;
        if (start < 0 || s_cu[b] < 0 || end > 0x7fffffffll) bad = TV_ST_BAD_SIZE;
        else if (s_cu[b + 1] > p.rows) bad = -1;                       // CTA 0 reports it
        else if ((end - 1) / TV_BLOCK_SIZE >= held) bad = TV_ST_BAD_BLOCK;
      }
      if (bad == 0) {
        blk = p.block_table[static_cast<size_t>(b) * p.max_blocks + slot / TV_BLOCK_SIZE];
        if (blk < 0 || blk >= p.num_blocks) bad = TV_ST_BAD_BLOCK;
        // the request's first row here checks the blocks of rows that lie in other CTAs
        if (bad == 0 && (r == 0 || t - 1 < s_cu[b]) && (s_cu[b] < t0 || s_cu[b + 1] > t0 + nrows)) {
          s_first[r] = start / TV_BLOCK_SIZE;
          s_pages[r] = static_cast<int>((end - 1) / TV_BLOCK_SIZE) - s_first[r] + 1;
        }
      }
      s_slot[r] = static_cast<int>(slot);
    }
    s_bad[r] = bad;
    s_blk[r] = blk;
  }
  __syncthreads();
  // at most two requests reach beyond this CTA's rows: the first and the last one
  for (int r = 0; r < nrows; ++r) {
    const int pages = s_pages[r];
    if (pages == 0) continue;
    const int32_t* row = p.block_table + static_cast<size_t>(s_req[r]) * p.max_blocks + s_first[r];
    bool bad = false;
    for (int e = threadIdx.x; e < pages; e += kAppendThreads) {
      const int blk = row[e];
      bad |= blk < 0 || blk >= p.num_blocks;
    }
    if (bad) s_bad[r] = TV_ST_BAD_BLOCK;
  }
  __syncthreads();
  if (threadIdx.x < nrows && s_req[threadIdx.x] >= 0) {
    // one bad row of a request holds all of its rows back
    const int r = threadIdx.x, b = s_req[r];
    int bad = s_bad[r];
    const int own = bad;
    for (int o = r - 1; o >= 0 && s_req[o] == b; --o) bad = max(bad, s_bad[o]);
    for (int o = r + 1; o < nrows && s_req[o] == b; ++o) bad = max(bad, s_bad[o]);
    if (bad != 0) s_blk[r] = -1;
    if (own > 0) atomicOr(p.status + b, own);
  }
  __syncthreads();
  uint8_t* codes = (isv ? p.v_cache : p.k_cache) + lane * 8;
  float* scales = isv ? p.v_scale : p.k_scale;
  for (int r0 = 0; r0 < nrows; r0 += kAppendBatch * p.slots) {
    if (r0 > 0) load(r0 + slot0);
#pragma unroll
    for (int e = 0; e < kAppendBatch; ++e) {
      if (r0 + e * p.slots >= nrows) break;                  // the same for all threads: the shuffles are whole
      const int r = r0 + slot0 + e * p.slots;
      const int blk = mine && r < nrows ? s_blk[r] : -1;
      const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
      // bits 14..0 of both halves order as integers: halves are compared apart
      uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                              __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, s));
      top = max(top & 0xffffu, top >> 16);
      if (blk < 0) continue;
      const KvRowScale sc = kv_row_scale<kFmt>(top);
      uint2 c = make_uint2(0u, 0u);
      if (sc.mul != 0.0f) {
        c.x = kv_encode2<kFmt>(bf16_lo(w[0]), bf16_hi(w[0]), sc) | (kv_encode2<kFmt>(bf16_lo(w[1]), bf16_hi(w[1]), sc) << 16);
        c.y = kv_encode2<kFmt>(bf16_lo(w[2]), bf16_hi(w[2]), sc) | (kv_encode2<kFmt>(bf16_lo(w[3]), bf16_hi(w[3]), sc) << 16);
      }
      const size_t row = (static_cast<size_t>(blk) * p.hkv + h) * TV_BLOCK_SIZE + s_slot[r] % TV_BLOCK_SIZE;
      *reinterpret_cast<uint2*>(codes + row * D) = c;
      if (lane == 0) scales[row] = sc.scale;
    }
  }
}

// ------------------------------------------------------------------ read back

constexpr int kReadThreads = 256;
constexpr int kReadBatch = 4;          // items a thread has in flight

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

// Pages that a request's range touches; a negative end is one page, so that
// some CTA meets the request and flags it.
__device__ __forceinline__ int read_pages(int first, int last) {
  if (first < 0 || last < 0) return 1;
  return last <= first ? 0 : (last - 1) / TV_BLOCK_SIZE - first / TV_BLOCK_SIZE + 1;
}

// An item is one head of one page, K and V: 32 D bytes of codes to 64 D bytes
// of bf16. All items are laid end to end and a CTA takes a contiguous range.
// A thread turns 8 codes (8 bytes) into one 16-byte store, so that a warp's
// stores cover whole 32-byte sectors (16 codes a thread and two stores a
// stride apart: 118 us for the 692 MB of the largest measured case).
template <int kFmt, int D>
__global__ void __launch_bounds__(kReadThreads) kv_quant_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kVecs = TV_BLOCK_SIZE * D / 8;               // 8-code vectors of K (or V) in an item
  constexpr int kPer = 2 * kVecs / kReadThreads;             // a thread's vectors in an item: 2 or 1
  grid_dependency_wait();
  grid_launch_dependents();
  const Share sh = find_share<kReadThreads>(p.batch, 1, [&](int b) {
    return static_cast<long long>(read_pages(p.first ? p.first[b] : 0, p.last[b])) * p.hkv;
  });
  long long at = sh.start;
  long long pos = sh.lo;
  for (int b = sh.b; b < p.batch && pos < sh.hi; ++b) {
    const int first = p.first ? p.first[b] : 0, last = p.last[b], st = p.status[b];
    const int pages = read_pages(first, last);
    const long long end = at + static_cast<long long>(pages) * p.hkv;
    if (pos >= end) { at = end; continue; }
    const long long stop = end < sh.hi ? end : sh.hi;
    const int page0 = max(first, 0) / TV_BLOCK_SIZE, page1 = page0 + pages - 1;
    const int32_t* from = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    const int32_t* to = p.out_table + static_cast<size_t>(b) * p.out_max_blocks;
    int bad = 0;
    if (first < 0 || last < 0) {
      bad = TV_ST_BAD_SIZE;
    } else if (page1 >= min(p.n_blocks[b], p.max_blocks) || page1 >= min(p.out_n_blocks[b], p.out_max_blocks)) {
      bad = TV_ST_BAD_BLOCK;
    } else {
      for (int e = page0 + threadIdx.x; e <= page1; e += kReadThreads) {
        const int s = from[e], d = to[e];
        if (s < 0 || s >= p.num_blocks || d < 0 || d >= p.out_num_blocks) bad = TV_ST_BAD_BLOCK;
      }
    }
    // status is only OR-ed into after this point of some CTA, by a CTA that found the same fault
    if (__syncthreads_or(bad | st)) {
      if (bad && st == 0) atomicOr(p.status + b, bad);
    } else {
      const int i0 = static_cast<int>((pos - at) % p.hkv);
      const int p0 = page0 + static_cast<int>((pos - at) / p.hkv);
      const int count = static_cast<int>(stop - pos);
      for (int base = 0; base < count; base += kReadBatch) {
        uint2 c[kReadBatch][kPer];
        float sc[kReadBatch][kPer];
        size_t dst[kReadBatch];
        bool live[kReadBatch][kPer];
#pragma unroll
        for (int e = 0; e < kReadBatch; ++e) {
          const int i = i0 + base + e;
          const int page = p0 + i / p.hkv, h = i % p.hkv;
          const bool there = base + e < count;
          const size_t src = there ? (static_cast<size_t>(from[page]) * p.hkv + h) * TV_BLOCK_SIZE : 0;
          dst[e] = there ? (static_cast<size_t>(to[page]) * p.hkv + h) * TV_BLOCK_SIZE : 0;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int idx = threadIdx.x + j * kReadThreads;
            const bool isv = idx >= kVecs;
            const int v = isv ? idx - kVecs : idx, row = v / (D / 8), slot = page * TV_BLOCK_SIZE + row;
            live[e][j] = there && slot >= first && slot < last;
            c[e][j] = make_uint2(0u, 0u);
            sc[e][j] = 0.0f;
            if (live[e][j]) {
              c[e][j] = __ldcs(reinterpret_cast<const uint2*>((isv ? p.v_cache : p.k_cache) + src * D) + v);
              sc[e][j] = __ldg((isv ? p.v_scale : p.k_scale) + src + row);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kReadBatch; ++e) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            if (!live[e][j]) continue;
            const int idx = threadIdx.x + j * kReadThreads;
            const bool isv = idx >= kVecs;
            const int v = isv ? idx - kVecs : idx;
            const float s = sc[e][j];
            const float2 f0 = kv_decode2<kFmt>(c[e][j].x & 0xffffu), f1 = kv_decode2<kFmt>(c[e][j].x >> 16);
            const float2 f2 = kv_decode2<kFmt>(c[e][j].y & 0xffffu), f3 = kv_decode2<kFmt>(c[e][j].y >> 16);
            reinterpret_cast<uint4*>((isv ? p.v_out : p.k_out) + dst[e] * D)[v] =
                make_uint4(pack_bf16x2(f0.x * s, f0.y * s), pack_bf16x2(f1.x * s, f1.y * s),
                           pack_bf16x2(f2.x * s, f2.y * s), pack_bf16x2(f3.x * s, f3.y * s));
          }
        }
      }
    }
    pos = stop;
    at = end;
  }
}

static int check_kv_format(const tv_geom* geom, int fmt) {
  // heads go to grid.y in blocks of 16 or 32
  return (fmt == TV_KV_E4M3 || fmt == TV_KV_INT8) && geom->num_kv_heads <= 4096 ? TV_OK : TV_ERR_BAD_GEOMETRY;
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
  rc = tv::check_kv_format(geom, kv_format);
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
  // A CTA takes up to 256 / (D / 8) heads of a row at a time, several rows at
  // a time when a row has fewer, and two batches of loads a thread where that
  // still gives every SM eight CTAs (fewer rows than that: down to one sweep).
  const int parts = tv::kAppendThreads / (geom->head_dim / 8), heads = 2 * p.hkv;
  p.cta_heads = heads < parts ? heads : parts;
  p.slots = parts / p.cta_heads;
  const int head_blocks = (heads + p.cta_heads - 1) / p.cta_heads;
  const long long ctas = 152 * 8 / head_blocks + 1;
  long long cta_rows = (rows + ctas - 1) / ctas;
  const long long most = 2ll * tv::kAppendBatch * p.slots;
  if (cta_rows > most) cta_rows = most;
  if (cta_rows > tv::kAppendMaxRows) cta_rows = tv::kAppendMaxRows;
  cta_rows = (cta_rows + p.slots - 1) / p.slots * p.slots;
  p.cta_rows = static_cast<int>(cta_rows);
  const size_t smem = sizeof(int) * (static_cast<size_t>(batch) + 1);
  const dim3 grid(static_cast<unsigned>((rows + cta_rows - 1) / cta_rows), head_blocks);
  const cudaError_t err = tv::launch_pdl(kernel, grid, dim3(tv::kAppendThreads), smem, tv::as_stream(stream), p);
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
  rc = tv::check_kv_format(geom, kv_format);
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
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
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
  // as many CTAs as are resident, or as there can be items
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  const long long pages = max_blocks_per_req < out_max_blocks_per_req ? max_blocks_per_req : out_max_blocks_per_req;
  const long long items = pages * batch * p.hkv, most = static_cast<long long>(sms) * 6;
  const dim3 grid(static_cast<unsigned>(items < most ? items : most));
  const cudaError_t err = tv::launch_pdl(kernel, grid, dim3(tv::kReadThreads), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
