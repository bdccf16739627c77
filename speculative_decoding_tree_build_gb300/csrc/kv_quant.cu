// tv_kv_quant_append and tv_kv_quant_read: rows written into the 8-bit paged
// KV cache and read back into bf16 pools.
//
// A row (one head's D values of one token) is quantised on its own: largest
// magnitude, scale, codes (tv_kv8.cuh). Both calls are bound by memory: the
// append reads 2 D bytes a row and writes D + 4, the read the other way round.
// A row is held by D / 16 neighbouring lanes, 32 bytes of bf16 each; its
// largest magnitude takes log2(D / 16) shuffles of a paired integer maximum.
// The append's rows are loaded before their slots are known, so the chain of
// small loads (offsets, lengths, block ids) overlaps the one large one.
#include "tv_kv8.cuh"
#include "tv_share.cuh"

namespace tv {

constexpr int kAppendThreads = 256;
constexpr int kAppendPerSm = 3;      // CTAs an SM: 2 / 3 / 4 took 46.6 / 41.8 / 42.1 us for 201 MB (4 spills)
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

// What the CTA knows of the row of K/V it handles.
struct AppendRow {
  int req;       // the request that owns it, -1: none (or one that is skipped)
  int head;      // the CTA's first row of that request: its verdict counts for all of them
  int slot;
  int blk;       // the slot's block
};

template <int kFmt, int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendPerSm) kv_quant_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16;       // lanes that hold one row, two pieces of 8 values each
  __shared__ AppendRow s_row[kAppendMaxRows];
  __shared__ int s_bad[kAppendMaxRows];                      // by head row
  __shared__ int s_cross[2][4];        // requests that reach past the CTA's rows, before and behind:
                                       // request, first page, pages, head row
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * p.cta_rows;
  const int nrows = min(p.cta_rows, p.rows - t0), t1 = t0 + nrows;
  // kLanes threads keep one head and step through the CTA's rows
  const int part = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int slot0 = part / p.cta_heads, head = blockIdx.y * p.cta_heads + part - slot0 * p.cta_heads;
  const bool mine = slot0 < p.slots && head < 2 * p.hkv;
  const bool isv = head >= p.hkv;
  const int h = isv ? head - p.hkv : head;
  const __nv_bfloat16* src = (isv ? p.v_new : p.k_new) + static_cast<long long>(h) * D + lane * 8;
  uint4 x[kAppendBatch][2];            // a warp's loads cover whole sectors: piece lane, piece lane + kLanes
  auto load = [&](int r0) {
#pragma unroll
    for (int e = 0; e < kAppendBatch; ++e) {
      const int r = r0 + e * p.slots;
      x[e][0] = x[e][1] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && r < nrows) {
        const __nv_bfloat16* from = src + (t0 + r) * p.kv_ld;
        x[e][0] = *reinterpret_cast<const uint4*>(from);
        x[e][1] = *reinterpret_cast<const uint4*>(from + kLanes * 8);
      }
    }
  };
  load(slot0);                         // on their way while the rows' slots are found

  // A thread looks at request i with all that it needs of it in one round
  // trip, and describes those of the CTA's rows that the request owns.
  if (threadIdx.x < kAppendMaxRows) {
    s_row[threadIdx.x].req = -1;
    s_bad[threadIdx.x] = 0;
  }
  if (threadIdx.x < 2) s_cross[threadIdx.x][2] = 0;
  __syncthreads();
#pragma unroll 2
  for (int i = threadIdx.x; i < p.batch; i += kAppendThreads) {
    const int c0 = p.cu_rows[i], c1 = p.cu_rows[i + 1], st = p.status[i], start = p.start_len[i];
    const int held = min(p.n_blocks[i], p.max_blocks);
    if (c1 <= c0 || st != 0) continue;
    if (blockIdx.x == 0 && blockIdx.y == 0 && (c1 > p.rows || c0 < 0 || start < 0)) atomicOr(p.status + i, TV_ST_BAD_SIZE);
    if (c0 < 0 || c1 > p.rows || start < 0 || c0 >= t1 || c1 <= t0) continue;
    const int first = max(c0, t0) - t0, last = min(c1, t1) - t0;
    const long long end = static_cast<long long>(start) + (c1 - c0);
    const bool fits = (end - 1) / TV_BLOCK_SIZE < held;      // (which also keeps slots below 2^31)
    if (!fits) s_bad[first] = TV_ST_BAD_BLOCK;
    for (int r = first; r < last; ++r) {
      AppendRow a;
      a.req = i;
      a.head = first;
      a.slot = fits ? start + (t0 + r - c0) : 0;
      a.blk = -1;
      s_row[r] = a;
    }
    if (fits && (c0 < t0 || c1 > t1)) {
      int* cross = s_cross[c0 < t0 ? 0 : 1];
      cross[0] = i;
      cross[1] = start / TV_BLOCK_SIZE;
      cross[3] = first;
      cross[2] = static_cast<int>((end - 1) / TV_BLOCK_SIZE) - cross[1] + 1;
    }
  }
  __syncthreads();
  // the rows' blocks, and all other blocks of a request that other CTAs have rows of
  if (threadIdx.x < nrows && s_row[threadIdx.x].req >= 0) {
    AppendRow& a = s_row[threadIdx.x];
    if (s_bad[a.head] == 0) {
      const int blk = p.block_table[static_cast<size_t>(a.req) * p.max_blocks + a.slot / TV_BLOCK_SIZE];
      a.blk = blk;
      if (blk < 0 || blk >= p.num_blocks) s_bad[a.head] = TV_ST_BAD_BLOCK;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int pages = s_cross[c][2];
    const int32_t* row = p.block_table + static_cast<size_t>(s_cross[c][0]) * p.max_blocks + s_cross[c][1];
    bool bad = false;
    for (int e = threadIdx.x; e < pages; e += kAppendThreads) {
      const int blk = row[e];
      bad |= blk < 0 || blk >= p.num_blocks;
    }
    if (bad) s_bad[s_cross[c][3]] = TV_ST_BAD_BLOCK;
  }

  uint2 code[kAppendBatch][2];
  float scale[kAppendBatch];
  auto encode = [&](int r0) {
#pragma unroll
    for (int e = 0; e < kAppendBatch; ++e) {
      if (r0 + e * p.slots >= nrows) break;                  // the same for all threads: the shuffles are whole
      // bits 14..0 of both halves order as integers: halves are compared apart
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[e][u].x & 0x7fff7fffu, x[e][u].y & 0x7fff7fffu),
                                     __vmaxu2(x[e][u].z & 0x7fff7fffu, x[e][u].w & 0x7fff7fffu)));
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, s));
      top = max(top & 0xffffu, top >> 16);
      const KvRowScale sc = kv_row_scale<kFmt>(top);
      scale[e] = sc.scale;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint2 c = make_uint2(0u, 0u);
        if (sc.mul != 0.0f) {
          c.x = kv_encode2<kFmt>(bf16_lo(x[e][u].x), bf16_hi(x[e][u].x), sc) | (kv_encode2<kFmt>(bf16_lo(x[e][u].y), bf16_hi(x[e][u].y), sc) << 16);
          c.y = kv_encode2<kFmt>(bf16_lo(x[e][u].z), bf16_hi(x[e][u].z), sc) | (kv_encode2<kFmt>(bf16_lo(x[e][u].w), bf16_hi(x[e][u].w), sc) << 16);
        }
        code[e][u] = c;
      }
    }
  };
  encode(0);                           // while the block ids are on their way
  __syncthreads();
  if (threadIdx.x < nrows && blockIdx.y == 0) {
    const AppendRow a = s_row[threadIdx.x];
    if (a.req >= 0 && a.head == static_cast<int>(threadIdx.x) && s_bad[a.head] != 0) atomicOr(p.status + a.req, s_bad[a.head]);
  }

  uint8_t* codes = (isv ? p.v_cache : p.k_cache) + lane * 8;
  float* scales = isv ? p.v_scale : p.k_scale;
  for (int r0 = 0; r0 < nrows; r0 += kAppendBatch * p.slots) {
    if (r0 > 0) {
      load(r0 + slot0);
      encode(r0);
    }
#pragma unroll
    for (int e = 0; e < kAppendBatch; ++e) {
      const int r = r0 + slot0 + e * p.slots;
      if (!mine || r >= nrows) break;
      const AppendRow a = s_row[r];
      if (a.req < 0 || s_bad[a.head] != 0) continue;
      const size_t row = (static_cast<size_t>(a.blk) * p.hkv + h) * TV_BLOCK_SIZE + a.slot % TV_BLOCK_SIZE;
      uint8_t* to = codes + row * D;
      *reinterpret_cast<uint2*>(to) = code[e][0];
      *reinterpret_cast<uint2*>(to + kLanes * 8) = code[e][1];
      if (lane == 0) scales[row] = scale[e];
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
              sc[e][j] = (isv ? p.v_scale : p.k_scale)[src + row];
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
  // heads go to grid.y in blocks of 32 or 64
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
  // A CTA takes up to 256 / (D / 16) heads of a row at a time, several rows at
  // a time when a row has fewer, and two batches of loads a thread where that
  // still gives every SM eight CTAs (fewer rows than that: down to one sweep).
  const int parts = tv::kAppendThreads / (geom->head_dim / 16), heads = 2 * p.hkv;
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
  const dim3 grid(static_cast<unsigned>((rows + cta_rows - 1) / cta_rows), head_blocks);
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
