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
// Measured: append 34.5 us for 201 MB (5.8 TB/s), read back 119 us for 692 MB
// (5.8 TB/s, two thirds of it writes).
#include <climits>

#include "tv_kv8.cuh"
#include "tv_share.cuh"

namespace tv {

constexpr int kAppendThreads = 256;
constexpr int kAppendPerSm = 3;      // CTAs an SM
constexpr int kAppendAhead = 4;      // rows whose loads a thread has in flight
constexpr int kAppendMaxRows = 256;  // rows of k_new / v_new per CTA at most (a thread describes a row)
static_assert(kAppendMaxRows == kAppendThreads, "arrays by row also serve by thread");

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
  uint32_t by_heads;                 // thread_divisor(cta_heads)
};

// A request's rows among the CTA's rows.
struct AppendRun {
  int req;
  int c0;        // the request's first row
  int start;     // that row's slot
  int last;      // one past the run, counted from the CTA's first row
};

// A CTA quantises a contiguous range of rows (all of them in one wave of CTAs
// where they fit), kLanes threads a row and head. Each thread keeps its head
// and steps through the rows with kAppendAhead of them in flight: a row's
// registers are loaded again as soon as it is encoded. (Loading a batch of
// four, then encoding and storing it, left the memory idle while the CTAs of
// an SM computed in step: 41.8 us for 201 MB.)
template <int kFmt, int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendPerSm) kv_quant_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16;       // lanes that hold one row, two pieces of 8 values each
  __shared__ AppendRun s_run[kAppendMaxRows];                // by the run's first row
  __shared__ int s_bad[kAppendMaxRows];                      // by the run's first row
  __shared__ uint32_t s_heads[kAppendMaxRows / 32];          // bit r: a run begins at row r
  __shared__ long long s_row[kAppendMaxRows];                // the row's place in the pool (head 0), -1: none
  __shared__ int s_head[kAppendMaxRows];
  __shared__ int s_cross[2][4];        // requests that reach past the CTA's rows, before and behind:
                                       // request, first page, pages, first row of the run
  grid_launch_dependents();
  const int t0 = blockIdx.x * p.cta_rows;
  const int nrows = min(p.cta_rows, p.rows - t0), t1 = t0 + nrows;
  const int part = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int slot0 = part * p.by_heads >> 16, head = blockIdx.y * p.cta_heads + part - slot0 * p.cta_heads;
  const bool mine = slot0 < p.slots && head < 2 * p.hkv;
  const bool isv = head >= p.hkv;
  const int h = isv ? head - p.hkv : head;
  const long long step = p.slots * p.kv_ld;
  const __nv_bfloat16* src = (isv ? p.v_new : p.k_new) + (t0 + slot0) * p.kv_ld + static_cast<long long>(h) * D + lane * 8;
  // A thread looks at request i with all that it needs of it in one round
  // trip. Its first request goes ahead of the rows, so as not to queue behind them.
  struct Request { int c0, c1, st, start, held; };
  auto look_at = [&](int i) {
    Request q = {0, 0, 0, 0, 0};
    if (i < p.batch) q = Request{p.cu_rows[i], p.cu_rows[i + 1], *const_cast<volatile int32_t*>(p.status + i), p.start_len[i], min(p.n_blocks[i], p.max_blocks)};
    return q;
  };
  if (threadIdx.x < kAppendMaxRows) s_bad[threadIdx.x] = 0;
  if (threadIdx.x < kAppendMaxRows / 32) s_heads[threadIdx.x] = 0u;
  if (threadIdx.x < 8) s_cross[threadIdx.x / 4][threadIdx.x % 4] = 0;
  grid_dependency_wait();              // (all of the above while the grid before this one ends)
  Request q = look_at(threadIdx.x);
  uint4 x[kAppendAhead][2];            // a warp's loads cover whole sectors: piece lane, piece lane + kLanes
  auto load = [&](uint4 (&to)[2], int r) {
    to[0] = to[1] = make_uint4(0u, 0u, 0u, 0u);
    if (mine && r < nrows) {
      to[0] = *reinterpret_cast<const uint4*>(src);
      to[1] = *reinterpret_cast<const uint4*>(src + kLanes * 8);
    }
    src += step;
  };
#pragma unroll
  for (int e = 0; e < kAppendAhead; ++e) load(x[e], slot0 + e * p.slots);    // on their way while slots are found

  __syncthreads();
  // the CTA's rows that each request owns (the first CTA reports bad offsets)
  auto claim = [&](int i, const Request& r, bool bad) {
    if ((r.c1 <= r.c0 && !bad) || r.st != 0) return;
    bad |= r.c1 > p.rows || r.c0 < 0 || r.start < 0;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status + i, TV_ST_BAD_SIZE);
    if (bad || r.c0 >= t1 || r.c1 <= t0) return;
    const int first = max(r.c0, t0) - t0;
    const long long end = static_cast<long long>(r.start) + (r.c1 - r.c0);
    const bool fits = (end - 1) / TV_BLOCK_SIZE < r.held;    // (which also keeps slots below 2^31)
    if (!fits) s_bad[first] = TV_ST_BAD_BLOCK;
    s_run[first] = AppendRun{i, r.c0, r.start, min(r.c1, t1) - t0};
    atomicOr(&s_heads[first / 32], 1u << (first % 32));
    if (fits && (r.c0 < t0 || r.c1 > t1)) {
      int* cross = s_cross[r.c0 < t0 ? 0 : 1];
      cross[0] = i;
      cross[1] = r.start / TV_BLOCK_SIZE;
      cross[3] = first;
      cross[2] = static_cast<int>((end - 1) / TV_BLOCK_SIZE) - cross[1] + 1;
    }
  };
  bool back = false;
  for (int i = threadIdx.x; i < p.batch; i += kAppendThreads, q = look_at(i)) {
    back |= q.c1 < q.c0;
    claim(i, q, false);
  }
  // Offsets that run backwards let requests claim the same rows: all is claimed
  // again, without the requests that begin before an earlier offset or end before
  // they begin. (Every CTA looks at all offsets, so all of them decide alike.)
  if (__syncthreads_or(back)) {
    const int per = (p.batch + kAppendThreads - 1) / kAppendThreads;
    const int i0 = min(p.batch, static_cast<int>(threadIdx.x) * per), i1 = min(p.batch, i0 + per);
    int most = INT_MIN;
    for (int i = i0; i < i1; ++i) most = max(most, p.cu_rows[i]);
    if (threadIdx.x < kAppendMaxRows) s_bad[threadIdx.x] = 0;
    if (threadIdx.x < kAppendMaxRows / 32) s_heads[threadIdx.x] = 0u;
    if (threadIdx.x < 8) s_cross[threadIdx.x / 4][threadIdx.x % 4] = 0;
    s_head[threadIdx.x] = most;
    __syncthreads();
    most = INT_MIN;                    // of the offsets before the thread's requests
    for (int t = 0; t < static_cast<int>(threadIdx.x); ++t) most = max(most, s_head[t]);
    for (int i = i0; i < i1; ++i) {
      const Request r = look_at(i);
      claim(i, r, r.c1 < r.c0 || (r.c1 > r.c0 && r.c0 < most));
      most = max(most, r.c0);
    }
    __syncthreads();
  }
  // the rows' blocks, and all other blocks of a request that other CTAs have rows of
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x;
    int w = r / 32, first = -1;
    uint32_t bits = s_heads[w] & (0xffffffffu >> (31 - r % 32));
    while (bits == 0u && w > 0) bits = s_heads[--w];
    if (bits != 0u) first = 32 * w + 31 - __clz(bits);
    s_row[r] = -1;
    s_head[r] = 0;
    if (first >= 0 && r < s_run[first].last && s_bad[first] == 0) {
      const AppendRun run = s_run[first];
      const int slot = run.start + (t0 + r - run.c0);
      const int page = slot / TV_BLOCK_SIZE;
      const int blk = slot >= 0 && page < p.max_blocks ? p.block_table[static_cast<size_t>(run.req) * p.max_blocks + page] : -1;
      s_row[r] = static_cast<long long>(blk) * p.hkv * TV_BLOCK_SIZE + slot % TV_BLOCK_SIZE;
      s_head[r] = first;
      if (blk < 0 || blk >= p.num_blocks) s_bad[first] = TV_ST_BAD_BLOCK;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int pages = min(s_cross[c][2], p.max_blocks - s_cross[c][1]);
    const int32_t* row = p.block_table + static_cast<size_t>(s_cross[c][0]) * p.max_blocks + s_cross[c][1];
    bool bad = false;
#pragma unroll 4
    for (int e = threadIdx.x; e < pages; e += kAppendThreads) {
      const int blk = row[e];
      bad |= blk < 0 || blk >= p.num_blocks;
    }
    if (bad) s_bad[s_cross[c][3]] = TV_ST_BAD_BLOCK;
  }
  __syncthreads();
  // one bad block holds all rows of its request back
  if (threadIdx.x < nrows) {
    const int r = threadIdx.x;
    if (s_bad[s_head[r]] != 0) s_row[r] = -1;
    if (s_bad[r] != 0 && blockIdx.y == 0) atomicOr(p.status + s_run[r].req, s_bad[r]);
  }
  __syncthreads();

  uint8_t* codes = (isv ? p.v_cache : p.k_cache) + lane * 8;
  float* scales = isv ? p.v_scale : p.k_scale;
  for (int r0 = 0; r0 < nrows; r0 += kAppendAhead * p.slots) {
#pragma unroll
    for (int e = 0; e < kAppendAhead; ++e) {
      if (r0 + e * p.slots >= nrows) break;                  // the same for all threads: the shuffles are whole
      const int r = r0 + slot0 + e * p.slots;
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
      uint2 code[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
      if (sc.mul != 0.0f) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          code[u] = make_uint2(kv_encode4<kFmt>(x[e][u].x, x[e][u].y, sc), kv_encode4<kFmt>(x[e][u].z, x[e][u].w, sc));
        }
      }
      load(x[e], r + kAppendAhead * p.slots);
      const long long place = mine && r < nrows ? s_row[r] : -1;
      if (place < 0) continue;
      const long long row = place + h * TV_BLOCK_SIZE;
      uint8_t* to = codes + row * D;
      *reinterpret_cast<uint2*>(to) = code[0];
      *reinterpret_cast<uint2*>(to + kLanes * 8) = code[1];
      if (lane == 0) scales[row] = sc.scale;
    }
  }
}

// ------------------------------------------------------------------ read back

constexpr int kReadThreads = 256;
constexpr int kReadPerSm = 4;          // CTAs an SM: 3 to 6 all take 117 to 119 us for 692 MB, small calls least with 4
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

// An item is the K or V rows of one head of one page: 16 D bytes of codes to
// 32 D bytes of bf16. All items are laid end to end, a CTA takes a contiguous
// range of them and its warps every eighth item. A lane turns 8 codes (8
// bytes) into one 16-byte store, so that a warp's stores cover whole 32-byte
// sectors, and a warp's loads of an item are all in flight together. The
// page's 16 scales come in one load and go round by shuffles.
template <int kFmt, int D>
__global__ void __launch_bounds__(kReadThreads, kReadPerSm) kv_quant_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kWarps = kReadThreads / 32;
  constexpr int kPerRow = D / 8;                             // 8-code vectors of a row
  constexpr int kPer = TV_BLOCK_SIZE * kPerRow / 32;         // a lane's vectors: 8 or 4
  grid_launch_dependents();
  grid_dependency_wait();
  const Share sh = find_share<kReadThreads>(p.batch, 1, [&](int b) {
    return static_cast<long long>(read_pages(p.first ? p.first[b] : 0, p.last[b])) * 2 * p.hkv;
  });
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t per_page = 2 * p.hkv;
  long long at = sh.start, pos = sh.lo;
  for (int b = sh.b; b < p.batch && pos < sh.hi; ++b) {
    const int first = p.first ? p.first[b] : 0, last = p.last[b], st = p.status[b];
    const int held = min(p.n_blocks[b], p.max_blocks), out_held = min(p.out_n_blocks[b], p.out_max_blocks);
    const int pages = read_pages(first, last);
    const long long end = at + static_cast<long long>(pages) * per_page;
    if (pos >= end) { at = end; continue; }
    const long long stop = end < sh.hi ? end : sh.hi;
    const int page0 = max(first, 0) / TV_BLOCK_SIZE, page1 = page0 + pages - 1;
    const int32_t* from = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    const int32_t* to = p.out_table + static_cast<size_t>(b) * p.out_max_blocks;
    int bad = 0;
    if (first < 0 || last < 0) {
      bad = TV_ST_BAD_SIZE;
    } else if (page1 >= held || page1 >= out_held) {
      bad = TV_ST_BAD_BLOCK;
    } else {
#pragma unroll 4
      for (int e = page0 + threadIdx.x; e <= page1; e += kReadThreads) {
        const int s = from[e], d = to[e];
        if (s < 0 || s >= p.num_blocks || d < 0 || d >= p.out_num_blocks) bad = TV_ST_BAD_BLOCK;
      }
    }
    // (the threads decide together: another CTA may flag the request meanwhile, having found the same)
    if (__syncthreads_or(bad | st)) {
      if (bad && st == 0) atomicOr(p.status + b, bad);
    } else {
      // item = page, K or V, head; the block ids of a warp's next item are on their way
      long long item = pos - at + warp;
      const long long items = stop - at;
      int page = 0, half = 0, sblk = 0, dblk = 0;
      auto look_up = [&](long long i, int& pg, int& hf, int& s, int& d) {
        if (i >= items) return;
        const uint32_t rel = static_cast<uint32_t>(divide(i, per_page));
        hf = static_cast<int>(i - static_cast<long long>(rel) * per_page);
        pg = page0 + static_cast<int>(rel);
        s = from[pg];
        d = to[pg];
      };
      look_up(item, page, half, sblk, dblk);
      while (item < items) {
        const bool isv = half >= p.hkv;
        const int h = isv ? half - p.hkv : half;
        const size_t srow = (static_cast<size_t>(sblk) * p.hkv + h) * TV_BLOCK_SIZE;
        const size_t drow = (static_cast<size_t>(dblk) * p.hkv + h) * TV_BLOCK_SIZE;
        const uint2* src = reinterpret_cast<const uint2*>((isv ? p.v_cache : p.k_cache) + srow * D) + lane;
        uint4* dst = reinterpret_cast<uint4*>((isv ? p.v_out : p.k_out) + drow * D) + lane;
        // rows [r0, r1) of the page
        const int r0 = max(first - page * TV_BLOCK_SIZE, 0), r1 = min(last - page * TV_BLOCK_SIZE, TV_BLOCK_SIZE);
        const int lane_row = lane / kPerRow;
        const float scale = (isv ? p.v_scale : p.k_scale)[srow + lane % TV_BLOCK_SIZE];
        uint2 c[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = i * (32 / kPerRow) + lane_row;
          c[i] = r >= r0 && r < r1 ? __ldcs(src + 32 * i) : make_uint2(0u, 0u);
        }
        item += kWarps;
        look_up(item, page, half, sblk, dblk);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = i * (32 / kPerRow) + lane_row;
          const float s = __shfl_sync(0xffffffffu, scale, r);
          const float2 f0 = kv_decode2<kFmt>(c[i].x & 0xffffu), f1 = kv_decode2<kFmt>(c[i].x >> 16);
          const float2 f2 = kv_decode2<kFmt>(c[i].y & 0xffffu), f3 = kv_decode2<kFmt>(c[i].y >> 16);
          if (r >= r0 && r < r1)
            dst[32 * i] = make_uint4(pack_bf16x2(f0.x * s, f0.y * s), pack_bf16x2(f1.x * s, f1.y * s),
                                     pack_bf16x2(f2.x * s, f2.y * s), pack_bf16x2(f3.x * s, f3.y * s));
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
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
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
  // a time when a row has fewer, and as many rows as fill the SMs once.
  const int parts = tv::kAppendThreads / (geom->head_dim / 16), heads = 2 * p.hkv;
  p.cta_heads = heads < parts ? heads : parts;
  p.slots = parts / p.cta_heads;
  p.by_heads = tv::thread_divisor(p.cta_heads);
  const int head_blocks = (heads + p.cta_heads - 1) / p.cta_heads;
  // (or a whole number of times)
  const long long work = static_cast<long long>(rows) * head_blocks, wave = static_cast<long long>(sms) * tv::kAppendPerSm;
  const long long waves = (work + wave * tv::kAppendMaxRows - 1) / (wave * tv::kAppendMaxRows);
  long long cta_rows = (work + waves * wave - 1) / (waves * wave);
  cta_rows = (cta_rows + p.slots - 1) / p.slots * p.slots;
  if (cta_rows > tv::kAppendMaxRows) cta_rows = tv::kAppendMaxRows;
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
  // As many CTAs as are resident, or as there can be pairs of items: fewer CTAs
  // with an item for each warp meet several short requests one after the other
  // (14 requests of 2 rows, one head: 6.1 us, with pairs 2.9; one item a CTA 2.9).
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  const long long pages = max_blocks_per_req < out_max_blocks_per_req ? max_blocks_per_req : out_max_blocks_per_req;
  const long long items = pages * batch * p.hkv, most = static_cast<long long>(sms) * tv::kReadPerSm;
  const dim3 grid(static_cast<unsigned>(items < most ? items : most));
  const cudaError_t err = tv::launch_pdl(kernel, grid, dim3(tv::kReadThreads), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
