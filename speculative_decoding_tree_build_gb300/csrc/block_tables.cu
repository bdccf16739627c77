// tv_block_tables and tv_slot_map: the pages that requests hold, kept on the
// device, and the slots that their rows go to.
//
// The free list is a stack. Three kinds of moves happen in a call, each
// numbered p = 0, 1, ... over requests ascending and blocks ascending:
//   1. ids that a commit released   -> free[base + total - 1 - p]
//   2. blocks past the wanted end   -> the same, on top of those
//   3. blocks that a request lacks  <- free[top - 1 - p]
// Push and pop mirror each other, so giving back what a call handed out
// restores list and tables exactly. The numbers are prefix sums of the
// requests' counts: no atomics on the list, the result depends on the
// arguments alone.
#include <algorithm>
#include <climits>

#include "tv_cluster.cuh"

namespace tv {

constexpr int kTableThreads = 512;
constexpr int kTableMaxBatch = 4096;
constexpr int kTablePer = kTableMaxBatch / kTableThreads;   // requests a thread looks at
constexpr int kTableCluster = 8;
constexpr int kTableAhead = 4;                              // moves of a thread in flight

struct TableParams {
  const int32_t* want_len;
  int32_t* table;
  int32_t* n_blocks;
  int32_t* free_blocks;
  int32_t* free_count;
  const int32_t* released;
  int32_t* released_count;
  int32_t* status;
  int batch, max_blocks, num_blocks, csize;
};

// Blocks of the requests before one: released, dropped, added.
struct TableSums {
  long long rel, drop, add;
};

__device__ __forceinline__ TableSums operator+(const TableSums& a, const TableSums& b) {
  return {a.rel + b.rel, a.drop + b.drop, a.add + b.add};
}

// Exclusive sums over the CTA's threads and the total.
__device__ __forceinline__ TableSums table_scan(const TableSums& mine, TableSums* s_warp, TableSums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  TableSums up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const TableSums v = {__shfl_up_sync(0xffffffffu, up.rel, o), __shfl_up_sync(0xffffffffu, up.drop, o),
                         __shfl_up_sync(0xffffffffu, up.add, o)};
    if (lane >= o) up = up + v;
  }
  __syncthreads();                        // s_warp may still be read from the scan before
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  TableSums before = {0, 0, 0};
  total = {0, 0, 0};
  for (int w = 0; w < kTableThreads / 32; ++w) {
    if (w == warp) before = total;
    total = total + s_warp[w];
  }
  return {before.rel + up.rel - mine.rel, before.drop + up.drop - mine.drop, before.add + up.add - mine.add};
}

// The last of n ascending numbers that is <= p (the first one is): with sums of
// counts, the request that has move p; with offsets, the one that has row p.
__device__ __forceinline__ int last_at_most(const int32_t* sums, int n, int p) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= p) lo = mid; else hi = mid;
  }
  return lo;
}

// A cluster makes the call: every CTA works the sums out for itself (4096
// requests are 8 a thread), then all moves are spread over the cluster's
// threads, each looking its request up in the sums. Latency binds it: a round
// trip for the requests, one for the ids, a barrier before anything is
// overwritten, and one between pushes and pops where both occur.
__global__ void __launch_bounds__(kTableThreads, 1) block_tables_kernel(const __grid_constant__ TableParams p) {
  extern __shared__ int32_t s_req[];      // by request: three sums, blocks held, blocks wanted
  __shared__ TableSums s_warp[kTableThreads / 32];
  __shared__ uint64_t s_faulty[kTableMaxBatch / 64];        // requests with an id outside the pool, seen by this CTA
  __shared__ uint64_t s_any;                                // (one of those words is not 0)
  __shared__ uint32_t s_all[kTableMaxBatch / 32];           // and by any CTA
  __shared__ int s_taken;                                   // blocks handed out
  int32_t* s_rel = s_req;
  int32_t* s_drop = s_rel + p.batch;
  int32_t* s_add = s_drop + p.batch;
  int32_t* s_held = s_add + p.batch;
  int32_t* s_need = s_held + p.batch;
  const int rank = p.csize > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = rank * kTableThreads + threadIdx.x, step = p.csize * kTableThreads;
  const int per = (p.batch + kTableThreads - 1) / kTableThreads;   // requests of a thread, side by side
  if (threadIdx.x < kTableMaxBatch / 64) s_faulty[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    s_any = 0;
    s_taken = 0;
  }
  grid_dependency_wait();
  grid_launch_dependents();

  const int count = *p.free_count;
  int held[kTablePer], need[kTablePer], rel[kTablePer], flag[kTablePer];   // flag: -1 leaves the request out
#pragma unroll
  for (int u = 0; u < kTablePer; ++u) {
    const int b = threadIdx.x * per + u;
    held[u] = need[u] = rel[u] = 0;
    flag[u] = -1;
    if (u >= per || b >= p.batch) continue;
    const int st = p.status[b], want = p.want_len[b];
    held[u] = p.n_blocks[b];
    rel[u] = p.released_count ? p.released_count[b] : 0;
    need[u] = want / TV_BLOCK_SIZE + (want % TV_BLOCK_SIZE > 0);
    if (st == 0)
      flag[u] = want < 0 || need[u] > p.max_blocks || held[u] < 0 || held[u] > p.max_blocks || rel[u] < 0 ||
                        rel[u] > p.max_blocks
                    ? TV_ST_BAD_SIZE : 0;
  }
  TableSums total = {0, 0, 0}, at;
  // where the i-th id that comes back stands, and whose it is
  auto back = [&](int i, int& b) -> const int32_t* {
    const bool is_rel = i < total.rel;
    const int q = is_rel ? i : i - static_cast<int>(total.rel);
    b = last_at_most(is_rel ? s_rel : s_drop, p.batch, q);
    const size_t row = static_cast<size_t>(b) * p.max_blocks;
    return is_rel ? p.released + row + (q - s_rel[b]) : p.table + row + s_need[b] + (q - s_drop[b]);
  };
  bool fail, checked = false;
  while (true) {
    TableSums mine = {0, 0, 0};
#pragma unroll
    for (int u = 0; u < kTablePer; ++u)
      if (flag[u] == 0) mine = mine + TableSums{rel[u], max(held[u] - need[u], 0), max(need[u] - held[u], 0)};
    at = table_scan(mine, s_warp, total);
    // a list too short for what comes back holds some of it already
    fail = count < 0 || count > p.num_blocks || total.rel + total.drop > p.num_blocks - count;
    if (fail) break;
    TableSums sum = at;
#pragma unroll
    for (int u = 0; u < kTablePer; ++u) {
      const int b = threadIdx.x * per + u;
      if (u >= per || b >= p.batch) continue;
      s_rel[b] = static_cast<int32_t>(sum.rel);
      s_drop[b] = static_cast<int32_t>(sum.drop);
      s_add[b] = static_cast<int32_t>(min(sum.add, static_cast<long long>(INT_MAX)));   // past any list
      s_held[b] = held[u];
      s_need[b] = need[u];
      if (flag[u] == 0) sum = sum + TableSums{rel[u], max(held[u] - need[u], 0), max(need[u] - held[u], 0)};
    }
    __syncthreads();
    const int pushes = static_cast<int>(total.rel + total.drop);
    if (checked || pushes == 0) break;
    // every id that comes back has to be one of the pool's
    checked = true;
    for (long long i0 = first; i0 < pushes; i0 += kTableAhead * step) {
      int b[kTableAhead], id[kTableAhead];
#pragma unroll
      for (int u = 0; u < kTableAhead; ++u) {
        const long long i = i0 + u * step;
        id[u] = 0;
        if (i < pushes) id[u] = *back(static_cast<int>(i), b[u]);
      }
#pragma unroll
      for (int u = 0; u < kTableAhead; ++u) {
        if (id[u] >= 0 && id[u] < p.num_blocks) continue;
        atomicOr(reinterpret_cast<uint32_t*>(s_faulty) + b[u] / 32, 1u << (b[u] % 32));
        s_any = 1;
      }
    }
    row_barrier(p.csize);
    uint64_t any = s_any;
    for (int r = 0; r < p.csize && p.csize > 1; ++r) any |= ld_cluster_u64(&s_any, r);
    if (any == 0) break;
    // requests with such an id stay as they are: once more without them
    if (threadIdx.x < kTableMaxBatch / 64) {
      uint64_t bits = s_faulty[threadIdx.x];
      for (int r = 0; r < p.csize && p.csize > 1; ++r) bits |= ld_cluster_u64(&s_faulty[threadIdx.x], r);
      s_all[2 * threadIdx.x] = static_cast<uint32_t>(bits);
      s_all[2 * threadIdx.x + 1] = static_cast<uint32_t>(bits >> 32);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTablePer; ++u) {
      const int b = threadIdx.x * per + u;
      if (flag[u] == 0 && (s_all[b / 32] >> (b % 32) & 1)) flag[u] = TV_ST_BAD_BLOCK;
    }
  }
  row_barrier(p.csize);                   // every CTA has read what is overwritten from here on
  const int pushes = fail ? 0 : static_cast<int>(total.rel + total.drop);
  const int top = count + pushes;
  for (long long i0 = first; i0 < pushes; i0 += kTableAhead * step) {
    const int32_t* from[kTableAhead];
    int id[kTableAhead];
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u) {
      const long long i = i0 + u * step;
      from[u] = nullptr;
      if (i >= pushes) continue;
      int b;
      from[u] = back(static_cast<int>(i), b);
      id[u] = *from[u];
    }
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u) {
      if (!from[u]) continue;
      const int i = static_cast<int>(i0) + u * step;
      if (i < total.rel) {
        p.free_blocks[count + static_cast<int>(total.rel) - 1 - i] = id[u];
      } else {
        p.free_blocks[top - 1 - (i - static_cast<int>(total.rel))] = id[u];
        *const_cast<int32_t*>(from[u]) = -1;
      }
    }
  }
  // First come, first served: a request whose blocks end past the list gets
  // none, nor does any growing one behind it.
  const int pops = fail ? 0 : static_cast<int>(min(total.add, static_cast<long long>(top)));
  if (pushes > 0 && pops > 0) row_barrier(p.csize);
  for (long long i0 = first; i0 < pops; i0 += kTableAhead * step) {
    int id[kTableAhead];
    int32_t* to[kTableAhead];
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u) {
      to[u] = nullptr;
      if (i0 + u * step >= pops) continue;
      const int i = static_cast<int>(i0) + u * step;
      id[u] = __ldcg(&p.free_blocks[top - 1 - i]);
      const int b = last_at_most(s_add, p.batch, i);
      const int held_b = s_held[b];
      if (s_add[b] <= top - (s_need[b] - held_b)) to[u] = p.table + static_cast<size_t>(b) * p.max_blocks + held_b + (i - s_add[b]);
    }
#pragma unroll
    for (int u = 0; u < kTableAhead; ++u)
      if (to[u]) *to[u] = id[u];
  }
  if (rank != 0) return;
  long long sum = at.add;
#pragma unroll
  for (int u = 0; u < kTablePer; ++u) {
    const int b = threadIdx.x * per + u;
    if (flag[u] < 0) continue;
    int set = fail ? TV_ST_BAD_SIZE : flag[u];
    if (set == 0) {
      const int add = max(need[u] - held[u], 0);
      sum += add;
      if (p.released_count) p.released_count[b] = 0;
      if (add > 0 && sum > top) set = TV_ST_NO_BLOCKS;
      else if (need[u] != held[u]) p.n_blocks[b] = need[u];
      if (add > 0 && sum <= top) atomicMax(&s_taken, static_cast<int>(sum));
    }
    if (set) atomicOr(&p.status[b], set);
  }
  __syncthreads();
  if (threadIdx.x == 0 && !fail) *p.free_count = top - s_taken;
}

// --------------------------------------------------------------------- slots

constexpr int kSlotThreads = 512;
constexpr int kSlotRows = 4;               // rows a thread in large calls

struct SlotParams {
  const int32_t* cu_rows;
  const int32_t* start_len;
  const int32_t* table;
  const int32_t* n_blocks;
  long long* slots;
  int32_t* status;
  int batch, rows, max_blocks, num_blocks, cta_rows;
  bool wide;               // slots lie on 16 bytes
};

// s_off[b] = the largest offset of a thread's requests [b0, b1) up to b, and the largest
// of all requests before b0, which is returned.
__device__ __forceinline__ int scan_offsets(const SlotParams& p, int32_t* s_off, int* s_warp, int& b0, int& b1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.batch + kSlotThreads - 1) / kSlotThreads;
  b0 = min(p.batch, static_cast<int>(threadIdx.x) * per);
  b1 = min(p.batch, b0 + per);
  int most = INT_MIN;
  for (int b = b0; b < b1; ++b) {
    most = max(most, p.cu_rows[b]);
    s_off[b] = most;
  }
  int up = most;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up = max(up, v);
  }
  if (lane == 31) s_warp[warp] = up;
  up = __shfl_up_sync(0xffffffffu, up, 1);
  __syncthreads();
  int before = lane > 0 ? up : INT_MIN;
  for (int w = 0; w < warp; ++w) before = max(before, s_warp[w]);
  return before;
}

// A CTA has a contiguous range of rows, kRows of them side by side a thread (they
// lie in one or two pages: one search, one or two table entries, one wide store). It
// takes the running maximum of all offsets (4 a thread for 2048 requests), in
// which a row finds its request and offsets that run backwards show. Requests that lie
// within the range are checked by their rows. In small calls (a row a thread) the ones
// at its two ends, which may have rows elsewhere, are checked in full by each CTA that has
// some of them. In large ones that would be quadratic in a request's length: a CTA checks
// its own rows alone, and slot_clear_kernel takes back what others wrote for a request
// that one of them flagged. One launch against two, us: 64 trees, 4591 rows 4.1 / 4.2;
// one prompt of 65536 4.1 / 4.2, of 262144 7.2 / 5.2, of 8.4M 1391 / 31; 64 prompts, 1.3M
// rows 13.4 / 10.4; 1000 requests of 1000 rows 13.0 / 10.7.
template <int kRows>
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const __grid_constant__ SlotParams p) {
  extern __shared__ int32_t s_off[];       // running maximum of the offsets, then a request's fault
  int32_t* s_bad = s_off + p.batch;
  __shared__ int s_warp[kSlotThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * p.cta_rows;                  // below rows, whose end may lie at 2^31 - 1
  const int t1 = static_cast<int>(min(static_cast<long long>(p.rows), static_cast<long long>(t0) + p.cta_rows));
  int b0, b1;
  const int before = scan_offsets(p, s_off, s_warp, b0, b1);
  // A request with rows begins where no earlier offset lies behind. Requests
  // that end before they begin have no rows: the first CTA reports them.
  for (int b = b0; b < b1; ++b) {
    const int c0 = p.cu_rows[b], c1 = p.cu_rows[b + 1];
    const int high = max(before, s_off[b]);
    s_off[b] = high;
    int bad = 0;
    if (c1 != c0) {
      const int start = p.start_len[b];
      if (c1 < c0 || c0 < high || c0 < 0 || c1 > p.rows || start < 0) bad = TV_ST_BAD_SIZE;
      else if ((static_cast<long long>(start) + (c1 - c0) - 1) / TV_BLOCK_SIZE >= min(p.n_blocks[b], p.max_blocks))
        bad = TV_ST_BAD_BLOCK;             // (which also keeps slots below 2^31)
      if (p.status[b] != 0) bad = -1;      // flagged before: left out
      else if (bad && blockIdx.x == 0) atomicOr(&p.status[b], bad);
    }
    s_bad[b] = bad;
  }
  __syncthreads();

  int req[kRows], slot[kRows], id[kRows];
  const uint32_t mine = t0 + threadIdx.x * kRows, end = t1;      // (may pass 2^31 - 1)
  int b = 0, c0 = 0, c1 = INT_MIN, start = 0;            // the request of the row before
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    req[u] = -1;
    if (mine + u >= end) continue;
    const int t = static_cast<int>(mine) + u;
    if (p.batch == 0 || s_off[0] > t) continue;
    if (u == 0 || t >= c1 || t < c0) {
      b = last_at_most(s_off, p.batch, t);
      c0 = p.cu_rows[b];
      c1 = p.cu_rows[b + 1];
      start = p.start_len[b];
    }
    if (s_bad[b] != 0 || t < c0 || t >= c1) continue;
    req[u] = b;
    slot[u] = start + (t - c0);
    if (u > 0 && req[u - 1] == b && slot[u] % TV_BLOCK_SIZE != 0) id[u] = id[u - 1];
    else id[u] = p.table[static_cast<size_t>(b) * p.max_blocks + slot[u] / TV_BLOCK_SIZE];
  }
  // the two requests that may have rows elsewhere
  int fault[2] = {-1, -1};
#pragma unroll
  for (int e = 0; e < (kRows == 1 ? 2 : 0); ++e) {
    const int t = e ? t1 - 1 : t0;
    if (p.batch == 0 || s_off[0] > t) continue;
    const int b = last_at_most(s_off, p.batch, t);
    const int c0 = p.cu_rows[b], c1 = p.cu_rows[b + 1];
    if (s_bad[b] != 0 || c1 <= c0 || (c0 >= t0 && c1 <= t1)) continue;
    const int start = p.start_len[b];
    const int page0 = start / TV_BLOCK_SIZE, page1 = (start + (c1 - c0 - 1)) / TV_BLOCK_SIZE;
    const int32_t* row = p.table + static_cast<size_t>(b) * p.max_blocks;
#pragma unroll 4
    for (int j = page0 + threadIdx.x; j <= page1; j += kSlotThreads)
      if (row[j] < 0 || row[j] >= p.num_blocks) fault[e] = b;
  }
  __syncthreads();                         // s_bad is read above and written below
#pragma unroll
  for (int u = 0; u < kRows; ++u)
    if (req[u] >= 0 && (id[u] < 0 || id[u] >= p.num_blocks)) s_bad[req[u]] = TV_ST_BAD_BLOCK;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (fault[e] >= 0) s_bad[fault[e]] = TV_ST_BAD_BLOCK;
  __syncthreads();
  long long out[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    out[u] = -1;
    if (mine + u >= end || req[u] < 0) continue;
    if (s_bad[req[u]] == 0) out[u] = static_cast<long long>(id[u]) * TV_BLOCK_SIZE + slot[u] % TV_BLOCK_SIZE;
    else if (mine + u == static_cast<uint32_t>(max(t0, p.cu_rows[req[u]]))) atomicOr(&p.status[req[u]], TV_ST_BAD_BLOCK);
  }
  if (kRows % 2 == 0 && p.wide && mine + kRows <= end) {
#pragma unroll
    for (int u = 0; u < kRows; u += 2) *reinterpret_cast<longlong2*>(p.slots + mine + u) = make_longlong2(out[u], out[u + 1 < kRows ? u + 1 : u]);
  } else {
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (mine + u < end) p.slots[mine + u] = out[u];
  }
}

// -1 for all rows of requests whose blocks the grid before found wanting. Where none
// is flagged so, a CTA has read the status and is done.
__global__ void __launch_bounds__(kSlotThreads) slot_clear_kernel(const __grid_constant__ SlotParams p) {
  extern __shared__ int32_t s_off[];       // as above, then whether a request's rows go
  int32_t* s_bad = s_off + p.batch;
  __shared__ int s_warp[kSlotThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  bool any = false;
  for (int b = threadIdx.x; b < p.batch; b += kSlotThreads) any |= (p.status[b] & TV_ST_BAD_BLOCK) != 0;
  if (!__syncthreads_or(any)) return;
  int b0, b1;
  const int before = scan_offsets(p, s_off, s_warp, b0, b1);
  for (int b = b0; b < b1; ++b) {          // (rows that two requests claim are not the flagged one's)
    const int c0 = p.cu_rows[b], c1 = p.cu_rows[b + 1];
    s_bad[b] = (p.status[b] & TV_ST_BAD_BLOCK) && c0 >= max(0, max(before, s_off[b])) && c1 <= p.rows;
  }
  __syncthreads();
  for (int b = 0; b < p.batch; ++b) {
    if (!s_bad[b]) continue;
    const int c1 = p.cu_rows[b + 1];
    for (long long t = p.cu_rows[b] + static_cast<long long>(blockIdx.x) * kSlotThreads + threadIdx.x; t < c1;
         t += static_cast<long long>(gridDim.x) * kSlotThreads)
      p.slots[t] = -1;
  }
}

}  // namespace tv

extern "C" int tv_block_tables(int32_t batch, const int32_t* want_len, int32_t* block_table,
                               int32_t* n_blocks, int32_t max_blocks_per_req, int32_t num_blocks,
                               int32_t* free_blocks, int32_t* free_count, const int32_t* released,
                               int32_t* released_count, int32_t* status, void* stream) {
  if (batch < 0 || batch > tv::kTableMaxBatch || max_blocks_per_req < 1 || num_blocks < 1) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!want_len || !block_table || !n_blocks || !free_blocks || !free_count || !status || !released != !released_count)
    return TV_ERR_NULL_POINTER;
  static tv::SmemLimit smem_limit;
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
  const size_t smem = static_cast<size_t>(batch) * 5 * sizeof(int32_t);
  if (!tv::ensure_smem(tv::block_tables_kernel, smem, smem_limit, dev)) return TV_ERR_CUDA;
  tv::TableParams p = {};
  p.want_len = want_len; p.table = block_table; p.n_blocks = n_blocks;
  p.free_blocks = free_blocks; p.free_count = free_count;
  p.released = released; p.released_count = released_count; p.status = status;
  p.batch = batch; p.max_blocks = max_blocks_per_req; p.num_blocks = num_blocks;
  p.csize = tv::kTableCluster;
  const cudaError_t err = tv::launch_cluster_smem_pdl(tv::block_tables_kernel, dim3(p.csize), dim3(tv::kTableThreads),
                                                      p.csize, smem, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

extern "C" int tv_slot_map(int32_t batch, int32_t rows, const int32_t* cu_rows,
                           const int32_t* start_len, const int32_t* block_table,
                           const int32_t* n_blocks, int32_t max_blocks_per_req, int32_t num_blocks,
                           int64_t* slots, int32_t* status, void* stream) {
  if (batch < 0 || batch > tv::kTableMaxBatch || rows < 0 || max_blocks_per_req < 1 || num_blocks < 1 ||
      max_blocks_per_req > (1 << 27))      // (token positions stay below 2^31)
    return TV_ERR_BAD_SIZE;
  if (rows == 0) return TV_OK;
  if (!slots || (batch > 0 && (!cu_rows || !start_len || !block_table || !n_blocks || !status)))
    return TV_ERR_NULL_POINTER;
  if (!tv::aligned(slots, 8)) return TV_ERR_MISALIGNED;
  const int dev = tv::current_device();
  const int sms = dev < 0 ? -1 : tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  tv::SlotParams p = {};
  p.cu_rows = cu_rows; p.start_len = start_len; p.table = block_table; p.n_blocks = n_blocks;
  p.slots = reinterpret_cast<long long*>(slots); p.status = status;
  p.batch = batch; p.rows = rows; p.max_blocks = max_blocks_per_req; p.num_blocks = num_blocks;
  // a row a thread while that leaves SMs with less than two CTAs
  const bool large = rows > static_cast<long long>(sms) * tv::kSlotThreads * 2;
  p.cta_rows = tv::kSlotThreads * (large ? tv::kSlotRows : 1);
  p.wide = tv::aligned(slots, 16);
  const size_t smem = static_cast<size_t>(batch) * 2 * sizeof(int32_t);
  const int ctas = static_cast<int>((rows + static_cast<long long>(p.cta_rows) - 1) / p.cta_rows);
  auto* kernel = large ? tv::slot_map_kernel<tv::kSlotRows> : tv::slot_map_kernel<1>;
  cudaError_t err = tv::launch_pdl(kernel, dim3(ctas), dim3(tv::kSlotThreads), smem, tv::as_stream(stream), p);
  if (err == cudaSuccess && large && batch > 0)
    err = tv::launch_pdl(tv::slot_clear_kernel, dim3(std::min(ctas, 2 * sms)), dim3(tv::kSlotThreads), smem,
                         tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
