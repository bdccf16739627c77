// tv_kv_rows_write and tv_kv_rows_read: K/V rows between [rows][Hkv][D] arrays
// and slots of the bf16 paged cache.
//
// A copy of 16-byte vectors, bound by memory (half reads, half writes). A row's
// vectors (K's heads, then V's) lie side by side in the array and D * 2 bytes
// at a time in the pool. A CTA takes a contiguous run of rows; its threads step
// through their vectors with kRowsAhead loads in flight. All slots of the run
// are fetched first, one round trip ahead of the rows.
#include "tv_common.cuh"

namespace tv {

constexpr int kRowsThreads = 256;
constexpr int kRowsAhead = 4;              // vectors a thread has in flight
constexpr int kRowsMax = 256;              // rows a CTA at most
constexpr int kRowsMaxHeads = 4096;

struct RowsParams {
  uint4* k_rows;
  uint4* v_rows;
  long long k_ld, v_ld;                    // in vectors
  const long long* slots;
  uint4* k_cache;
  uint4* v_cache;
  long long num_slots;
  int rows, hkv, cta_rows;
};

template <bool kWrite, int kVecs>          // kVecs: vectors of a head's row
__global__ void __launch_bounds__(kRowsThreads) kv_rows_kernel(const __grid_constant__ RowsParams p) {
  __shared__ long long s_slot[kRowsMax];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long t0 = static_cast<long long>(blockIdx.x) * p.cta_rows;
  const int nrows = static_cast<int>(min(static_cast<long long>(p.cta_rows), p.rows - t0));
  for (int r = threadIdx.x; r < nrows; r += kRowsThreads) {
    const long long s = p.slots[t0 + r];
    s_slot[r] = s >= 0 && s < p.num_slots ? s : -1;
  }
  __syncthreads();
  const uint32_t row_vecs = 2u * p.hkv * kVecs;
  const long long total = static_cast<long long>(nrows) * row_vecs;
  for (long long i0 = threadIdx.x; i0 < total; i0 += kRowsAhead * kRowsThreads) {
    const uint4* from[kRowsAhead];
    uint4* to[kRowsAhead];
    uint4 x[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const long long i = i0 + u * kRowsThreads;
      to[u] = nullptr;
      if (i >= total) continue;
      const uint32_t r = static_cast<uint32_t>(i / row_vecs), e = static_cast<uint32_t>(i - static_cast<long long>(r) * row_vecs);
      const long long slot = s_slot[r];
      if (slot < 0) continue;
      const bool isv = e >= row_vecs / 2;
      const uint32_t c = isv ? e - row_vecs / 2 : e;       // the vector among K's or V's
      uint4* row = (isv ? p.v_rows : p.k_rows) + (t0 + r) * (isv ? p.v_ld : p.k_ld) + c;
      uint4* pool = (isv ? p.v_cache : p.k_cache) +
                    ((slot / TV_BLOCK_SIZE * p.hkv + c / kVecs) * TV_BLOCK_SIZE + slot % TV_BLOCK_SIZE) * kVecs + c % kVecs;
      from[u] = kWrite ? row : pool;
      to[u] = kWrite ? pool : row;
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (to[u]) x[u] = *from[u];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (to[u]) *to[u] = x[u];
  }
}

template <bool kWrite>
static int launch_rows(const tv_geom* geom, int rows, const void* k_rows, long long k_ld, const void* v_rows,
                       long long v_ld, const int64_t* slots, const void* k_cache, const void* v_cache,
                       int num_blocks, void* stream) {
  int rc = check_geom(geom);
  if (rc != TV_OK) return rc;
  if (geom->num_kv_heads > kRowsMaxHeads) return TV_ERR_BAD_GEOMETRY;
  const long long width = static_cast<long long>(geom->num_kv_heads) * geom->head_dim;
  if (rows < 0 || num_blocks < 1 || k_ld < width || v_ld < width) return TV_ERR_BAD_SIZE;
  if (rows == 0) return TV_OK;
  if (!k_rows || !v_rows || !slots || !k_cache || !v_cache) return TV_ERR_NULL_POINTER;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || (k_ld & 7) || (v_ld & 7) || !aligned(slots, 8) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return TV_ERR_MISALIGNED;
  RowsParams p = {};
  p.k_rows = static_cast<uint4*>(const_cast<void*>(k_rows));
  p.v_rows = static_cast<uint4*>(const_cast<void*>(v_rows));
  p.k_ld = k_ld / 8; p.v_ld = v_ld / 8;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.k_cache = static_cast<uint4*>(const_cast<void*>(k_cache));
  p.v_cache = static_cast<uint4*>(const_cast<void*>(v_cache));
  p.num_slots = static_cast<long long>(num_blocks) * TV_BLOCK_SIZE;
  p.rows = rows; p.hkv = geom->num_kv_heads;
  // the rows that kRowsAhead vectors a thread cover
  const long long each = static_cast<long long>(kRowsThreads) * kRowsAhead * 8 / (2 * width);
  p.cta_rows = static_cast<int>(each < 1 ? 1 : each > kRowsMax ? kRowsMax : each);
  const dim3 grid(static_cast<unsigned>((rows + static_cast<long long>(p.cta_rows) - 1) / p.cta_rows));
  auto* kernel = geom->head_dim == 64 ? kv_rows_kernel<kWrite, 8> : kv_rows_kernel<kWrite, 16>;
  return launch_pdl(kernel, grid, dim3(kRowsThreads), 0, as_stream(stream), p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv

extern "C" int tv_kv_rows_write(const tv_geom* geom, int32_t rows, const void* k_new, int64_t k_ld,
                                const void* v_new, int64_t v_ld, const int64_t* slots, void* k_cache,
                                void* v_cache, int32_t num_blocks, void* stream) {
  return tv::launch_rows<true>(geom, rows, k_new, k_ld, v_new, v_ld, slots, k_cache, v_cache, num_blocks, stream);
}

extern "C" int tv_kv_rows_read(const tv_geom* geom, int32_t rows, const int64_t* slots,
                               const void* k_cache, const void* v_cache, int32_t num_blocks,
                               void* k_out, int64_t k_ld, void* v_out, int64_t v_ld, void* stream) {
  return tv::launch_rows<false>(geom, rows, k_out, k_ld, v_out, v_ld, slots, k_cache, v_cache, num_blocks, stream);
}
