// tv_decode_attention: attention of one new token per request over its paged
// cache, bf16 or 8 bits.
//
//   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
//
// One warp per query head; a lane holds D / 32 columns and the warp walks the
// cache with the running maximum and sum of the softmax.
#include "tv_kv8.cuh"

namespace tv {

struct DecodeParams {
  const __nv_bfloat16* q;
  long long q_ld;
  const int32_t* seq_len;
  const int32_t* block_table;
  const int32_t* n_blocks;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
  int batch, hq, hkv, group, max_blocks, num_blocks;
  float scale_log2;
};

template <int kFmt, int N>
__device__ __forceinline__ void decode_load(const void* cache, size_t elem, float (&x)[N]) {
  if constexpr (kFmt == TV_KV_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[elem + i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(cache) + elem + i);
      const float2 f = kv_decode2<kFmt>(w);
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}

template <int kFmt, int D>
__global__ void __launch_bounds__(512) decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int N = D / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.x / p.hkv, kvh = blockIdx.x % p.hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int st = p.status[b], n = p.seq_len[b], held = min(p.n_blocks[b], p.max_blocks);
  if (st != 0) return;
  const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  int bad = n < 0 ? TV_ST_BAD_SIZE : 0;
  const int pages = n > 0 ? (n - 1) / TV_BLOCK_SIZE + 1 : 0;
  if (!bad && pages > held) bad = TV_ST_BAD_BLOCK;
  if (!bad) {
    for (int e = threadIdx.x; e < pages; e += blockDim.x) {
      const int blk = row[e];
      if (blk < 0 || blk >= p.num_blocks) bad = TV_ST_BAD_BLOCK;
    }
  }
  if (__syncthreads_or(bad)) {
    if (bad) atomicOr(p.status + b, bad);
    return;
  }
  const int h = kvh * p.group + warp;
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  decode_load<TV_KV_BF16, N>(p.q, static_cast<size_t>(b) * p.q_ld + static_cast<size_t>(h) * D + lane * N, q);
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.0f;
  for (int j = 0; j < n; ++j) {
    const size_t r = (static_cast<size_t>(row[j / TV_BLOCK_SIZE]) * p.hkv + kvh) * TV_BLOCK_SIZE + j % TV_BLOCK_SIZE;
    float k[N], v[N], s = 0.0f;
    decode_load<kFmt, N>(p.k_cache, r * D + lane * N, k);
    decode_load<kFmt, N>(p.v_cache, r * D + lane * N, v);
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    float vs = 1.0f;
    if (kFmt != TV_KV_BF16) {
      s *= p.k_scale[r];
      vs = p.v_scale[r];
    }
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.0f : mn;
    const float down = exp2f(m - ref), e = exp2f(s - ref);
    l = l * down + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * down + e * vs * v[i];
    m = mn;
  }
  const float inv = n == 0 ? 0.0f : 1.0f / l;
  __nv_bfloat16* out = p.out + (static_cast<size_t>(b) * p.hq + h) * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __float2bfloat16_rn(o[i] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<size_t>(b) * p.hq + h] = n == 0 ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace tv

extern "C" int tv_decode_workspace_bytes(const tv_geom* geom, int32_t batch, size_t* bytes) {
  int rc = tv::check_geom(geom);
  if (rc != TV_OK) return rc;
  if (bytes == nullptr) return TV_ERR_NULL_POINTER;
  if (batch < 0 || batch > tv::kKvMaxBatch) return TV_ERR_BAD_SIZE;
  *bytes = 256;
  return TV_OK;
}

extern "C" int tv_decode_attention(const tv_geom* geom, int32_t kv_format, int32_t batch,
                                   const void* q, int64_t q_ld, const int32_t* seq_len,
                                   const int32_t* block_table, const int32_t* n_blocks,
                                   int32_t max_blocks_per_req, const void* k_cache,
                                   const void* v_cache, const float* k_scale,
                                   const float* v_scale, int32_t num_blocks, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int32_t* status,
                                   void* stream) {
  int rc = tv::check_geom(geom);
  if (rc != TV_OK) return rc;
  if (kv_format != TV_KV_BF16 && kv_format != TV_KV_E4M3 && kv_format != TV_KV_INT8) return TV_ERR_BAD_GEOMETRY;
  if (batch < 0 || batch > tv::kKvMaxBatch || max_blocks_per_req < 1 || num_blocks < 1 ||
      q_ld < static_cast<long long>(geom->num_q_heads) * geom->head_dim)
    return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  const bool scaled = kv_format != TV_KV_BF16;
  if (!q || !seq_len || !block_table || !n_blocks || !k_cache || !v_cache || !out || !workspace || !status ||
      (scaled && (!k_scale || !v_scale)))
    return TV_ERR_NULL_POINTER;
  if (!tv::aligned(q, 16) || q_ld % 8 != 0 || !tv::aligned(k_cache, 16) || !tv::aligned(v_cache, 16) ||
      !tv::aligned(out, 16) || (lse && !tv::aligned(lse, 4)) || !tv::aligned(workspace, 256) ||
      (scaled && (!tv::aligned(k_scale, 16) || !tv::aligned(v_scale, 16))))
    return TV_ERR_MISALIGNED;
  size_t need = 0;
  rc = tv_decode_workspace_bytes(geom, batch, &need);
  if (rc != TV_OK) return rc;
  if (workspace_bytes < need) return TV_ERR_WORKSPACE;
  tv::DecodeParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_ld = q_ld;
  p.seq_len = seq_len; p.block_table = block_table; p.n_blocks = n_blocks;
  p.k_cache = k_cache; p.v_cache = v_cache; p.k_scale = k_scale; p.v_scale = v_scale;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse; p.status = status;
  p.batch = batch; p.hq = geom->num_q_heads; p.hkv = geom->num_kv_heads;
  p.group = geom->num_q_heads / geom->num_kv_heads;
  p.max_blocks = max_blocks_per_req; p.num_blocks = num_blocks;
  const float scale = geom->softmax_scale > 0.0f ? geom->softmax_scale : 1.0f / sqrtf(static_cast<float>(geom->head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  void (*kernel)(tv::DecodeParams) = nullptr;
  const bool d64 = geom->head_dim == 64;
  if (kv_format == TV_KV_BF16) kernel = d64 ? tv::decode_kernel<TV_KV_BF16, 64> : tv::decode_kernel<TV_KV_BF16, 128>;
  else if (kv_format == TV_KV_E4M3) kernel = d64 ? tv::decode_kernel<TV_KV_E4M3, 64> : tv::decode_kernel<TV_KV_E4M3, 128>;
  else kernel = d64 ? tv::decode_kernel<TV_KV_INT8, 64> : tv::decode_kernel<TV_KV_INT8, 128>;
  const cudaError_t err = tv::launch_pdl(kernel, dim3(batch * p.hkv), dim3(32 * p.group), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
