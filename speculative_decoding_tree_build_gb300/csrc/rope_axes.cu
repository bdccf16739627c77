// tv_rope_axes: rotary positions with several axes (time, height, width).
//
// Pair i of row t turns by positions[axis(i)][t] * inv_freq[i]. The angle is
// wanted modulo one turn, and float32 has no digits left for that at far
// positions (at position 10^6 its last bit is 0.06 rad). So inv_freq is held
// as a 64-bit fraction of a turn, F = frac(inv_freq / 2 pi) * 2^64, and the
// integer product position * F modulo 2^64 IS the angle's fraction of a turn,
// with an error of |position| * 2^-64 turns from F's own rounding (and of
// 2^-53 of the angle from inv_freq / 2 pi in float64). Its top 32 bits go to
// sincospif.
//
// Memory bound: every value is read and written once, 6 float operations a
// pair. One CTA rotates a few rows; the sines and cosines of a row are
// computed once in shared memory and used by all of its heads.
#include "tv_common.cuh"

namespace tv {

constexpr int kRopeAxThreads = 256;
constexpr int kRopeAxMaxPairs = 256;
constexpr int kRopeAxRows = 4;         // rows per CTA

struct RopeAxParams {
  const void* q;
  const void* k;
  const int32_t* positions;
  const float* inv_freq;
  void* q_out;
  void* k_out;
  long long q_ld, k_ld, q_out_ld, k_out_ld, pos_ld;
  int rows, hq, hkv, d, pairs, style;
  uint8_t axis[kRopeAxMaxPairs];
};

__device__ __forceinline__ float rope_load(const float* p) { return *p; }
__device__ __forceinline__ float rope_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void rope_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// cos and sin of position * inv_freq
__device__ __forceinline__ float2 rope_cos_sin(int position, float inv_freq) {
  double turns = static_cast<double>(inv_freq) * 0.15915494309189533577;   // 1 / (2 pi)
  turns -= floor(turns);
  const unsigned long long f = __double2ull_rn(turns * 18446744073709551616.0);
  const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(position)) * f;
  // the fraction of a turn in [-1/2, 1/2), in half turns for sincospif
  const float half_turns = static_cast<float>(static_cast<int>(a >> 32)) * (1.0f / 2147483648.0f);
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

template <typename T>
__global__ void __launch_bounds__(kRopeAxThreads) rope_axes_kernel(const __grid_constant__ RopeAxParams p) {
  __shared__ float2 s_cs[kRopeAxRows * kRopeAxMaxPairs];
  grid_dependency_wait();
  grid_launch_dependents();
  const int row0 = blockIdx.x * kRopeAxRows;
  const int nrows = min(kRopeAxRows, p.rows - row0);
  for (int i = threadIdx.x; i < nrows * p.pairs; i += blockDim.x) {
    const int r = i / p.pairs, pr = i % p.pairs;
    s_cs[i] = rope_cos_sin(p.positions[p.axis[pr] * p.pos_ld + row0 + r], p.inv_freq[pr]);
  }
  __syncthreads();
  // one thread per pair (or pair of passed-through columns) of one head
  const int half = p.d / 2, rest = p.d - 2 * p.pairs, units = p.pairs + (rest + 1) / 2;
  (void)half;
  const int heads = p.hq + p.hkv;
  for (int i = threadIdx.x; i < nrows * heads * units; i += blockDim.x) {
    const int r = i / (heads * units), h = i / units % heads, u = i % units;
    const long long row = row0 + r;
    const bool isq = h < p.hq;
    const T* src = isq ? static_cast<const T*>(p.q) + row * p.q_ld + static_cast<long long>(h) * p.d
                       : static_cast<const T*>(p.k) + row * p.k_ld + static_cast<long long>(h - p.hq) * p.d;
    T* dst = isq ? static_cast<T*>(p.q_out) + row * p.q_out_ld + static_cast<long long>(h) * p.d
                 : static_cast<T*>(p.k_out) + row * p.k_out_ld + static_cast<long long>(h - p.hq) * p.d;
    if (u < p.pairs) {
      const int ca = p.style ? u : 2 * u, cb = p.style ? u + p.pairs : 2 * u + 1;
      const float2 cs = s_cs[r * p.pairs + u];
      const float a = rope_load(src + ca), b = rope_load(src + cb);
      rope_store(dst + ca, a * cs.x - b * cs.y);
      rope_store(dst + cb, b * cs.x + a * cs.y);
    } else {
      const int c = 2 * u;
      dst[c] = src[c];
      if (c + 1 < p.d) dst[c + 1] = src[c + 1];
    }
  }
}

}  // namespace tv

extern "C" int tv_rope_axes(const tv_rope_axes_geom* g, int32_t rows, int32_t dtype, const void* q,
                            int64_t q_ld, const void* k, int64_t k_ld, const int32_t* positions,
                            int64_t pos_ld, const float* inv_freq, void* q_out, int64_t q_out_ld,
                            void* k_out, int64_t k_out_ld, void* stream) {
  if (g == nullptr) return TV_ERR_NULL_POINTER;
  if (g->num_q_heads < 1 || g->num_kv_heads < 0 || g->num_q_heads > 65536 || g->num_kv_heads > 65536 ||
      g->head_dim < 2 || g->head_dim > 2 * tv::kRopeAxMaxPairs || (g->rope_style != 0 && g->rope_style != 1) ||
      g->num_axes < 1 || g->num_axes > TV_MAX_ROPE_AXES || (g->section_order != 0 && g->section_order != 1))
    return TV_ERR_BAD_GEOMETRY;
  int pairs = 0;
  for (int a = 0; a < g->num_axes; ++a) {
    if (g->section[a] < 0 || g->section[a] > g->head_dim / 2) return TV_ERR_BAD_GEOMETRY;
    pairs += g->section[a];
  }
  if (pairs < 1 || pairs > g->head_dim / 2) return TV_ERR_BAD_GEOMETRY;
  if (dtype != TV_DTYPE_BF16 && dtype != TV_DTYPE_F32) return TV_ERR_BAD_GEOMETRY;
  const bool keys = g->num_kv_heads > 0;
  const long long qn = static_cast<long long>(g->num_q_heads) * g->head_dim;
  const long long kn = static_cast<long long>(g->num_kv_heads) * g->head_dim;
  if (rows < 0 || pos_ld < rows || q_ld < qn || q_out_ld < qn || (keys && (k_ld < kn || k_out_ld < kn)))
    return TV_ERR_BAD_SIZE;
  if (rows == 0) return TV_OK;
  if (!q || !q_out || !positions || !inv_freq || (keys && (!k || !k_out))) return TV_ERR_NULL_POINTER;
  const uintptr_t size = dtype == TV_DTYPE_BF16 ? 2 : 4;
  if (!tv::aligned(q, size) || !tv::aligned(q_out, size) || !tv::aligned(positions, 4) ||
      !tv::aligned(inv_freq, 4) || (keys && (!tv::aligned(k, size) || !tv::aligned(k_out, size))))
    return TV_ERR_MISALIGNED;
  tv::RopeAxParams p = {};
  p.q = q; p.k = k; p.positions = positions; p.inv_freq = inv_freq; p.q_out = q_out; p.k_out = k_out;
  p.q_ld = q_ld; p.k_ld = k_ld; p.q_out_ld = q_out_ld; p.k_out_ld = k_out_ld; p.pos_ld = pos_ld;
  p.rows = rows; p.hq = g->num_q_heads; p.hkv = g->num_kv_heads; p.d = g->head_dim; p.pairs = pairs;
  p.style = g->rope_style;
  int left[TV_MAX_ROPE_AXES] = {0};
  for (int a = 0; a < g->num_axes; ++a) left[a] = g->section[a];
  for (int i = 0, a = 0; i < pairs;) {
    if (left[a] > 0) {
      p.axis[i++] = static_cast<uint8_t>(a);
      --left[a];
      if (g->section_order == 1) a = (a + 1) % g->num_axes;
    } else {
      a = (a + 1) % g->num_axes;
    }
  }
  const dim3 grid((rows + tv::kRopeAxRows - 1) / tv::kRopeAxRows);
  const cudaError_t err = dtype == TV_DTYPE_BF16
      ? tv::launch_pdl(tv::rope_axes_kernel<__nv_bfloat16>, grid, dim3(tv::kRopeAxThreads), 0, tv::as_stream(stream), p)
      : tv::launch_pdl(tv::rope_axes_kernel<float>, grid, dim3(tv::kRopeAxThreads), 0, tv::as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
