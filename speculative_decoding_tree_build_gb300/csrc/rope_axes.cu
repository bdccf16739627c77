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
// pair. One CTA rotates a few rows (or some heads of one row); the sines and
// cosines of a row are computed once in shared memory and used by all of its
// heads, and each thread's first vectors are in flight meanwhile.
#include "tv_common.cuh"

namespace tv {

constexpr int kRopeAxThreads = 256;
constexpr int kRopeAxMaxPairs = 256;
constexpr int kRopeAxMaxRows = 8;      // rows per CTA at most
constexpr int kRopeAxBatch = 4;        // items a thread has in flight

struct RopeAxParams {
  const void* q;
  const void* k;
  const int32_t* positions;
  const float* inv_freq;
  void* q_out;
  void* k_out;
  long long q_ld, k_ld, q_out_ld, k_out_ld, pos_ld;
  int rows, hq, heads, d, pairs;
  int cta_rows, cta_heads, groups;     // a CTA's rows and heads; head groups per row block
  int units, rot_units;                // items of a head; those of them that rotate
  uint32_t units_magic, heads_magic;   // ceil(2^32 / units), ceil(2^32 / cta_heads)
  uint8_t axis[kRopeAxMaxPairs];
};

template <typename T, int N>
struct alignas(sizeof(T) * N) RopeVec {
  T x[N];
};

__device__ __forceinline__ float rope_float(float x) { return x; }
__device__ __forceinline__ float rope_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void rope_round(float& y, float x) { y = x; }
__device__ __forceinline__ void rope_round(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// i / n for i * n < 2^32
__device__ __forceinline__ int rope_div(int i, int n, uint32_t magic) {
  return n == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), magic));
}

// T: element, N: elements of a vector, kHalves: rotary style 1 (a pair's two
// columns lie in two vectors; else N = 1 or both are in one vector).
template <typename T, int N, bool kHalves>
__global__ void __launch_bounds__(kRopeAxThreads) rope_axes_kernel(const __grid_constant__ RopeAxParams p) {
  // pairs of an item, and whether it holds a second vector
  constexpr int P = kHalves ? N : (N == 1 ? 1 : N / 2);
  constexpr bool kTwo = kHalves || N == 1;
  using Vec = RopeVec<T, N>;
  __shared__ unsigned long long s_f[kRopeAxMaxPairs];
  __shared__ __align__(16) float s_cos[kRopeAxMaxRows * kRopeAxMaxPairs];
  __shared__ __align__(16) float s_sin[kRopeAxMaxRows * kRopeAxMaxPairs];
  grid_dependency_wait();
  grid_launch_dependents();
  const int block = blockIdx.x / p.groups, group = blockIdx.x - block * p.groups;
  const int row0 = block * p.cta_rows, nrows = min(p.cta_rows, p.rows - row0);
  const int head0 = group * p.cta_heads;
  const int total = nrows * p.cta_heads * p.units;

  Vec va[kRopeAxBatch], vb[kRopeAxBatch];
  auto place = [&](int i, int& u, int& r, int& h) {
    const int rh = rope_div(i, p.units, p.units_magic);
    u = i - rh * p.units;
    r = rope_div(rh, p.cta_heads, p.heads_magic);
    h = head0 + rh - r * p.cta_heads;
  };
  // the columns of an item's two vectors
  auto columns = [&](int u, int& ca, int& cb) {
    if (u < p.rot_units) {
      ca = kHalves ? u * N : u * (N == 1 ? 2 : N);
      cb = kHalves ? ca + p.pairs : ca + 1;
    } else {
      ca = 2 * p.pairs + (u - p.rot_units) * N;
      cb = -1;
    }
  };
  auto load = [&](int base) {
#pragma unroll
    for (int e = 0; e < kRopeAxBatch; ++e) {
      const int i = base + e * kRopeAxThreads;
      if (i >= total) break;
      int u, r, h, ca, cb;
      place(i, u, r, h);
      if (h >= p.heads) continue;
      columns(u, ca, cb);
      const long long row = row0 + r;
      const T* src = h < p.hq ? static_cast<const T*>(p.q) + row * p.q_ld + static_cast<long long>(h) * p.d
                              : static_cast<const T*>(p.k) + row * p.k_ld + static_cast<long long>(h - p.hq) * p.d;
      va[e] = *reinterpret_cast<const Vec*>(src + ca);
      if (kTwo && cb >= 0) vb[e] = *reinterpret_cast<const Vec*>(src + cb);
    }
  };
  load(threadIdx.x);                   // the first items are on their way while the angles are made

  // inv_freq as a 64-bit fraction of a turn
  for (int i = threadIdx.x; i < p.pairs; i += kRopeAxThreads) {
    double turns = static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= floor(turns);
    s_f[i] = __double2ull_rn(turns * 18446744073709551616.0);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nrows * p.pairs; i += kRopeAxThreads) {
    const int r = i / p.pairs, pr = i - r * p.pairs;
    const long long position = p.positions[p.axis[pr] * p.pos_ld + row0 + r];
    const unsigned long long a = static_cast<unsigned long long>(position) * s_f[pr];
    // the fraction of a turn in [-1/2, 1/2), in half turns for sincospif
    const float half_turns = static_cast<float>(static_cast<int>(a >> 32)) * (1.0f / 2147483648.0f);
    sincospif(half_turns, &s_sin[i], &s_cos[i]);
  }
  __syncthreads();

  for (int base = threadIdx.x; base < total; base += kRopeAxBatch * kRopeAxThreads) {
    if (base != static_cast<int>(threadIdx.x)) load(base);
#pragma unroll
    for (int e = 0; e < kRopeAxBatch; ++e) {
      const int i = base + e * kRopeAxThreads;
      if (i >= total) break;
      int u, r, h, ca, cb;
      place(i, u, r, h);
      if (h >= p.heads) continue;
      columns(u, ca, cb);
      const long long row = row0 + r;
      T* dst = h < p.hq ? static_cast<T*>(p.q_out) + row * p.q_out_ld + static_cast<long long>(h) * p.d
                        : static_cast<T*>(p.k_out) + row * p.k_out_ld + static_cast<long long>(h - p.hq) * p.d;
      if (u < p.rot_units) {
        const float* cs = s_cos + r * p.pairs + u * P;
        const float* sn = s_sin + r * p.pairs + u * P;
#pragma unroll
        for (int j = 0; j < P; ++j) {
          T& xa = kTwo ? va[e].x[j] : va[e].x[2 * j];
          T& xb = kTwo ? vb[e].x[j] : va[e].x[2 * j + (N > 1 ? 1 : 0)];
          const float a = rope_float(xa), b = rope_float(xb);
          rope_round(xa, a * cs[j] - b * sn[j]);
          rope_round(xb, b * cs[j] + a * sn[j]);
        }
        if (kTwo) *reinterpret_cast<Vec*>(dst + cb) = vb[e];
      }
      *reinterpret_cast<Vec*>(dst + ca) = va[e];
    }
  }
}

template <typename T, int N>
static cudaError_t launch_rope_axes(RopeAxParams p, bool halves, cudaStream_t stream) {
  const int per_unit = halves ? N : (N == 1 ? 1 : N / 2);
  p.rot_units = p.pairs / per_unit;
  p.units = p.rot_units + (p.d - 2 * p.pairs) / N;
  // Rows and heads of a CTA: four to ten items a thread when there is work
  // for every SM, down to one item a thread (a head group of one row) when
  // there is little, so that few rows still spread over the chip.
  const long long row_items = static_cast<long long>(p.heads) * p.units;
  long long per = row_items * p.rows / (152 * 8);
  per = per < kRopeAxThreads ? kRopeAxThreads : per > 10 * kRopeAxThreads ? 10 * kRopeAxThreads : per;
  if (per >= row_items) {
    p.cta_rows = static_cast<int>(per / row_items);
    if (p.cta_rows > kRopeAxMaxRows) p.cta_rows = kRopeAxMaxRows;
    p.cta_heads = p.heads;
    p.groups = 1;
  } else {
    p.cta_rows = 1;
    const long long groups = (row_items + per - 1) / per;
    p.cta_heads = static_cast<int>((p.heads + groups - 1) / groups);
    p.groups = (p.heads + p.cta_heads - 1) / p.cta_heads;
  }
  p.units_magic = static_cast<uint32_t>(((1ull << 32) + p.units - 1) / p.units);
  p.heads_magic = static_cast<uint32_t>(((1ull << 32) + p.cta_heads - 1) / p.cta_heads);
  const long long blocks = (p.rows + p.cta_rows - 1) / p.cta_rows * static_cast<long long>(p.groups);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  auto* kernel = halves ? rope_axes_kernel<T, N, true> : rope_axes_kernel<T, N, false>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRopeAxThreads), 0, stream, p);
}

// The widest vector (16 or 8 bytes, else single elements) that the addresses,
// strides, head dimension and pairs allow.
template <typename T>
static cudaError_t launch_rope_axes_any(const RopeAxParams& p, bool halves, bool keys, cudaStream_t stream) {
  auto fits = [&](int n) {
    const uintptr_t bytes = n * sizeof(T);
    const int cols = halves ? p.pairs : 2 * p.pairs;
    return p.d % n == 0 && cols % n == 0 && p.q_ld % n == 0 && p.q_out_ld % n == 0 && aligned(p.q, bytes) &&
           aligned(p.q_out, bytes) &&
           (!keys || (p.k_ld % n == 0 && p.k_out_ld % n == 0 && aligned(p.k, bytes) && aligned(p.k_out, bytes)));
  };
  constexpr int kFull = 16 / sizeof(T);
  if (fits(kFull)) return launch_rope_axes<T, kFull>(p, halves, stream);
  if (fits(kFull / 2)) return launch_rope_axes<T, kFull / 2>(p, halves, stream);
  return launch_rope_axes<T, 1>(p, halves, stream);
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
  p.rows = rows; p.hq = g->num_q_heads; p.heads = g->num_q_heads + g->num_kv_heads; p.d = g->head_dim; p.pairs = pairs;
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
  const bool halves = g->rope_style == 1;
  const cudaError_t err = dtype == TV_DTYPE_BF16
      ? tv::launch_rope_axes_any<__nv_bfloat16>(p, halves, keys, tv::as_stream(stream))
      : tv::launch_rope_axes_any<float>(p, halves, keys, tv::as_stream(stream));
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
