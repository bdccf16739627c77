// tv_rope_axes: rotary positions with several axes (time, height, width).
//
// Pair i of row t turns by positions[axis(i)][t] * inv_freq[i]. The angle is
// wanted modulo one turn, and float32 has no digits left for that at far
// positions (at position 10^6 its last bit is 0.06 rad). So inv_freq is held
// as a 64-bit fraction of a turn, F = frac(inv_freq / 2 pi) * 2^64, made from
// the float's significand and the bits of 1 / 2 pi by integer arithmetic, and
// the integer product position * F modulo 2^64 IS the angle's fraction of a
// turn, within |position| * 2^-63 turns. Its top 32 bits (the angle, cut off to
// 2^-32 turns, 1.5e-9 rad) give the quadrant and a remainder of at most an eighth
// of a turn, for which the Taylor series of sine and cosine end below float32's
// last bit after five and six terms.
//
// Memory bound: every value is read and written once, 6 float operations a
// pair. One CTA rotates a few rows (or some heads of one row); the sines and
// cosines of a row are computed once in shared memory. A thread keeps the same
// columns and the same (at most four or eight) heads of every row it takes, so it
// reads a row's sines once into registers and steps its pointers by a fixed
// stride; its first vectors are in flight while the angles are made. 56 us for
// 16201 rows of 40 heads of 128 (332 MB, 5.9 TB/s, half of it writes).
// (Items numbered across rows, heads and columns, with divisions for each,
// float64 for F and sincospif took 175 instructions a vector and were bound
// by issue: 93 us for 332 MB. A small call's time went into divisions of thread
// numbers by variables, and into working out the layout behind the wait for the
// grid before: 8 rows 2.3 us, 2.1 with multiplications, 1.8 with that ahead of
// the wait.)
#include <cstring>

#include "tv_common.cuh"

namespace tv {

constexpr int kRopeAxThreads = 256;
constexpr int kRopeAxMaxPairs = 256;
constexpr int kRopeAxAngles = 2048;    // rows x pairs of a CTA at most
constexpr int kRopeAxBatch = 4;        // heads of a row that a thread takes at most,
constexpr int kRopeAxNarrow = 8;       // and with vectors of 4 or 8 bytes, of rows with more heads than that

struct RopeAxParams {
  const void* q;
  const void* k;
  const int32_t* positions;
  const float* inv_freq;
  void* q_out;
  void* k_out;
  long long q_ld, k_ld, q_out_ld, k_out_ld, pos_ld;
  long long q_step, k_step, q_out_step, k_out_step;   // row_slots rows on
  int rows, hq, heads, d, pairs;
  int cta_rows, cta_heads, groups;     // a CTA's rows and heads; head groups per row block
  int units, rot_units;                // column units of a head; those of them that rotate
  int head_slots, row_slots;           // heads and rows that the CTA's threads take at a time
  int angle_rows;                      // rows whose angles they make at a time
  uint32_t by_span, by_head_slots, by_pairs;          // divisors of thread numbers (thread_divisor)
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

// inv_freq as a 64-bit fraction of a turn, F = frac(inv_freq / 2 pi) 2^64, within
// 2 of its units. |inv_freq| = m 2^(e - 150) with an integer m < 2^24. Below 8, 64
// bits of 1 / 2 pi = C 2^-66 are enough: F = m C 2^(e - 152) modulo 2^64, where
// half a unit of C weighs inv_freq / 8. Above, the bits of 1 / 2 pi ahead of the
// e - 150th make whole turns, and F comes from the 128 bits from there on (the
// reduction of Payne and Hanek, 1983).
__device__ __forceinline__ unsigned long long rope_turns(float inv_freq) {
  constexpr unsigned long long kC = 11743562013128004906ull;         // 2^66 / 2 pi
  const uint32_t bits = __float_as_uint(inv_freq);
  const uint32_t field = (bits >> 23) & 0xffu;
  const unsigned long long m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
  unsigned long long f;
  if (field < 130) {
    const int shift = 152 - static_cast<int>(field ? field : 1u);
    const unsigned long long lo = m * kC, hi = __umul64hi(m, kC);
    if (shift < 64) f = (lo >> shift) | (hi << (64 - shift));
    else f = shift < 128 ? hi >> (shift - 64) : 0ull;
  } else {
    constexpr unsigned long long kB0 = 0x28be60db9391054aull, kB1 = 0x7f09d5f47d4d3770ull;     // 1 / 2 pi
    constexpr unsigned long long kB2 = 0x36d8a5664f10e410ull, kB3 = 0x7f9458eaf7aef158ull;
    const int at = static_cast<int>(field) - 86;                     // the first bit, 64 zeros going ahead
    const int word = at / 64, shift = at % 64;
    const unsigned long long w0 = word == 0 ? 0ull : word == 1 ? kB0 : kB1;
    const unsigned long long w1 = word == 0 ? kB0 : word == 1 ? kB1 : kB2;
    const unsigned long long w2 = word == 0 ? kB1 : word == 1 ? kB2 : kB3;
    const unsigned long long hi = (w0 << shift) | (w1 >> 1 >> (63 - shift)), lo = (w1 << shift) | (w2 >> 1 >> (63 - shift));
    f = m * hi + __umul64hi(m, lo);
  }
  return bits >> 31 ? 0ull - f : f;
}

// (cos, sin) of position * F / 2^64 turns.
__device__ __forceinline__ float2 rope_cos_sin(int position, unsigned long long f) {
  const uint32_t lo = static_cast<uint32_t>(f), hi = static_cast<uint32_t>(f >> 32), pos = static_cast<uint32_t>(position);
  // bits 63..32 of the product: the angle in 2^-32 turns
  const uint32_t a = __umulhi(pos, lo) + pos * hi - (position < 0 ? lo : 0u);
  const uint32_t quarter = (a + 0x20000000u) >> 30;                  // nearest quarter turn
  const float x = static_cast<float>(static_cast<int>(a - (quarter << 30))) * 1.46291807926715968e-9f;   // 2 pi 2^-32
  const float z = x * x;
  // Taylor: |x| <= pi / 4, the first term left out is below 2^-29
  float s = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(z, s, 1.0f / 120.0f);
  s = fmaf(z, s, -1.0f / 6.0f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = fmaf(z, c, -1.0f / 720.0f);
  c = fmaf(z, c, 1.0f / 24.0f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const bool swap = quarter & 1u;
  const float cs = swap ? s : c, sn = swap ? c : s;
  return make_float2(quarter == 1u || quarter == 2u ? -cs : cs, quarter & 2u ? -sn : sn);
}

// Turn the N values of a vector of a pair-interleaved head (N / 2 pairs; the
// first `pairs` of them), or the pairs of two vectors.
template <typename T, int N, int P, bool kTwo>
__device__ __forceinline__ void rope_turn(RopeVec<T, N>& va, RopeVec<T, N>& vb, const float2 (&cs)[P], int pairs) {
#pragma unroll
  for (int j = 0; j < P; ++j) {
    if (j >= pairs) break;
    T& xa = kTwo ? va.x[j] : va.x[2 * j];
    T& xb = kTwo ? vb.x[j] : va.x[2 * j + (N > 1 ? 1 : 0)];
    const float a = rope_float(xa), b = rope_float(xb);
    const float ra = a * cs[j].x - b * cs[j].y, rb = b * cs[j].x + a * cs[j].y;
    rope_round(xa, ra);
    rope_round(xb, rb);
  }
}

// The same for bf16 vectors, two values a conversion.
template <int N, int P, bool kTwo>
__device__ __forceinline__ void rope_turn_bf16(RopeVec<__nv_bfloat16, N>& va, RopeVec<__nv_bfloat16, N>& vb, const float2 (&cs)[P]) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&va);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&vb);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    if constexpr (kTwo) {
      const float a0 = bf16_lo(wa[j]), a1 = bf16_hi(wa[j]), b0 = bf16_lo(wb[j]), b1 = bf16_hi(wb[j]);
      const float2 c0 = cs[2 * j], c1 = cs[2 * j + 1];
      wa[j] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
      wb[j] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
    } else {
      const float a = bf16_lo(wa[j]), b = bf16_hi(wa[j]);
      wa[j] = pack_bf16x2(a * cs[j].x - b * cs[j].y, b * cs[j].x + a * cs[j].y);
    }
  }
}

// T: element, N: elements of a vector, kHalves: rotary style 1 (a pair's two
// columns lie in two vectors; else N = 1 or both are in one vector), kEdge:
// the rotated columns end inside a vector (where both are in one), kBatch: heads
// of a row that a thread takes at most.
template <typename T, int N, bool kHalves, bool kEdge, int kBatch>
__global__ void __launch_bounds__(kRopeAxThreads, kHalves ? 3 : 4) rope_axes_kernel(const __grid_constant__ RopeAxParams p) {
  // pairs of a unit, and whether it holds a second vector
  constexpr int P = kHalves ? N : (N == 1 ? 1 : N / 2);
  constexpr bool kTwo = kHalves || N == 1;
  constexpr bool kPacked = sizeof(T) == 2 && N > 1;
  using Vec = RopeVec<T, N>;
  __shared__ __align__(16) float2 s_cs[kRopeAxAngles];
  grid_launch_dependents();
  const int block = p.groups == 1 ? blockIdx.x : blockIdx.x / p.groups, group = blockIdx.x - block * p.groups;
  const int row0 = block * p.cta_rows, nrows = min(p.cta_rows, p.rows - row0);
  const int head_end = min(p.heads, (group + 1) * p.cta_heads);
  // a thread's first column unit, row and heads (more units than threads: one row and head)
  const int span = min(p.units, kRopeAxThreads);
  const int slot = threadIdx.x * p.by_span >> 16, u0 = threadIdx.x - slot * span;
  const int first_row = slot * p.by_head_slots >> 16;
  const int head0 = first_row < p.row_slots ? group * p.cta_heads + slot - first_row * p.head_slots : head_end;
  const bool at_work = first_row < nrows && head0 < head_end;

  // the columns of a unit's two vectors
  auto columns = [&](int u, int& ca, int& cb) {
    if (u < p.rot_units) {
      ca = kHalves ? u * N : u * (N == 1 ? 2 : N);
      cb = kHalves ? ca + p.pairs : ca + 1;
    } else {                           // (a pair-interleaved head's units of two columns or more cover it in order)
      ca = kTwo ? 2 * p.pairs + (u - p.rot_units) * N : u * N;
      cb = ca;
    }
  };
  Vec va[kBatch], vb[kBatch];
  // the row's heads of q and of k, and the thread's heads in them
  const T *qs, *ks;
  T *qd, *kd;
  int off[kBatch];
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    const int h = head0 + e * p.head_slots;
    off[e] = (h < p.hq ? h : h - p.hq) * p.d;
  }
  int ca, cb;
  columns(u0, ca, cb);
  auto is_q = [&](int e) { return head0 + e * p.head_slots < p.hq; };
  auto point = [&]() {
    const long long row = row0 + first_row;
    qs = static_cast<const T*>(p.q) + row * p.q_ld;
    ks = static_cast<const T*>(p.k) + row * p.k_ld;
    qd = static_cast<T*>(p.q_out) + row * p.q_out_ld;
    kd = static_cast<T*>(p.k_out) + row * p.k_out_ld;
  };
  auto load = [&]() {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (head0 + e * p.head_slots >= head_end) break;
      const T* src = (is_q(e) ? qs : ks) + off[e];
      va[e] = *reinterpret_cast<const Vec*>(src + ca);
      if (kTwo) vb[e] = *reinterpret_cast<const Vec*>(src + cb);
    }
  };
  // the angles' inputs go ahead of the first row, which is on its way while the angles are made
  const int step = p.angle_rows;                             // rows taken at a time, a thread keeps its pair
  const int r0 = threadIdx.x * p.by_pairs >> 16, pr = threadIdx.x - r0 * p.pairs;
  const bool turning = r0 < step && r0 < nrows;
  const int32_t* position = p.positions + p.axis[turning ? pr : 0] * p.pos_ld + row0;
  float inv_freq = 0.0f;
  int pos = 0;
  if (at_work) point();
  grid_dependency_wait();              // (all of the above while the grid before this one ends)
  if (turning) {
    inv_freq = *const_cast<const volatile float*>(p.inv_freq + pr);
    pos = *const_cast<const volatile int32_t*>(position + r0);
  }
  if (at_work) load();
  if (turning) {
    const unsigned long long f = rope_turns(inv_freq);
    s_cs[r0 * p.pairs + pr] = rope_cos_sin(pos, f);
    constexpr int kAhead = 4;                                // further positions in flight together
    for (int r = r0 + step; r < nrows; r += kAhead * step) {
      int next[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = r + i * step < nrows ? *const_cast<const volatile int32_t*>(position + r + i * step) : 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r + i * step < nrows) s_cs[(r + i * step) * p.pairs + pr] = rope_cos_sin(next[i], f);
    }
  }
  __syncthreads();
  if (!at_work) return;

  for (int u = u0; u < p.units; u += kRopeAxThreads) {
    if (u != u0) {
      columns(u, ca, cb);
      point();
    }
    const bool turns = u < p.rot_units;
    for (int r = first_row; r < nrows; r += p.row_slots) {
      if (u != u0 || r != first_row) load();
      float2 cs[P];
      if (turns) {
#pragma unroll
        for (int j = 0; j < P; ++j) cs[j] = s_cs[kEdge ? min(r * p.pairs + u * P + j, kRopeAxAngles - 1) : r * p.pairs + u * P + j];
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (head0 + e * p.head_slots >= head_end) break;
        if (turns) {
          if (kPacked && (!kEdge || u * P + P <= p.pairs)) {
            if constexpr (kPacked) rope_turn_bf16<N, P, kTwo>(va[e], vb[e], cs);
          } else {
            rope_turn<T, N, P, kTwo>(va[e], vb[e], cs, kEdge ? p.pairs - u * P : P);
          }
        }
        T* dst = (is_q(e) ? qd : kd) + off[e];
        *reinterpret_cast<Vec*>(dst + ca) = va[e];
        if (kTwo && turns) *reinterpret_cast<Vec*>(dst + cb) = vb[e];
      }
      qs += p.q_step;
      ks += p.k_step;
      qd += p.q_out_step;
      kd += p.k_out_step;
    }
  }
}

template <typename T, int N, int kBatch>
static cudaError_t launch_rope_axes_with(RopeAxParams& p, bool halves, int sms, cudaStream_t stream) {
  const int per_unit = halves ? N : (N == 1 ? 1 : N / 2);
  p.rot_units = (p.pairs + per_unit - 1) / per_unit;
  p.units = halves || N == 1 ? p.rot_units + (p.d - 2 * p.pairs) / N : p.d / N;
  const int slots = p.units < kRopeAxThreads ? kRopeAxThreads / p.units : 1;
  // Little work (less than a vector a thread for eight CTAs an SM): a CTA takes
  // one sweep, of as many rows as still leave two CTAs for every SM, where
  // those fit at once. Else about ten vectors a thread: all heads of some rows,
  // in the 1 to 4 sweeps over a row's heads that leave the fewest threads idle
  // (40 heads of 8 units: 32 + 8 heads would idle 3 threads in 8; 4 x 10 heads of
  // 3 rows 1 in 16). Single sweeps that do not fit at once cost a second wave:
  // 502 rows of 20 heads of 17 units 3.3 us in 1004 CTAs, 1.8 us in 502.
  const long long row_items = static_cast<long long>(p.heads) * p.units;
  const long long per = row_items * p.rows / (sms * 8);
  p.head_slots = p.heads < slots ? p.heads : slots;
  p.cta_heads = p.head_slots;
  p.row_slots = slots / p.head_slots;
  if (p.row_slots > p.rows / (sms * 2)) p.row_slots = p.rows / (sms * 2);
  if (p.row_slots > kRopeAxAngles / p.pairs) p.row_slots = kRopeAxAngles / p.pairs;
  if (p.row_slots < 1) p.row_slots = 1;
  p.cta_rows = p.row_slots;
  auto row_blocks = [&] { return (static_cast<long long>(p.rows) + p.cta_rows - 1) / p.cta_rows; };    // (rows up to 2^31 - 1)
  const long long sweeps = row_blocks() * ((p.heads + p.cta_heads - 1) / p.cta_heads);
  if (per >= kRopeAxThreads || sweeps > sms * 4) {
    p.cta_heads = p.heads < kBatch * slots ? p.heads : kBatch * slots;
    const long long items = static_cast<long long>(p.cta_heads) * p.units;
    // (twenty narrow vectors: 10181 rows of 26 heads with 50 pairs, float32, 63.5 -> 55.3 us; single elements not)
    constexpr long long kMost = (N > 1 && N * sizeof(T) < 16 ? 20ll : 10ll) * kRopeAxThreads;
    long long rows = (per > kMost ? kMost : per) / items;
    int best = 0;
    for (int k = 1; k <= kBatch; ++k) {
      const int hs = (p.cta_heads + k - 1) / k;
      if (hs > slots) continue;
      // threads at work, in sixteenths of a slot; of two equals the one with more loads in flight a
      // thread, where there are rows enough for it (38 heads of 10 units: 45.7 -> 38.2 us)
      const int busy = slots / hs * p.cta_heads * 16 / k;
      if (busy < best || (busy == best && slots / hs > rows)) continue;
      best = busy;
      p.head_slots = hs;
      p.row_slots = slots / hs;
    }
    if (p.row_slots > kRopeAxAngles / p.pairs) p.row_slots = kRopeAxAngles / p.pairs;
    rows = (rows + p.row_slots - 1) / p.row_slots * p.row_slots;
    if (rows > kRopeAxAngles / p.pairs) rows = kRopeAxAngles / p.pairs;
    p.cta_rows = rows < 1 ? 1 : static_cast<int>(rows);
  }
  p.q_step = p.row_slots * p.q_ld;
  p.k_step = p.row_slots * p.k_ld;
  p.q_out_step = p.row_slots * p.q_out_ld;
  p.k_out_step = p.row_slots * p.k_out_ld;
  p.groups = (p.heads + p.cta_heads - 1) / p.cta_heads;
  p.angle_rows = kRopeAxThreads / p.pairs;
  p.by_span = thread_divisor(p.units < kRopeAxThreads ? p.units : kRopeAxThreads);
  p.by_head_slots = thread_divisor(p.head_slots);
  p.by_pairs = thread_divisor(p.pairs);
  const long long blocks = row_blocks() * p.groups;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  auto* kernel = halves ? rope_axes_kernel<T, N, true, false, kBatch> : rope_axes_kernel<T, N, false, false, kBatch>;
  if constexpr (N > 1) {
    if (!halves && 2 * p.pairs % N != 0) kernel = rope_axes_kernel<T, N, false, true, kBatch>;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRopeAxThreads), 0, stream, p);
}

// Narrow vectors leave little in flight with four heads a thread: with eight, 16
// heads with 59 pairs, float32, 18602 rows 85 -> 73 us, 26 heads with 50 pairs 55
// -> 49 us. With few heads there is nothing to gain (2 + 2 heads with 41 pairs 23 ->
// 26 us), nor with single bf16 values (32 heads with 63 pairs 23 -> 29 us).
template <typename T, int N>
static cudaError_t launch_rope_axes(RopeAxParams& p, bool halves, int sms, cudaStream_t stream) {
  if constexpr (N * sizeof(T) == 4 || N * sizeof(T) == 8) {
    if (p.heads > kRopeAxNarrow) return launch_rope_axes_with<T, N, kRopeAxNarrow>(p, halves, sms, stream);
  }
  return launch_rope_axes_with<T, N, kRopeAxBatch>(p, halves, sms, stream);
}

// The widest vector (16, 8 or 4 bytes, else single elements) that the addresses,
// strides, head dimension and, for pairs of two halves, the pairs allow.
template <typename T>
static cudaError_t launch_rope_axes_any(RopeAxParams& p, bool halves, bool keys, int sms, cudaStream_t stream) {
  auto fits = [&](int n) {
    const uintptr_t bytes = n * sizeof(T);
    return p.d % n == 0 && (!halves || p.pairs % n == 0) && p.q_ld % n == 0 && p.q_out_ld % n == 0 && aligned(p.q, bytes) &&
           aligned(p.q_out, bytes) &&
           (!keys || (p.k_ld % n == 0 && p.k_out_ld % n == 0 && aligned(p.k, bytes) && aligned(p.k_out, bytes)));
  };
  constexpr int kFull = 16 / sizeof(T);
  if (fits(kFull)) return launch_rope_axes<T, kFull>(p, halves, sms, stream);
  if (fits(kFull / 2)) return launch_rope_axes<T, kFull / 2>(p, halves, sms, stream);
  if constexpr (kFull / 4 > 1) {
    if (fits(kFull / 4)) return launch_rope_axes<T, kFull / 4>(p, halves, sms, stream);
  }
  return launch_rope_axes<T, 1>(p, halves, sms, stream);
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
  if (rows < 0 || (pos_ld != 0 && pos_ld < rows) || q_ld < qn || q_out_ld < qn || (keys && (k_ld < kn || k_out_ld < kn)))
    return TV_ERR_BAD_SIZE;
  if (rows == 0) return TV_OK;
  if (!q || !q_out || !positions || !inv_freq || (keys && (!k || !k_out))) return TV_ERR_NULL_POINTER;
  const uintptr_t size = dtype == TV_DTYPE_BF16 ? 2 : 4;
  if (!tv::aligned(q, size) || !tv::aligned(q_out, size) || !tv::aligned(positions, 4) ||
      !tv::aligned(inv_freq, 4) || (keys && (!tv::aligned(k, size) || !tv::aligned(k_out, size))))
    return TV_ERR_MISALIGNED;
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  tv::RopeAxParams p = {};
  p.q = q; p.k = k; p.positions = positions; p.inv_freq = inv_freq; p.q_out = q_out; p.k_out = k_out;
  p.q_ld = q_ld; p.k_ld = k_ld; p.q_out_ld = q_out_ld; p.k_out_ld = k_out_ld; p.pos_ld = pos_ld;
  p.rows = rows; p.hq = g->num_q_heads; p.heads = g->num_q_heads + g->num_kv_heads; p.d = g->head_dim; p.pairs = pairs;
  if (g->section_order == 0) {
    for (int i = 0, a = 0; a < g->num_axes; i += g->section[a++]) memset(p.axis + i, a, g->section[a]);
  } else {
    int left[TV_MAX_ROPE_AXES] = {0};
    for (int a = 0; a < g->num_axes; ++a) left[a] = g->section[a];
    for (int i = 0; i < pairs;) {
      for (int a = 0; a < g->num_axes; ++a) {
        if (left[a] == 0) continue;
        p.axis[i++] = static_cast<uint8_t>(a);
        --left[a];
      }
    }
  }
  const bool halves = g->rope_style == 1;
  const cudaError_t err = dtype == TV_DTYPE_BF16
      ? tv::launch_rope_axes_any<__nv_bfloat16>(p, halves, keys, sms, tv::as_stream(stream))
      : tv::launch_rope_axes_any<float>(p, halves, keys, sms, tv::as_stream(stream));
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}
