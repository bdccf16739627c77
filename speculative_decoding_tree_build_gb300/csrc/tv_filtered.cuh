// tv_sample_filtered and tv_filter_logits: temperature, top-k, top-p, min-p.
//
// A row's tokens are ordered by (logit descending, index ascending); what is
// kept is a prefix of that order, so a filter is one place in it: the last kept
// token. Places are 64-bit numbers, the logit's order key above the inverted
// index, and comparing two of them is comparing integers; ties need no care
// anywhere else.
//
// Finding the place without sorting the row:
//   1. a sample of the row in 128-byte lines gives a place above which some
//      hundred tokens of the row lie;
//   2. one pass over the row lists those (shared memory) and, where top-p needs
//      the total, sums the weights of the others in float32 with a bound on the
//      error;
//   3. on the list, a histogram over places finds the bin in which the count
//      (top-k) or the sum of weights (top-p) is reached; its few tokens are
//      ranked by one warp.
// Where the place is not on the list (top-k larger than the list, a flat row whose
// top-p set is a tenth of the vocabulary, many equal logits), another pass lists
// the tokens around a place that a sample gives and sums those above and below
// with a tighter bound. Every pass shrinks the bounds on the place, and from the
// fifth on it halves them. Where a bound on the sums leaves the border open, a
// pass with exact weights settles it.
//
// Weights of listed tokens are integers (tv_weight.cuh) and their sums exact: no
// result depends on the order of the atomics that build lists and histograms.
//
// One CTA has a row, or a cluster where rows are few: its CTAs pass over slices,
// exchange lists and sums through distributed shared memory, and all of them take
// the same decisions.
#pragma once

#include <cfloat>
#include <cuda_bf16.h>

#include "tv_cluster.cuh"
#include "tv_filter_params.h"
#include "tv_weight.cuh"

// A unit names its space and its CTA's size before it includes this; filtered.cu chooses.
namespace tv {
namespace TV_FILT_SPACE {

constexpr int kFiltThreads = TV_FILT_THREADS;
constexpr int kFiltWarps = kFiltThreads / 32;
constexpr int kFiltPerSm = 1024 / kFiltThreads;    // CTAs an SM
constexpr int kFiltMaxCluster = 8;
constexpr int kListCap = kFiltThreads == 256 ? 3840 : 4864;   // (with kLocalCap, what shared memory holds)
constexpr int kLocalCap = 4 * kFiltThreads;        // a CTA's own part of the list in a cluster
constexpr int kSampleEach = 8;             // sampled tokens a thread
constexpr int kSampleSize = kSampleEach * kFiltThreads;
constexpr int kSamplePieces = 4;           // samples that a second look takes
constexpr int kFirstList = 256;            // tokens that the first list is made for without top-k
constexpr int kBinBits = kFiltThreads == 512 ? 11 : kFiltThreads == 256 ? 10 : 9, kBins = 1 << kBinBits;
static_assert(kBins == 4 * kFiltThreads, "a thread clears 16 bytes of them and sums four");
constexpr int kHits = 4 * kBins;           // noted vectors of a pass (where the bins lie otherwise)
constexpr int kSmall = 32;                 // tokens that a warp ranks
constexpr int kSampledTurns = 4, kTurns = kSampledTurns + 64;
constexpr int kFiltUnroll = 2;             // 16-byte loads in flight a thread, first look
constexpr float kInf = __builtin_huge_valf();

// Places: (order key, ~index). -inf has no place: it is never kept.
constexpr uint64_t kLowest = static_cast<uint64_t>(0x00800000u) << 32;   // just above -inf (order key 0x007fffff)
constexpr uint64_t kHighest = ~0ull;

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float place_value(uint64_t c) { return key_value(static_cast<uint32_t>(c >> 32)); }

struct FiltSmem {
  uint32_t bins[4][kBins];                 // counts; weights in three parts
  WeightTable table;
  uint64_t red[6][kFiltWarps];
  uint64_t small[kSmall];
  uint64_t found, before, weight;          // of select
  uint64_t stat[6];                        // of a pass: listed, above, three sums, the largest key
  int bin, bin_count, n_small, n_list, n_hits;
  int rank, lo_bin, hi_bin;                // of a bracket
  uint64_t list[kListCap];                 // in a cluster the CTA's own part follows
};

// ---------------------------------------------------------------- reductions

// Three parts of 22 bits: sums of 32 fit a register, and a warp adds a register
// in one instruction.
__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
  const uint64_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0x3fffffu);
  const uint64_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 22) & 0x3fffffu);
  const uint64_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 44));
  return a + (b << 22) + (c << 44);
}
// The larger high half, then the larger low half of those that have it.
__device__ __forceinline__ uint64_t warp_top_u64(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32), high = __reduce_max_sync(0xffffffffu, hi);
  return static_cast<uint64_t>(high) << 32 | __reduce_max_sync(0xffffffffu, hi == high ? static_cast<uint32_t>(v) : 0u);
}

// Sums (or, from kMax on, maxima) of kN numbers over the CTA.
template <int kN, int kMax>
__device__ __forceinline__ void block_reduce(uint64_t (&v)[kN], FiltSmem& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = i >= kMax ? warp_top_u64(v[i]) : warp_sum_u64(v[i]);
  __syncthreads();                         // what was there is read
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) s.red[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kFiltWarps; ++w) {
      const uint64_t x = s.red[i][w];
      all = i >= kMax ? (x > all ? x : all) : all + x;
    }
    v[i] = all;
  }
}

__device__ __forceinline__ uint64_t block_sum(uint64_t v, FiltSmem& s) {
  uint64_t x[1] = {v};
  block_reduce<1, 1>(x, s);
  return x[0];
}
__device__ __forceinline__ uint64_t block_max(uint64_t v, FiltSmem& s) {
  uint64_t x[1] = {v};
  block_reduce<1, 0>(x, s);
  return x[0];
}
__device__ __forceinline__ float block_sum(float v, FiltSmem& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[0][threadIdx.x >> 5] = __float_as_uint(v);
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) t += __uint_as_float(static_cast<uint32_t>(s.red[0][w]));
  return t;
}

// ------------------------------------------------------------------ the row

template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int kLen = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int kLen = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
  }
  // values that were bf16 before
  static __device__ __forceinline__ uint4 pack(const float* x) {
    auto two = [](float a, float b) { return __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xffff0000u); };
    return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
  }
};

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) {
  *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(__float_as_uint(x) >> 16);
}

// A row and the CTA's slice [v0, v1) of it; v0 is a multiple of 8.
template <typename T>
struct Row {
  const T* x;
  int vocab, v0, v1;
  int rank, csize;
  float inv_t;
  int bits;
};

__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// f.many<n>(x, first index) for all entries of the slice, n at a time (the
// ragged end one by one). kAhead > 0: the first look at the row, lines that far ahead
// (in steps of the loop) are fetched to L2, since 32 bytes a thread in flight leave
// the memory idle; two loads at a time (4112 rows of 151936: 580 us, with one load ahead
// of the work 603). Later looks find the row in L2 more often than not, with one load ahead of
// the work (24 ragged requests masked: 349 us, with two loads at a time 377).
template <int kAhead, typename T, typename F>
__device__ __forceinline__ void for_slice(const Row<T>& row, F& f) {
  constexpr int kLen = Vec<T>::kLen;
  const uint4* vecs = reinterpret_cast<const uint4*>(row.x + row.v0);
  const int n = (row.v1 - row.v0) / kLen;
  if constexpr (kAhead > 0) {
    for (int j0 = threadIdx.x; j0 < n; j0 += kFiltUnroll * kFiltThreads) {
      uint4 v[kFiltUnroll];
#pragma unroll
      for (int u = 0; u < kFiltUnroll; ++u)
        if (j0 + u * kFiltThreads < n) v[u] = vecs[j0 + u * kFiltThreads];
      if (threadIdx.x < kFiltUnroll * kFiltThreads / 8) {
        const int line = (j0 - static_cast<int>(threadIdx.x)) + kAhead * kFiltUnroll * kFiltThreads + threadIdx.x * 8;
        if (line < n) prefetch_line(vecs + line);
      }
#pragma unroll
      for (int u = 0; u < kFiltUnroll; ++u) {
        const int j = j0 + u * kFiltThreads;
        if (j >= n) break;
        float x[kLen];
        Vec<T>::unpack(v[u], x);
        f.template many<kLen>(x, row.v0 + j * kLen);
      }
    }
  } else {
    uint4 next;
    if (threadIdx.x < n) next = vecs[threadIdx.x];
    for (int j = threadIdx.x; j < n; j += kFiltThreads) {
      const uint4 v = next;
      if (j + kFiltThreads < n) next = vecs[j + kFiltThreads];
      float x[kLen];
      Vec<T>::unpack(v, x);
      f.template many<kLen>(x, row.v0 + j * kLen);
    }
  }
  const int i = row.v0 + n * kLen + threadIdx.x;
  if (i < row.v1) {
    float x[1] = {load_one(row.x + i)};
    f.template many<1>(x, i);
  }
}

// Sum (or maximum) over the cluster of what each CTA left in s.stat: a lane reads
// a CTA's (clusters are powers of two up to 8). For whole warps.
template <bool kMax>
__device__ __forceinline__ uint64_t cluster_stat(const FiltSmem& s, int i, int csize) {
  if (csize == 1) return s.stat[i];
  uint64_t v = ld_cluster_u64(&s.stat[i], (threadIdx.x & 31) & (csize - 1));
  for (int o = csize >> 1; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? (w > v ? w : v) : v + w;
  }
  return v;
}

// ------------------------------------------------------------------ the pass

// What a pass does with the tokens that it does not list: nothing; sum the
// weights below the list, cheaply; sum those below and above within 2^-28; weigh
// exactly.
enum class Weigh { kNone, kBelow, kClose, kExact };

// One pass over the row: places in [lo, hi] are listed (as many as fit, all are
// counted), those above are counted. Weights are relative to the scale given.
struct Bracket {
  uint64_t lo, hi;
  int n_in, n_above;
  uint64_t m_above, below, total;    // (kBelow: below alone, kClose: not below)
  bool whole;                        // the list holds all places in [lo, hi]
  float top;                         // the largest logit from lo on
  bool any;                          // there is one
};

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// A float32 sum with its roundings beside it.
struct FloatSum {
  float sum, low;
  __device__ __forceinline__ void add(float part) {
    const float all = sum + part, back = all - sum;
    low += (sum - (all - back)) + (part - back);
    sum = all;
  }
  __device__ __forceinline__ void scale(float factor) {
    const float all = sum * factor;
    low = __fmaf_rn(low, factor, __fmaf_rn(sum, factor, -all));
    sum = all;
  }
  __device__ __forceinline__ uint64_t steps(float unit) const {
    return static_cast<uint64_t>(__float2ll_rn(sum * unit) + __float2ll_rn(low * unit));
  }
};

// A sum of close weights of at most 2: the multiples of 2^-12 in w add up without
// rounding below 2^12; what is left of w, and w q, is small.
struct ClosePart {                   // of one vector
  float high, low;
  __device__ __forceinline__ void add(const CloseWeight& c) {
    constexpr float kGrid = 0x1.8p11f;                                   // last bit 2^-12
    const float grid = (c.w + kGrid) - kGrid;
    high += grid;
    low += __fmaf_rn(c.w, c.q, c.w - grid);
  }
};
struct CloseSum {
  float high;
  FloatSum low;
  uint64_t put;                      // moved out of `high`, in steps
  __device__ __forceinline__ void add(const ClosePart& p, float unit) {
    high += p.high;
    low.add(p.low);
    if (high >= 2048.0f) {
      put += static_cast<uint64_t>(__float2ll_rn(high * unit));
      high = 0.0f;
    }
  }
  __device__ __forceinline__ uint64_t steps(float unit) const {
    return put + static_cast<uint64_t>(__float2ll_rn(high * unit)) + low.steps(unit);
  }
};

template <Weigh kWeigh, typename T>
struct PassBody {
  FiltSmem& s;
  const Row<T>& row;
  uint64_t* list;                    // the CTA's own
  int cap;
  uint64_t lo, hi;
  float lo_value, hi_value, to_y, y_off, unit;
  WeightScale scale;
  uint32_t best;                     // the largest order key from lo on
  int n_above;
  uint64_t m_in, m_above, below;
  FloatSum f_below;                  // kBelow
  CloseSum c_all, c_above;           // kClose: of all tokens, of those above the bracket

  // 2^(y - k), y = x to_y: the factor's rounding makes the exponent good to |y| 2^-22.8.
  __device__ __forceinline__ float cheap(float x) const { return fast_exp2(__fmaf_rn(x, to_y, y_off)); }

  __device__ __forceinline__ CloseWeight close(float x) const { return close_weight(__fmul_rn(x, row.inv_t), scale, s.table); }
  // (a logit of -inf weighs nothing, also where all others are scaled to -inf and weigh 1)
  __device__ __forceinline__ uint64_t exact(float x) const {
    return x == -kInf ? 0ull : weight_of(__fmul_rn(x, row.inv_t), scale, s.table);
  }

  // a token that may lie in the bracket
  __device__ __forceinline__ void take(float x, int i) {
    const uint32_t key = order_key(x);
    const uint64_t c = pack_best(key, i);
    if (c < lo || c > hi) {
      if (c < lo) {
        if (kWeigh == Weigh::kExact) below += exact(x);
        if (kWeigh == Weigh::kBelow) f_below.add(cheap(x));
      } else {
        best = key > best ? key : best;
        ++n_above;
        if (kWeigh == Weigh::kExact) m_above += exact(x);
      }
      if (kWeigh == Weigh::kClose && c > hi) {
        ClosePart part = {0.0f, 0.0f};
        part.add(close(x));
        c_above.add(part, unit);
      }
      return;
    }
    best = key > best ? key : best;
    const int at = atomicAdd(&s.n_list, 1);
    if (at < cap) list[at] = c;
    if (kWeigh == Weigh::kExact) m_in += exact(x);
  }

  // those of a vector (or of a single entry at the slice's end) that may
  template <int kLen>
  __device__ __forceinline__ void take_all(int i0) {
    float x[kLen];
    if constexpr (kLen > 1) Vec<T>::unpack(*reinterpret_cast<const uint4*>(row.x + i0), x);
    else x[0] = load_one(row.x + i0);
#pragma unroll
    for (int e = 0; e < kLen; ++e)
      if (!(x[e] < lo_value) && (kWeigh == Weigh::kBelow || !(x[e] > hi_value))) take(x[e], i0 + e);
  }
  __device__ __forceinline__ void take_hits() {
    constexpr int kLen = Vec<T>::kLen;
    const int n = min(s.n_hits, kHits);
    for (int h = threadIdx.x; h < n; h += kFiltThreads) {
      const int i0 = static_cast<int>(s.bins[0][h]);
      if (i0 + kLen <= row.v1) take_all<kLen>(i0);
      else take_all<1>(i0);
    }
  }

  // Vectors with such tokens are noted, and looked at when all threads have some: one in a
  // hundred vectors has one, and a warp that stopped for it would stop nearly always.
  template <int kLen>
  __device__ __forceinline__ void note(int i0) {
    const int at = atomicAdd(&s.n_hits, 1);
    if (at < kHits) s.bins[0][at] = i0;
    else take_all<kLen>(i0);
  }

  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
    if (kWeigh == Weigh::kNone || kWeigh == Weigh::kBelow) {
      // most vectors lie below the list as a whole (a NaN does not)
      float high = x[0];
#pragma unroll
      for (int e = 1; e < kLen; ++e) high = max_or_nan(high, x[e]);
      if (kWeigh == Weigh::kBelow) {       // (for all of a warp's vectors alike: no lane waits for others)
        float low = 0.0f;
#pragma unroll
        for (int e = 0; e < kLen; ++e) low += x[e] < lo_value ? cheap(x[e]) : 0.0f;
        f_below.add(low);
      }
      if (high < lo_value) return;
      if (kWeigh == Weigh::kBelow || hi_value == kInf) {         // the list goes up to the largest
        note<kLen>(i0);
        return;
      }
    }
    uint32_t in = 0;
    float top = -kInf;
    ClosePart all = {0.0f, 0.0f}, part = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      const bool under = x[e] < lo_value, over = x[e] > hi_value;      // (a NaN is neither)
      if (kWeigh == Weigh::kClose) {
        const CloseWeight c = close(x[e]);
        all.add(c);
        if (over) part.add(c);
      }
      if (kWeigh == Weigh::kExact) {
        const uint64_t w = exact(x[e]);
        if (under) below += w;
        if (over) m_above += w;
      }
      if (over) {
        top = fmaxf(top, x[e]);
        ++n_above;
      }
      if (!under && !over) in |= 1u << e;
    }
    if (in) note<kLen>(i0);
    if (kWeigh == Weigh::kClose) {
      c_all.add(all, unit);
      c_above.add(part, unit);
    }
    if (top > -kInf) best = max(best, order_key(top));
  }
};

template <Weigh kWeigh, typename T>
__device__ __noinline__ Bracket pass(const Row<T>& row, uint64_t lo, uint64_t hi, const WeightScale& scale, FiltSmem& s) {
  uint64_t* own = row.csize > 1 ? s.list + kListCap : s.list;
  const int cap = row.csize > 1 ? kLocalCap : kListCap;
  __syncwarp();
  row_barrier(row.csize);                  // the lists and sums of the pass before are read
  if (threadIdx.x == 0) s.n_list = s.n_hits = 0;
  __syncthreads();
  // a weight is at most 2: sums stay below 2^31, in steps of 2^-F below 2^63
  const float unit = exp2f(static_cast<float>(row.bits));
  PassBody<kWeigh, T> body = {s, row, own, cap, lo, hi, place_value(lo), hi == kHighest ? kInf : place_value(hi),
                              row.inv_t * kLog2e, -static_cast<float>(scale.k), unit, scale,
                              0u, 0, 0, 0, 0, {}, {}, {}};
  for_slice<kWeigh == Weigh::kNone || kWeigh == Weigh::kBelow ? 3 : 0>(row, body);
  __syncthreads();
  body.take_hits();
  Bracket out;
  out.lo = lo;
  out.hi = hi;
  uint64_t v[5] = {static_cast<uint64_t>(body.n_above), body.m_in, body.m_above, body.below, body.best};
  if (kWeigh == Weigh::kBelow) v[3] = body.f_below.steps(unit);
  if (kWeigh == Weigh::kClose) {
    v[1] = body.c_all.steps(unit);
    v[2] = body.c_above.steps(unit);
  }
  block_reduce<5, 4>(v, s);                // (its barriers close the list too)
  const int listed = s.n_list;
  if (row.csize > 1) {
    if (threadIdx.x == 0) {
      s.stat[0] = listed;
#pragma unroll
      for (int i = 0; i < 5; ++i) s.stat[i + 1] = v[i];
    }
    __syncwarp();
    cluster_sync_all();
    // one round trip for all numbers (lane by lane: number i of CTA r), one for the lists
    const int lane = threadIdx.x & 31, shift = __ffs(row.csize) - 1;
    uint64_t got[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int q = lane + 32 * j;
      got[j] = q < 6 * row.csize ? ld_cluster_u64(&s.stat[q >> shift], q & (row.csize - 1)) : 0ull;
    }
    int end[kFiltMaxCluster], longest = 0;
    out.n_in = 0;
#pragma unroll
    for (int r = 0; r < kFiltMaxCluster; ++r) {
      const int n = __shfl_sync(0xffffffffu, static_cast<int>(got[0]), r);
      if (r < row.csize) {
        out.n_in += n;
        longest = max(longest, n);
      }
      end[r] = out.n_in;
    }
    for (int o = row.csize >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, got[j], o);
        got[j] = (lane + 32 * j) >> shift == 5 ? (w > got[j] ? w : got[j]) : got[j] + w;
      }
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int q = (i + 1) << shift;
      v[i] = __shfl_sync(0xffffffffu, q < 32 ? got[0] : got[1], q & 31);
    }
    out.whole = out.n_in <= kListCap && longest <= kLocalCap;
    if (out.whole) {
#pragma unroll 4
      for (int i = threadIdx.x; i < out.n_in; i += kFiltThreads) {
        int r = 0, from = 0;
#pragma unroll
        for (int u = 0; u < kFiltMaxCluster - 1; ++u) {
          if (u < row.csize - 1 && i >= end[u]) {
            r = u + 1;
            from = end[u];
          }
        }
        s.list[i] = ld_cluster_u64(&own[i - from], r);
      }
    }
    __syncthreads();
  } else {
    out.n_in = listed;
    out.whole = listed <= kListCap;
  }
  out.n_above = static_cast<int>(v[0]);
  out.total = kWeigh == Weigh::kExact ? v[1] + v[2] + v[3] : v[1];
  out.m_above = v[2];
  out.below = v[3];
  out.any = v[4] != 0;
  out.top = key_value(static_cast<uint32_t>(v[4]));
  return out;
}

// ------------------------------------------------------------- the selection

struct Target {
  uint64_t least, most;    // reached by the sum of amounts; the place looked for is that of `most`
  float share;             // > 0: of the sum of all, which lies within `off` of (those listed + below)
  uint64_t below, off;
};

// Among the n places of the list that lie in [a, b]: the first one, from the
// largest down, at which the sum of amounts reaches the target: amounts are
// weights, or 1 each. Returns 0 where all of them do not reach it, and leaves their
// sum in `sum`; else the sum in front of the place and its own amount are in
// s.before and s.weight.
template <bool kWeights>
__device__ __noinline__ uint64_t select(int n, uint64_t a, uint64_t b, Target& target, uint64_t& sum, float inv_t,
                                        const WeightScale& scale, FiltSmem& s) {
  auto amount = [&](uint64_t c) -> uint64_t {
    return kWeights ? weight_of(__fmul_rn(place_value(c), inv_t), scale, s.table) : 1ull;
  };
  constexpr int kAhead = 4, kEach = kBins / kFiltThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t base = 0;
  for (bool first = true;; first = false) {
    // bins of 2^sh places, counted from b down
    const int sh = b > a ? max(0, 64 - kBinBits - __clzll(b - a)) : 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < (kWeights ? 4 : 1); ++u) reinterpret_cast<uint4*>(s.bins[u])[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
      s.bin = -1;
      s.n_small = 0;
    }
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kFiltThreads) {
      uint64_t c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) c[u] = i0 + u * kFiltThreads < n ? s.list[i0 + u * kFiltThreads] : 0ull;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (c[u] < a || c[u] > b) continue;
        const int j = static_cast<int>((b - c[u]) >> sh);
        atomicAdd(&s.bins[0][j], 1u);
        if (kWeights) {                    // at most 5120 parts of 16 bits: 64-bit additions to shared memory are
          const uint64_t w = amount(c[u]); // loops (14 us for 4096 of them, three parts 1 us)
          atomicAdd(&s.bins[1][j], static_cast<uint32_t>(w) & 0xffffu);
          atomicAdd(&s.bins[2][j], static_cast<uint32_t>(w >> 16) & 0xffffu);
          atomicAdd(&s.bins[3][j], static_cast<uint32_t>(w >> 32));
        }
      }
    }
    __syncthreads();
    uint32_t count[kEach];
    uint64_t mine[kEach], own = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int j = threadIdx.x * kEach + u;
      count[u] = s.bins[0][j];
      mine[u] = kWeights ? (static_cast<uint64_t>(s.bins[3][j]) << 32) + (static_cast<uint64_t>(s.bins[2][j]) << 16) + s.bins[1][j] : count[u];
      own += mine[u];
    }
    uint64_t up = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) s.red[0][warp] = up;
    __syncthreads();
    uint64_t at = base + up - own, all = base;
#pragma unroll
    for (int w = 0; w < kFiltWarps; ++w) {
      const uint64_t v = s.red[0][w];
      if (w < warp) at += v;
      all += v;
    }
    if (first) {
      sum = all;
      if (kWeights && target.share > 0.0f) {
        const uint64_t z = all + target.below;
        target.least = share_of(target.share, z > target.off ? z - target.off : 0);
        target.most = target.off ? share_of(target.share, z + target.off) : target.least;
      }
      if (all < target.most) return 0;     // (the same for all threads)
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (at < target.most && target.most <= at + mine[u]) {
        s.bin = threadIdx.x * kEach + u;
        s.before = at;
        s.weight = mine[u];
        s.bin_count = static_cast<int>(count[u]);
      }
      at += mine[u];
    }
    __syncthreads();
    const int bin = s.bin;
    if (bin < 0) return 0;                 // (does not happen: the sum reaches it)
    base = s.before;
    b -= static_cast<uint64_t>(bin) << sh;
    if (sh == 0) return b;
    const uint64_t end = b - ((1ull << sh) - 1);
    a = end > a && end <= b ? end : a;
    if (s.bin_count > kSmall) continue;
    // one warp ranks what is in the bin
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kFiltThreads) {
      uint64_t c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) c[u] = i0 + u * kFiltThreads < n ? s.list[i0 + u * kFiltThreads] : 0ull;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c[u] >= a && c[u] <= b) s.small[atomicAdd(&s.n_small, 1)] = c[u];
    }
    __syncthreads();
    if (warp == 0) {
      const int held = s.n_small;
      const uint64_t c = lane < held ? s.small[lane] : 0ull;
      const uint64_t w = lane < held ? amount(c) : 0ull;
      uint64_t before = base;
      for (int o = 0; o < held; ++o) {
        const uint64_t oc = __shfl_sync(0xffffffffu, c, o), ow = __shfl_sync(0xffffffffu, w, o);
        if (oc > c) before += ow;
      }
      if (w != 0 && before < target.most && target.most <= before + w) {
        s.found = c;
        s.before = before;
        s.weight = w;
      }
    }
    __syncthreads();
    return s.found;
  }
}

template <typename T>
__device__ __forceinline__ uint64_t select_rank(const Bracket& view, uint64_t rank, const Row<T>& row, FiltSmem& s) {
  Target target = {rank, rank, 0.0f, 0, 0};
  uint64_t sum;
  const uint64_t top = static_cast<uint64_t>(order_key(view.top)) << 32 | 0xffffffffu;
  return select<false>(view.n_in, view.lo, top < view.hi ? top : view.hi, target, sum, row.inv_t, weight_scale(0.0f, row.bits), s);
}

template <typename T>
__device__ __forceinline__ uint64_t select_weight(const Bracket& view, uint64_t from, Target& target, uint64_t& sum,
                                                  const WeightScale& scale, const Row<T>& row, FiltSmem& s) {
  const uint64_t top = static_cast<uint64_t>(order_key(view.top)) << 32 | 0xffffffffu;
  return select<true>(view.n_in, from, top < view.hi ? top : view.hi, target, sum, row.inv_t, scale, s);
}

// ------------------------------------------------------------------ the place

// Bounds of the place that is looked for: it lies in [lo, hi], n places with weight
// m (about) lie above hi, and w (about, 0: not known) is the weight within.
struct Bounds {
  uint64_t lo, hi;
  int n;
  uint64_t m, w;
};

// The part of the bounds that a sample of the row says to look at. `pieces` times
// 2048 tokens, 128 bytes at a time evenly over the row (`turn` moves them), are
// sorted into bins of equal width below the largest one. In them the rank is found
// at which `missing` tokens are counted or, with kWeights, at which the weights from
// the lowest bin up reach `beneath` (-p: all but a share p of them; the light tokens below a place are many and
// tell its rank far better than the few heavy ones above it). Bins a margin of ranks
// above and below it are the bracket's ends. They go down to 32 below the largest
// scaled logit; what lies further below shares the last one.
template <bool kWeights, typename T>
__device__ __noinline__ void sample_bracket(const Row<T>& row, const Bounds& in, float missing, float beneath, int turn,
                                            int pieces, float sigmas, float most, const WeightScale& scale, FiltSmem& s,
                                            uint64_t& lo, uint64_t& hi) {
  constexpr int kLen = Vec<T>::kLen, kVecs = kSampleEach / kLen, kLines = kSampleSize / kLen / 8;
  constexpr int kSorts = kWeights ? 2 * kBins : kBins, kEach = kSorts / kFiltThreads;
  uint32_t* counts = s.bins[0];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lo = in.lo;
  hi = in.hi;
  const int lines = row.vocab / (8 * kLen);        // >= kLines: the row does not fit the list
  if (row.vocab < pieces * kSampleSize) pieces = 1;
  const float lo_value = place_value(in.lo), hi_value = place_value(in.hi);
  // a piece's vectors; bit e of the answer: x[e] lies within the bounds
  auto fetch = [&](int piece, float* x) -> uint32_t {
    uint4 v[kVecs];
    int first[kVecs];
    const uint32_t shift = static_cast<uint32_t>(piece) * (lines / 4) + static_cast<uint32_t>(turn) * (lines / 29);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t at = u * kFiltThreads + threadIdx.x;
      const uint32_t line = static_cast<uint32_t>((static_cast<uint64_t>(at / 8) * lines + shift) / kLines);   // shift < lines
      first[u] = (line * 8 + at % 8) * kLen;
      v[u] = *reinterpret_cast<const uint4*>(row.x + first[u]);
    }
    uint32_t on = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      Vec<T>::unpack(v[u], x + u * kLen);
#pragma unroll
      for (int e = 0; e < kLen; ++e) {
        const float y = x[u * kLen + e];
        bool mine = !(y < lo_value) && !(y > hi_value);
        if (mine && (y == lo_value || y == hi_value || y != y)) {
          const uint64_t c = pack_best(order_key(y), first[u] + e);
          mine = c >= in.lo && c <= in.hi;
        }
        if (mine) on |= 1u << (u * kLen + e);
      }
    }
    return on;
  };
  float x[kSampleEach];
  uint32_t on = fetch(0, x);
  float high = -kInf, low = kInf;
#pragma unroll
  for (int e = 0; e < kSampleEach; ++e) {
    if ((on >> e & 1) && fabsf(x[e]) < kInf) {
      high = fmaxf(high, x[e]);
      low = fminf(low, x[e]);
    }
  }
  // (of the first piece: how many, and the ends of the finite ones, the lower one inverted)
  const uint32_t up_key = __reduce_max_sync(0xffffffffu, order_key(high)), low_key = __reduce_max_sync(0xffffffffu, order_key(-low));
  const uint32_t here = __reduce_add_sync(0xffffffffu, __popc(on));
  __syncthreads();                         // what was there is read
  if (lane == 0) {
    s.red[0][warp] = static_cast<uint64_t>(up_key) << 32 | low_key;
    s.red[1][warp] = here;
  }
#pragma unroll
  for (int u = 0; u < kSorts / 4 / kFiltThreads; ++u) reinterpret_cast<uint4*>(counts)[threadIdx.x + u * kFiltThreads] = make_uint4(0u, 0u, 0u, 0u);
  if (threadIdx.x == 0) {
    s.lo_bin = kSorts;
    s.hi_bin = -1;
    s.rank = -1;
  }
  __syncthreads();
  uint32_t all_up = 0, all_low = 0;
  int m = 0;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) {
    const uint64_t v = s.red[0][w];
    all_up = max(all_up, static_cast<uint32_t>(v >> 32));
    all_low = max(all_low, static_cast<uint32_t>(v));
    m += static_cast<int>(s.red[1][w]);
  }
  high = key_value(all_up);
  low = -key_value(all_low);
  if (m == 0 || !(high >= low)) return;
  // one of the sample stands for `each` of the row
  const float each = static_cast<float>(row.vocab) / (kSampleSize * pieces);
  const float width = fminf(high - low, 32.0f / row.inv_t);
  // the weight of the largest sampled token
  const float unit = kWeights ? fast_exp2(fmaxf(fminf((__fmul_rn(high, row.inv_t) - scale.ref) * kLog2e - static_cast<float>(scale.k), 2.0f), -100.0f)) : 1.0f;
  if (!(width > 0.0f)) {                   // equal logits: their indices lie evenly, for all that is known
    const uint32_t key = order_key(high);
    const float i0 = in.hi >> 32 == key ? static_cast<float>(min(~static_cast<uint32_t>(in.hi), static_cast<uint32_t>(row.vocab))) : 0.0f;
    const float i1 = in.lo >> 32 == key ? static_cast<float>(min(~static_cast<uint32_t>(in.lo), static_cast<uint32_t>(row.vocab))) : static_cast<float>(row.vocab);
    const float ties = static_cast<float>(m) * row.vocab / kSampleSize;
    const float part = missing / unit / ties, span = most / ties;
    const float end = part + span, start = part - span;
    const uint64_t base = static_cast<uint64_t>(key) << 32;
    if (end < 1.0f) lo = max(lo, base | ~static_cast<uint32_t>(i0 + end * (i1 - i0)));
    if (start > 0.0f) hi = min(hi, base | ~static_cast<uint32_t>(i0 + start * (i1 - i0)));
    if (lo > hi) {
      lo = in.lo;
      hi = in.hi;
    }
    return;
  }
  const float per = kSorts / width;
  for (int piece = 0; piece < pieces; ++piece) {
    if (piece > 0) on = fetch(piece, x);
#pragma unroll
    for (int e = 0; e < kSampleEach; ++e) {
      if (!(on >> e & 1)) continue;
      const int j = fabsf(x[e]) < kInf ? max(0, min(static_cast<int>((high - x[e]) * per), kSorts - 1)) : 0;
      atomicAdd(&counts[j], 1u);
    }
  }
  __syncthreads();
  uint32_t n[kEach], up_n = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u) up_n += n[u] = counts[threadIdx.x * kEach + u];
  const uint32_t own_n = up_n;
  // weights in the middle of their bins, relative to the largest sampled one; sums from
  // the lowest bin up, added in an order of their own
  const float step = row.inv_t * kLog2e / per;
  float own_w = 0.0f, up_w;
  if (kWeights) {
#pragma unroll
    for (int u = kEach - 1; u >= 0; --u)
      own_w += n[u] * fast_exp2(-step * (static_cast<float>(threadIdx.x * kEach + u) + 0.5f));
  }
  up_w = own_w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, up_n, o);
    const float b = kWeights ? __shfl_down_sync(0xffffffffu, up_w, o) : 0.0f;
    if (lane >= o) up_n += a;
    if (lane < 32 - o) up_w += b;
  }
  if (lane == 31) s.red[0][warp] = up_n;
  if (lane == 0) s.red[1][warp] = __float_as_uint(up_w);
  __syncthreads();
  uint32_t at_n = up_n - own_n, all_n = 0;
  float after_w = 0.0f;                    // of the warps behind
#pragma unroll
  for (int q = 0; q < kFiltWarps; ++q) {
    if (q < warp) at_n += static_cast<uint32_t>(s.red[0][q]);
    all_n += static_cast<uint32_t>(s.red[0][q]);
  }
  float rank, margin;
  if (kWeights) {
#pragma unroll
    for (int q = kFiltWarps - 1; q >= 0; --q)
      if (q > warp) after_w += __uint_as_float(static_cast<uint32_t>(s.red[1][q]));
    float all_w = 0.0f;
#pragma unroll
    for (int q = 0; q < kFiltWarps; ++q) all_w += __uint_as_float(static_cast<uint32_t>(s.red[1][q]));
    const float want = beneath < 0.0f ? (1.0f + beneath) * all_w : beneath / (each * unit);
    float a_w = after_w + (up_w - own_w);
    uint32_t a_n = at_n + own_n;
#pragma unroll
    for (int u = kEach - 1; u >= 0; --u) {
      const int j = threadIdx.x * kEach + u;
      const float next = a_w + n[u] * fast_exp2(-step * (static_cast<float>(j) + 0.5f));
      a_n -= n[u];
      // (roundings may let two threads say so)
      if (a_w <= want && want < next) atomicMax(&s.rank, j << 16 | static_cast<int>(a_n + n[u] / 2));
      a_w = next;
    }
    __syncthreads();
    const int found = max(s.rank, 0);      // nothing: all lies beneath
    rank = static_cast<float>(found & 0xffff);
    // the deviation of the weight beneath, in tokens of the place's own weight: none beneath is heavier
    margin = sigmas * sqrtf(want / fast_exp2(fmaxf(-step * (static_cast<float>(found >> 16) + 0.5f), -100.0f))) + 6.0f;
  } else {
    rank = missing / each;
    margin = sigmas * sqrtf(rank) + 3.0f;
  }
  margin = fminf(margin, most / each);
  const int down = static_cast<int>(fminf(rank + margin, 1e9f)) + 1, up = static_cast<int>(rank - margin);
  uint32_t a_n = at_n;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int next = static_cast<int>(a_n + n[u]), before = static_cast<int>(a_n);
    if (before < down && down <= next) s.lo_bin = threadIdx.x * kEach + u;
    if (before < up && up <= next) s.hi_bin = threadIdx.x * kEach + u;
    a_n += n[u];
  }
  __syncthreads();
  const int lo_bin = s.lo_bin, hi_bin = s.hi_bin;
  if (lo_bin < kSorts - 1) lo = max(lo, static_cast<uint64_t>(order_key(high - static_cast<float>(lo_bin + 1) / per)) << 32);
  if (hi_bin > 0) hi = min(hi, static_cast<uint64_t>(order_key(high - static_cast<float>(hi_bin) / per)) << 32 | 0xffffffffu);
  if (lo < kLowest) lo = kLowest;
  if (lo > hi) {                           // (roundings of a narrow range)
    lo = in.lo;
    hi = in.hi;
  }
}

// The next bracket within the bounds: four times around what a sample says, then
// half of the bounds.
template <bool kWeights, typename T>
__device__ __forceinline__ void next_bracket(const Row<T>& row, const Bounds& in, float missing, float beneath, int turn,
                                             const WeightScale& scale, FiltSmem& s, uint64_t& lo, uint64_t& hi) {
  lo = in.lo;
  hi = in.hi;
  if (row.vocab <= kListCap) return;       // (one CTA, and all of the row on the list)
  if (turn <= kSampledTurns) {
    sample_bracket<kWeights>(row, in, missing, beneath, turn, kSamplePieces, 3.0f, 0.4f * kListCap, scale, s, lo, hi);
  } else {
    lo = in.lo + (in.hi - in.lo) / 2 + 1;
    if (lo > in.hi) lo = in.hi;
  }
}

// The place of rank k within the bounds (or their lowest place, where there are
// fewer). Leaves the last bracket in `view`, its places on the list.
template <typename T>
__device__ __noinline__ uint64_t locate_rank(const Row<T>& row, Bounds in, int k, FiltSmem& s, Bracket& view) {
  const WeightScale none = weight_scale(0.0f, row.bits);
  for (int turn = 1; turn <= kTurns; ++turn) {
    uint64_t lo, hi;
    next_bracket<false>(row, in, static_cast<float>(k - in.n), 0.0f, turn, none, s, lo, hi);
    view = pass<Weigh::kNone>(row, lo, hi, none, s);
    const int with = view.n_above + view.n_in;
    if (view.n_above >= k) {
      in.lo = hi + 1;                      // (hi < in.hi, above which there are fewer)
    } else if (with < k) {
      if (lo == in.lo) return in.lo;       // all that there is
      in.hi = lo - 1;
      in.n = with;
    } else if (view.whole) {
      return select_rank(view, k - view.n_above, row, s);
    } else {
      in = {lo, hi, view.n_above, 0, 0};
    }
  }
  return in.lo;                            // (not reached: 64 halvings leave one place)
}

// The place within the bounds at which the weight from the top reaches the target:
// target.share of all weights, or target.most itself where share is 0 (target.most
// is a guess otherwise). `from` > 0 is where the first bracket begins. Leaves the
// last bracket in `view`, its places on the list, and the weight from the top down
// to the place in `mass`.
template <typename T>
__device__ __noinline__ uint64_t locate_weight(const Row<T>& row, Bounds in, Target target, uint64_t from,
                                               const WeightScale& scale, FiltSmem& s, Bracket& view, uint64_t& mass) {
  bool exact = scale.tie, again = from != 0;
  uint64_t lo = from, hi = in.hi;
  for (int turn = 1; turn <= kTurns; ++turn) {
    if (!again) {
      const uint64_t missing = target.most > in.m ? target.most - in.m : 0, beneath = in.w > missing ? in.w - missing : 0;
      const float unit = exp2f(static_cast<float>(-row.bits));
      next_bracket<true>(row, in, static_cast<float>(missing) * unit, in.w ? static_cast<float>(beneath) * unit : -target.share, turn,
                         scale, s, lo, hi);
    }
    again = false;
    view = exact ? pass<Weigh::kExact>(row, lo, hi, scale, s) : pass<Weigh::kClose>(row, lo, hi, scale, s);
    uint64_t sum = 0;                      // of the bracket
    if (view.whole) {                      // listed weights are exact
      for (int i = threadIdx.x; i < view.n_in; i += kFiltThreads) sum += weight_of(__fmul_rn(place_value(s.list[i]), row.inv_t), scale, s.table);
      sum = block_sum(sum, s);
    } else {
      const uint64_t out = view.m_above + view.below;
      sum = exact && view.total > out ? view.total - out : 0;
    }
    // sums of close weights are within `off`: 2^-29.5 of a weight, 2^-28.5 of a vector's sum; exact weights are
    // rounded to a step each
    const uint64_t off = exact ? 0 : static_cast<uint64_t>(static_cast<float>(view.total) * 0x1p-27f) + row.vocab;
    uint64_t least = target.most, most = target.most;
    if (target.share > 0.0f) {
      least = share_of(target.share, view.total > off ? view.total - off : 0);
      most = off ? share_of(target.share, view.total + off) : least;
      target.most = most;
    }
    const uint64_t above_least = view.m_above > off ? view.m_above - off : 0, above_most = view.m_above + off;
    if (above_least >= most) {             // above the bracket
      in.lo = hi + 1;
      in.w = view.m_above > in.m ? view.m_above - in.m : 0;
    } else if (!view.whole && !exact) {
      // the bracket's own weight is not known: another one, and the second time exact weights, which tell
      if (above_most < least) {
        in.hi = hi;
        in.n = view.n_above;
        in.m = view.m_above;
        in.w = view.total > view.m_above ? view.total - view.m_above : 0;
      }
      exact = turn >= 2;
    } else if (above_most + sum < least) { // below it
      if (lo == in.lo) return in.lo;       // all that there is
      in.hi = lo - 1;
      in.n = view.n_above + view.n_in;
      in.m = view.m_above + sum;
      in.w = view.total > in.m ? view.total - in.m : 0;
    } else if (!view.whole) {              // in it, and more than the list holds
      in = {lo, hi, view.n_above, view.m_above, sum};
    } else {
      Target inner = {least > above_most ? least - above_most : 0, most - above_least, 0.0f, 0, 0};
      const uint64_t at = inner.least > 0 && inner.most <= sum ? select_weight(view, lo, inner, sum, scale, row, s) : 0;
      if (at != 0 && s.before < inner.least) {
        mass = view.m_above + s.before + s.weight;
        return at;
      }
      if (exact) return in.lo;             // (does not happen)
      exact = again = true;                // the border is within the bound: the same bracket, exactly
    }
  }
  return in.lo;                            // (not reached: 64 halvings leave one place)
}

// The order key of the smallest logit x with fl(x * inv_t) >= least (which +inf
// fulfils): a quotient's key is within a few of it, but where products
// underflow or overflow many logits share one.
__device__ __forceinline__ uint32_t smallest_key(float least, float inv_t) {
  constexpr uint32_t kFirst = 0x00800000u, kLast = 0xff800000u;      // -FLT_MAX, +inf
  auto enough = [&](uint32_t key) { return __fmul_rn(key_value(key), inv_t) >= least; };
  const uint32_t near = min(max(order_key(__fdiv_rn(least, inv_t)), kFirst + 4), kLast - 4);
  uint32_t no = near - 4, yes = near + 4;  // the border lies between
  if (!enough(yes)) { no = yes; yes = kLast; }
  else if (enough(no)) { yes = no; no = kFirst - 1; }
  while (yes - no > 1) {
    const uint32_t mid = no + (yes - no) / 2;
    if (enough(mid)) yes = mid; else no = mid;
  }
  return yes;
}

struct RowResult {
  uint64_t cut;            // the last place that is kept
  uint64_t mass;           // the weight of all that is kept, 0: not known
  bool empty;              // nothing above -inf
  bool listed;             // all that is kept is on the list
  int n_list, n_above;     // on the list, and above it
  WeightScale scale;
};

template <typename T>
__device__ __forceinline__ RowResult find_cut(const Row<T>& row, int k, float p, float min_p, FiltSmem& s) {
  const bool by_k = k > 0 && k < row.vocab, by_p = p < 1.0f, by_m = min_p > 0.0f;
  const int vocab = row.vocab;
  uint64_t lo = kLowest, hi = kHighest;
  const WeightScale none = weight_scale(0.0f, row.bits);
  // 1. where the list begins (and ends, for a top-k set that no list holds)
  if (vocab > kListCap) {
    const float wanted = static_cast<float>(by_k ? k : kFirstList);
    const bool large = wanted >= 0.5f * kListCap;
    sample_bracket<false>(row, Bounds{kLowest, kHighest, 0, 0, 0}, wanted, 0.0f, 0, large ? kSamplePieces : 1, 3.0f,
                          0.4f * kListCap, none, s, lo, hi);
    if (!large) hi = kHighest;
  }
  // 2. the list; weights below it relative to its first place, a power of two
  // from the row's (not where the reduction differs, nor where 1 / T times log2 e
  // would be infinite, from 2.36e38 on)
  const bool total = by_p && !by_k;
  const float s_lo = __fmul_rn(place_value(lo), row.inv_t);
  const WeightScale low_scale = weight_scale(s_lo, row.bits);
  const bool low_fits = fabsf(s_lo) < (row.inv_t < 2.3e38f ? kWeightSpan : 0.0f);
  Bracket view = total && low_fits ? pass<Weigh::kBelow>(row, lo, hi, low_scale, s)
                                   : pass<Weigh::kNone>(row, lo, hi, none, s);
  if (!view.any && lo > kLowest)           // (a bracket's end need not be a token's place)
    view = pass<Weigh::kNone>(row, kLowest, kHighest, none, s);
  if (!view.any) return RowResult{kHighest, 0, true, true, 0, 0, none};
  const WeightScale scale = weight_scale(__fmul_rn(view.top, row.inv_t), row.bits);
  uint64_t cut = kLowest, mass = 0;
  // 3. top-k
  if (by_k) {
    const int with = view.n_above + view.n_in;
    if (view.n_above >= k) {
      cut = locate_rank(row, Bounds{view.hi + 1, kHighest, 0, 0, 0}, k, s, view);
    } else if (with < k) {                 // (from the lowest place on fewer than k: all stay)
      if (view.lo > kLowest) cut = locate_rank(row, Bounds{kLowest, view.lo - 1, with, 0, 0}, k, s, view);
    } else if (view.whole) {
      cut = select_rank(view, k - view.n_above, row, s);
    } else {
      cut = locate_rank(row, Bounds{view.lo, view.hi, view.n_above, 0, 0}, k, s, view);
    }
  }
  // 4. top-p of what top-k leaves
  if (by_p) {
    const bool listed = view.hi == kHighest && view.whole;      // the list holds all from view.lo on
    uint64_t at = 0, sum = 0;
    Target target = {1, 1, p, 0, 0};
    if (by_k) {
      if (listed && cut >= view.lo) {
        at = select_weight(view, cut, target, sum, scale, row, s);
        mass = s.before + s.weight;
      } else {
        view = pass<Weigh::kExact>(row, cut, kHighest, scale, s);
        target = {0, share_of(p, view.total - view.below), 0.0f, 0, 0};
        target.least = target.most;
        if (view.whole) {
          at = select_weight(view, cut, target, sum, scale, row, s);
          mass = s.before + s.weight;
        } else {
          at = locate_weight(row, Bounds{cut, kHighest, 0, 0, view.total - view.below}, target, 0, scale, s, view, mass);
        }
      }
    } else {
      Bounds in = {kLowest, kHighest, 0, 0, 0};
      uint64_t from = 0;
      if (listed && low_fits && scale.ref == 0.0f && !scale.tie) {
        // The total lies within target.off. A weight's exponent y is off by less than |y| 2^-22.8 (the rounded
        // product, its factor, log2 e) and |y - k| 2^-24, exp2 by 2^-22, a vector's sum by 2^-21; tokens with
        // y - k below -20 are covered by the second term.
        const int down = scale.k - low_scale.k;
        const float rel = (fabsf(static_cast<float>(low_scale.k)) + 24.0f) * 0x1p-22f;
        const uint64_t few = static_cast<uint64_t>(vocab) << max(row.bits - 42, 0);
        target.below = down < 64 ? view.below >> down : 0ull;
        target.off = static_cast<uint64_t>(static_cast<float>(target.below) * rel) + (down < 64 ? few >> down : 0ull) + 2;
        at = select_weight(view, view.lo, target, sum, scale, row, s);
        if (at != 0 && s.before < target.least) mass = s.before + s.weight;      // all targets fall on one token
        else if (sum >= target.least) { at = 0; from = view.lo; }                 // on the list, or close to its end
        else if (view.lo > kLowest) { at = 0; in = {kLowest, view.lo - 1, view.n_in, sum, target.below}; }
        else at = 0;
        target.below = target.off = 0;
      }
      if (at == 0) at = locate_weight(row, in, target, from, scale, s, view, mass);
    }
    if (at > cut) cut = at;
  }
  // 5. min-p
  if (by_m) {
    float least = scale.s_max;
    if (!scale.tie) least = __double2float_ru(static_cast<double>(scale.s_max) + log(static_cast<double>(min_p)));
    const uint32_t key = scale.s_max != scale.s_max ? 0xffffffffu : smallest_key(least, row.inv_t);
    const uint64_t at = static_cast<uint64_t>(key) << 32;
    if (at > cut) {
      cut = at;
      mass = 0;
    }
  }
  return RowResult{cut, mass, false, view.hi == kHighest && view.whole && cut >= view.lo, view.n_in, view.n_above, scale};
}

// ------------------------------------------------------------------- endings

// ln of the kept share of a token: its weight over the sum of all kept ones.
__device__ __forceinline__ float log_share(float s_tok, uint64_t sum, const WeightScale& w, const WeightTable& table) {
  const uint64_t mine = weight_of(s_tok, w, table);
  if (mine >= sum && mine > 0) return 0.0f;              // (a close sum may lie below its one term)
  if (mine > sum / 2) return log1pf(-(static_cast<float>(sum - mine) / static_cast<float>(sum)));
  const float total = static_cast<float>(sum) * exp2f(static_cast<float>(-w.bits));
  if (w.tie) return mine ? -logf(total) : -kInf;
  const float s = s_tok - w.ref;
  const float yh = __fmul_rn(s, kLog2e);
  const float yl = __fmaf_rn(s, kLog2eLow, __fmaf_rn(s, kLog2e, -yh));
  return kLn2 * ((yh - static_cast<float>(w.k)) + yl) - logf(total);
}

// f.many<n>(x, noise, first index) for all entries of the slice, the noise fetched
// beside the logits.
template <typename T, typename F>
__device__ __forceinline__ void for_slice_noise(const Row<T>& row, const float* noise, F& f) {
  constexpr int kLen = Vec<T>::kLen, kUnroll = 2;
  const uint4* vecs = reinterpret_cast<const uint4*>(row.x + row.v0);
  const float4* more = reinterpret_cast<const float4*>(noise + row.v0);
  const int n = (row.v1 - row.v0) / kLen;
  for (int j0 = threadIdx.x; j0 < n; j0 += kUnroll * kFiltThreads) {
    uint4 v[kUnroll];
    float4 w[kUnroll][kLen / 4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * kFiltThreads;
      if (j >= n) continue;
      v[u] = vecs[j];
#pragma unroll
      for (int q = 0; q < kLen / 4; ++q) w[u][q] = __ldcs(more + j * (kLen / 4) + q);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * kFiltThreads;
      if (j >= n) break;
      float x[kLen], g[kLen];
      Vec<T>::unpack(v[u], x);
#pragma unroll
      for (int q = 0; q < kLen / 4; ++q) {
        g[4 * q] = w[u][q].x; g[4 * q + 1] = w[u][q].y; g[4 * q + 2] = w[u][q].z; g[4 * q + 3] = w[u][q].w;
      }
      f.template many<kLen>(x, g, row.v0 + j * kLen);
    }
  }
  const int i = row.v0 + n * kLen + threadIdx.x;
  if (i < row.v1) {
    float x[1] = {load_one(row.x + i)}, g[1] = {noise[i]};
    f.template many<1>(x, g, i);
  }
}

// The largest of fl(s + noise), the first one of equal ones: a thread meets
// indices in increasing order, and few values pass the ones before them.
struct Draw {
  float value;             // of `best`, for a first look (a NaN at first, which all pass)
  uint64_t best;
  __device__ __forceinline__ bool passes(float v) const { return !(v <= value); }       // (a NaN does)
  __device__ __forceinline__ void offer(float v, int i) {
    const uint64_t c = pack_best(order_key(v), i);
    if (c > best) {
      best = c;
      value = v;
    }
  }
};

__device__ __forceinline__ Draw no_draw() { return {__int_as_float(0x7fffffff), 0}; }

template <typename T>
struct DrawBody {
  const Row<T>& row;
  const float* noise;
  uint64_t cut;
  float cut_value;
  bool weigh;
  WeightScale scale;
  const WeightTable& table;
  Draw draw;
  uint64_t sum;            // of weights: exact for few tokens,
  CloseSum close;          // within 2^-27 for many (no decision hangs on it)
  float unit;

  __device__ __forceinline__ bool keeps(float x, int i) const {
    return !(x < cut_value) && (x > cut_value || pack_best(order_key(x), i) >= cut);
  }
  __device__ __forceinline__ void take(float x, float g, int i) {
    const float sx = __fmul_rn(x, row.inv_t);
    draw.offer(__fadd_rn(sx, g), i);
    if (weigh) sum += weight_of(sx, scale, table);
  }
  // few are kept: their noise alone is read
  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
#pragma unroll
    for (int e = 0; e < kLen; ++e)
      if (keeps(x[e], i0 + e)) take(x[e], noise[i0 + e], i0 + e);
  }
  template <int kLen>
  __device__ __forceinline__ void many(const float* x, const float* g, int i0) {
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      const float v = __fadd_rn(__fmul_rn(x[e], row.inv_t), g[e]);
      if (draw.passes(v) && keeps(x[e], i0 + e)) draw.offer(v, i0 + e);
    }
    if (weigh) {
      ClosePart part = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < kLen; ++e)
        if (keeps(x[e], i0 + e)) part.add(close_weight(__fmul_rn(x[e], row.inv_t), scale, table));
      close.add(part, unit);
    }
  }
};

// No filter: all of the noise is read beside the logits, the sum of weights is
// float32 relative to a running maximum (nothing is decided by it). The reference
// moves where a value lies more than 1 above it: a row in ascending order would
// move it at every vector otherwise, and the factors' errors would add up (3.7e-5 of the
// sum in 2^20 entries that rise by 0.012). Sums fall by e at least with every move, so those
// of n entries of a thread count ln n + 2 moves at most before they are a small part
// of what comes; each is off by 2^-22.4 (expf, the difference).
struct FreeBody {
  float inv_t;
  Draw draw;
  float top, nans;
  FloatSum sum;            // (beside one heavy token hundreds of light ones would each lose up to 2^-25 of it)

  template <int kLen>
  __device__ __forceinline__ void many(const float* x, const float* g, int i0) {
    float s[kLen], high = top, part = 0.0f;
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      s[e] = __fmul_rn(x[e], inv_t);
      high = fmaxf(high, s[e]);
      const float v = __fadd_rn(s[e], g[e]);
      if (draw.passes(v) && x[e] != -kInf) draw.offer(v, i0 + e);
    }
    if (high > top + 1.0f) {
      sum.scale(expf(top - high));
      top = high;
    }
#pragma unroll
    for (int e = 0; e < kLen; ++e) {       // equal infinities weigh 1
      if (s[e] != s[e]) nans += 1.0f;
      else part += s[e] == top ? 1.0f : fast_exp2((s[e] - top) * kLog2e);
    }
    sum.add(part);
  }
};

struct TopBody {
  Draw draw;
  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
#pragma unroll
    for (int e = 0; e < kLen; ++e)
      if (draw.passes(x[e])) draw.offer(x[e], i0 + e);
  }
};

template <typename T>
struct MaskBody {
  T* out;
  uint64_t cut;
  float cut_value;
  uint64_t kept;

  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
    float y[kLen];
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      bool keep = !(x[e] < cut_value);
      if (keep && !(x[e] > cut_value)) keep = pack_best(order_key(x[e]), i0 + e) >= cut;
      y[e] = keep ? x[e] : -kInf;
      kept += keep;
    }
    if constexpr (kLen == 1) store_one(out + i0, y[0]);
    else __stcs(reinterpret_cast<uint4*>(out + i0), Vec<T>::pack(y));      // (the logits stay in L2 for other rows)
  }
};

// Each look at a row is a function of its own, with registers of its own.
template <typename T>
__device__ __noinline__ uint64_t top_row(const Row<T>& row, FiltSmem& s) {
  TopBody body = {no_draw()};
  for_slice<3>(row, body);
  return block_max(body.draw.best, s);
}

template <typename T>
__device__ __noinline__ uint64_t mask_row(const Row<T>& row, T* out, uint64_t cut, FiltSmem& s) {
  MaskBody<T> body = {out, cut, place_value(cut), 0};
  for_slice<0>(row, body);
  return block_sum(body.kept, s);
}

struct FreeResult {
  uint64_t best;
  float top, sum, nans;
};
template <typename T>
__device__ __noinline__ FreeResult free_row(const Row<T>& row, const float* noise, FiltSmem& s) {
  FreeBody body = {row.inv_t, no_draw(), -FLT_MAX, 0.0f, {0.0f, 0.0f}};
  for_slice_noise(row, noise, body);
  FreeResult out;
  const float sum = body.sum.sum + body.sum.low;
  out.best = block_max(body.draw.best, s);
  out.top = key_value(static_cast<uint32_t>(block_max(order_key(body.top), s)));
  out.sum = block_sum(body.top == out.top ? sum : sum * fast_exp2((body.top - out.top) * kLog2e), s);
  out.nans = block_sum(body.nans, s);
  if (out.sum == 0.0f && out.nans == 0.0f) {             // all are scaled to -inf: those that are not -inf weigh 1
    float n = 0.0f;
    for (int i = row.v0 + threadIdx.x; i < row.v1; i += kFiltThreads) n += load_one(row.x + i) == -kInf ? 0.0f : 1.0f;
    out.top = -kInf;
    out.sum = block_sum(n, s);
  }
  return out;
}

struct DrawResult {
  uint64_t best, sum;
};
// `dense`: so many are kept that all of the noise is read.
template <typename T>
__device__ __noinline__ DrawResult draw_row(const Row<T>& row, const float* noise, const RowResult& res, bool weigh, bool dense, FiltSmem& s) {
  DrawBody<T> body = {row, noise, res.cut, place_value(res.cut), weigh, res.scale, s.table,
                      no_draw(), 0, {}, exp2f(static_cast<float>(row.bits))};
  if (res.listed) {
    for (int i = row.rank * kFiltThreads + threadIdx.x; i < res.n_list; i += row.csize * kFiltThreads) {
      const uint64_t c = s.list[i];
      if (c >= res.cut) body.take(place_value(c), noise[best_index(c)], best_index(c));
    }
  } else if (dense) {
    for_slice_noise(row, noise, body);
    body.sum = body.close.steps(body.unit);
  } else {
    for_slice<0>(row, body);
  }
  DrawResult out;
  out.best = block_max(body.draw.best, s);
  out.sum = weigh ? block_sum(body.sum, s) : 0;
  return out;
}

// A row of the call, as a CTA meets it.
struct Job {
  bool on;                 // there is something to do
  int b;
  size_t t;
  float temp, inv_t, top_p, min_p;
  int k;
};

template <bool kSampling>
__device__ __forceinline__ Job job_of(const FiltParams& p, int id) {
  Job job;
  job.on = false;
  if (id >= p.rows) return job;
  job.b = id / p.max_nodes;
  const int node = id - job.b * p.max_nodes;
  const int st = p.status[job.b];
  const int t0 = p.cu_nodes[job.b], n = p.cu_nodes[job.b + 1] - t0;
  job.temp = p.temperature[job.b];
  job.k = p.top_k ? p.top_k[job.b] : 0;
  job.top_p = p.top_p ? p.top_p[job.b] : 1.0f;
  job.min_p = p.min_p ? p.min_p[job.b] : 0.0f;
  if (st != 0 || (node >= n && n >= 0)) return job;
  job.inv_t = job.temp > 0.0f ? __frcp_rn(job.temp) : 1.0f;
  int flag = 0;
  if (n > p.max_nodes || n < 0 || t0 < 0) flag |= TV_ST_BAD_SIZE;
  if (!(job.temp >= 0.0f) || job.temp == kInf || job.inv_t == kInf || (kSampling && job.temp > 0.0f && !p.gumbel))
    flag |= TV_ST_BAD_TEMPERATURE;
  if (job.k < 0 || !(job.top_p >= 0.0f && job.top_p <= 1.0f) || !(job.min_p >= 0.0f && job.min_p <= 1.0f)) flag |= TV_ST_BAD_FILTER;
  if (flag) {
    if (node == 0 && threadIdx.x == 0) atomicOr(&p.status[job.b], flag);       // (all CTAs that meet the row say the same)
    return job;
  }
  job.t = static_cast<size_t>(t0) + node;
  job.on = true;
  return job;
}

// One row, by the csize CTAs of a cluster together.
template <typename T, bool kSampling>
__device__ __forceinline__ void do_row(const FiltParams& p, const Job& job, int csize, int rank, FiltSmem& s) {
  const size_t t = job.t;
  const float inv_t = job.inv_t, top_p = job.top_p, min_p = job.min_p;
  const int k = job.k;
  Row<T> row = {static_cast<const T*>(p.logits) + t * p.logits_ld, p.vocab, 0, p.vocab, rank, csize, inv_t, p.bits};
  if (csize > 1) {
    const int per = ((p.vocab + csize - 1) / csize + 7) & ~7;
    row.v0 = min(p.vocab, rank * per);
    row.v1 = min(p.vocab, row.v0 + per);
  }
  const bool greedy = job.temp == 0.0f;
  const bool filtered = !greedy && ((k > 0 && k < p.vocab) || top_p < 1.0f || min_p > 0.0f);

  // Each CTA's part of an ending goes to s.stat; the first CTA combines them.
  auto publish = [&](uint64_t a, uint64_t b2, uint64_t c) {
    __syncwarp();
    row_barrier(csize);                    // what a pass left there is read
    if (threadIdx.x == 0) {
      s.stat[0] = a;
      s.stat[1] = b2;
      s.stat[2] = c;
    }
    __syncwarp();
    row_barrier(csize);
  };
  RowResult res = {kLowest, 0, false, false, 0, 0, weight_scale(0.0f, p.bits)};
  if (greedy) {
    publish(top_row(row, s), 0, 0);
    const uint64_t best = cluster_stat<true>(s, 0, csize);
    res.empty = best < kLowest;
    res.cut = res.empty ? kHighest : best;
    if (kSampling) {
      if (threadIdx.x == 0 && rank == 0) {
        p.tokens[t] = res.empty ? 0 : best_index(best);
        if (p.logp) p.logp[t] = res.empty ? -kInf : 0.0f;
      }
      return;
    }
  } else if (filtered) {
    res = find_cut(row, k, top_p, min_p, s);
  }

  if constexpr (kSampling) {
    const float* noise = p.gumbel + t * p.gumbel_ld;
    if (!filtered) {
      const FreeResult own = free_row(row, noise, s);
      publish(own.best, static_cast<uint64_t>(__float_as_uint(own.sum)) << 32 | order_key(own.top), __float_as_uint(own.nans));
      const uint64_t best = cluster_stat<true>(s, 0, csize);
      if (threadIdx.x == 0 && rank == 0) {
        const int token = best ? best_index(best) : 0;
        p.tokens[t] = token;
        if (p.logp) {
          float top = -kInf, sum = 0.0f, nans = 0.0f;
          for (int r = 0; r < csize; ++r) {
            const uint64_t v = csize > 1 ? ld_cluster_u64(&s.stat[1], r) : s.stat[1];
            top = fmaxf(top, key_value(static_cast<uint32_t>(v)));
            nans += __uint_as_float(static_cast<uint32_t>(csize > 1 ? ld_cluster_u64(&s.stat[2], r) : s.stat[2]));
          }
          for (int r = 0; r < csize; ++r) {
            const uint64_t v = csize > 1 ? ld_cluster_u64(&s.stat[1], r) : s.stat[1];
            const float its = key_value(static_cast<uint32_t>(v)), part = __uint_as_float(static_cast<uint32_t>(v >> 32));
            sum += its == top ? part : part * fast_exp2((its - top) * kLog2e);
          }
          const float mine = __fmul_rn(load_one(row.x + token), inv_t);
          float out = (mine == top ? 0.0f : mine - top) - logf(sum);
          if (nans > 0.0f) out = mine != mine ? -logf(nans) : -kInf;
          p.logp[t] = best ? out : -kInf;
        }
      }
      return;
    }
    if (res.empty) {
      if (threadIdx.x == 0 && rank == 0) {
        p.tokens[t] = 0;
        if (p.logp) p.logp[t] = -kInf;
      }
      return;
    }
    const bool weigh = p.logp != nullptr && res.mass == 0;
    const DrawResult own = draw_row(row, noise, res, weigh, res.n_list + res.n_above > p.vocab / 32 && !res.scale.tie, s);
    publish(own.best, own.sum, 0);
    const int token = best_index(cluster_stat<true>(s, 0, csize));
    const uint64_t sum = weigh ? cluster_stat<false>(s, 1, csize) : res.mass;
    if (threadIdx.x == 0 && rank == 0) {
      p.tokens[t] = token;
      if (p.logp) {
        p.logp[t] = log_share(__fmul_rn(load_one(row.x + token), inv_t), sum, res.scale, s.table);
      }
    }
  } else {
    // (in place: no CTA of the cluster writes before all have read the row)
    __syncwarp();
    row_barrier(csize);
    publish(mask_row(row, static_cast<T*>(p.out) + t * p.out_ld, res.cut, s), 0, 0);
    const int kept = static_cast<int>(cluster_stat<false>(s, 0, csize));
    if (p.kept && threadIdx.x == 0 && rank == 0) p.kept[t] = kept;
  }
}

// The row of a CTA (of a cluster). Where there are more rows than fit at once, the
// requests with top-p alone come first: their flat rows take four times as long as
// others, and one that started last would be waited for alone.
__device__ __forceinline__ int row_of(const FiltParams& p, FiltSmem& s) {
  const int id = blockIdx.x / p.csize;
  if (!p.reorder) return id;
  const int place = id / p.max_nodes, b = threadIdx.x, lane = b & 31, warp = b >> 5;
  bool slow = false;
  if (b < p.batch) {
    const int k = p.top_k ? p.top_k[b] : 0;
    slow = p.top_p && p.top_p[b] < 1.0f && (k == 0 || k >= p.vocab);
  }
  const uint32_t who = __ballot_sync(0xffffffffu, slow);
  if (lane == 0) s.red[0][warp] = who;
  __syncthreads();
  int all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) {
    const int n = __popc(static_cast<uint32_t>(s.red[0][w]));
    if (w < warp) before += n;
    all += n;
  }
  before += __popc(who & ((1u << lane) - 1));              // slow requests in front of b
  if (b < p.batch && place == (slow ? before : all + (b - before))) s.bin = b;
  __syncthreads();
  return s.bin * p.max_nodes + (id - place * p.max_nodes);
}

template <typename T, bool kSampling>
__global__ void __launch_bounds__(kFiltThreads, kFiltPerSm) filtered_kernel(const __grid_constant__ FiltParams p) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  FiltSmem& s = *reinterpret_cast<FiltSmem*>(s_raw);
  if (threadIdx.x < kWeightTable) fill_weight_table(s.table, threadIdx.x);
  grid_dependency_wait();
  grid_launch_dependents();
  const int place = p.csize > 1 ? static_cast<int>(cluster_rank()) : 0;
  const Job job = job_of<kSampling>(p, row_of(p, s));
  if (!job.on) return;                     // (the same in all CTAs of a cluster)
  __syncthreads();
  do_row<T, kSampling>(p, job, p.csize, place, s);
  __syncwarp();
  if (p.csize > 1) cluster_sync_all();     // no CTA goes while its memory may be read
}

// ------------------------------------------------------------------ host side

template <bool kSampling>
static int launch_filtered(int dtype, FiltParams& p, void* stream) {
  static SmemLimit smem_limit[2];
  const int dev = current_device();
  const int sms = dev < 0 ? -1 : device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  const bool f32 = dtype == TV_DTYPE_F32;
  auto* kernel = f32 ? filtered_kernel<float, kSampling> : filtered_kernel<__nv_bfloat16, kSampling>;
  const long long rows = static_cast<long long>(p.batch) * p.max_nodes;
  p.rows = static_cast<int>(rows);
  p.bits = weight_bits(p.vocab);
  // a cluster a row where all of them are resident at once
  p.csize = 1;
  while (p.csize < kFiltMaxCluster && rows * p.csize * 2 <= sms * kFiltPerSm && p.vocab > kListCap) p.csize *= 2;
  p.reorder = p.top_p && p.batch > 1 && p.batch <= kFiltThreads && rows * p.csize > sms * kFiltPerSm;
  const size_t smem = sizeof(FiltSmem) + (p.csize > 1 ? kLocalCap * sizeof(uint64_t) : 0);
  if (!ensure_smem(kernel, smem, smem_limit[f32], dev)) return TV_ERR_CUDA;
  const cudaError_t err = launch_cluster_smem_pdl(kernel, dim3(static_cast<unsigned>(rows * p.csize)), dim3(kFiltThreads), p.csize,
                                                  smem, as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace TV_FILT_SPACE
}  // namespace tv
