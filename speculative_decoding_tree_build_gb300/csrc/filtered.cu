// tv_sample_filtered and tv_filter_logits: temperature, top-k, top-p, min-p.
//
// A row's tokens are ordered by (logit descending, index ascending); what is
// kept is a prefix of that order, so a filter is one place in it: the last kept
// token. Places are 64-bit numbers, the logit's order key above the inverted
// index, and comparing two of them is comparing integers; ties need no care
// anywhere else.
//
// Finding the place without sorting the row:
//   1. a sample of the row in 128-byte lines gives a place below which some
//      thousand tokens of the row lie above;
//   2. one pass over the row lists those (shared memory) and sums the weights
//      of the others where top-p needs the total;
//   3. on the list, a histogram over places finds the bin in which the count
//      (top-k) or the sum of weights (top-p) is reached; its few tokens are
//      ranked by one warp.
// Where the place is not on the list (top-k larger than the list, a flat row
// whose top-p set is a tenth of the vocabulary, many equal logits), bounds on
// the place are narrowed by another sample and another pass. Every pass shrinks
// the bounds, and from the fifth on it halves them.
//
// Sums are integers (tv_weight.cuh): no result depends on the order of the
// atomics that build lists and histograms.
#include <cuda_bf16.h>

#include "tv_cluster.cuh"
#include "tv_weight.cuh"

namespace tv {

constexpr int kFiltThreads = 512;
constexpr int kFiltWarps = kFiltThreads / 32;
constexpr int kListCap = 8192;
constexpr int kSampleSize = 4096;
constexpr int kBins = 1024;
constexpr int kSmall = 32;                 // tokens that a warp ranks
constexpr int kSampledTurns = 4, kTurns = kSampledTurns + 64;
constexpr int kFiltUnroll = 4;             // 16-byte loads in flight a thread
constexpr float kInf = __builtin_huge_valf();

// Places: (order key, ~index). -inf has no place: it is never kept.
constexpr uint64_t kLowest = static_cast<uint64_t>(0x00800000u) << 32;   // just above -inf (order key 0x007fffff)
constexpr uint64_t kHighest = ~0ull;

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float place_value(uint64_t c) { return key_value(static_cast<uint32_t>(c >> 32)); }

struct FiltParams {
  const void* logits;
  long long logits_ld;
  const float* gumbel;
  long long gumbel_ld;
  const int32_t* cu_nodes;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int max_nodes, vocab, bits;
  int32_t* tokens;
  float* logp;
  void* out;
  long long out_ld;
  int32_t* kept;
  int32_t* status;
};

struct FiltSmem {
  uint64_t list[kListCap];
  unsigned long long hist[kBins];
  uint32_t count[kBins];
  unsigned long long table[kWeightTable];
  uint64_t red[kFiltWarps];
  uint64_t small[kSmall];
  uint64_t found, base;
  int bin, bin_count, n_small;
  int n_list;
};

// ---------------------------------------------------------------- reductions

__device__ __forceinline__ uint64_t block_sum(uint64_t v, FiltSmem& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t t = 0;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) t += s.red[w];
  return t;
}

__device__ __forceinline__ float block_sum(float v, FiltSmem& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = __float_as_uint(v);
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) t += __uint_as_float(static_cast<uint32_t>(s.red[w]));
  return t;
}

__device__ __forceinline__ uint64_t block_max(uint64_t v, FiltSmem& s) {
  v = warp_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t t = 0;
#pragma unroll
  for (int w = 0; w < kFiltWarps; ++w) t = s.red[w] > t ? s.red[w] : t;
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

// f.many<n>(x, first index) for all entries of the row, n at a time (the ragged
// end one by one).
template <typename T, typename F>
__device__ __forceinline__ void for_row(const T* row, int vocab, F& f) {
  constexpr int kLen = Vec<T>::kLen;
  const uint4* vecs = reinterpret_cast<const uint4*>(row);
  const int n = vocab / kLen;
  for (int j0 = threadIdx.x; j0 < n; j0 += kFiltUnroll * kFiltThreads) {
    uint4 v[kFiltUnroll];
#pragma unroll
    for (int u = 0; u < kFiltUnroll; ++u)
      if (j0 + u * kFiltThreads < n) v[u] = vecs[j0 + u * kFiltThreads];
#pragma unroll
    for (int u = 0; u < kFiltUnroll; ++u) {
      const int j = j0 + u * kFiltThreads;
      if (j >= n) break;
      float x[kLen];
      Vec<T>::unpack(v[u], x);
      f.template many<kLen>(x, j * kLen);
    }
  }
  const int i = n * kLen + threadIdx.x;
  if (i < vocab) {
    float x[1] = {load_one(row + i)};
    f.template many<1>(x, i);
  }
}

// ------------------------------------------------------------------ the pass

// One pass over the row: places in [lo, hi] are listed (as many as fit, all
// are counted), those above are counted, those below weighed (kBelow); the
// others are weighed with kWeigh.
struct Bracket {
  uint64_t lo, hi;
  int n_in, n_above;
  uint64_t m_in, m_above, below;     // weights
  uint64_t best;                     // the largest place from lo on, 0 if there is none
};

template <bool kBelow, bool kWeigh>
struct PassBody {
  FiltSmem& s;
  uint64_t lo, hi;
  float lo_value, inv_t;
  WeightScale scale;
  uint64_t n_above, m_in, m_above, below, best;

  __device__ __forceinline__ void take(float x, int i) {
    const uint64_t c = pack_best(order_key(x), i);
    if (c < lo) {
      if (kBelow) below += weight_of(__fmul_rn(x, inv_t), scale, s.table);
      return;
    }
    if (c > best) best = c;
    const uint64_t w = kWeigh ? weight_of(__fmul_rn(x, inv_t), scale, s.table) : 0ull;
    if (c > hi) {
      ++n_above;
      m_above += w;
    } else {
      const int at = atomicAdd(&s.n_list, 1);
      if (at < kListCap) s.list[at] = c;
      m_in += w;
    }
  }

  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < kLen; ++e) any |= !(x[e] < lo_value);        // (a NaN is not below)
    if (kBelow) {
#pragma unroll
      for (int e = 0; e < kLen; ++e)
        if (x[e] < lo_value) below += weight_of(__fmul_rn(x[e], inv_t), scale, s.table);
    }
    if (any) {
#pragma unroll
      for (int e = 0; e < kLen; ++e)
        if (!(x[e] < lo_value)) take(x[e], i0 + e);
    }
  }
};

template <bool kBelow, bool kWeigh, typename T>
__device__ __noinline__ Bracket pass(const T* row, int vocab, uint64_t lo, uint64_t hi, float inv_t,
                                     const WeightScale& scale, FiltSmem& s) {
  __syncthreads();
  if (threadIdx.x == 0) s.n_list = 0;
  __syncthreads();
  PassBody<kBelow, kWeigh> body = {s, lo, hi, place_value(lo), inv_t, scale, 0, 0, 0, 0, 0};
  for_row(row, vocab, body);
  Bracket out;
  out.lo = lo;
  out.hi = hi;
  out.best = block_max(body.best, s);        // (its barriers close the list too)
  out.n_in = s.n_list;
  out.n_above = static_cast<int>(block_sum(body.n_above, s));
  out.m_in = out.m_above = out.below = 0;
  if (kWeigh) {
    out.m_in = block_sum(body.m_in, s);
    out.m_above = block_sum(body.m_above, s);
  }
  if (kBelow) out.below = block_sum(body.below, s);
  return out;
}

// ------------------------------------------------------------- the selection

// Among the n places of the list that lie in [a, b]: the first one, from the
// largest down, at which the sum of amounts reaches `target` (>= 1): amounts
// are weights, or 1 each. The sum of all of them has to reach it.
template <bool kWeigh>
__device__ __noinline__ uint64_t select(int n, uint64_t a, uint64_t b, uint64_t target, float inv_t,
                                        const WeightScale& scale, FiltSmem& s) {
  auto amount = [&](uint64_t c) -> uint64_t {
    return kWeigh ? weight_of(__fmul_rn(place_value(c), inv_t), scale, s.table) : 1ull;
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t base = 0, high = 0, low = 0;     // (low: inverted, so that 0 is nothing)
  for (int i = threadIdx.x; i < n; i += kFiltThreads) {
    const uint64_t c = s.list[i];
    if (c < a || c > b) continue;
    high = c > high ? c : high;
    low = ~c > low ? ~c : low;
  }
  b = block_max(high, s);
  a = ~block_max(low, s);
  if (a > b) return b;                     // nothing there (callers see to it that there is)
  while (true) {
    // bins of 2^sh places, counted from b down
    const int sh = b > a ? max(0, 54 - __clzll(b - a)) : 0;
    __syncthreads();
    for (int j = threadIdx.x; j < kBins; j += kFiltThreads) {
      s.hist[j] = 0;
      s.count[j] = 0;
    }
    if (threadIdx.x == 0) {
      s.bin = -1;
      s.n_small = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kFiltThreads) {
      const uint64_t c = s.list[i];
      if (c < a || c > b) continue;
      const int j = static_cast<int>((b - c) >> sh);
      atomicAdd(&s.count[j], 1u);
      if (kWeigh) atomicAdd(&s.hist[j], static_cast<unsigned long long>(amount(c)));
    }
    __syncthreads();
    constexpr int kEach = kBins / kFiltThreads;
    uint64_t mine[kEach], sum = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int j = threadIdx.x * kEach + u;
      mine[u] = kWeigh ? static_cast<uint64_t>(s.hist[j]) : s.count[j];
      sum += mine[u];
    }
    uint64_t up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    if (lane == 31) s.red[warp] = up;
    __syncthreads();
    uint64_t at = base + up - sum;
#pragma unroll
    for (int w = 0; w < kFiltWarps; ++w)
      if (w < warp) at += s.red[w];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (at < target && target <= at + mine[u]) {
        const int j = threadIdx.x * kEach + u;
        s.bin = j;
        s.base = at;
        s.bin_count = static_cast<int>(s.count[j]);
      }
      at += mine[u];
    }
    __syncthreads();
    const int bin = s.bin;
    if (bin < 0) return a;                 // not reached (as above)
    base = s.base;
    b -= static_cast<uint64_t>(bin) << sh;
    if (sh == 0) return b;
    const uint64_t end = b - ((1ull << sh) - 1);
    a = end > a && end <= b ? end : a;
    if (s.bin_count > kSmall) continue;
    // one warp ranks what is in the bin
    for (int i = threadIdx.x; i < n; i += kFiltThreads) {
      const uint64_t c = s.list[i];
      if (c >= a && c <= b) s.small[atomicAdd(&s.n_small, 1)] = c;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t c = lane < s.n_small ? s.small[lane] : 0ull;
      const uint64_t w = lane < s.n_small ? amount(c) : 0ull;
      uint64_t before = base;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const uint64_t oc = __shfl_sync(0xffffffffu, c, o), ow = __shfl_sync(0xffffffffu, w, o);
        if (oc > c) before += ow;
      }
      if (w != 0 && before < target && target <= before + w) s.found = c;
    }
    __syncthreads();
    return s.found;
  }
}

// A sample of the row's places in [a, b] becomes the list; returns how many.
// 128-byte lines lie evenly over the row, `turn` moves them.
template <typename T>
__device__ __noinline__ int sample_row(const T* row, int vocab, uint64_t a, uint64_t b, int turn, FiltSmem& s) {
  constexpr int kLine = 128 / sizeof(T), kLines = kSampleSize / kLine, kEach = kLine / 32;
  const int lines = vocab / kLine;         // >= kLines: the row does not fit the list
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (threadIdx.x == 0) s.n_list = 0;
  __syncthreads();
  float x[kLines / kFiltWarps][kEach];
  int at[kLines / kFiltWarps];
#pragma unroll
  for (int u = 0; u < kLines / kFiltWarps; ++u) {
    const int l = warp + u * kFiltWarps;
    const long long line = (static_cast<long long>(l) * lines + static_cast<long long>(turn) * (lines / 7 + 1)) / kLines;
    at[u] = static_cast<int>(line % lines) * kLine + lane;
#pragma unroll
    for (int e = 0; e < kEach; ++e) x[u][e] = load_one(row + at[u] + e * 32);
  }
#pragma unroll
  for (int u = 0; u < kLines / kFiltWarps; ++u) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint64_t c = pack_best(order_key(x[u][e]), at[u] + e * 32);
      const bool in = c >= a && c <= b;
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      int first = 0;
      if (lane == 0 && who) first = atomicAdd(&s.n_list, __popc(who));
      first = __shfl_sync(0xffffffffu, first, 0);
      if (in) s.list[first + __popc(who & ((1u << lane) - 1))] = c;
    }
  }
  __syncthreads();
  return s.n_list;
}

// ------------------------------------------------------------------ the place

// Bounds of the place that is looked for: it lies in [lo, hi], and n places
// with weight m lie above hi.
struct Bounds {
  uint64_t lo, hi;
  int n;
  uint64_t m;
};

// The next bracket inside the bounds, around the place where the count (or the
// weight) still missing is reached by a sample. From the fifth try on the
// bounds are cut in half.
template <bool kWeigh, typename T>
__device__ __forceinline__ void next_bracket(const T* row, int vocab, const Bounds& in, uint64_t target, int turn,
                                             float inv_t, const WeightScale& scale, FiltSmem& s, uint64_t& lo,
                                             uint64_t& hi) {
  lo = in.lo;
  hi = in.hi;
  if (vocab <= kListCap) return;
  if (turn > kSampledTurns) {
    lo = in.lo + (in.hi - in.lo) / 2 + 1;
    if (lo > in.hi) lo = in.hi;
    return;
  }
  const int m = sample_row(row, vocab, in.lo, in.hi, turn, s);
  if (m == 0) return;
  // one of the sample stands for `each` of the row
  const float each = static_cast<float>(vocab) / kSampleSize;
  float rank;
  if (kWeigh) {
    const uint64_t missing = max(1ull, static_cast<unsigned long long>(static_cast<float>(target - in.m) / each));
    uint64_t all = 0;
    for (int i = threadIdx.x; i < m; i += kFiltThreads)
      all += weight_of(__fmul_rn(place_value(s.list[i]), inv_t), scale, s.table);
    all = block_sum(all, s);
    if (all < missing) {
      rank = static_cast<float>(m);
    } else {
      const uint64_t c = select<true>(m, in.lo, in.hi, missing, inv_t, scale, s);
      uint64_t r = 0;
      for (int i = threadIdx.x; i < m; i += kFiltThreads) r += s.list[i] >= c;
      rank = static_cast<float>(block_sum(r, s));
    }
  } else {
    rank = static_cast<float>(target - in.n) / each;
  }
  const float margin = 4.0f * sqrtf(rank) + 8.0f;
  const int down = static_cast<int>(fminf(rank + margin, 1e9f)), up = static_cast<int>(rank - margin);
  if (down <= m) lo = select<false>(m, in.lo, in.hi, down, inv_t, scale, s);
  if (up >= 1 && up <= m) hi = select<false>(m, in.lo, in.hi, up, inv_t, scale, s);
}

// The place at which the count (or the weight) from the top reaches target,
// within the bounds. Leaves the last bracket in `view`, its places on the list.
template <bool kWeigh, typename T>
__device__ __noinline__ uint64_t locate(const T* row, int vocab, Bounds in, uint64_t target, float inv_t,
                                        const WeightScale& scale, FiltSmem& s, Bracket& view) {
  for (int turn = 1; turn <= kTurns; ++turn) {
    uint64_t lo, hi;
    next_bracket<kWeigh>(row, vocab, in, target, turn, inv_t, scale, s, lo, hi);
    view = pass<false, kWeigh>(row, vocab, lo, hi, inv_t, scale, s);
    const uint64_t above = kWeigh ? view.m_above : static_cast<uint64_t>(view.n_above);
    const uint64_t with = above + (kWeigh ? view.m_in : static_cast<uint64_t>(view.n_in));
    if (above >= target) {
      in.lo = hi + 1;                      // (hi < in.hi, above which the target is not reached)
    } else if (with < target) {
      if (lo == in.lo) return in.lo;       // all that there is
      in.hi = lo - 1;
      in.n = view.n_above + view.n_in;
      in.m = view.m_above + view.m_in;
    } else if (view.n_in <= kListCap) {
      return select<kWeigh>(view.n_in, lo, hi, target - above, inv_t, scale, s);
    } else {
      in.lo = lo;
      in.hi = hi;
      in.n = view.n_above;
      in.m = view.m_above;
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
  bool empty;              // nothing above -inf
  bool listed;             // all that is kept is on the list
  int n_list;
  WeightScale scale;
};

template <typename T>
__device__ __forceinline__ RowResult find_cut(const T* row, int vocab, int bits, float inv_t, int k, float p,
                                              float min_p, FiltSmem& s) {
  const bool by_k = k > 0 && k < vocab, by_p = p < 1.0f, by_m = min_p > 0.0f;
  uint64_t lo = kLowest, hi = kHighest;
  const WeightScale none = weight_scale(0.0f, bits);
  // 1. where the list begins (and ends, for a top-k set that no list holds)
  if (vocab > kListCap) {
    const int m = sample_row(row, vocab, kLowest, kHighest, 0, s);
    const float rank = static_cast<float>(by_k ? k : 1024) * kSampleSize / vocab;
    const float margin = 3.0f * sqrtf(rank) + 8.0f;
    const int down = static_cast<int>(fminf(rank + margin, 1e9f)), up = static_cast<int>(rank - margin);
    if (down <= m) lo = select<false>(m, kLowest, kHighest, down, inv_t, none, s);
    if (static_cast<float>(down) * vocab / kSampleSize > kListCap && up >= 1 && up <= m)
      hi = select<false>(m, kLowest, kHighest, up, inv_t, none, s);
  }
  // 2. the list; weights below it relative to its first place, a power of two
  // from the row's (not where the reduction differs)
  const bool total = by_p && !by_k;
  const float s_lo = __fmul_rn(place_value(lo), inv_t);
  const WeightScale low_scale = weight_scale(s_lo, bits);
  const bool low_fits = fabsf(s_lo) < kWeightSpan;
  Bracket view = total && low_fits ? pass<true, false>(row, vocab, lo, hi, inv_t, low_scale, s)
                                   : pass<false, false>(row, vocab, lo, hi, inv_t, none, s);
  if (view.best == 0) return RowResult{kHighest, true, true, 0, none};       // (lo is kLowest then)
  const WeightScale scale = weight_scale(__fmul_rn(place_value(view.best), inv_t), bits);
  uint64_t cut = kLowest;
  // 3. top-k
  if (by_k) {
    const int with = view.n_above + view.n_in;
    if (view.n_above >= k) {
      cut = locate<false>(row, vocab, Bounds{view.hi + 1, kHighest, 0, 0}, k, inv_t, scale, s, view);
    } else if (with < k) {                 // (from the lowest place on fewer than k: all stay)
      if (view.lo > kLowest) cut = locate<false>(row, vocab, Bounds{kLowest, view.lo - 1, with, 0}, k, inv_t, scale, s, view);
    } else if (view.n_in <= kListCap) {
      cut = select<false>(view.n_in, view.lo, view.hi, k - view.n_above, inv_t, scale, s);
    } else {
      cut = locate<false>(row, vocab, Bounds{view.lo, view.hi, view.n_above, 0}, k, inv_t, scale, s, view);
    }
  }
  // 4. top-p of what top-k leaves
  if (by_p) {
    uint64_t z;
    bool whole = view.hi == kHighest && view.n_in <= kListCap;      // the list holds all from view.lo on
    if (total ? !(low_fits && whole && scale.ref == 0.0f && !scale.tie) : !(whole && cut >= view.lo)) {
      // the sum in a pass of its own, the list anew beside it
      view = pass<false, true>(row, vocab, cut, kHighest, inv_t, scale, s);
      z = view.m_in;
      whole = view.n_in <= kListCap;
    } else {
      uint64_t sum = 0;
      const uint64_t from = by_k ? cut : view.lo;
      for (int i = threadIdx.x; i < view.n_in; i += kFiltThreads)
        if (s.list[i] >= from) sum += weight_of(__fmul_rn(place_value(s.list[i]), inv_t), scale, s.table);
      view.m_in = block_sum(sum, s);
      z = view.m_in;
      if (total) {
        const int down = scale.k - low_scale.k;
        z += down < 64 ? view.below >> down : 0ull;
      }
    }
    const uint64_t target = share_of(p, z);
    uint64_t at;
    if (whole && view.m_in >= target) {
      at = select<true>(view.n_in, view.lo > cut ? view.lo : cut, kHighest, target, inv_t, scale, s);
    } else {
      Bounds in = {cut, kHighest, 0, 0};
      if (whole && view.lo > cut) in = {cut, view.lo - 1, view.n_in, view.m_in};
      at = locate<true>(row, vocab, in, target, inv_t, scale, s, view);
    }
    if (at > cut) cut = at;
  }
  // 5. min-p
  if (by_m) {
    float least = scale.s_max;
    if (!scale.tie) least = __double2float_ru(static_cast<double>(scale.s_max) + log(static_cast<double>(min_p)));
    const uint32_t key = scale.s_max != scale.s_max ? 0xffffffffu : smallest_key(least, inv_t);
    const uint64_t at = static_cast<uint64_t>(key) << 32;
    if (at > cut) cut = at;
  }
  return RowResult{cut, false, view.hi == kHighest && view.n_in <= kListCap && cut >= view.lo, view.n_in, scale};
}

// ------------------------------------------------------------------- endings

// ln of the kept share of a token: its weight over the sum of all kept ones.
__device__ __forceinline__ float log_share(float s_tok, uint64_t sum, const WeightScale& w, const unsigned long long* table) {
  const uint64_t mine = weight_of(s_tok, w, table);
  if (mine > sum / 2) return log1pf(-(static_cast<float>(sum - mine) / static_cast<float>(sum)));
  const float total = static_cast<float>(sum) * exp2f(static_cast<float>(-w.bits));
  if (w.tie) return mine ? -logf(total) : -kInf;
  const float s = s_tok - w.ref;
  const float yh = __fmul_rn(s, kLog2e);
  const float yl = __fmaf_rn(s, kLog2eLow, __fmaf_rn(s, kLog2e, -yh));
  return kLn2 * ((yh - static_cast<float>(w.k)) + yl) - logf(total);
}

struct DrawBody {
  const float* noise;
  uint64_t cut;
  float cut_value, inv_t;
  bool weigh;
  WeightScale scale;
  const unsigned long long* table;
  uint64_t best, sum;

  __device__ __forceinline__ void take(float x, int i) {
    if (pack_best(order_key(x), i) < cut) return;
    const float sx = __fmul_rn(x, inv_t);
    const uint64_t c = pack_best(order_key(__fadd_rn(sx, noise[i])), i);
    if (c > best) best = c;
    if (weigh) sum += weight_of(sx, scale, table);
  }
  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
#pragma unroll
    for (int e = 0; e < kLen; ++e)
      if (!(x[e] < cut_value)) take(x[e], i0 + e);
  }
};

// No filter: all of the noise is read beside the logits, the sum of weights is
// float32 relative to a running maximum (nothing is decided by it).
struct FreeBody {
  const float* noise;
  float inv_t;
  uint64_t best;
  float top, sum, nans;

  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
    float s[kLen], g[kLen], high = top;
    if constexpr (kLen % 4 == 0) {
#pragma unroll
      for (int e = 0; e < kLen; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(noise + i0 + e);
        g[e] = v.x; g[e + 1] = v.y; g[e + 2] = v.z; g[e + 3] = v.w;
      }
    } else {
      g[0] = noise[i0];
    }
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      s[e] = __fmul_rn(x[e], inv_t);
      high = fmaxf(high, s[e]);
      const uint64_t c = pack_best(order_key(__fadd_rn(s[e], g[e])), i0 + e);
      if (x[e] != -kInf && c > best) best = c;
    }
    if (high > top) {
      sum *= fast_exp2((top - high) * kLog2e);
      top = high;
    }
#pragma unroll
    for (int e = 0; e < kLen; ++e) {       // equal infinities weigh 1
      if (s[e] != s[e]) nans += 1.0f;
      else sum += s[e] == top ? 1.0f : fast_exp2((s[e] - top) * kLog2e);
    }
  }
};

struct TopBody {
  uint64_t best;
  template <int kLen>
  __device__ __forceinline__ void many(const float* x, int i0) {
#pragma unroll
    for (int e = 0; e < kLen; ++e) {
      const uint64_t c = pack_best(order_key(x[e]), i0 + e);
      if (c > best) best = c;
    }
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
    else reinterpret_cast<uint4*>(out)[i0 / kLen] = Vec<T>::pack(y);
  }
};

template <typename T, bool kSampling>
__global__ void __launch_bounds__(kFiltThreads, 2) filtered_kernel(const __grid_constant__ FiltParams p) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  FiltSmem& s = *reinterpret_cast<FiltSmem*>(s_raw);
  if (threadIdx.x < kWeightTable) s.table[threadIdx.x] = c_weight_table[threadIdx.x];
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.y, node = blockIdx.x;
  const int st = p.status[b];
  const int t0 = p.cu_nodes[b], n = p.cu_nodes[b + 1] - t0;
  const float temp = p.temperature[b];
  const int k = p.top_k ? p.top_k[b] : 0;
  const float top_p = p.top_p ? p.top_p[b] : 1.0f, min_p = p.min_p ? p.min_p[b] : 0.0f;
  if (st != 0 || (node >= n && n >= 0)) return;
  const float inv_t = temp > 0.0f ? __frcp_rn(temp) : 1.0f;
  int flag = 0;
  if (n > p.max_nodes || n < 0 || t0 < 0) flag |= TV_ST_BAD_SIZE;
  if (!(temp >= 0.0f) || temp == kInf || inv_t == kInf || (kSampling && temp > 0.0f && !p.gumbel)) flag |= TV_ST_BAD_TEMPERATURE;
  if (k < 0 || !(top_p >= 0.0f && top_p <= 1.0f) || !(min_p >= 0.0f && min_p <= 1.0f)) flag |= TV_ST_BAD_FILTER;
  if (flag) {
    if (node == 0 && threadIdx.x == 0) atomicOr(&p.status[b], flag);
    return;
  }
  const size_t t = static_cast<size_t>(t0) + node;
  const T* row = static_cast<const T*>(p.logits) + t * p.logits_ld;
  const int vocab = p.vocab;
  const bool greedy = temp == 0.0f;
  const bool filtered = !greedy && ((k > 0 && k < vocab) || top_p < 1.0f || min_p > 0.0f);
  __syncthreads();

  RowResult res = {kLowest, false, false, 0, weight_scale(0.0f, p.bits)};
  if (greedy) {
    TopBody body = {0};
    for_row(row, vocab, body);
    const uint64_t best = block_max(body.best, s);
    res.empty = best < kLowest;
    res.cut = res.empty ? kHighest : best;
    if (kSampling) {
      if (threadIdx.x == 0) {
        p.tokens[t] = res.empty ? 0 : best_index(best);
        if (p.logp) p.logp[t] = res.empty ? -kInf : 0.0f;
      }
      return;
    }
  } else if (filtered) {
    res = find_cut(row, vocab, p.bits, inv_t, k, top_p, min_p, s);
  }

  if constexpr (kSampling) {
    const float* noise = p.gumbel + t * p.gumbel_ld;
    if (!filtered) {
      FreeBody body = {noise, inv_t, 0, -kInf, 0.0f, 0.0f};
      for_row(row, vocab, body);
      const uint64_t best = block_max(body.best, s);
      const int token = best ? best_index(best) : 0;
      if (threadIdx.x == 0) p.tokens[t] = token;
      if (p.logp) {
        const float top = key_value(static_cast<uint32_t>(block_max(order_key(body.top), s)));
        const float sum = block_sum(body.top == top ? body.sum : body.sum * fast_exp2((body.top - top) * kLog2e), s);
        const float nans = block_sum(body.nans, s);
        if (threadIdx.x == 0) {
          const float mine = __fmul_rn(load_one(row + token), inv_t);
          float out = (mine == top ? 0.0f : mine - top) - logf(sum);
          if (nans > 0.0f) out = mine != mine ? -logf(nans) : -kInf;
          p.logp[t] = best ? out : -kInf;
        }
      }
      return;
    }
    if (res.empty) {
      if (threadIdx.x == 0) {
        p.tokens[t] = 0;
        if (p.logp) p.logp[t] = -kInf;
      }
      return;
    }
    DrawBody body = {noise, res.cut, place_value(res.cut), inv_t, p.logp != nullptr, res.scale, s.table, 0, 0};
    if (res.listed) {
      for (int i = threadIdx.x; i < res.n_list; i += kFiltThreads) {
        const uint64_t c = s.list[i];
        if (c >= res.cut) body.take(place_value(c), best_index(c));
      }
    } else {
      for_row(row, vocab, body);
    }
    const uint64_t best = block_max(body.best, s);
    const uint64_t sum = p.logp ? block_sum(body.sum, s) : 0;
    if (threadIdx.x == 0) {
      const int token = best_index(best);
      p.tokens[t] = token;
      if (p.logp) p.logp[t] = log_share(__fmul_rn(load_one(row + token), inv_t), sum, res.scale, s.table);
    }
  } else {
    MaskBody<T> body = {static_cast<T*>(p.out) + t * p.out_ld, res.cut, place_value(res.cut), 0};
    for_row(row, vocab, body);
    if (p.kept) {
      const uint64_t kept = block_sum(body.kept, s);
      if (threadIdx.x == 0) p.kept[t] = static_cast<int>(kept);
    }
  }
}

// ------------------------------------------------------------------ host side

static int check_filter(int dtype, const void* logits, long long ld, int batch, int max_nodes, int vocab) {
  if (dtype != TV_DTYPE_BF16 && dtype != TV_DTYPE_F32) return TV_ERR_BAD_GEOMETRY;
  if (batch < 0 || batch > 65535 || max_nodes < 1 || max_nodes > TV_MAX_NODES || vocab < 1 || vocab > (1 << 30) || ld < vocab)
    return TV_ERR_BAD_SIZE;
  return TV_OK;
}

template <bool kSampling>
static int launch_filtered(int dtype, FiltParams& p, int batch, void* stream) {
  static size_t smem_set[2][kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return TV_ERR_CUDA;
  auto* kernel = dtype == TV_DTYPE_F32 ? filtered_kernel<float, kSampling> : filtered_kernel<__nv_bfloat16, kSampling>;
  if (!ensure_smem(kernel, sizeof(FiltSmem), smem_set[dtype], dev)) return TV_ERR_CUDA;
  p.bits = weight_bits(p.vocab);
  const cudaError_t err = launch_pdl(kernel, dim3(p.max_nodes, batch), dim3(kFiltThreads), sizeof(FiltSmem), as_stream(stream), p);
  return err == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace tv

extern "C" int tv_sample_filtered(int32_t dtype, const void* logits, int64_t logits_ld, const float* gumbel,
                                  int64_t gumbel_ld, const int32_t* cu_nodes, const float* temperature,
                                  const int32_t* top_k, const float* top_p, const float* min_p, int32_t batch,
                                  int32_t max_nodes, int32_t vocab, int32_t* tokens, float* logp, int32_t* status,
                                  void* stream) {
  int rc = tv::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (gumbel && gumbel_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !tokens || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || (gumbel && (!tv::aligned(gumbel, 16) || gumbel_ld % 4)))
    return TV_ERR_MISALIGNED;
  tv::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld; p.gumbel = gumbel; p.gumbel_ld = gumbel_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.max_nodes = max_nodes; p.vocab = vocab; p.tokens = tokens; p.logp = logp; p.status = status;
  return tv::launch_filtered<true>(dtype, p, batch, stream);
}

extern "C" int tv_filter_logits(int32_t dtype, const void* logits, int64_t logits_ld, const int32_t* cu_nodes,
                                const float* temperature, const int32_t* top_k, const float* top_p,
                                const float* min_p, int32_t batch, int32_t max_nodes, int32_t vocab, void* out,
                                int64_t out_ld, int32_t* kept, int32_t* status, void* stream) {
  int rc = tv::check_filter(dtype, logits, logits_ld, batch, max_nodes, vocab);
  if (rc != TV_OK) return rc;
  if (out_ld < vocab) return TV_ERR_BAD_SIZE;
  if (batch == 0) return TV_OK;
  if (!logits || !cu_nodes || !temperature || !out || !status) return TV_ERR_NULL_POINTER;
  const int per = dtype == TV_DTYPE_F32 ? 4 : 8;
  if (!tv::aligned(logits, 16) || logits_ld % per || !tv::aligned(out, 16) || out_ld % per) return TV_ERR_MISALIGNED;
  tv::FiltParams p = {};
  p.logits = logits; p.logits_ld = logits_ld;
  p.cu_nodes = cu_nodes; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.max_nodes = max_nodes; p.vocab = vocab; p.out = out; p.out_ld = out_ld; p.kept = kept; p.status = status;
  return tv::launch_filtered<false>(dtype, p, batch, stream);
}
