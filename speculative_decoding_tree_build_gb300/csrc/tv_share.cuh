// A CTA's share of a ragged batch: the work of all requests laid end to end
// and cut into equal contiguous ranges, computed on the device from the
// per-request lengths (no host round trip, no atomics).
#pragma once

#include "tv_common.cuh"

namespace tv {

// a / b for b > 0; in 32 bits where they fit (a 64-bit division is a routine of
// some hundred instructions, and the shares stand ahead of all other loads).
__device__ __forceinline__ long long divide(long long a, long long b) {
  if ((static_cast<unsigned long long>(a) | static_cast<unsigned long long>(b)) >> 32) return a / b;
  return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

struct Share {
  long long lo, hi;      // the CTA's range of the sequence; lo >= hi: nothing to do
  long long total;       // the whole sequence
  long long start;       // where request b starts in it
  int b;                 // the request that holds lo
  int ctas;              // CTAs that share the work: the first `longer` take each + 1 of it, the others each
  int longer;            // (those come in the order of the SMs: longer shares strewn among the others 20.2 us, first
                         // 19.4 us for 168 units of 8 to 69 tiles)
  long long each;

  __device__ __forceinline__ long long start_of(int cta) const { return each * cta + min(cta, longer); }
  // the CTA that has position x of the sequence
  __device__ __forceinline__ int owner(long long x) const {
    const long long edge = (each + 1) * longer;
    return static_cast<int>(x < edge ? divide(x, each + 1) : longer + divide(x - edge, each));
  }
};

// work(b) >= 0 is request b's amount. At least `least` of it goes to a CTA.
// Every thread of the CTA (kThreads of them) calls this and gets the same
// answer: each sums the work of a run of requests, a scan over the threads
// gives the total, and the thread whose run holds the range's start walks it.
template <int kThreads, typename Work>
__device__ __forceinline__ Share find_share(int batch, int least, Work work) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_start;
  __shared__ int s_b;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = (batch + kThreads - 1) / kThreads;
  const int r0 = min(batch, static_cast<int>(threadIdx.x) * per), r1 = min(batch, r0 + per);
  long long mine = 0;
  for (int b = r0; b < r1; ++b) mine += work(b);
  long long upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += o;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  Share r;
  r.total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_sum[w];
    r.total += s_sum[w];
  }
  const long long before = upto - mine;
  const long long most = (r.total + least - 1) / least;
  r.ctas = static_cast<int>(most < static_cast<long long>(gridDim.x) ? most : gridDim.x);
  const int cta = blockIdx.x;
  r.each = divide(r.total, max(r.ctas, 1));
  r.longer = static_cast<int>(r.total - r.each * r.ctas);
  r.lo = cta < r.ctas ? r.start_of(cta) : r.total;
  r.hi = cta < r.ctas ? r.start_of(cta + 1) : r.total;
  r.b = 0;
  r.start = 0;
  if (r.lo >= r.hi) return r;
  if (mine > 0 && r.lo >= before && r.lo < upto) {
    long long at = before;
    int b = r0;
    for (; b + 1 < r1; ++b) {
      const long long c = work(b);
      if (r.lo < at + c) break;
      at += c;
    }
    s_b = b;
    s_start = at;
  }
  __syncthreads();
  r.b = s_b;
  r.start = s_start;
  return r;
}

}  // namespace tv
