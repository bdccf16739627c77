// tv_decode_attention: attention of one new token per request over its paged
// cache, bf16 or 8 bits.
//
//   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
//
// What bounds it: the cache is read once and a byte of it takes 2 G / size
// multiply-adds (G query heads to a cached head), far below the tensor
// cores' rate per byte, so the floor is the cache's bytes at HBM bandwidth.
// The design follows from that:
//  - The G <= 16 query heads that share a cached head go together, so every
//    cached row is read once. They are the N side of mma.sync m16n8k16 and the
//    cached rows the M side: S^T = K Q^T (16 keys x 8 queries), O^T = V^T P^T
//    (16 columns of D x 8 queries). At this intensity a tcgen05 tile of 128
//    rows would be 7/8 empty, and the register path needs no staging:
//  - Cached rows go from global memory straight to registers in the layout
//    that the MMA wants. The contraction may run over D and over the keys in
//    any order, so each thread takes whole 16-byte pieces: of K the pieces
//    t, t + 4, ... of rows g and g + 8, of V the piece g of rows 2t, 2t + 1,
//    2t + 8, 2t + 9 (g = lane / 4, t = lane % 4). V's two rows are interleaved
//    by byte permutes on the way into the MMA. No shared memory, no barriers
//    in the loop: 12 to 16 warps an SM with a page each of K and V in flight.
//  - 8-bit codes become f16 exactly (e4m3 by the hardware's conversion, int8
//    through the 1024 + u trick). Queries are scaled to f16 by a power of two
//    per head, which is exact but for elements 2^-14 below the head's largest.
//  - The softmax's reference is not the exact running maximum: it moves only
//    when a score exceeds it by 2^8, so the common page takes one warp vote
//    and no reduction; weights stay below 2^8. A value row's scale joins the
//    exponent: w_j = 2^(s_j + log2 vscale_j - M), with its own reference M that
//    moves to 2^7 below the largest: that one is 2^7 to 2^15 in f16 whatever the
//    scales are, and half of f16's smallest step at most 2^-32 of it. The sum of
//    the softmax is float32 of unrounded terms. DecTraits::kTwice tells in how
//    many parts the weights go.
//
// Work plan: a unit is (request, KV head), its tiles are 64 keys (a page for
// each of the CTA's four warps). All units' tiles are laid end to end and
// every CTA takes a contiguous share, whatever the mix of lengths; the share
// is computed by each CTA from seq_len, so no host round trip. A unit cut
// between CTAs leaves one partial result a CTA in the workspace and a second
// grid joins them in order. Where the block table is short and there are few
// units, every unit goes to a cluster of 1 to 8 CTAs of 4 or 8 warps instead,
// which join their results through distributed shared memory: one launch, and one
// round trip less ahead of the first cached row (launch_decode has the rule).
//
// Measured: 64 requests of 4096 to 32768 keys, 32/8 heads of 128, e4m3 (1.9
// GB) 295 us, 6.4 TB/s; one of 32768 keys, bf16 (134 MB) 28 us, of which the
// first grid 20.
#include <cuda_fp16.h>

#include <type_traits>

#include "tv_cluster.cuh"
#include "tv_kv8.cuh"
#include "tv_share.cuh"

namespace tv {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecTileKeys = TV_BLOCK_SIZE * kDecWarps;
constexpr int kDecUnitCost = 2;        // fixed cost of a unit, in tiles
constexpr int kDecMinShare = 3;        // least cost worth a CTA of its own: a unit of one tile
constexpr int kDecMaxCluster = 8;
constexpr int kFewWarps = 8;           // warps an SM that are few, and pages of a warp up to which a
constexpr int kClusterPagesFew = 3;    // unit's warps are not doubled with no more than those
constexpr int kClusterPages = 4;       // or with more
constexpr int kOneGridPages = 16;      // pages of a warp at most in the one-launch form,
constexpr int kOneGridExcess = 5;      // and how many more than in an even share
constexpr int kDecMaxPerSm = 4;        // CTAs an SM at most, for the workspace
constexpr int kDecMaxHeads = 4096;     // KV heads at most: unit numbers stay below 2^24
constexpr int kMergeWarps = 4;         // warps of a joining CTA at least
constexpr int kMergeMaxParts = 8;      // warps that share a query head's partials at most
constexpr int kMergeBatch = 8;         // partials whose sums a warp has in flight
constexpr float kRefBelow = 7.0f;      // log2 of the largest weight over 8-bit values when its reference moves
constexpr float kLowest = -3.4028234663852886e38f;

// What the CTA that begins a unit tells the joining grid: the CTAs that work
// on the unit (its own partial is its slot 1, the others' their slot 0).
// last < 0: nothing to join.
struct DecBegin {
  int unit, first, last, pad;
};

struct DecodeParams {
  const __nv_bfloat16* q;
  long long q_ld;
  const int32_t* seq_len;
  const int32_t* block_table;
  const int32_t* n_blocks;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;
  float* lse;
  DecBegin* begins;    // by unit, or by CTA where there are more units than CTAs
  int* mids;           // [CTAs] the unit whose partial is in slot 0, -1: none
  float* partials;     // two slots a CTA: [group][D] sums, then [group] x (m, M, l, -)
  int32_t* status;
  int batch, hq, hkv, group, max_blocks, num_blocks;
  int cluster;         // CTAs of a unit in the one-launch form
  int by_unit;         // how begins is indexed
  int parts;           // warps that share a query head's partials
  float scale_log2;
};

__host__ __device__ constexpr size_t dec_slot_floats(int group, int d) { return static_cast<size_t>(group) * (d + 4); }

// ------------------------------------------------------------------ pieces

// Loads that stay where they are written, ahead of the branches that follow.
// (Not .nc: the grid may be resident while the one before it still writes.)

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ uint2 ldg_stream8(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

__device__ __forceinline__ int ldg_int(const int32_t* p) {
  int r;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

__device__ __forceinline__ float ldg_float(const float* p) {
  float r;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(r) : "l"(p));
  return r;
}

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (kHalf) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Transpose of an 8 x 8 matrix of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a weight w >= 0 cut off to the bf16 number h leaves, never 0 beside an h
// above 0: two positive parts carry an infinite value to the output, where a
// second part of 0 or below would make inf * 0 or inf - inf of it. It is taken as
// 2^-24 of h (float32's own rounding) at least, and as the smallest bf16 number
// where that underflows. The parts miss w by 2^-16 of it at the most: the rest is
// below 2^-7 of w's power of two and is rounded to 8 bits.
__device__ __forceinline__ float weight_rest(float w, float h) {
  return fmaxf(fmaxf(w - h, h * 0x1p-24f), fminf(h, 0x1p-133f));
}

// Four codes of a word to two f16x2: (byte 0, byte 1) and (byte 2, byte 3).
template <int kFmt>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kFmt == TV_KV_E4M3) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    // code + 128 = u in the last bits of f16 1024 + u, then minus 1152: exact
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// Tiles of a request; a request without keys, or one that will be flagged, is
// one tile that computes nothing.
__device__ __forceinline__ int dec_tiles(int n, int max_blocks) {
  if (n <= 0 || n > static_cast<long long>(max_blocks) * TV_BLOCK_SIZE) return 1;
  return (n - 1) / kDecTileKeys + 1;
}

// Two columns of a query head's output from the joined sums, and its log-sum-exp.
template <int D>
__device__ __forceinline__ void dec_store(const DecodeParams& p, int b, int h, int qi, int d, int n, float2 acc, float mm, float mr, float ll) {
  const size_t at = static_cast<size_t>(b) * p.hq + static_cast<size_t>(h) * p.group + qi;
  const float f = n == 0 ? 0.0f : fast_exp2(mr - mm) / ll;
  *reinterpret_cast<uint32_t*>(p.out + at * D + d) = pack_bf16x2(acc.x * f, acc.y * f);
  if (p.lse != nullptr && d == 0) p.lse[at] = n == 0 ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
}

__device__ __forceinline__ float2 as_float2(uint64_t v) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// ------------------------------------------------------------------ the kernel

// kQ: query heads to a cached head at most, 4, 8 or 16.
template <int kFmt, int D, int kQ>
struct DecTraits {
  static constexpr int NT = kQ > 8 ? 2 : 1;                    // MMA tiles of eight queries
  // A weight goes to the MMA as a number of the values' 16-bit type. In one part
  // bf16's rounding would add as much to the error as the output's own does, so
  // over bf16 pools it goes in two parts. f16's is an eighth of that: 0.00167
  // against 64 bits, where the output's own rounding makes 0.00166.
  // Up to four queries stand twice among the MMA's eight, the first four for the
  // first parts and the others for the second, so there two parts cost no product
  // (e4m3, 1.9 GB: 293.7 -> 295.4 us) and are taken for all formats. With more
  // queries over 8-bit pools it is one part: a second product takes 27.2 -> 29.1
  // us (101 MB, 8 queries, int8) for a hundredth of the error.
  static constexpr bool kTwice = kQ == 4;
  static constexpr bool kHalf = kFmt != TV_KV_BF16;
  static constexpr int kElem = kHalf ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kKPieces = kRowBytes / 64;              // 16-byte pieces of a K row a thread holds
  static constexpr int kSteps = D / 16;                        // MMA steps over D (QK), tiles of D (PV)
  static constexpr int kVPieces = kRowBytes >= 128 ? kRowBytes / 128 : 1;    // of a V row (8 bytes at 64)
  // Pages that a warp takes at a time: two of the smallest ones, whose chain of
  // products, exponentials and waits would else be as long for half the bytes
  // (64 sequences of 4096 to 16384 keys, D = 64, e4m3: 129 -> 110 us).
  static constexpr int kPages = kRowBytes == 64 && NT == 1 ? 2 : 1;
  // CTAs an SM: registers for the pages, the queries and the output
  // accumulators. More warps are worth more than more pages a warp (D = 128,
  // e4m3, 1.9 GB: 4 CTAs 293 us, 3 CTAs 309 us, 3 CTAs with two pages in
  // flight a warp 357 us), until the registers spill (two groups of queries,
  // D = 128: 2 CTAs 21 us, 3 CTAs 23 us).
  static constexpr int kPerSm = NT == 2 ? (D == 64 ? 3 : 2) : kRowBytes == 256 ? 3 : 4;
  // Warps of a CTA at most in the one-launch form: two CTAs' worth where that
  // leaves a thread its registers.
  static constexpr int kMaxWarps = kPerSm == 4 ? 2 * kDecWarps : kDecWarps;
};

// kOneGrid: a unit belongs to a cluster of p.cluster CTAs, whose kWarps warps
// take its pages in turn; else a CTA takes a share of all units' tiles.
template <int kFmt, int D, int kQ, bool kOneGrid, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (DecTraits<kFmt, D, kQ>::kPerSm * kDecWarps / kWarps))
decode_kernel(const __grid_constant__ DecodeParams p) {
  using Tr = DecTraits<kFmt, D, kQ>;
  constexpr int NT = Tr::NT;
  constexpr bool kTwice = Tr::kTwice;
  static_assert(kOneGrid || kWarps == kDecWarps, "a tile is a page for each warp");
  constexpr bool kHalf = Tr::kHalf;
  constexpr int kRowBytes = Tr::kRowBytes, kKPieces = Tr::kKPieces, kVPieces = Tr::kVPieces, kSteps = Tr::kSteps;
  constexpr int kPages = Tr::kPages;
  constexpr int kRowPad = D + 4;
  extern __shared__ float s_o[];                               // [warps][8 NT][D + 4]
  constexpr int kThreads = 32 * kWarps;
  __shared__ float4 s_stat[kWarps][16];                        // (m, M, l, -)
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  auto query = [&](int x) { return kTwice ? g % 4 : x * 8 + g; };        // of the MMA's column g
  grid_launch_dependents();
  if (!kOneGrid) grid_dependency_wait();

  __shared__ float4 s_joined[16];                              // the CTA's (m, M, l, faulty) for its cluster
  const int cta = blockIdx.x;
  int b, h, n, nt, tile0 = 0, rank = 0;
  __shared__ Share s_share;            // thread 0's, for the end of a unit
  long long hi = 0;
  long long unit = 0;                  // where the unit starts in the sequence of costs
  int mid = -1;                        // the unit whose partial this CTA leaves in slot 0
  DecBegin begun = {0, 0, -1, 0};      // the unit that it begins and does not finish
  if constexpr (kOneGrid) {
    rank = blockIdx.x;
    h = blockIdx.y;
    b = blockIdx.z;
    nt = 1;
  } else {
    // ---- this CTA's share of the tiles
    const Share share = find_share<kDecThreads>(p.batch, kDecMinShare, [&](int i) {
      return static_cast<long long>(p.hkv) * (kDecUnitCost + dec_tiles(p.seq_len[i], p.max_blocks));
    });
    hi = share.hi;
    if (threadIdx.x == 0) s_share = share;
    if (share.lo >= share.hi) {
      if (threadIdx.x == 0) {
        p.mids[cta] = -1;
        if (!p.by_unit) p.begins[cta] = begun;
      }
      return;
    }
    b = share.b;
    n = p.seq_len[b];
    nt = dec_tiles(n, p.max_blocks);
    const long long cost = kDecUnitCost + nt, rel = share.lo - share.start;
    h = static_cast<int>(divide(rel, cost));
    const long long off = rel - h * cost;
    unit = share.start + h * cost;
    // tile 0 starts at 0, tile k at kDecUnitCost + k
    tile0 = off == 0 ? 0 : off <= kDecUnitCost + 1 ? 1 : static_cast<int>(off - kDecUnitCost);
  }

  for (;;) {
    // ---- the next unit, or part of one
    if (tile0 >= nt) {
      if (kOneGrid) break;
      unit += kDecUnitCost + nt;
      tile0 = 0;
      if (++h == p.hkv) {
        h = 0;
        if (++b == p.batch) break;
        n = p.seq_len[b];
        nt = dec_tiles(n, p.max_blocks);
      }
      continue;
    }
    if (!kOneGrid && (tile0 == 0 ? unit >= hi : unit + kDecUnitCost + tile0 >= hi)) break;
    int tile1 = nt;
    if (!kOneGrid && hi - unit - kDecUnitCost < nt) tile1 = max(tile0 + 1, static_cast<int>(hi - unit - kDecUnitCost));

    // the loads that need nothing but (b, h): status, held blocks, the first block ids, the queries
    const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    // pages of a warp: first, first + stride, ...
    const int stride = kOneGrid ? kWarps * p.cluster : kWarps;
    const int first = (kOneGrid ? rank : tile0) * kWarps + warp;
    // queries: the thread's columns of query g (and g + 8), as MMA operands
    const __nv_bfloat16* q_row[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x)
      q_row[x] = p.q + static_cast<long long>(b) * p.q_ld + (static_cast<long long>(h) * p.group + min(query(x), p.group - 1)) * D;
    if (kOneGrid) {                    // (all of the above while the grid before this one ends)
      grid_dependency_wait();
      n = ldg_int(p.seq_len + b);
    }
    int ids_first = 0;
    if (kOneGrid && first + lane * stride < p.max_blocks) ids_first = ldg_int(row + first + lane * stride);
    const bool fits = n >= 0 && n <= static_cast<long long>(p.max_blocks) * TV_BLOCK_SIZE;
    const int pages = fits && n > 0 ? (n - 1) / TV_BLOCK_SIZE + 1 : 0;
    const int page_end = !kOneGrid && tile1 < nt ? tile1 * kDecWarps : pages;
    int iters = page_end > first ? (page_end - first + stride - 1) / stride : 0;
    auto fetch_ids = [&](int base) { return base + lane < iters ? ldg_int(row + first + (base + lane) * stride) : 0; };
    if (!kOneGrid) ids_first = fetch_ids(0);
    const int st = *const_cast<volatile int32_t*>(p.status + b), held = min(ldg_int(p.n_blocks + b), p.max_blocks);

    uint32_t qf[NT][kSteps][2];
    float fac[NT][2];                  // score factor of queries 2t and 2t + 1
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int s = 0; s < kSteps; s += 2) {
        // 8 values: bf16 pieces t + 4 c of the row, or half a 16-value piece
        const uint4 w = ldg_stream(kHalf ? q_row[x] + (t + 4 * (s / 4)) * 16 + 4 * (s % 4) : q_row[x] + (t + 2 * s) * 8);
        qf[x][s][0] = w.x; qf[x][s][1] = w.y;
        qf[x][s + 1][0] = w.z; qf[x][s + 1][1] = w.w;
      }
    }
    int bad = n < 0 ? TV_ST_BAD_SIZE : (!fits || pages > held) ? TV_ST_BAD_BLOCK : 0;
    // another CTA may flag the request while this one's threads read its status: they decide
    // together. (The barrier also keeps the last unit's shared sums until they are read.)
    int hold = __syncthreads_or(st | bad);
    if (hold) {
      if (st == 0 && threadIdx.x == 0) atomicOr(p.status + b, bad);
      if (kOneGrid) {
        iters = 0;                     // on to the cluster's barriers with nothing, reported once
        bad = 0;
      } else {
        if (tile0 == 0 && p.by_unit && threadIdx.x == 0) p.begins[b * p.hkv + h] = DecBegin{0, 0, -1, 0};
        tile0 = nt;
        continue;
      }
    }
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      if (query(x) >= p.group) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) qf[x][s][0] = qf[x][s][1] = 0u;
      }
      if constexpr (!kHalf) {
        fac[x][0] = fac[x][1] = p.scale_log2;
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) top = max(top, max(qf[x][s][e] & 0x7fffu, (qf[x][s][e] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e <= largest magnitude < 2^(e+1); queries are held as q / 2^e
        const int e = min(max(static_cast<int>(top >> 7) - 127, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float mine_fac = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qf[x][s][u] = pack_half2(bf16_lo(qf[x][s][u]) * down, bf16_hi(qf[x][s][u]) * down);
        fac[x][0] = __shfl_sync(0xffffffffu, mine_fac, 8 * t);
        fac[x][1] = __shfl_sync(0xffffffffu, mine_fac, 8 * t + 4);
      }
    }

    float o[NT][kSteps][4];
    float m[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][s][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) { m[x][e] = ref[x][e] = kLowest; l[x][e] = 0.0f; }
    }

    // ---- pages: block ids a warp-load at a time, rows a page ahead
    int ids = 0, ids_next = 0;
    auto valid = [&](int blk) {
      if (blk < 0 || blk >= p.num_blocks) { bad = TV_ST_BAD_BLOCK; blk = 0; }
      return blk;
    };
    uint4 kf[kPages][2][kKPieces], vf[kPages][4][kVPieces];
    float ks[kPages][2], vs[kPages][2];
    auto head_row = [&](int it) {      // the page's first row of this head, as a row number of the pool
      const int blk = __shfl_sync(0xffffffffu, ids, it % 32);
      return (static_cast<size_t>(blk) * p.hkv + h) * TV_BLOCK_SIZE;
    };
    auto load_k = [&](int pg, size_t r) {
      const uint8_t* base = p.k_cache + r * kRowBytes + t * 16;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < kKPieces; ++c) kf[pg][u][c] = ldg_stream(base + (g + 8 * u) * kRowBytes + c * 64);
      if constexpr (kHalf) {
        ks[pg][0] = ldg_float(p.k_scale + r + g);
        ks[pg][1] = ldg_float(p.k_scale + r + g + 8);
      }
    };
    auto load_v = [&](int pg, size_t r) {
      const uint8_t* base = p.v_cache + r * kRowBytes;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint8_t* src = base + (2 * t + (u & 1) + (u >> 1) * 8) * kRowBytes;
        if constexpr (kRowBytes >= 128) {
#pragma unroll
          for (int c = 0; c < kVPieces; ++c) vf[pg][u][c] = ldg_stream(src + g * 16 + c * 128);
        } else {
          const uint2 w = ldg_stream8(src + g * 8);
          vf[pg][u][0] = make_uint4(w.x, w.y, 0u, 0u);
        }
      }
      if constexpr (kHalf) {
        vs[pg][0] = ldg_float(p.v_scale + r + g);
        vs[pg][1] = ldg_float(p.v_scale + r + g + 8);
      }
    };
    // the segment's keys end here; a page from here on is not loaded and masked like any tail
    const int key_end = !kOneGrid && tile1 < nt ? page_end * TV_BLOCK_SIZE : n;
    const int next_page = stride * TV_BLOCK_SIZE;              // keys from a page of the warp to its next one
    size_t rows[kPages];
    if (iters > 0) {
      ids = valid(lane < iters ? ids_first : 0);
#pragma unroll
      for (int pg = 0; pg < kPages; ++pg) {
        if (pg < iters) {
          rows[pg] = head_row(pg);
          load_k(pg, rows[pg]);
          load_v(pg, rows[pg]);
        } else {                       // (masked; zeroed so that nothing is read that was never set)
#pragma unroll
          for (int c = 0; c < kKPieces; ++c) kf[pg][0][c] = kf[pg][1][c] = make_uint4(0u, 0u, 0u, 0u);
          ks[pg][0] = ks[pg][1] = vs[pg][0] = vs[pg][1] = 0.0f;
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < kVPieces; ++c) vf[pg][u][c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      ids_next = fetch_ids(32);
    }
    for (int it = 0; it < iters; it += kPages) {
      const int left = key_end - (first + it * stride) * TV_BLOCK_SIZE; // keys from the first page's first on
      const bool tail = left < (kPages - 1) * next_page + TV_BLOCK_SIZE;
      // scores of 16 keys a page: thread holds keys g, g + 8 of queries 2t, 2t + 1
      float s[kPages][NT][4], k0[kPages], k1[kPages];
#pragma unroll
      for (int pg = 0; pg < kPages; ++pg) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[pg][x][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < kKPieces; ++c) {
          const uint4 &ka = kf[pg][0][c], &kb = kf[pg][1][c];
          const uint32_t a[4] = {ka.x, ka.y, ka.z, ka.w};
          const uint32_t e[4] = {kb.x, kb.y, kb.z, kb.w};
          if constexpr (kHalf) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t a0, a1, a2, a3;
              codes_to_half<kFmt>(a[j], a0, a2);
              codes_to_half<kFmt>(e[j], a1, a3);
#pragma unroll
              for (int x = 0; x < NT; ++x) mma16816<true>(s[pg][x], a0, a1, a2, a3, qf[x][4 * c + j][0], qf[x][4 * c + j][1]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int x = 0; x < NT; ++x)
                mma16816<false>(s[pg][x], a[2 * j], e[2 * j], a[2 * j + 1], e[2 * j + 1], qf[x][2 * c + j][0], qf[x][2 * c + j][1]);
          }
        }
        k0[pg] = kHalf ? ks[pg][0] : 1.0f;
        k1[pg] = kHalf ? ks[pg][1] : 1.0f;
      }
      const int next = it + kPages;
      if (next < iters) {
        if (next % 32 == 0) {
          ids = valid(ids_next);
          ids_next = fetch_ids(next + 32);
        }
#pragma unroll
        for (int pg = 0; pg < kPages; ++pg) {
          if (next + pg < iters) {
            rows[pg] = head_row(next + pg);
            load_k(pg, rows[pg]);
          }
        }
      }
      bool live[kPages][2];
      float lv[kPages][2];
      bool over = false;
#pragma unroll
      for (int pg = 0; pg < kPages; ++pg) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          live[pg][u] = !tail || pg * next_page + g + 8 * u < left;
          lv[pg][u] = kHalf ? __log2f(vs[pg][u]) : 0.0f;
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = kHalf ? fac[x][e & 1] * (e < 2 ? k0[pg] : k1[pg]) : fac[x][e & 1];
            s[pg][x][e] = live[pg][e / 2] ? s[pg][x][e] * f : -INFINITY;
            over |= s[pg][x][e] > m[x][e & 1] + 8.0f;
            if (kHalf) over |= s[pg][x][e] + lv[pg][e / 2] > ref[x][e & 1] + 8.0f + kRefBelow;
          }
        }
      }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = kLowest, c = kLowest;
#pragma unroll
            for (int pg = 0; pg < kPages; ++pg) {
              a = fmaxf(a, fmaxf(s[pg][x][e], s[pg][x][e + 2]));
              if (kHalf) c = fmaxf(c, fmaxf(s[pg][x][e] + (live[pg][0] ? lv[pg][0] : 0.0f), s[pg][x][e + 2] + (live[pg][1] ? lv[pg][1] : 0.0f)));
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
              if (kHalf) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, d));
            }
            a = fmaxf(a, m[x][e]);
            l[x][e] *= fast_exp2(m[x][e] - a);
            m[x][e] = a;
            c = kHalf ? fmaxf(c - kRefBelow, ref[x][e]) : a;
            const float down = fast_exp2(ref[x][e] - c);
            ref[x][e] = c;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) { o[x][i][e] *= down; o[x][i][e + 2] *= down; }
          }
        }
      }
#pragma unroll
      for (int pg = 0; pg < kPages; ++pg) {
        // weights, transposed into the MMA's B operand: query g, keys 2t, 2t + 1 (and + 8), in the
        // parts that DecTraits::kTwice tells of
        uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = fast_exp2(s[pg][x][e] - m[x][e & 1]);
            l[x][e & 1] += w[e];
            if (kHalf) {
              w[e] = fast_exp2(s[pg][x][e] + lv[pg][e / 2] - ref[x][e & 1]);
              if (tail && !live[pg][e / 2]) w[e] = 0.0f;
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t hi, rest;
            if constexpr (kHalf) {
              hi = pack_half2(w[2 * u], w[2 * u + 1]);
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              rest = pack_half2(w[2 * u] - h.x, w[2 * u + 1] - h.y);
            } else {
              hi = __byte_perm(__float_as_uint(w[2 * u]), __float_as_uint(w[2 * u + 1]), 0x7632);
              rest = pack_bf16x2(weight_rest(w[2 * u], bf16_lo(hi)), weight_rest(w[2 * u + 1], bf16_hi(hi)));
            }
            pf[x][u] = transpose8x8(kTwice && t >= 2 ? rest : hi);
            if (!kHalf && !kTwice) pl[x][u] = transpose8x8(rest);
          }
        }
        if (tail) {                    // rows past the end may hold anything, NaN among it
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (pg * next_page + 2 * t + (u & 1) + (u >> 1) * 8 < left) continue;
#pragma unroll
            for (int c = 0; c < kVPieces; ++c) vf[pg][u][c] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int c = 0; c < kVPieces; ++c) {
          const uint4 (&v)[4][kVPieces] = vf[pg];
          const uint32_t v0[4] = {v[0][c].x, v[0][c].y, v[0][c].z, v[0][c].w};
          const uint32_t v1[4] = {v[1][c].x, v[1][c].y, v[1][c].z, v[1][c].w};
          const uint32_t v2[4] = {v[2][c].x, v[2][c].y, v[2][c].z, v[2][c].w};
          const uint32_t v3[4] = {v[3][c].x, v[3][c].y, v[3][c].z, v[3][c].w};
          constexpr int kWords = kRowBytes >= 128 ? 4 : 2;
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            if constexpr (kHalf) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {      // two columns of two rows, by bytes
                const uint32_t sel = i ? 0x7362 : 0x5140;
                uint32_t a0, a1, a2, a3;
                codes_to_half<kFmt>(__byte_perm(v0[j], v1[j], sel), a0, a1);
                codes_to_half<kFmt>(__byte_perm(v2[j], v3[j], sel), a2, a3);
#pragma unroll
                for (int x = 0; x < NT; ++x) mma16816<true>(o[x][2 * j + i], a0, a1, a2, a3, pf[x][0], pf[x][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632);
              const uint32_t a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                mma16816<false>(o[x][4 * c + j], a0, a1, a2, a3, pf[x][0], pf[x][1]);
                if (!kTwice) mma16816<false>(o[x][4 * c + j], a0, a1, a2, a3, pl[x][0], pl[x][1]);
              }
            }
          }
        }
        if (next + pg < iters) load_v(pg, rows[pg]);
      }
    }

    // ---- join the warps
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], d);
        const int qi = 8 * x + 2 * t + e;
        if (g == 0) s_stat[warp][qi] = make_float4(m[x][e], ref[x][e], l[x][e], 0.0f);
        float* dst = s_o + (static_cast<size_t>(warp) * 8 * NT + qi) * kRowPad;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          // the column of tile i's row g (and the next one in its row g + 8)
          const int d = kRowBytes == 256 ? 8 * g + 64 * (i / 4) + 2 * (i % 4) : kRowBytes == 128 && kHalf ? 16 * g + 2 * i : 8 * g + 2 * i;
          *reinterpret_cast<float2*>(dst + d) = make_float2(o[x][i][e], o[x][i][e + 2]);
        }
      }
    const bool any_bad = __syncthreads_or(bad | hold);
    if (bad) atomicOr(p.status + b, bad);
    const bool whole = kOneGrid ? p.cluster == 1 : tile0 == 0 && tile1 == nt;
    // where the CTA's sums go: the output, its cluster's sight, or a slot of the workspace
    float* const s_part = s_o + kWarps * 8 * NT * kRowPad;     // [group][D]
    float* const slot = kOneGrid ? s_part : p.partials + (static_cast<size_t>(cta) * 2 + (tile0 == 0 ? 1 : 0)) * dec_slot_floats(p.group, D);
    if (!any_bad || !whole) {
      for (int i = threadIdx.x; i < p.group * (D / 2); i += kThreads) {
        const int qi = i / (D / 2), d = i % (D / 2) * 2;
        float mm = kLowest, mr = kLowest, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          mm = fmaxf(mm, s_stat[w][qi].x);
          mr = fmaxf(mr, s_stat[w][qi].y);
        }
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 s4 = s_stat[w][qi];
          const float f = fast_exp2(s4.y - mr);
          const float* sums = s_o + (static_cast<size_t>(w) * 8 * NT + qi) * kRowPad + d;
          float2 v = *reinterpret_cast<const float2*>(sums);
          if (kTwice) {
            const float2 rest = *reinterpret_cast<const float2*>(sums + 4 * kRowPad);
            v.x += rest.x;
            v.y += rest.y;
          }
          acc.x += v.x * f;
          acc.y += v.y * f;
          ll += s4.z * fast_exp2(s4.x - mm);
        }
        if (whole) {
          dec_store<D>(p, b, h, qi, d, n, acc, mm, mr, ll);
        } else {
          *reinterpret_cast<float2*>(slot + static_cast<size_t>(qi) * D + d) = acc;
          if (d == 0) {
            const float4 stat = make_float4(mm, mr, ll, any_bad ? 1.0f : 0.0f);
            if (kOneGrid) s_joined[qi] = stat;
            else *reinterpret_cast<float4*>(slot + static_cast<size_t>(p.group) * D + 4 * qi) = stat;
          }
        }
      }
    }
    if constexpr (kOneGrid) {
      if (p.cluster > 1) {
        // the CTAs of the cluster share the output's columns and read each other's sums
        __syncwarp();
        cluster_sync_all();
        for (int i = rank * kThreads + threadIdx.x; i < p.group * (D / 2); i += kThreads * p.cluster) {
          const int qi = i / (D / 2), d = i % (D / 2) * 2;
          float2 v[kDecMaxCluster], mM[kDecMaxCluster], lf[kDecMaxCluster];
#pragma unroll
          for (int r = 0; r < kDecMaxCluster; ++r) {
            if (r >= p.cluster) break;
            v[r] = as_float2(ld_cluster_u64(s_part + qi * D + d, r));
            mM[r] = as_float2(ld_cluster_u64(&s_joined[qi].x, r));
            lf[r] = as_float2(ld_cluster_u64(&s_joined[qi].z, r));
          }
          float mm = kLowest, mr = kLowest, ll = 0.0f, faulty = 0.0f;
          float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int r = 0; r < kDecMaxCluster; ++r) {
            if (r >= p.cluster) break;
            mm = fmaxf(mm, mM[r].x);
            mr = fmaxf(mr, mM[r].y);
            faulty += lf[r].y;
          }
#pragma unroll
          for (int r = 0; r < kDecMaxCluster; ++r) {
            if (r >= p.cluster) break;
            const float f = fast_exp2(mM[r].y - mr);
            acc.x += v[r].x * f;
            acc.y += v[r].y * f;
            ll += lf[r].x * fast_exp2(mM[r].x - mm);
          }
          if (faulty == 0.0f) dec_store<D>(p, b, h, qi, d, n, acc, mm, mr, ll);
        }
        __syncwarp();
        cluster_sync_all();            // a CTA's shared memory outlives its readers
      }
      return;
    }
    if (tile0 > 0) {
      mid = b * p.hkv + h;
    } else {
      DecBegin d = {b * p.hkv + h, cta, -1, 0};
      if (!whole && threadIdx.x == 0) {
        d.last = s_share.owner(unit + kDecUnitCost + nt - 1);  // of the unit's last tile
        begun = d;
      }
      if (p.by_unit && threadIdx.x == 0) p.begins[d.unit] = d;
    }
    if (tile1 < nt) break;
    tile0 = nt;
  }
  if (!kOneGrid && threadIdx.x == 0) {
    p.mids[cta] = mid;
    if (!p.by_unit) p.begins[cta] = begun;
  }
}

// Join the partials of unit blockIdx.x. A warp takes a query head, or one of
// p.parts interleaved parts of its partials where a unit is cut into many. A
// lane looks up one of up to 32 partials (does that CTA's slot hold this unit,
// its references and sum), while the first sums are already on their way.
template <int D>
__global__ void __launch_bounds__(32 * kMergeMaxParts) decode_merge_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kVec = D / 32;         // columns of a lane
  using Vec = typename std::conditional<kVec == 4, float4, float2>::type;
  __shared__ float s_acc[kMergeMaxParts][D];
  __shared__ float4 s_stat[kMergeMaxParts];
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int part = warp % p.parts, qi = blockIdx.y * (warps / p.parts) + warp / p.parts;
  grid_dependency_wait();
  const DecBegin task = p.begins[blockIdx.x];
  if (task.last < 0) return;
  const int b = task.unit / p.hkv, h = task.unit - b * p.hkv;
  const bool live = qi < p.group;
  float acc[kVec], mm = kLowest, mr = kLowest, ll = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
  const int st = p.status[b], count = task.last - task.first + 1;
  const int mine = live && part < count ? (count - part - 1) / p.parts + 1 : 0;     // this warp's partials
  auto slot_of = [&](int i) {
    const int k = part + i * p.parts;
    return p.partials + (static_cast<size_t>(task.first + k) * 2 + (k == 0 ? 1 : 0)) * dec_slot_floats(p.group, D);
  };
  for (int base = 0; base < mine; base += 32) {
    const int here = min(32, mine - base);
    Vec v[kMergeBatch];
    auto load = [&](int from) {
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u)
        v[u] = *reinterpret_cast<const Vec*>(slot_of(base + min(from + u, here - 1)) + static_cast<size_t>(qi) * D + kVec * lane);
    };
    load(0);
    float4 s = make_float4(kLowest, kLowest, 0.0f, 0.0f);
    bool has = false;
    if (lane < here) {
      const int k = part + (base + lane) * p.parts;
      has = k == 0 || p.mids[task.first + k] == task.unit;
      s = *reinterpret_cast<const float4*>(slot_of(base + lane) + static_cast<size_t>(p.group) * D + 4 * qi);
    }
    float nm = has ? fmaxf(mm, s.x) : mm, nr = has ? fmaxf(mr, s.y) : mr;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
      nr = fmaxf(nr, __shfl_xor_sync(0xffffffffu, nr, d));
    }
    float sum = has ? s.z * fast_exp2(s.x - nm) : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    ll = ll * fast_exp2(mm - nm) + sum;
    const float down = fast_exp2(mr - nr);
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] *= down;
    mm = nm;
    mr = nr;
    const float f = fast_exp2(s.y - nr);
    const unsigned hold = __ballot_sync(0xffffffffu, has);
    for (int from = 0; from < here; from += kMergeBatch) {
      if (from > 0) load(from);
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        const float w = __shfl_sync(0xffffffffu, f, (from + u) % 32);
        if (from + u < here && (hold >> (from + u) & 1u)) {
          const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] += x[i] * w;
        }
      }
    }
  }
  if (p.parts > 1) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) s_acc[warp][kVec * lane + i] = acc[i];
    if (lane == 0) s_stat[warp] = make_float4(mm, mr, ll, 0.0f);
    __syncthreads();
    if (part != 0) return;
    float nm = mm, nr = mr;
    for (int w = 1; w < p.parts; ++w) {
      nm = fmaxf(nm, s_stat[warp + w].x);
      nr = fmaxf(nr, s_stat[warp + w].y);
    }
    ll = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] = 0.0f;
    for (int w = 0; w < p.parts; ++w) {
      const float4 s4 = s_stat[warp + w];
      const float f = fast_exp2(s4.y - nr);
      ll += s4.z * fast_exp2(s4.x - nm);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] += s_acc[warp + w][kVec * lane + i] * f;
    }
    mm = nm;
    mr = nr;
  }
  if (!live || st != 0) return;
  const size_t at = static_cast<size_t>(b) * p.hq + static_cast<size_t>(h) * p.group + qi;
  const float f = fast_exp2(mr - mm) / ll;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + at * D + kVec * lane);
#pragma unroll
  for (int i = 0; i < kVec; i += 2) out[i / 2] = pack_bf16x2(acc[i] * f, acc[i + 1] * f);
  if (p.lse != nullptr && lane == 0) p.lse[at] = (mm + log2f(ll)) * 0.69314718055994531f;
}

template <int kFmt, int D, int kQ, int kWarps>
static int launch_decode_one(const DecodeParams& p, int dev, cudaStream_t stream) {
  constexpr size_t smem = sizeof(float) * 8 * DecTraits<kFmt, D, kQ>::NT * (kWarps * (D + 4) + D);
  static SmemLimit smem_limit;
  auto* kernel = decode_kernel<kFmt, D, kQ, true, kWarps>;
  if (!ensure_smem(kernel, smem, smem_limit, dev)) return TV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cluster, p.hkv, p.batch);             // (no divisions by variables in the kernel)
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

template <int kFmt, int D, int kQ>
static int launch_decode(DecodeParams p, int sms, int dev, cudaStream_t stream) {
  using Tr = DecTraits<kFmt, D, kQ>;
  constexpr size_t sums = sizeof(float) * kDecWarps * 8 * Tr::NT * (D + 4);
  const int grid = sms * Tr::kPerSm, units = p.batch * p.hkv;
  const long long all_warps = static_cast<long long>(grid) * kDecWarps;
  auto fits = [&](long long unit_warps, long long most) { return units * unit_warps <= most; };
  // The warps of a unit in the one-launch form: doubled while the table's
  // longest request leaves each enough pages and all fit at once (powers of
  // two: clusters of 5 or 7 CTAs start late, 28 -> 35 us). One CTA of eight
  // warps rather than two of four saves the cluster (296 units, 16 pages, int8:
  // 6.7 / 8.2 us) and reaches twice the warps (12 units, 298 pages: 7.8 / 10.2),
  // but clusters of four-warp CTAs are the lighter ones in between (128 units,
  // 256 pages: 27.4 / 28.2). Past a few warps an SM another doubling adds loads in
  // flight but no SM, and needs more pages to pay for its cluster (96 units, 29
  // pages: 5.0 with 8 warps, 5.7 with 16; 15 units, 30 pages: 5.7 and 5.0).
  int unit_warps = kDecWarps;
  while (unit_warps < kDecMaxCluster * Tr::kMaxWarps) {
    const int pages = unit_warps < Tr::kMaxWarps ? Tr::kPages : fits(2 * unit_warps, kFewWarps * sms) ? kClusterPagesFew : kClusterPages;
    if (unit_warps * pages >= p.max_blocks || !fits(2 * unit_warps, all_warps)) break;
    unit_warps *= 2;
  }
  const bool wide = unit_warps == Tr::kMaxWarps || unit_warps == kDecMaxCluster * Tr::kMaxWarps;
  p.cluster = unit_warps / (wide ? Tr::kMaxWarps : kDecWarps);
  // One launch saves the joining grid and a round trip, but its CTAs are as
  // uneven as the requests and may leave SMs without work. So it is taken up to
  // kOneGridPages pages a warp, kOneGridExcess of them above an even share. One
  // launch against two, us: 35 heads, 287 keys 4.3 / 8.2; 8 x 512..2048 keys,
  // bf16 14.6 / 15.8; 32 units, 7683 keys, int8 11.0 / 14.2; 64 x 1000 keys, int8
  // 28.4 / 34.9; it loses with 32 pages a warp (128 x 100..2048 keys, e4m3 47.8 /
  // 41.7) or an excess of 5.1 (16 units, 9002 keys, int8 17.2 / 15.2).
  const long long by_unit = static_cast<long long>(units) * unit_warps;
  if (p.max_blocks <= unit_warps * kOneGridPages &&
      p.max_blocks * (all_warps - by_unit) <= kOneGridExcess * unit_warps * all_warps) {
    if constexpr (Tr::kMaxWarps > kDecWarps) {
      if (wide) return launch_decode_one<kFmt, D, kQ, Tr::kMaxWarps>(p, dev, stream);
    }
    return launch_decode_one<kFmt, D, kQ, kDecWarps>(p, dev, stream);
  }
  static SmemLimit smem_limit;
  auto* kernel = decode_kernel<kFmt, D, kQ, false, kDecWarps>;
  if (!ensure_smem(kernel, sums, smem_limit, dev)) return TV_ERR_CUDA;
  p.by_unit = units <= grid ? 1 : 0;
  p.parts = 1;
  if (launch_pdl(kernel, dim3(grid), dim3(kDecThreads), sums, stream, p) != cudaSuccess) return TV_ERR_CUDA;
  // a unit's partials: about grid / units and both ends; eight of them a warp
  const int partials = grid / units + 2;
  while (p.parts < kMergeMaxParts && p.parts * kMergeBatch < partials) p.parts *= 2;
  const int join_warps = p.parts > kMergeWarps ? p.parts : kMergeWarps, heads = join_warps / p.parts;
  if (launch_pdl(decode_merge_kernel<D>, dim3(p.by_unit ? units : grid, (p.group + heads - 1) / heads), dim3(32 * join_warps), 0, stream, p) != cudaSuccess)
    return TV_ERR_CUDA;
  return TV_OK;
}

template <int kFmt>
static int launch_decode_fmt(const DecodeParams& p, int d, int sms, int dev, cudaStream_t stream) {
  if (d == 64) {
    if (p.group <= 4) return launch_decode<kFmt, 64, 4>(p, sms, dev, stream);
    return p.group <= 8 ? launch_decode<kFmt, 64, 8>(p, sms, dev, stream) : launch_decode<kFmt, 64, 16>(p, sms, dev, stream);
  }
  if (p.group <= 4) return launch_decode<kFmt, 128, 4>(p, sms, dev, stream);
  return p.group <= 8 ? launch_decode<kFmt, 128, 8>(p, sms, dev, stream) : launch_decode<kFmt, 128, 16>(p, sms, dev, stream);
}

static size_t dec_task_bytes(int ctas) { return ((sizeof(DecBegin) + sizeof(int)) * ctas + 255) / 256 * 256; }

}  // namespace tv

extern "C" int tv_decode_workspace_bytes(const tv_geom* geom, int32_t batch, size_t* bytes) {
  int rc = tv::check_geom(geom);
  if (rc != TV_OK) return rc;
  if (bytes == nullptr) return TV_ERR_NULL_POINTER;
  if (batch < 0 || batch > tv::kKvMaxBatch) return TV_ERR_BAD_SIZE;
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  const int ctas = sms * tv::kDecMaxPerSm;
  *bytes = tv::dec_task_bytes(ctas) +
           sizeof(float) * 2 * ctas * tv::dec_slot_floats(geom->num_q_heads / geom->num_kv_heads, geom->head_dim);
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
  if ((kv_format != TV_KV_BF16 && kv_format != TV_KV_E4M3 && kv_format != TV_KV_INT8) || geom->num_kv_heads > tv::kDecMaxHeads)
    return TV_ERR_BAD_GEOMETRY;
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
      (scaled && (!tv::aligned(k_scale, 4) || !tv::aligned(v_scale, 4))))
    return TV_ERR_MISALIGNED;
  size_t need = 0;
  rc = tv_decode_workspace_bytes(geom, batch, &need);
  if (rc != TV_OK) return rc;
  if (workspace_bytes < need) return TV_ERR_WORKSPACE;
  const int dev = tv::current_device();
  if (dev < 0) return TV_ERR_CUDA;
  const int sms = tv::device_sm_count(dev);
  if (sms <= 0) return TV_ERR_CUDA;
  tv::DecodeParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_ld = q_ld;
  p.seq_len = seq_len; p.block_table = block_table; p.n_blocks = n_blocks;
  p.k_cache = static_cast<const uint8_t*>(k_cache); p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale; p.v_scale = v_scale;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse; p.status = status;
  p.begins = static_cast<tv::DecBegin*>(workspace);
  p.mids = reinterpret_cast<int*>(p.begins + sms * tv::kDecMaxPerSm);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + tv::dec_task_bytes(sms * tv::kDecMaxPerSm));
  p.batch = batch; p.hq = geom->num_q_heads; p.hkv = geom->num_kv_heads;
  p.group = geom->num_q_heads / geom->num_kv_heads;
  p.max_blocks = max_blocks_per_req; p.num_blocks = num_blocks;
  const float scale = geom->softmax_scale > 0.0f ? geom->softmax_scale : 1.0f / sqrtf(static_cast<float>(geom->head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t s = tv::as_stream(stream);
  if (kv_format == TV_KV_BF16) return tv::launch_decode_fmt<TV_KV_BF16>(p, geom->head_dim, sms, dev, s);
  if (kv_format == TV_KV_E4M3) return tv::launch_decode_fmt<TV_KV_E4M3>(p, geom->head_dim, sms, dev, s);
  return tv::launch_decode_fmt<TV_KV_INT8>(p, geom->head_dim, sms, dev, s);
}
