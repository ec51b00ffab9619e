// Token sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// The answer is a whole number decided by borders of running sums, so the sums are exact: each weight
// w_i = exp((x_i - m) / T) is a 64-bit fixed-point number (`bits` fraction bits) evaluated to
// about 31 significant bits, and integer sums do not depend on their order.  Every threshold is then
// an integer comparison: a token is in the nucleus iff the weight before it is below
// ceil(top_p * Z), and the sampled one is the first whose running sum exceeds floor(u * Z_kept).
//
// A row is one cluster of C CTAs; each CTA keeps its slice of the row in shared memory (fp32), so
// the logits are read from memory once and every later pass runs out of shared memory.  One
// pass over the slice evaluates every weight: it gives the whole weight, the weight kept by
// min-p for each warp's stretch of the slice, and a histogram over the span of logits, of counts for
// top-k or of weights for top-p.  Without top-k and top-p the warp in which the running sum
// passes its target is then known, and it alone walks its stretch again.  With them, the histogram
// gives the bin in which the running measure, from the largest logit down, crosses its target; the
// tokens down to that bin, if they are few, go to one CTA as a list, which settles top-k, top-p, min-p
// and the choice by sorting them (bitonic, one token per thread).  A longer list stays where it is: the
// bin's span is divided by further histograms until its logits are few or equal, and one more pass sums
// what is kept and counts the ties, which are taken in index order.
//
// What bounds it is instructions, not the logits' bytes: the 31-bit weights cost about 60 of the 90
// instructions per 32 logits without filters (120 with all of them), issued at 56 % of the peak,
// the rest being waits for their results and at the barriers between the passes.  256 rows of 131072
// fp32 logits: 140 us at a temperature alone, 207-222 us with every filter (20 us to read them once at
// the copy rate); 64 rows of 50001 bf16 logits with nuclei of thousands 52 us, at a temperature alone 21;
// 16 rows of 32000 11 us (as a node of a graph).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <cstring>

#include "pg_internal.h"

namespace pg {

namespace cg = cooperative_groups;

namespace {

// Small CTAs, several to an SM: a row's passes are separated by barriers over its CTA and its cluster, and
// other CTAs' warps fill those waits.  256 rows of 131072 logits with every filter: 256 threads 233 us,
// 512 with the same slices 261, 1024 with twice the slice 274.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kBinBits = 8;
constexpr int kMaxCluster = 8;
constexpr int kList = 256;      // longest list of candidates settled by one CTA
typedef unsigned long long u64;

// 2^(j / 64) in 1.31 fixed point, and times 2^31 in fp32.
struct Exp2Table {
  uint2 e[64];
};

// ---------------------------------------------------------------------------------- logits --
// NaN counts as -inf and -0 as 0, so that comparisons order the logits.
__device__ __forceinline__ float canonical(float x) { return x != x ? -INFINITY : x + 0.f; }

// Order-preserving unsigned image of a canonical logit.
__device__ __forceinline__ uint32_t to_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

// --------------------------------------------------------------------------------- weights --
// w = exp((x - m) / T) = 2^t, t = (x - m) log2(e) / T, as a fixed-point number with `bits` fraction
// bits (31 <= bits <= 45).  x - m and the product are carried as unevaluated sums of two floats;
// 2^t = 2^n 2^(j/64) e^(r ln 2), |r| <= 2^-7 + rounding, the last factor by its Taylor series.  The
// significand (1.31 bits, relative error below 2^-31) is scaled by 2^(n + bits - 31) and rounded.
struct Weigher {
  float m, ch, cl;   // the row's maximum; log2(e) / T as ch + cl
  float cut;         // t at or below it: weight 0
  int bits;
  bool inf;          // the maximum is +inf: its weight is 1, any other 0
  const uint2* tab;
  // log2(e) / T as a sum of two floats: the quotient, and its remainder over T again.
  __device__ __forceinline__ void init(float max, float temp, int bits_, const uint2* tab_) {
    constexpr float kHi = 1.44269502162933349609375f;   // log2(e) rounded to fp32 ...
    constexpr float kLo = 1.9259629911266174681e-8f;    // ... and the rest
    m = max;
    // an infinite T: every t is 0 (-inf x 0 is NaN, which is no weight)
    ch = temp < INFINITY ? fminf(kHi / temp, 3.4e38f) : 0.f;
    cl = ch > 0.f && ch < 3.4e38f ? (fmaf(-ch, temp, kHi) + kLo) / temp : 0.f;
    bits = bits_;
    cut = -(float)(bits + 1);
    inf = max == INFINITY;
    tab = tab_;
  }
  // t as th + tl
  __device__ __forceinline__ float exponent(float x, float& tl) const {
    const float dh = x - m, bb = dh - x;
    const float de = (x - (dh - bb)) - (m + bb);
    const float th = dh * ch;
    tl = fmaf(dh, ch, -th) + fmaf(dh, cl, de * ch);
    return th;
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    if (inf) return x == INFINITY ? 1ull << bits : 0ull;
    float tl;
    const float th = exponent(x, tl);
    if (!(th > cut)) return 0;
    const float kf = fmaf(th, 64.f, 12582912.f);     // 1.5 x 2^23: rounds th x 64 to a whole number
    const int k = __float_as_int(kf) - 0x4b400000;
    const float r = fmaf(kf - 12582912.f, -1.f / 64.f, th) + tl;
    // e^(r ln 2) - 1 by its Taylor series: (ln 2)^i / i!
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 0.009618129107628477f, 0.05550410866482158f),
                                     0.2402265069591007f), 0.6931471805599453f);
    const uint2 e = tab[k & 63];
    const uint32_t sig = e.x + (uint32_t)__float2int_rn(__uint_as_float(e.y) * p);
    // sig x 2^sh, -32 <= sh <= 14: a product, of which negative sh takes the upper word, rounded
    const int sh = (k >> 6) + bits - 31;
    const u64 wide = (u64)sig * (1u << (sh & 31));
    return sh >= 0 ? wide : (wide + 0x80000000ull) >> 32;
  }
  // ln of the weight's share of the whole weight Z: ln 2 (t - log2 Z), with Z = 2^e 2^(j/64) (1 + q),
  // 0 <= q < 0.011.  q comes from an integer product with the table's 2^(-j/64) (error 2^-32), ln(1 + q)
  // from its series (2^-23 q), and t - e - j/64 and its product with ln 2 are sums of two floats.
  __device__ __forceinline__ float log_share(float x, u64 Z) const {
    float th = 0.f, tl = 0.f;
    if (x != m) th = exponent(x, tl);
    const int e = 63 - __clzll((long long)Z);
    const u64 z = Z << (63 - e);                                      // 1.63 bits, in [1, 2)
    const float f = __uint_as_float((uint32_t)(z >> 40 & 0x7fffffu) | 0x3f800000u);
    int j = 0;                                                        // the largest j with 2^(j/64) <= f
#pragma unroll
    for (int b = 32; b > 0; b >>= 1)
      if (__uint_as_float(tab[j + b].y) * 0x1p-31f <= f) j += b;
    const u64 scaled = j == 0 ? z : __umul64hi(z, (u64)tab[64 - j].x << 32);
    const float q = (float)((long long)(scaled - (1ull << 63))) * 0x1p-63f;
    const float l1p = q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 0.2f, -0.25f), 0.333333343f), -0.5f), 1.f);
    const float c = (float)(e - bits) + (float)j * (1.f / 64.f);      // exact
    const float a = th - c, ab = a - th;
    const float al = (th - (a - ab)) - (c + ab) + tl;
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.9046543e-9f;
    const float hi = a * kLn2Hi;
    const float lo = fmaf(a, kLn2Hi, -hi) + fmaf(a, kLn2Lo, al * kLn2Hi) - l1p;
    return hi + lo;
  }
};

// floor(a * f) for f = frac / 2^64.
__device__ __forceinline__ u64 mul_frac(u64 a, u64 frac) { return __umul64hi(a, frac); }

// x 2^n for x in (0, 1), 0 <= n <= 64, rounded down or up to a whole number (below 2^64).
__device__ __forceinline__ u64 scaled(float x, int n, bool up) {
  const uint32_t b = __float_as_uint(x);
  const int ex = max((int)(b >> 23), 1);
  const u64 sig = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);     // x = sig 2^(ex - 150)
  const int sh = ex - 150 + n;
  if (sh >= 0) return sig << sh;
  if (sh <= -24) return up && sig ? 1 : 0;
  return (sig + (up ? (1ull << -sh) - 1 : 0)) >> -sh;
}

// ------------------------------------------------------------------------- shared memory ----
struct Sums {
  u64 a, b;
};

struct Smem {
  uint2 tab[64];
  uint32_t lo[kBins], hi[kBins];   // counts (lo), or weights as two words
  u64 warp_sum[2][kWarps];
  u64 scan[kWarps];
  Sums slot[2];           // this CTA's contribution to a cluster sum (two, used in turn)
  uint32_t slot_lo[2], slot_hi[2];
  u64 found_above;        // the crossing bin: the measure of its predecessors, its own
  u64 found_in;
  int found_bin;
  int found_idx;
  int list_n;             // this CTA's candidates
  float list_x[kList];
  int list_idx[kList];
  u64 sort[kList];
};

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

// kFits: the whole slice is in shared memory, with up to three entries of -inf in front (so that
// 16 bytes of it are 16 aligned bytes of the row) and behind (so that its length is a multiple of 4).
template <typename T, bool kFits>
struct Row {
  const T* x;
  float* kept;        // shared memory, the first `cap` of the slice
  int begin, n, cap;  // slice [begin, begin + n) of the row
  __device__ __forceinline__ float at(int i) const {
    return kFits || i < cap ? kept[i] : canonical(load_logit(x + begin + i));
  }
  // f(i, x) for every entry of [w0, w1) (w0 a multiple of 4), the lanes of a warp side by side.
  template <typename F>
  __device__ __forceinline__ void each(int w0, int w1, F&& f) const {
    const int lane = threadIdx.x & 31;
    if (kFits) {
#pragma unroll 1
      for (int i = w0 + 4 * lane; i < w1; i += 128) {
        const float4 v = *reinterpret_cast<const float4*>(kept + i);
        f(i, v.x);
        f(i + 1, v.y);
        f(i + 2, v.z);
        f(i + 3, v.w);
      }
    } else {
#pragma unroll 2
      for (int i = w0 + lane; i < w1; i += 32) f(i, at(i));
    }
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the 8 lanes (or 16) that hold one value per CTA (per warp).
template <int kLanes>
__device__ __forceinline__ u64 lanes_sum(u64 v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the cluster of per-lane values, and over the CTAs of lower rank; every thread gets them.
// `turn` alternates between the two slots, so a CTA may write its next contribution while another
// still reads the previous one.
__device__ __forceinline__ Sums cluster_sums(Sums v, Smem& sm, int& turn, int C, int rank,
                                             Sums& before) {
  static_assert(kWarps == 8 && kMaxCluster == 8, "lanes that hold one value per warp, per CTA");
  const int lane = threadIdx.x & 31;
  v.a = warp_sum(v.a);
  v.b = warp_sum(v.b);
  __syncthreads();
  if (lane == 0) {
    sm.warp_sum[0][threadIdx.x >> 5] = v.a;
    sm.warp_sum[1][threadIdx.x >> 5] = v.b;
  }
  __syncthreads();
  Sums s{lanes_sum<8>(sm.warp_sum[0][lane & 7]), lanes_sum<8>(sm.warp_sum[1][lane & 7])};
  before = Sums{0, 0};
  if (C == 1) return s;
  cg::cluster_group cl = cg::this_cluster();
  if (threadIdx.x == 0) sm.slot[turn] = s;
  cl.sync();
  // lane c (and c + 8, ...) reads CTA c's contribution
  const int c = lane & 7;
  Sums o{0, 0};
  if (c < C) o = *cl.map_shared_rank(&sm.slot[turn], c);
  turn ^= 1;
  before = Sums{lanes_sum<8>(c < rank ? o.a : 0), lanes_sum<8>(c < rank ? o.b : 0)};
  return Sums{lanes_sum<8>(o.a), lanes_sum<8>(o.b)};
}
__device__ __forceinline__ u64 cluster_sum(u64 v, Smem& sm, int& turn, int C, int rank) {
  Sums before;
  return cluster_sums(Sums{v, 0}, sm, turn, C, rank, before).a;
}

// The largest and smallest key of the cluster's slices among those passed in; `turn` as for the sums.
__device__ __forceinline__ void cluster_minmax(uint32_t& lo, uint32_t& hi, Smem& sm, int& turn, int C) {
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if (threadIdx.x == 0) {
    sm.slot_lo[turn] = 0xffffffffu;
    sm.slot_hi[turn] = 0;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    atomicMin(&sm.slot_lo[turn], lo);
    atomicMax(&sm.slot_hi[turn], hi);
  }
  if (C == 1) {
    __syncthreads();
    lo = sm.slot_lo[turn];
    hi = sm.slot_hi[turn];
  } else {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int c = min((int)(threadIdx.x & 31), C - 1);
    lo = __reduce_min_sync(0xffffffffu, *cl.map_shared_rank(&sm.slot_lo[turn], c));
    hi = __reduce_max_sync(0xffffffffu, *cl.map_shared_rank(&sm.slot_hi[turn], c));
  }
  turn ^= 1;
}

// Bin of a logit in a histogram over [lo, hi]: linear in the logit, or in its key; 0 for the largest.
struct Bins {
  float lo, hi, scale;
  bool linear;
  int shift;
  __device__ __forceinline__ Bins(float lo_, float hi_, bool want_linear) : lo(lo_), hi(hi_) {
    const float span = hi - lo;
    scale = (float)kBins / span;
    // a span that vanishes, overflows or is too small for its reciprocal goes by key
    linear = want_linear && span > 0.f && span < INFINITY && scale < INFINITY && scale > 0.f;
    const uint32_t width = to_key(hi) - to_key(lo);
    shift = width < (uint32_t)kBins ? 0 : 32 - __clz(width) - kBinBits;
  }
  __device__ __forceinline__ int operator()(float x) const {
    return linear ? min((int)((hi - x) * scale), kBins - 1)
                  : (int)((to_key(hi) - to_key(x)) >> shift);
  }
};

__device__ __forceinline__ void add_weight(Smem& sm, int bin, u64 w) {
  const uint32_t lo = (uint32_t)w;
  const uint32_t old = atomicAdd(&sm.lo[bin], lo);
  const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(&sm.hi[bin], hi);
}

// The bin in which the cluster's histograms, from bin 0 on, cross `target`: above < target <= above + in.
// All CTAs' histograms must be complete (a cluster barrier), and are free after another one.  -1: none,
// above and in stay as they were.  wide: weights, whose upper words count.
__device__ __forceinline__ int find_bin(Smem& sm, u64 target, u64 base, int C, bool wide, u64& above,
                                        u64& in) {
  const int t = threadIdx.x, lane = t & 31;
  if (t == 0) sm.found_bin = -1;
  u64 mine = 0, inc = 0;
  if (t < kBins) {
    if (C == 1) {
      mine = (u64)sm.hi[t] << 32 | sm.lo[t];
    } else {
      // Word t of a CTA's histogram, by its 32-bit address in the cluster's shared memory: with sixteen
      // 64-bit addresses the kernel needs 80 registers, so 64 (64 rows of 50001: 60 us, 52 here).
      const auto word = [&](const uint32_t* p, int c) {
        uint32_t at, v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p + t)), "r"(c));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
        return v;
      };
      uint32_t l[kMaxCluster], h[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        l[c] = c < C ? word(sm.lo, c) : 0;
        h[c] = wide && c < C ? word(sm.hi, c) : 0;
      }
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) mine += (u64)h[c] << 32 | l[c];
    }
    inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sm.scan[t >> 5] = inc;
  }
  __syncthreads();
  if (t < kBins) {
    u64 run = base + inc - mine;
    for (int i = 0; i < (t >> 5); ++i) run += sm.scan[i];
    if (run < target && target <= run + mine) {
      sm.found_bin = t;
      sm.found_above = run;
      sm.found_in = mine;
    }
  }
  __syncthreads();
  const int bin = sm.found_bin;
  if (bin >= 0) {
    above = sm.found_above;
    in = sm.found_in;
  }
  return bin;
}

__device__ __forceinline__ void cluster_barrier(int C) {
  if (C > 1) cg::this_cluster().sync();
  else __syncthreads();
}

// Empty histograms; whoever reads the present ones has done so before the barrier.
__device__ __forceinline__ void clear_bins(Smem& sm, int C) {
  cluster_barrier(C);
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.lo[i] = sm.hi[i] = 0;
  __syncthreads();
}

// Sorts one key per thread, the first `size` (a power of two, at least 32) of them, ascending: the
// bitonic network, steps within a warp by shuffles, wider ones through shared memory.
__device__ __forceinline__ u64 block_sort(u64 key, int size, Smem& sm) {
  static_assert(kList == kThreads, "one candidate per thread");
  const int t = threadIdx.x;
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      u64 other;
      if (j >= 32) {
        __syncthreads();
        sm.sort[t] = key;
        __syncthreads();
        other = sm.sort[t ^ j];
      } else {
        other = __shfl_xor_sync(0xffffffffu, key, j);
      }
      const bool up = (t & k) == 0, low = (t & j) == 0;    // ascending run; lower of the two
      key = (key < other) == (up == low) ? key : other;
    }
  }
  return key;
}

// Exclusive scan of one value per thread; total: the sum.
__device__ __forceinline__ u64 block_scan(u64 v, u64& total, Smem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) sm.scan[warp] = inc;
  __syncthreads();
  const u64 w = sm.scan[lane & 7];
  total = lanes_sum<8>(w);
  return lanes_sum<8>((lane & 7) < warp ? w : 0) + inc - v;
}

// A token as a sorting key: logits descending, equal ones by index.
__device__ __forceinline__ u64 token_key(float x, int idx) {
  return (u64)(~to_key(x)) << 32 | (uint32_t)idx;
}
__device__ __forceinline__ int sort_size(int n) { return n <= 32 ? 32 : 1 << (32 - __clz(n - 1)); }

// The logits for which `in` holds into this CTA's list, if they are few; list_n above kList if not.
template <typename R, typename F>
__device__ __forceinline__ void collect(const R& row, Smem& sm, int w0, int w1, F&& in) {
  row.each(w0, w1, [&](int i, float x) {
    if (in(x)) {
      const int at = atomicAdd(&sm.list_n, 1);
      if (at < kList) {
        sm.list_x[at] = x;
        sm.list_idx[at] = row.begin + i;
      }
    }
  });
}

// After a cluster barrier: the lists' sizes, lane c the size of CTA c's, and their sum.
__device__ __forceinline__ int list_sizes(Smem& sm, int C, int& n) {
  const int lane = threadIdx.x & 31;
  int cnt = 0;
  if (lane < C) cnt = C > 1 ? *cg::this_cluster().map_shared_rank(&sm.list_n, lane) : sm.list_n;
  n = __reduce_add_sync(0xffffffffu, min(cnt, kList + 1));
  return cnt;
}

// Entry t of the cluster's lists put one after another (t below their sum).
__device__ __forceinline__ void list_entry(Smem& sm, int C, int cnt, int t, int n, float& x, int& idx) {
  int at = t, c = 0;
  for (int cc = 0; cc < C - 1; ++cc) {
    const int m = __shfl_sync(0xffffffffu, cnt, cc);
    if (c == cc && at >= m) {
      at -= m;
      ++c;
    }
  }
  if (t < n) {
    x = C > 1 ? cg::this_cluster().map_shared_rank(sm.list_x, c)[at] : sm.list_x[at];
    idx = C > 1 ? cg::this_cluster().map_shared_rank(sm.list_idx, c)[at] : sm.list_idx[at];
  }
}

// The logit at which a measure running from the largest down crosses `target`, given the bin of a
// first, linear histogram in which it does.  above: the measure of all greater logits.  lo, hi: the
// smallest and largest key of the bin's logits that this thread has read, if `known`.  kWeights: the
// measure is the weight, else the count.  The bin's span is divided by further histograms, until one
// value is left or the logits in the span are few enough for every CTA to sort them.
template <bool kWeights, typename R>
__device__ float refine(const R& row, const Weigher& w, const Bins& first, int bin, u64 target,
                        u64& above, Smem& sm, int& turn, int C, int w0, int w1, bool known,
                        uint32_t lo, uint32_t hi) {
  if (!known) {
    lo = 0xffffffffu;
    hi = 0;
    row.each(w0, w1, [&](int, float x) {
      if (x >= first.lo && x <= first.hi && first(x) == bin) {
        lo = min(lo, to_key(x));
        hi = max(hi, to_key(x));
      }
    });
  }
  cluster_minmax(lo, hi, sm, turn, C);
  u64 in = 0;
  while (lo < hi) {
    const float xlo = from_key(lo), xhi = from_key(hi);
    const Bins bins(xlo, xhi, false);
    clear_bins(sm, C);
    row.each(w0, w1, [&](int, float x) {
      if (x >= xlo && x <= xhi) {
        if (kWeights) {
          const u64 v = w(x);
          if (v) add_weight(sm, bins(x), v);
        } else {
          atomicAdd(&sm.lo[bins(x)], 1u);
        }
      }
    });
    if (threadIdx.x == 0) sm.list_n = 0;
    cluster_barrier(C);
    const int b = find_bin(sm, target, above, C, kWeights, above, in);
    if (b < 0) return xlo;       // not reached: the target is within the measure
    const u64 low = ((u64)b + 1) << bins.shift;
    if ((u64)hi + 1 > low + lo) lo = (uint32_t)((u64)hi + 1 - low);
    hi -= (uint32_t)((u64)b << bins.shift);
    if (lo >= hi) break;
    const float nlo = from_key(lo), nhi = from_key(hi);
    collect(row, sm, w0, w1, [&](float x) { return x >= nlo && x <= nhi; });
    cluster_barrier(C);
    int n;
    const int cnt = list_sizes(sm, C, n);
    if (n > kList) continue;
    float x = 0.f;
    int idx = 0;
    const int t = threadIdx.x;
    if (t == 0) sm.found_idx = __float_as_int(nlo);    // (the scan's barriers come before the next write)
    list_entry(sm, C, cnt, t, n, x, idx);
    cluster_barrier(C);          // every list has been read
    const u64 key = block_sort(t < n ? token_key(x, idx) : ~0ull, sort_size(n), sm);
    x = from_key(~(uint32_t)(key >> 32));
    const u64 v = t < n ? (kWeights ? w(x) : 1ull) : 0;
    u64 total;
    const u64 run = above + block_scan(v, total, sm);
    if (t < n && run < target && target <= run + v) sm.found_idx = __float_as_int(x);
    __syncthreads();
    const float border = __int_as_float(sm.found_idx);
    block_scan(t < n && x > border ? v : 0, total, sm);
    above += total;
    return border;
  }
  return from_key(lo);
}

template <typename T>
struct Quad;   // 16 bytes of logits
template <>
struct Quad<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[N]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Quad<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// The slice into shared memory (its first `cap`), the largest key, and the smallest that is finite:
// 16-byte loads between the aligned ends, four in flight per thread.
template <typename T, bool kFits>
__device__ __forceinline__ void load_slice(Row<T, kFits>& row, uint32_t& lo, uint32_t& hi) {
  constexpr int N = Quad<T>::N, U = 4;
  const T* src = row.x + row.begin;
  float xl = INFINITY, xh = -INFINITY;
  auto see = [&](float v) {
    const float x = canonical(v);
    xh = fmaxf(xh, x);
    if (x > -INFINITY) xl = fminf(xl, x);
    return x;
  };
  const int n = row.n;
  const int head = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / sizeof(T)));
  const int pad = kFits ? -head & 3 : 0;      // entry i of the row is at pad + i
  const int vecs = (n - head) / N;
  const uint4* v = reinterpret_cast<const uint4*>(src + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * U) {
    uint4 q[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i0 + j * kThreads < vecs) q[j] = __ldcs(v + i0 + j * kThreads);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j * kThreads;
      if (i >= vecs) continue;
      float x[N];
      Quad<T>::get(q[j], x);
      const int at = pad + head + i * N;
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 f = make_float4(see(x[e]), see(x[e + 1]), see(x[e + 2]), see(x[e + 3]));
        if (kFits) {
          *reinterpret_cast<float4*>(row.kept + at + e) = f;
        } else {
          if (at + e < row.cap) row.kept[at + e] = f.x;
          if (at + e + 1 < row.cap) row.kept[at + e + 1] = f.y;
          if (at + e + 2 < row.cap) row.kept[at + e + 2] = f.z;
          if (at + e + 3 < row.cap) row.kept[at + e + 3] = f.w;
        }
      }
    }
  }
  auto single = [&](int i) {
    const float x = see(load_logit(src + i));
    if (kFits || i < row.cap) row.kept[pad + i] = x;
  };
  if ((int)threadIdx.x < head) single(threadIdx.x);
  const int done = head + vecs * N;
  if ((int)threadIdx.x < n - done) single(done + threadIdx.x);
  if (kFits) {
    const int t = threadIdx.x, total = pad + n;
    if (t < pad) row.kept[t] = -INFINITY;
    if (t < (-total & 3)) row.kept[total + t] = -INFINITY;
    row.begin -= pad;
    row.n = (total + 3) & ~3;
  }
  lo = to_key(xl);
  hi = to_key(xh);
}

template <typename T, bool kFits>
__global__ void __launch_bounds__(kThreads, 4)
sample_kernel(const T* __restrict__ logits, long long ld, int vocab, const float* __restrict__ u,
              const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
              const float* __restrict__ top_p, const float* __restrict__ min_p,
              int32_t* __restrict__ tokens, float* __restrict__ logprobs, int C, int slice, int cap,
              int bits, const __grid_constant__ Exp2Table table) {
  __shared__ Smem sm;
  extern __shared__ __align__(16) float stored[];
  const long long r = blockIdx.x / C;
  const int rank = (int)(blockIdx.x % C);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int turn = 0;
  if (threadIdx.x < 64) sm.tab[threadIdx.x] = table.e[threadIdx.x];
  if (threadIdx.x == 0) sm.list_n = 0;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.lo[i] = sm.hi[i] = 0;
  Row<T, kFits> row;
  row.x = logits + r * ld;
  row.begin = min(rank * slice, vocab);
  row.n = min(slice, vocab - row.begin);
  row.cap = min(cap, row.n);
  row.kept = stored;
  float temp = temperature ? temperature[r] : 1.f;
  const bool greedy = !(temp > 0.f);
  if (greedy) temp = 1.f;
  float pr = top_p ? top_p[r] : 1.f, mp = min_p ? min_p[r] : 0.f;
  // Only the first token of the order is kept: greedy, a min_p that no weight reaches, a NaN filter.
  const bool lone = greedy || !(mp <= 1.f) || pr != pr;
  if (lone) {
    pr = 1.f;
    mp = 0.f;
  }
  const int k = top_k && !lone ? top_k[r] : 0;
  const float ur = u[r];

  uint32_t hi_key, lo_key;
  load_slice(row, lo_key, hi_key);
  cluster_minmax(lo_key, hi_key, sm, turn, C);
  const float hi = from_key(hi_key);
  if (hi == -INFINITY) {     // nothing to choose from (uniform over the cluster)
    if (rank == 0 && threadIdx.x == 0) {
      tokens[r] = -1;
      if (logprobs) logprobs[r] = -INFINITY;
    }
    cluster_barrier(C);
    return;
  }

  Weigher w;
  w.init(hi, temp, bits, sm.tab);
  const u64 one = 1ull << bits;
  const u64 wmin = mp == 1.f ? one : (mp > 0.f ? scaled(mp, bits, true) : 0ull);
  // A largest logit of +inf leaves weights of 1 and 0 only: nothing below it is a candidate.
  const float floor_x = w.inf || lone ? hi : from_key(lo_key);
  const bool by_count = k > 0 && k < vocab, by_weight = !by_count && pr < 1.f;
  // Weights vanish below m - bits T ln 2: the histogram of weights ends there.
  float first_lo = floor_x;
  if (by_weight && !w.inf) first_lo = fmaxf(floor_x, hi - (float)(bits + 2) / w.ch);
  const Bins first(first_lo, hi, true);

  // Every weight once: the whole vocabulary's, min-p's share by warps, and the histogram.
  const int per_warp = ((row.n + kWarps - 1) / kWarps + 127) & ~127;
  const int w0 = min(warp * per_warp, row.n), w1 = min(w0 + per_warp, row.n);
  Sums s{0, 0};
  if (by_count) {
    row.each(w0, w1, [&](int, float x) {
      s.a += w(x);
      if (x >= floor_x) atomicAdd(&sm.lo[first(x)], 1u);
    });
  } else if (by_weight) {
    row.each(w0, w1, [&](int, float x) {
      const u64 v = w(x);
      s.a += v;
      if (v && x >= first_lo) add_weight(sm, first(x), v);
    });
  } else {
    row.each(w0, w1, [&](int, float x) {
      const u64 v = w(x);
      s.a += v;
      if (v >= wmin) s.b += v;
    });
  }
  Sums before;
  const Sums all = cluster_sums(s, sm, turn, C, rank, before);
  const u64 Z = all.a;
  auto finish = [&](int idx, float x) {
    tokens[r] = idx;
    if (logprobs) logprobs[r] = w.log_share(x, Z);
  };
  auto pick = [&](u64 kept) -> u64 {     // floor(u x kept), u cut to [0, 1)
    return ur > 0.f ? (ur < 1.f ? mul_frac(kept, scaled(ur, 64, false)) : kept - 1) : 0;
  };
  // ceil(top_p x weight), at least 1: before < p x weight  <=>  before < its ceiling, for whole numbers
  auto nucleus = [&](u64 weight) -> u64 {
    const u64 frac = pr > 0.f ? scaled(pr, 64, false) : 0ull;
    return max(mul_frac(weight, frac) + (weight * frac != 0ull ? 1ull : 0ull), 1ull);
  };

  // Kept: logits above thr, and of those equal to it the first `quota`.
  float thr = floor_x;
  u64 quota = lone ? 1 : ~0ull;
  u64 above = 0, in = 0;
  int bin = by_count ? find_bin(sm, (u64)k, 0, C, false, above, in) : -1;
  const bool cut_k = bin >= 0;      // else k is above the number of finite logits
  bool recount = lone || by_count;   // the pass above did not sum what is kept
  const bool late_weight = by_count && !cut_k && pr < 1.f;   // top-k cuts nothing after all
  if (late_weight) {
    clear_bins(sm, C);
    row.each(w0, w1, [&](int, float x) {
      const u64 v = w(x);
      if (v && x >= first_lo) add_weight(sm, first(x), v);
    });
    cluster_barrier(C);
  }
  if (cut_k || by_weight || late_weight) {
    const u64 target = cut_k ? (u64)k : nucleus(Z);
    if (!cut_k) bin = find_bin(sm, target, 0, C, true, above, in);
    if (bin >= 0) {
      // The tokens down to that bin, into this CTA's list if they are few.
      const bool listed = !cut_k || above + in <= (u64)kList;
      uint32_t bin_lo = 0xffffffffu, bin_hi = 0;     // the bin's own, should they be too many
      if (listed) {
        const float bound = bin < kBins - 1 ? (float)(bin + 1) : INFINITY;
        // in a linear bin up to `bin`, or by its key
        collect(row, sm, w0, w1, [&](float x) {
          const bool c =
              x >= first_lo && (first.linear ? (hi - x) * first.scale < bound : first(x) <= bin);
          if (c && first(x) == bin) {
            bin_lo = min(bin_lo, to_key(x));
            bin_hi = max(bin_hi, to_key(x));
          }
          return c;
        });
      } else if (threadIdx.x == 0) {
        sm.list_n = kList + 1;
      }
      cluster_barrier(C);
      int n;
      const int cnt = list_sizes(sm, C, n);
      if (n <= kList) {
        // The cluster's first CTA settles it: sorted by logit, a thread's number is its token's rank.
        float x = 0.f;
        int idx = 0;
        const int t = threadIdx.x, size = sort_size(n);
        if (rank == 0) list_entry(sm, C, cnt, t, n, x, idx);
        cluster_barrier(C);         // every list has been read
        if (rank != 0) return;
        u64 key = block_sort(t < n ? token_key(x, idx) : ~0ull, size, sm);
        x = from_key(~(uint32_t)(key >> 32));
        const bool in_k = t < n && (!cut_k || t < k);
        u64 v = in_k ? w(x) : 0, Zk, Zkept;
        const u64 prior = block_scan(v, Zk, sm);
        // top-p's share is of the weight that top-k leaves
        if (!cut_k) Zk = Z;
        const bool kept = in_k && (pr >= 1.f || prior < nucleus(Zk)) && v >= wmin;
        // what is kept, by index
        key = block_sort(kept ? key << 32 | (uint32_t)~(key >> 32) : ~0ull, size, sm);
        x = from_key((uint32_t)key);
        v = key != ~0ull ? w(x) : 0;
        const u64 run = block_scan(v, Zkept, sm);
        const u64 goal = pick(Zkept);
        if (run <= goal && goal < run + v) finish((int)(key >> 32), x);
        return;
      }
      // Too many for a list: the border's logit, then top-p's within top-k's.
      if (cut_k) {
        thr = refine<false>(row, w, first, bin, target, above, sm, turn, C, w0, w1, listed, bin_lo,
                            bin_hi);
        quota = (u64)k - above;
        if (pr < 1.f) {
          u64 part = 0;
          const Bins second(thr, hi, true);
          clear_bins(sm, C);
          row.each(w0, w1, [&](int, float x) {
            if (x > thr) {
              const u64 v = w(x);
              part += v;
              if (v) add_weight(sm, second(x), v);
            }
          });
          const u64 top = cluster_sum(part, sm, turn, C, rank), tie = w(thr);
          const u64 goal = nucleus(top + quota * tie);
          const int b = goal <= top ? find_bin(sm, goal, 0, C, true, above, in) : -1;
          if (b >= 0) {
            // among the logits above top-k's border (which the last bin would take in as well)
            Bins inner = second;
            inner.lo = from_key(to_key(thr) + 1);
            thr = refine<true>(row, w, inner, b, goal, above, sm, turn, C, w0, w1, false, 0, 0);
            const u64 wt = w(thr);
            quota = wt ? (goal - above + wt - 1) / wt : 1;
          } else {
            quota = min(quota, tie ? (goal - top + tie - 1) / tie : 1ull);
          }
        }
      } else {
        thr = refine<true>(row, w, first, bin, target, above, sm, turn, C, w0, w1, listed, bin_lo,
                           bin_hi);
        const u64 wt = w(thr);
        quota = wt ? (target - above + wt - 1) / wt : 1;
      }
      recount = true;
    }
  }

  // The kept weight by warps, in index order: the logits above thr and, of the ties in index order, the
  // first `quota`.  (The warps' shares of a cluster sum stay in sm.warp_sum until the next one.)
  u64 tie_w = w(thr);
  if (tie_w < wmin) tie_w = 0;
  u64 Zkept, run, mine, ties = 0;      // the row's; before this warp; this warp's; ties before this warp
  if (recount) {
    Sums part{0, 0};
    row.each(w0, w1, [&](int, float x) {
      if (x > thr) {
        const u64 v = w(x);
        part.a += v >= wmin ? v : 0;
      } else {
        part.b += x == thr;
      }
    });
    const Sums sum = cluster_sums(part, sm, turn, C, rank, before);
    Zkept = sum.a + min(sum.b, quota) * tie_w;
    run = before.a;
    ties = before.b;
    for (int i = 0; i < warp; ++i) {
      run += sm.warp_sum[0][i];
      ties += sm.warp_sum[1][i];
    }
    const u64 first_ties = min(ties, quota), last_ties = min(ties + sm.warp_sum[1][warp], quota);
    run += first_ties * tie_w;
    mine = sm.warp_sum[0][warp] + (last_ties - first_ties) * tie_w;
  } else {
    Zkept = all.b;
    run = before.b;
    for (int i = 0; i < warp; ++i) run += sm.warp_sum[1][i];
    mine = sm.warp_sum[1][warp];
  }

  // The warp in which the running sum passes u Zkept walks its stretch.
  const u64 target = pick(Zkept);
  if (run <= target && target < run + mine) {
    // This lane's kept weight among the 32 tokens from i; `ties` moves past theirs.
    const auto step = [&](int i) -> u64 {
      const float x = i + lane < w1 ? row.at(i + lane) : -INFINITY;
      const unsigned m = __ballot_sync(0xffffffffu, x == thr);
      u64 v = 0;
      if (x > thr) {
        v = w(x);
        if (v < wmin) v = 0;
      } else if (x == thr && ties + __popc(m & ((1u << lane) - 1u)) < quota) {
        v = tie_w;
      }
      ties += __popc(m);
      return v;
    };
    // four steps of 32 tokens at a time, then the one in which it happens
    int i = w0;
    while (i + 128 < w1) {
      const u64 ties0 = ties;
      u64 v = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) v += step(i + e * 32);
      v = warp_sum(v);
      if (run + v > target) {
        ties = ties0;
        break;
      }
      run += v;
      i += 128;
    }
    for (; i < w1; i += 32) {
      u64 inc = step(i);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, run + inc > target);
      if (m) {
        if (lane == __ffs(m) - 1) finish(row.begin + i + lane, row.at(i + lane));
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (C > 1) cg::this_cluster().sync();   // no CTA leaves while another may read its slots
}

const Exp2Table& exp2_table() {
  static const Exp2Table t = [] {
    Exp2Table x{};
    for (int j = 0; j < 64; ++j) {
      const double v = exp2(j / 64.0);
      const float f = (float)(v * 2147483648.0);
      x.e[j].x = (uint32_t)(v * 2147483648.0 + 0.5);
      memcpy(&x.e[j].y, &f, sizeof(f));
    }
    return x;
  }();
  return t;
}

template <typename T>
pg_status launch(int64_t rows, int32_t vocab, const void* logits, int64_t ld, const float* u,
                 const float* temperature, const int32_t* top_k, const float* top_p,
                 const float* min_p, int32_t* tokens, float* logprobs, cudaStream_t s) {
  // CTAs per row: enough for slices of 8192 logits (32 KB; the registers allow four CTAs per SM), at most
  // a cluster of eight, and more than that needs while the rows alone do not fill the GPU and slices
  // stay above 2048 logits.  (64 rows of 50001: slices of 6251 logits 58 us, of 12501 74; 256 rows of
  // 131072: slices of 16384 logits 209 us, of 8192 in clusters of sixteen 263.)
  int C = 1;
  while (C < kMaxCluster && ((vocab + C - 1) / C > 8192 ||
                             (rows * C * 2 <= 152 && (vocab + 2 * C - 1) / (2 * C) >= 2048)))
    C *= 2;
  const int slice = (vocab + C - 1) / C;
  const int cap = std::min(slice, 49152);
  int lg = 0;
  while ((1 << lg) < vocab) ++lg;
  const int bits = std::min(45, 62 - lg);
  auto kern = cap == slice ? sample_kernel<T, true> : sample_kernel<T, false>;
  const size_t smem = (size_t)(cap + 8) * 4;
  static OncePerDevice once[2];
  pg_status st = once[cap == slice].run([&] {
    return allow_smem(kern, (size_t)(49152 + 8) * 4, "sample smem attributes");
  });
  if (st != PG_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  prof_begin(PG_KERNEL_SAMPLE, s);
  st = cuda_check(cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(logits), (long long)ld,
                                     (int)vocab, u, temperature, top_k, top_p, min_p, tokens,
                                     logprobs, C, slice, cap, bits, exp2_table()),
                  "sample launch");
  prof_end(PG_KERNEL_SAMPLE, s);
  return st;
}

}  // namespace

}  // namespace pg

using namespace pg;

extern "C" pg_status pg_sample(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits,
                               int64_t ld, const float* u, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p,
                               int32_t* tokens, float* logprobs, pg_stream_t stream) {
  const char* who = "pg_sample";
  const uintptr_t unit = dtype == PG_F32 ? 4 : 2;
  if ((dtype != PG_F32 && dtype != PG_BF16) || rows < 1 || rows > (1 << 24) || vocab < 1 ||
      vocab > (1 << 20) || ld < vocab) {
    set_error("%s: needs dtype f32 or bf16, 1 <= rows <= 2^24, 1 <= vocab <= 2^20 and ld >= vocab",
              who);
    return PG_ERR_INVALID_ARG;
  }
  if (!logits || !u || !tokens || (reinterpret_cast<uintptr_t>(logits) % unit)) {
    set_error("%s: logits, u and tokens must be non-NULL, logits aligned to its type", who);
    return PG_ERR_INVALID_ARG;
  }
  for (const void* p : {(const void*)u, (const void*)temperature, (const void*)top_k,
                        (const void*)top_p, (const void*)min_p, (const void*)tokens,
                        (const void*)logprobs})
    if (reinterpret_cast<uintptr_t>(p) % 4) {
      set_error("%s: per-row arrays must be 4-byte aligned", who);
      return PG_ERR_INVALID_ARG;
    }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == PG_F32 ? launch<float>(rows, vocab, logits, ld, u, temperature, top_k, top_p,
                                         min_p, tokens, logprobs, s)
                         : launch<__nv_bfloat16>(rows, vocab, logits, ld, u, temperature, top_k,
                                                 top_p, min_p, tokens, logprobs, s);
}
