// Token sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// The answer is a whole number decided by borders of running sums, so the sums are exact: each weight
// w_i = exp((x_i - m) / T) is a 64-bit fixed-point number (weight_bits fraction bits) evaluated to
// about 31 significant bits, and integer sums do not depend on their order.  Every threshold is then
// an integer comparison: a token is in the nucleus iff the weight before it is below
// ceil(top_p * Z), and the sampled one is the first whose running sum exceeds floor(u * Z_kept).
//
// A row is one cluster of C CTAs; each CTA keeps its slice of the row in shared memory as ordered
// 32-bit keys, so the logits are read from memory once and every later pass (total, thresholds,
// selection) runs out of shared memory.  The top-k and top-p borders are found without sorting: a
// histogram of 2048 bins (of counts, or of weights) over the span of logits gives the bin in which
// the running measure, from the largest logit down, crosses its target; the bin's span of keys is
// divided into 2048 again until it is a single key, and ties of that key are taken in index order.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "pg_internal.h"

namespace pg {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kMaxCluster = 8;
typedef unsigned long long u64;

// 2^((j - 32) / 64) in 2.62 fixed point and in fp32.
struct Exp2Table {
  u64 fixed[65];
  float f[65];
};

// ------------------------------------------------------------------------------------ keys --
// Order-preserving unsigned image of a logit: -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t to_key(float x) {
  if (x != x) x = -INFINITY;
  if (x == 0.f) x = 0.f;
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kNegInfKey = 0x007fffffu;   // to_key(-inf)
constexpr uint32_t kPosInfKey = 0xff800000u;   // to_key(+inf)

// --------------------------------------------------------------------------------- weights --
// w = exp((x - m) / T) = 2^t, t = (x - m) log2(e) / T, as a fixed-point number with `bits` fraction
// bits.  x - m and the product are carried as unevaluated sums of two floats; 2^t = 2^n 2^(j/64) e^(r ln 2)
// with |r| <= 2^-7 + rounding, the last factor by its Taylor series.
struct Weigher {
  float m, ch, cl;   // the row's maximum; log2(e) / T as ch + cl
  uint32_t max_key;
  int bits;
  const u64* tab;
  const float* tabf;
  __device__ __forceinline__ u64 operator()(uint32_t key) const {
    const u64 one = 1ull << bits;
    if (key == max_key) return one;
    if (max_key == kPosInfKey || key <= kNegInfKey) return 0;
    const float x = from_key(key);
    const float dh = x - m, bb = dh - x;
    const float de = (x - (dh - bb)) + (-m - bb);
    const float th = dh * ch;
    if (!(th > -(float)(bits + 2))) return 0;
    const float tl = fmaf(dh, ch, -th) + fmaf(dh, cl, de * ch);
    const float n = rintf(th);
    const float fr = th - n;                         // exact
    const float j = rintf(fr * 64.f);
    const float r = fmaf(j, -1.f / 64.f, fr) + tl;
    // e^(r ln 2) - 1 by its Taylor series: (ln 2)^i / i!
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 0.009618129107628477f, 0.05550410866482158f),
                                     0.2402265069591007f), 0.6931471805599453f);
    const int ji = (int)j + 32;
    const float add = tabf[ji] * p;                  // |add| < 2^-7
    const long long w62 = (long long)tab[ji] + ((long long)__float2int_rn(add * 0x1p37f) << 25);
    const int sh = 62 - bits - (int)n;               // >= 62 - bits > 1
    if (sh > 63) return 0;
    const u64 w = ((u64)w62 + (1ull << (sh - 1))) >> sh;
    return w > one ? one : w;
  }
};

// floor(a * f) for f = frac / 2^64.
__device__ __forceinline__ u64 mul_frac(u64 a, u64 frac) { return __umul64hi(a, frac); }

// x in (0, 1) as 0.64 fixed point (exact for x >= 2^-40, else cut to 2^-64).
__device__ __forceinline__ u64 to_frac(float x) { return (u64)((double)x * 18446744073709551616.0); }

// ------------------------------------------------------------------------- shared memory ----
struct Smem {
  u64 tab[65];
  float tabf[65];
  u64 hist[kBins];        // counts or weights
  u64 warp_sum[kWarps];
  u64 scan[kWarps];
  u64 slot[2];            // this CTA's contribution to a cluster reduction (two, used in turn)
  uint32_t slot_lo, slot_hi;
  u64 found_above;        // the crossing bin's predecessors
  int found_bin;
  int found_idx;
};

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

template <typename T>
struct Row {
  const T* x;
  uint32_t* keys;     // shared memory, the first `cap` of the slice
  int begin, n, cap;  // slice [begin, begin + n) of the row
  __device__ __forceinline__ uint32_t key(int i) const {
    return i < cap ? keys[i] : to_key(load_logit(x + begin + i));
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ u64 block_sum(u64 v, Smem& sm) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) s += sm.warp_sum[i];
  return s;
}

// Sum over the cluster and over the CTAs of lower rank.  `turn` alternates between the two slots, so a
// CTA may write its next contribution while another still reads the previous one.
__device__ __forceinline__ u64 cluster_sum(u64 block_total, Smem& sm, int& turn, int C, int rank,
                                           u64& before) {
  before = 0;
  if (C == 1) return block_total;
  cg::cluster_group cl = cg::this_cluster();
  if (threadIdx.x == 0) sm.slot[turn] = block_total;
  cl.sync();
  u64 s = 0;
  for (int c = 0; c < C; ++c) {
    const u64 v = *cl.map_shared_rank(&sm.slot[turn], c);
    if (c < rank) before += v;
    s += v;
  }
  turn ^= 1;
  return s;
}

// The largest and smallest key of the cluster's slices among those passed in.
__device__ __forceinline__ void cluster_minmax(uint32_t& lo, uint32_t& hi, Smem& sm, int C) {
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if (threadIdx.x == 0) {
    sm.slot_lo = 0xffffffffu;
    sm.slot_hi = 0;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    atomicMin(&sm.slot_lo, lo);
    atomicMax(&sm.slot_hi, hi);
  }
  if (C == 1) {
    __syncthreads();
    lo = sm.slot_lo;
    hi = sm.slot_hi;
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  lo = 0xffffffffu;
  hi = 0;
  for (int c = 0; c < C; ++c) {
    lo = min(lo, *cl.map_shared_rank(&sm.slot_lo, c));
    hi = max(hi, *cl.map_shared_rank(&sm.slot_hi, c));
  }
  cl.sync();
}

// Level-1 bin of a key: linear in the logit, 0 for the largest.
struct LinearBins {
  float m, scale;
  __device__ __forceinline__ int operator()(uint32_t key) const {
    return min((int)((m - from_key(key)) * scale), kBins - 1);
  }
};

// The key at which a measure running from the largest logit down crosses `target` (at least 1, at
// most the whole measure): above = measure of all greater keys < target <= above + measure of the key.
// kWeights: the measure is the weight, else the count.  Only keys >= floor_key take part.
template <bool kWeights, typename T>
__device__ uint32_t crossing(const Row<T>& row, const Weigher& w, u64 target, uint32_t floor_key,
                             uint32_t lo, uint32_t hi, Smem& sm, int C, u64& above) {
  above = 0;
  bool linear = true;
  // lo and hi: the smallest and largest finite key that can be the answer.
  while (lo < hi) {
    const float mx = from_key(hi), span = mx - from_key(lo);
    // linear needs a finite scale; a span that overflows or vanishes goes by key at once
    const float scale = (float)kBins / span;
    if (linear && !(span > 0.f && span < INFINITY && scale < INFINITY)) linear = false;
    const LinearBins lb{mx, scale};
    const uint32_t width = hi - lo;
    const int shift = width < (uint32_t)kBins ? 0 : 32 - __clz(width) - 11;   // (hi - key) >> shift < 2048
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
      const uint32_t key = row.key(i);
      if (key < lo || key > hi || key < floor_key) continue;
      const int b = linear ? lb(key) : (int)((hi - key) >> shift);
      const u64 add = kWeights ? w(key) : 1ull;
      if (add) atomicAdd(&sm.hist[b], add);
    }
    u64 bins[kBinsPerThread], mine = 0;
    if (C == 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kBinsPerThread; ++e) bins[e] = sm.hist[threadIdx.x * kBinsPerThread + e];
    } else {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
#pragma unroll
      for (int e = 0; e < kBinsPerThread; ++e) bins[e] = 0;
      for (int c = 0; c < C; ++c) {
        const u64* h = cl.map_shared_rank(sm.hist, c) + threadIdx.x * kBinsPerThread;
#pragma unroll
        for (int e = 0; e < kBinsPerThread; ++e) bins[e] += h[e];
      }
    }
#pragma unroll
    for (int e = 0; e < kBinsPerThread; ++e) mine += bins[e];
    // exclusive scan over the threads
    u64 inc = mine;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (threadIdx.x == 0) sm.found_bin = -1;
    if (lane == 31) sm.scan[threadIdx.x >> 5] = inc;
    __syncthreads();
    u64 run = above + inc - mine;
    for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) run += sm.scan[i];
#pragma unroll
    for (int e = 0; e < kBinsPerThread; ++e) {
      if (run < target && target <= run + bins[e]) {
        sm.found_bin = threadIdx.x * kBinsPerThread + e;
        sm.found_above = run;
      }
      run += bins[e];
    }
    if (C > 1) cg::this_cluster().sync();   // the histogram may be cleared after this
    else __syncthreads();
    const int bin = sm.found_bin;
    above = sm.found_above;
    if (bin < 0) return lo;                 // not reached: target is within the whole measure
    // the span of the keys in that bin
    uint32_t klo = 0xffffffffu, khi = 0;
    if (linear) {
      for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const uint32_t key = row.key(i);
        if (key < lo || key > hi || key < floor_key || lb(key) != bin) continue;
        klo = min(klo, key);
        khi = max(khi, key);
      }
      cluster_minmax(klo, khi, sm, C);
      linear = false;
    } else {
      const u64 top = (u64)hi - ((u64)bin << shift);
      khi = (uint32_t)top;
      const u64 low = ((u64)bin + 1) << shift;
      klo = (u64)hi + 1 > low ? (uint32_t)((u64)hi + 1 - low) : 0u;
      klo = max(klo, lo);
      __syncthreads();
    }
    lo = klo;
    hi = khi;
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
sample_kernel(const T* __restrict__ logits, long long ld, int vocab, const float* __restrict__ u,
              const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
              const float* __restrict__ top_p, const float* __restrict__ min_p,
              int32_t* __restrict__ tokens, float* __restrict__ logprobs, int C, int slice, int cap,
              int bits, const __grid_constant__ Exp2Table table) {
  __shared__ Smem sm;
  extern __shared__ uint32_t keys[];
  const long long r = blockIdx.x / C;
  const int rank = (int)(blockIdx.x % C);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int turn = 0;
  for (int i = threadIdx.x; i < 65; i += kThreads) {
    sm.tab[i] = table.fixed[i];
    sm.tabf[i] = table.f[i];
  }
  Row<T> row;
  row.x = logits + r * ld;
  row.begin = min(rank * slice, vocab);
  row.n = min(slice, vocab - row.begin);
  row.cap = min(cap, row.n);
  row.keys = keys;
  float temp = temperature ? temperature[r] : 1.f;
  const bool greedy = !(temp > 0.f);
  if (greedy) temp = 1.f;

  // The slice's keys, the largest, and the smallest that is finite.
  uint32_t hi = 0, lo = 0xffffffffu;
  for (int i = threadIdx.x; i < row.n; i += kThreads) {
    const uint32_t k = to_key(load_logit(row.x + row.begin + i));
    if (i < row.cap) keys[i] = k;
    hi = max(hi, k);
    if (k > kNegInfKey) lo = min(lo, k);
  }
  cluster_minmax(lo, hi, sm, C);
  if (hi <= kNegInfKey) {     // nothing to choose from (uniform over the cluster)
    if (rank == 0 && threadIdx.x == 0) {
      tokens[r] = -1;
      if (logprobs) logprobs[r] = -INFINITY;
    }
    return;
  }

  Weigher w;
  const double c = 1.4426950408889634074 / (double)temp;
  w.m = from_key(hi);
  w.ch = (float)c;
  w.cl = (float)(c - (double)w.ch);
  w.max_key = hi;
  w.bits = bits;
  w.tab = sm.tab;
  w.tabf = sm.tabf;

  // The whole vocabulary's weight.
  u64 sum = 0, before;
  for (int i = threadIdx.x; i < row.n; i += kThreads) sum += w(row.key(i));
  const u64 Z = cluster_sum(block_sum(sum, sm), sm, turn, C, rank, before);

  // Kept: keys above thr, and of those equal to it the first `quota`.
  uint32_t thr = kNegInfKey + 1;
  u64 quota = ~0ull;
  if (greedy || hi == kPosInfKey) {
    // Equal weights 1 for the largest logits, 0 for all others: top-k and top-p count ties.
    thr = hi;
    if (greedy) quota = 1;
  }
  u64 Zk = Z;
  if (!greedy) {
    const int k = top_k ? top_k[r] : 0;
    if (k > 0 && k < vocab) {
      // Among k or fewer finite logits all are kept; cnt finite ones in all.
      u64 cnt = 0;
      for (int i = threadIdx.x; i < row.n; i += kThreads) cnt += row.key(i) >= thr;
      cnt = cluster_sum(block_sum(cnt, sm), sm, turn, C, rank, before);
      if ((u64)k < cnt) {
        u64 above;
        thr = crossing<false>(row, w, (u64)k, thr, max(lo, thr), hi, sm, C, above);
        quota = (u64)k - above;
        u64 part = 0;
        for (int i = threadIdx.x; i < row.n; i += kThreads) {
          const uint32_t key = row.key(i);
          if (key > thr) part += w(key);
        }
        Zk = cluster_sum(block_sum(part, sm), sm, turn, C, rank, before) + quota * w(thr);
      }
    }
    const float p = top_p ? top_p[r] : 1.f;
    if (p < 1.f) {
      const u64 frac = p > 0.f ? to_frac(p) : 0ull;
      // ceil(p Zk), at least 1: before < p Zk  <=>  before < ceil(p Zk) for whole numbers
      u64 target = mul_frac(Zk, frac) + (Zk * frac != 0ull);
      if (target == 0) target = 1;
      u64 above;
      const uint32_t key = crossing<true>(row, w, target, thr, max(lo, thr), hi, sm, C, above);
      const u64 wt = w(key);
      const u64 need = wt ? (target - above + wt - 1) / wt : 1;
      quota = key == thr ? min(quota, need) : need;   // top-k's quota is for its own border
      thr = key;
    }
  }
  u64 wmin = 0;
  if (min_p && !greedy) {
    const float mp = min_p[r];
    const u64 one = 1ull << bits;
    if (mp >= 1.f) wmin = one;
    else if (mp > 0.f) {
      const double x = ceil((double)mp * (double)one);
      wmin = (u64)x;
    }
  }

  // The index of the last tie that is kept: ties are taken in index order.
  const int per_warp = ((row.n + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(warp * per_warp, row.n), w1 = min(w0 + per_warp, row.n);
  int last_tie = vocab;      // all
  if (quota != ~0ull) {
    u64 ties = 0;
    for (int i = w0 + lane; i < w1; i += 32) ties += row.key(i) == thr;
    ties = warp_sum(ties);
    __syncthreads();
    if (lane == 0) sm.scan[warp] = ties;
    if (threadIdx.x == 0) sm.found_idx = -1;
    __syncthreads();
    u64 in_block = 0, in_warps = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) in_warps += sm.scan[i];
      in_block += sm.scan[i];
    }
    u64 lower;
    cluster_sum(in_block, sm, turn, C, rank, lower);
    u64 run = lower + in_warps;
    if (run < quota && quota <= run + ties) {
      for (int i = w0; i < w1; i += 32) {
        const bool tie = i + lane < w1 && row.key(i + lane) == thr;
        const unsigned m = __ballot_sync(0xffffffffu, tie);
        if (run + __popc(m) >= quota) {
          const int rank_in = __popc(m & ((1u << lane) - 1u));
          if (tie && run + rank_in + 1 == quota) sm.found_idx = row.begin + i + lane;
          break;
        }
        run += __popc(m);
      }
    }
    __syncthreads();
    // found by at most one CTA; none: every tie is kept
    const u64 found = cluster_sum((u64)(sm.found_idx + 1), sm, turn, C, rank, lower);
    if (found) last_tie = (int)found - 1;
  }
  auto kept = [&](int i, uint32_t key) -> u64 {
    if (key < thr || (key == thr && row.begin + i > last_tie)) return 0;
    const u64 x = w(key);
    return x >= wmin ? x : 0;
  };

  // The kept weight by warps, in index order, and the warp in which the running sum passes u Zkept.
  u64 mine = 0;
  for (int i = w0 + lane; i < w1; i += 32) mine += kept(i, row.key(i));
  mine = warp_sum(mine);
  __syncthreads();
  if (lane == 0) sm.scan[warp] = mine;
  __syncthreads();
  u64 in_block = 0, run = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) run += sm.scan[i];
    in_block += sm.scan[i];
  }
  u64 lower;
  const u64 Zkept = cluster_sum(in_block, sm, turn, C, rank, lower);
  run += lower;
  const float ur = u[r];
  u64 target = ur > 0.f ? (ur < 1.f ? mul_frac(Zkept, to_frac(ur)) : Zkept - 1) : 0;
  if (run <= target && target < run + mine) {
    for (int i = w0; i < w1; i += 32) {
      const uint32_t key = i + lane < w1 ? row.key(i + lane) : 0;
      const u64 x = i + lane < w1 ? kept(i + lane, key) : 0;
      u64 inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, run + inc > target);
      if (m) {
        if (lane == __ffs(m) - 1) {
          tokens[r] = row.begin + i + lane;
          if (logprobs) {
            const double total = ldexp((double)Z, -bits);
            const double d = key == hi ? 0.0 : ((double)from_key(key) - (double)w.m) / (double)temp;
            logprobs[r] = (float)(d - log(total));
          }
        }
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
    for (int j = 0; j <= 64; ++j) {
      const long double v = exp2l((j - 32) / 64.0L);
      x.fixed[j] = (u64)(v * 4611686018427387904.0L + 0.5L);
      x.f[j] = (float)v;
    }
    return x;
  }();
  return t;
}

template <typename T>
pg_status launch(int64_t rows, int32_t vocab, const void* logits, int64_t ld, const float* u,
                 const float* temperature, const int32_t* top_k, const float* top_p,
                 const float* min_p, int32_t* tokens, float* logprobs, cudaStream_t s) {
  // CTAs per row: enough that a slice of 16384 keys (64 KB) stays in shared memory, and more while
  // the rows alone do not fill the GPU and slices stay above 2048 keys.
  int C = 1;
  while (C < kMaxCluster && ((vocab + C - 1) / C > 16384 ||
                             (rows * C * 2 <= 152 && (vocab + 2 * C - 1) / (2 * C) >= 2048)))
    C *= 2;
  const int slice = (vocab + C - 1) / C;
  const int cap = std::min(slice, 49152);
  int lg = 0;
  while ((1 << lg) < vocab) ++lg;
  const int bits = std::min(45, 62 - lg);
  auto kern = sample_kernel<T>;
  const size_t smem = (size_t)cap * 4;
  pg_status st = cuda_check(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 49152 * 4),
      "sample smem attribute");
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
