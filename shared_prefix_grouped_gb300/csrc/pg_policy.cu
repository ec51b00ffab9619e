// The clipped policy loss with a KL term from the logits, and its gradient.
//
// With c = log2 e / T and m a row's largest logit, p_i = 2^(c (x_i - m)) / sum_j 2^(c (x_j - m)); a token's
// log-probability gives its loss and d loss / d log-probability g in closed form, and the row's gradient
// is 1/T (sum of g at the tokens' places - p sum g).  So a row is needed twice: for its maximum and sum,
// then for p.  It is read once: a row is a cluster of C CTAs whose threads hold its logits in registers as
// they came (16-byte vectors, kVec of them per thread) from the first pass to the second.  Each thread
// takes the maximum of its own logits and their sum against it; the pairs (maximum, sum) meet by
// shuffles, in shared memory and through the cluster's distributed shared memory, one cluster barrier
// per row.  Rows longer than a cluster's registers go through in several pieces, and once more for the
// gradient (out of L2, unless the rows in flight exceed it).
//
// Every thread works out the row's token by itself (a few broadcast reads), so that the common row of
// one target needs no further barrier; a row with several (a prefix's last row) takes one more.
//
// The backward alone needs a row once, so its CTAs take any length in pieces.
//
// Bound by memory: two bytes read and two written per bf16 logit.  The backward of 4096 rows of 131072 bf16 logits
// takes 312 us (6.9 TB/s), of 4096 rows of 32000 fp32 159 us (6.6 TB/s); of 16 rows of 32000 fp32 the forward takes
// 7.6 us with the sum of the loss, most of it launches and the chain of reads row_starts, tokens, logits.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "../../include/pg_policy.h"
#include "pg_internal.h"
#include "pg_sm100.cuh"

namespace pg {

namespace cg = cooperative_groups;
using namespace sm100;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kListed = 512;         // targets of a row that a CTA keeps a list of
constexpr int kSMs = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ int s_status_policy = 0;

__device__ __forceinline__ void report(int code) { atomicCAS(&s_status_policy, 0, code); }

enum Mode { kForward = 0, kStep = 1, kBackward = 2 };

struct PolicyArgs {
  const void* logits;
  void* dlogits;
  long long ld, ldd, n_tokens;
  const int32_t *row_starts, *tokens;
  const float *old_lp, *ref_lp, *adv, *weights, *grad_output;
  float *lse, *logprobs, *token_loss, *token_grad;
  int vocab, C;
  float c, inv_t, lo, hi, kl;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of a row.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint4 lowest() {        // of -inf
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    return fmaxf(fmax3(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)),
                 __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint4 lowest() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __forceinline__ float get(const uint4& v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    const __nv_bfloat162 a = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&v.x),
                                     *reinterpret_cast<const __nv_bfloat162*>(&v.y));
    const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&v.z),
                                     *reinterpret_cast<const __nv_bfloat162*>(&v.w));
    const float2 f = __bfloat1622float2(__hmax2(a, b));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// (maximum, sum of 2^(c (x - maximum))): the pair of two sets of logits.  -inf: an empty set.
__device__ __forceinline__ float2 join(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, a.y + b.y);      // (a NaN stays in the sum)
  return make_float2(m, a.y * ex2(c * (a.x - m)) + b.y * ex2(c * (b.x - m)));
}

// A token's terms, from its log-probability.
struct Term {
  float loss, grad;
};
__device__ __forceinline__ Term term_of(const PolicyArgs& a, float lp, bool dead, float old, float ref,
                                        float adv, float w) {
  Term t{0.f, 0.f};
  if (w == 0.f || dead) return t;
  const float ratio = a.old_lp ? expf(lp - old) : (lp != lp ? lp : 1.f);
  const float free = ratio * adv, held = fminf(fmaxf(ratio, a.lo), a.hi) * adv;
  t.loss = ratio != ratio ? ratio : -fminf(free, held);
  t.grad = ratio != ratio ? ratio : (free <= held ? -free : 0.f);
  if (a.ref_lp) {
    const float gap = ref - lp, em1 = expm1f(gap);
    t.loss += a.kl * (em1 - gap);
    t.grad -= a.kl * em1;
  }
  t.loss *= w;
  t.grad *= w;
  return t;
}
__device__ __forceinline__ Term term(const PolicyArgs& a, long long n, float lp, bool dead) {
  return term_of(a, lp, dead, a.old_lp ? a.old_lp[n] : 0.f, a.ref_lp ? a.ref_lp[n] : 0.f, a.adv[n],
                 a.weights ? a.weights[n] : 1.f);
}

// A target of a row of several: its place (-1: none, or none of this CTA's), its gradient and its logit.
struct Target {
  int y;
  float g, z;
};

// The gradient at the places of a row's k listed targets, whose vectors have been stored without them (a barrier
// ago): of equal ones the first takes all, in order.  p: the row's -sum g / T times the probability of a
// logit.  380 rows of 131072 bf16 logits, one of them with 64, 256 or 1024 targets: 47, 54 and 102 us, with one 46.6
// (a walk over the targets at every vector, as rows with more than the list holds take it: 118, 332 and 1179).
template <typename T, typename P>
__device__ __forceinline__ void add_targets(T* drow, const Target* list, int k, int tid, int threads, float gt,
                                            P&& p) {
  for (int j = tid; j < k; j += threads) {
    const Target t = list[j];
    bool first = t.y >= 0;
    for (int i = 0; first && i < j; ++i) first = list[i].y != t.y;
    if (!first) continue;
    float g = t.g;
    for (int i = j + 1; i < k; ++i)
      if (list[i].y == t.y) g += list[i].g;
    drow[t.y] = (T)fmaf(g, gt, p(t.z));
  }
}

template <typename T, int kVec, int kMode>
__global__ void __launch_bounds__(kThreads)
policy_kernel(const PolicyArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr int kTile = kThreads * kVec;              // vectors a CTA holds
  __shared__ float2 part[kWarps], slot[kMaxCluster];
  __shared__ float red[kWarps];
  __shared__ Target list[kMode == kForward ? 1 : kListed];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.C, rank = C > 1 ? (int)(blockIdx.x % C) : 0;
  const long long r = blockIdx.x / C;

  long long t0 = r, t1 = r + 1;
  if (a.row_starts) {
    const long long s0 = a.row_starts[r], s1 = a.row_starts[r + 1];
    t0 = min(max(s0, 0ll), a.n_tokens);
    t1 = min(max(s1, t0), a.n_tokens);
    // (a token before the first row's or behind the last row's is nobody's)
    const bool loose = (r == 0 && s0 != 0) || (r == (long long)gridDim.x / C - 1 && s1 != a.n_tokens);
    if ((t0 != s0 || t1 != s1 || loose) && rank == 0 && tid == 0) report(PG_ERR_DEVICE);
  }
  const int k = (int)min(t1 - t0, 1ll << 30);

  const T* row = static_cast<const T*>(a.logits) + r * a.ld;
  T* drow = kMode == kForward ? nullptr : static_cast<T*>(a.dlogits) + r * a.ldd;
  // Vector v of the row: logits [v N - ph, v N - ph + N), on 16-byte boundaries of memory.
  const int ph = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const bool same_phase =
      kMode != kForward && (int)((reinterpret_cast<uintptr_t>(drow) & 15) / sizeof(T)) == ph;
  const int nv = (a.vocab + ph + N - 1) / N;
  const int per = (nv + C - 1) / C;
  const int v_lo = min(rank * per, nv), v_hi = min(v_lo + per, nv);
  const int tiles = (per + kTile - 1) / kTile;        // the same for every CTA of the cluster

  auto store = [&](int v, const float (&f)[N]) {
    const int i = v * N - ph;
    if (same_phase && i >= 0 && i + N <= a.vocab) {
      *reinterpret_cast<uint4*>(drow + i) = V::pack(f);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (i + e >= 0 && i + e < a.vocab) drow[i + e] = (T)f[e];
    }
  };
  auto zero_row = [&] {
    float f[N];
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = 0.f;
    for (int v = v_lo + tid; v < v_hi; v += kThreads) store(v, f);
  };
  // A token's place in the vocabulary, or -1.
  auto token = [&](long long n) {
    const int y = a.tokens[n];
    if (y >= a.vocab && rank == 0) report(PG_ERR_DEVICE);
    return y >= 0 && y < a.vocab ? y : -1;
  };

  if (k == 0) {
    if (kMode != kBackward && rank == 0 && tid == 0) a.lse[r] = 0.f;
    if (kMode != kForward) zero_row();
    return;                                           // (the whole cluster)
  }

  // The sum over the row's tokens of their gradients, and whether any is not 0; in every thread.
  const float go = kMode == kBackward && a.grad_output ? a.grad_output[0] : 1.f;
  float g_sum = 0.f;
  bool any = false;
  int y1 = -1;                                        // the token of a row of one
  auto sum_grads = [&] {
    float s = 0.f;
    bool nz = false;
    for (long long n = t0 + tid; n < t1; n += kThreads) {
      const int y = a.tokens[n];
      const float g = y >= 0 && y < a.vocab ? a.token_grad[n] : 0.f;
      s += g;
      nz |= g != 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[warp] = s;
    any = __syncthreads_or(nz);
    g_sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) g_sum += red[w];
  };
  if (kMode == kBackward) {
    if (k == 1) {
      y1 = token(t0);
      g_sum = y1 >= 0 ? a.token_grad[t0] : 0.f;
      any = g_sum != 0.f;
    } else {
      for (long long n = t0 + tid; n < t1; n += kThreads) token(n);
      sum_grads();
    }
    if (!any) {
      zero_row();
      return;
    }
  }

  uint4 x[kVec];
  auto load = [&](int tile) {
    const int v0 = v_lo + tile * kTile + tid;
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int v = v0 + u * kThreads, i = v * N - ph;
      float f[N];
      if (v < v_hi && i >= 0 && i + N <= a.vocab) {
        x[u] = *reinterpret_cast<const uint4*>(row + i);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          f[e] = v < v_hi && i + e >= 0 && i + e < a.vocab ? to_f(row[i + e]) : -INFINITY;
        x[u] = V::pack(f);
      }
    }
  };

  // p = 2^(px (ax x - rx)) * scale: c (x - m) over the sum, or log2 e (x / T - lse).
  float ax, rx, px, scale;
  if (kMode == kBackward) {
    load(0);
    const float l = a.lse[r];
    ax = a.inv_t;
    rx = l == -INFINITY ? INFINITY : l;
    px = kLog2e;
    scale = 1.f;
  } else {
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    float2 ms = make_float2(-INFINITY, 0.f);
    float xy = -INFINITY;
    for (int t = 0; t < tiles; ++t) {
      load(t);
      if (t == 0 && k == 1) {          // with the row on its way; before anything is overwritten
        y1 = token(t0);
        if (y1 >= 0) xy = to_f(row[y1]);
      }
      float m = V::vmax(x[0]);
#pragma unroll
      for (int u = 1; u < kVec; ++u) m = fmaxf(m, V::vmax(x[u]));
      // (x - m before the product: c m may overflow where every logit is the type's lowest)
      const float ref = m == -INFINITY ? 0.f : m;
      const uint64_t c2 = f2_pack(a.c, a.c), r2 = f2_pack(-ref, -ref);
      uint64_t s2 = f2_pack(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kVec; ++u)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          float b0, b1;
          f2_unpack(f2_mul(f2_add(f2_pack(V::get(x[u], e), V::get(x[u], e + 1)), r2), c2), b0, b1);
          s2 = f2_add(s2, f2_pack(ex2(b0), ex2(b1)));
        }
      float s0, s1;
      f2_unpack(s2, s0, s1);
      ms = t == 0 ? make_float2(m, s0 + s1) : join(ms, make_float2(m, s0 + s1), a.c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float2 other = make_float2(__shfl_xor_sync(0xffffffffu, ms.x, o),
                                       __shfl_xor_sync(0xffffffffu, ms.y, o));
      // (the lower lane's pair first, so that every lane computes the same)
      ms = lane & o ? join(other, ms, a.c) : join(ms, other, a.c);
    }
    if (lane == 0) part[warp] = ms;
    __syncthreads();
    ms = part[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) ms = join(ms, part[w], a.c);
    if (C > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");       // every CTA has started
      if (tid < C) cg::this_cluster().map_shared_rank(slot, tid)[rank] = ms;
      cg::this_cluster().sync();
      ms = slot[0];
      for (int i = 1; i < C; ++i) ms = join(ms, slot[i], a.c);
    }
    const bool dead = ms.x == -INFINITY && ms.y == 0.f;       // nothing but -inf
    ax = 1.f;
    rx = ms.x == -INFINITY ? 0.f : ms.x;
    px = a.c;
    scale = 1.f / ms.y;
    const float ls = log2f(ms.y);
    auto logprob = [&](float z) { return dead ? -INFINITY : (fmaf(z - rx, a.c, -ls)) * kLn2; };
    if (rank == 0 && tid == 0) a.lse[r] = dead ? -INFINITY : fmaf(rx, a.inv_t, ls * kLn2);
    auto settle = [&](long long n, int y, float z, bool write) {
      Term t{0.f, 0.f};
      const float lp = y >= 0 ? logprob(z) : 0.f;
      if (y >= 0 && a.adv) t = term(a, n, lp, dead);
      if (write) {
        a.logprobs[n] = lp;
        if (a.adv) {
          a.token_loss[n] = t.loss;
          a.token_grad[n] = t.grad;
        }
      }
      return t.grad;
    };
    if (k == 1) {
      if (kMode == kStep || (rank == 0 && tid == 0)) g_sum = settle(t0, y1, xy, rank == 0 && tid == 0);
      any = g_sum != 0.f;
    } else {
      if (rank == 0)
        for (long long n = t0 + tid; n < t1; n += kThreads) {
          const int y = token(n);
          settle(n, y, y >= 0 ? to_f(row[y]) : 0.f, true);
        }
      if (kMode == kStep) {
        // The tokens' gradients, written by the first CTA, to all; the row is overwritten after this.
        if (C > 1) cg::this_cluster().sync();
        else __syncthreads();
        sum_grads();
      }
    }
    if (kMode == kForward) return;
    if (!any) {
      zero_row();
      return;
    }
  }
  if (kMode == kForward) return;

  const float gt = go * a.inv_t;
  // fp32 throughout: -sum g / T * p, and g / T at the tokens' places.
  const float coef = -(g_sum * gt) * scale;
  const uint64_t a2 = f2_pack(ax, ax), r2 = f2_pack(-rx, -rx), p2 = f2_pack(px, px),
                 k2 = f2_pack(coef, coef);
  const int vy1 = k == 1 ? (y1 + ph) / N : -1;
  const bool listed = k > 1 && k <= kListed;
  if (listed) {
    for (int j = tid; j < k; j += kThreads) {
      const int y = a.tokens[t0 + j], v = (y + ph) / N;
      const bool mine = y >= 0 && y < a.vocab && v >= v_lo && v < v_hi;
      list[j] = mine ? Target{y, a.token_grad[t0 + j], to_f(row[y])} : Target{-1, 0.f, 0.f};
    }
    __syncthreads();                                  // (before anything of the row is overwritten)
  }
  for (int t = 0; t < tiles; ++t) {
    if (tiles > 1 && !(kMode == kBackward && t == 0)) load(t);
    const int v0 = v_lo + t * kTile + tid;
    uint32_t hit = 0;
    if (k == 1) {
      const int d = vy1 - v0;
      if (y1 >= 0 && d >= 0 && d < kTile && d % kThreads == 0) hit = 1u << (d / kThreads);
    } else if (!listed) {
      for (long long n = t0; n < t1; ++n) {
        const int y = a.tokens[n], d = (y + ph) / N - v0;
        if (y >= 0 && y < a.vocab && d >= 0 && d < kTile && d % kThreads == 0)
          hit |= 1u << (d / kThreads);
      }
    }
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const int v = v0 + u * kThreads;
      if (v >= v_hi) break;
      float f[N];
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float b0, b1;
        f2_unpack(f2_mul(f2_fma(f2_pack(V::get(x[u], e), V::get(x[u], e + 1)), a2, r2), p2), b0, b1);
        f2_unpack(f2_mul(f2_pack(ex2(b0), ex2(b1)), k2), f[e], f[e + 1]);
      }
      if (hit >> u & 1) {
        for (long long n = t0; n < t1; ++n) {
          const int y = k == 1 ? y1 : a.tokens[n];
          const float g = k == 1 ? g_sum : a.token_grad[n];
          const int at = y < 0 || y >= a.vocab ? -1 : y + ph - v * N;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (at == e) f[e] = fmaf(g, gt, f[e]);
        }
      }
      store(v, f);
    }
  }
  if (listed) {
    __syncthreads();
    add_targets(drow, list, k, tid, kThreads, gt, [&](float z) { return ex2(fmaf(z, ax, -rx) * px) * coef; });
  }
}

// ---------------------------------------------------------------------------------------------
// Many long rows: persistent CTAs through whose shared memory the rows stream, one row after another per
// cluster of C CTAs (C = 1 while a row, or for the forward any part of it, fits).  A warp keeps the ring of
// 32 KB chunks full by bulk copies, chunks of the next row into what the second pass of this one has
// freed, so that reads never wait for a row's reductions; another reads the rows' tokens and what belongs to
// them, 32 rows at a time.  The 16 other warps add up a row's chunks as they arrive, exchange
// (maximum, sum) with the cluster's other CTAs by remote stores that complete on a barrier, and go
// through the chunks again for the gradient.
// A thread's sum is against the logit of the row's token, which is near the largest or at least below it: no
// maximum is looked for unless a chunk brings the sum past 2^100 (or the row has no such logit), when
// the chunk, still in registers, is gone through again, with a maximum that may then lag behind by 2^kLag.
// Sums and probabilities cost 3 and 3.5 instructions per bf16 logit; what bounds the kernel beside memory is
// their issue, and, of rows below 100 KB, what a row costs however short it is (its reductions and the wait
// for its first chunk).  Loss and gradient of 8192 rows of 131072 bf16 logits take 681 us (6.3 TB/s; the kernel
// above 2047), the forward 320 us (6.7 TB/s; 642).
// ---------------------------------------------------------------------------------------------
constexpr int kMetaRows = 32;
constexpr float kLag = 40.f;
constexpr float kExact = 0x1p24f;     // products below it are off by half at most
constexpr uint64_t kWaitNs = 2000000000ull;

// One CTA of 16 workers' warps per SM, or two of 8 or four of 4 with their share of the ring, which hide
// each other's reductions.  Chunks in vectors of 16 bytes.
struct Wide {
  static constexpr int kWorkers = 512, kChunk = 2048, kRing = 6, kPerSm = 1, kListed = 1024;
};
struct Pair {
  static constexpr int kWorkers = 256, kChunk = 1280, kRing = 5, kPerSm = 2, kListed = 512;
};
struct Quad {
  static constexpr int kWorkers = 128, kChunk = 1024, kRing = 3, kPerSm = 4, kListed = 256;
};

// A row's tokens; of a row of one token, its place, its logit and what belongs to it.
struct RowMeta {
  int t0, k, y;
  float x, old, ref, adv, w;
};

template <typename Shape>
struct StreamSmem {
  uint4 ring[Shape::kRing][Shape::kChunk];
  RowMeta meta[2][kMetaRows];
  Target list[Shape::kListed];
  float2 part[2][Shape::kWorkers / 32], slot[2][kMaxCluster];
  float red[Shape::kWorkers / 32];
  uint64_t full[Shape::kRing], empty[Shape::kRing];
  uint64_t meta_full[2], meta_empty[2], exchange[2], tokens_read;
};
static_assert(sizeof(StreamSmem<Wide>) + 128 + 1024 <= 233472 &&
                  2 * (sizeof(StreamSmem<Pair>) + 128 + 1024) <= 233472 &&
                  4 * (sizeof(StreamSmem<Quad>) + 128 + 1024) <= 233472,
              "policy stream shared memory");

__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

template <typename T, int kMode, typename Shape>
__global__ void __launch_bounds__(Shape::kWorkers + 64, Shape::kPerSm)
policy_stream_kernel(const PolicyArgs a, long long rows, int groups) {
  using V = Vec<T>;
  constexpr int N = V::N, kRing = Shape::kRing, kChunk = Shape::kChunk;
  constexpr int kWorkers = Shape::kWorkers;
  constexpr int kWorkerWarps = kWorkers / 32, kPerThread = kChunk / kWorkers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  StreamSmem<Shape>& sm = *reinterpret_cast<StreamSmem<Shape>*>(base);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.C, rank = C > 1 ? (int)(blockIdx.x % C) : 0;
  const long long first = blockIdx.x / C;
  // (each of more targets than the list holds keeps its row's workers for a microsecond or two)
  const uint64_t wait_ns = kWaitNs + 4000ull * (uint64_t)a.n_tokens;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWorkerWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.meta_full[i], 1);
      mbar_init(&sm.meta_empty[i], kWorkerWarps + 1);
      mbar_init(&sm.exchange[i], 1);
    }
    mbar_init(&sm.tokens_read, C);
    fence_mbar_init();
  }
  __syncthreads();
  if (C > 1) cg::this_cluster().sync();

  // Vectors of a row as in the kernel above; those of this CTA, and of them the whole ones.
  struct Slice {
    int ph, lo, hi, whole_lo, whole_hi;
  };
  auto slice_of = [&](long long r) {
    Slice s;
    const T* row = static_cast<const T*>(a.logits) + r * a.ld;
    s.ph = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int nv = (a.vocab + s.ph + N - 1) / N, per = (nv + C - 1) / C;
    s.lo = min(rank * per, nv);
    s.hi = min(s.lo + per, nv);
    s.whole_lo = s.lo == 0 && s.ph > 0 ? min(1, s.hi) : s.lo;
    s.whole_hi = s.hi == nv && (a.vocab + s.ph) % N ? max(s.hi - 1, s.whole_lo) : s.hi;
    return s;
  };

  if (warp == kWorkerWarps) {
    // ------------------------------------------------------------------ the ring ---------
    if (lane == 0) {
      bool ok = true;
      unsigned count = 0;
      long long r = first;
      for (unsigned b = 0; ok && r < rows; ++b) {
        ok = mbar_wait(&sm.meta_full[b & 1], (b >> 1) & 1, wait_ns);
        for (int i = 0; ok && i < kMetaRows && r < rows; ++i, r += groups) {
          if (sm.meta[b & 1][i].k == 0) continue;
          const Slice s = slice_of(r);
          const T* src = static_cast<const T*>(a.logits) + r * a.ld - s.ph;
          for (int v = s.whole_lo; ok && v < s.whole_hi; v += kChunk, ++count) {
            const int at = count % kRing;
            ok = mbar_wait(&sm.empty[at], ((count / kRing) & 1) ^ 1, wait_ns);
            if (!ok) break;
            const uint32_t bytes = (uint32_t)min(kChunk, s.whole_hi - v) * 16u;
            mbar_expect_tx(&sm.full[at], bytes);
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    smem_u32(sm.ring[at])),
                "l"(src + (long long)v * N), "r"(bytes), "r"(smem_u32(&sm.full[at]))
                : "memory");
          }
        }
        if (ok) mbar_arrive(&sm.meta_empty[b & 1]);
      }
      if (!ok) report(PG_ERR_TIMEOUT);
      // Leave no copy in flight.
      for (unsigned j = count > kRing ? count - kRing : 0; j < count; ++j)
        mbar_wait(&sm.full[j % kRing], (j / kRing) & 1, wait_ns);
    }
  } else if (warp == kWorkerWarps + 1) {
    // ------------------------------------------------------------------ tokens -----------
    bool ok = true;
    long long r = first + (long long)lane * groups;
    for (unsigned b = 0; ok && first + (long long)b * kMetaRows * groups < rows; ++b) {
      RowMeta m{0, 0, -1, 0.f, 0.f, 0.f, 0.f, 1.f};
      if (r < rows) {
        long long t0 = r, t1 = r + 1;
        if (a.row_starts) {
          const long long s0 = a.row_starts[r], s1 = a.row_starts[r + 1];
          t0 = min(max(s0, 0ll), a.n_tokens);
          t1 = min(max(s1, t0), a.n_tokens);
          const bool loose = (r == 0 && s0 != 0) || (r == rows - 1 && s1 != a.n_tokens);
          if ((t0 != s0 || t1 != s1 || loose) && rank == 0) report(PG_ERR_DEVICE);
        }
        m.t0 = (int)t0;
        m.k = (int)(t1 - t0);
        if (m.k == 1) {
          const int y = a.tokens[t0];
          if (a.adv) {
            m.adv = a.adv[t0];
            if (a.old_lp) m.old = a.old_lp[t0];
            if (a.ref_lp) m.ref = a.ref_lp[t0];
            if (a.weights) m.w = a.weights[t0];
          }
          if (y >= a.vocab && rank == 0) report(PG_ERR_DEVICE);
          m.y = y >= 0 && y < a.vocab ? y : -1;
          if (m.y >= 0) m.x = to_f(static_cast<const T*>(a.logits)[r * a.ld + m.y]);
        }
      }
      ok = warp_wait(&sm.meta_empty[b & 1], ((b >> 1) & 1) ^ 1, wait_ns);
      if (!ok) break;
      sm.meta[b & 1][lane] = m;
      warp_arrive(&sm.meta_full[b & 1]);
      r += (long long)kMetaRows * groups;
    }
    if (!ok && lane == 0) report(PG_ERR_TIMEOUT);
  } else {
    // ------------------------------------------------------------------ the rows ---------
    // (ok: this thread's waits; all: every thread's, by which they leave together.)
    bool ok = true, all = true;
    unsigned count = 0, live = 0, shared_rows = 0;
    long long r = first;
    for (unsigned b = 0; all && r < rows; ++b) {
      ok = ok && mbar_wait(&sm.meta_full[b & 1], (b >> 1) & 1, wait_ns);
      all = named_bar_and(1, kWorkers, ok);
      for (int i = 0; all && i < kMetaRows && r < rows; ++i, r += groups) {
        const RowMeta meta = sm.meta[b & 1][i];
        const Slice s = slice_of(r);
        const T* row = static_cast<const T*>(a.logits) + r * a.ld;
        T* drow = kMode == kForward ? nullptr : static_cast<T*>(a.dlogits) + r * a.ldd;
        const bool same_phase =
            kMode != kForward && (int)((reinterpret_cast<uintptr_t>(drow) & 15) / sizeof(T)) == s.ph;
        auto store = [&](int v, const float (&f)[N]) {
          const int at = v * N - s.ph;
          if (same_phase && at >= 0 && at + N <= a.vocab) {
            *reinterpret_cast<uint4*>(drow + at) = V::pack(f);
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (at + e >= 0 && at + e < a.vocab) drow[at + e] = (T)f[e];
          }
        };
        auto zero_row = [&] {
          float f[N];
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] = 0.f;
          for (int v = s.lo + tid; v < s.hi; v += kWorkers) store(v, f);
        };
        if (meta.k == 0) {
          if (rank == 0 && tid == 0) a.lse[r] = 0.f;
          if (kMode != kForward) zero_row();
          continue;
        }
        // The row's first and last vector, where they are not whole: threads 0 and 32 have them.
        const int edge_v = tid == 0 && s.whole_lo > s.lo  ? s.lo
                           : tid == 32 && s.whole_hi < s.hi ? s.hi - 1
                                                            : -1;
        float edge[N];
        if (edge_v >= 0)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const int at = edge_v * N - s.ph + e;
            edge[e] = at >= 0 && at < a.vocab ? to_f(row[at]) : -INFINITY;
          }

        // First pass.
        // (Exponents are one product and sum while the reference's own product is below kExact: rounding that
        // product, mc, multiplies all terms by 2^d, d = m c - mc, at most half.  The sum is kept times 2^d, and
        // freed of it at the end, so that a log-probability knows nothing of what a row's logits have in common.)
        const float by = meta.k == 1 && meta.y >= 0 && meta.x > -INFINITY ? meta.x : -INFINITY;
        float m = by;
        uint64_t s2 = f2_pack(0.f, 0.f);
        const uint64_t c2 = f2_pack(a.c, a.c);
        auto excess = [&](float x) {         // d of the reference x
          const float xc = x * a.c;
          return fabsf(xc) < kExact ? fmaf(x, a.c, -xc) : 0.f;
        };
        auto raise = [&](float top) {        // a new maximum for this thread's sum
          const float f = m == -INFINITY ? 0.f : ex2(a.c * (m - top) + (excess(top) - excess(m)));
          s2 = f2_mul(s2, f2_pack(f, f));
          m = top;
        };
        unsigned at = count;
        for (int v0 = s.whole_lo; v0 < s.whole_hi; v0 += kChunk, ++at) {
          const int slot = at % kRing;
          ok = ok && mbar_wait(&sm.full[slot], (at / kRing) & 1, wait_ns);
          uint4 x[kPerThread];
          const uint4* src = sm.ring[slot] + tid;
          if (v0 + kChunk <= s.whole_hi) {
#pragma unroll
            for (int u = 0; u < kPerThread; ++u) x[u] = src[u * kWorkers];
          } else {
#pragma unroll
            for (int u = 0; u < kPerThread; ++u)
              x[u] = v0 + u * kWorkers + tid < s.whole_hi ? src[u * kWorkers] : V::lowest();
          }
          const uint64_t before = s2;
          const float mc = m * a.c;
          bool done = false;
          if (fabsf(mc) < kExact) {
            const uint64_t r2 = f2_pack(-mc, -mc);
#pragma unroll
            for (int u = 0; u < kPerThread; ++u)
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                float b0, b1;
                f2_unpack(f2_fma(f2_pack(V::get(x[u], e), V::get(x[u], e + 1)), c2, r2), b0, b1);
                s2 = f2_add(s2, f2_pack(ex2(b0), ex2(b1)));
              }
            float s0, s1;
            f2_unpack(s2, s0, s1);
            done = s0 < 0x1p100f && s1 < 0x1p100f;
          }
          if (!done) {
            s2 = before;
            float top = V::vmax(x[0]);
#pragma unroll
            for (int u = 1; u < kPerThread; ++u) top = fmaxf(top, V::vmax(x[u]));
            if (top > m && a.c * (top - m) > kLag) raise(top);
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t r2 = f2_pack(-ref, -ref);
            uint64_t t2 = f2_pack(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < kPerThread; ++u)
#pragma unroll
              for (int e = 0; e < N; e += 2) {
                float b0, b1;
                f2_unpack(f2_mul(f2_add(f2_pack(V::get(x[u], e), V::get(x[u], e + 1)), r2), c2), b0, b1);
                t2 = f2_add(t2, f2_pack(ex2(b0), ex2(b1)));
              }
            const float up = ex2(excess(m));
            s2 = f2_fma(t2, f2_pack(up, up), s2);
          }
          if (kMode == kForward) warp_arrive(&sm.empty[slot]);
        }
        if (edge_v >= 0) {
          float top = edge[0];
#pragma unroll
          for (int e = 1; e < N; ++e) top = fmaxf(top, edge[e]);
          if (top > m && a.c * (top - m) > kLag) raise(top);
          const float ref = m == -INFINITY ? 0.f : m, up = ex2(excess(m));
#pragma unroll
          for (int e = 0; e < N; ++e) s2 = f2_add(s2, f2_pack(ex2(a.c * (edge[e] - ref)) * up, 0.f));
        }
        float s0, s1;
        f2_unpack(s2, s0, s1);
        const float sum_m = (s0 + s1) * ex2(-excess(m));
        // (maximum, sum) of a warp, of the CTA, of the cluster: the largest first, then the sums against it.
        auto meet = [&](float2 v, int width) {
          float top = v.x, sum = v.y;
          if (!__all_sync(0xffffffffu, v.x == by)) {
            for (int o = width / 2; o > 0; o >>= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (v.x != -INFINITY) sum *= ex2(a.c * (v.x - top));
          }
          for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          return make_float2(top, sum);
        };
        float2 ms = meet(make_float2(m, sum_m), 32);
        const int side = live & 1;
        if (lane == 0) sm.part[side][warp] = ms;
        all = named_bar_and(1, kWorkers, ok);
        if (!all) break;
        ms = meet(sm.part[side][lane % kWorkerWarps], kWorkerWarps);
        if (C > 1) {
          if (tid == 0) mbar_expect_tx(&sm.exchange[side], 8u * (uint32_t)C);
          if (tid < C)
            asm volatile(
                "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                    remote(&sm.slot[side][rank], tid)),
                "r"(__float_as_uint(ms.x)), "r"(__float_as_uint(ms.y)),
                "r"(remote(&sm.exchange[side], tid))
                : "memory");
          ok = cluster_wait(&sm.exchange[side], (live >> 1) & 1, wait_ns) && ok;
          ms = sm.slot[side][0];
          for (int j = 1; j < C; ++j) ms = join(ms, sm.slot[side][j], a.c);
        }
        ++live;
        const bool dead = ms.x == -INFINITY && ms.y == 0.f;
        const float rx = ms.x == -INFINITY ? 0.f : ms.x, ls = log2f(ms.y);
        auto logprob = [&](float z) { return dead ? -INFINITY : fmaf(z - rx, a.c, -ls) * kLn2; };
        const bool writer = rank == 0 && tid == 0;
        if (writer) a.lse[r] = dead ? -INFINITY : fmaf(rx, a.inv_t, ls * kLn2);
        float g_sum = 0.f;
        bool any;
        const bool listed = kMode == kStep && meta.k > 1 && meta.k <= Shape::kListed;
        if (meta.k == 1) {
          if (kMode == kStep || writer) {
            const float lp = meta.y >= 0 ? logprob(meta.x) : 0.f;
            Term t{0.f, 0.f};
            if (meta.y >= 0 && a.adv)
              t = term_of(a, lp, dead, meta.old, meta.ref, meta.adv, meta.w);
            g_sum = t.grad;
            if (writer) {
              a.logprobs[meta.t0] = lp;
              if (a.adv) {
                a.token_loss[meta.t0] = t.loss;
                a.token_grad[meta.t0] = t.grad;
              }
            }
          }
          any = g_sum != 0.f;
        } else {
          // Every CTA works out all tokens; the first one stores them.
          bool nz = false;
          if (kMode == kStep || rank == 0)
            for (int j = tid; j < meta.k; j += kWorkers) {
              const long long n = (long long)meta.t0 + j;
              const int y = a.tokens[n];
              if (y >= a.vocab && rank == 0) report(PG_ERR_DEVICE);
              Term t{0.f, 0.f};
              float lp = 0.f, z = 0.f;
              if (y >= 0 && y < a.vocab) {
                z = to_f(row[y]);
                lp = logprob(z);
                if (a.adv) t = term(a, n, lp, dead);
              }
              if (listed) {
                const int v = (y + s.ph) / N;
                sm.list[j] = Target{y >= 0 && y < a.vocab && v >= s.lo && v < s.hi ? y : -1, t.grad, z};
              }
              if (rank == 0) {
                a.logprobs[n] = lp;
                if (a.adv) {
                  a.token_loss[n] = t.loss;
                  a.token_grad[n] = t.grad;
                }
              }
              g_sum += t.grad;
              nz |= t.grad != 0.f;
            }
          if (kMode == kStep) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) g_sum += __shfl_xor_sync(0xffffffffu, g_sum, o);
            if (lane == 0) sm.red[warp] = g_sum;
            any = !named_bar_and(1, kWorkers, !nz);
            g_sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWorkerWarps; ++w) g_sum += sm.red[w];
            if (C > 1) {
              // The row may be overwritten once every CTA has read its tokens' logits.
              if (tid < C)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 remote(&sm.tokens_read, tid))
                             : "memory");
              ok = cluster_wait(&sm.tokens_read, shared_rows & 1, wait_ns) && ok;
              ++shared_rows;
            }
          }
        }
        if (kMode == kForward) {
          count = at;
          continue;
        }
        // Second pass.
        // (the factor 2^d of its exponents, as in the first pass, is taken back by the coefficient)
        const float rc = rx * a.c;
        const bool in_range = fabsf(rc) < kExact;
        const float coef = -(g_sum * a.inv_t) / ms.y * ex2(-excess(rx));
        const uint64_t r2 = f2_pack(-rx, -rx), k2 = f2_pack(coef, coef);
        const int y_at = meta.k == 1 && meta.y >= 0 ? meta.y + s.ph : INT_MIN / 2;
        const uint64_t rc2 = f2_pack(-rc, -rc);
        auto gradient = [&](int v, const float (&z)[N], float (&f)[N]) {
          if (in_range) {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              float b0, b1;
              f2_unpack(f2_fma(f2_pack(z[e], z[e + 1]), c2, rc2), b0, b1);
              f2_unpack(f2_mul(f2_pack(ex2(b0), ex2(b1)), k2), f[e], f[e + 1]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              float b0, b1;
              f2_unpack(f2_mul(f2_add(f2_pack(z[e], z[e + 1]), r2), c2), b0, b1);
              f2_unpack(f2_mul(f2_pack(ex2(b0), ex2(b1)), k2), f[e], f[e + 1]);
            }
          }
          if (meta.k == 1) {
            const int d = y_at - v * N;
            if ((unsigned)d < (unsigned)N) {
#pragma unroll
              for (int e = 0; e < N; ++e)
                if (d == e) f[e] = fmaf(g_sum, a.inv_t, f[e]);
            }
          } else if (!listed) {
            for (int j = 0; j < meta.k; ++j) {
              const long long n = (long long)meta.t0 + j;
              const int y = a.tokens[n], d = y + s.ph - v * N;
              if (y >= 0 && y < a.vocab && d >= 0 && d < N) {
#pragma unroll
                for (int e = 0; e < N; ++e)
                  if (d == e) f[e] = fmaf(term(a, n, logprob(z[e]), dead).grad, a.inv_t, f[e]);
              }
            }
          }
        };
        if (!any) zero_row();
        at = count;
        for (int v0 = s.whole_lo; v0 < s.whole_hi; v0 += kChunk, ++at) {
          const int slot = at % kRing;
          if (any) {
            const uint4* src = sm.ring[slot] + tid;
#pragma unroll
            for (int u = 0; u < kPerThread; ++u) {
              const int v = v0 + u * kWorkers + tid;
              if (v >= s.whole_hi) break;
              const uint4 x = src[u * kWorkers];
              float z[N], f[N];
#pragma unroll
              for (int e = 0; e < N; ++e) z[e] = V::get(x, e);
              gradient(v, z, f);
              if (same_phase) *reinterpret_cast<uint4*>(drow + (v * N - s.ph)) = V::pack(f);
              else store(v, f);
            }
          }
          warp_arrive(&sm.empty[slot]);
        }
        count = at;
        if (any && edge_v >= 0) {
          float f[N];
          gradient(edge_v, edge, f);
          store(edge_v, f);
        }
        if (listed && any) {
          all = named_bar_and(1, kWorkers, ok);
          if (!all) break;
          add_targets(drow, sm.list, meta.k, tid, kWorkers, a.inv_t, [&](float z) {
            return ex2(in_range ? fmaf(z, a.c, -rc) : (z - rx) * a.c) * coef;
          });
        }
      }
      if (all) warp_arrive(&sm.meta_empty[b & 1]);
    }
    if (!ok) report(PG_ERR_TIMEOUT);
  }
  // No CTA leaves while another may store to it.
  __syncwarp();
  if (C > 1) cg::this_cluster().sync();
}

// loss = sum of the tokens' losses: one block, partial sums in fp64 in a fixed order.  It starts under the
// kernel before it.
__global__ void __launch_bounds__(1024)
policy_sum_kernel(const float* token_loss, long long n, float* loss) {
  __shared__ double red[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s = 0;
  for (long long i = threadIdx.x; i < n; i += 1024) s += (double)token_loss[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = red[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) *loss = (float)s;
  }
}

// The kernel whose threads hold the CTA's `per` vectors, or as many as pay off: only the step reads them
// twice.
template <typename T, int kMode>
auto kernel_for(int64_t per) {
  if (per <= kThreads) return policy_kernel<T, 1, kMode>;
  if constexpr (kMode == kBackward) {
    return policy_kernel<T, 4, kMode>;
  } else if constexpr (kMode == kForward) {
    return per <= kThreads * 4 ? policy_kernel<T, 4, kMode> : policy_kernel<T, 8, kMode>;
  } else {
    return per <= kThreads * 2   ? policy_kernel<T, 2, kMode>
           : per <= kThreads * 4 ? policy_kernel<T, 4, kMode>
           : per <= kThreads * 8 ? policy_kernel<T, 8, kMode>
                                 : policy_kernel<T, 16, kMode>;
  }
}

// How many clusters of 2, 4 or 8 CTAs of a kernel run at once, asked once per device.
class ClustersPerDevice {
 public:
  template <typename F>
  pg_status get(int C, F&& ask, int* n) {
    int dev = 0;
    pg_status st = cuda_check(cudaGetDevice(&dev), "current device");
    if (st != PG_OK) return st;
    std::atomic<int>* kept = dev >= 0 && dev < 64 ? &kept_[dev][C == 2 ? 0 : C == 4 ? 1 : 2] : nullptr;
    *n = kept ? kept->load(std::memory_order_relaxed) : 0;
    if (*n > 0) return PG_OK;
    st = cuda_check(ask(n), "policy loss clusters");
    if (st != PG_OK) return st;
    *n = std::max(*n, 1);
    if (kept) kept->store(*n, std::memory_order_relaxed);
    return PG_OK;
  }

 private:
  std::atomic<int> kept_[64][3] = {};
};

// CTAs per row of the streaming kernel with this shape, 0 if rows do not fit it; more than a row needs while the
// rows alone do not fill the GPU (forward of 64 rows of 256 KB: two CTAs per row 10.3 us, one 11.0).
template <int kMode, typename Shape>
int stream_cluster(int64_t nv, int64_t rows) {
  int C = 1;
  if (kMode == kStep)
    while (C < kMaxCluster && (nv + C - 1) / C > (int64_t)Shape::kRing * Shape::kChunk) C *= 2;
  if (kMode == kStep && (nv + C - 1) / C > (int64_t)Shape::kRing * Shape::kChunk) return 0;
  while (C < kMaxCluster && rows * C * 2 <= kSMs) C *= 2;
  return C;
}

template <typename T, int kMode, typename Shape>
pg_status launch_stream(int64_t rows, int C, PolicyArgs a, cudaStream_t s) {
  a.C = C;
  auto kern = policy_stream_kernel<T, kMode, Shape>;
  const size_t smem = sizeof(StreamSmem<Shape>) + 128;
  static OncePerDevice once;
  pg_status st = once.run([&] { return allow_smem(kern, smem, "policy stream smem attributes"); });
  if (st != PG_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3(Shape::kWorkers + 64);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  // As many clusters as run at once (an SM whose neighbours are taken has no place for one), each with its
  // share of the rows.
  static ClustersPerDevice at_once;
  int most = kSMs * Shape::kPerSm;
  if (C > 1) st = at_once.get(C, [&](int* n) { return cudaOccupancyMaxActiveClusters(n, kern, &cfg); }, &most);
  if (st != PG_OK) return st;
  const int64_t groups = std::min<int64_t>(rows, most);
  cfg.gridDim = dim3((unsigned)(groups * C));
  prof_begin(PG_KERNEL_POLICY, s);
  st = cuda_check(cudaLaunchKernelEx(&cfg, kern, a, (long long)rows, (int)groups),
                  "policy loss stream launch");
  prof_end(PG_KERNEL_POLICY, s);
  return st;
}

// Which kernel: at few bytes the streaming kernel's setup costs 2-4 us.  Loss and gradient of rows of 64 KB that
// lie in L2, registers against streaming: 4 MB 9.9 and 12.0 us, 8 MB 16.7 and 12.2, 16 MB 23.1 and 13.8; of rows of
// 256 KB, eight CTAs each in registers: 8 MB 13.6 and 12.0, 16 MB 22.0 and 14.3.  The forward, registers against streaming:
// rows of 32 KB 8 MB 12.9 and 9.2, of 64 KB 8 MB 9.3 and 9.4, of 256 KB 8 MB 9.2 and 10.0, 12 MB 9.9 and 10.7, 16 MB 11.7
// and 11.0, of 200 KB (fp32) 8 MB 9.6 and 10.2, 12 MB 11.2 and 10.3.  Which shape (512 MB of bf16
// logits, us; memory alone: 158 for the step, 79 for the forward):
//   row             40 KB  48 KB  64 KB  80 KB  100 KB  128 KB  256 KB
//   step    Quad      212    247    205    208     247     209     224
//           Pair      207    219    204    182     214     211     222
//           Wide      293    260    210    213     196     175     185
//   forward Quad                     92             88      89      93
//           Wide                    108            104      87      89
constexpr int64_t kWideStep = 100 << 10, kPairStep = 48 << 10, kWideForward = 128 << 10,
                  kStreamBytes = 8 << 20, kStreamWideForward = 12 << 20;

template <typename T, int kMode>
pg_status launch(int64_t rows, PolicyArgs a, cudaStream_t s) {
  if constexpr (kMode != kBackward) {
    const int64_t bytes = (int64_t)a.vocab * sizeof(T), vecs = bytes / 16 + 2;
    const bool wide = bytes >= (kMode == kStep ? kWideStep : kWideForward);
    const bool pair = kMode == kStep && !wide && bytes >= kPairStep;
    const int C = wide   ? stream_cluster<kMode, Wide>(vecs, rows)
                  : pair ? stream_cluster<kMode, Pair>(vecs, rows)
                         : stream_cluster<kMode, Quad>(vecs, rows);
    if (C > 0 && rows * bytes >= (kMode == kForward && wide ? kStreamWideForward : kStreamBytes)) {
      if (wide) return launch_stream<T, kMode, Wide>(rows, C, a, s);
      if constexpr (kMode == kStep)
        if (pair) return launch_stream<T, kMode, Pair>(rows, C, a, s);
      return launch_stream<T, kMode, Quad>(rows, C, a, s);
    }
  }
  // CTAs per row, at most a cluster of eight: enough that a thread holds eight vectors (32 KB per CTA), and
  // more while the rows alone do not fill the GPU and a thread has a vector.  The backward, which holds nothing, goes
  // by the latter alone: two CTAs per SM (eight CTAs per row against one: 4096 rows of 131072 bf16 347 and 318 us,
  // 4096 of 50001 158 and 133, but 64 of 131072 8 and 12; one, two, four CTAs per SM: 256 rows 33, 26 and 27 us, 512 of
  // 50001 19, 19 and 21).
  const int64_t nv = ((int64_t)a.vocab * sizeof(T) + 31) / 16;
  int C = 1;
  while (C < kMaxCluster && nv > (int64_t)C * kThreads &&
         (kMode == kBackward ? rows * C < 2 * kSMs : nv > (int64_t)C * kThreads * 8 || rows * C * 2 <= kSMs))
    C *= 2;
  a.C = C;
  const int64_t per = (nv + C - 1) / C;
  auto kern = kernel_for<T, kMode>(per);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  prof_begin(PG_KERNEL_POLICY, s);
  const pg_status st = cuda_check(cudaLaunchKernelEx(&cfg, kern, a), "policy loss launch");
  prof_end(PG_KERNEL_POLICY, s);
  return st;
}

pg_status launch_sum(const PolicyArgs& a, float* loss, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  prof_begin(PG_KERNEL_POLICY, s);
  const pg_status st = cuda_check(
      cudaLaunchKernelEx(&cfg, policy_sum_kernel, (const float*)a.token_loss, a.n_tokens, loss),
      "policy loss sum launch");
  prof_end(PG_KERNEL_POLICY, s);
  return st;
}

template <int kMode>
pg_status launch_typed(pg_dtype dtype, int64_t rows, const PolicyArgs& a, cudaStream_t s) {
  return dtype == PG_F32 ? launch<float, kMode>(rows, a, s) : launch<__nv_bfloat16, kMode>(rows, a, s);
}

// What both calls ask of the rows.
pg_status check_rows(const char* who, pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits,
                     int64_t ld, int64_t n_tokens, const int32_t* row_starts, const int32_t* tokens,
                     float temperature, const void* dlogits, int64_t ldd) {
  if ((dtype != PG_F32 && dtype != PG_BF16) || rows < 1 || rows > (1 << 27) || vocab < 1 ||
      vocab >= (1 << 30) || ld < vocab || n_tokens < 0 || n_tokens >= (1ll << 31)) {
    set_error("%s: needs dtype f32 or bf16, 1 <= rows <= 2^27, 1 <= vocab < 2^30, ld >= vocab and "
              "0 <= n_tokens < 2^31", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!row_starts && n_tokens != rows) {
    set_error("%s: without row_starts every row has one token", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!(temperature >= 0x1p-126f) || !(temperature <= 3.4e38f)) {
    set_error("%s: temperature must be finite and at least 2^-126", who);
    return PG_ERR_INVALID_ARG;
  }
  const uintptr_t unit = dtype == PG_F32 ? 4 : 2;
  if (!logits || (n_tokens > 0 && !tokens) || reinterpret_cast<uintptr_t>(logits) % unit ||
      reinterpret_cast<uintptr_t>(dlogits) % unit || (dlogits && ldd < vocab) ||
      (dlogits == logits && ldd != ld)) {
    set_error("%s: logits and tokens must be non-NULL, logits and dlogits aligned to their type, ldd >= "
              "vocab, and ldd = ld when dlogits is logits", who);
    return PG_ERR_INVALID_ARG;
  }
  return PG_OK;
}

bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 4) return false;
  return true;
}

}  // namespace

pg_status read_status_policy(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_policy, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_policy, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg

using namespace pg;

extern "C" {

pg_status pg_policy_loss(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits, int64_t ld,
                         int64_t n_tokens, const int32_t* row_starts, const int32_t* tokens,
                         const float* old_logprobs, const float* ref_logprobs,
                         const float* advantages, const float* weights, const pg_policy_opts* opts,
                         float* lse, float* logprobs, float* token_loss, float* token_grad,
                         float* loss, void* dlogits, int64_t ldd, pg_stream_t stream) {
  const char* who = "pg_policy_loss";
  if (!opts) {
    set_error("%s: opts is NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  pg_status st = check_rows(who, dtype, rows, vocab, logits, ld, n_tokens, row_starts, tokens,
                            opts->temperature, dlogits, ldd);
  if (st != PG_OK) return st;
  if (!(opts->clip_low >= 0.f) || !(opts->clip_high >= 0.f) || !(opts->kl_coef >= 0.f) ||
      !(opts->kl_coef <= 3.4e38f)) {
    set_error("%s: clip_low, clip_high and kl_coef must be >= 0, kl_coef finite", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!lse || (n_tokens > 0 && !logprobs)) {
    set_error("%s: lse and logprobs must be non-NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  const bool scored = advantages != nullptr || (n_tokens == 0 && loss != nullptr);
  if (scored ? (!loss || (n_tokens > 0 && (!token_loss || !token_grad)))
             : (old_logprobs || ref_logprobs || weights || token_loss || token_grad || loss || dlogits)) {
    set_error("%s: with advantages token_loss, token_grad and loss must be non-NULL, without them those, "
              "old_logprobs, ref_logprobs, weights and dlogits must be NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!aligned4({row_starts, tokens, old_logprobs, ref_logprobs, advantages, weights, lse, logprobs,
                 token_loss, token_grad, loss})) {
    set_error("%s: arrays per row and per token must be 4-byte aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  PolicyArgs a{};
  a.logits = logits;
  a.dlogits = dlogits;
  a.ld = ld;
  a.ldd = ldd;
  a.n_tokens = n_tokens;
  a.row_starts = row_starts;
  a.tokens = tokens;
  a.old_lp = old_logprobs;
  a.ref_lp = opts->kl_coef > 0.f ? ref_logprobs : nullptr;
  a.adv = advantages;
  a.weights = weights;
  a.lse = lse;
  a.logprobs = logprobs;
  a.token_loss = token_loss;
  a.token_grad = token_grad;
  a.vocab = vocab;
  a.inv_t = (float)(1.0 / (double)opts->temperature);
  a.c = (float)(1.4426950408889634 / (double)opts->temperature);
  a.lo = 1.f - opts->clip_low;
  a.hi = 1.f + opts->clip_high;
  a.kl = opts->kl_coef;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = dlogits ? launch_typed<kStep>(dtype, rows, a, s) : launch_typed<kForward>(dtype, rows, a, s);
  if (st == PG_OK && loss) st = launch_sum(a, loss, s);
  return st;
}

pg_status pg_policy_loss_bwd(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits,
                             int64_t ld, int64_t n_tokens, const int32_t* row_starts,
                             const int32_t* tokens, float temperature, const float* lse,
                             const float* token_grad, const float* grad_output, void* dlogits,
                             int64_t ldd, pg_stream_t stream) {
  const char* who = "pg_policy_loss_bwd";
  pg_status st = check_rows(who, dtype, rows, vocab, logits, ld, n_tokens, row_starts, tokens,
                            temperature, dlogits, ldd);
  if (st != PG_OK) return st;
  if (!dlogits || !lse || (n_tokens > 0 && !token_grad) ||
      !aligned4({row_starts, tokens, lse, token_grad, grad_output})) {
    set_error("%s: lse, token_grad and dlogits must be non-NULL, arrays per row and per token 4-byte "
              "aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  PolicyArgs a{};
  a.logits = logits;
  a.dlogits = dlogits;
  a.ld = ld;
  a.ldd = ldd;
  a.n_tokens = n_tokens;
  a.row_starts = row_starts;
  a.tokens = tokens;
  a.lse = const_cast<float*>(lse);
  a.token_grad = const_cast<float*>(token_grad);
  a.grad_output = grad_output;
  a.vocab = vocab;
  a.inv_t = (float)(1.0 / (double)temperature);
  a.c = (float)(1.4426950408889634 / (double)temperature);
  return launch_typed<kBackward>(dtype, rows, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
