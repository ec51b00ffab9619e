// The rollout's paged cache and attention step: append with rotation, the plan of the attention
// step, its fp32-arithmetic kernel and the merge of partial results.
#include <math.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "pg_decode.h"
#include "pg_e4m3.cuh"
#include "pg_headrows.cuh"

namespace pg {

using namespace headrows;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 152;

__device__ int s_status_rollout = 0;

__device__ __forceinline__ void report(int code) { atomicCAS(&s_status_rollout, 0, code); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool page_size_ok(int32_t ps) {
  return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256;
}

// ---------------------------------------------------------------------------------------------
// Append.  A row is one head of one token: the heads of q, then of k, then of v.  As in the q / k norm
// a warp takes a token (or, with few tokens, a share of its rows), so the page table is read and the
// angles are computed once for all its rows.  Bound by memory, and for one token per response
// by the latency of a launch and two dependent reads (index, page).  The rows' loads are issued before the
// page is looked up and the angles are computed.  The frequencies go through shared memory: lanes reading
// different words of a parameter take turns.  8 x 2048 tokens of 8 heads take 28.8 us (4.7 TB/s), 33 us
// with the frequencies read from the parameter, 43 us with the lookup first and half as many rows in
// flight; without a rotation 27 us.  One token of 16 responses 3.6 us (as a node of a graph).
// ---------------------------------------------------------------------------------------------
constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;
template <typename T>
constexpr int kAppendRows = sizeof(T) == 2 ? 8 : 4;   // rows in flight per group of lanes

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
cache_append_kernel(const T* q, long long ldq, T* q_out, const T* __restrict__ k, long long ldk,
                    const T* __restrict__ v, long long ldv, const int32_t* __restrict__ positions,
                    const __grid_constant__ RopeFreq f, int rope, T* __restrict__ k_cache,
                    T* __restrict__ v_cache, long long num_pages, int page_size,
                    const int32_t* __restrict__ pages, int num_page_rows, int pages_per_row,
                    long long pages_stride, const int32_t* __restrict__ page_rows,
                    const int32_t* __restrict__ cache_pos, long long N, int Hq, int Hkv, int chunks,
                    int per_chunk) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kAppendRows<T>;
  __shared__ uint64_t turn[D / 2];
  if (rope) {
    if (threadIdx.x < D / 2) turn[threadIdx.x] = f.turn[threadIdx.x];
    __syncthreads();
  }
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const unsigned item = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);   // below 2^31 + kAppendWarps
  const long long n = item / (unsigned)chunks;
  if (n >= N) return;
  const int rows = Hq + 2 * Hkv;
  const int r_begin = (int)(item % (unsigned)chunks) * per_chunk, r_end = min(r_begin + per_chunk, rows);
  const int cp = cache_pos[n];
  const long long table_row = page_rows ? (long long)page_rows[n] : n;
  const int pos = positions ? positions[n] : cp;
  float c[4], s[4];
  long long slot = -1;
  for (int r0 = r_begin; r0 < r_end; r0 += RPW * U) {
    RawRow<T, D> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(r0 + u * RPW + sub, r_end - 1);
      const T* src = r < Hq ? q + n * ldq + (long long)r * D
                            : (r < Hq + Hkv ? k + n * ldk + (long long)(r - Hq) * D
                                            : v + n * ldv + (long long)(r - Hq - Hkv) * D);
      raw[u].load(src, l);
    }
    if (r0 == r_begin) {
      // With the first rows on their way: where the token goes, and its angles.
      if (cp >= 0) {
        const int pi = cp / page_size;
        long long page = -1;
        if (table_row >= 0 && table_row < num_page_rows && pi < pages_per_row)
          page = pages[table_row * pages_stride + pi];
        if (page >= 0 && page < num_pages) slot = page * page_size + cp % page_size;
        else if (lane == 0) report(PG_ERR_DEVICE);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
      }
      if (rope) {
        Angles<D> a;
        a.init(turn, lane);
        a.at(pos, lane, c, s);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r >= r_end) continue;
      Row<T, D> x;
      x.from(raw[u]);
      if (r < Hq + Hkv) x.rotate(c, s);
      if (r < Hq) {
        x.store(q_out + ((size_t)n * Hq + r) * D, l);
      } else if (slot >= 0) {
        const bool is_k = r < Hq + Hkv;
        const int h = r - Hq - (is_k ? 0 : Hkv);
        x.store((is_k ? k_cache : v_cache) + ((size_t)slot * Hkv + h) * D, l);
      }
    }
  }
}

template <typename T, int D>
pg_status append_t(int64_t n, int Hq, int Hkv, const void* q, int64_t ldq, void* q_out,
                   const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                   float theta, void* kc, void* vc, int64_t num_pages, int page_size,
                   const int32_t* pages, int num_page_rows, int pages_per_row, int64_t pages_stride,
                   const int32_t* page_rows, const int32_t* cache_pos, cudaStream_t s) {
  constexpr int kStep = 256 / D;
  const int rows = Hq + 2 * Hkv, steps = (rows + kStep - 1) / kStep;
  // As for the q / k norm: one warp per token once the tokens fill the GPU, else the rows are shared.
  const int want = (int)std::min<int64_t>(steps, std::max<int64_t>(1, (int64_t)kSMs * 32 / n));
  const int per = (steps + want - 1) / want * kStep;
  const int chunks = (rows + per - 1) / per;
  const int64_t blocks = (n * chunks + kAppendWarps - 1) / kAppendWarps;
  prof_begin(PG_KERNEL_CACHE_APPEND, s);
  cache_append_kernel<T, D><<<(unsigned)blocks, kAppendThreads, 0, s>>>(
      static_cast<const T*>(q), ldq, static_cast<T*>(q_out), static_cast<const T*>(k), ldk,
      static_cast<const T*>(v), ldv, positions, rope_freq(D, theta), theta > 0.f,
      static_cast<T*>(kc), static_cast<T*>(vc), num_pages, page_size, pages, num_page_rows,
      pages_per_row, pages_stride, page_rows, cache_pos, n, Hq, Hkv, chunks, per);
  prof_end(PG_KERNEL_CACHE_APPEND, s);
  return cuda_check(cudaGetLastError(), "cache append launch");
}

// ---------------------------------------------------------------------------------------------
// Attention, fp32 arithmetic: a block takes one response, one key/value head, up to four of its
// query heads and one part of the response's keys (prefix, then own).  Eight lanes share a key (D / 8
// dimensions each), so a block has 16 keys in flight; every key group keeps its own running maximum
// and sum, and the groups meet in shared memory.  It reads the prefix once per response: the plain
// form for fp32 caches, and the independent check of the tensor-core kernels.  A cache in 8 bits
// (C = uint8_t) has a scale per 16 slots and head.
// ---------------------------------------------------------------------------------------------
constexpr int kHeadsPerBlock = 4;
constexpr int kKeyGroups = 16;

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float t[4];
    load4(p + i, t);
    v[i] = t[0]; v[i + 1] = t[1]; v[i + 2] = t[2]; v[i + 3] = t[3];
  }
}

template <int N>
__device__ __forceinline__ void load_n(const uint8_t* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float t[4];
    e4m3::decode4(*reinterpret_cast<const uint32_t*>(p + i), t);
    v[i] = t[0]; v[i + 1] = t[1]; v[i + 2] = t[2]; v[i + 3] = t[3];
  }
}

template <typename T, typename Cache, int D>
__global__ void __launch_bounds__(128)
decode_simt_kernel(const T* __restrict__ q, const Cache* __restrict__ kc,
                   const Cache* __restrict__ vc, const float* __restrict__ k_scales,
                   const float* __restrict__ v_scales, long long num_pages,
                   const int32_t* __restrict__ prefix_pages, long long prefix_stride,
                   const int32_t* __restrict__ own_pages, long long own_stride, const int32_t* __restrict__ own_lens,
                   const DecodeSeq* __restrict__ seqs, int Hq, int Hkv, int page_size,
                   int own_cap, float scale_log2, float* __restrict__ part_o,
                   float* __restrict__ part_lse, int S) {
  constexpr int N = D / 8, HC = kHeadsPerBlock;
  __shared__ float sm_m[kKeyGroups][HC], sm_l[kKeyGroups][HC];
  __shared__ float sm_o[kKeyGroups][HC][D];
  const int hp = Hq / Hkv, nhc = (hp + HC - 1) / HC;
  int x = blockIdx.x;
  const int hc = x % nhc;
  x /= nhc;
  const int kh = x % Hkv, s = x / Hkv;
  const int h0 = kh * hp + hc * HC, nh = min(HC, hp - hc * HC);
  const DecodeSeq sq = seqs[s];
  int own = own_cap > 0 ? own_lens[s] : 0;
  if (own > own_cap) {
    if (threadIdx.x == 0) report(PG_ERR_DEVICE);
    own = own_cap;
  }
  const int total = sq.prefix_len + max(own, 0);
  const int chunk = (total + gridDim.y - 1) / gridDim.y;
  const int lo = (int)min((long long)blockIdx.y * chunk, (long long)total);
  const int hi = min(lo + chunk, total);
  const int lane8 = threadIdx.x & 7, group = threadIdx.x >> 3;
  const unsigned mask = 0xffu << (threadIdx.x & 24);
  float qr[HC][N], acc[HC][N], m[HC], l[HC];
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    load_n<T, N>(q + ((size_t)s * Hq + h0 + min(i, nh - 1)) * D + lane8 * N, qr[i]);
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      qr[i][e] *= scale_log2;
      acc[i][e] = 0.f;
    }
  }
  for (int key = lo + group; key < hi; key += kKeyGroups) {
    const bool pre = key < sq.prefix_len;
    const int idx = pre ? key : key - sq.prefix_len;
    const long long page = pre ? prefix_pages[sq.group * prefix_stride + idx / page_size]
                               : own_pages[s * own_stride + idx / page_size];
    const bool bad = page < 0 || page >= num_pages;
    if (bad) report(PG_ERR_DEVICE);
    const size_t slot = (size_t)(bad ? 0 : page) * page_size + idx % page_size;
    const size_t off = (slot * Hkv + kh) * D + lane8 * N;
    float kv[N], sc[HC], k_scale = 1.f, v_scale = 1.f;
    if constexpr (sizeof(Cache) == 1) {
      k_scale = k_scales[(slot >> 4) * Hkv + kh];
      v_scale = v_scales[(slot >> 4) * Hkv + kh];
      load_n<N>(kc + off, kv);
#pragma unroll
      for (int e = 0; e < N; ++e) kv[e] *= k_scale;
    } else {
      load_n<T, N>(kc + off, kv);
    }
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) d = fmaf(qr[i][e], kv[e], d);
      d += __shfl_xor_sync(mask, d, 1);
      d += __shfl_xor_sync(mask, d, 2);
      d += __shfl_xor_sync(mask, d, 4);
      sc[i] = bad ? 0.f : d;     // a page that is out of range reads as zero keys and values
    }
    if constexpr (sizeof(Cache) == 1) {
      load_n<N>(vc + off, kv);
#pragma unroll
      for (int e = 0; e < N; ++e) kv[e] *= v_scale;
    } else {
      load_n<T, N>(vc + off, kv);
    }
    if (bad)
#pragma unroll
      for (int e = 0; e < N; ++e) kv[e] = 0.f;
#pragma unroll
    for (int i = 0; i < HC; ++i) {
      const float mn = fmaxf(m[i], sc[i]);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[i] - ref), p = exp2f(sc[i] - ref);
      m[i] = mn;
      l[i] = l[i] * corr + p;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[i][e] = fmaf(acc[i][e], corr, p * kv[e]);
    }
  }
#pragma unroll
  for (int i = 0; i < HC; ++i) {
    if (lane8 == 0) {
      sm_m[group][i] = m[i];
      sm_l[group][i] = l[i];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sm_o[group][i][lane8 * N + e] = acc[i][e];
  }
  __syncthreads();
  const size_t rows = (size_t)S * Hq;
  for (int i = threadIdx.x; i < nh * D; i += 128) {
    const int h = i / D, e = i % D;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int g = 0; g < kKeyGroups; ++g) M = fmaxf(M, sm_m[g][h]);
    const float ref = M == -INFINITY ? 0.f : M;
    for (int g = 0; g < kKeyGroups; ++g) {
      const float w = exp2f(sm_m[g][h] - ref);
      L += w * sm_l[g][h];
      O += w * sm_o[g][h][e];
    }
    const size_t row = blockIdx.y * rows + (size_t)s * Hq + h0 + h;
    part_o[row * D + e] = L > 0.f ? O / L : O;   // O is 0 without a key, NaN with a NaN score
    if (e == 0) part_lse[row] = L > 0.f ? M + log2f(L) : (L == 0.f ? -INFINITY : L);
  }
}

// ---------------------------------------------------------------------------------------------
// Merge: o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over a row's partial results, M the
// largest of their log-sum-exps.  The slots in use are the first prefix_parts (of prefix_slots) and
// the last rest_slots.  Four warps per row: warp w adds slots w, w + 4, ..., four loads in flight, and
// the four sums are added in the order of the warps; with few slots one warp does it all.  Bound by the
// latency of its few dependent loads: 512 rows of 27 slots 7 us, 18 us with one warp per row adding
// one slot after another.
// ---------------------------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <typename T, int D, int kMergeWarps>
__global__ void __launch_bounds__(256)
decode_combine_kernel(const float* part_o, const float* part_lse,
                      const DecodeSeq* __restrict__ seqs, T* __restrict__ o,
                      float* __restrict__ lse, int S, int Hq, int prefix_slots, int rest_slots,
                      const int32_t* own_lens, int own_cap, int own_fill) {
  // (part_o and part_lse are not __restrict__: their reads may not move above the wait.)
  constexpr int N = D / 32, U = kMergeWarps == 1 ? 4 : 8, kMergeRows = kMergeThreads / 32 / kMergeWarps;
  __shared__ float red[kMergeRows][kMergeWarps][D], wred[kMergeRows][kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rl = warp / kMergeWarps, wr = warp % kMergeWarps;
  const long long row = (long long)blockIdx.x * kMergeRows + rl;
  const long long rows = (long long)S * Hq;
  const bool live = row < rows;
  const int s = (int)(row / Hq), h = (int)(row % Hq);
  const int np = live && prefix_slots > 0 ? seqs[s].prefix_parts : 0;
  // (own_lens, complete before the first kernel began: of rest_slots those that the response's own keys fill)
  const int rest = live && own_lens
                       ? own_parts_e4m3(min(own_lens[s], own_cap), own_fill, rest_slots).n
                       : rest_slots;
  const int n = live ? np + rest : 0;
  auto slot = [&](int i) { return (size_t)(i < np ? i : prefix_slots + i - np) * rows + row; };
  asm volatile("griddepcontrol.wait;" ::: "memory");     // the partial results
  // The first outputs are read with the log-sum-exps that weigh them: one round trip less.
  float v[U][N];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMergeWarps;
      if (i >= n) continue;
      const float* src = part_o + slot(i) * D + lane * N;
      if (N == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[u][0] = f.x; v[u][1] = f.y; v[u][N - 2] = f.z; v[u][N - 1] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[u][0] = f.x; v[u][1] = f.y;
      }
    }
  };
  load(wr);
  float M = -INFINITY;
  bool nan = false;
  for (int i = lane; i < n; i += 32) {
    const float x = part_lse[slot(i)];
    nan |= x != x;
    M = fmaxf(M, x);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  nan = __any_sync(0xffffffffu, nan);
  const float ref = M == -INFINITY ? 0.f : M;
  float W = 0.f, acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
  for (int i0 = wr; i0 < n; i0 += U * kMergeWarps) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMergeWarps;
      const float w = i < n ? exp2f(part_lse[slot(i)] - ref) : 0.f;
      W += w;
      if (w != 0.f) {            // a slot without keys holds no output
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
      }
    }
    load(i0 + U * kMergeWarps);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) red[rl][wr][lane * N + e] = acc[e];
  if (lane == 0) wred[rl][wr] = W;
  __syncthreads();
  if (!live || wr != 0) return;
#pragma unroll
  for (int i = 1; i < kMergeWarps; ++i) {
    W += wred[rl][i];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] += red[rl][i][lane * N + e];
  }
  if (nan) W = NAN;
  const float inv = W == 0.f ? 0.f : 1.f / W;
  T* dst = o + row * D + lane * N;
#pragma unroll
  for (int e = 0; e < N; ++e) dst[e] = (T)(acc[e] * inv);
  if (lane == 0)
    lse[(size_t)h * S + s] = nan ? NAN : (W > 0.f ? (M + log2f(W)) * kLn2 : -INFINITY);
}

template <typename T, int D>
pg_status combine_t(const DecodeArgs& a, int prefix_slots, int rest_slots,
                    const int32_t* own_lens = nullptr) {
  const pg_decode_plan* p = a.plan;
  const int64_t rows = (int64_t)p->num_seqs * p->heads_q;
  cudaLaunchConfig_t cfg{};
  // One warp per row while a row's slots are four loads in flight or two rounds of them.
  const bool wide = prefix_slots + rest_slots > 8;
  const int block_rows = kMergeThreads / 32 / (wide ? 4 : 1);
  auto kern = wide ? decode_combine_kernel<T, D, 4> : decode_combine_kernel<T, D, 1>;
  cfg.gridDim = dim3((unsigned)((rows + block_rows - 1) / block_rows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  prof_begin(PG_KERNEL_DECODE_COMBINE, a.stream);
  const pg_status st = cuda_check(
      cudaLaunchKernelEx(&cfg, kern, (const float*)a.part_o,
                         (const float*)a.part_lse, decode_seqs(p), static_cast<T*>(a.o), a.lse,
                         (int)p->num_seqs, (int)p->heads_q, prefix_slots, rest_slots,
                         own_lens, (int)(p->own_pages * p->page_size), (int)p->own_slots),
      "decode combine launch");
  prof_end(PG_KERNEL_DECODE_COMBINE, a.stream);
  return st;
}

template <typename T, typename Cache, int D>
pg_status simt_t(const DecodeArgs& a) {
  const pg_decode_plan* p = a.plan;
  const int hp = p->heads_q / p->heads_kv, nhc = (hp + kHeadsPerBlock - 1) / kHeadsPerBlock;
  dim3 grid((unsigned)((int64_t)p->num_seqs * p->heads_kv * nhc), (unsigned)p->simt_splits);
  prof_begin(PG_KERNEL_DECODE, a.stream);
  decode_simt_kernel<T, Cache, D><<<grid, 128, 0, a.stream>>>(
      static_cast<const T*>(a.q), static_cast<const Cache*>(a.k_cache),
      static_cast<const Cache*>(a.v_cache), a.k_scales, a.v_scales, a.num_pages, a.prefix_pages,
      a.prefix_stride, a.own_pages, a.own_stride, a.own_lens, decode_seqs(p), p->heads_q, p->heads_kv,
      p->page_size, p->own_pages * p->page_size, a.scale_log2, a.part_o, a.part_lse, p->num_seqs);
  prof_end(PG_KERNEL_DECODE, a.stream);
  pg_status st = cuda_check(cudaGetLastError(), "decode simt launch");
  if (st != PG_OK) return st;
  return combine_t<T, D>(a, 0, p->simt_splits);
}

// ---------------------------------------------------------------------------------------------
// The plan.
// ---------------------------------------------------------------------------------------------
struct DecodePlan {
  pg_decode_plan p{};
  std::vector<DecodeSeq> seqs;
  std::vector<DecodeItem> items;
};

int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Partial results per query row with own_slots of own keys, and the workspace that holds them.
int64_t decode_slots(const pg_decode_plan& p, int own_slots) {
  return std::max<int64_t>(p.simt_splits, p.prefix_slots + own_slots);
}
size_t decode_bytes(const pg_decode_plan& p, int own_slots) {
  const int64_t rows = decode_slots(p, own_slots) * p.num_seqs * p.heads_q;
  return (size_t)align_up(rows * p.head_dim * 4, 256) + (size_t)align_up(rows * 4, 256);
}

pg_status make_plan(int32_t B, const int32_t* plens, const int32_t* gsizes, pg_dtype dt, int32_t Hq,
                    int32_t Hkv, int32_t d, int32_t ps, int32_t own_pages, DecodePlan* out) {
  const char* who = "pg_plan_decode";
  if (B < 1 || !plens || !gsizes) {
    set_error("%s: num_groups must be >= 1 and arrays non-NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  if ((dt != PG_F32 && dt != PG_BF16) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 65536 ||
      (d != 64 && d != 128)) {
    set_error("%s: dtype f32 or bf16, heads_q a positive multiple of heads_kv, head_dim 64 or 128",
              who);
    return PG_ERR_INVALID_ARG;
  }
  if (!page_size_ok(ps) || own_pages < 0 || (int64_t)own_pages * ps >= (1ll << 30)) {
    set_error("%s: page_size must be 16, 32, 64, 128 or 256 and own_pages * page_size in [0, 2^30)",
              who);
    return PG_ERR_INVALID_ARG;
  }
  int64_t S = 0, max_prefix = 0;
  for (int32_t b = 0; b < B; ++b) {
    if (plens[b] < 0 || plens[b] >= (1 << 30) || gsizes[b] < 0) {
      set_error("%s: group %d has a negative size or a prefix length outside [0, 2^30)", who, b);
      return PG_ERR_INVALID_ARG;
    }
    S += gsizes[b];
    if (gsizes[b] > 0) max_prefix = std::max<int64_t>(max_prefix, plens[b]);
  }
  if (S < 1 || S >= (1 << 20) || S * Hq >= (1ll << 31)) {
    set_error("%s: needs between 1 and 2^20 - 1 responses, got %lld", who, (long long)S);
    return PG_ERR_INVALID_ARG;
  }
  pg_decode_plan& p = out->p;
  p.num_groups = B;
  p.num_seqs = (int32_t)S;
  p.heads_q = Hq;
  p.heads_kv = Hkv;
  p.head_dim = d;
  p.dtype = dt;
  p.page_size = ps;
  p.own_pages = own_pages;
  p.max_prefix = max_prefix;
  const int hp = Hq / Hkv;
  const int64_t own_cap = (int64_t)own_pages * ps;
  // SIMT: parts enough for a few blocks per SM, none shorter than 64 keys.
  const int64_t nhc = (hp + kHeadsPerBlock - 1) / kHeadsPerBlock, blocks = S * Hkv * nhc;
  int64_t ns = std::max<int64_t>(1, (int64_t)kSMs * 8 / blocks);
  ns = std::min<int64_t>(ns, std::max<int64_t>(1, (max_prefix + own_cap) / 64));
  p.simt_splits = (int32_t)std::min<int64_t>(ns, 32);
  // Tensor cores: how many tiles a prefix item takes.  An item costs its tiles and about three more
  // (launch, first loads, merge of the streams); items run in waves of one per SM; every part
  // adds a partial result per query row, written and read in fp32, to be weighed in tiles of K and V.
  // The own-key CTAs run in what the prefix CTAs leave of an SM, but start when the last of those
  // has: a second wave has to gain a quarter to be worth it (four groups of 64 over 32768 keys: one
  // wave on 128 SMs 237 us, three waves 276 us).
  int64_t chunk = 1;
  if (dt == PG_BF16 && hp <= kMaxRows) {
    p.seqs_per_item = kMaxRows / hp;
    const int64_t longest = (max_prefix + kDecodeTile - 1) / kDecodeTile;
    const double slot_cost = (double)S * Hq * d * 8 / ((double)kSMs * kDecodeTile * d * 4);
    double best = 0;
    for (int64_t parts = 1; parts <= std::min<int64_t>(longest, 64); ++parts) {
      const int64_t per = (longest + parts - 1) / parts;
      int64_t items = 0;
      for (int32_t b = 0; b < B; ++b) {
        const int64_t tiles = (plens[b] + kDecodeTile - 1) / kDecodeTile;
        items += (tiles + per - 1) / per * ((gsizes[b] + p.seqs_per_item - 1) / p.seqs_per_item);
      }
      const int64_t waves = (items * Hkv + kSMs - 1) / kSMs;
      const double cost = (waves > 1 ? 1.25 : 1.0) * (double)waves * (double)(per + 3) +
                          slot_cost * (double)((longest + per - 1) / per);
      if (parts == 1 || cost < best) {
        best = cost;
        chunk = per;
      }
    }
    // Own keys: parts enough for nine one-warp CTAs per SM, none that could not hold more than 64 keys.
    // (16 responses of 8 heads and 256-1024 keys: one part 51 us, four 35, eight 33; 128 responses of
    // 0-512 keys: one 53, two 51, eight 58, as partial results add up.)  At d = 128 eight fit at a time,
    // at d = 64 sixteen; parts for exactly those instead take 28.0 instead of 28.6 us on 16 responses over
    // 16384 keys, but 45.6 instead of 42.6 on 32 with 1000-2048 own keys over 500, and at d = 64
    // 22.6 instead of 20.6 on the first.
    if (own_cap > 0) {
      const int64_t ctas = S * Hkv * ((hp + 15) / 16);
      int64_t parts = ((int64_t)kSMs * 9 + ctas - 1) / ctas;
      parts = std::min<int64_t>(std::min<int64_t>(parts, 16), std::max<int64_t>(1, own_cap / 64));
      p.own_slots = (int32_t)parts;
      // In 8 bits a CTA is bound by the instructions between its loads rather than by bytes in flight, and
      // the longest response ends the kernel: up to four parts, fewer where there is no room for 1024 keys
      // each, of which a step uses what its responses' lengths ask for (own_parts_e4m3).  A part that is not
      // used costs an empty CTA.  (256 responses, 8 heads, room for 16384 keys, with 32, 300 or 1500 of them
      // at present: 2, 4 and 16 parts 15.0, 41.9, 135; 18.0, 42.5, 135; 55.7, 76.2, 161 us.  With 1-8000
      // keys and room for 8192: 372, 349 and (8 parts) 339; one response of 8000 among those of 200: 118, 76, 61.)
      p.own_slots_e4m3 = (int32_t)std::max<int64_t>(parts, std::min<int64_t>((own_cap + 1023) / 1024, 4));
    }
  }
  int32_t s0 = 0;
  for (int32_t b = 0; b < B; ++b) {
    const int64_t keys = (int64_t)chunk * kDecodeTile;
    const int32_t parts = p.seqs_per_item > 0 ? (int32_t)((plens[b] + keys - 1) / keys) : 0;
    for (int32_t i = 0; i < gsizes[b]; ++i) out->seqs.push_back({b, plens[b], parts, 0});
    for (int32_t c = 0; c < parts; ++c)
      for (int32_t i = 0; i < gsizes[b]; i += p.seqs_per_item)
        out->items.push_back({b, s0 + i, std::min(p.seqs_per_item, gsizes[b] - i),
                              (int32_t)(c * keys),
                              (int32_t)std::min<int64_t>(plens[b], (c + 1) * keys), c, 0, 0});
    if (gsizes[b] > 0) p.prefix_slots = std::max(p.prefix_slots, parts);
    s0 += gsizes[b];
  }
  p.n_items = (int32_t)out->items.size();
  if ((int64_t)p.n_items * Hkv >= (1ll << 31) ||
      S * Hkv * ((hp + 15) / 16) * std::max({p.own_slots, p.own_slots_e4m3, 1}) >= (1ll << 31)) {
    set_error("%s: too many work items", who);
    return PG_ERR_INVALID_ARG;
  }
  int64_t off = 0;
  p.off_seqs = off;
  off = align_up(off + S * (int64_t)sizeof(DecodeSeq), 256);
  p.off_items = off;
  off = align_up(off + (int64_t)out->items.size() * (int64_t)sizeof(DecodeItem), 256);
  p.table_bytes = off;
  p.workspace_bytes = decode_bytes(p, p.own_slots);
  p.workspace_bytes_e4m3 = decode_bytes(p, p.own_slots_e4m3);
  return PG_OK;
}

void write_tables(const DecodePlan& pl, void* tables) {
  char* t = static_cast<char*>(tables);
  memcpy(t + pl.p.off_seqs, pl.seqs.data(), pl.seqs.size() * sizeof(DecodeSeq));
  if (!pl.items.empty())
    memcpy(t + pl.p.off_items, pl.items.data(), pl.items.size() * sizeof(DecodeItem));
}

// What the attention calls ask of their arguments, and a launch's arguments from them.
pg_status make_args(const char* who, const pg_decode_plan* plan, const void* q, const void* k_cache,
                    const void* v_cache, int64_t num_pages, const int32_t* prefix_pages,
                    int64_t prefix_stride, const int32_t* own_pages, int64_t own_stride,
                    const int32_t* own_lens, int own_slots, void* o, float* lse, const pg_opts* opts,
                    void* workspace, size_t workspace_bytes, pg_stream_t stream, DecodeArgs* out) {
  if (!plan || !plan->tables || plan->num_seqs < 1) {
    set_error("%s: plan missing or empty (call pg_plan_decode first)", who);
    return PG_ERR_INVALID_ARG;
  }
  const int64_t prefix_pages_needed = (plan->max_prefix + plan->page_size - 1) / plan->page_size;
  if (num_pages < 0 || num_pages * plan->page_size >= (1ll << 31) ||
      (num_pages < 1 && (plan->max_prefix > 0 || plan->own_pages > 0))) {
    set_error("%s: num_pages * page_size must be below 2^31 and the cache non-empty", who);
    return PG_ERR_INVALID_ARG;
  }
  if ((plan->max_prefix > 0 && (!prefix_pages || prefix_stride < prefix_pages_needed)) ||
      (plan->own_pages > 0 && (!own_pages || !own_lens || own_stride < plan->own_pages))) {
    set_error("%s: page tables must be non-NULL and their rows cover the longest prefix (%lld pages) "
              "and the plan's own_pages (%d), own_lens non-NULL", who,
              (long long)prefix_pages_needed, plan->own_pages);
    return PG_ERR_INVALID_ARG;
  }
  if (opts && (!(opts->softmax_scale >= 0.f) || opts->rope_theta != 0.f || opts->debug != 0u ||
               (opts->flags & ~PG_FLAG_SIMT))) {
    set_error("%s: softmax_scale must be >= 0, rope_theta and debug 0, flags 0 or PG_FLAG_SIMT", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!q || !k_cache || !v_cache || !o || !lse || !workspace || !aligned16(q) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(workspace) || workspace_bytes < plan->workspace_bytes) {
    set_error("%s: q, the caches, o, lse and the workspace must be non-NULL and 16-byte aligned, the "
              "workspace >= %zu bytes", who, plan->workspace_bytes);
    return PG_ERR_INVALID_ARG;
  }
  DecodeArgs& a = *out;
  a.plan = plan;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = num_pages;
  a.prefix_pages = prefix_pages;
  a.prefix_stride = prefix_stride;
  a.own_pages = own_pages;
  a.own_stride = own_stride;
  a.own_lens = own_lens;
  a.o = o;
  a.lse = lse;
  const float scale = opts && opts->softmax_scale > 0.f ? opts->softmax_scale
                                                        : 1.0f / sqrtf((float)plan->head_dim);
  a.scale_log2 = scale * kLog2e;
  // (own_slots as far as the workspace goes, the plan's for its own type at least)
  a.own_slots = own_slots;
  while (a.own_slots > plan->own_slots && decode_bytes(*plan, a.own_slots) > workspace_bytes) --a.own_slots;
  const int64_t slots = decode_slots(*plan, a.own_slots);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(
      static_cast<char*>(workspace) +
      align_up(slots * plan->num_seqs * plan->heads_q * plan->head_dim * 4, 256));
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return PG_OK;
}

// Whether a call goes to the tensor-core kernels.
bool tensor_cores(const pg_decode_plan* plan, const pg_opts* opts) {
  return plan->seqs_per_item > 0 && !(opts && (opts->flags & PG_FLAG_SIMT));
}

// The prefix parts, the own keys and their merge.
pg_status run_tensor_cores(const DecodeArgs& a, pg_status (*prefix)(const DecodeArgs&),
                           pg_status (*own)(const DecodeArgs&, bool)) {
  const pg_decode_plan* plan = a.plan;
  pg_status st = PG_OK;
  if (plan->n_items > 0) st = prefix(a);
  if (st == PG_OK && a.own_slots > 0) st = own(a, plan->n_items > 0);
  if (st != PG_OK) return st;
  const int32_t* lens = a.k_scales && a.own_slots > 0 ? a.own_lens : nullptr;
  return plan->head_dim == 64
             ? combine_t<__nv_bfloat16, 64>(a, plan->prefix_slots, a.own_slots, lens)
             : combine_t<__nv_bfloat16, 128>(a, plan->prefix_slots, a.own_slots, lens);
}

// A C entry never lets an exception out.
template <typename F>
pg_status guarded(const char* who, F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    set_error("%s: %s", who, e.what());
    return PG_ERR_INVALID_ARG;
  }
}

}  // namespace

pg_status read_status_rollout(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_rollout, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_rollout, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg

using namespace pg;

extern "C" {

pg_status pg_cache_append(pg_dtype dtype, int64_t n_tokens, int32_t heads_q, int32_t heads_kv,
                          int32_t head_dim, const void* q, int64_t ldq, void* q_out, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                          float rope_theta, void* k_cache, void* v_cache, int64_t num_pages,
                          int32_t page_size, const int32_t* pages, int32_t num_page_rows,
                          int32_t pages_per_row, int64_t pages_stride, const int32_t* page_rows,
                          const int32_t* cache_pos, pg_stream_t stream) {
  const char* who = "pg_cache_append";
  if ((dtype != PG_F32 && dtype != PG_BF16) || n_tokens < 1 || n_tokens >= (1ll << 31) ||
      heads_q < 0 || heads_q > 65536 || heads_kv < 1 || heads_kv > 65536 ||
      (head_dim != 64 && head_dim != 128) || !(rope_theta >= 0.f)) {
    set_error("%s: needs dtype f32 or bf16, 1 <= n_tokens < 2^31, heads_kv >= 1, head_dim 64 or 128, "
              "rope_theta >= 0", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!page_size_ok(page_size) || num_pages < 1 || num_page_rows < 1 || pages_per_row < 1 ||
      pages_stride < pages_per_row || (!page_rows && num_page_rows < n_tokens)) {
    set_error("%s: page_size must be 16, 32, 64, 128 or 256, the cache and the page table non-empty, "
              "pages_stride >= pages_per_row, and without page_rows a table row per token", who);
    return PG_ERR_INVALID_ARG;
  }
  const int64_t unit = dtype == PG_F32 ? 4 : 8, kv_row = (int64_t)heads_kv * head_dim;
  if (!k || !v || !k_cache || !v_cache || !pages || !cache_pos || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) || ldk % unit || ldv % unit || ldk < kv_row ||
      ldv < kv_row) {
    set_error("%s: k, v and the caches must be non-NULL and 16-byte aligned, ldk and ldv multiples of "
              "16 bytes covering a row, pages and cache_pos non-NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  if (heads_q > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out) || ldq % unit ||
                      ldq < (int64_t)heads_q * head_dim)) {
    set_error("%s: q and q_out must be non-NULL and 16-byte aligned, ldq a multiple of 16 bytes "
              "covering a row", who);
    return PG_ERR_INVALID_ARG;
  }
  auto fn = dtype == PG_F32
                ? (head_dim == 64 ? append_t<float, 64> : append_t<float, 128>)
                : (head_dim == 64 ? append_t<__nv_bfloat16, 64> : append_t<__nv_bfloat16, 128>);
  return fn(n_tokens, heads_q, heads_kv, q, ldq, q_out, k, ldk, v, ldv, positions, rope_theta,
            k_cache, v_cache, num_pages, page_size, pages, num_page_rows, pages_per_row,
            pages_stride, page_rows, cache_pos, reinterpret_cast<cudaStream_t>(stream));
}

pg_status pg_plan_decode_size(int32_t num_groups, const int32_t* prefix_lens,
                              const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                              int32_t heads_kv, int32_t head_dim, int32_t page_size,
                              int32_t own_pages, int64_t* table_bytes) {
  return guarded("pg_plan_decode_size", [&] {
    if (!table_bytes) {
      set_error("pg_plan_decode_size: table_bytes is NULL");
      return PG_ERR_INVALID_ARG;
    }
    DecodePlan pl;
    pg_status st = make_plan(num_groups, prefix_lens, group_sizes, dtype, heads_q, heads_kv,
                             head_dim, page_size, own_pages, &pl);
    if (st == PG_OK) *table_bytes = pl.p.table_bytes;
    return st;
  });
}

pg_status pg_plan_decode_host(int32_t num_groups, const int32_t* prefix_lens,
                              const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                              int32_t heads_kv, int32_t head_dim, int32_t page_size,
                              int32_t own_pages, void* tables, int64_t table_bytes,
                              pg_decode_plan* plan) {
  return guarded("pg_plan_decode_host", [&] {
    DecodePlan pl;
    pg_status st = make_plan(num_groups, prefix_lens, group_sizes, dtype, heads_q, heads_kv,
                             head_dim, page_size, own_pages, &pl);
    if (st != PG_OK) return st;
    if (!tables || !plan || table_bytes < pl.p.table_bytes) {
      set_error("pg_plan_decode_host: NULL buffer or table buffer smaller than %lld bytes",
                (long long)pl.p.table_bytes);
      return PG_ERR_INVALID_ARG;
    }
    write_tables(pl, tables);
    *plan = pl.p;
    plan->tables = tables;
    return PG_OK;
  });
}

pg_status pg_plan_decode(int32_t num_groups, const int32_t* prefix_lens,
                         const int32_t* group_sizes, pg_dtype dtype, int32_t heads_q,
                         int32_t heads_kv, int32_t head_dim, int32_t page_size, int32_t own_pages,
                         void* tables_dev, int64_t table_bytes, pg_decode_plan* plan,
                         pg_stream_t stream) {
  return guarded("pg_plan_decode", [&] {
    DecodePlan pl;
    pg_status st = make_plan(num_groups, prefix_lens, group_sizes, dtype, heads_q, heads_kv,
                             head_dim, page_size, own_pages, &pl);
    if (st != PG_OK) return st;
    if (!tables_dev || !plan || !aligned16(tables_dev) || table_bytes < pl.p.table_bytes) {
      set_error("pg_plan_decode: NULL or misaligned buffer or table buffer smaller than %lld bytes",
                (long long)pl.p.table_bytes);
      return PG_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    st = cuda_check(cudaStreamIsCapturing(s, &capture), "pg_plan_decode: capture status");
    if (st != PG_OK) return st;
    if (capture != cudaStreamCaptureStatusNone) {
      // a replay would copy from the temporary buffer, which is gone by then
      set_error("pg_plan_decode: not to be captured into a graph (make the plan before)");
      return PG_ERR_INVALID_ARG;
    }
    std::vector<char> host((size_t)pl.p.table_bytes, 0);
    write_tables(pl, host.data());
    st = cuda_check(cudaMemcpyAsync(tables_dev, host.data(), host.size(), cudaMemcpyHostToDevice, s),
                    "pg_plan_decode: copy");
    if (st != PG_OK) return st;
    *plan = pl.p;
    plan->tables = tables_dev;
    return PG_OK;
  });
}

pg_status pg_decode_attn(const pg_decode_plan* plan, const void* q, const void* k_cache,
                         const void* v_cache, int64_t num_pages, const int32_t* prefix_pages,
                         int64_t prefix_stride, const int32_t* own_pages, int64_t own_stride,
                         const int32_t* own_lens, void* o, float* lse, const pg_opts* opts,
                         void* workspace, size_t workspace_bytes, pg_stream_t stream) {
  DecodeArgs a{};
  const pg_status st = make_args("pg_decode_attn", plan, q, k_cache, v_cache, num_pages, prefix_pages,
                                 prefix_stride, own_pages, own_stride, own_lens, plan ? plan->own_slots : 0,
                                 o, lse, opts, workspace, workspace_bytes, stream, &a);
  if (st != PG_OK) return st;
  if (tensor_cores(plan, opts)) return run_tensor_cores(a, launch_decode_prefix, launch_decode_own);
  if (plan->dtype == PG_F32)
    return plan->head_dim == 64 ? simt_t<float, float, 64>(a) : simt_t<float, float, 128>(a);
  return plan->head_dim == 64 ? simt_t<__nv_bfloat16, __nv_bfloat16, 64>(a)
                              : simt_t<__nv_bfloat16, __nv_bfloat16, 128>(a);
}

pg_status pg_decode_attn_e4m3(const pg_decode_plan* plan, const void* q, const void* k_codes,
                              const void* v_codes, const float* k_scales, const float* v_scales,
                              int64_t num_pages, const int32_t* prefix_pages,
                              int64_t prefix_stride, const int32_t* own_pages, int64_t own_stride,
                              const int32_t* own_lens, void* o, float* lse, const pg_opts* opts,
                              void* workspace, size_t workspace_bytes, pg_stream_t stream) {
  const char* who = "pg_decode_attn_e4m3";
  DecodeArgs a{};
  const pg_status st = make_args(who, plan, q, k_codes, v_codes, num_pages, prefix_pages,
                                 prefix_stride, own_pages, own_stride, own_lens,
                                 plan ? plan->own_slots_e4m3 : 0, o, lse, opts, workspace,
                                 workspace_bytes, stream, &a);
  if (st != PG_OK) return st;
  if (!k_scales || !v_scales || !aligned16(k_scales) || !aligned16(v_scales)) {
    set_error("%s: the scales must be non-NULL and 16-byte aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  if (tensor_cores(plan, opts))
    return run_tensor_cores(a, launch_decode_prefix_e4m3, launch_decode_own_e4m3);
  if (plan->dtype == PG_F32)
    return plan->head_dim == 64 ? simt_t<float, uint8_t, 64>(a) : simt_t<float, uint8_t, 128>(a);
  return plan->head_dim == 64 ? simt_t<__nv_bfloat16, uint8_t, 64>(a)
                              : simt_t<__nv_bfloat16, uint8_t, 128>(a);
}

}  // extern "C"
