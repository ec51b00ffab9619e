// Per-head RMSNorm of q and k with the position rotation in the same pass, forward and backward.
//
//   forward   y = R(pos) (x r g),  r = 1 / sqrt(mean_j x_j^2 + eps)
//   backward  dy = R(pos)^-1 dout;  dx = r (g dy - xhat mean_j(xhat g dy)),  xhat = x r;
//             dg_j = sum over tokens and heads of dy_j xhat_j
//
// Bound by memory: every element is read once and written once (forward), or x and dout are read and
// dx written (backward); r is recomputed in the backward from the x it reads anyway.  A warp owns a
// token (or, with few tokens, a share of a token's heads) and walks its heads, D / 8 lanes to a
// row, so the token's angles are computed once and used for every head of q and k.  The gain
// gradients are summed per lane over all its rows, then over the block, and the blocks' partial
// sums are added in a fixed order by a second launch: the result is the same from run to run.
#include <algorithm>

#include "pg_headrows.cuh"
#include "pg_internal.h"

namespace pg {

using namespace headrows;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdBlocks = 152 * 2;   // one wave of resident blocks: as many partial gain gradients
constexpr int kSMs = 152;

// Heads [h0, h1) of token t: which share of the work a warp takes.
struct Split {
  int chunks;      // warps per token
  int per_chunk;   // heads per warp, a multiple of the rows a warp takes at once
};

// One warp per token once the tokens alone fill the GPU's warps; a token's heads are shared out
// among warps below that, down to one step's rows a warp, since a warp's rows follow one another.
Split split_heads(int64_t T, int heads, int rows_per_step) {
  const int steps = (heads + rows_per_step - 1) / rows_per_step;
  const int64_t want = std::max<int64_t>(1, (int64_t)kSMs * 32 / std::max<int64_t>(T, 1));
  const int chunks = (int)std::min<int64_t>(steps, want);
  const int per = (steps + chunks - 1) / chunks * rows_per_step;
  return {(heads + per - 1) / per, per};
}

// Heads [h0, h1) of one tensor of one token: x (rows of D from `x`) to y.  The loads of kFwdRows rows
// per group of lanes are in flight at once, kept as bf16 until used: with them converted, 89 registers
// leave two blocks per SM, and 32768 tokens of 32 + 8 heads took 154 us instead of 106 (6.3 TB/s).
constexpr int kFwdRows = 4;
// In the backward x and dy are both read: four rows of each in bf16 fill the registers of two blocks per
// SM, and 26601 tokens take 141.5 us (5.8 TB/s; with two rows 164).  fp32 rows take twice the registers.
template <typename T>
constexpr int kBwdRows = sizeof(T) == 2 ? 4 : 2;

template <typename T, int D>
__device__ __forceinline__ void norm_heads(const T* x, T* y, const T* __restrict__ gain, int h0, int h1,
                                           const float (&c)[4], const float (&s)[4], float eps, int l,
                                           int sub) {
  constexpr int RPW = 256 / D, U = kFwdRows;
  if (h0 >= h1) return;
  Row<T, D> g;
  g.load(gain, l);
  for (int h = h0; h < h1; h += RPW * U) {
    RawRow<T, D> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)       // past the end: the last head again
      raw[u].load(x + (size_t)min(h + u * RPW + sub, h1 - 1) * D, l);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Row<T, D> v;
      v.from(raw[u]);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss += v.lo[e] * v.lo[e] + v.hi[e] * v.hi[e];
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v.lo[e] = v.lo[e] * r * g.lo[e];
        v.hi[e] = v.hi[e] * r * g.hi[e];
      }
      v.rotate(c, s);
      const int row = h + u * RPW + sub;
      if (row < h1) v.store(y + (size_t)row * D, l);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
qk_norm_fwd_kernel(const T* q, long long ldq, const T* k, long long ldk, const T* __restrict__ gq,
                   const T* __restrict__ gk, T* q_out, T* k_out, const int32_t* __restrict__ pos,
                   const __grid_constant__ RopeFreq f, int rope, float eps, long long Ttot, int Hq,
                   int Hkv, Split sp) {
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long t = item / sp.chunks;
  if (t >= Ttot) return;
  const int h_begin = (int)(item % sp.chunks) * sp.per_chunk;
  const int h_end = min(h_begin + sp.per_chunk, Hq + Hkv);
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (rope) {
    Angles<D> a;
    a.init(f.turn, lane);
    a.at(pos[t], lane, c, s);
  }
  norm_heads<T, D>(q + t * ldq, q_out + (size_t)t * Hq * D, gq, h_begin, min(h_end, Hq), c, s, eps, l,
                   sub);
  norm_heads<T, D>(k + t * ldk, k_out + (size_t)t * Hkv * D, gk, max(h_begin - Hq, 0), h_end - Hq, c,
                   s, eps, l, sub);
}

// The backward of norm_heads: dx from x and dy (the gradient of y), and the lane's sums of dy xhat.
template <typename T, int D>
__device__ __forceinline__ void norm_heads_bwd(const T* x, const T* dy, T* dx,
                                               const T* __restrict__ gain, int h0, int h1,
                                               const float (&c)[4], const float (&s)[4], float eps,
                                               int l, int sub, float (&acc)[8]) {
  constexpr int RPW = 256 / D, U = kBwdRows<T>;
  if (h0 >= h1) return;
  Row<T, D> g;
  g.load(gain, l);
  for (int h = h0; h < h1; h += RPW * U) {
    RawRow<T, D> rx[U], ry[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t at = (size_t)min(h + u * RPW + sub, h1 - 1) * D;
      rx[u].load(x + at, l);
      ry[u].load(dy + at, l);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = h + u * RPW + sub;
      const bool valid = row < h1;
      Row<T, D> v, d;
      v.from(rx[u]);
      d.from(ry[u]);
      // the inverse rotation
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float b0 = d.lo[e], b1 = d.hi[e];
        d.lo[e] = b0 * c[e] + b1 * s[e];
        d.hi[e] = b1 * c[e] - b0 * s[e];
      }
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ss += v.lo[e] * v.lo[e] + v.hi[e] * v.hi[e];
        dot += v.lo[e] * (g.lo[e] * d.lo[e]) + v.hi[e] * (g.hi[e] * d.hi[e]);
      }
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
      const float mean = row_sum<D>(dot) * r * (1.f / D);   // of xhat g dy
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = v.lo[e] * r, x1 = v.hi[e] * r;
        if (valid) {
          acc[e] += d.lo[e] * x0;
          acc[4 + e] += d.hi[e] * x1;
        }
        v.lo[e] = r * (g.lo[e] * d.lo[e] - x0 * mean);
        v.hi[e] = r * (g.hi[e] * d.hi[e] - x1 * mean);
      }
      if (valid) v.store(dx + (size_t)row * D, l);
    }
  }
}

// part[block][2][D]: the block's sums of dy xhat, for q and for k.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_bwd_kernel(const T* __restrict__ q, long long ldq, const T* __restrict__ k, long long ldk,
                   const T* __restrict__ gq, const T* __restrict__ gk, const T* dq_out,
                   const T* dk_out, T* dq, T* dk, float* __restrict__ part,
                   const int32_t* __restrict__ pos, const __grid_constant__ RopeFreq f, int rope,
                   float eps, long long Ttot, int Hq, int Hkv, Split sp) {
  constexpr int LPR = D / 8;
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  Angles<D> a;
  if (rope) a.init(f.turn, lane);
  float acc[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[0][e] = acc[1][e] = 0.f;
  const long long items = Ttot * sp.chunks, step = (long long)gridDim.x * kWarps;
  for (long long item = (long long)blockIdx.x * kWarps + warp; item < items; item += step) {
    const long long t = item / sp.chunks;
    const int h_begin = (int)(item % sp.chunks) * sp.per_chunk;
    const int h_end = min(h_begin + sp.per_chunk, Hq + Hkv);
    if (rope) a.at(pos[t], lane, c, s);
    norm_heads_bwd<T, D>(q + t * ldq, dq_out + (size_t)t * Hq * D, dq + (size_t)t * Hq * D, gq, h_begin,
                         min(h_end, Hq), c, s, eps, l, sub, acc[0]);
    norm_heads_bwd<T, D>(k + t * ldk, dk_out + (size_t)t * Hkv * D, dk + (size_t)t * Hkv * D, gk,
                         max(h_begin - Hq, 0), h_end - Hq, c, s, eps, l, sub, acc[1]);
  }
  // the rows of a warp, then the warps of the block, in a fixed order
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) acc[w][e] += __shfl_xor_sync(0xffffffffu, acc[w][e], o);
      if (sub == 0) red[warp][w][(e < 4 ? 4 * l + e : D / 2 + 4 * l + e - 4)] = acc[w][e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += red[w][i / D][i % D];
    part[(size_t)blockIdx.x * 2 * D + i] = x;
  }
}

// One block per column of part [n][cols]: each thread adds every 128th partial sum, then the
// threads are added up by halves.
__global__ void __launch_bounds__(128)
gain_grad_kernel(const float* __restrict__ part, int n, int cols, int d, float* __restrict__ dgq,
                 float* __restrict__ dgk) {
  __shared__ float red[128];
  const int col = blockIdx.x;
  float x = 0.f;
  for (int i = threadIdx.x; i < n; i += 128) x += part[(size_t)i * cols + col];
  red[threadIdx.x] = x;
  __syncthreads();
  for (int o = 64; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    float* dst = col < d ? dgq : dgk;
    if (dst) dst[col < d ? col : col - d] = red[0];
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pg_status check(const char* who, pg_dtype dt, int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                const void* q, int64_t ldq, const void* k, int64_t ldk, const void* gq,
                const void* gk, float eps, const int32_t* pos, float theta) {
  if ((dt != PG_F32 && dt != PG_BF16) || T < 1 || T >= (1ll << 31) || Hq < 0 || Hkv < 0 ||
      Hq > 65536 || Hkv > 65536 || Hq + Hkv < 1 || (d != 64 && d != 128)) {
    set_error("%s: needs dtype f32 or bf16, 1 <= T < 2^31, at least one head and head_dim 64 or 128",
              who);
    return PG_ERR_INVALID_ARG;
  }
  if (!(eps >= 0.f) || !(theta >= 0.f) || (theta > 0.f && !pos)) {
    set_error("%s: eps and rope_theta must be >= 0, and a rotation needs positions", who);
    return PG_ERR_INVALID_ARG;
  }
  const int64_t unit = dt == PG_F32 ? 4 : 8;
  for (int w = 0; w < 2; ++w) {
    const int64_t H = w ? Hkv : Hq, ld = w ? ldk : ldq;
    if (H == 0) continue;
    if (!(w ? k : q) || !(w ? gk : gq) || !aligned16(w ? k : q) || !aligned16(w ? gk : gq)) {
      set_error("%s: %c and its gain must be non-NULL and 16-byte aligned", who, w ? 'k' : 'q');
      return PG_ERR_INVALID_ARG;
    }
    if (ld % unit || ld < H * d) {
      set_error("%s: the row stride of %c must be a multiple of 16 bytes and cover its heads", who,
                w ? 'k' : 'q');
      return PG_ERR_INVALID_ARG;
    }
  }
  return PG_OK;
}

template <typename T, int D>
pg_status fwd_t(int64_t n, int Hq, int Hkv, const void* q, int64_t ldq, const void* k, int64_t ldk,
                const void* gq, const void* gk, float eps, const int32_t* pos, float theta,
                void* qo, void* ko, cudaStream_t s) {
  const Split sp = split_heads(n, Hq + Hkv, 256 / D);
  const int64_t items = n * sp.chunks;
  const int64_t blocks = (items + kWarps - 1) / kWarps;
  const RopeFreq f = rope_freq(D, theta);
  prof_begin(PG_KERNEL_QK_NORM, s);
  qk_norm_fwd_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(
      static_cast<const T*>(q), ldq, static_cast<const T*>(k), ldk, static_cast<const T*>(gq),
      static_cast<const T*>(gk), static_cast<T*>(qo), static_cast<T*>(ko), pos, f, theta > 0.f, eps,
      n, Hq, Hkv, sp);
  prof_end(PG_KERNEL_QK_NORM, s);
  return cuda_check(cudaGetLastError(), "qk norm fwd launch");
}

int bwd_blocks(int64_t n, int heads, int d) {
  const Split sp = split_heads(n, heads, 256 / d);
  return (int)std::min<int64_t>(kBwdBlocks, (n * sp.chunks + kWarps - 1) / kWarps);
}

template <typename T, int D>
pg_status bwd_t(int64_t n, int Hq, int Hkv, const void* q, int64_t ldq, const void* k, int64_t ldk,
                const void* gq, const void* gk, float eps, const void* dqo, const void* dko,
                const int32_t* pos, float theta, void* dq, void* dk, float* dgq, float* dgk,
                float* part, cudaStream_t s) {
  const Split sp = split_heads(n, Hq + Hkv, 256 / D);
  const int blocks = bwd_blocks(n, Hq + Hkv, D);
  const RopeFreq f = rope_freq(D, theta);
  prof_begin(PG_KERNEL_QK_NORM, s);
  qk_norm_bwd_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(
      static_cast<const T*>(q), ldq, static_cast<const T*>(k), ldk, static_cast<const T*>(gq),
      static_cast<const T*>(gk), static_cast<const T*>(dqo), static_cast<const T*>(dko),
      static_cast<T*>(dq), static_cast<T*>(dk), part, pos, f, theta > 0.f, eps, n, Hq, Hkv, sp);
  gain_grad_kernel<<<2 * D, 128, 0, s>>>(part, blocks, 2 * D, D, Hq > 0 ? dgq : nullptr,
                                         Hkv > 0 ? dgk : nullptr);
  prof_end(PG_KERNEL_QK_NORM, s);
  return cuda_check(cudaGetLastError(), "qk norm bwd launch");
}

}  // namespace

}  // namespace pg

using namespace pg;

extern "C" {

pg_status pg_qk_norm_rope_fwd(pg_dtype dtype, int64_t T, int32_t heads_q, int32_t heads_kv,
                              int32_t head_dim, const void* q, int64_t ldq, const void* k,
                              int64_t ldk, const void* gain_q, const void* gain_k, float eps,
                              const int32_t* positions, float rope_theta, void* q_out, void* k_out,
                              pg_stream_t stream) {
  const char* who = "pg_qk_norm_rope_fwd";
  pg_status st = check(who, dtype, T, heads_q, heads_kv, head_dim, q, ldq, k, ldk, gain_q, gain_k,
                       eps, positions, rope_theta);
  if (st != PG_OK) return st;
  if ((heads_q > 0 && (!q_out || !aligned16(q_out))) ||
      (heads_kv > 0 && (!k_out || !aligned16(k_out)))) {
    set_error("%s: outputs must be non-NULL and 16-byte aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  auto fn = dtype == PG_F32 ? (head_dim == 64 ? fwd_t<float, 64> : fwd_t<float, 128>)
                            : (head_dim == 64 ? fwd_t<__nv_bfloat16, 64> : fwd_t<__nv_bfloat16, 128>);
  return fn(T, heads_q, heads_kv, q, ldq, k, ldk, gain_q, gain_k, eps, positions, rope_theta, q_out,
            k_out, reinterpret_cast<cudaStream_t>(stream));
}

size_t pg_qk_norm_rope_bwd_workspace(int64_t T, int32_t heads_q, int32_t heads_kv,
                                     int32_t head_dim) {
  (void)T;
  (void)heads_q;
  (void)heads_kv;
  return (size_t)kBwdBlocks * 2 * head_dim * sizeof(float);
}

pg_status pg_qk_norm_rope_bwd(pg_dtype dtype, int64_t T, int32_t heads_q, int32_t heads_kv,
                              int32_t head_dim, const void* q, int64_t ldq, const void* k,
                              int64_t ldk, const void* gain_q, const void* gain_k, float eps,
                              const void* dq_out, const void* dk_out, const int32_t* positions,
                              float rope_theta, void* dq, void* dk, float* dgain_q, float* dgain_k,
                              void* workspace, size_t workspace_bytes, pg_stream_t stream) {
  const char* who = "pg_qk_norm_rope_bwd";
  pg_status st = check(who, dtype, T, heads_q, heads_kv, head_dim, q, ldq, k, ldk, gain_q, gain_k,
                       eps, positions, rope_theta);
  if (st != PG_OK) return st;
  const bool bad_q = heads_q > 0 && (!dq_out || !dq || !dgain_q || !aligned16(dq_out) || !aligned16(dq));
  const bool bad_k = heads_kv > 0 && (!dk_out || !dk || !dgain_k || !aligned16(dk_out) || !aligned16(dk));
  if (bad_q || bad_k) {
    set_error("%s: gradients must be non-NULL and 16-byte aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pg_qk_norm_rope_bwd_workspace(T, heads_q, heads_kv, head_dim)) {
    set_error("%s: workspace must be 16-byte aligned and >= %zu bytes", who,
              pg_qk_norm_rope_bwd_workspace(T, heads_q, heads_kv, head_dim));
    return PG_ERR_INVALID_ARG;
  }
  auto fn = dtype == PG_F32 ? (head_dim == 64 ? bwd_t<float, 64> : bwd_t<float, 128>)
                            : (head_dim == 64 ? bwd_t<__nv_bfloat16, 64> : bwd_t<__nv_bfloat16, 128>);
  return fn(T, heads_q, heads_kv, q, ldq, k, ldk, gain_q, gain_k, eps, dq_out, dk_out, positions,
            rope_theta, dq, dk, dgain_q, dgain_k, static_cast<float*>(workspace),
            reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
