// The paged cache in 8 bits: append with rotation and block scales, and reading back.
//
// A block is 16 consecutive slots of a page and one head.  Its scale is the least power of two 2^e with all
// its values within 448 2^e, the range of e4m3, and a slot holds round(x 2^-e).  A power of two costs
// no accuracy against a scale of 24 bits (the code's relative step is the same all over its range, only
// values 2^-15 of the largest and below lose bits), and it makes a block that grows cheap to keep: when a
// new token exceeds the range, the codes already there are multiplied by a power of two, which changes none of
// them but those that fall below the normal range.
//
// Append.  A CTA takes a window of 16 tokens of the call and some heads; 8 (d = 128) or 4 (d = 64) lanes hold
// a row of one head and the rows of 16 tokens are handled side by side, the next head's on their way.  Tokens of
// the window that follow one another in a block form a group, whose largest value is found through shared memory;
// a group that starts in the window and ends in the next belongs to this one (a second round of rows), so
// nobody else writes its blocks.  A window whose first block is full and begins in it (a prompt's pages)
// takes one round; 16 responses of one token each are 16 groups of one.
//
// The read back is bound by memory: 8 prompts of 2048 tokens, 8 key/value heads of 128, bf16, 101 MB in 17 us (5.9
// TB/s), fp32 168 MB in 30 us (5.6).  The append of the same takes 34 us (3.0 TB/s), of fp32 48 us (3.5), and waits
// rather than reads: 260 instructions per warp and head fill 43 % of the issue slots of 16 warps per SM, each with a
// chain of two barriers, two reductions and the reads of its turn.  (Against 37 us then, rows brought through shared
// memory up to three heads ahead: 36 us; fewer registers and more warps: 39.)  A step of one token per response is
// bound by the latency of a launch and two dependent reads (index, page): 16 responses, append and read back, 6.6
// us.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pg_e4m3.cuh"
#include "pg_headrows.cuh"
#include "pg_internal.h"
#include "pg_sm100.cuh"

namespace pg {

using namespace headrows;
using namespace e4m3;

namespace {

constexpr int kSMs = 152;
constexpr int kBlock = 16;            // tokens that share a scale
constexpr int kWindow = 16;           // tokens of a CTA

__device__ int s_status_cache8 = 0;

__device__ __forceinline__ void report(int code) { atomicCAS(&s_status_cache8, 0, code); }

struct Cache8 {
  uint8_t *k, *v;
  float *ks, *vs;
  long long num_pages, pages_stride;
  const int32_t *pages, *page_rows, *cache_pos;
  int page_size, num_page_rows, pages_per_row;

  // The slot of index cp of a page table row; -1: none.  `ok` false if it is out of range.
  __device__ __forceinline__ long long slot(long long row, int cp, bool& ok) const {
    const int pi = cp / page_size;
    long long page = -1;
    if (row >= 0 && row < num_page_rows && pi < pages_per_row) page = pages[row * pages_stride + pi];
    ok = page >= 0 && page < num_pages;
    return ok ? page * page_size + cp % page_size : -1;
  }
};

// A lane's share of a row: its elements [8 l, 8 l + 8) and [D/2 + 8 l, D/2 + 8 l + 8), both ends of eight
// rotate-half pairs; as they are in memory, and in fp32.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = *(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4& u = v[sizeof(T) / 2 == 2 ? i : 0];
        x[4 * i] = __uint_as_float(u.x);
        x[4 * i + 1] = __uint_as_float(u.y);
        x[4 * i + 2] = __uint_as_float(u.z);
        x[4 * i + 3] = __uint_as_float(u.w);
      }
    }
  }
};
template <typename T, int D>
struct RawHalves {
  Raw8<T> lo, hi;
  __device__ __forceinline__ void load(const T* row, int l) {
    lo.load(row + 8 * l);
    hi.load(row + D / 2 + 8 * l);
  }
};
struct Halves {
  float lo[8], hi[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) lo[e] = hi[e] = 0.f;
  }
  template <typename T, int D>
  __device__ __forceinline__ void from(const RawHalves<T, D>& r) {
    r.lo.get(lo);
    r.hi.get(hi);
  }
  __device__ __forceinline__ void rotate(const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = lo[e], b = hi[e];
      lo[e] = a * c[e] - b * s[e];
      hi[e] = b * c[e] + a * s[e];
    }
  }
  // The codes under the scale 1 / inv, 8 bytes to either place.
  __device__ __forceinline__ void encode(uint8_t* p, uint8_t* q, float inv, bool inf) const {
    auto codes = [&](const float (&x)[8]) {
      const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
      return inf ? make_uint2(encode4(a, inv), encode4(b, inv))
                 : make_uint2(encode4_finite(a, inv), encode4_finite(b, inv));
    };
    *reinterpret_cast<uint2*>(p) = codes(lo);
    *reinterpret_cast<uint2*>(q) = codes(hi);
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(sm100::pack_bf16x2(x[0], x[1]), sm100::pack_bf16x2(x[2], x[3]),
                   sm100::pack_bf16x2(x[4], x[5]), sm100::pack_bf16x2(x[6], x[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(D, 512 / D)
append_e4m3_kernel(const T* q, long long ldq, T* q_out, const T* __restrict__ k, long long ldk,
                   const T* __restrict__ v, long long ldv, const int32_t* __restrict__ positions,
                   const __grid_constant__ RopeFreq f, int rope, const Cache8 c, long long N, int Hq,
                   int Hkv, int chunks, int per_chunk) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  static_assert(D / LPR == kWindow, "a row per token of the window");
  __shared__ uint64_t turn[D / 2];
  __shared__ float row_max[2][2 * kWindow];        // [k, v][token]
  __shared__ float held[2][kWindow];               // [k, v][leader]: the scale before the call
  __shared__ float2 grown[2][kWindow];             // [k, v][leader]: that and the new one, if larger
  if (rope) {
    if (threadIdx.x < D / 2) turn[threadIdx.x] = f.turn[threadIdx.x];
    __syncthreads();
  }
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const int i0 = (threadIdx.x >> 5) * RPW + lane / LPR;        // this row's token of the window
  const long long w0 = (long long)(blockIdx.x / (unsigned)chunks) * kWindow;
  const int u_begin = (int)(blockIdx.x % (unsigned)chunks) * per_chunk;
  const int u_end = min(u_begin + per_chunk, Hq + Hkv);

  // Lane t looks at token w0 + t: is it in the block of the token before it, behind that?
  const long long nt = w0 + lane;
  const int cp_t = nt < N ? c.cache_pos[nt] : -1;
  const long long row_t = nt < N ? (c.page_rows ? (long long)c.page_rows[nt] : nt) : -1;
  int cp_b = __shfl_up_sync(0xffffffffu, cp_t, 1);
  long long row_b = __shfl_up_sync(0xffffffffu, row_t, 1);
  if (lane == 0 && w0 > 0) {
    cp_b = c.cache_pos[w0 - 1];
    row_b = c.page_rows ? (long long)c.page_rows[w0 - 1] : w0 - 1;
  }
  const bool linked = nt > 0 && nt < N && cp_t > 0 && cp_b >= 0 && row_t == row_b &&
                      cp_t == cp_b + 1 && cp_t % kBlock != 0;
  const uint32_t links = __ballot_sync(0xffffffffu, linked);
  // The first token of i's group, -1 if it lies before the window.
  auto leader_of = [&](int i) { return 31 - __clz(~links & (0xffffffffu >> (31 - i))); };
  const bool more = leader_of(kWindow) < kWindow && w0 + kWindow < N;   // the last group goes on
  const bool whole = (links & 0x1ffffu) == 0xfffeu;     // the window is one group (a prompt's block)

  // A lane's token of the window (or 16 further on): its place, its group, whether it is stored from here.
  struct Token {
    long long slot;
    int lead, end, off;      // of the group: its first token, one behind its last, its first slot in the block
    bool live;
  };
  auto token = [&](int i) {
    Token x;
    x.lead = leader_of(i);
    const int src = max(x.lead, 0);
    const uint32_t ends = x.lead < 31 ? ~links & (0xfffffffeu << src) : 0u;
    x.end = ends ? __ffs(ends) - 1 : 32;
    const int cp = __shfl_sync(0xffffffffu, cp_t, i);
    const long long row = __shfl_sync(0xffffffffu, row_t, i);
    x.off = __shfl_sync(0xffffffffu, cp_t, src) % kBlock;
    x.live = cp >= 0 && x.lead >= 0 && x.lead < kWindow && w0 + i < N;
    x.slot = 0;
    if (x.live) {
      bool ok;
      const long long at = c.slot(row, cp, ok);
      if (!ok && l == 0) report(PG_ERR_DEVICE);
      x.live = ok;
      if (ok) x.slot = at;
    }
    return x;
  };
  const Token mine = token(i0);
  auto angles = [&](long long n, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
    if (!rope || n >= N) return;
    const int pos = positions ? positions[n] : c.cache_pos[n];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // In half turns times 2^31, of which a float takes 24 bits and d the rest, in radians: an angle that is off
      // by more than a sine's rounding would bring more codes to the far side of a border.
      const int32_t h = (int32_t)(uint32_t)((uint64_t)(int64_t)pos * turn[8 * l + e] >> 32);
      const float x = __int2float_rz(h), d = (float)(h - __float2int_rz(x)) * (3.14159265f * 0x1p-31f);
      float sine, cosine;
      sincospif(x * 0x1p-31f, &sine, &cosine);
      sn[e] = fmaf(d, cosine, sine);
      cs[e] = fmaf(-d, sine, cosine);
    }
  };
  const T* k_row = k + (w0 + i0) * ldk;
  const T* v_row = v + (w0 + i0) * ldv;
  uint8_t* k_codes = c.k + (size_t)mine.slot * Hkv * D + 8 * l;
  uint8_t* v_codes = c.v + (size_t)mine.slot * Hkv * D + 8 * l;
  float* ks_row = c.ks + (size_t)(mine.slot / kBlock) * Hkv;
  float* vs_row = c.vs + (size_t)(mine.slot / kBlock) * Hkv;
  // A head's rows of this lane's token, and the scales that their blocks have so far.
  struct Rows {
    RawHalves<T, D> k, v;
    float old_k, old_v;
  };
  auto load = [&](int h) {
    Rows x;
    x.k.load(k_row + h * D, l);
    x.v.load(v_row + h * D, l);
    x.old_k = mine.off > 0 ? ks_row[h] : 0.f;
    x.old_v = mine.off > 0 ? vs_row[h] : 0.f;
    return x;
  };
  // (the first head's rows on their way before the angles are computed)
  const int h_begin = max(u_begin - Hq, 0), h_end = max(u_end - Hq, 0);
  Rows next;
  if (mine.live && h_begin < h_end) next = load(h_begin);
  float cs[8], sn[8];
  angles(w0 + i0, cs, sn);

  for (int u = u_begin; u < min(u_end, Hq); ++u) {
    const long long n = w0 + i0;
    if (n < N) {
      RawHalves<T, D> raw;
      raw.load(q + n * ldq + (long long)u * D, l);
      Halves x;
      x.from(raw);
      if (rope) x.rotate(cs, sn);
      T* dst = q_out + ((size_t)n * Hq + u) * D + 8 * l;
      store8(dst, x.lo);
      store8(dst + D / 2, x.hi);
    }
  }
  // The largest of a row, to shared memory.  (fmax passes over NaN; infinities are looked for only where there
  // is one.)  Returns whether the warp has one.
  auto row_top = [&](const Halves& x, int w, int i) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(fmaxf(m, fabsf(x.lo[e])), fabsf(x.hi[e]));
    const bool inf = __any_sync(0xffffffffu, m == INFINITY);
    if (inf) {
      m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(finite_abs(x.lo[e]), finite_abs(x.hi[e])));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (l == 0) row_max[w][i] = m;
    return inf;
  };
  // The largest of a token's group.
  auto group_top = [&](int w, const Token& x) {
    float m = 0.f;
    if (whole) {
      m = row_max[w][lane % kWindow];
#pragma unroll
      for (int o = kWindow / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    } else {
      for (int i = max(x.lead, 0); i < x.end; ++i) m = fmaxf(m, row_max[w][i]);
    }
    return m;
  };
  // The row of the token 16 further on, where the window's last group goes on to it: read for its maximum,
  // and once more for its codes.
  auto behind = [&](const Token& x, int h, Halves& yk, Halves& yv) {
    yk.zero();
    yv.zero();
    if (!x.live) return;
    const long long n = w0 + i0 + kWindow;
    RawHalves<T, D> raw;
    raw.load(k + n * ldk + (long long)h * D, l);
    yk.from(raw);
    raw.load(v + n * ldv + (long long)h * D, l);
    yv.from(raw);
    if (rope) {
      float c1[8], s1[8];
      angles(n, c1, s1);
      yk.rotate(c1, s1);
    }
  };
  // (a loop of its own for the windows with a second round, which needs more registers)
  auto heads = [&](auto goes_on) {
    for (int h = h_begin; h < h_end; ++h) {
      // (the value row stays as it is in memory until it is encoded)
      Halves xk;
      const RawHalves<T, D> raw_v = next.v;
      const float old_k = mine.live ? next.old_k : 0.f, old_v = mine.live ? next.old_v : 0.f;
      bool inf_v;
      {
        Halves xv;
        xk.zero();
        xv.zero();
        if (mine.live) {
          xk.from(next.k);
          xv.from(raw_v);
          if (h + 1 < h_end) next = load(h + 1);
        }
        inf_v = row_top(xv, 1, i0);
      }
      if (rope) xk.rotate(cs, sn);   // (not by an angle of 0: a NaN would reach its partner)
      const bool inf_k = row_top(xk, 0, i0);
      if (l == 0) {
        held[0][i0] = old_k;
        held[1][i0] = old_v;
      }
      if constexpr (decltype(goes_on)::value) {
        const Token last = token(i0 + kWindow);
        Halves yk, yv;
        behind(last, h, yk, yv);
        row_top(yk, 0, i0 + kWindow);
        row_top(yv, 1, i0 + kWindow);
      }
      __syncthreads();
      const float sk = fmaxf(block_scale(group_top(0, mine)), old_k);
      const float sv = fmaxf(block_scale(group_top(1, mine)), old_v);
      const bool leads = mine.live && mine.lead == i0;
      const bool grows_k = leads && mine.off > 0 && sk > old_k, grows_v = leads && mine.off > 0 && sv > old_v;
      if (mine.live) {
        xk.encode(k_codes + h * D, k_codes + h * D + D / 2, inverse_scale(sk), inf_k);
        Halves xv;
        xv.from(raw_v);
        xv.encode(v_codes + h * D, v_codes + h * D + D / 2, inverse_scale(sv), inf_v);
      }
      if (l == 0) {
        if (leads) {
          ks_row[h] = sk;
          vs_row[h] = sv;
        }
        grown[0][i0] = grows_k ? make_float2(old_k, sk) : make_float2(0.f, 0.f);
        grown[1][i0] = grows_v ? make_float2(old_v, sv) : make_float2(0.f, 0.f);
      }
      if constexpr (decltype(goes_on)::value) {
        const Token last = token(i0 + kWindow);
        Halves yk, yv;
        behind(last, h, yk, yv);
        const float tk = group_top(0, last), tv = group_top(1, last);
        if (last.live) {
          const size_t at = ((size_t)last.slot * Hkv + h) * D + 8 * l;
          yk.encode(c.k + at, c.k + at + D / 2, inverse_scale(fmaxf(block_scale(tk), held[0][last.lead])), true);
          yv.encode(c.v + at, c.v + at + D / 2, inverse_scale(fmaxf(block_scale(tv), held[1][last.lead])), true);
        }
      }
      // Blocks whose scale grew: their earlier codes, a row per group of lanes.
      if (__syncthreads_or(grows_k || grows_v)) {
        for (int i = 0; i < kWindow; ++i) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float2 g = grown[w][i];
            if (g.y == 0.f) continue;
            const int cp = __shfl_sync(0xffffffffu, cp_t, i);
            const long long row = __shfl_sync(0xffffffffu, row_t, i);
            bool ok;
            const long long at = c.slot(row, cp / kBlock * kBlock, ok) + i0;
            if (i0 >= cp % kBlock || !ok) continue;
            const float ratio = g.x * inverse_scale(g.y);
            uint32_t* p = reinterpret_cast<uint32_t*>((w ? c.v : c.k) + ((size_t)at * Hkv + h) * D + 16 * l);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y[4];
              decode4(p[e], y);
              p[e] = encode4(y, ratio);
            }
          }
        }
      }
    }
  };
  if (more) heads(std::true_type{});
  else heads(std::false_type{});
}

// ---------------------------------------------------------------------------------------------
// Reading back: a warp takes a token (or, with few tokens, a share of its rows), lanes that write 16 bytes
// each a row of one head, first of k, then of v.
// ---------------------------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadRows = 8;          // rows in flight per group of lanes

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads)
read_e4m3_kernel(const Cache8 c, T* __restrict__ k, T* __restrict__ v, long long N, int Hkv, int chunks,
                 int per_chunk) {
  constexpr int E = 16 / sizeof(T), LPR = D / E, RPW = 32 / LPR, U = kReadRows;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const unsigned item = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
  const long long n = item / (unsigned)chunks;
  if (n >= N) return;
  const int rows = 2 * Hkv;
  const int r_begin = (int)(item % (unsigned)chunks) * per_chunk, r_end = min(r_begin + per_chunk, rows);
  const int cp = c.cache_pos[n];
  bool ok = false;
  long long slot = -1;
  if (cp >= 0) {
    slot = c.slot(c.page_rows ? (long long)c.page_rows[n] : n, cp, ok);
    if (!ok && lane == 0) report(PG_ERR_DEVICE);
  }
  for (int r0 = r_begin; r0 < r_end; r0 += RPW * U) {
    uint32_t raw[U][E / 4];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) raw[u][e] = 0u;
      s[u] = 0.f;
      if (r < r_end && ok) {
        const int h = r < Hkv ? r : r - Hkv;
        const uint8_t* src = (r < Hkv ? c.k : c.v) + ((size_t)slot * Hkv + h) * D + E * l;
        if constexpr (E == 8) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          raw[u][0] = x.x;
          raw[u][E / 4 - 1] = x.y;
        } else {
          raw[u][0] = *reinterpret_cast<const uint32_t*>(src);
        }
        s[u] = (r < Hkv ? c.ks : c.vs)[(size_t)(slot / kBlock) * Hkv + h];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r >= r_end) continue;
      const int h = r < Hkv ? r : r - Hkv;
      T* dst = (r < Hkv ? k : v) + ((size_t)n * Hkv + h) * D + E * l;
      float y[E / 4][4];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        decode4(raw[u][e], y[e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[e][i] *= s[u];
      }
      if constexpr (E == 8)
        *reinterpret_cast<uint4*>(dst) = make_uint4(
            sm100::pack_bf16x2(y[0][0], y[0][1]), sm100::pack_bf16x2(y[0][2], y[0][3]),
            sm100::pack_bf16x2(y[E / 4 - 1][0], y[E / 4 - 1][1]),
            sm100::pack_bf16x2(y[E / 4 - 1][2], y[E / 4 - 1][3]));
      else store4(dst, y[0]);
    }
  }
}

template <typename T, int D>
pg_status append_t(int64_t n, int Hq, int Hkv, const void* q, int64_t ldq, void* q_out,
                   const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* positions,
                   float theta, const Cache8& c, cudaStream_t s) {
  // A CTA per window once the windows fill the GPU, else its heads are shared (16 tokens, 40 heads: append
  // and read back 6.6 us, without 23.5; 2048 windows 52.6 and 51.7).
  const int units = Hq + Hkv;
  const int64_t windows = (n + kWindow - 1) / kWindow;
  const int want = (int)std::min<int64_t>(units, std::max<int64_t>(1, (int64_t)kSMs * 16 / windows));
  const int per = (units + want - 1) / want, chunks = (units + per - 1) / per;
  prof_begin(PG_KERNEL_CACHE_APPEND, s);
  append_e4m3_kernel<T, D><<<(unsigned)(windows * chunks), D, 0, s>>>(
      static_cast<const T*>(q), ldq, static_cast<T*>(q_out), static_cast<const T*>(k), ldk,
      static_cast<const T*>(v), ldv, positions, rope_freq(D, theta), theta > 0.f, c, n, Hq, Hkv,
      chunks, per);
  prof_end(PG_KERNEL_CACHE_APPEND, s);
  return cuda_check(cudaGetLastError(), "e4m3 cache append launch");
}

template <typename T, int D>
pg_status read_t(int64_t n, int Hkv, const Cache8& c, void* k, void* v, cudaStream_t s) {
  constexpr int kStep = 32 / (D / (16 / (int)sizeof(T)));        // rows that a warp takes at a time
  const int rows = 2 * Hkv, steps = (rows + kStep - 1) / kStep;
  const int want = (int)std::min<int64_t>(steps, std::max<int64_t>(1, (int64_t)kSMs * 32 / n));
  const int per = (steps + want - 1) / want * kStep, chunks = (rows + per - 1) / per;
  const int64_t blocks = (n * chunks + kReadThreads / 32 - 1) / (kReadThreads / 32);
  prof_begin(PG_KERNEL_CACHE_READ, s);
  read_e4m3_kernel<T, D><<<(unsigned)blocks, kReadThreads, 0, s>>>(
      c, static_cast<T*>(k), static_cast<T*>(v), n, Hkv, chunks, per);
  prof_end(PG_KERNEL_CACHE_READ, s);
  return cuda_check(cudaGetLastError(), "e4m3 cache read launch");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What both calls ask of the cache and the tokens.
pg_status check_cache(const char* who, pg_dtype dtype, int64_t n_tokens, int32_t heads_kv,
                      int32_t head_dim, const Cache8& c) {
  const int32_t ps = c.page_size;
  if ((dtype != PG_F32 && dtype != PG_BF16) || n_tokens < 1 || n_tokens >= (1ll << 27) ||
      heads_kv < 1 || heads_kv > 65536 || (head_dim != 64 && head_dim != 128)) {
    set_error("%s: needs dtype f32 or bf16, 1 <= n_tokens < 2^27, heads_kv >= 1, head_dim 64 or 128", who);
    return PG_ERR_INVALID_ARG;
  }
  if ((ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) || c.num_pages < 1 ||
      c.num_page_rows < 1 || c.pages_per_row < 1 || c.pages_stride < c.pages_per_row ||
      (!c.page_rows && c.num_page_rows < n_tokens)) {
    set_error("%s: page_size must be 16, 32, 64, 128 or 256, the cache and the page table non-empty, "
              "pages_stride >= pages_per_row, and without page_rows a table row per token", who);
    return PG_ERR_INVALID_ARG;
  }
  if (!c.k || !c.v || !c.ks || !c.vs || !c.pages || !c.cache_pos || !aligned16(c.k) ||
      !aligned16(c.v) || !aligned16(c.ks) || !aligned16(c.vs)) {
    set_error("%s: the caches and their scales must be non-NULL and 16-byte aligned, pages and cache_pos "
              "non-NULL", who);
    return PG_ERR_INVALID_ARG;
  }
  return PG_OK;
}

}  // namespace

pg_status read_status_cache8(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_cache8, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_cache8, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg

using namespace pg;

extern "C" {

pg_status pg_cache_append_e4m3(pg_dtype dtype, int64_t n_tokens, int32_t heads_q, int32_t heads_kv,
                               int32_t head_dim, const void* q, int64_t ldq, void* q_out,
                               const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const int32_t* positions, float rope_theta, void* k_codes,
                               void* v_codes, float* k_scales, float* v_scales, int64_t num_pages,
                               int32_t page_size, const int32_t* pages, int32_t num_page_rows,
                               int32_t pages_per_row, int64_t pages_stride,
                               const int32_t* page_rows, const int32_t* cache_pos,
                               pg_stream_t stream) {
  const char* who = "pg_cache_append_e4m3";
  const Cache8 c{static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(v_codes), k_scales, v_scales,
                 num_pages, pages_stride, pages, page_rows, cache_pos, page_size, num_page_rows,
                 pages_per_row};
  pg_status st = check_cache(who, dtype, n_tokens, heads_kv, head_dim, c);
  if (st != PG_OK) return st;
  const int64_t unit = dtype == PG_F32 ? 4 : 8, kv_row = (int64_t)heads_kv * head_dim;
  if (!(rope_theta >= 0.f) || !k || !v || !aligned16(k) || !aligned16(v) || ldk % unit || ldv % unit ||
      ldk < kv_row || ldv < kv_row) {
    set_error("%s: rope_theta must be >= 0, k and v non-NULL and 16-byte aligned, ldk and ldv multiples of "
              "16 bytes covering a row", who);
    return PG_ERR_INVALID_ARG;
  }
  if (heads_q < 0 || heads_q > 65536 ||
      (heads_q > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out) || ldq % unit ||
                       ldq < (int64_t)heads_q * head_dim))) {
    set_error("%s: heads_q must be in [0, 65536], q and q_out non-NULL and 16-byte aligned, ldq a multiple of "
              "16 bytes covering a row", who);
    return PG_ERR_INVALID_ARG;
  }
  auto fn = dtype == PG_F32
                ? (head_dim == 64 ? append_t<float, 64> : append_t<float, 128>)
                : (head_dim == 64 ? append_t<__nv_bfloat16, 64> : append_t<__nv_bfloat16, 128>);
  return fn(n_tokens, heads_q, heads_kv, q, ldq, q_out, k, ldk, v, ldv, positions, rope_theta, c,
            reinterpret_cast<cudaStream_t>(stream));
}

pg_status pg_cache_read_e4m3(pg_dtype dtype, int64_t n_tokens, int32_t heads_kv, int32_t head_dim,
                             const void* k_codes, const void* v_codes, const float* k_scales,
                             const float* v_scales, int64_t num_pages, int32_t page_size,
                             const int32_t* pages, int32_t num_page_rows, int32_t pages_per_row,
                             int64_t pages_stride, const int32_t* page_rows,
                             const int32_t* cache_pos, void* k, void* v, pg_stream_t stream) {
  const char* who = "pg_cache_read_e4m3";
  const Cache8 c{static_cast<uint8_t*>(const_cast<void*>(k_codes)),
                 static_cast<uint8_t*>(const_cast<void*>(v_codes)), const_cast<float*>(k_scales),
                 const_cast<float*>(v_scales), num_pages, pages_stride, pages, page_rows, cache_pos,
                 page_size, num_page_rows, pages_per_row};
  pg_status st = check_cache(who, dtype, n_tokens, heads_kv, head_dim, c);
  if (st != PG_OK) return st;
  if (!k || !v || !aligned16(k) || !aligned16(v)) {
    set_error("%s: k and v must be non-NULL and 16-byte aligned", who);
    return PG_ERR_INVALID_ARG;
  }
  auto fn = dtype == PG_F32 ? (head_dim == 64 ? read_t<float, 64> : read_t<float, 128>)
                            : (head_dim == 64 ? read_t<__nv_bfloat16, 64> : read_t<__nv_bfloat16, 128>);
  return fn(n_tokens, heads_kv, c, k, v, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
