// One-token attention over the shared prefix on the 5th-generation tensor cores, for a cache in 8 bits:
// the form of pg_attn_decode_sm100.cu (work items, two streams of tiles per CTA, roles, TMEM) for e4m3
// codes with a scale per 16 slots and head.
//
// The products are of 8-bit numbers, so a code goes from memory to the tensor core as it is.  (Making bf16
// tiles of the codes would move 224 KB through shared memory per 128-key tile, 0.9 us, while its 32 KB arrive
// in 0.74.)  What is not in 8 bits enters as a sum of two 8-bit numbers, at twice the
// rate of 16-bit ones:
//   q = (q1 + q2) 2^a, both e4m3, 2^a the row's scale as of a block of the cache: a bf16 number has 8 bits,
//     q1 takes four of them and q2 the rest, exact but for half of its least
//     step of 2^-9, the row's largest element being 224 at least: 2^-17 of that.
//   w = w1 + w2: with f the softmax scale times log2 e times 2^a and the key's scale, and 2^e the value's scale,
//     the weight that meets a value's code is w = 2^(f s + e - m + 7), m the running maximum of f s + e (w may reach
//     2^11 before the reference m moves).  As an fp16 number, w1 is its nearest e5m2 number (the upper byte
//     of an fp16 number) and w2 the rest as e4m3: off by 2^-7 of w at most, and at w < 2^-3, 2^-10 of a
//     weight of the maximum or less, by 2^-10 or 2^-3 of w, the smaller; so no weight is lost down to 2^-23
//     of the largest, however many small ones there are.
// The row's sum adds the fp32 w 2^(E - e), 2^E the sum's unit: the largest scale of a value so far, or 2^60 times the
// least of a tile where that is less (keys of the largest scores may have values of zeros, whose block has the
// scale 2^-126, and weigh 2^118 of others).  A unit is raised as long as the sum stays below 2^64; where it lags behind,
// what is added meanwhile is added to 2^63 or more.  A scale below 2^-118 of the largest so far counts as that.
//
// Pages, tiles and what happens at a prefix's end are as in pg_attn_decode_sm100.cu.
//
// Four threads share a query row and stream: each has half of a tile's columns, so that its 32 + 32 scores pass
// through registers in two halves (two threads a row: 229 us for the step below, spilling).  The weights of 32 columns
// go over their own scores, and the product of tile j and the scores of tile j + 2 follow one another in
// the same columns.
// Keys, values and scales have a warp each that brings them: a tile's loads are a chain of short instructions beside
// 16 busy warps, 0.9 us of a single warp's time (loads alone 102 us for the step below; with three warps 59).
// 4 groups of 64 responses, 4 query heads to a key/value head, over 32768 keys: 149 us for 269 MB (of which each half
// is read by two CTAs: 538 MB), 1.17 us per tile and CTA; the whole step 200.  What bounds it is the softmax
// (122 us without the products) and the products (111 without the softmax; a stream's tile waits for the
// scores, the scores for the products before them).  The tensor pipe is busy for 41 % of the time, the issue slots
// for 51 %.  Tried without gain: a third buffer of scores with one output (204), halves of tiles in work at a time
// (219), scores kept in registers between the maximum and the weights, five stages or three (202, 206), one pass over
// the scores that is repeated where a maximum has grown (181 for the kernel).
#include <math.h>

#include <algorithm>

#include "pg_decode.h"
#include "pg_e4m3.cuh"
#include "pg_rowsoftmax.cuh"
#include "pg_sm100.cuh"
#include "pg_tmap.h"

namespace pg {

using namespace sm100;
using namespace rowsoftmax;
using namespace e4m3;

namespace {

constexpr int BM = 128;                 // query rows
constexpr int BN = kDecodeTile;         // keys per tile
constexpr int NS = 4;                   // stages of each ring
constexpr int kBlock = 16;              // keys that share a scale
constexpr int kTileBlocks = BN / kBlock;
constexpr int NTHREADS = 640;            // warps: keys, MMA issuer, 16 of the softmax, values, scales
constexpr int kSoftmaxThreads = 512;
constexpr float kRescaleThreshold = 4.0f;
constexpr float kShift = 7.f;           // weights enter the product times 2^kShift
constexpr int kScaleRange = 118;   // exponents of scales that are told apart
constexpr int kUnitRange = 60;     // and the largest that a weight is multiplied by
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ int s_status_decode8 = 0;

__device__ __forceinline__ void fail(int code) { atomicCAS(&s_status_decode8, 0, code); }

template <int D>
struct PrefixSmem {
  uint8_t q[2][BM * D];          // q1, q2
  uint8_t k[NS][BN * D];
  uint8_t v[NS][BN * D];
  float scale[NS][2 * kTileBlocks];    // of a tile's keys and values
  float amax[4][BM];             // of quarters of a query row
  float top[2][2][BM];           // [stream][half of a tile] the largest score of a row's tile
  float m[2][BM];                // the streams' maxima
  float l[4][BM], x[4][BM];      // of their halves the sums as l 2^x, 1 <= l < 2
  uint64_t q_full;
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t scale_full[NS], s_full[2], p_full[2], pv_done[2];
  uint64_t mma_done;
  uint32_t tmem;
};
static_assert(sizeof(PrefixSmem<128>) + 1024 <= 232448, "prefix attention shared memory");

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D>
__device__ __forceinline__ uint64_t tile_desc(const uint8_t* p) {    // rows of D bytes
  return D == 128 ? sdesc_sw128(smem_u32(p), 16, 1024) : sdesc_sw64(smem_u32(p), 16, 512);
}

__device__ __forceinline__ float pow2i(int i) { return __int_as_float((i + 127) << 23); }
__device__ __forceinline__ int exponent(float s) { return (__float_as_int(s) >> 23 & 0xff) - 127; }

// l 2^x of a sum l: 0 stays 0 (x may be NaN or out of range then).
__device__ __forceinline__ float scaled(float l, float x) { return l == 0.f ? 0.f : l * ex2(x); }

// Four weights: their e5m2 neighbours w1 (upper bytes of fp16 numbers), and what those leave of their fp16
// values, as e4m3, w2.
__device__ __forceinline__ void split4(const float (&p)[4], uint32_t& w1, uint32_t& w2) {
  uint32_t h[2];
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e5m2x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e5m2x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}"
      : "=r"(w1)
      : "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(p[1]), "f"(p[0]));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(p[3]), "f"(p[2]));
  const uint32_t u[2] = {__byte_perm(w1, 0u, 0x1404), __byte_perm(w1, 0u, 0x3424)};
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[0]) : "r"(u[0]));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[1]) : "r"(u[1]));
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}"
      : "=r"(w2)
      : "r"(h[0]), "r"(h[1]));
}

// The scores of 32 columns (c0 .. of a tile with `len` keys) that belong to no key.
__device__ __forceinline__ void mask32(uint32_t (&r)[32], int c0, int len) {
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = c0 + i < len ? r[i] : 0xff800000u;
}

// w = 2^(s k + d) of the 16 raw scores of a block, as w1 and w2 words (four weights each); returns their sum.
__device__ __forceinline__ float weights16(const uint32_t* r, float k, float d, uint32_t* w1, uint32_t* w2) {
  const uint64_t k2 = f2_pack(k, k), d2 = f2_pack(d, d);
  uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float e0, e1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(r[4 * i + j]), __uint_as_float(r[4 * i + j + 1])), k2, d2),
                e0, e1);
      p[j] = ex2(e0);
      p[j + 1] = ex2(e1);
      sum2 = f2_add(sum2, f2_pack(p[j], p[j + 1]));
    }
    split4(p, w1[i], w2[i]);
  }
  float s0, s1;
  f2_unpack(sum2, s0, s1);
  return s0 + s1;
}

// 16 consecutive columns.
__device__ __forceinline__ float top16(const uint32_t* r) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 16; i += 2) top = fmax3(top, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
  return top;
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
decode_prefix_e4m3_kernel(const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const float* __restrict__ k_scales,
                          const float* __restrict__ v_scales, const __nv_bfloat16* __restrict__ q,
                          const DecodeItem* __restrict__ items, const int32_t* __restrict__ pages,
                          long long pages_stride, int num_pages, int page_shift,
                          float* __restrict__ part_o, float* __restrict__ part_lse, int S, int Hq,
                          int Hkv, float scale_log2) {
  const int page_size = 1 << page_shift;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  PrefixSmem<D>& sm = *reinterpret_cast<PrefixSmem<D>*>(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const DecodeItem it = items[blockIdx.x / Hkv];     // the plan's: written long before
  const int kh = blockIdx.x % Hkv, hp = Hq / Hkv;
  const int rows = it.n_seq * hp;
  const int n = (it.key_hi - it.key_lo + BN - 1) / BN;      // key tiles, at least one

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, kSoftmaxThreads / 32);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
      mbar_init(&sm.scale_full[s], 2 * kTileBlocks);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftmaxThreads / 64);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // Every role has its resources: the own-key kernel's CTAs may start beside this grid.
  launch_dependents();

  constexpr int kValues = 18, kScales = 19;
  if (warp == 0 || warp == kValues) {
    // ------------------------------------------------------------------ TMA producers ----
    // One for the keys and one for the values.
    const int R = min(page_size, BN), pieces = BN / R;
    const int32_t* row = pages + (long long)it.group * pages_stride;
    const int oob = num_pages * page_size;     // a box of zeros
    const CUtensorMap* map = warp == 0 ? &tk : &tv;
    uint8_t(*ring)[BN * D] = warp == 0 ? sm.k : sm.v;
    uint64_t *full = warp == 0 ? sm.k_full : sm.v_full, *empty = warp == 0 ? sm.k_empty : sm.v_empty;
    // This lane's page of tile j, read two tiles ahead and looked at when the tile is loaded.
    auto has_box = [&](int j) { return j < n && lane < pieces && it.key_lo + j * BN + lane * R < it.key_hi; };
    auto read_page = [&](int j) { return has_box(j) ? row[(it.key_lo + j * BN + lane * R) >> page_shift] : 0; };
    if (lane == 0) prefetch_tmap(map);
    int page = read_page(0), page1 = read_page(1), issued = 0;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int page2 = read_page(j + 2), s = j % NS;
      int y = -1;              // the cache row that the box starts at
      if (has_box(j)) {
        y = (page << page_shift) + ((it.key_lo + j * BN + lane * R) & (page_size - 1));
        if (page < 0 || page >= num_pages) {
          fail(PG_ERR_DEVICE);
          y = oob;
        }
      }
      ok = warp_wait(&empty[s], ((j / NS) & 1) ^ 1, kWaitNs);
      if (!ok) break;
      const int left = it.key_hi - (it.key_lo + j * BN);
      if (lane == 0) mbar_expect_tx(&full[s], (uint32_t)(min((left + R - 1) / R, pieces) * R) * (uint32_t)D);
      __syncwarp();
      if (y >= 0) tma_load_2d(ring[s] + lane * R * D, map, &full[s], kh * D, y);
      ++issued;
      page = page1;
      page1 = page2;
    }
    __syncwarp();
    if (!ok && lane == 0) fail(PG_ERR_TIMEOUT);
    // Leave no copy in flight: the last stages' loads must have landed before exit.
    for (int j = max(issued - NS, 0); j < issued; ++j) mbar_wait(&full[j % NS], (j / NS) & 1, kWaitNs);
    __syncwarp();
  } else if (warp == kScales) {
    // ------------------------------------------------------------------ the scales -------
    // Lane b < 8 fetches the key scale of block b of a tile, lanes 8-15 the value scales, into the stage of the
    // values.  A block without keys (or on a bad page) counts with the least scale.
    const int32_t* row = pages + (long long)it.group * pages_stride;
    auto key_of = [&](int j) { return it.key_lo + j * BN + (lane & (kTileBlocks - 1)) * kBlock; };
    auto has = [&](int j) { return j < n && lane < 2 * kTileBlocks && key_of(j) < it.key_hi; };
    auto read_page = [&](int j) { return has(j) ? row[key_of(j) >> page_shift] : -1; };
    int page = read_page(0), page1 = read_page(1);
    for (int j = 0; j < n; ++j) {
      const int page2 = read_page(j + 2), s = j % NS;
      if (!warp_wait(&sm.v_empty[s], ((j / NS) & 1) ^ 1, kWaitNs)) break;     // (the values' warp reports it)
      if (lane < 2 * kTileBlocks) {
        float* dst = &sm.scale[s][lane];
        if (page >= 0 && page < num_pages) {
          const int slot = (page << page_shift) + (key_of(j) & (page_size - 1));
          const float* src = (lane < kTileBlocks ? k_scales : v_scales) + (size_t)(slot / kBlock) * Hkv + kh;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.scale_full[s]))
                       : "memory");
        } else {
          *dst = pow2i(-126);
          mbar_arrive(&sm.scale_full[s]);
        }
      }
      page = page1;
      page1 = page2;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer -------
    // S(0), S(1), then for each tile j its P V product and the scores of tile j + 2, which overwrite
    // the columns P(j) was read from: the tensor core executes them in issue order.
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_f8(BM, BN, 0, 0, 0, 0);
      constexpr uint32_t idesc_w1 = idesc_f8(BM, D, 1, 0, 0, 1), idesc_w2 = idesc_f8(BM, D, 0, 0, 0, 1);
      const uint64_t qd = tile_desc<D>(sm.q[0]);
      const uint64_t kd0 = tile_desc<D>(sm.k[0]);
      const uint64_t vd0 = tile_desc<D>(sm.v[0]);
      auto keys = [&](int j) { return mbar_wait(&sm.k_full[j % NS], (j / NS) & 1, kWaitNs); };
      auto issue_s = [&](int j) {
        const uint64_t kd = desc_add(kd0, (j % NS) * BN * D);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma8_ss(tmem + 128 * (j & 1), desc_add(qd, i * BM * D + kk * 32), desc_add(kd, kk * 32),
                    idesc_s, (i | kk) != 0);
        mma_commit(&sm.s_full[j & 1]);
        mma_commit(&sm.k_empty[j % NS]);
      };
      bool ok = mbar_wait(&sm.q_full, 0, kWaitNs) && keys(0) && (n < 2 || keys(1));
      if (ok) {
        tc_fence_after();
        issue_s(0);
        if (n > 1) issue_s(1);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int i = j & 1;
        // (the weights last: what they release is ready then)
        ok = mbar_wait(&sm.v_full[j % NS], (j / NS) & 1, kWaitNs) && (j + 2 >= n || keys(j + 2)) &&
             mbar_wait(&sm.p_full[i], (j >> 1) & 1, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = desc_add(vd0, (j % NS) * BN * D);
#pragma unroll
        for (int kk = 0; kk < BN / 32; ++kk) {
          mma8_ts(tmem + 256 + 128 * i, tmem + 128 * i + 32 * kk, desc_add(vd, kk * 32 * D), idesc_w1,
                  kk == 0 ? (uint32_t)(j >= 2) : 1u);
          mma8_ts(tmem + 256 + 128 * i, tmem + 128 * i + 32 * kk + 8, desc_add(vd, kk * 32 * D),
                  idesc_w2, 1u);
        }
        mma_commit(&sm.pv_done[i]);
        mma_commit(&sm.v_empty[j % NS]);
        if (j + 2 < n) issue_s(j + 2);
      }
      if (!ok) fail(PG_ERR_TIMEOUT);
      mma_commit(&sm.mma_done);
      mbar_wait(&sm.mma_done, 0, kWaitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax ----------
    // Two warps per 32 rows and stream, each for half of a tile's columns.
    const int i = (warp - 2) >> 3, half = (warp - 2) >> 2 & 1, part = 2 * i + half;
    const int quarter = warp & 3;
    const int m = quarter * 32 + lane;               // query row
    const bool valid = m < rows;
    const bool any_valid = __any_sync(0xffffffffu, valid);
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + 128 * i + 64 * half + lane_addr;
    const uint32_t t_o = tmem + 256 + 128 * i + D / 2 * half + lane_addr;
    const int s = it.s0 + (valid ? m / hp : 0), h = kh * hp + m % hp;
    float f;
    {
      // The four threads of a row bring it into shared memory, as q1 and q2.
      constexpr int QD = D / 4;
      uint4 raw[QD / 8];
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < QD / 8; ++e) {
        raw[e] = make_uint4(0u, 0u, 0u, 0u);
        if (valid)
          raw[e] = *reinterpret_cast<const uint4*>(q + ((size_t)s * Hq + h) * D + part * QD + 8 * e);
      }
#pragma unroll
      for (int e = 0; e < QD / 8; ++e)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t w = u == 0 ? raw[e].x : u == 1 ? raw[e].y : u == 2 ? raw[e].z : raw[e].w;
          amax = fmaxf(amax, fmaxf(finite_abs(__uint_as_float(w << 16)),
                                   finite_abs(__uint_as_float(w & 0xffff0000u))));
        }
      sm.amax[part][m] = amax;
      named_bar_sync(1, kSoftmaxThreads);
      amax = fmaxf(fmaxf(sm.amax[0][m], sm.amax[1][m]), fmaxf(sm.amax[2][m], sm.amax[3][m]));
      const float scale = block_scale(amax), inv = inverse_scale(scale);
      f = scale_log2 * scale;
#pragma unroll
      for (int c = 0; c < QD / 16; ++c) {
        uint32_t w1[4], w2[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4& v = raw[2 * c + (u >> 1)];
          const uint32_t a = u & 1 ? v.z : v.x, b = u & 1 ? v.w : v.y;
          const float x[4] = {__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u),
                              __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)};
          float y[4];
          w1[u] = encode4(x, inv);
          decode4(w1[u], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = fmaf(x[e], inv, -y[e]);
          w2[u] = encode4(y, 1.f);
        }
        const uint32_t chunk = part * (QD / 16) + c;
        const uint32_t off = D == 128 ? sw128_offset(m, chunk) : sw64_offset(m, chunk);
        *reinterpret_cast<uint4*>(sm.q[0] + off) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        *reinterpret_cast<uint4*>(sm.q[1] + off) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
      }
      fence_proxy_async_smem();
      warp_arrive(&sm.q_full);
    }

    constexpr int kHalfBlocks = kTileBlocks / 2;
    int e_ref = -126, unit = -126;   // the largest scale of a value so far, and the sum's unit
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    int c = 0;
    for (int j = i; j < n; j += 2, ++c) {
      const int st = j % NS;
      ok = ok && warp_wait(&sm.scale_full[st], (j / NS) & 1, kWaitNs);
      ok = ok && warp_wait(&sm.s_full[i], c & 1, kWaitNs);
      const int len = min(it.key_hi - (it.key_lo + j * BN), BN);
      const bool full_tile = len == BN;
      if (!full_tile) {
        // The prefix ends in this tile: zero the value rows behind its end.
        ok = ok && warp_wait(&sm.v_full[st], (j / NS) & 1, kWaitNs);
        const int t = ((warp - 2) & 7) * 32 + lane;
        for (int idx = t; idx < (BN - len) * (D / 16); idx += kSoftmaxThreads / 2)
          *reinterpret_cast<uint4*>(sm.v[st] + len * D + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
      }
      if (!any_valid) {
        // Rows of no response: keep the barrier protocol; their outputs are never stored.  (Both halves.)
        if (!ok) break;
        warp_arrive(&sm.p_full[i]);
        continue;
      }
      // The tile's scales, and the unit they ask for.
      const float4 ks4 = *reinterpret_cast<const float4*>(&sm.scale[st][half * kHalfBlocks]);
      const float4 vs4 = *reinterpret_cast<const float4*>(&sm.scale[st][kTileBlocks + half * kHalfBlocks]);
      const int4 e4 = make_int4(exponent(vs4.x), exponent(vs4.y), exponent(vs4.z), exponent(vs4.w));
      e_ref = max(max(max(e4.x, e4.y), max(e4.z, e4.w)), e_ref);
      const int e_least = e_ref - kScaleRange;
      // (a factor of 0 would make NaN of -inf)
      const float ks[kHalfBlocks] = {fmaxf(f * ks4.x, 0x1p-126f), fmaxf(f * ks4.y, 0x1p-126f),
                                     fmaxf(f * ks4.z, 0x1p-126f), fmaxf(f * ks4.w, 0x1p-126f)};
      const int eb[kHalfBlocks] = {max(e4.x, e_least), max(e4.y, e_least), max(e4.z, e_least),
                                   max(e4.w, e_least)};
      const int aim = min(e_ref, min(min(eb[0], eb[1]), min(eb[2], eb[3])) + kUnitRange);
      float mx = -INFINITY;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t sr[32];
        tmem_ld32(t_s + 32 * g, sr);
        tmem_ld_wait();
        if (!full_tile) mask32(sr, 64 * half + 32 * g, len);
#pragma unroll
        for (int b = 0; b < 2; ++b)
          mx = fmaxf(mx, fmaf(top16(sr + 16 * b), ks[2 * g + b], (float)eb[2 * g + b]));
      }
      // The row's largest, with the other half's thread.
      sm.top[i][half][m] = mx;
      ok = named_bar_and(2 + 4 * i + quarter, 64, ok);
      if (!ok) break;                              // (both warps)
      mx = fmaxf(mx, sm.top[i][half ^ 1][m]);
      // The reference moves when a row's maximum has grown past the rescale threshold; rescaling O needs
      // this stream's previous P V product done.
      const float m_old = m_used;
      const bool grow = mx > m_used + kRescaleThreshold;
      if (grow) {
        m_used = mx;
        l = scaled(l, m_old - mx);
      }
      if (aim != unit) {
        const int all = aim - unit, up = l == 0.f ? all : min(all, max(64 - exponent(l), 0));
        l = l * pow2i(up >> 1) * pow2i(up - (up >> 1));
        unit += up;
      }
      if (c > 0 && __any_sync(0xffffffffu, grow)) {
        ok = warp_wait(&sm.pv_done[i], (c - 1) & 1, kWaitNs);
        const float corr = grow ? (m_old == -INFINITY ? 0.f : ex2(m_old - m_used)) : 1.f;
        tc_fence_after();
#pragma unroll
        for (int q4 = 0; q4 < D / 64; ++q4) {
          uint32_t orr[32];
          tmem_ld32(t_o + q4 * 32, orr);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * corr);
          tmem_st32(t_o + q4 * 32, orr);
        }
      }
      const float ref = (m_used == -INFINITY ? 0.f : m_used) - kShift;
      const int from = max(unit, e_ref - 126);      // (further behind than a factor can say: next to 2^63)
      // The weights of 32 columns go over their scores: w1 in eight columns, w2 in the next.
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t sr[32], w[16];
        tmem_ld32(t_s + 32 * g, sr);
        tmem_ld_wait();
        if (!full_tile) mask32(sr, 64 * half + 32 * g, len);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int e = eb[2 * g + b];
          l = fmaf(weights16(sr + 16 * b, ks[2 * g + b], (float)e - ref, w + 4 * b, w + 8 + 4 * b),
                   pow2i(from - e), l);
        }
        tmem_st16(t_s + 32 * g, w);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm.p_full[i]);
    }
    // Merge the streams, once both have done their last product.
    // (This stream's own last product first: products complete in order, so the other stream then has
    // at most one phase to go, which its parity tells from the one before.)
    const int n1 = n / 2, mine = (n + 1 - i) / 2, other = n - mine;
    if (mine > 0) ok = ok && warp_wait(&sm.pv_done[i], (mine - 1) & 1, kWaitNs);
    if (other > 0) ok = ok && warp_wait(&sm.pv_done[i ^ 1], (other - 1) & 1, kWaitNs);
    tc_fence_after();
    sm.m[i][m] = m_used;
    // (m_used, the unit and the sum itself may be far from one another: only their sum is sure to be in range)
    const int e_l = exponent(l);
    sm.l[part][m] = l * pow2i(-e_l);
    sm.x[part][m] = l == 0.f ? -INFINITY : m_used + (float)(e_l - unit);
    ok = named_bar_and(1, kSoftmaxThreads, ok);
    if (ok && any_valid) {
      const float ma = sm.m[0][m], mb = n1 > 0 ? sm.m[1][m] : -INFINITY;
      const float M = fmaxf(ma, mb), ref = M == -INFINITY ? 0.f : M;
      float xs[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) xs[k] = k < 2 || n1 > 0 ? sm.x[k][m] : -INFINITY;
      float top = fmaxf(fmaxf(xs[0], xs[1]), fmaxf(xs[2], xs[3]));
      if (top == -INFINITY) top = 0.f;
      float L = 0.f;                       // the row's sum is L 2^top
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < 2 || n1 > 0) L = fmaf(sm.l[k][m], ex2(xs[k] - top), L);
      const float inv = L == 0.f ? 0.f : 1.f / L, out = ex2(0.5f * (ref - top));
      const float wa = ex2(ma - ref) * inv * out, wb = ex2(mb - ref) * inv * out;
      const size_t row = ((size_t)it.slot * S + s) * Hq + h;
      const bool al32 = (reinterpret_cast<uintptr_t>(part_o) & 31) == 0;
      // The row's four threads write a part of the columns each (D = 64: two of them).
#pragma unroll 1
      for (int q4 = part; q4 < D / 32; q4 += 4) {
        uint32_t xa[32], xb[32];
        tmem_ld32(tmem + 256 + lane_addr + q4 * 32, xa);
        if (n1 > 0) tmem_ld32(tmem + 384 + lane_addr + q4 * 32, xb);
        tmem_ld_wait();
        if (!valid) continue;
        float* prow = part_o + row * D + q4 * 32;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            float x = __uint_as_float(xa[e + u]) * wa;
            if (n1 > 0) x = fmaf(__uint_as_float(xb[e + u]), wb, x);
            w[u] = __float_as_uint(x * out);
          }
          if (al32) {
            st_global_v8(prow + e, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
          } else {
            *reinterpret_cast<uint4*>(prow + e) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(prow + e + 4) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
      // L is NaN when a score is; a row without weight has no log
      if (valid && part == 0)
        part_lse[row] = L == 0.f ? -INFINITY : top - kShift + log2f(L);
    }
    if (!ok && lane == 0) fail(PG_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
pg_status launch_t(const DecodeArgs& a) {
  const pg_decode_plan* p = a.plan;
  const int Hq = p->heads_q, Hkv = p->heads_kv, S = p->num_seqs;
  const uint64_t slots = (uint64_t)a.num_pages * p->page_size, row = (uint64_t)Hkv * D;
  const uint32_t R = (uint32_t)std::min<int32_t>(p->page_size, BN);
  int shift = 0;
  while ((1 << shift) < p->page_size) ++shift;
  CUtensorMap tk, tv;
  pg_status st = make_tmap_2d_u8(&tk, a.k_cache, row, slots, row, D, R);
  if (st == PG_OK) st = make_tmap_2d_u8(&tv, a.v_cache, row, slots, row, D, R);
  if (st != PG_OK) return st;
  auto kern = decode_prefix_e4m3_kernel<D>;
  const size_t smem = sizeof(PrefixSmem<D>) + 1024;
  static OncePerDevice once;
  st = once.run([&] { return allow_smem(kern, smem, "decode prefix e4m3 smem attributes"); });
  if (st != PG_OK) return st;
  prof_begin(PG_KERNEL_DECODE, a.stream);
  // (In plain stream order, for the reason at the bf16 kernel's launch.)
  const dim3 grid((unsigned)(p->n_items * Hkv));
  kern<<<grid, NTHREADS, smem, a.stream>>>(
      tk, tv, a.k_scales, a.v_scales, static_cast<const __nv_bfloat16*>(a.q), decode_items(p),
      a.prefix_pages, (long long)a.prefix_stride, (int)a.num_pages, shift, a.part_o,
      a.part_lse, S, Hq, Hkv, a.scale_log2);
  st = cuda_check(cudaGetLastError(), "decode prefix e4m3 launch");
  prof_end(PG_KERNEL_DECODE, a.stream);
  return st;
}

}  // namespace

pg_status launch_decode_prefix_e4m3(const DecodeArgs& a) {
  return a.plan->head_dim == 64 ? launch_t<64>(a) : launch_t<128>(a);
}

pg_status read_status_decode_e4m3(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_decode8, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_decode8, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg
