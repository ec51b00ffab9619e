// One-token attention over a response's own keys in 8 bits: the form of pg_attn_own.cu for a cache of
// e4m3 codes with a scale per 16 slots and head, whose split (one warp per response, key/value head, up to
// 16 query rows and part of the keys) and reasons it shares.
//
// A stage is 32 keys: boxes of 16 slots by TMA, and the four scales by asynchronous copies that arrive on
// the same barrier.  Every e4m3 number is an fp16 number, so the codes become fp16 in registers and the
// products are fp16 warp MMAs (16 x 8, 16 deep), exact up to their fp32 sums.  (The 8-bit warp MMAs are no
// choice: this architecture makes several instructions of one, 713 per stage in all, and such a kernel was slower.)
// Keys and dimensions are on the long side, the query rows on the short one, which eight rows
// (Hq / Hkv <= 8) fill:
//   S^T = K Q^T       A = 16 keys x 16 dimensions.  A matrix load moves 16-bit pairs of codes, so a lane gets four
//     consecutive dimensions of a key; the product's order over the dimensions is free, and q's fragments take
//     the same one.  The query enters as fp16, scaled by a power of two so that its largest element lies in
//     [128, 256) (a bf16 number has 8 bits, fp16 11).
//   O^T += V^T W^T    A = 16 dimensions x 16 keys.  A transposing load gives a lane (key, dimension) pairs, 2 x 2;
//     a byte permutation and two conversions make the pairs of keys of an even and an odd dimension: rows 0-7
//     of A are the even dimensions of 16, rows 8-15 the odd ones.  The weights go through an 8 x 8
//     transposition between the products.
// With f the softmax scale times log2 e times the key scale, and 2^e a value's scale, the weight that meets
// the code is w = 2^(f s + e - m), m the running maximum of f s + e: accuracy is relative to the largest
// product of weight and scale.  w enters the product as fp16 times 2^10 (11 bits down to 2^-24 of the
// largest).  The row's sum, in fp32, is of w 2^(E - e), 2^E the row's unit: the largest scale so far, or 2^60 times
// the least of a stage where that is less (keys of the largest scores may have values of zeros, whose block has the scale
// 2^-126, and weigh 2^118 of others).  A unit is raised as long as the sum stays below 2^64; where it lags
// behind, what is added meanwhile is added to 2^63 or more.  A scale below 2^-118 of the largest so far counts as that, so
// that w keeps clear of underflow.
// Every lane holds the running reference of its two query rows and its own keys' part of their sums; the
// reference moves, and lanes exchange their maxima, only when one has grown past it by kRescale.
//
// A response's keys are shared by their present number (own_parts_e4m3); the CTAs of parts that it does not fill leave.
// Bound by the bytes read, with few responses by the latency of their chain (length, page, boxes, products):
// 256 responses of 1-1537 keys, 404 MB, in 77 us with the merge (5.2 TB/s), of 512-2048 keys, 671 MB, in 119 (5.6),
// 128 responses of 0-512 keys in 22 us alone.  Three stages: two or four of them take 37.8 and 39.2 us of the latter's whole step against 37.5, but beside a long prefix, where
// two leave room for three CTAs on a prefix kernel's SM, 256 responses over 32768 keys take 192 us with two and
// 201 with three (16 over 16384 27.0 and 26.4).
#include <math.h>

#include "pg_decode.h"
#include "pg_rowsoftmax.cuh"
#include "pg_sm100.cuh"
#include "pg_tmap.h"

namespace pg {

using namespace sm100;
using rowsoftmax::ex2;

namespace {

constexpr int kKeys = 32;        // keys per stage
constexpr int kBlock = 16;       // keys per box and per scale
constexpr int kStages = 3;
constexpr int kRows = 16;        // query rows per CTA
constexpr int kScaleLanes = 2 * kKeys / kBlock;
constexpr float kShift = 10.f;   // weights enter the product times 2^kShift
constexpr float kRescale = 4.f;
constexpr int kScaleRange = 118;   // exponents of scales that are told apart
constexpr int kUnitRange = 60;     // and the largest that a weight is multiplied by
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ int s_status_own8 = 0;

__device__ __forceinline__ void fail(int code) { atomicCAS(&s_status_own8, 0, code); }

template <int D>
struct OwnSmem {
  uint8_t k[kStages][kKeys * D];
  uint8_t v[kStages][kKeys * D];
  float scale[kStages][kScaleLanes];     // k, k, v, v
  uint64_t full[kStages];
};

template <int D>
__device__ __forceinline__ uint32_t chunk_offset(uint32_t row, uint32_t chunk) {
  return D == 128 ? sw128_offset(row, chunk) : sw64_offset(row, chunk);
}

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], fp16 with fp32 accumulation.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The low and the high pair of four codes as fp16 pairs.
__device__ __forceinline__ void halves(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Transposes an 8 x 8 matrix of 16-bit elements, lane 4 i + j holding (i, 2 j) and (i, 2 j + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// l 2^x of a sum l, x at most 0: 0 stays 0 (x may be NaN then).
__device__ __forceinline__ float scaled(float l, float x) { return l == 0.f ? 0.f : l * ex2(x); }
// 2^i, -126 <= i <= 127; the exponent of a power of two (0: -127).
__device__ __forceinline__ float pow2i(int i) { return __int_as_float((i + 127) << 23); }
__device__ __forceinline__ int exponent(float s) { return (__float_as_int(s) >> 23 & 0xff) - 127; }

// RG: groups of eight query rows.
template <int D, int RG>
__global__ void __launch_bounds__(32)
decode_own_e4m3_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const float* __restrict__ k_scales, const float* __restrict__ v_scales,
                       const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ pages,
                       long long pages_stride, const int32_t* __restrict__ own_lens, int num_pages,
                       int page_shift, int own_cap, int first_slot, int fill, int parts, int row_tiles,
                       int S, int Hq, int Hkv, float scale_log2, float* __restrict__ part_o,
                       float* __restrict__ part_lse) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  OwnSmem<D>& sm = *reinterpret_cast<OwnSmem<D>*>(base);
  const int lane = threadIdx.x;
  // (As in pg_attn_own.cu: all that is read here was complete before the prefix kernel began.)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int x = blockIdx.x;
  const int kh = x % Hkv;
  x /= Hkv;
  const int rt = x % row_tiles;
  x /= row_tiles;
  const int part = x % parts, s = x / parts;
  const int hp = Hq / Hkv, h0 = kh * hp + rt * kRows, nrows = min(kRows, hp - rt * kRows);
  const int32_t* row = pages + s * pages_stride;
  const int table = own_cap >> page_shift;      // entries of a page table row
  int len = own_lens[s];
  int pg = row[min(lane, table - 1)];           // with a short table, the pages need no second wait
  if (len > own_cap) {
    if (lane == 0) fail(PG_ERR_DEVICE);
    len = own_cap;
  }
  const int part_keys = own_parts_e4m3(len, fill, parts).keys;
  const int lo = part * part_keys, hi = min(len, lo + part_keys);
  const size_t row0 = ((size_t)(first_slot + part) * S + s) * Hq + h0;
  const int g = lane >> 2, t4 = lane & 3;       // lane 4 g + t4 of the fragments

  if (lo < hi) {                 // (the merge knows as well which parts there are)
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[i], 1 + kScaleLanes);
      fence_mbar_init();
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
    __syncwarp();
    const int nt = (hi - lo + kKeys - 1) / kKeys;
    // Page numbers 32 at a time, one per lane, the next 32 read ahead.
    const int last_page = (hi - 1) >> page_shift;
    auto read_page = [&](int i) { return i <= last_page ? row[i] : 0; };
    int pbase = 0, pg_next = 0;
    if (last_page >= 32) {
      pbase = lo >> page_shift;
      pg = read_page(pbase + lane);
      pg_next = read_page(pbase + 32 + lane);
    }
    auto issue = [&](int t) {        // every lane; t in order
      const int key0 = lo + t * kKeys;
      if (key0 >> page_shift >= pbase + 32) {
        pbase += 32;
        pg = pg_next;
        pg_next = read_page(pbase + 32 + lane);
      }
      // Lanes 0, 1 load the keys of the stage's two blocks, 2, 3 the values, and their scales.  (Both
      // blocks' pages are in reach: 16-slot pages begin at even ones of the 32.)
      const int b = lane & 1, key = key0 + b * kBlock, pi = key >> page_shift;
      const int page = __shfl_sync(0xffffffffu, pg, min(pi - pbase, 31));
      const int st = t % kStages;
      if (lane == 0) mbar_expect_tx(&sm.full[st], (key0 + kBlock < hi ? 2 : 1) * 2 * kBlock * D);
      __syncwarp();
      if (lane < kScaleLanes) {
        const bool is_v = lane >= kScaleLanes / 2;
        bool copied = false;
        if (key < hi) {
          const bool bad = page < 0 || page >= num_pages;
          if (bad) fail(PG_ERR_DEVICE);        // a box behind the cache reads as zeros
          const int y = bad ? num_pages << page_shift
                            : (page << page_shift) + (key & ((1 << page_shift) - 1));
          tma_load_2d((is_v ? sm.v : sm.k)[st] + b * kBlock * D, is_v ? &tv : &tk, &sm.full[st],
                      kh * D, y);
          if (!bad) {
            const float* src = (is_v ? v_scales : k_scales) + (size_t)(y >> 4) * Hkv + kh;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                             smem_u32(&sm.scale[st][lane])),
                         "l"(src)
                         : "memory");
            copied = true;
          }
        }
        if (copied) {
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&sm.full[st]))
                       : "memory");
        } else {                 // no keys, or zeros: the least scale
          sm.scale[st][lane] = pow2i(-126);
          mbar_arrive(&sm.full[st]);
        }
      }
    };
    int issued = 0;
    for (; issued < min(kStages, nt); ++issued) issue(issued);
    // The query rows as the B operand: row g of a group; of each 16 dimensions 4 t4, 4 t4 + 1 and 4 t4 + 2,
    // 4 t4 + 3 stand where the fragment has 2 t4, 2 t4 + 1 and 2 t4 + 8, 2 t4 + 9.
    uint32_t qb[RG][D / 16][2];
    float f[RG][2];                              // of rows 2 t4 and 2 t4 + 1
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      uint2 raw[D / 16];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        raw[c] = make_uint2(0u, 0u);
        if (8 * r + g < nrows)
          raw[c] = *reinterpret_cast<const uint2*>(q + ((size_t)s * Hq + h0 + 8 * r + g) * D + 16 * c +
                                                   4 * t4);
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        amax = fmaxf(fmax3(amax, fabsf(__uint_as_float(raw[c].x << 16)),
                           fabsf(__uint_as_float(raw[c].x & 0xffff0000u))),
                     fmaxf(fabsf(__uint_as_float(raw[c].y << 16)),
                           fabsf(__uint_as_float(raw[c].y & 0xffff0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = min(max(7 - exponent(amax), -120), 126);    // (an infinity stays one)
      const float up = pow2i(e);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        qb[r][c][0] = pack_f16x2(__uint_as_float(raw[c].x << 16) * up,
                                 __uint_as_float(raw[c].x & 0xffff0000u) * up);
        qb[r][c][1] = pack_f16x2(__uint_as_float(raw[c].y << 16) * up,
                                 __uint_as_float(raw[c].y & 0xffff0000u) * up);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        f[r][u] = scale_log2 * __shfl_sync(0xffffffffu, pow2i(-e), 4 * (2 * t4 + u));
    }
    // O^T: chunk i of 16 dimensions: [0], [1] dimension 2 g of rows 2 t4, 2 t4 + 1, [2], [3] dimension 2 g + 1.
    float oacc[RG][D / 16][4], m[RG][2], l[RG][2];
#pragma unroll
    for (int r = 0; r < RG; ++r) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[r][i][e] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[r][u] = -INFINITY;
        l[r][u] = 0.f;
      }
    }
    int e_ref = -126;            // the largest scale so far
    int unit[RG][2];             // E of the rows' sums
    int aim = e_ref;             // what it is to be
    bool behind = false;         // is any of them below that?
#pragma unroll
    for (int r = 0; r < RG; ++r) unit[r][0] = unit[r][1] = e_ref;
    // This lane's row and chunk of a matrix load: slots 0-7 and 8-15 of a 16-byte chunk and of the next.
    const int mrow = lane & 15, mchunk = lane >> 4;
    bool ok = true;

    for (int t = 0; t < nt; ++t) {
      const int st = t % kStages;
      if (!warp_wait(&sm.full[st], (t / kStages) & 1, kWaitNs)) { ok = false; break; }
      const int valid = hi - (lo + t * kKeys);      // keys of this stage
      const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
      if (valid < kKeys) {                          // the last stage: no copy follows into it
        for (int i = lane; i < (kKeys - valid) * (D / 16); i += 32)
          *reinterpret_cast<uint4*>(sm.v[st] + valid * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      const int e0 = exponent(sm.scale[st][2]), e1 = exponent(sm.scale[st][3]);
      e_ref = max(e_ref, max(e0, e1));
      const int eb[2] = {max(e0, e_ref - kScaleRange), max(e1, e_ref - kScaleRange)};
      const int aim_old = aim;
      aim = min(e_ref, (valid > kBlock ? min(eb[0], eb[1]) : eb[0]) + kUnitRange);
      // S^T of two blocks of 16 keys: [0], [1] key g of rows 2 t4, 2 t4 + 1, [2], [3] key g + 8.
      float z[RG][2][4];
#pragma unroll
      for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[r][b][e] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; c += 2)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t x[4];
          ldm4(kb + chunk_offset<D>(b * kBlock + mrow, c + mchunk), x);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t a[4];
            halves(x[2 * k], a[0], a[2]);
            halves(x[2 * k + 1], a[1], a[3]);
#pragma unroll
            for (int r = 0; r < RG; ++r) mma16(z[r][b], a, qb[r][c + k][0], qb[r][c + k][1]);
          }
        }
      // In log2 units, with the scale of the value.
      bool grow = false;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float ks = sm.scale[st][b], add = (float)eb[b];
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[r][b][e] = fmaf(z[r][b][e], f[r][e & 1] * ks, add);
            if (b * kBlock + g + 8 * (e >> 1) >= valid) z[r][b][e] = -INFINITY;
            grow |= z[r][b][e] > m[r][e & 1] + kRescale;
          }
      }
      if (__any_sync(0xffffffffu, grow) || aim != aim_old) {
        bool low = false;
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float mx = fmaxf(fmax3(z[r][0][u], z[r][0][2 + u], z[r][1][u]), z[r][1][2 + u]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = mx > m[r][u] + kRescale ? mx : m[r][u];
            const float corr = mn == m[r][u] ? 1.f : ex2(m[r][u] - mn);
            if (mn != m[r][u]) l[r][u] = scaled(l[r][u], m[r][u] - mn);
            m[r][u] = mn;
            if (t == 0) {
              unit[r][u] = aim;
            } else if (aim != aim_old || behind) {
              // The unit goes up as far as the row's largest part of the sum lets it.
              int top = l[r][u] == 0.f ? -127 : exponent(l[r][u]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              const int all = aim - unit[r][u], up = top == -127 ? all : min(all, max(64 - top, 0));
              l[r][u] = l[r][u] * pow2i(up >> 1) * pow2i(up - (up >> 1));
              unit[r][u] += up;
              low |= up != all;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              oacc[r][i][u] *= corr;
              oacc[r][i][2 + u] *= corr;
            }
          }
        behind = __any_sync(0xffffffffu, low);
      }
      // The weights, as B operands: of row g and a block's keys 2 t4, 2 t4 + 1 and 8 + 2 t4, 9 + 2 t4.
      uint32_t wb[RG][2][2];
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float ref[2] = {(m[r][0] == -INFINITY ? 0.f : m[r][0]) - kShift,
                              (m[r][1] == -INFINITY ? 0.f : m[r][1]) - kShift};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float back[2], p[4];
          back[0] = back[1] = pow2i(aim - eb[b]);
          if (behind)
#pragma unroll
            for (int u = 0; u < 2; ++u) back[u] = pow2i(max(unit[r][u] - eb[b], -126));
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2(z[r][b][e] - ref[e & 1]);
          l[r][0] = fmaf(p[0] + p[2], back[0], l[r][0]);
          l[r][1] = fmaf(p[1] + p[3], back[1], l[r][1]);
          wb[r][b][0] = transpose8(pack_f16x2(p[0], p[1]));
          wb[r][b][1] = transpose8(pack_f16x2(p[2], p[3]));
        }
      }
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t x[4];
          ldm4_t(vb + chunk_offset<D>(b * kBlock + mrow, i + mchunk), x);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t a[4];
            halves(__byte_perm(x[2 * k], 0u, 0x3120), a[0], a[1]);
            halves(__byte_perm(x[2 * k + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
            for (int r = 0; r < RG; ++r) mma16(oacc[r][i + k], a, wb[r][b][0], wb[r][b][1]);
          }
        }
      }
      __syncwarp();                                 // every lane has read the stage
      if (issued < nt) issue(issued++);
    }
    if (ok) {
#pragma unroll
      for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float out = pow2i(min(unit[r][u], 127));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[r][u] += __shfl_xor_sync(0xffffffffu, l[r][u], o);
          const float inv = l[r][u] == 0.f ? 0.f : 1.f / l[r][u];
          const int n = 8 * r + 2 * t4 + u;
          if (n >= nrows) continue;
          float* dst = part_o + (row0 + n) * D + 2 * g;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2*>(dst + 16 * i) =
                make_float2(oacc[r][i][u] * inv * out, oacc[r][i][2 + u] * inv * out);
          if (g == 0)       // l is NaN when a score is; a row without weight has no log
            part_lse[row0 + n] =
                l[r][u] == 0.f ? -INFINITY
                               : m[r][u] - kShift - (float)unit[r][u] + log2f(l[r][u]);
        }
    } else {
      if (lane == 0) fail(PG_ERR_TIMEOUT);
      // leave no copy in flight
      for (int t = max(issued - kStages, 0); t < issued; ++t)
        mbar_wait(&sm.full[t % kStages], (t / kStages) & 1, kWaitNs);
    }
  }
  // (As in pg_attn_own.cu: this grid does not end before the prefix kernel has.)
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int RG>
pg_status launch_t(const DecodeArgs& a, bool after_prefix) {
  const pg_decode_plan* p = a.plan;
  const int hp = p->heads_q / p->heads_kv, row_tiles = (hp + kRows - 1) / kRows;
  const uint64_t slots = (uint64_t)a.num_pages * p->page_size, row = (uint64_t)p->heads_kv * D;
  int shift = 0;
  while ((1 << shift) < p->page_size) ++shift;
  CUtensorMap tk, tv;
  pg_status st = make_tmap_2d_u8(&tk, a.k_cache, row, slots, row, D, kBlock);
  if (st == PG_OK) st = make_tmap_2d_u8(&tv, a.v_cache, row, slots, row, D, kBlock);
  if (st != PG_OK) return st;
  auto kern = decode_own_e4m3_kernel<D, RG>;
  const size_t smem = sizeof(OwnSmem<D>) + 1024;
  static OncePerDevice once;
  st = once.run([&] { return allow_smem(kern, smem, "decode own e4m3 smem attributes"); });
  if (st != PG_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p->num_seqs * a.own_slots * row_tiles * p->heads_kv));
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after_prefix ? 1 : 0;
  prof_begin(PG_KERNEL_DECODE, a.stream);
  st = cuda_check(
      cudaLaunchKernelEx(&cfg, kern, tk, tv, a.k_scales, a.v_scales,
                         static_cast<const __nv_bfloat16*>(a.q), a.own_pages, (long long)a.own_stride,
                         a.own_lens, (int)a.num_pages, shift, (int)(p->own_pages * p->page_size),
                         (int)p->prefix_slots, (int)p->own_slots, a.own_slots, row_tiles,
                         (int)p->num_seqs, (int)p->heads_q, (int)p->heads_kv, a.scale_log2, a.part_o, a.part_lse),
      "decode own e4m3 launch");
  prof_end(PG_KERNEL_DECODE, a.stream);
  return st;
}

}  // namespace

pg_status launch_decode_own_e4m3(const DecodeArgs& a, bool after_prefix) {
  // (a group of eight rows without a row costs what one with rows does: four query heads per key/value head,
  // 128 responses of 0-512 keys, 37.5 us for the step with one group and 43.4 with two)
  if (a.plan->heads_q <= 8 * a.plan->heads_kv)
    return a.plan->head_dim == 64 ? launch_t<64, 1>(a, after_prefix) : launch_t<128, 1>(a, after_prefix);
  return a.plan->head_dim == 64 ? launch_t<64, 2>(a, after_prefix) : launch_t<128, 2>(a, after_prefix);
}

pg_status read_status_decode_own_e4m3(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_own8, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_own8, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg
