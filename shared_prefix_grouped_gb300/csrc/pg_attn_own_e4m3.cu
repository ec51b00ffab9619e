// One-token attention over a response's own keys in 8 bits: the form of pg_attn_own.cu for a cache of
// e4m3 codes with a scale per 16 slots and head, whose split (one warp per response, key/value head, up to
// 16 query rows and part of the keys) and reasons it shares.
//
// A stage is 32 keys: boxes of 16 slots by TMA, and the four scales by asynchronous copies that arrive on
// the same barrier.  Every e4m3 number is an fp16 number, so the codes become fp16 in registers and the
// products use the 16-row fp16 warp MMA, exact up to its fp32 sums: the query enters as fp16, scaled by a
// power of two so that its largest element lies in [128, 256) (a bf16 number has 8 bits, fp16 11).
//   K fragments: the matrix loads move 16-bit pairs of codes, so a lane gets four consecutive dimensions
//     of a key; the product's order over the dimensions is free, and q's fragments take the same one.
//   V fragments: a transposing load gives a lane (key, dimension) pairs (2 x 2); a byte permutation and two
//     conversions make the pairs of keys of an even and an odd dimension, whose outputs are then
//     neighbours.
// With f the softmax scale times log2 e times the key scale, and 2^e a value's scale, the weight that
// meets the code is w = 2^(f s + e - m), m the running maximum of f s + e: accuracy is relative to the largest
// product of weight and scale.  w enters the product as fp16 times 2^10 (11 bits down to 2^-24 of the
// largest, to 2^-35 absolutely).  The row's sum, in fp32, is of w 2^(E - e) with 2^E the largest scale so far,
// so it stays in range whatever the scales are.  A scale below 2^-64 of the largest so far counts as
// that, so that w keeps clear of underflow (a block of zeros has the scale 2^-126).
#include <cuda_fp16.h>
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
constexpr int kScaleRange = 64;
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
// 2^i, -126 <= i <= 127; the exponent of a power of two (0: -127).
__device__ __forceinline__ float pow2i(int i) { return __int_as_float((i + 127) << 23); }
__device__ __forceinline__ int exponent(float s) { return (__float_as_int(s) >> 23 & 0xff) - 127; }

template <int D>
__global__ void __launch_bounds__(32)
decode_own_e4m3_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const float* __restrict__ k_scales, const float* __restrict__ v_scales,
                       const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ pages,
                       long long pages_stride, const int32_t* __restrict__ own_lens, int num_pages,
                       int page_shift, int own_cap, int first_slot, int parts, int row_tiles, int S,
                       int Hq, int Hkv, float scale_log2, float* __restrict__ part_o,
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
  const int chunk = ((len + parts - 1) / parts + kKeys - 1) / kKeys * kKeys;
  const int lo = part * chunk, hi = min(len, lo + chunk);
  const size_t row0 = ((size_t)(first_slot + part) * S + s) * Hq + h0;
  const int g = lane >> 2, t4 = lane & 3;       // this lane's rows g, g + 8

  if (len <= 0 || lo >= hi) {
    if (lane < nrows) part_lse[row0 + lane] = -INFINITY;
  } else {
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
    // The query rows as the A operand: of each 16 dimensions 4 t, 4 t + 1 and 4 t + 2, 4 t + 3 stand where
    // the fragment has 2 t, 2 t + 1 and 2 t + 8, 2 t + 9.
    uint32_t qa[D / 16][4];
    float f[2];
    {
      uint2 raw[2][D / 16];
      float amax[2] = {0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          raw[r][kk] = make_uint2(0u, 0u);
          if (g + 8 * r < nrows)
            raw[r][kk] = *reinterpret_cast<const uint2*>(q + ((size_t)s * Hq + h0 + g + 8 * r) * D +
                                                         kk * 16 + 4 * t4);
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = e ? raw[r][kk].y : raw[r][kk].x;
            amax[r] = fmax3(amax[r], fabsf(__uint_as_float(w << 16)),
                            fabsf(__uint_as_float(w & 0xffff0000u)));
          }
        amax[r] = fmaxf(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 1));
        amax[r] = fmaxf(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 2));
        const int e = min(max(7 - exponent(amax[r]), -120), 126);    // (an infinity stays one)
        const float up = pow2i(e);
        f[r] = scale_log2 * pow2i(-e);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = i ? raw[r][kk].y : raw[r][kk].x;
            qa[kk][2 * i + r] = pack_f16x2(__uint_as_float(w << 16) * up,
                                           __uint_as_float(w & 0xffff0000u) * up);
          }
      }
    }
    float oacc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[i][e] = 0.f;
    int e_ref = -126;            // the largest scale so far
    bool ok = true;

    for (int t = 0; t < nt; ++t) {
      const int st = t % kStages;
      if (!warp_wait(&sm.full[st], (t / kStages) & 1, kWaitNs)) { ok = false; break; }
      const int valid = hi - (lo + t * kKeys);      // keys of this stage
      const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
      if (valid < kKeys) {                          // the last stage: no copy follows into it
        for (int i = lane; i < (kKeys - valid) * (D / 16); i += 32)
          *reinterpret_cast<uint4*>(sm.v[st] + (valid + i / (D / 16)) * D + i % (D / 16) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      float kf[2][2], add[2], back[2];              // [block][row]; per block
      const int e_old = e_ref;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float ks = sm.scale[st][b];
        kf[b][0] = f[0] * ks;
        kf[b][1] = f[1] * ks;
        e_ref = max(e_ref, exponent(sm.scale[st][2 + b]));
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int e = max(exponent(sm.scale[st][2 + b]), e_ref - kScaleRange);
        add[b] = (float)e;
        back[b] = pow2i(e_ref - e);
      }
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t c[4];
        ldm4(kb + chunk_offset<D>(lane, kk), c);    // keys 0-7, 8-15, 16-23, 24-31 of 16 dimensions
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          halves(c[i], b0, b1);
          mma16(sc[i], qa[kk], b0, b1);
        }
      }
      // In log2 units, with the scale of the value.
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[i][e] = fmaf(sc[i][e], kf[i >> 1][e >> 1], add[i >> 1]);
          if (i * 8 + t4 * 2 + (e & 1) >= valid) sc[i][e] = -INFINITY;
        }
      float corr[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(fmax3(sc[0][2 * r], sc[0][2 * r + 1], sc[1][2 * r]),
                               fmax3(sc[1][2 * r + 1], sc[2][2 * r], sc[2][2 * r + 1])),
                         fmaxf(sc[3][2 * r], sc[3][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx);
        moved |= mn > m[r];
        corr[r] = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
        if (mn != -INFINITY) l[r] *= ex2(m[r] - mn + (float)(e_ref - e_old));
        m[r] = mn;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          oacc[i][0] *= corr[0];
          oacc[i][1] *= corr[0];
          oacc[i][2] *= corr[1];
          oacc[i][3] *= corr[1];
        }
      }
      float p[4][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ref = (m[r] == -INFINITY ? 0.f : m[r]) - kShift;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float sum = 0.f;
#pragma unroll
          for (int i = 2 * b; i < 2 * b + 2; ++i)
#pragma unroll
            for (int e = 2 * r; e < 2 * r + 2; ++e) {
              p[i][e] = ex2(sc[i][e] - ref);
              sum += p[i][e];
            }
          l[r] = fmaf(sum, back[b], l[r]);
        }
      }
      uint32_t pa[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          pa[b][e] = pack_f16x2(p[2 * b + (e >> 1)][2 * (e & 1)], p[2 * b + (e >> 1)][2 * (e & 1) + 1]);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t c[4], even[4], odd[4];
        ldm4_t(vb + chunk_offset<D>(lane, i), c);
#pragma unroll
        for (int e = 0; e < 4; ++e) halves(__byte_perm(c[e], 0u, 0x3120), even[e], odd[e]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          mma16(oacc[2 * i], pa[b], even[2 * b], even[2 * b + 1]);
          mma16(oacc[2 * i + 1], pa[b], odd[2 * b], odd[2 * b + 1]);
        }
      }
      __syncwarp();                                 // every lane has read the stage
      if (issued < nt) issue(issued++);
    }
    if (ok) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r], out = pow2i(min(e_ref, 127));
        if (g + 8 * r < nrows) {
          float* dst = part_o + (row0 + g + 8 * r) * D + 4 * t4;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float4*>(dst + i * 16) =
                make_float4(oacc[2 * i][2 * r] * inv * out, oacc[2 * i + 1][2 * r] * inv * out,
                            oacc[2 * i][2 * r + 1] * inv * out,
                            oacc[2 * i + 1][2 * r + 1] * inv * out);
          if (t4 == 0)       // l is NaN when a score is; a row without weight has no log
            part_lse[row0 + g + 8 * r] =
                l[r] == 0.f ? -INFINITY : m[r] - kShift - (float)e_ref + log2f(l[r]);
        }
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

template <int D>
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
  auto kern = decode_own_e4m3_kernel<D>;
  const size_t smem = sizeof(OwnSmem<D>) + 1024;
  static OncePerDevice once;
  st = once.run([&] { return allow_smem(kern, smem, "decode own e4m3 smem attributes"); });
  if (st != PG_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p->num_seqs * p->own_slots * row_tiles * p->heads_kv));
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
                         (int)p->prefix_slots, (int)p->own_slots, row_tiles, (int)p->num_seqs,
                         (int)p->heads_q, (int)p->heads_kv, a.scale_log2, a.part_o, a.part_lse),
      "decode own e4m3 launch");
  prof_end(PG_KERNEL_DECODE, a.stream);
  return st;
}

}  // namespace

pg_status launch_decode_own_e4m3(const DecodeArgs& a, bool after_prefix) {
  return a.plan->head_dim == 64 ? launch_t<64>(a, after_prefix) : launch_t<128>(a, after_prefix);
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
