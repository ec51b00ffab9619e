// One-token attention over a response's own keys (bf16 caches): the other part of the rollout's
// attention step.  No key is shared between responses, so a key meets only the Hq / Hkv query
// rows of its key/value head: a few FLOPs per byte, bound by memory and, with short
// answers, by the number of bytes that many small pieces of work keep in flight.
//
// A CTA is one warp: it takes one response, one key/value head, up to 16 of its query rows and one part
// of the keys.  A 128-row tile would be almost empty here, so the products use the 16-row warp MMA, with
// the output accumulator, the running maximum and the sum in registers; no other warp has to be
// waited for or merged with.  K and V of 16 keys at a time arrive by TMA (one box each, 128-byte
// swizzle) into a ring of kStages, issued by the warp itself as soon as a stage is free.  Eight
// such CTAs fit on an SM (d = 128: 26 KB of shared memory each, with the slack for alignment and
// the system's share; d = 64: sixteen) and keep up to 192 KB in flight, and the hardware's CTA scheduler
// balances responses of different lengths.  Without the slack nine fit, and the step as graph replays takes
// 29.4 instead of 28.6 us on one group of 16 over 16384 keys, 45.2 instead of 44.2 on eight groups of 16,
// 227.5 instead of 223.8 on four of 64.  More stages in fewer CTAs hide less of a CTA's start (own length,
// pages, first copies: three round trips): eight groups of 16 / four of 64 took 49 / 228 us with
// three stages, 51 / 238 with four, 52 / 252 with six, other kernels alike.  A CTA of four warps that
// merged their accumulators and copied with 16-byte asynchronous copies read 3.5 TB/s, this one 5.7
// (256 responses, 769 own keys each on average).
//
// 16 divides every page size, so a stage never crosses pages; the value rows behind a response's last
// key are zeroed before the product reads them (P is 0 there, 0 x NaN is not).
#include <math.h>

#include "pg_decode.h"
#include "pg_rowsoftmax.cuh"
#include "pg_sm100.cuh"
#include "pg_tmap.h"

namespace pg {

using namespace sm100;
using rowsoftmax::ex2;

namespace {

constexpr int kKeys = 16;        // keys per stage
constexpr int kStages = 3;
constexpr int kRows = 16;        // query rows per CTA
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ int s_status_own = 0;

__device__ __forceinline__ void fail(int code) { atomicCAS(&s_status_own, 0, code); }

template <int D>
struct OwnSmem {
  uint8_t k[kStages][D / 64][kKeys * 128];   // [dim half][16 rows x 128 bytes]
  uint8_t v[kStages][D / 64][kKeys * 128];
  uint64_t full[kStages];
};

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
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 with fp32 accumulation.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(32)
decode_own_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ pages,
                  long long pages_stride, const int32_t* __restrict__ own_lens, int num_pages,
                  int page_shift, int own_cap, int first_slot, int parts, int row_tiles, int S, int Hq,
                  int Hkv, float scale_log2, float* __restrict__ part_o,
                  float* __restrict__ part_lse) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  OwnSmem<D>& sm = *reinterpret_cast<OwnSmem<D>*>(base);
  const int lane = threadIdx.x;
  // Everything read here was complete before the prefix kernel began (see its launch), beside which this
  // grid may run: nothing of the prefix kernel's is read.
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
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;    // this lane's rows r0, r0 + 8 and first column

  if (len <= 0 || lo >= hi) {
    if (lane < nrows) part_lse[row0 + lane] = -INFINITY;
  } else {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[i], 1);
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
      const int key = lo + t * kKeys, pi = key >> page_shift;
      if (pi >= pbase + 32) {
        pbase += 32;
        pg = pg_next;
        pg_next = read_page(pbase + 32 + lane);
      }
      const int page = __shfl_sync(0xffffffffu, pg, pi - pbase);
      if (lane == 0) {
        const bool bad = page < 0 || page >= num_pages;
        if (bad) fail(PG_ERR_DEVICE);        // a box behind the cache reads as zeros
        const int y = bad ? num_pages << page_shift
                          : (page << page_shift) + (key & ((1 << page_shift) - 1));
        const int st = t % kStages;
        mbar_expect_tx(&sm.full[st], 2 * kKeys * D * 2);
        tma_load_3d(sm.k[st], &tk, &sm.full[st], 0, y, kh * (D / 64));
        tma_load_3d(sm.v[st], &tv, &sm.full[st], 0, y, kh * (D / 64));
      }
    };
    int issued = 0;
    for (; issued < min(kStages, nt); ++issued) issue(issued);
    // The query rows as the A operand: rows r0 and r0 + 8, columns c0 + {0, 1, 8, 9} of each 16.
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int rr = r0 + (e & 1) * 8;
        qa[kk][e] = rr < nrows ? *reinterpret_cast<const uint32_t*>(
                                     q + ((size_t)s * Hq + h0 + rr) * D + kk * 16 + c0 + (e >> 1) * 8)
                               : 0u;
      }
    float oacc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[i][e] = 0.f;
    const int mrow = lane & 7, mid = lane >> 3;     // row and matrix this lane addresses
    bool ok = true;

    for (int t = 0; t < nt; ++t) {
      const int st = t % kStages;
      if (!warp_wait(&sm.full[st], (t / kStages) & 1, kWaitNs)) { ok = false; break; }
      const int valid = hi - (lo + t * kKeys);      // keys of this stage
      const uint32_t kb = smem_u32(sm.k[st]), vb = smem_u32(sm.v[st]);
      if (valid < kKeys) {                          // the last stage: no copy follows into it
        for (int i = lane; i < (kKeys - valid) * 8 * (D / 64); i += 32)
          *reinterpret_cast<uint4*>(sm.v[st][i / ((kKeys - valid) * 8)] +
                                    (valid + i % ((kKeys - valid) * 8) / 8) * 128 + (i & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        // keys 0-7 and 8-15 by columns 0-7 and 8-15 of the step
        uint32_t b[4];
        ldm4(kb + (kk >> 2) * (kKeys * 128) +
                 sw128_offset((mid >> 1) * 8 + mrow, (kk & 3) * 2 + (mid & 1)), b);
        mma16(sc[0], qa[kk], b[0], b[1]);
        mma16(sc[1], qa[kk], b[2], b[3]);
      }
      if (valid < kKeys) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i * 8 + c0 + (e & 1) >= valid) sc[i][e] = -INFINITY;
      }
      float corr[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx * scale_log2);
        moved |= mn > m[r];
        corr[r] = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
        m[r] = mn;
        l[r] *= corr[r];
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
      float p[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1;
          const float ref = m[r] == -INFINITY ? 0.f : m[r];
          p[i][e] = ex2(fmaf(sc[i][e], scale_log2, -ref));
          l[r] += p[i][e];
        }
      // The weights are rounded to bf16 for the product; the sum keeps them in fp32 (the reasons are at
      // the prefix kernel).
      const uint32_t pa[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                              pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3])};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldm4_t(vb + (i >> 2) * (kKeys * 128) +
                   sw128_offset((mid & 1) * 8 + mrow, (i & 3) * 2 + (mid >> 1)), b);
        mma16(oacc[2 * i], pa, b[0], b[1]);
        mma16(oacc[2 * i + 1], pa, b[2], b[3]);
      }
      __syncwarp();                                 // every lane has read the stage
      if (issued < nt) issue(issued++);
    }
    if (ok) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        if (r0 + 8 * r < nrows) {
          float* dst = part_o + (row0 + r0 + 8 * r) * D + c0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(dst + i * 8) =
                make_float2(oacc[i][2 * r] * inv, oacc[i][2 * r + 1] * inv);
          if (c0 == 0)       // l is NaN when a score is; a row without weight has no log
            part_lse[row0 + r0 + 8 * r] = l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
        }
      }
    } else {
      if (lane == 0) fail(PG_ERR_TIMEOUT);
      // leave no copy in flight
      for (int t = max(issued - kStages, 0); t < issued; ++t)
        mbar_wait(&sm.full[t % kStages], (t / kStages) & 1, kWaitNs);
    }
  }
  // The merge kernel waits for this grid, which must therefore not end before the prefix kernel has: its
  // last CTA sees to that (all of them would hold their SM's shared memory while they wait).
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
pg_status launch_t(const DecodeArgs& a, bool after_prefix) {
  const pg_decode_plan* p = a.plan;
  const int hp = p->heads_q / p->heads_kv, row_tiles = (hp + kRows - 1) / kRows;
  const uint64_t slots = (uint64_t)a.num_pages * p->page_size, row = (uint64_t)p->heads_kv * D * 2;
  int shift = 0;
  while ((1 << shift) < p->page_size) ++shift;
  // [64-dim halves of all heads][slots][64 dims]: a box is both halves of 16 slots of a head.
  CUtensorMap tk, tv;
  pg_status st = make_tmap_3d_bf16(&tk, a.k_cache, 64, slots, (uint64_t)p->heads_kv * (D / 64), row, 128,
                                   64, kKeys, D / 64);
  if (st == PG_OK)
    st = make_tmap_3d_bf16(&tv, a.v_cache, 64, slots, (uint64_t)p->heads_kv * (D / 64), row, 128, 64,
                           kKeys, D / 64);
  if (st != PG_OK) return st;
  auto kern = decode_own_kernel<D>;
  const size_t smem = sizeof(OwnSmem<D>) + 1024;
  static OncePerDevice once;
  st = once.run([&] { return allow_smem(kern, smem, "decode own smem attributes"); });
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
      cudaLaunchKernelEx(&cfg, kern, tk, tv, static_cast<const __nv_bfloat16*>(a.q), a.own_pages,
                         (long long)a.own_stride, a.own_lens, (int)a.num_pages, shift,
                         (int)(p->own_pages * p->page_size), (int)p->prefix_slots,
                         (int)p->own_slots, row_tiles, (int)p->num_seqs, (int)p->heads_q,
                         (int)p->heads_kv, a.scale_log2, a.part_o, a.part_lse),
      "decode own launch");
  prof_end(PG_KERNEL_DECODE, a.stream);
  return st;
}

}  // namespace

pg_status launch_decode_own(const DecodeArgs& a, bool after_prefix) {
  return a.plan->head_dim == 64 ? launch_t<64>(a, after_prefix) : launch_t<128>(a, after_prefix);
}

pg_status read_status_decode_own(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_own, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_own, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg
