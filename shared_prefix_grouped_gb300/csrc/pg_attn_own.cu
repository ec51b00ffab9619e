// One-token attention over a response's own keys (bf16 caches): the other part of the rollout's
// attention step.  No key is shared between responses, so a key meets only the Hq / Hkv query
// rows of its key/value head: a few FLOPs per byte, bound by memory and, with short
// answers, by the number of bytes that many small pieces of work keep in flight.
//
// A CTA takes one response, one key/value head, up to 16 of its query rows and one part of the
// keys.  A tile of 128 rows would be almost empty here, so the products use the 16-row warp MMA: each of the
// four warps takes 16 of a tile's 64 keys with a running maximum, sum and accumulator of its own, K and
// V arrive by 16-byte asynchronous copies into a ring of three tiles (XOR-swizzled rows, so that
// the matrix loads meet no bank conflict), and the warps are merged at the end.  Two CTAs per SM keep up to
// 128 KB in flight.  Rows behind the last key are filled with zeros by the copy itself.
#include <math.h>

#include "pg_decode.h"
#include "pg_rowsoftmax.cuh"

namespace pg {

using rowsoftmax::ex2;
using sm100::pack_bf16x2;
using sm100::smem_u32;

namespace {

constexpr int kTile = 64;        // keys per tile
constexpr int kStages = 3;
constexpr int kRows = 16;        // query rows per CTA

__device__ int s_status_own = 0;

__device__ __forceinline__ void fail(int code) { atomicCAS(&s_status_own, 0, code); }

template <int D>
struct OwnSmem {
  __nv_bfloat16 k[kStages][kTile * D];
  __nv_bfloat16 v[kStages][kTile * D];
  int32_t page[kOwnPagesPerPart];
  float m[4][kRows], l[4][kRows];
};

// 16 bytes into shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 with fp32 accumulation.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(128)
decode_own_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kc,
                  const __nv_bfloat16* __restrict__ vc, const int32_t* __restrict__ pages,
                  long long pages_stride, const int32_t* __restrict__ own_lens, int num_pages,
                  int page_size, int own_cap, int first_slot, int parts, int row_tiles, int S, int Hq,
                  int Hkv, float scale_log2, float* __restrict__ part_o,
                  float* __restrict__ part_lse) {
  constexpr int CPR = D / 8;                 // 16-byte chunks per row
  constexpr int RPI = 128 / CPR;             // rows per round of copies
  extern __shared__ uint8_t smem_raw[];
  OwnSmem<D>& sm = *reinterpret_cast<OwnSmem<D>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int x = blockIdx.x;
  const int kh = x % Hkv;
  x /= Hkv;
  const int rt = x % row_tiles;
  x /= row_tiles;
  const int part = x % parts, s = x / parts;
  const int hp = Hq / Hkv, h0 = kh * hp + rt * kRows, nrows = min(kRows, hp - rt * kRows);
  int len = own_lens[s];
  if (len > own_cap) {
    if (threadIdx.x == 0) fail(PG_ERR_DEVICE);
    len = own_cap;
  }
  const int chunk = ((len + parts - 1) / parts + kTile - 1) / kTile * kTile;
  const int lo = part * chunk, hi = min(len, lo + chunk);
  const size_t row0 = ((size_t)(first_slot + part) * S + s) * Hq + h0;

  if (len <= 0 || lo >= hi) {
    if (threadIdx.x < nrows) part_lse[row0 + threadIdx.x] = -INFINITY;
  } else {
    const int p0 = lo / page_size, np = (hi - 1) / page_size - p0 + 1;    // at most kOwnPagesPerPart
    for (int i = threadIdx.x; i < np; i += 128) {
      const int pg = pages[s * pages_stride + p0 + i];
      const bool bad = pg < 0 || pg >= num_pages;
      if (bad) fail(PG_ERR_DEVICE);
      sm.page[i] = bad ? -1 : pg;
    }
    __syncthreads();
    const int nt = (hi - lo + kTile - 1) / kTile;
    const int cr = threadIdx.x / CPR, cc = threadIdx.x % CPR;
    auto issue = [&](int t) {
      if (t < nt) {
        const uint32_t kb = smem_u32(sm.k[t % kStages]), vb = smem_u32(sm.v[t % kStages]);
#pragma unroll
        for (int i = 0; i < kTile / RPI; ++i) {
          const int r = cr + i * RPI, key = lo + t * kTile + r;
          const int pg = key < hi ? sm.page[key / page_size - p0] : -1;
          const size_t off =
              pg >= 0 ? (((size_t)pg * page_size + key % page_size) * Hkv + kh) * D + cc * 8 : 0;
          copy16(kb + at<D>(r, cc), kc + off, pg >= 0);
          copy16(vb + at<D>(r, cc), vc + off, pg >= 0);
        }
      }
      copy_commit();       // an empty group past the end keeps the count
    };
    for (int t = 0; t < kStages - 1; ++t) issue(t);
    // The query rows as the A operand: lane holds rows lane / 4 and + 8, columns 2 (lane % 4) + {0, 1, 8, 9}.
    uint32_t qa[D / 16][4];
    {
      const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = r + (e & 1) * 8;
          qa[kk][e] = rr < nrows ? *reinterpret_cast<const uint32_t*>(
                                       q + ((size_t)s * Hq + h0 + rr) * D + kk * 16 + c + (e >> 1) * 8)
                                 : 0u;
        }
    }
    float oacc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[i][e] = 0.f;
    const int mrow = lane & 7, mid = lane >> 3;     // row and matrix this lane addresses

    for (int t = 0; t < nt; ++t) {
      copy_wait<kStages - 2>();
      __syncthreads();
      issue(t + kStages - 1);
      const int k0 = lo + t * kTile + warp * 16;    // this warp's 16 keys
      if (k0 >= hi) continue;
      const uint32_t kb = smem_u32(sm.k[t % kStages]), vb = smem_u32(sm.v[t % kStages]);
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        // keys 0-7 and 8-15 by columns 0-7 and 8-15 of the step
        uint32_t b[4];
        ldm4(kb + at<D>(warp * 16 + (mid >> 1) * 8 + mrow, kk * 2 + (mid & 1)), b);
        mma16(sc[0], qa[kk], b[0], b[1]);
        mma16(sc[1], qa[kk], b[2], b[3]);
      }
      if (k0 + 16 > hi) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k0 + i * 8 + (lane & 3) * 2 + (e & 1) >= hi) sc[i][e] = -INFINITY;
      }
      float mx[2], corr[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float mn = fmaxf(m[r], mx[r] * scale_log2);
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
      // The weights are rounded to bf16 for the product; the sum keeps them in fp32.
      const uint32_t pa[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                              pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3])};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldm4_t(vb + at<D>(warp * 16 + (mid & 1) * 8 + mrow, i * 2 + (mid >> 1)), b);
        mma16(oacc[2 * i], pa, b[0], b[1]);
        mma16(oacc[2 * i + 1], pa, b[2], b[3]);
      }
    }
    copy_wait<0>();
    // Merge the warps through the (now free) ring: O as fp32 [warp][16][D].
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        sm.m[warp][(lane >> 2) + 8 * r] = m[r];
        sm.l[warp][(lane >> 2) + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float* ob = reinterpret_cast<float*>(smem_raw);
    static_assert(4 * kRows * D * 4 <= sizeof(sm.k) + sizeof(sm.v), "merge buffer");
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float2*>(ob + ((warp * kRows + (lane >> 2) + 8 * r) * D + i * 8 +
                                         (lane & 3) * 2)) =
            make_float2(oacc[i][2 * r], oacc[i][2 * r + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < nrows * (D / 4); i += 128) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, sm.m[w][r]);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(sm.m[w][r] - ref);
        L = fmaf(f, sm.l[w][r], L);
        const float4 v = *reinterpret_cast<const float4*>(ob + (w * kRows + r) * D + c);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<float4*>(part_o + (row0 + r) * D + c) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (c == 0) part_lse[row0 + r] = L == 0.f ? -INFINITY : M + log2f(L);
    }
  }
  // The merge kernel waits for this grid: this grid must not end before the prefix kernel has.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
pg_status launch_t(const DecodeArgs& a, bool after_prefix) {
  const pg_decode_plan* p = a.plan;
  const int hp = p->heads_q / p->heads_kv, row_tiles = (hp + kRows - 1) / kRows;
  auto kern = decode_own_kernel<D>;
  const size_t smem = sizeof(OwnSmem<D>);
  pg_status st = cuda_check(
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem),
      "decode own smem attribute");
  if (st != PG_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)p->num_seqs * p->own_slots * row_tiles * p->heads_kv));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after_prefix ? 1 : 0;
  prof_begin(PG_KERNEL_DECODE, a.stream);
  st = cuda_check(
      cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16*>(a.q),
                         static_cast<const __nv_bfloat16*>(a.k_cache),
                         static_cast<const __nv_bfloat16*>(a.v_cache), a.own_pages,
                         (long long)a.own_stride, a.own_lens, (int)a.num_pages, (int)p->page_size,
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
