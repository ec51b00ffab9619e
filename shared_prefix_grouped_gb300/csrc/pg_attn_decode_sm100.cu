// One-token attention over the shared prefix on the 5th-generation tensor cores (bf16 caches): the
// prefix part of the rollout's attention step.
//
//   for the query rows (response s, head h) of a group and key/value head:
//   S = Q K^T;  P = exp2(scale S - m);  O = P V;  partial o = O / sum P,  lse = m + log2 sum P
//
// The rows of up to 128 / (Hq / Hkv) responses and the Hq / Hkv heads that share a key/value head fill
// one M = 128 tile, so a prefix key and value are read once for all of them: 4 x 128 rows FLOPs per
// byte at most, below the ridge of the tensor cores, hence bound by memory.  Work is split over the
// keys (parts of a prefix, chosen by the plan for whole waves of one CTA per SM); the parts' partial
// results meet in the merge kernel.
//
// A CTA keeps 2 + 2 stages of 128-key K and V tiles (128 KB) in flight, which leaves an SM room for two
// of the one-warp CTAs that do the responses' own keys: they start as soon as every prefix CTA has
// (programmatic launch) and use the bandwidth that the prefix CTAs' first loads and merges leave.  The
// tiles alternate between two independent streams, each with its own scores, running maximum, sum
// and output accumulator in TMEM (S_i in columns [128 i, 128 i + 128), P_i written over its first 64,
// O_i in [256 + 128 i, ...)), so that one stream's softmax runs under the other's products; the streams
// are merged at the end.  Roles as in the scoring forward: warp 0 the TMA producer, warp 1 issues
// every MMA, warps 2..9 the softmax of streams 0 and 1, one thread per row.  Every wait is bounded.
//
// The weights P enter the product with V as bf16, the type of V and of the matrix instruction, and their
// sum is of the fp32 ones, as in the training kernels.  A weight is off by half a step (2^-8 of it) at
// most, each by its own amount, and o by 0.0023 of its norm from fp64 attention, of which the rounding
// of o itself is 0.0017.  The remainders as a second bf16 operand would need a third product per tile:
// two take 0.67 us of the 1.02 us per tile below at the tensor cores' rate, three 1.01, no longer hidden
// by the loads.  PG_FLAG_SIMT has fp32 weights.
//
// Measured: 128 CTAs of 128 tiles (four groups of 64 responses over 32768 keys, two row blocks per
// group) 130 us, 64 GB/s of keys and values into each SM; one group of 16 responses over 16384 keys,
// seven tiles per CTA, 13 us, of which about 4 are the start and the merge.
//
// Pages.  A cache is a matrix of num_pages * page_size rows (slots) for TMA; a 128-key tile is loaded
// as 128 / min(page_size, 128) boxes, one lane of the producer warp per box, each with its page number
// read one tile ahead.  In a prefix's last tile the pages behind the end are not loaded, and
// the value rows behind it are zeroed before the product reads them: P is 0 there, but 0 x NaN is not.
#include <math.h>

#include <algorithm>

#include "pg_decode.h"
#include "pg_rowsoftmax.cuh"
#include "pg_sm100.cuh"
#include "pg_tmap.h"

namespace pg {

using namespace sm100;
using namespace rowsoftmax;

namespace {

constexpr int BM = 128;                 // query rows
constexpr int BN = kDecodeTile;         // keys per tile
constexpr int NS = 2;                   // stages of each ring
constexpr uint32_t HALF = BN * 128;     // [128 rows][64 dims] bf16
constexpr int NTHREADS = 320;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ int s_status_decode = 0;

__device__ __forceinline__ void fail(int code) { atomicCAS(&s_status_decode, 0, code); }

template <int D>
struct PrefixSmem {
  uint8_t q[D / 64][HALF];
  uint8_t k[NS][D / 64][HALF];
  uint8_t v[NS][D / 64][HALF];
  uint64_t q_full;
  uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t mma_done;
  uint32_t tmem;
};
static_assert(sizeof(PrefixSmem<128>) + 1024 <= 232448, "prefix attention shared memory");

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
decode_prefix_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const DecodeItem* __restrict__ items,
                     const int32_t* __restrict__ pages, long long pages_stride, int num_pages,
                     int page_size, float* __restrict__ part_o, float* __restrict__ part_lse, int S,
                     int Hq, int Hkv, int q_box_rows, float scale_log2) {
  constexpr int NH = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  PrefixSmem<D>& sm = *reinterpret_cast<PrefixSmem<D>*>(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const DecodeItem it = items[blockIdx.x / Hkv];     // the plan's: written long before
  const int kh = blockIdx.x % Hkv, hp = Hq / Hkv;
  const int rows = it.n_seq * hp;
  const int n = (it.key_hi - it.key_lo + BN - 1) / BN;      // key tiles, at least one

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
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

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer -----
    const int R = min(page_size, BN), pieces = BN / R;
    const int32_t* row = pages + (long long)it.group * pages_stride;
    const int oob = num_pages * page_size;     // a box of zeros
    // This lane's box of tile j: the cache row it starts at, or -1 if it lies behind the end.
    auto box = [&](int j) -> int {
      const int key = it.key_lo + j * BN + lane * R;
      if (j >= n || lane >= pieces || key >= it.key_hi) return -1;
      const int page = row[key / page_size];
      if (page < 0 || page >= num_pages) {
        fail(PG_ERR_DEVICE);
        return oob;
      }
      return page * page_size + key % page_size;
    };
    auto tile_bytes = [&](int j) -> uint32_t {
      const int left = it.key_hi - (it.key_lo + j * BN);
      return (uint32_t)(min((left + R - 1) / R, pieces) * R) * 128u * NH;
    };
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
      mbar_expect_tx(&sm.q_full, (uint32_t)q_box_rows * 128u * NH);
#pragma unroll
      for (int hf = 0; hf < NH; ++hf)
        tma_load_3d(sm.q[hf], &tq, &sm.q_full, 64 * hf, kh * hp, it.s0);
    }
    auto load = [&](const CUtensorMap* map, uint8_t (*ring)[NH][HALF], uint64_t* full,
                    uint64_t* empty, int j, int y) -> bool {
      const int s = j % NS;
      if (!warp_wait(&empty[s], ((j / NS) & 1) ^ 1, kWaitNs)) return false;
      if (lane == 0) mbar_expect_tx(&full[s], tile_bytes(j));
      __syncwarp();
      if (y >= 0)
#pragma unroll
        for (int hf = 0; hf < NH; ++hf)
          tma_load_2d(ring[s][hf] + lane * R * 128, map, &full[s], kh * D + 64 * hf, y);
      __syncwarp();
      return true;
    };
    int y0 = box(0), y1 = box(1), k_issued = 0, v_issued = 0;
    bool ok = load(&tk, sm.k, sm.k_full, sm.k_empty, 0, y0);
    if (ok) ++k_issued;
    for (int j = 0; ok && j < n; ++j) {
      const int y2 = box(j + 2);
      if (j + 1 < n) {
        ok = load(&tk, sm.k, sm.k_full, sm.k_empty, j + 1, y1);
        if (!ok) break;
        ++k_issued;
      }
      ok = load(&tv, sm.v, sm.v_full, sm.v_empty, j, y0);
      if (!ok) break;
      ++v_issued;
      y0 = y1;
      y1 = y2;
    }
    if (!ok && lane == 0) fail(PG_ERR_TIMEOUT);
    // Leave no copy in flight: the last stages' loads must have landed before exit.
    mbar_wait(&sm.q_full, 0, kWaitNs);
    for (int j = max(k_issued - NS, 0); j < k_issued; ++j)
      mbar_wait(&sm.k_full[j % NS], (j / NS) & 1, kWaitNs);
    for (int j = max(v_issued - NS, 0); j < v_issued; ++j)
      mbar_wait(&sm.v_full[j % NS], (j / NS) & 1, kWaitNs);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer -------
    // S(0), S(1), then for each tile j its P V product and the scores of tile j + 2, which overwrite
    // the columns P(j) was read from: the tensor core executes them in issue order.
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(BM, D, 0, 1);
      const uint64_t qd = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(sm.k[0][0]), 16, 1024);
      const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0][0]), HALF, 1024);
      auto issue_s = [&](int j) -> bool {
        if (!mbar_wait(&sm.k_full[j % NS], (j / NS) & 1, kWaitNs)) return false;
        tc_fence_after();
        const uint64_t kd = desc_add(kd0, (j % NS) * NH * HALF);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + 128 * (j & 1), desc_add(qd, (kk >> 2) * HALF + (kk & 3) * 32),
                 desc_add(kd, (kk >> 2) * HALF + (kk & 3) * 32), idesc_s, kk != 0);
        mma_commit(&sm.s_full[j & 1]);
        mma_commit(&sm.k_empty[j % NS]);
        return true;
      };
      bool ok = mbar_wait(&sm.q_full, 0, kWaitNs) && issue_s(0) && (n < 2 || issue_s(1));
      for (int j = 0; ok && j < n; ++j) {
        const int i = j & 1;
        ok = mbar_wait(&sm.v_full[j % NS], (j / NS) & 1, kWaitNs) &&
             mbar_wait(&sm.p_full[i], (j >> 1) & 1, kWaitNs);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = desc_add(vd0, (j % NS) * NH * HALF);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + kk * 8, desc_add(vd, kk * 2048), idesc_pv,
                 kk == 0 ? (uint32_t)(j >= 2) : 1u);
        mma_commit(&sm.pv_done[i]);
        mma_commit(&sm.v_empty[j % NS]);
        if (j + 2 < n) ok = issue_s(j + 2);
      }
      if (!ok) fail(PG_ERR_TIMEOUT);
      mma_commit(&sm.mma_done);
      mbar_wait(&sm.mma_done, 0, kWaitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax ----------
    const int i = (warp - 2) >> 2;                   // stream
    const int quarter = warp & 3;
    const int m = quarter * 32 + lane;               // query row
    const bool valid = m < rows;
    const bool any_valid = __any_sync(0xffffffffu, valid);
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + 128 * i + lane_addr, t_o = tmem + 256 + 128 * i + lane_addr;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    int c = 0;
    for (int j = i; j < n; j += 2, ++c) {
      if (!warp_wait(&sm.s_full[i], c & 1, kWaitNs)) { ok = false; break; }
      const int len = min(it.key_hi - (it.key_lo + j * BN), BN);
      const bool full_tile = len == BN;
      if (!full_tile) {
        // The prefix ends in this tile: zero the value rows behind its end.
        const int s = j % NS;
        if (!warp_wait(&sm.v_full[s], (j / NS) & 1, kWaitNs)) { ok = false; break; }
        const int t = ((warp - 2) & 3) * 32 + lane;
        for (int idx = t; idx < (BN - len) * 8 * NH; idx += 128) {
          const int hf = idx / ((BN - len) * 8), rem = idx % ((BN - len) * 8);
          *reinterpret_cast<uint4*>(sm.v[s][hf] + (len + rem / 8) * 128 + (rem % 8) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      if (!any_valid) {
        // Rows of no response: keep the barrier protocol; their outputs are never stored.
        warp_arrive(&sm.p_full[i]);
        continue;
      }
      tc_fence_after();
      // Row handling as in the scoring forward: an exact pass on the first tile and whenever a row's
      // maximum grows past the rescale threshold, else one pass against the running reference.
      uint32_t sr[64];
      bool stored = false;
      if (c > 0) {
        uint32_t pa[32], pb[32];
        float mxk = -INFINITY;
        const float mref0 = (m_used == -INFINITY) ? 0.f : m_used;
        load64(t_s, sr);
        const float sa = full_tile ? exp64_keep<false>(sr, 0, 0, len, scale_log2, mref0, pa, mxk)
                                   : exp64_keep<true>(sr, 0, 0, len, scale_log2, mref0, pa, mxk);
        load64(t_s + 64, sr);
        const float sb = full_tile ? exp64_keep<false>(sr, 64, 0, len, scale_log2, mref0, pb, mxk)
                                   : exp64_keep<true>(sr, 64, 0, len, scale_log2, mref0, pb, mxk);
        const bool grow = fmaxf(m_used, mxk * scale_log2) > m_used + kRescaleThreshold;
        if (!__any_sync(0xffffffffu, grow)) {
          tmem_st16(t_s, pa);
          tmem_st16(t_s + 16, pa + 16);
          tmem_st16(t_s + 32, pb);
          tmem_st16(t_s + 48, pb + 16);
          l += sa;
          l += sb;
          stored = true;
        }
      }
      if (!stored) {
        load64(t_s + 64, sr);
        float mx = full_tile ? max64<false>(sr, 64, 0, len) : max64<true>(sr, 64, 0, len);
        load64(t_s, sr);
        mx = fmaxf(mx, full_tile ? max64<false>(sr, 0, 0, len) : max64<true>(sr, 0, 0, len));
        const float m_new = fmaxf(m_used, mx * scale_log2);
        const bool rescale = m_new > m_used + kRescaleThreshold;
        float corr = 1.f;
        if (rescale) {
          corr = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_new);
          m_used = m_new;
          l *= corr;
        }
        const float mref = (m_used == -INFINITY) ? 0.f : m_used;
        // Rescaling O needs this stream's previous P V product done.
        if (__any_sync(0xffffffffu, rescale) && c > 0) {
          if (!warp_wait(&sm.pv_done[i], (c - 1) & 1, kWaitNs)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t orr[32];
            tmem_ld32(t_o + q4 * 32, orr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * corr);
            tmem_st32(t_o + q4 * 32, orr);
          }
        }
        l += full_tile ? exp64<false>(sr, 0, 0, len, scale_log2, mref, t_s)
                       : exp64<true>(sr, 0, 0, len, scale_log2, mref, t_s);
        load64(t_s + 64, sr);
        l += full_tile ? exp64<false>(sr, 64, 0, len, scale_log2, mref, t_s + 32)
                       : exp64<true>(sr, 64, 0, len, scale_log2, mref, t_s + 32);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm.p_full[i]);
    }
    // Merge the streams.  Once both have done their last product every MMA is complete, and the
    // query buffer carries the maxima and sums from one stream's threads to the other's.
    // (This stream's own last product first: products complete in order, so the other stream then has
    // at most one phase to go, which its parity tells from the one before.)
    const int n1 = n / 2, mine = (n + 1 - i) / 2, other = n - mine;
    if (mine > 0) ok = ok && warp_wait(&sm.pv_done[i], (mine - 1) & 1, kWaitNs);
    if (other > 0) ok = ok && warp_wait(&sm.pv_done[i ^ 1], (other - 1) & 1, kWaitNs);
    tc_fence_after();
    float2* ml = reinterpret_cast<float2*>(sm.q[0]);      // [2][128] (maximum, sum)
    ml[i * BM + m] = make_float2(m_used, l);
    ok = named_bar_and(1, 256, ok);
    if (ok && any_valid) {
      const float2 a = ml[m], b = ml[BM + m];
      const float M = fmaxf(a.x, b.x), ref = M == -INFINITY ? 0.f : M;
      const float fa = ex2(a.x - ref), fb = n1 > 0 ? ex2(b.x - ref) : 0.f;
      const float L = a.y * fa + (n1 > 0 ? b.y * fb : 0.f);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const float wa = fa * inv, wb = fb * inv;
      const int s = it.s0 + (valid ? m / hp : 0), h = kh * hp + m % hp;
      const size_t row = ((size_t)it.slot * S + s) * Hq + h;
      const bool al32 = (reinterpret_cast<uintptr_t>(part_o) & 31) == 0;
      // Stream i's warps write half of the columns.
#pragma unroll 1
      for (int q4 = i * (D / 64); q4 < (i + 1) * (D / 64); ++q4) {
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
            w[u] = __float_as_uint(x);
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
      if (valid && i == 0) part_lse[row] = L == 0.f ? -INFINITY : M + log2f(L);
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
  const int Hq = p->heads_q, Hkv = p->heads_kv, S = p->num_seqs, hp = Hq / Hkv;
  const uint32_t tb = (uint32_t)std::min<int64_t>(BM / hp, S);
  const uint64_t slots = (uint64_t)a.num_pages * p->page_size, row = (uint64_t)Hkv * D * 2;
  const uint32_t R = (uint32_t)std::min<int32_t>(p->page_size, BN);
  CUtensorMap tq, tk, tv;
  pg_status st = make_tmap_3d_bf16(&tq, a.q, D, (uint64_t)Hq, (uint64_t)S, D * 2,
                                   (uint64_t)Hq * D * 2, 64, (uint32_t)hp, tb);
  if (st == PG_OK) st = make_tmap_2d_bf16(&tk, a.k_cache, (uint64_t)Hkv * D, slots, row, 64, R);
  if (st == PG_OK) st = make_tmap_2d_bf16(&tv, a.v_cache, (uint64_t)Hkv * D, slots, row, 64, R);
  if (st != PG_OK) return st;
  auto kern = decode_prefix_kernel<D>;
  const size_t smem = sizeof(PrefixSmem<D>) + 1024;
  static OncePerDevice once;
  st = once.run([&] { return allow_smem(kern, smem, "decode prefix smem attributes"); });
  if (st != PG_OK) return st;
  prof_begin(PG_KERNEL_DECODE, a.stream);
  // In plain stream order: what the work before the step writes (the appended keys, q, page tables, own
  // lengths) is complete before this grid begins, hence also before the own-key grid, whose programmatic
  // launch relaxes its order to this grid alone.  (Were this launch programmatic too, with a
  // griddepcontrol.wait in the kernel, that wait would order the earlier work for this grid only; the
  // own-key grid starts on launch_dependents, which makes nothing visible to it.)
  const dim3 grid((unsigned)(p->n_items * Hkv));
  kern<<<grid, NTHREADS, smem, a.stream>>>(
      tq, tk, tv, decode_items(p), a.prefix_pages, (long long)a.prefix_stride, (int)a.num_pages,
      (int)p->page_size, a.part_o, a.part_lse, S, Hq, Hkv, (int)tb * hp, a.scale_log2);
  st = cuda_check(cudaGetLastError(), "decode prefix launch");
  prof_end(PG_KERNEL_DECODE, a.stream);
  return st;
}

}  // namespace

pg_status launch_decode_prefix(const DecodeArgs& a) {
  return a.plan->head_dim == 64 ? launch_t<64>(a) : launch_t<128>(a);
}

pg_status read_status_decode_sm100(bool clear, int32_t* code) {
  int32_t v = 0;
  pg_status st = cuda_check(cudaMemcpyFromSymbol(&v, s_status_decode, sizeof(v)), "read status");
  if (st != PG_OK) return st;
  if (clear && v != 0) {
    int32_t z = 0;
    st = cuda_check(cudaMemcpyToSymbol(s_status_decode, &z, sizeof(z)), "clear status");
    if (st != PG_OK) return st;
  }
  if (*code == 0) *code = v;
  return PG_OK;
}

}  // namespace pg
