// Internal declarations of the rollout's attention step: the plan's records and the launches of its
// kernels.
#pragma once
#include "pg_internal.h"

namespace pg {

// One response (record s of the plan): its group, the group's prefix length and number of parts.
struct DecodeSeq {
  int32_t group, prefix_len, prefix_parts, pad;
};

constexpr int kDecodeTile = 128;          // keys per tile of the prefix kernel
constexpr int kMaxRows = 128;             // query rows of a prefix item

// Keys [key_lo, key_hi) (key_lo a multiple of kDecodeTile, key_lo < key_hi) of group `group`'s prefix
// for the responses [s0, s0 + n_seq): the partial results of part `slot`.
struct DecodeItem {
  int32_t group, s0, n_seq, key_lo, key_hi, slot, pad0, pad1;
};

// How a response's own keys in 8 bits are shared: parts of `keys` keys (a multiple of 32), `n` of them.  By the
// present length, not by the room for it: `fill` parts, which fill the GPU, or as many as hold kOwnPart
// keys each, at most `most`.  (256 responses over prefixes of 2000 keys, own keys 300 each: parts of 128, 256 and 512
// take 61.0, 59.0 and 61.9 us; 1-1537 keys 97.9, 95.6 and 99.3; 1500 keys 152, 151 and 154.)
constexpr int kOwnPart = 256;
struct OwnParts {
  int keys, n;
};
__host__ __device__ inline OwnParts own_parts_e4m3(int len, int fill, int most) {
  if (len <= 0) return {32, 0};
  int n = (len + kOwnPart - 1) / kOwnPart;
  n = n < fill ? fill : n > most ? most : n;
  if (n == 1) return {(len + 31) / 32 * 32, 1};
  const int keys = ((len + n - 1) / n + 31) / 32 * 32;
  return {keys, (len + keys - 1) / keys};
}

static_assert(sizeof(DecodeSeq) == 16 && sizeof(DecodeItem) == 32, "plan records");

// Keys of a response in one paged cache.
struct DecodeArgs {
  const pg_decode_plan* plan;
  const void *q, *k_cache, *v_cache;
  const float *k_scales, *v_scales;      // of a cache in 8 bits
  int64_t num_pages;
  const int32_t *prefix_pages, *own_pages, *own_lens;
  int64_t prefix_stride, own_stride;
  void* o;
  float* lse;
  int own_slots;         // partial results of the own keys: at most (in 8 bits), or as many
  float scale_log2;      // softmax scale x log2 e
  float *part_o, *part_lse;   // [slot][S x Hq][d], [slot][S x Hq] (log2 units)
  cudaStream_t stream;
};

inline const DecodeSeq* decode_seqs(const pg_decode_plan* p) {
  return reinterpret_cast<const DecodeSeq*>(static_cast<const char*>(p->tables) + p->off_seqs);
}
inline const DecodeItem* decode_items(const pg_decode_plan* p) {
  return reinterpret_cast<const DecodeItem*>(static_cast<const char*>(p->tables) + p->off_items);
}

// The tensor-core kernels: partial results of the prefix parts (slots [0, prefix_slots)) and of the
// responses' own keys (slots from prefix_slots on).  The first starts after all work before it in the
// stream; with after_prefix the second may start while the first still runs, and ends after it.
pg_status launch_decode_prefix(const DecodeArgs& a);
pg_status launch_decode_own(const DecodeArgs& a, bool after_prefix);
// The same over a cache in 8 bits, where a response's slots are those of own_parts_e4m3, at most a.own_slots.
pg_status launch_decode_prefix_e4m3(const DecodeArgs& a);
pg_status launch_decode_own_e4m3(const DecodeArgs& a, bool after_prefix);

}  // namespace pg
