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

static_assert(sizeof(DecodeSeq) == 16 && sizeof(DecodeItem) == 32, "plan records");

// Keys of a response in one paged cache.
struct DecodeArgs {
  const pg_decode_plan* plan;
  const void *q, *k_cache, *v_cache;
  int64_t num_pages;
  const int32_t *prefix_pages, *own_pages, *own_lens;
  int64_t prefix_stride, own_stride;
  void* o;
  float* lse;
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

}  // namespace pg
