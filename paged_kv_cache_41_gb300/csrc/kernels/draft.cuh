// draft.cuh -- what the draft-tree attention kernels share: a sequence's
// drafted rows, their masks and the checks of the device data that describes
// them.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

// Rows of one sequence at most: positions rounded up to a tile stay in 32 bits.
constexpr long long kDraftMaxLen = 0x7fffff00ll;

// The drafted rows of sequence r: query rows [row0, row0 + n) of q, at cache
// positions [ctx, ctx + n).  n = 0 (the sequence is skipped) for a range that
// is empty, or that the checks refuse; those set PKV_DEVERR_LENGTH.
struct DraftSeq {
  int row0, n, ctx;
};

__device__ __forceinline__ DraftSeq draft_seq(const DraftArgs& a, int r, bool report) {
  DraftSeq s;
  s.row0 = __ldg(a.draft_ptr + r);
  const int end = __ldg(a.draft_ptr + r + 1);
  s.ctx = __ldg(a.ctx_lens + r);
  // in 64 bits: the differences and sums of bad data may pass 32
  const long long n = (long long)end - s.row0;
  const bool ok = s.row0 >= 0 && n >= 0 && end <= a.num_rows && n <= a.max_draft && s.ctx >= 0 &&
                  s.ctx + n <= (long long)a.max_blocks * a.block_size && s.ctx + n <= kDraftMaxLen;
  if (!ok && report) atomicOr(a.err, PKV_DEVERR_LENGTH);
  s.n = ok ? (int)n : 0;
  return s;
}

// The drafted rows that drafted row i (of n) attends, one bit each.
__device__ __forceinline__ uint64_t draft_mask(const DraftArgs& a, const DraftSeq& s, int i) {
  const uint64_t all = s.n >= 64 ? ~0ull : (1ull << s.n) - 1;
  const uint64_t m = a.masks ? __ldg(reinterpret_cast<const unsigned long long*>(a.masks) + s.row0 + i)
                             : (i >= 63 ? ~0ull : (2ull << i) - 1);
  return m & all;
}

// The work list of plan.cuh: a sequence's rows, and its segments.
__device__ __forceinline__ int plan_len(const DraftArgs& a, int r, int, bool report) {
  const DraftSeq s = draft_seq(a, r, report);
  return s.n > 0 ? s.ctx + s.n : 0;
}
__device__ __forceinline__ int plan_heads(const DraftArgs& a) {
  return a.num_kv_heads * a.row_tiles;
}

}  // namespace pkv
