// Device side of sequences of different lengths: their rows, what their tokens
// see, and which block of work a CTA takes.
#pragma once

#include "varlen.h"

namespace tpmlp {

struct SeqSpan {
  int first, count;  // rows
  int past;          // tokens before the first row's; < 0: inactive
};

// Sequence b's rows, held inside [0, rows), and its past, held inside a cache
// of `cap` tokens (cap < 0: no limit); what lies outside is reported.
__device__ __forceinline__ SeqSpan seq_span(const SeqRows& s, int b, int64_t cap, bool* bad) {
  SeqSpan r;
  const int rows = (int)s.rows;
  if (s.cu_rows) {
    const int lo = s.cu_rows[b], hi = s.cu_rows[b + 1];
    *bad |= lo < 0 || hi < lo || hi > rows;
    r.first = min(max(lo, 0), rows);
    r.count = min(max(hi, r.first), rows) - r.first;
  } else {
    r.first = b * s.rows_per_seq;
    r.count = s.rows_per_seq;
    if (s.new_lens) r.count = min(max(s.new_lens[b], 0), r.count);
  }
  r.past = s.past_lens ? s.past_lens[b] : 0;
  if (cap >= 0 && r.past >= 0 && r.count > 0 && (int64_t)r.past + r.count > cap) {
    *bad = true;
    r.past = (int)max((int64_t)0, cap - r.count);
  }
  return r;
}

// First of the block slots of sequence b: its blocks of `tokens` rows have the
// slots base + i.  Slots of different sequences are different, because
// first[b+1] >= first[b] + count[b]; there are rows / tokens + batch of them.
__device__ __forceinline__ int slot_base(int first, int b, int tokens) { return first / tokens + b; }

// The sequence whose slots hold `slot`, by the lanes of one warp: a search with
// 32 probes a step.  Returns the last b whose base does not exceed the slot.
__device__ __forceinline__ int find_slot(const SeqRows& s, int slot, int tokens, int lane) {
  int lo = 0, hi = s.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    bool le = false;
    if (b < hi) {
      const int first = s.cu_rows ? min(max(s.cu_rows[b], 0), (int)s.rows) : b * s.rows_per_seq;
      le = slot_base(first, b, tokens) <= slot;
    }
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    lo += max(n - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace tpmlp
