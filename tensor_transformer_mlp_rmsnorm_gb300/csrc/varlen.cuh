// Device side of SeqRows: a sequence's rows and what its tokens see.
#pragma once

#include "varlen.h"

namespace tpmlp {

struct SeqSpan {
  int first, count;  // rows
  int past;          // tokens before the first row's; < 0: inactive
};

// Sequence b's rows, held inside [0, rows); what lies outside is reported.
__device__ __forceinline__ SeqSpan seq_span(const SeqRows& s, int b, bool* bad) {
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
  return r;
}

// Whether the token at position p sees the one at position t.
__device__ __forceinline__ bool sees(int p, int t, int window, int sinks) {
  return t <= p && (window == 0 || p - t < window || t < sinks);
}

}  // namespace tpmlp
