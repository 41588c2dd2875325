// Device side of sequences of different lengths: their rows, what their tokens
// see, and which block of work a CTA takes.
#pragma once

#include <cuda_bf16.h>

#include "tma_maps.cuh"
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

// The sequence that a row belongs to if to any: the last one that does not
// begin behind it.  By the lanes of one warp.
__device__ __forceinline__ int find_row(const SeqRows& s, int row, int lane) {
  if (!s.cu_rows) return row / s.rows_per_seq;
  int lo = 0, hi = s.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, b < hi && s.cu_rows[b] <= row));
    lo += max(n - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Blocks are ordered by length up to this many sequences.  Looking at all of
// them costs a CTA about a microsecond at 512; with more there are many blocks,
// and the last ones count for little.
constexpr int LPT_BATCH = 512;

// The rank-th block, longest first (more steps before fewer), by the lanes of
// one warp over the sequences' (past, count) in shared memory.  The number of
// blocks of at least x steps of a sequence is a closed form, so the steps of
// the rank-th block are found by bisection.  A step is KB tokens.
template <int KB>
__device__ __forceinline__ void find_by_length(const int2* sq, int batch, int rank, int block_tok, int cap, int lane,
                                               int* b_out, int* i_out) {
  auto blocks_from = [&](int2 s, int x) -> int {  // blocks with at least x steps
    const int nblk = (s.y + block_tok - 1) / block_tok;
    if (x <= 1) return nblk;
    if (x > cap || s.x < 0) return 0;
    const int64_t y = (int64_t)(x - 1) * KB + 1;  // tokens that x steps need
    if ((int64_t)s.x + s.y < y) return 0;
    const int64_t before = (y - s.x + block_tok - 1) / block_tok - 1;
    return nblk - (int)max((int64_t)0, before);
  };
  auto count = [&](int x) -> int {
    int c = 0;
    for (int b = lane; b < batch; b += 32) c += blocks_from(sq[b], x);
    return __reduce_add_sync(0xffffffffu, c);
  };
  int most = 1;
  for (int b = lane; b < batch; b += 32) most = max(most, (int)min(((int64_t)max(sq[b].x, 0) + sq[b].y + KB - 1) / KB, (int64_t)cap));
  most = __reduce_max_sync(0xffffffffu, most);
  *b_out = -1;
  if (count(1) <= rank) return;
  int lo = 1, hi = most + 1;  // count(lo) > rank >= count(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count(mid) > rank) lo = mid;
    else hi = mid;
  }
  int left = rank - count(hi);
  for (int b0 = 0; b0 < batch; b0 += 32) {
    const int b = b0 + lane;
    int mine = 0, longer = 0, nblk = 0;
    if (b < batch) {
      longer = blocks_from(sq[b], hi);
      nblk = blocks_from(sq[b], 1);
      mine = blocks_from(sq[b], lo) - longer;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t has = __ballot_sync(0xffffffffu, upto > left);
    if (has) {
      const int src = __ffs(has) - 1;
      const int i = nblk - longer - mine + (left - (upto - mine));
      *b_out = b0 + src;
      *i_out = __shfl_sync(0xffffffffu, i, src);
      return;
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
// {64 columns, mid, rows} boxes of a tensor {d, mid count, rows} with strides in elements.
inline bool map3(CUtensorMap* m, const void* ptr, int d, int mid, int64_t rows, int64_t ld, int box_mid, int box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)mid, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_mid, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tpmlp
