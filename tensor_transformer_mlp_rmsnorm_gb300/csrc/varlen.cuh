// Device side of sequences of different lengths: their rows, what their tokens
// see, and which block of work a CTA takes.
#pragma once

#include <cuda_bf16.h>

#include "ptx_sm103.cuh"
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

// One warp a CTA, while the others work: every sequence is looked at, for the report.
__device__ __forceinline__ void report_bad(const SeqRows& s, int64_t cap, uint32_t* status, int lane) {
  bool bad = false;
  for (int64_t b = (int64_t)blockIdx.x * 32 + lane; b < s.batch; b += (int64_t)gridDim.x * 32) seq_span(s, (int)b, cap, &bad);
  if (bad) atomicOr(status, STATUS_BAD_INDEX);
}

// Block slots: every block of `tokens` rows of every sequence has one of its own,
// slot(b) + i, found from either side without looking at the other sequences.
// Sequences of the same number of rows, and a single one: per_seq slots each.
// Else slot(b) = first[b] / tokens + b: those of different sequences are
// different, because first[b+1] >= first[b] + count[b].
struct Slots {
  int tokens, per_seq;  // per_seq 0: by rows
  int64_t count;
};
inline Slots make_slots(const SeqRows& s, int tokens) {
  Slots r;
  r.tokens = tokens;
  const int64_t rows = s.batch == 1 ? s.rows : s.cu_rows ? 0 : s.rows_per_seq;
  r.per_seq = (int)((rows + tokens - 1) / tokens);
  r.count = r.per_seq > 0 ? (int64_t)r.per_seq * s.batch : s.rows / tokens + s.batch;
  return r;
}
__device__ __forceinline__ int slot_base(const Slots& t, int first, int b) {
  return t.per_seq > 0 ? b * t.per_seq : first / t.tokens + b;
}

// The sequence whose slots hold `slot`, by the lanes of one warp: a search with
// 32 probes a step.  Returns the last b whose base does not exceed the slot.
__device__ __forceinline__ int find_slot(const SeqRows& s, const Slots& t, int slot, int lane) {
  if (t.per_seq > 0) return slot / t.per_seq;
  int lo = 0, hi = s.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const bool le = b < hi && slot_base(t, min(max(s.cu_rows[b], 0), (int)s.rows), b) <= slot;
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

// Blocks are ordered by length up to this many sequences, two a lane, and by place
// from the end with more.  That is worse where a long sequence lies first: 16384 tokens
// before 64 x 100 take 1676 us, before 63 x 100 1530 (1626 by place); behind them 1600 and
// 1550.  19 sequences of 8192 tokens: 72 us by length, 81 by place.
constexpr int LPT_BATCH = 64;

// Finds the blocks of units of work, longest first (more steps of KB tokens
// before fewer), by the lanes of one warp.  The number of blocks of at least x
// steps of a sequence is a closed form, so the steps of the rank-th block are
// found by bisection.
template <int KB>
struct ByLength {
  int past[2], count[2], blocks[2];  // of the sequences lane + 32 k
  int most;                          // steps of the longest block that is not found yet
  int block_tok, cap;                // tokens of a block; steps that a window leaves at most
  uint64_t inverse;                  // 2^64 / block_tok, rounded up: exact quotients of 32-bit numbers

  __device__ __forceinline__ int div_up(int n) const {
    return block_tok == 1 ? n : (int)__umul64hi((uint64_t)(n + block_tok - 1), inverse);
  }
  // blocks of sequence k with at least x steps
  __device__ __forceinline__ int from(int k, int x) const {
    if (x <= 1) return blocks[k];
    if (x > cap || past[k] < 0) return 0;
    const int y = (x - 1) * KB + 1;  // tokens that x steps need
    if (past[k] + count[k] < y) return 0;
    return y <= past[k] ? blocks[k] : blocks[k] - div_up(y - past[k]) + 1;
  }
  __device__ __forceinline__ int total(int x) const {
    int c = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      c += from(k, x);
    return __reduce_add_sync(0xffffffffu, c);
  }
  // limit: tokens of the cache, or -1; packed: past counts as 0
  __device__ __forceinline__ void init(const SeqRows& s, int64_t limit, int block_tok_, int cap_, int lane) {
    block_tok = block_tok_;
    cap = cap_;
    inverse = ~0ull / (uint32_t)block_tok + 1;
    int m = 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      past[k] = count[k] = blocks[k] = 0;
      if (lane + 32 * k < s.batch) {
        bool bad = false;  // reported elsewhere
        const SeqSpan sp = seq_span(s, lane + 32 * k, limit, &bad);
        past[k] = sp.past;
        count[k] = sp.count;
        blocks[k] = div_up(sp.count);
        m = max(m, min((max(sp.past, 0) + sp.count + KB - 1) / KB, cap));
      }
    }
    most = __reduce_max_sync(0xffffffffu, m);
  }
  // The rank-th block: block i of sequence b, or b = -1.  Ranks are asked for in
  // ascending order, so the steps only descend.
  __device__ __forceinline__ void find(int rank, int lane, int* b, int* i) {
    *b = -1;
    *i = 0;
    if (total(1) <= rank) return;
    int lo = 1, hi = most + 1;  // total(lo) > rank >= total(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (total(mid) > rank) lo = mid;
      else hi = mid;
    }
    most = lo;
    int left = rank - total(hi);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int longer = from(k, hi), mine = from(k, lo) - longer;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t has = __ballot_sync(0xffffffffu, upto > left);
      if (has) {
        const int src = __ffs(has) - 1;
        *b = 32 * k + src;
        *i = __shfl_sync(0xffffffffu, blocks[k] - longer - mine + (left - (upto - mine)), src);
        return;
      }
      left -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
};

// The unit of work of CTA c in its k-th turn among n CTAs: every other turn in
// reverse, so that with units longest first nobody has the longer one each time.
__device__ __forceinline__ int64_t snake(int k, int c, int n) {
  return (int64_t)k * n + ((k & 1) ? n - 1 - c : c);
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Four lanes (4 i to 4 i + 3) have four pieces of 16 bytes of a row each: afterwards
// lane 4 i + j has piece j of the four rows, so that a store of the k-th fills 64
// bytes of each of 8 rows.  (One of 16 bytes in each of 32 rows takes some 250 cycles.)
__device__ __forceinline__ void turn_pieces(uint4 (&u)[4], int lane) {
  auto swap = [&](uint4& a, uint4& b, int bit) {  // a lane without the bit gives b, one with it gives a
    const bool has = lane & bit;
    uint4 g = has ? a : b;
    g.x = __shfl_xor_sync(0xffffffffu, g.x, bit);
    g.y = __shfl_xor_sync(0xffffffffu, g.y, bit);
    g.z = __shfl_xor_sync(0xffffffffu, g.z, bit);
    g.w = __shfl_xor_sync(0xffffffffu, g.w, bit);
    if (has) a = g;
    else b = g;
  };
  swap(u[0], u[1], 1);
  swap(u[2], u[3], 1);
  swap(u[0], u[2], 2);
  swap(u[1], u[3], 2);
}

// Bits 0 to n - 1 of a word.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
// {64 columns, mid, rows} boxes of a tensor {d, mid count, rows} with strides in elements.
inline bool map3(CUtensorMap* m, const void* ptr, int d, int mid, int64_t rows, int64_t ld, int box_mid, int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)mid, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_mid, (cuuint32_t)box_rows};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace tpmlp
