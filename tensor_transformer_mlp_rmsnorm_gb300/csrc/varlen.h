// Attention of sequences of different lengths: kernel arguments, shared by the
// calls over packed rows and over a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tpmlp_internal.h"

namespace tpmlp {

// Parts of blocks that are split over the length of a cache at most, and the floats of one.
constexpr int VAR_MAX_PARTS = 320;
inline size_t var_part_floats(int d) { return (size_t)(d <= 128 ? 256 : 128) * (d + 2); }

// Which rows are whose.  Sequence b has `count` rows from `first` on, the i-th
// of them at position past + i; past < 0: an inactive sequence.
struct SeqRows {
  const int32_t* cu_rows;    // [batch + 1], or null: rows_per_seq rows each
  const int32_t* new_lens;   // [batch] tokens among them, or null: all
  const int32_t* past_lens;  // [batch], or null: 0
  int batch;
  int rows_per_seq;
  int64_t rows;
};

// Blocks of a call (those of all sequences, times key heads) are numbered in 31 bits, with
// room for the turn behind them.  A tile has 128 rows of (token, head): the bound counts
// blocks of one tile; those of two are fewer.
constexpr int64_t VAR_MAX_BLOCKS = 0x7fffffff / 2;
inline bool var_fits(const SeqRows& s, int nq, int nkv) {
  const int hpg = nq / nkv, ht = hpg < 128 ? hpg : 128, tok = 128 / ht;
  const int64_t heads = (int64_t)nkv * ((hpg + ht - 1) / ht);
  const int64_t slots = s.cu_rows && s.batch > 1 ? s.rows / tok + s.batch
                        : (int64_t)((s.rows / s.batch + tok - 1) / tok) * s.batch;
  return slots <= VAR_MAX_BLOCKS / heads;
}

// Forward: q, out [rows, >= nq d] bf16, lse [rows, nq] natural log or null.
// Keys and values: rows of their own (packed), or a paged cache.
struct VarFwdArgs {
  SeqRows seq;
  const void *q, *k, *v;  // k, v: packed only
  int64_t ld_q, ld_k, ld_v;
  void* out;
  int64_t ld_out;
  float* lse;
  int nq, nkv, d;
  float scale;
  int window, sinks;  // window 0: no limit
  uint32_t* status;
  // the cache
  bool paged, e4m3;
  const int32_t* table;
  int64_t ld_table;
  int max_pages, page_size;
  int64_t num_pages;
  const void *k_cache, *v_cache;
  int64_t stride_page, stride_head, stride_slot;
  const float *k_inv_scale, *v_inv_scale;  // E4M3: [nkv] or null
  float* part;  // scratch for parts, or null: blocks are not split
  size_t part_floats;
  uint64_t* launches;  // counts the kernels behind the first, or null
};

// The kernels add to and subtract from `window` and `sinks` in 32 bits.  Where no
// sequence is longer than `longest` tokens, a window of so many is none, and sinks
// behind it are all alike.
inline void limit_window(int* window, int* sinks, int64_t longest) {
  if (*window >= longest) *window = 0;
  if (*sinks > longest) *sinks = (int)longest;
}

// Backward over packed rows.
struct VarBwdArgs {
  SeqRows seq;
  const void *q, *k, *v, *out, *dout;
  int64_t ld_q, ld_k, ld_v, ld_out, ld_dout;
  const float* lse;
  void *dq, *dk, *dv;
  int64_t ld_dq, ld_dk, ld_dv;
  float2* stats;  // scratch [rows, nq]
  int nq, nkv, d;
  float scale;
  int window, sinks;
  uint32_t* status;
  uint64_t* launches;  // as above
};

// For each row its position (pos, or null), and zeros in rows of z and dz (row
// bytes, multiples of 16; null: none) that are no sequence's.  past is not used.
cudaError_t launch_packed_rows(const SeqRows& s, int32_t* pos, void* z, int64_t z_bytes, void* dz, int64_t dz_bytes,
                               int num_sms, cudaStream_t st);
cudaError_t launch_var_fwd(const VarFwdArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_var_bwd(const VarBwdArgs& a, int num_sms, cudaStream_t st);

}  // namespace tpmlp
