// Query/key norm and rotation, and the cache append: kernel arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tpmlp_internal.h"

namespace tpmlp {

constexpr int ROPE_MAX_PAIRS = 128;    // rot <= 256
constexpr int ROPE_MAX_PARTS = 1024;   // blocks of the backward kernel

// Rotation per position of each pair, in turns as a 64-bit fraction.
struct RopeFreqs {
  int32_t rot;          // rotated values of a head (a multiple of 16; 0: none)
  int32_t interleaved;  // pairs (2j, 2j + 1) instead of (j, j + rot / 2)
  uint64_t turn[ROPE_MAX_PAIRS];
};

struct RopeArgs {
  const void* in;  // rows of nq query heads, nkv key heads (append: and nkv value heads)
  int64_t ld_in;
  void* out;       // rotated rows (append: query heads only, may be null)
  int64_t ld_out;
  void* save;      // optional copy of the rows as read
  int64_t ld_save;
  int64_t rows;
  int nq, nkv;
  const void *q_norm_w, *k_norm_w;  // [d] or null
  float eps;
  const int32_t* pos;  // [rows], or null: row % seq (seq 0: row)
  int64_t seq;
  int splits;
  // append
  int batch;
  int rows_per_seq;
  const int32_t *cu_rows, *new_lens, *past_lens, *table;
  int64_t ld_table;
  int max_pages;  // pages of a sequence that the table holds
  int page_size;
  int64_t num_pages;
  void *k_cache, *v_cache;
  int64_t stride_page, stride_head, stride_slot;
  const float *k_inv_scale, *v_inv_scale;
  uint32_t* status;
};

struct RopeBwdArgs {
  const void* x;  // the rows before the norm (unused without norm weights)
  int64_t ld_x;
  const void* dout;
  int64_t ld_dout;
  void* dx;  // may be dout
  int64_t ld_dx;
  int64_t rows;
  int nq, nkv;
  const void *q_norm_w, *k_norm_w;
  float eps;
  const int32_t* pos;
  int64_t seq;
  int splits;
  float* part;  // [ROPE_MAX_PARTS][2][d] scratch for the weight gradients, or null
};

// dtype: 0 = f32, 1 = bf16; d: 64, 128, 192 or 256.
cudaError_t launch_qk_rope(int dtype, int d, const RopeArgs& a, const RopeFreqs& fr, int num_sms, cudaStream_t st);
cudaError_t launch_qk_rope_bwd(int dtype, int d, const RopeBwdArgs& a, const RopeFreqs& fr, int num_sms,
                               cudaStream_t st, float* dq_w, float* dk_w);
cudaError_t launch_kv_append(bool e4m3, int d, const RopeArgs& a, const RopeFreqs& fr, int num_sms, cudaStream_t st);

}  // namespace tpmlp
