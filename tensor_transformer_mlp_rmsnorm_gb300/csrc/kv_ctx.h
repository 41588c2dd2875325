// The cache context, shared by its own entry points and the attention
// sublayer's calls that store into or read from a cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/tpmlp.h"
#include "kv_decode.h"
#include "qk_rope.h"

namespace tpmlp {
constexpr int KV_MAX_WORKERS = 512;  // CTAs of the decode kernel
}

struct tpkv_ctx {
  tpkv_config cfg{};
  cudaStream_t stream = nullptr;
  int device = 0, num_sms = 0, box_tokens = 64, workers = 0;
  uint32_t *status = nullptr, *counters = nullptr;
  float* part = nullptr;
  // The clears of status and counters: an event behind them until the host has
  // seen it, their stream, and the last other stream that waits for it.
  cudaEvent_t cleared = nullptr;
  bool clear_pending = false;
  cudaStream_t clear_stream = nullptr, clear_seen = nullptr;
  void *k = nullptr, *v = nullptr;
  int64_t stride_page = 0, stride_head = 0, stride_slot = 0;
  const float *k_inv_scale = nullptr, *v_inv_scale = nullptr;
  CUtensorMap kmap, vmap;
  tpmlp::RopeFreqs freqs{};
  const void *q_norm_w = nullptr, *k_norm_w = nullptr;
  float eps = 0.0f;
  uint64_t launches = 0;
  const char* err = "";  // static text
  tpmlp_status fail(tpmlp_status s, const char* m) {
    err = m;
    return s;
  }
};

namespace tpmlp {

// What is done to queries and keys on the way (nothing by default).
struct QkTransform {
  const RopeFreqs* freqs = nullptr;
  const void *q_norm_w = nullptr, *k_norm_w = nullptr;
  float eps = 0.0f;
};
const char* rotary_error(const tpattn_rotary* r, int d);
RopeFreqs freqs_of(const tpattn_rotary* r);

// Checks that every cache call makes; the caller has checked its own tensors
// before the two launches below.  past_lens null: all 0.
tpmlp_status kv_check_call(tpkv_ctx* c, int64_t batch, const int32_t* lens, const int32_t* table, int64_t ld_table,
                           int32_t max_pages);
tpmlp_status kv_check_append(tpkv_ctx* c);
tpmlp_status kv_run_append(tpkv_ctx* c, int64_t rows, int32_t batch, const void* qkv, int64_t ld_qkv,
                           const int32_t* cu_rows, const int32_t* new_lens, const int32_t* past_lens,
                           const int32_t* table, int64_t ld_table, int32_t max_pages, const QkTransform& tr,
                           void* q_out, int64_t ld_q, cudaStream_t st);
tpmlp_status kv_run_decode(tpkv_ctx* c, int32_t batch, const void* q, int64_t ld_q, const int32_t* lens,
                           int32_t len_add, const int32_t* table, int64_t ld_table, int32_t max_pages, float scale,
                           int32_t window, int32_t sinks, void* out, int64_t ld_out, float* lse, cudaStream_t st);

}  // namespace tpmlp
