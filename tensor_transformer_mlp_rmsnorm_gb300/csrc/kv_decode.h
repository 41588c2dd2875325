// Attention of one new token per sequence over a paged cache: kernel arguments.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tpmlp_internal.h"

namespace tpmlp {

struct DecodeArgs {
  const void* q;  // bf16 [batch, >= nq d], row stride ld_q
  int64_t ld_q;
  void* out;  // bf16 [batch, >= nq d], row stride ld_out
  int64_t ld_out;
  float* lse;  // [batch, nq] natural log-sum-exp, or null
  const int32_t* lens;  // [batch]
  int len_add;          // tokens attended = lens[b] + len_add
  const int32_t* table;
  int64_t ld_table;
  int max_pages;  // pages of a sequence that the table holds
  int page_size;
  int64_t num_pages;
  int batch, nq, nkv;
  int hpg;     // query heads of a key head
  int chunks;  // groups of HT query heads a key head is worked on in
  float scale_log2;  // softmax scale * log2(e)
  int window, sinks;  // window 0: no limit
  const float *k_inv_scale, *v_inv_scale;  // E4M3: [nkv] or null
  int box_tokens;  // tokens a TMA box holds: 8 to 128, dividing page_size and the tile
  int workers;     // CTAs the work is divided over
  float* part;     // partial results, 2 per worker (kv_decode_part_floats)
  uint32_t* counters;  // 3 per worker, zero between launches
  uint32_t* status;
};

// Query heads worked on together: the smallest tile that holds a key head's, at most 32.
inline int kv_decode_head_tile(int hpg) { return hpg <= 8 ? 8 : hpg <= 16 ? 16 : 32; }
// Tokens of a tile.
int kv_decode_tile(int d);
// CTAs the kernel runs with.
int kv_decode_workers(int num_sms);
inline size_t kv_decode_part_floats(int d, int hpg) {
  return (size_t)kv_decode_head_tile(hpg) * (d + 2);
}
// Tensor map of a cache [num_pages, nkv, page_size, d] with element strides.
bool make_cache_map(CUtensorMap* m, const void* ptr, bool e4m3, int d, int page_size, int nkv, int64_t num_pages,
                    int64_t stride_page, int64_t stride_head, int64_t stride_slot, int box_tokens);
cudaError_t launch_kv_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int d, bool e4m3,
                             cudaStream_t st);

}  // namespace tpmlp
