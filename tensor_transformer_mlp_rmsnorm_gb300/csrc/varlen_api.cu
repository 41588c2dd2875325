// C ABI of causal attention over packed sequences (tpattn_packed_*): argument
// checks, the workspace and the launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/tpmlp.h"
#include "varlen.h"

using namespace tpmlp;

namespace {

tpmlp_status bad(tpmlp_status s, const char* m) {
  set_thread_error(m);
  return s;
}
bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define PK_TRY(expr)                \
  do {                              \
    const tpmlp_status s_ = (expr); \
    if (s_ != TPMLP_OK) return s_;  \
  } while (0)

SeqRows rows_of(const tpattn_packed_desc* p) {
  SeqRows s{};
  s.cu_rows = p->cu_rows;
  s.batch = p->batch;
  s.rows = p->rows;
  return s;
}

tpmlp_status check_desc(const tpattn_packed_desc* p) {
  if (!p) return bad(TPMLP_ERR_ARG, "descriptor is NULL");
  if (p->reserved != 0) return bad(TPMLP_ERR_ARG, "reserved must be 0");
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 192 && p->head_dim != 256)
    return bad(TPMLP_ERR_SHAPE, "head_dim must be 64, 128, 192 or 256");
  if (p->n_heads < 1 || p->n_kv_heads < 1 || p->n_heads > 65536 || p->n_heads % p->n_kv_heads != 0)
    return bad(TPMLP_ERR_SHAPE, "n_heads must be a positive multiple of n_kv_heads, at most 65536");
  if (p->rows < 0 || p->rows > (1 << 28)) return bad(TPMLP_ERR_SHAPE, "rows out of range (at most 2^28)");
  if (p->batch < 0 || p->batch > (1 << 20)) return bad(TPMLP_ERR_SHAPE, "batch out of range (at most 2^20)");
  if (p->batch > 0 && !p->cu_rows) return bad(TPMLP_ERR_ARG, "cu_rows is NULL");
  if (reinterpret_cast<uintptr_t>(p->cu_rows) & 3u) return bad(TPMLP_ERR_ARG, "index tensor not 4-byte aligned");
  if (!std::isfinite(p->scale)) return bad(TPMLP_ERR_ARG, "scale must be finite");
  if (p->window < 0 || p->sinks < 0) return bad(TPMLP_ERR_ARG, "window and sinks must be >= 0");
  if (p->rows > 0 && p->batch > 0 && !var_fits(rows_of(p), p->n_heads, p->n_kv_heads))
    return bad(TPMLP_ERR_SHAPE, "too many blocks: sequences and rows times key heads");
  return TPMLP_OK;
}

tpmlp_status check_rows(const void* p, int64_t ld, int64_t width) {
  if (ld % 8 != 0 || ld < width || ld > ((int64_t)1 << 36))
    return bad(TPMLP_ERR_SHAPE, "row strides must be multiples of 8 and hold a row");
  if (!p) return bad(TPMLP_ERR_ARG, "NULL tensor");
  if (!a16(p)) return bad(TPMLP_ERR_ARG, "tensor not 16-byte aligned");
  return TPMLP_OK;
}

// Multiprocessors of the current device if it is an sm_103.
tpmlp_status current_sms(int* sms) {
  static int cached[64] = {};  // written with one value only
  int dev = 0, major = 0, minor = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return bad(TPMLP_ERR_CUDA, "no CUDA device");
  if (dev >= 0 && dev < 64 && cached[dev]) {
    *sms = cached[dev];
    return TPMLP_OK;
  }
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev))
    return bad(TPMLP_ERR_CUDA, "no CUDA device");
  if (major != 10 || minor != 3) return bad(TPMLP_ERR_UNSUPPORTED, "needs an sm_103 device");
  if (dev >= 0 && dev < 64) cached[dev] = n;
  *sms = n;
  return TPMLP_OK;
}

}  // namespace

extern "C" {

tpmlp_status tpattn_packed_forward(const tpattn_packed_desc* p, const void* q, int64_t ld_q, const void* k,
                                   int64_t ld_k, const void* v, int64_t ld_v, void* out, int64_t ld_out, float* lse,
                                   uint32_t* status, void* stream) {
  PK_TRY(check_desc(p));
  if (p->rows == 0 || p->batch == 0) return TPMLP_OK;
  const int64_t zq = (int64_t)p->n_heads * p->head_dim, zk = (int64_t)p->n_kv_heads * p->head_dim;
  PK_TRY(check_rows(q, ld_q, zq));
  PK_TRY(check_rows(k, ld_k, zk));
  PK_TRY(check_rows(v, ld_v, zk));
  PK_TRY(check_rows(out, ld_out, zq));
  if (!status) return bad(TPMLP_ERR_ARG, "status is NULL");
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(status)) & 3u)
    return bad(TPMLP_ERR_ARG, "lse or status not 4-byte aligned");
  if (out == q && ld_out != ld_q && p->rows > 1) return bad(TPMLP_ERR_ARG, "in place needs equal strides");
  if (out == k || out == v) return bad(TPMLP_ERR_ARG, "out is the keys or values");
  int sms = 0;
  PK_TRY(current_sms(&sms));
  VarFwdArgs a{};
  a.seq = rows_of(p);
  a.q = q;
  a.ld_q = ld_q;
  a.k = k;
  a.ld_k = ld_k;
  a.v = v;
  a.ld_v = ld_v;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.nq = p->n_heads;
  a.nkv = p->n_kv_heads;
  a.d = p->head_dim;
  a.scale = p->scale;
  a.window = p->window;
  a.sinks = p->sinks;
  limit_window(&a.window, &a.sinks, p->rows);
  a.status = status;
  const cudaError_t e = launch_var_fwd(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPMLP_OK : bad(TPMLP_ERR_CUDA, cudaGetErrorString(e));
}

size_t tpattn_packed_workspace_bytes(int64_t rows, int32_t n_heads) {
  if (rows < 0 || rows > (1 << 28) || n_heads < 1 || n_heads > 65536) return 0;
  return ((size_t)rows * n_heads * sizeof(float2) + 255) & ~size_t(255);
}

tpmlp_status tpattn_packed_backward(const tpattn_packed_desc* p, const void* q, int64_t ld_q, const void* k,
                                    int64_t ld_k, const void* v, int64_t ld_v, const void* out, int64_t ld_out,
                                    const float* lse, const void* dout, int64_t ld_dout, void* dq, int64_t ld_dq,
                                    void* dk, int64_t ld_dk, void* dv, int64_t ld_dv, void* workspace,
                                    size_t workspace_bytes, uint32_t* status, void* stream) {
  PK_TRY(check_desc(p));
  if (p->rows == 0 || p->batch == 0) return TPMLP_OK;
  const int64_t zq = (int64_t)p->n_heads * p->head_dim, zk = (int64_t)p->n_kv_heads * p->head_dim;
  PK_TRY(check_rows(q, ld_q, zq));
  PK_TRY(check_rows(k, ld_k, zk));
  PK_TRY(check_rows(v, ld_v, zk));
  PK_TRY(check_rows(out, ld_out, zq));
  PK_TRY(check_rows(dout, ld_dout, zq));
  PK_TRY(check_rows(dq, ld_dq, zq));
  PK_TRY(check_rows(dk, ld_dk, zk));
  PK_TRY(check_rows(dv, ld_dv, zk));
  if (!lse || !status) return bad(TPMLP_ERR_ARG, "lse or status is NULL");
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(status)) & 3u)
    return bad(TPMLP_ERR_ARG, "lse or status not 4-byte aligned");
  const void* const written[] = {dq, dk, dv};
  for (int i = 0; i < 3; ++i) {
    for (const void* in : {q, k, v, out, dout})
      if (written[i] == in) return bad(TPMLP_ERR_ARG, "a gradient is one of the inputs");
    for (int j = 0; j < i; ++j)
      if (written[i] == written[j]) return bad(TPMLP_ERR_ARG, "the same tensor for two gradients");
  }
  if (!workspace || !a16(workspace)) return bad(TPMLP_ERR_ARG, "workspace must be 16-byte aligned");
  if (workspace_bytes < tpattn_packed_workspace_bytes(p->rows, p->n_heads))
    return bad(TPMLP_ERR_ARG, "workspace too small");
  int sms = 0;
  PK_TRY(current_sms(&sms));
  VarBwdArgs a{};
  a.seq = rows_of(p);
  a.q = q;
  a.ld_q = ld_q;
  a.k = k;
  a.ld_k = ld_k;
  a.v = v;
  a.ld_v = ld_v;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.dout = dout;
  a.ld_dout = ld_dout;
  a.dq = dq;
  a.ld_dq = ld_dq;
  a.dk = dk;
  a.ld_dk = ld_dk;
  a.dv = dv;
  a.ld_dv = ld_dv;
  a.stats = static_cast<float2*>(workspace);
  a.nq = p->n_heads;
  a.nkv = p->n_kv_heads;
  a.d = p->head_dim;
  a.scale = p->scale;
  a.window = p->window;
  a.sinks = p->sinks;
  limit_window(&a.window, &a.sinks, p->rows);
  a.status = status;
  const cudaError_t e = launch_var_bwd(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPMLP_OK : bad(TPMLP_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
