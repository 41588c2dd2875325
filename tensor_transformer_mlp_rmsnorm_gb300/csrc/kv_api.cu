// C ABI of the query/key norm and rotation (tpattn_rotary_init, tpattn_qk_rope_*)
// and of the paged key/value cache (tpkv_*): argument checks, the rotation's
// fixed-point frequencies, the workspace layout and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "../../include/tpmlp.h"
#include "kv_ctx.h"

namespace tpmlp {

// Null if `r` is a rotation that heads of d values can take.
const char* rotary_error(const tpattn_rotary* r, int d) {
  if (!r) return nullptr;
  if (r->rot_dim < 0 || r->rot_dim % 16 != 0 || r->rot_dim > d) return "rot_dim must be a multiple of 16 within head_dim";
  if (r->interleaved != 0 && r->interleaved != 1) return "interleaved must be 0 or 1";
  return nullptr;
}

RopeFreqs freqs_of(const tpattn_rotary* r) {
  RopeFreqs f{};
  if (r) {
    f.rot = r->rot_dim;
    f.interleaved = r->interleaved;
    for (int i = 0; i < r->rot_dim / 2; ++i) f.turn[i] = r->turn[i];
  }
  return f;
}

}  // namespace tpmlp

using namespace tpmlp;

namespace {

thread_local const char* g_kv_err = "";

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t al256(size_t v) { return (v + 255) & ~size_t(255); }
bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 192 || d == 256; }

tpmlp_status bad(tpmlp_status s, const char* m) {
  set_thread_error(m);
  return s;
}

constexpr int MAX_DEV = 64;

// Multiprocessors of the current device if it is an sm_103, looked up once a device.
tpmlp_status current_sms(int* sms) {
  static int cached[MAX_DEV] = {};  // written with one value only
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return bad(TPMLP_ERR_CUDA, "no CUDA device");
  if (dev >= 0 && dev < MAX_DEV && cached[dev]) {
    *sms = cached[dev];
    return TPMLP_OK;
  }
  int major = 0, minor = 0, n = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev))
    return bad(TPMLP_ERR_CUDA, "no CUDA device");
  if (major != 10 || minor != 3) return bad(TPMLP_ERR_UNSUPPORTED, "needs an sm_103 device");
  if (dev >= 0 && dev < MAX_DEV) cached[dev] = n;
  *sms = n;
  return TPMLP_OK;
}

// Checks of both directions of the row call.
tpmlp_status check_desc(const tpattn_qk_desc* q, const tpattn_rotary* rot) {
  if (!q) return bad(TPMLP_ERR_ARG, "descriptor is NULL");
  if (q->reserved != 0) return bad(TPMLP_ERR_ARG, "reserved must be 0");
  if (q->dtype != TPMLP_F32 && q->dtype != TPMLP_BF16) return bad(TPMLP_ERR_UNSUPPORTED, "unknown dtype");
  if (!head_dim_ok(q->head_dim)) return bad(TPMLP_ERR_SHAPE, "head_dim must be 64, 128, 192 or 256");
  if (q->rows < 0 || q->rows > ((int64_t)1 << 40)) return bad(TPMLP_ERR_SHAPE, "rows out of range");
  if (q->n_heads < 0 || q->n_kv_heads < 0 || q->n_heads > 65536 || q->n_kv_heads > 65536)
    return bad(TPMLP_ERR_SHAPE, "head counts out of range");
  if (q->seq < 0) return bad(TPMLP_ERR_SHAPE, "seq must be >= 0");
  if (!(q->eps >= 0.0f) || !std::isfinite(q->eps)) return bad(TPMLP_ERR_ARG, "eps must be finite and >= 0");
  if (!q->positions && (q->seq == 0 ? q->rows : q->seq) > 0x7fffffff)
    return bad(TPMLP_ERR_SHAPE, "positions must fit 32 bits");
  if (reinterpret_cast<uintptr_t>(q->positions) & 3u) return bad(TPMLP_ERR_ARG, "positions not 4-byte aligned");
  if (!a16(q->q_norm_w) || !a16(q->k_norm_w)) return bad(TPMLP_ERR_ARG, "norm weight not 16-byte aligned");
  if (const char* m = rotary_error(rot, q->head_dim)) return bad(TPMLP_ERR_SHAPE, m);
  return TPMLP_OK;
}

tpmlp_status check_rows(const char* what_null, const void* p, int64_t ld, int64_t width, bool empty) {
  if (ld % 8 != 0 || ld < width || ld > ((int64_t)1 << 40))
    return bad(TPMLP_ERR_SHAPE, "row strides must be multiples of 8 and hold a row");
  if (!p && !empty) return bad(TPMLP_ERR_ARG, what_null);
  if (!a16(p)) return bad(TPMLP_ERR_ARG, "tensor not 16-byte aligned");
  return TPMLP_OK;
}

#define KV_TRY(expr)                \
  do {                              \
    const tpmlp_status s_ = (expr); \
    if (s_ != TPMLP_OK) return s_;  \
  } while (0)

const char* kv_config_error(const tpkv_config* c, tpmlp_status* s) {
  *s = TPMLP_ERR_ARG;
  if (!c) return "config is NULL";
  if (c->reserved != 0) return "reserved must be 0";
  *s = TPMLP_ERR_UNSUPPORTED;
  if (c->cache_dtype != TPKV_BF16 && c->cache_dtype != TPKV_E4M3) return "unknown cache dtype";
  *s = TPMLP_ERR_SHAPE;
  if (c->num_pages < 1 || c->num_pages > 0x7fffffff) return "num_pages out of range";
  if (c->page_size < 8 || c->page_size % 8 != 0 || c->page_size > 65536)
    return "page_size must be a multiple of 8, at most 65536";
  if (c->max_batch < 1 || c->max_batch > (1 << 20)) return "max_batch out of range";
  if (c->n_kv_heads < 1 || c->n_heads < 1 || c->n_heads > 65536 || c->n_heads % c->n_kv_heads != 0)
    return "n_heads must be a positive multiple of n_kv_heads";
  if (!head_dim_ok(c->head_dim)) return "head_dim must be 64, 128, 192 or 256";
  *s = TPMLP_OK;
  return nullptr;
}

struct KvLayout {
  size_t status, counters, part, total;
};
// Sized for the largest worker count, so that it does not depend on the device.
KvLayout kv_layout(const tpkv_config& c) {
  KvLayout L{};
  L.status = 0;
  L.counters = 256;
  L.part = al256(L.counters + 3 * (size_t)KV_MAX_WORKERS * sizeof(uint32_t));
  L.total = al256(L.part + 2 * (size_t)KV_MAX_WORKERS *
                               kv_decode_part_floats(c.head_dim, c.n_heads / c.n_kv_heads) * sizeof(float));
  return L;
}

// The context's device while a call runs.
struct OnDevice {
  int prev = -1;
  explicit OnDevice(int dev) {
    int cur = -1;
    if (cudaGetDevice(&cur) == cudaSuccess && cur != dev && cudaSetDevice(dev) == cudaSuccess) prev = cur;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Clears `bytes` of the workspace on the context's stream; launches on other
// streams wait for it (wait_for_clear).
cudaError_t clear_workspace(tpkv_ctx* c, void* p, size_t bytes) {
  cudaError_t e = cudaMemsetAsync(p, 0, bytes, c->stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (e == cudaSuccess) e = cudaStreamIsCapturing(c->stream, &cap);
  if (e != cudaSuccess) return e;
  c->clear_pending = cap == cudaStreamCaptureStatusNone;  // in a graph it is ordered by the graph
  if (!c->clear_pending) return cudaSuccess;
  c->clear_stream = c->clear_seen = c->stream;
  return cudaEventRecord(c->cleared, c->stream);
}

// Orders what is launched on `st` next behind the last clear.  A captured
// launch cannot wait for an event from outside its graph, so the host does.
cudaError_t wait_for_clear(tpkv_ctx* c, cudaStream_t st) {
  if (!c->clear_pending) return cudaSuccess;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(st, &cap);
  if (e != cudaSuccess) return e;
  if (cap != cudaStreamCaptureStatusNone) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    e = cudaEventSynchronize(c->cleared);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) c->clear_pending = false;
    return e != cudaSuccess ? e : back;
  }
  if (st == c->clear_stream || st == c->clear_seen) return cudaSuccess;
  e = cudaStreamWaitEvent(st, c->cleared, 0);
  if (e == cudaSuccess) c->clear_seen = st;
  return e;
}

}  // namespace

extern "C" {

tpmlp_status tpattn_rotary_init(tpattn_rotary* r, int32_t rot_dim, int32_t interleaved, const double* inv_freq) {
  if (!r) return bad(TPMLP_ERR_ARG, "rotary is NULL");
  if (rot_dim < 0 || rot_dim % 16 != 0 || rot_dim > TPATTN_MAX_ROT_DIM)
    return bad(TPMLP_ERR_SHAPE, "rot_dim must be a multiple of 16, at most 256");
  if (interleaved != 0 && interleaved != 1) return bad(TPMLP_ERR_ARG, "interleaved must be 0 or 1");
  if (rot_dim > 0 && !inv_freq) return bad(TPMLP_ERR_ARG, "inv_freq is NULL");
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!(std::fabs(inv_freq[i]) <= 1048576.0)) return bad(TPMLP_ERR_ARG, "a frequency is not finite or above 2^20");
  r->rot_dim = rot_dim;
  r->interleaved = interleaved;
  // 1 / 2pi as the sum of two doubles; the product's rounding error is taken along
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  for (int i = 0; i < TPATTN_MAX_ROT_DIM / 2; ++i) r->turn[i] = 0;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double p = inv_freq[i] * hi;
    const double e = std::fma(inv_freq[i], hi, -p) + inv_freq[i] * lo;
    double frac = p - std::nearbyint(p);  // exact, within half a turn
    if (frac >= 0.5) frac -= 1.0;
    // both parts as multiples of 2^-64, added mod 1
    uint64_t t = (uint64_t)(int64_t)std::ldexp(frac, 64);
    t += (uint64_t)(int64_t)std::nearbyint(std::ldexp(e, 64));
    r->turn[i] = t;
  }
  return TPMLP_OK;
}

tpmlp_status tpattn_qk_rope_forward(const tpattn_qk_desc* q, const tpattn_rotary* rot, const void* x, int64_t ld_x,
                                    void* out, int64_t ld_out, void* stream) {
  KV_TRY(check_desc(q, rot));
  const int64_t width = (int64_t)(q->n_heads + q->n_kv_heads) * q->head_dim;
  const bool empty = q->rows == 0 || width == 0;
  KV_TRY(check_rows("x is NULL", x, ld_x, width, empty));
  KV_TRY(check_rows("out is NULL", out, ld_out, width, empty));
  if (x == out && ld_x != ld_out && q->rows > 1) return bad(TPMLP_ERR_ARG, "in place needs equal strides");
  if (empty) return TPMLP_OK;
  int sms = 0;
  KV_TRY(current_sms(&sms));
  RopeArgs a{};
  a.in = x;
  a.ld_in = ld_x;
  a.out = out;
  a.ld_out = ld_out;
  a.rows = q->rows;
  a.nq = q->n_heads;
  a.nkv = q->n_kv_heads;
  a.q_norm_w = q->q_norm_w;
  a.k_norm_w = q->k_norm_w;
  a.eps = q->eps;
  a.pos = q->positions;
  a.seq = q->seq;
  const cudaError_t e =
      launch_qk_rope(q->dtype, q->head_dim, a, freqs_of(rot), sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPMLP_OK : bad(TPMLP_ERR_CUDA, cudaGetErrorString(e));
}

size_t tpattn_qk_rope_workspace_bytes(int32_t head_dim) {
  return head_dim_ok(head_dim) ? (size_t)ROPE_MAX_PARTS * 2 * head_dim * sizeof(float) : 0;
}

tpmlp_status tpattn_qk_rope_backward(const tpattn_qk_desc* q, const tpattn_rotary* rot, const void* x, int64_t ld_x,
                                     const void* dout, int64_t ld_dout, void* dx, int64_t ld_dx, float* dq_norm_w,
                                     float* dk_norm_w, void* workspace, size_t workspace_bytes, void* stream) {
  KV_TRY(check_desc(q, rot));
  const int64_t width = (int64_t)(q->n_heads + q->n_kv_heads) * q->head_dim;
  const bool empty = q->rows == 0 || width == 0, norm = q->q_norm_w || q->k_norm_w;
  if (norm) KV_TRY(check_rows("x is NULL", x, ld_x, width, empty));
  KV_TRY(check_rows("dout is NULL", dout, ld_dout, width, empty));
  KV_TRY(check_rows("dx is NULL", dx, ld_dx, width, empty));
  if (dout == dx && ld_dout != ld_dx && q->rows > 1) return bad(TPMLP_ERR_ARG, "in place needs equal strides");
  if (!q->q_norm_w != !dq_norm_w || !q->k_norm_w != !dk_norm_w)
    return bad(TPMLP_ERR_ARG, "weight gradients are given exactly for the norm weights");
  if (dq_norm_w && dq_norm_w == dk_norm_w) return bad(TPMLP_ERR_ARG, "the same tensor for both weight gradients");
  if (!a16(dq_norm_w) || !a16(dk_norm_w)) return bad(TPMLP_ERR_ARG, "tensor not 16-byte aligned");
  if (norm && !empty) {
    if (!workspace || !a16(workspace)) return bad(TPMLP_ERR_ARG, "workspace must be 16-byte aligned");
    if (workspace_bytes < tpattn_qk_rope_workspace_bytes(q->head_dim)) return bad(TPMLP_ERR_ARG, "workspace too small");
  }
  if (empty && !norm) return TPMLP_OK;
  int sms = 0;
  KV_TRY(current_sms(&sms));
  RopeBwdArgs a{};
  a.x = x;
  a.ld_x = ld_x;
  a.dout = dout;
  a.ld_dout = ld_dout;
  a.dx = dx;
  a.ld_dx = ld_dx;
  a.rows = q->rows;
  a.nq = q->n_heads;
  a.nkv = q->n_kv_heads;
  a.q_norm_w = q->q_norm_w;
  a.k_norm_w = q->k_norm_w;
  a.eps = q->eps;
  a.pos = q->positions;
  a.seq = q->seq;
  a.part = norm ? static_cast<float*>(workspace) : nullptr;
  const cudaError_t e = launch_qk_rope_bwd(q->dtype, q->head_dim, a, freqs_of(rot), sms,
                                           static_cast<cudaStream_t>(stream), dq_norm_w, dk_norm_w);
  return e == cudaSuccess ? TPMLP_OK : bad(TPMLP_ERR_CUDA, cudaGetErrorString(e));
}

size_t tpkv_workspace_bytes(const tpkv_config* cfg) {
  tpmlp_status s;
  return kv_config_error(cfg, &s) ? 0 : kv_layout(*cfg).total;
}

tpmlp_status tpkv_create(const tpkv_config* cfg, void* stream, tpkv_ctx** out) {
  if (!out) return TPMLP_ERR_ARG;
  *out = nullptr;
  tpmlp_status s;
  if (const char* m = kv_config_error(cfg, &s)) {
    g_kv_err = m;
    return s;
  }
  int sms = 0, dev = 0;
  s = current_sms(&sms);
  if (s != TPMLP_OK) {
    g_kv_err = s == TPMLP_ERR_UNSUPPORTED ? "needs an sm_103 device" : "no CUDA device";
    return s;
  }
  cudaGetDevice(&dev);
  tpkv_ctx* c = new (std::nothrow) tpkv_ctx();
  if (!c) {
    g_kv_err = "out of host memory";
    return TPMLP_ERR_CUDA;
  }
  const cudaError_t e = cudaEventCreateWithFlags(&c->cleared, cudaEventDisableTiming);
  if (e != cudaSuccess) {
    g_kv_err = cudaGetErrorString(e);
    delete c;
    return TPMLP_ERR_CUDA;
  }
  c->cfg = *cfg;
  c->stream = static_cast<cudaStream_t>(stream);
  c->device = dev;
  c->num_sms = sms;
  c->box_tokens = kv_decode_tile(cfg->head_dim);
  while (cfg->page_size % c->box_tokens) c->box_tokens /= 2;  // ends at 8 at the latest
  c->workers = kv_decode_workers(sms);
  if (c->workers > KV_MAX_WORKERS) c->workers = KV_MAX_WORKERS;
  *out = c;
  return TPMLP_OK;
}

tpmlp_status tpkv_bind_workspace(tpkv_ctx* c, void* dev, size_t bytes) {
  if (!c) return TPMLP_ERR_ARG;
  if (!dev || (reinterpret_cast<uintptr_t>(dev) & 255u))
    return c->fail(TPMLP_ERR_ARG, "workspace must be 256-byte aligned");
  const KvLayout L = kv_layout(c->cfg);
  if (bytes < L.total) return c->fail(TPMLP_ERR_ARG, "workspace too small");
  OnDevice on(c->device);
  // the status word and the arrival counters; partial results need no initial contents
  const cudaError_t e = clear_workspace(c, dev, L.part);
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  uint8_t* w = static_cast<uint8_t*>(dev);
  c->status = reinterpret_cast<uint32_t*>(w + L.status);
  c->counters = reinterpret_cast<uint32_t*>(w + L.counters);
  c->part = reinterpret_cast<float*>(w + L.part);
  return TPMLP_OK;
}

tpmlp_status tpkv_set_stream(tpkv_ctx* c, void* stream) {
  if (!c) return TPMLP_ERR_ARG;
  c->stream = static_cast<cudaStream_t>(stream);
  return TPMLP_OK;
}

tpmlp_status tpkv_bind_cache(tpkv_ctx* c, void* k, void* v, int64_t stride_page, int64_t stride_head,
                             int64_t stride_slot, const float* k_inv_scale, const float* v_inv_scale) {
  if (!c) return TPMLP_ERR_ARG;
  if (!k || !v) return c->fail(TPMLP_ERR_ARG, "NULL cache");
  if (!a16(k) || !a16(v)) return c->fail(TPMLP_ERR_ARG, "cache not 16-byte aligned");
  const tpkv_config& cf = c->cfg;
  const bool f8 = cf.cache_dtype == TPKV_E4M3;
  const int64_t unit = f8 ? 16 : 8, most = ((int64_t)1 << 39);
  for (int64_t s : {stride_page, stride_head, stride_slot})
    if (s <= 0 || s % unit != 0 || s > most)
      return c->fail(TPMLP_ERR_SHAPE, "cache strides must be positive multiples of 16 bytes");
  if (stride_slot < cf.head_dim || (cf.n_kv_heads > 1 && stride_head < cf.head_dim))
    return c->fail(TPMLP_ERR_SHAPE, "a cache stride is below head_dim");
  if (!f8 && (k_inv_scale || v_inv_scale)) return c->fail(TPMLP_ERR_ARG, "a bf16 cache has no scales");
  if ((reinterpret_cast<uintptr_t>(k_inv_scale) | reinterpret_cast<uintptr_t>(v_inv_scale)) & 3u)
    return c->fail(TPMLP_ERR_ARG, "scales not 4-byte aligned");
  CUtensorMap km, vm;
  if (!make_cache_map(&km, k, f8, cf.head_dim, cf.page_size, cf.n_kv_heads, cf.num_pages, stride_page, stride_head,
                      stride_slot, c->box_tokens) ||
      !make_cache_map(&vm, v, f8, cf.head_dim, cf.page_size, cf.n_kv_heads, cf.num_pages, stride_page, stride_head,
                      stride_slot, c->box_tokens))
    return c->fail(TPMLP_ERR_CUDA, "the cache's tensor map could not be made");
  c->kmap = km;
  c->vmap = vm;
  c->k = k;
  c->v = v;
  c->stride_page = stride_page;
  c->stride_head = stride_head;
  c->stride_slot = stride_slot;
  c->k_inv_scale = k_inv_scale;
  c->v_inv_scale = v_inv_scale;
  return TPMLP_OK;
}

tpmlp_status tpkv_set_rotary(tpkv_ctx* c, const tpattn_rotary* rot, const void* q_norm_w, const void* k_norm_w,
                             float eps) {
  if (!c) return TPMLP_ERR_ARG;
  if (const char* m = rotary_error(rot, c->cfg.head_dim)) return c->fail(TPMLP_ERR_SHAPE, m);
  if (!a16(q_norm_w) || !a16(k_norm_w)) return c->fail(TPMLP_ERR_ARG, "norm weight not 16-byte aligned");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return c->fail(TPMLP_ERR_ARG, "eps must be finite and >= 0");
  c->freqs = freqs_of(rot);
  c->q_norm_w = q_norm_w;
  c->k_norm_w = k_norm_w;
  c->eps = eps;
  return TPMLP_OK;
}

tpmlp_status tpkv_append(tpkv_ctx* c, int64_t rows, int32_t batch, const void* qkv, int64_t ld_qkv,
                         const int32_t* cu_rows, const int32_t* new_lens, const int32_t* past_lens,
                         const int32_t* table, int64_t ld_table, int32_t max_pages, int32_t transform, void* q_out,
                         int64_t ld_q) {
  if (!c) return TPMLP_ERR_ARG;
  KV_TRY(kv_check_call(c, batch, past_lens, table, ld_table, max_pages));
  KV_TRY(kv_check_append(c));
  const tpkv_config& cf = c->cfg;
  const int64_t W = (int64_t)(cf.n_heads + 2 * cf.n_kv_heads) * cf.head_dim, Z = (int64_t)cf.n_heads * cf.head_dim;
  if (rows < 0 || rows > 0x7fffffff) return c->fail(TPMLP_ERR_SHAPE, "rows out of range");
  if (cu_rows && new_lens) return c->fail(TPMLP_ERR_ARG, "cu_rows or new_lens, not both");
  if (!cu_rows && (batch == 0 ? rows != 0 : rows % batch != 0))
    return c->fail(TPMLP_ERR_SHAPE, "without cu_rows, rows must be a multiple of batch");
  if ((reinterpret_cast<uintptr_t>(cu_rows) | reinterpret_cast<uintptr_t>(new_lens)) & 3u)
    return c->fail(TPMLP_ERR_ARG, "index tensor not 4-byte aligned");
  if (transform != 0 && transform != 1) return c->fail(TPMLP_ERR_ARG, "transform must be 0 or 1");
  if (ld_qkv % 8 != 0 || ld_qkv < W || (q_out && (ld_q % 8 != 0 || ld_q < Z)))
    return c->fail(TPMLP_ERR_SHAPE, "row strides must be multiples of 8 and hold a row");
  if (rows == 0 || batch == 0) return TPMLP_OK;
  if (!qkv) return c->fail(TPMLP_ERR_ARG, "qkv is NULL");
  if (!a16(qkv) || !a16(q_out)) return c->fail(TPMLP_ERR_ARG, "tensor not 16-byte aligned");
  if (q_out == qkv && ld_q != ld_qkv && rows > 1) return c->fail(TPMLP_ERR_ARG, "in place needs equal strides");
  QkTransform tr;
  if (transform) tr = {&c->freqs, c->q_norm_w, c->k_norm_w, c->eps};
  return kv_run_append(c, rows, batch, qkv, ld_qkv, cu_rows, new_lens, past_lens, table, ld_table, max_pages, tr,
                       q_out, ld_q, c->stream);
}

tpmlp_status tpkv_decode(tpkv_ctx* c, int32_t batch, const void* q, int64_t ld_q, const int32_t* lens, int32_t len_add,
                         const int32_t* table, int64_t ld_table, int32_t max_pages, float scale, int32_t window,
                         int32_t sinks, void* out, int64_t ld_out, float* lse) {
  if (!c) return TPMLP_ERR_ARG;
  KV_TRY(kv_check_call(c, batch, lens, table, ld_table, max_pages));
  const int64_t Z = (int64_t)c->cfg.n_heads * c->cfg.head_dim;
  if (ld_q % 8 != 0 || ld_q < Z || ld_out % 8 != 0 || ld_out < Z)
    return c->fail(TPMLP_ERR_SHAPE, "row strides must be multiples of 8 and hold a row");
  if (!std::isfinite(scale)) return c->fail(TPMLP_ERR_ARG, "scale must be finite");
  if (window < 0 || sinks < 0) return c->fail(TPMLP_ERR_ARG, "window and sinks must be >= 0");
  if (batch == 0) return TPMLP_OK;
  if (!q || !out) return c->fail(TPMLP_ERR_ARG, "NULL tensor");
  if (!a16(q) || !a16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return c->fail(TPMLP_ERR_ARG, "tensor not 16-byte aligned");
  if (q == out && ld_q != ld_out && batch > 1) return c->fail(TPMLP_ERR_ARG, "in place needs equal strides");
  return kv_run_decode(c, batch, q, ld_q, lens, len_add, table, ld_table, max_pages, scale, window, sinks, out, ld_out,
                       lse, c->stream);
}

tpmlp_status tpkv_sync(tpkv_ctx* c) {
  if (!c) return TPMLP_ERR_ARG;
  OnDevice on(c->device);
  cudaError_t e = cudaStreamSynchronize(c->stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  if (c->clear_stream == c->stream) c->clear_pending = false;  // it is done
  if (!c->status) return TPMLP_OK;
  uint32_t st = 0;
  e = cudaMemcpy(&st, c->status, sizeof st, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  if (!st) return TPMLP_OK;
  // a CTA that gave up has not counted its arrival: the counters, which lie
  // behind the status word, then start anew too
  const KvLayout L = kv_layout(c->cfg);
  e = clear_workspace(c, c->status, st & STATUS_TIMEOUT ? L.part - L.status : sizeof st);
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  if (st & STATUS_TIMEOUT) return c->fail(TPMLP_ERR_TIMEOUT, "a bounded device wait gave up");
  return c->fail(TPMLP_ERR_ARG, "a page or a length was outside the cache");
}

uint64_t tpkv_launch_count(const tpkv_ctx* c) { return c ? c->launches : 0; }
const char* tpkv_last_error(const tpkv_ctx* c) { return c ? c->err : g_kv_err; }
void tpkv_destroy(tpkv_ctx* c) {
  if (!c) return;
  cudaEventDestroy(c->cleared);
  delete c;
}

}  // extern "C"

namespace tpmlp {

tpmlp_status kv_check_call(tpkv_ctx* c, int64_t batch, const int32_t* lens, const int32_t* table, int64_t ld_table,
                           int32_t max_pages) {
  if (!c->status) return c->fail(TPMLP_ERR_ORDER, "no workspace bound");
  if (!c->k) return c->fail(TPMLP_ERR_ORDER, "no cache bound");
  if (batch < 0 || batch > c->cfg.max_batch) return c->fail(TPMLP_ERR_SHAPE, "batch exceeds max_batch");
  if (max_pages < 0 || ld_table < max_pages || (int64_t)max_pages * c->cfg.page_size > (1 << 30))
    return c->fail(TPMLP_ERR_SHAPE, "block table out of range (at most 2^30 tokens a sequence)");
  if (batch > 0 && (!lens || (!table && max_pages > 0))) return c->fail(TPMLP_ERR_ARG, "NULL lengths or block table");
  if ((reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(table)) & 3u)
    return c->fail(TPMLP_ERR_ARG, "index tensor not 4-byte aligned");
  return TPMLP_OK;
}

tpmlp_status kv_check_append(tpkv_ctx* c) {
  return c->k == c->v ? c->fail(TPMLP_ERR_ARG, "keys and values are the same tensor, which cannot be appended to")
                      : TPMLP_OK;
}

tpmlp_status kv_run_append(tpkv_ctx* c, int64_t rows, int32_t batch, const void* qkv, int64_t ld_qkv,
                           const int32_t* cu_rows, const int32_t* new_lens, const int32_t* past_lens,
                           const int32_t* table, int64_t ld_table, int32_t max_pages, const QkTransform& tr,
                           void* q_out, int64_t ld_q, cudaStream_t st) {
  const tpkv_config& cf = c->cfg;
  RopeArgs a{};
  a.in = qkv;
  a.ld_in = ld_qkv;
  a.out = q_out;
  a.ld_out = ld_q;
  a.rows = rows;
  a.nq = cf.n_heads;
  a.nkv = cf.n_kv_heads;
  a.q_norm_w = tr.q_norm_w;
  a.k_norm_w = tr.k_norm_w;
  a.eps = tr.eps;
  a.batch = batch;
  a.rows_per_seq = (int)(rows / batch);
  a.cu_rows = cu_rows;
  a.new_lens = new_lens;
  a.past_lens = past_lens;
  a.table = table;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  a.page_size = cf.page_size;
  a.num_pages = cf.num_pages;
  a.k_cache = c->k;
  a.v_cache = c->v;
  a.stride_page = c->stride_page;
  a.stride_head = c->stride_head;
  a.stride_slot = c->stride_slot;
  a.k_inv_scale = c->k_inv_scale;
  a.v_inv_scale = c->v_inv_scale;
  a.status = c->status;
  OnDevice on(c->device);
  cudaError_t e = wait_for_clear(c, st);
  if (e == cudaSuccess)
    e = launch_kv_append(cf.cache_dtype == TPKV_E4M3, cf.head_dim, a, tr.freqs ? *tr.freqs : RopeFreqs{}, c->num_sms,
                         st);
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  ++c->launches;
  return TPMLP_OK;
}

tpmlp_status kv_run_decode(tpkv_ctx* c, int32_t batch, const void* q, int64_t ld_q, const int32_t* lens,
                           int32_t len_add, const int32_t* table, int64_t ld_table, int32_t max_pages, float scale,
                           int32_t window, int32_t sinks, void* out, int64_t ld_out, float* lse, cudaStream_t st) {
  const tpkv_config& cf = c->cfg;
  DecodeArgs a{};
  a.q = q;
  a.ld_q = ld_q;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.lens = lens;
  a.len_add = len_add;
  a.table = table;
  a.ld_table = ld_table;
  a.max_pages = max_pages;
  a.page_size = cf.page_size;
  a.num_pages = cf.num_pages;
  a.batch = batch;
  a.nq = cf.n_heads;
  a.nkv = cf.n_kv_heads;
  a.hpg = cf.n_heads / cf.n_kv_heads;
  const int ht = kv_decode_head_tile(a.hpg);
  a.chunks = (a.hpg + ht - 1) / ht;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window;
  a.sinks = sinks;
  a.k_inv_scale = c->k_inv_scale;
  a.v_inv_scale = c->v_inv_scale;
  a.box_tokens = c->box_tokens;
  a.workers = c->workers;
  a.part = c->part;
  a.counters = c->counters;
  a.status = c->status;
  OnDevice on(c->device);
  cudaError_t e = wait_for_clear(c, st);
  if (e == cudaSuccess) e = launch_kv_decode(a, c->kmap, c->vmap, cf.head_dim, cf.cache_dtype == TPKV_E4M3, st);
  if (e != cudaSuccess) return c->fail(TPMLP_ERR_CUDA, cudaGetErrorString(e));
  ++c->launches;
  return TPMLP_OK;
}

}  // namespace tpmlp
