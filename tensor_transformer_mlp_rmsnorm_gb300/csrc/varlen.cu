// Attention of sequences of different lengths, one warp a row and head:
//   s_t = scale q . k_t over the tokens t that the row's token sees,
//   out = softmax(s) V,  lse = log sum exp s,
// and its gradients
//   P = exp(s - lse), D = sum_t P dP, dP = dO V^T, dS = scale P (dP - D),
//   dQ = dS K, dK = sum over the group's heads dS^T Q, dV = sum P^T dO.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "varlen.cuh"

namespace tpmlp {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row -> its sequence's span; false: nobody's.
__device__ bool row_span(const SeqRows& s, int row, SeqSpan* out, int* b_out, uint32_t* status) {
  bool bad = false;
  if (!s.cu_rows) {
    const int b = row / s.rows_per_seq;
    *out = seq_span(s, b, &bad);
    *b_out = b;
    return row - out->first < out->count;
  }
  for (int b = 0; b < s.batch; ++b) {
    const SeqSpan r = seq_span(s, b, &bad);
    if (row >= r.first && row - r.first < r.count) {
      *out = r;
      *b_out = b;
      if (bad) atomicOr(status, STATUS_BAD_INDEX);
      return true;
    }
  }
  if (bad) atomicOr(status, STATUS_BAD_INDEX);
  return false;
}

template <int D>
__device__ __forceinline__ void load_bf16(const void* p, int64_t off, int lane, float* f) {
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p) + off;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) f[i] = __bfloat162float(x[lane + 32 * i]);
}
template <int D>
__device__ __forceinline__ void store_bf16(void* p, int64_t off, int lane, const float* f) {
  __nv_bfloat16* x = static_cast<__nv_bfloat16*>(p) + off;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[lane + 32 * i] = __float2bfloat16(f[i]);
}

template <int D>
__global__ void __launch_bounds__(128) var_fwd_kernel(const VarFwdArgs a) {
  constexpr int V = D / 32;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= a.seq.rows * a.nq) return;
  const int row = (int)(id / a.nq), h = (int)(id % a.nq), g = h / (a.nq / a.nkv);
  SeqSpan sp;
  int b;
  if (!row_span(a.seq, row, &sp, &b, a.status)) return;
  float q[V], acc[V], m = -INFINITY, l = 0.0f;
  load_bf16<D>(a.q, (int64_t)row * a.ld_q + h * D, lane, q);
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  float ks = 1.0f, vs = 1.0f;
  if (a.e4m3 && a.k_inv_scale) ks = a.k_inv_scale[g];
  if (a.e4m3 && a.v_inv_scale) vs = a.v_inv_scale[g];
  const bool active = sp.past >= 0;
  int64_t p = (int64_t)sp.past + (row - sp.first);
  if (a.paged) {
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    if (p >= cap) {
      if (active && lane == 0) atomicOr(a.status, STATUS_BAD_INDEX);
      p = cap - 1;
    }
  }
  for (int t = 0; active && t <= (int)p; ++t) {
    if (!sees((int)p, t, a.window, a.sinks)) continue;
    float k[V], v[V];
    if (a.paged) {
      const int page = a.table[(int64_t)b * a.ld_table + t / a.page_size];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicOr(a.status, STATUS_BAD_INDEX);
        continue;
      }
      const int64_t off = (int64_t)page * a.stride_page + (int64_t)g * a.stride_head + (int64_t)(t % a.page_size) * a.stride_slot;
      if (a.e4m3) {
        const __nv_fp8_e4m3 *kc = static_cast<const __nv_fp8_e4m3*>(a.k_cache) + off,
                            *vc = static_cast<const __nv_fp8_e4m3*>(a.v_cache) + off;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          k[i] = (float)kc[lane + 32 * i];
          v[i] = (float)vc[lane + 32 * i];
        }
      } else {
        load_bf16<D>(a.k_cache, off, lane, k);
        load_bf16<D>(a.v_cache, off, lane, v);
      }
    } else {
      load_bf16<D>(a.k, (int64_t)(sp.first + t) * a.ld_k + g * D, lane, k);
      load_bf16<D>(a.v, (int64_t)(sp.first + t) * a.ld_v + g * D, lane, v);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(q[i], k[i], s);
    s = warp_sum(s) * (a.scale * ks);
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - base), w = expf(s - base);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(w, v[i], acc[i] * f);
  }
  const float r = active ? vs / l : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = active && p >= 0 ? acc[i] * r : 0.0f;
  store_bf16<D>(a.out, (int64_t)row * a.ld_out + h * D, lane, acc);
  if (a.lse && lane == 0) a.lse[id] = active ? m + logf(l) : -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(128) var_bwd_dq_kernel(const VarBwdArgs a) {
  constexpr int V = D / 32;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= a.seq.rows * a.nq) return;
  const int row = (int)(id / a.nq), h = (int)(id % a.nq), g = h / (a.nq / a.nkv);
  SeqSpan sp;
  int b;
  if (!row_span(a.seq, row, &sp, &b, a.status)) return;
  float q[V], go[V], acc[V], D_ = 0.0f, l = 0.0f;
  load_bf16<D>(a.q, (int64_t)row * a.ld_q + h * D, lane, q);
  load_bf16<D>(a.dout, (int64_t)row * a.ld_dout + h * D, lane, go);
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  const int p = row - sp.first;
  const float lse = a.lse[id];
  for (int pass = 0; pass < 2; ++pass) {
    for (int t = 0; t <= p; ++t) {
      if (!sees(p, t, a.window, a.sinks)) continue;
      float k[V], v[V], s = 0.0f, dp = 0.0f;
      load_bf16<D>(a.k, (int64_t)(sp.first + t) * a.ld_k + g * D, lane, k);
      load_bf16<D>(a.v, (int64_t)(sp.first + t) * a.ld_v + g * D, lane, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s = fmaf(q[i], k[i], s);
        dp = fmaf(go[i], v[i], dp);
      }
      s = warp_sum(s) * a.scale;
      dp = warp_sum(dp);
      const float w = expf(s - lse);
      if (pass == 0) {
        D_ = fmaf(w, dp, D_);
        l += w;
      } else {
        const float ds = w / l * (dp - D_) * a.scale;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
      }
    }
    if (pass == 0) D_ /= l;
  }
  store_bf16<D>(a.dq, (int64_t)row * a.ld_dq + h * D, lane, acc);
  if (lane == 0) a.stats[id] = make_float2(lse + logf(l), D_);
}

template <int D>
__global__ void __launch_bounds__(128) var_bwd_dkv_kernel(const VarBwdArgs a) {
  constexpr int V = D / 32;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= a.seq.rows * a.nkv) return;
  const int row = (int)(id / a.nkv), g = (int)(id % a.nkv), hpg = a.nq / a.nkv;
  SeqSpan sp;
  int b;
  if (!row_span(a.seq, row, &sp, &b, a.status)) return;
  float k[V], v[V], dk[V], dv[V];
  load_bf16<D>(a.k, (int64_t)row * a.ld_k + g * D, lane, k);
  load_bf16<D>(a.v, (int64_t)row * a.ld_v + g * D, lane, v);
#pragma unroll
  for (int i = 0; i < V; ++i) dk[i] = dv[i] = 0.0f;
  const int t = row - sp.first;
  for (int p = t; p < sp.count; ++p) {
    if (!sees(p, t, a.window, a.sinks)) continue;
    for (int h = g * hpg; h < (g + 1) * hpg; ++h) {
      float q[V], go[V], s = 0.0f, dp = 0.0f;
      load_bf16<D>(a.q, (int64_t)(sp.first + p) * a.ld_q + h * D, lane, q);
      load_bf16<D>(a.dout, (int64_t)(sp.first + p) * a.ld_dout + h * D, lane, go);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s = fmaf(q[i], k[i], s);
        dp = fmaf(go[i], v[i], dp);
      }
      s = warp_sum(s) * a.scale;
      dp = warp_sum(dp);
      const float2 st = a.stats[(int64_t)(sp.first + p) * a.nq + h];
      const float w = expf(s - st.x), ds = w * (dp - st.y) * a.scale;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dv[i] = fmaf(w, go[i], dv[i]);
        dk[i] = fmaf(ds, q[i], dk[i]);
      }
    }
  }
  store_bf16<D>(a.dk, (int64_t)row * a.ld_dk + g * D, lane, dk);
  store_bf16<D>(a.dv, (int64_t)row * a.ld_dv + g * D, lane, dv);
}

__global__ void __launch_bounds__(256) packed_rows_kernel(const SeqRows s, int32_t* pos, uint4* z, int64_t z16,
                                                          uint4* dz, int64_t dz16, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < s.rows; row += (int64_t)gridDim.x * 8) {
    SeqSpan sp;
    int b;
    const bool mine = row_span(s, (int)row, &sp, &b, status);
    if (pos && lane == 0) pos[row] = mine ? (int)row - sp.first : 0;
    if (mine) continue;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = lane; z && i < z16; i += 32) z[row * z16 + i] = zero;
    for (int64_t i = lane; dz && i < dz16; i += 32) dz[row * dz16 + i] = zero;
  }
}

template <int D>
cudaError_t bwd_d(const VarBwdArgs& a, cudaStream_t st) {
  var_bwd_dq_kernel<D><<<(unsigned)((a.seq.rows * a.nq + 3) / 4), 128, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  var_bwd_dkv_kernel<D><<<(unsigned)((a.seq.rows * a.nkv + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_rows(const SeqRows& s, int32_t* pos, void* z, int64_t z_bytes, void* dz, int64_t dz_bytes,
                               uint32_t* status, int num_sms, cudaStream_t st) {
  const int64_t want = (s.rows + 7) / 8, most = 8LL * num_sms;
  packed_rows_kernel<<<(unsigned)(want < most ? want : most), 256, 0, st>>>(
      s, pos, static_cast<uint4*>(z), z_bytes / 16, static_cast<uint4*>(dz), dz_bytes / 16, status);
  return cudaGetLastError();
}

cudaError_t launch_var_fwd(const VarFwdArgs& a, int, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.seq.rows * a.nq + 3) / 4);
  switch (a.d) {
    case 64: var_fwd_kernel<64><<<blocks, 128, 0, st>>>(a); break;
    case 128: var_fwd_kernel<128><<<blocks, 128, 0, st>>>(a); break;
    case 192: var_fwd_kernel<192><<<blocks, 128, 0, st>>>(a); break;
    case 256: var_fwd_kernel<256><<<blocks, 128, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_var_bwd(const VarBwdArgs& a, int, cudaStream_t st) {
  switch (a.d) {
    case 64: return bwd_d<64>(a, st);
    case 128: return bwd_d<128>(a, st);
    case 192: return bwd_d<192>(a, st);
    case 256: return bwd_d<256>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tpmlp
