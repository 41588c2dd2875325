// Attention of sequences of different lengths, one warp a row and head:
//   s_t = scale q . k_t over the tokens t that the row's token sees,
//   out = softmax(s) V,  lse = log sum exp s,
// and its gradients
//   P = exp(s - lse), D = sum_t P dP, dP = dO V^T, dS = scale P (dP - D),
//   dQ = dS K, dK = sum over the group's heads dS^T Q, dV = sum P^T dO.
#include <cuda_bf16.h>

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
    *out = seq_span(s, b, -1, &bad);
    *b_out = b;
    return row - out->first < out->count;
  }
  for (int b = 0; b < s.batch; ++b) {
    const SeqSpan r = seq_span(s, b, -1, &bad);
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
      if (!(t <= p && (a.window == 0 || p - t < a.window || t < a.sinks))) continue;
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
    if (!(t <= p && (a.window == 0 || p - t < a.window || t < a.sinks))) continue;
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
