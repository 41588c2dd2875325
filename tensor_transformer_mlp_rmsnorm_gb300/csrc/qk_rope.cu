// Queries and keys of the attention sublayer: the RMS norm of each head and
// the position rotation in one pass over the packed projection rows, its
// backward pass, and the same pass for new tokens with the keys and values
// stored into a paged cache on the way.
//
// A head x of d values at position p:
//   y = x * rsqrt(mean(x^2) + eps) * w                        (only with norm weights)
//   (z1, z2) = (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = p * f_j, for pair j
// over the first rot values; the others pass.  Backward, g the rotation of dz
// by -a and xh = x rstd:  dw = sum g xh,  dx = rstd (w g - xh mean(w g xh)).
//
// Angles.  a / 2pi mod 1 is what matters, so a frequency is kept in turns per
// position as a 64-bit fraction and the angle is the product with the position
// mod 2^64: exact for every 32-bit position, with no 64-bit floating point (a
// slow pipe here) and no table to read.  The top 32 bits go through
// sincospif; that is 2^-25 of a half turn, the rounding of the f32 result.
//
// What bounds it: memory (about 8 flops a byte are far below the f32 rate).
// A head belongs to d / 16 lanes; a lane holds two 16-byte (bf16) chunks whose
// values are each other's rotation partners, so the rotation needs no shuffle
// and the norm three or four.  A warp works on one row at a time (four heads
// at d = 128), takes the row's sines and cosines once, shared through shared
// memory, and loads ROPE_UNROLL heads a lane group ahead of their arithmetic.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "qk_rope.h"
#include "vec.cuh"

namespace tpmlp {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
#ifndef P_RU
#define P_RU 2
#define P_RB 3
#define P_BU 2
#define P_BB 2
#endif
constexpr int ROPE_UNROLL = P_RU;   // heads a lane group has in flight
constexpr int ROWS_BLOCKS = P_RB;
constexpr int BWD_UNROLL = P_BU;
constexpr int BWD_BLOCKS = P_BB;

// 8 consecutive elements as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void get(float* f) const { Vec<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(&v), f); }
  __device__ void set(const float* f) { Vec<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(&v), f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// E4M3 code of v: round to nearest even, saturated to +-448 (NaN stays NaN).
__device__ __forceinline__ uint2 e4m3x8(const float* f) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

// Lanes of a head, and where a lane's two chunks of 8 lie.
template <int D>
struct HeadLanes {
  static constexpr int UNITS = D / 16;                       // lanes with work: 4, 8, 12, 16
  static constexpr int LANES = UNITS == 12 ? 16 : UNITS;     // lanes a head takes
  static constexpr int GROUPS = 32 / LANES;                  // heads a warp works on at once
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  static __device__ __forceinline__ void sum2(float& v, float& y) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
  }
};

// The two chunks of unit u: partners 8u + i and rot/2 + 8u + i for pairs
// (j, j + rot/2), or 16 neighbouring values; either way the unit's pairs have
// the frequencies 8u .. 8u + 7.
__device__ __forceinline__ void unit_offsets(int u, int rot, bool interleaved, int& a, int& b) {
  const bool half = !interleaved && u < rot / 16;
  a = half ? 8 * u : 16 * u;
  b = half ? rot / 2 + 8 * u : 16 * u + 8;
}

// Rotates a lane's 16 values by the unit's eight angles (sn = -sin for the inverse).
__device__ __forceinline__ void rotate16(float* a, float* b, const float* cs, const float* sn, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = a0 * cs[i] - a1 * sn[i];
      a[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
      b[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
      b[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i] - y * sn[i];
      b[i] = y * cs[i] + x * sn[i];
    }
  }
}

// Cosine and sine of position * turn: one frequency a lane, left in shared memory.
template <int D>
__device__ __forceinline__ void row_angles(const uint64_t* turn, int nfreq, int pos, float2* cs_warp) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the previous row's readers are done
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const int f = lane + 32 * k;
    if (f < nfreq) {
      const uint64_t ph = turn[k] * (uint64_t)(int64_t)pos;  // turns mod 1
      float s, c;
      sincospif((float)(int32_t)(uint32_t)(ph >> 32) * 0x1p-31f, &s, &c);
      cs_warp[f] = make_float2(c, s);
    }
  }
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void load_turns(const RopeFreqs& fr, uint64_t* turn) {
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const int f = (threadIdx.x & 31) + 32 * k;
    turn[k] = f < fr.rot / 2 ? fr.turn[f] : 0;
  }
}

// Eight angles of unit u (identity where the unit lies behind the rotated part).
__device__ __forceinline__ void unit_angles(const float2* cs_warp, int u, int rot, float sign, float* cs, float* sn) {
  if (u < rot / 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(cs_warp)[4 * u + i];
      cs[2 * i] = t.x;
      sn[2 * i] = sign * t.y;
      cs[2 * i + 1] = t.z;
      sn[2 * i + 1] = sign * t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
    }
  }
}

// The sequence whose rows [cu[b], cu[b+1]) hold row r, by 32-way search; -1 if none.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool below = i < n && cu[lo + i] <= r;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int cnt = m == 0xffffffffu ? 32 : __ffs(~m) - 1;  // leading true answers
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  return cu[lo] <= r && r < cu[lo + 1] ? lo : -1;
}

// An append row's position, and where its key and value go in the cache
// (elements; negative: nowhere).
__device__ __forceinline__ int append_place(const RopeArgs& a, int64_t row, int64_t& slot_off) {
  slot_off = -1;
  int b, at;
  if (a.cu_rows) {
    b = find_sequence(a.cu_rows, a.batch, (int)row);
    if (b < 0) return 0;
    at = (int)row - a.cu_rows[b];
  } else {
    b = (int)row / a.rows_per_seq;
    at = (int)row - b * a.rows_per_seq;
    if (a.new_lens && at >= a.new_lens[b]) return 0;
  }
  const int past = a.past_lens[b];
  if (past < 0) return 0;  // an inactive sequence
  const uint32_t p = (uint32_t)past + (uint32_t)at;
  const uint32_t pi = p / (uint32_t)a.page_size;
  int page = -1;
  if (pi < (uint32_t)a.max_pages) page = a.table[(int64_t)b * a.ld_table + pi];
  if (page < 0 || page >= a.num_pages) {  // nowhere to store: reported, not written
    if ((threadIdx.x & 31) == 0) atomicOr(a.status, STATUS_BAD_INDEX);
    return 0;
  }
  slot_off = (int64_t)page * a.stride_page + (int64_t)(p - pi * a.page_size) * a.stride_slot;
  return (int)p;
}

// KIND 0: rows to rows (RopeArgs); 1, 2: append to a bf16 or E4M3 cache.
template <typename T, int D, int KIND>
__global__ void __launch_bounds__(THREADS, ROWS_BLOCKS) rope_rows_kernel(const __grid_constant__ RopeArgs a,
                                                            const __grid_constant__ RopeFreqs fr) {
  using HL = HeadLanes<D>;
  __shared__ __align__(16) float2 s_cs[WARPS][ROPE_MAX_PAIRS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % HL::LANES, group = lane / HL::LANES;
  const bool active = u < HL::UNITS;
  const bool il = fr.interleaved != 0, norm = a.q_norm_w != nullptr || a.k_norm_w != nullptr;
  const int rot = fr.rot;
  int oa, ob;
  unit_offsets(active ? u : 0, rot, il, oa, ob);
  uint64_t turn[D / 64];
  load_turns<D>(fr, turn);
  const int h_end = a.nq + a.nkv + (KIND ? a.nkv : 0);
  const int h_begin = KIND && !a.out ? a.nq : 0;  // an append without a query output skips the queries
  const int64_t items = a.rows * a.splits, stride = (int64_t)gridDim.x * WARPS;
  for (int64_t it = (int64_t)blockIdx.x * WARPS + warp; it < items; it += stride) {
    const int64_t row = it / a.splits;
    const int split = (int)(it - row * a.splits);
    const T* in = static_cast<const T*>(a.in) + row * a.ld_in;
    const int hstep = a.splits * HL::GROUPS;
    float cs[8], sn[8];
    int64_t slot_off = 0;
    bool placed = false;
    for (int h0 = h_begin + split * HL::GROUPS + group; h0 - group < h_end; h0 += ROPE_UNROLL * hstep) {
      Raw8<T> xa[ROPE_UNROLL], xb[ROPE_UNROLL];
#pragma unroll
      for (int k = 0; k < ROPE_UNROLL; ++k) {
        const int h = h0 + k * hstep;
        if (active && h < h_end) {
          xa[k].load(in + (int64_t)h * D + oa);
          xb[k].load(in + (int64_t)h * D + ob);
        } else {
          const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          xa[k].set(z);
          xb[k].set(z);
        }
      }
      if (!placed) {  // behind the first loads, which do not wait for it
        const int pos = KIND ? append_place(a, row, slot_off) : a.pos ? a.pos[row] : (int)(a.seq > 0 ? row % a.seq : row);
        if (KIND && slot_off < 0) break;
        if (rot) row_angles<D>(turn, rot / 2, pos, s_cs[warp]);
        unit_angles(s_cs[warp], u, rot, 1.0f, cs, sn);
        placed = true;
      }
#pragma unroll
      for (int k = 0; k < ROPE_UNROLL; ++k) {
        const int h = h0 + k * hstep;
        if (h - group >= h_end) break;  // the same for the whole warp
        const bool is_q = h < a.nq, is_v = KIND && h >= a.nq + a.nkv;
        float fa[8], fb[8];
        xa[k].get(fa);
        xb[k].get(fb);
        if (norm) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], ss));
          ss = HL::sum(ss);
          const T* w = static_cast<const T*>(is_q ? a.q_norm_w : a.k_norm_w);
          if (active && h < h_end && !is_v && w) {
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
            Raw8<T> wr;
            float wf[8];
            wr.load(w + oa);
            wr.get(wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) fa[i] *= r * wf[i];
            wr.load(w + ob);
            wr.get(wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) fb[i] *= r * wf[i];
          }
        }
        if (!active || h >= h_end) continue;
        if (!is_v) rotate16(fa, fb, cs, sn, il);
        if (KIND == 0 || is_q) {
          if (KIND == 0 && a.save) {  // the values before the norm, for the backward pass
            T* sv = static_cast<T*>(a.save) + row * a.ld_save + (int64_t)h * D;
            xa[k].store(sv + oa);
            xb[k].store(sv + ob);
          }
          T* out = static_cast<T*>(a.out) + row * a.ld_out + (int64_t)h * D;
          xa[k].set(fa);
          xb[k].set(fb);
          xa[k].store(out + oa);
          xb[k].store(out + ob);
        } else {
          const int g = is_v ? h - a.nq - a.nkv : h - a.nq;
          const int64_t off = slot_off + g * a.stride_head;
          if (KIND == 1) {
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + off;
            Raw8<__nv_bfloat16> t;
            t.set(fa);
            t.store(c + oa);
            t.set(fb);
            t.store(c + ob);
          } else {
            uint8_t* c = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + off;
            const float* isc = is_v ? a.v_inv_scale : a.k_inv_scale;
            const float sc = isc ? isc[g] : 1.0f;
            if (isc) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                fa[i] = __fdiv_rn(fa[i], sc);
                fb[i] = __fdiv_rn(fb[i], sc);
              }
            }
            *reinterpret_cast<uint2*>(c + oa) = e4m3x8(fa);
            *reinterpret_cast<uint2*>(c + ob) = e4m3x8(fb);
          }
        }
      }
    }
  }
}

// Backward.  All rows' query heads are taken first, then their key heads, so
// that a lane holds its 16 columns of one weight gradient at a time in registers; blocks leave their sums as partials, added in a fixed order by
// rope_dw_kernel, so the gradients are the same every run.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS) rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a,
                                                           const __grid_constant__ RopeFreqs fr) {
  using HL = HeadLanes<D>;
  constexpr int UN = BWD_UNROLL;
  __shared__ __align__(16) float2 s_cs[WARPS][ROPE_MAX_PAIRS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % HL::LANES, group = lane / HL::LANES;
  const bool active = u < HL::UNITS;
  const bool il = fr.interleaved != 0;
  const int rot = fr.rot;
  int oa, ob;
  unit_offsets(active ? u : 0, rot, il, oa, ob);
  uint64_t turn[D / 64];
  load_turns<D>(fr, turn);
  __shared__ float s_dw[WARPS][2][D];
  const int64_t items = a.rows * a.splits, stride = (int64_t)gridDim.x * WARPS;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int h_begin = part ? a.nq : 0, h_end = part ? a.nq + a.nkv : a.nq;
    const T* w = static_cast<const T*>(part ? a.k_norm_w : a.q_norm_w);
    const int hstep = a.splits * HL::GROUPS;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int64_t it = (int64_t)blockIdx.x * WARPS + warp; it < items; it += stride) {
      const int64_t row = it / a.splits;
      const int split = (int)(it - row * a.splits);
      float cs[8], sn[8];
      bool placed = false;
      for (int h0 = h_begin + split * HL::GROUPS + group; h0 - group < h_end; h0 += UN * hstep) {
        Raw8<T> ga[UN], gb[UN], xa[UN], xb[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int h = h0 + k * hstep;
          const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          ga[k].set(z);
          gb[k].set(z);
          xa[k].set(z);
          xb[k].set(z);
          if (active && h < h_end) {
            const T* g = static_cast<const T*>(a.dout) + row * a.ld_dout + (int64_t)h * D;
            ga[k].load(g + oa);
            gb[k].load(g + ob);
            if (w) {
              const T* x = static_cast<const T*>(a.x) + row * a.ld_x + (int64_t)h * D;
              xa[k].load(x + oa);
              xb[k].load(x + ob);
            }
          }
        }
        if (!placed) {  // behind the first loads, which do not wait for it
          const int pos = a.pos ? a.pos[row] : (int)(a.seq > 0 ? row % a.seq : row);
          if (rot) row_angles<D>(turn, rot / 2, pos, s_cs[warp]);
          unit_angles(s_cs[warp], u, rot, -1.0f, cs, sn);
          placed = true;
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int h = h0 + k * hstep;
          if (h - group >= h_end) break;  // the same for the whole warp
          float fa[8], fb[8];
          ga[k].get(fa);
          gb[k].get(fb);
          rotate16(fa, fb, cs, sn, il);
          if (w) {
            float va[8], vb[8];
            xa[k].get(va);
            xb[k].get(vb);
            float wa[8], wb[8];
            Raw8<T> wr;
            wr.load(w + oa);
            wr.get(wa);
            wr.load(w + ob);
            wr.get(wb);
            // both sums at once: sum x^2 and sum w g x = mean(w g xh) d / r
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
              dot = fmaf(wa[i] * fa[i], va[i], fmaf(wb[i] * fb[i], vb[i], dot));
            }
            HL::sum2(ss, dot);
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
            const float c = dot * (1.0f / D) * r * r * r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i] = fmaf(fa[i], va[i] * r, acc[i]);
              acc[8 + i] = fmaf(fb[i], vb[i] * r, acc[8 + i]);
              fa[i] = fmaf(r * wa[i], fa[i], -c * va[i]);
              fb[i] = fmaf(r * wb[i], fb[i], -c * vb[i]);
            }
          }
          if (!active || h >= h_end) continue;
          T* dx = static_cast<T*>(a.dx) + row * a.ld_dx + (int64_t)h * D;
          ga[k].set(fa);
          gb[k].set(fb);
          ga[k].store(dx + oa);
          gb[k].store(dx + ob);
        }
      }
    }
    // lanes of the same unit
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = HL::LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (active && group == 0) s_dw[warp][part][(i < 8 ? oa : ob - 8) + i] = v;
    }
  }
  if (!a.part) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += THREADS) {  // the warps of the block in order
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += (&s_dw[k][0][0])[c];
    a.part[(int64_t)blockIdx.x * 2 * D + c] = v;
  }
}

// dw[c] = sum over blocks of part[block][c]: 32 columns a block, 32 rows of threads.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, int nparts, int d,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;  // d is a multiple of 32
  float v = 0.0f;
  for (int p = threadIdx.y; p < nparts; p += 32) v += part[(int64_t)p * 2 * d + c];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x == 0) {
    const int cc = blockIdx.x * 32 + threadIdx.y;
    float* dst = cc < d ? dq_w : dk_w;
    if (dst) dst[cc < d ? cc : cc - d] = v;
  }
}

// Warps a row's heads are split over: one once the rows alone fill the machine
// (32 warps an SM), as many as there are head groups for a single row.
int head_splits(int64_t rows, int heads, int groups, int num_sms) {
  const int64_t want = (32LL * num_sms + rows - 1) / rows;
  const int most = (heads + groups - 1) / groups;
  return (int)(want < 1 ? 1 : want > most ? most : want);
}

template <int KIND, typename T>
cudaError_t launch_rows(RopeArgs a, const RopeFreqs& fr, int d, int num_sms, cudaStream_t st) {
  const int heads = (KIND && !a.out ? 0 : a.nq) + a.nkv + (KIND ? a.nkv : 0);
  const int groups = d == 64 ? 8 : d == 128 ? 4 : 2;
  a.splits = head_splits(a.rows, heads, groups, num_sms);
  const int64_t items = a.rows * a.splits;
  int64_t blocks = (items + WARPS - 1) / WARPS;
  if (blocks > 16LL * num_sms) blocks = 16LL * num_sms;
  switch (d) {
    case 64: rope_rows_kernel<T, 64, KIND><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 128: rope_rows_kernel<T, 128, KIND><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 192: rope_rows_kernel<T, 192, KIND><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 256: rope_rows_kernel<T, 256, KIND><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(RopeBwdArgs a, const RopeFreqs& fr, int d, int num_sms, cudaStream_t st, int* blocks_out) {
  const int groups = d == 64 ? 8 : d == 128 ? 4 : 2;
  a.splits = head_splits(a.rows, a.nq + a.nkv, groups, num_sms);
  const int64_t items = a.rows * a.splits;
  int64_t blocks = (items + WARPS - 1) / WARPS;
  if (blocks > 4LL * num_sms) blocks = 4LL * num_sms;
  if (blocks > ROPE_MAX_PARTS) blocks = ROPE_MAX_PARTS;
  *blocks_out = (int)blocks;
  switch (d) {
    case 64: rope_bwd_kernel<T, 64><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 128: rope_bwd_kernel<T, 128><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 192: rope_bwd_kernel<T, 192><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    case 256: rope_bwd_kernel<T, 256><<<(unsigned)blocks, THREADS, 0, st>>>(a, fr); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_rope(int dtype, int d, const RopeArgs& a, const RopeFreqs& fr, int num_sms, cudaStream_t st) {
  if (a.rows <= 0 || a.nq + a.nkv <= 0) return cudaSuccess;
  return dtype == 0 ? launch_rows<0, float>(a, fr, d, num_sms, st)
                    : launch_rows<0, __nv_bfloat16>(a, fr, d, num_sms, st);
}

cudaError_t launch_kv_append(bool e4m3, int d, const RopeArgs& a, const RopeFreqs& fr, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  return e4m3 ? launch_rows<2, __nv_bfloat16>(a, fr, d, num_sms, st)
              : launch_rows<1, __nv_bfloat16>(a, fr, d, num_sms, st);
}

cudaError_t launch_qk_rope_bwd(int dtype, int d, const RopeBwdArgs& a, const RopeFreqs& fr, int num_sms,
                               cudaStream_t st, float* dq_w, float* dk_w) {
  const bool dw = a.part && (dq_w || dk_w);
  if (a.rows <= 0 || a.nq + a.nkv <= 0) {
    cudaError_t e = cudaSuccess;
    for (float* p : {dq_w, dk_w})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, d * sizeof(float), st);
    return e;
  }
  int nparts = 0;
  cudaError_t e = dtype == 0 ? launch_bwd<float>(a, fr, d, num_sms, st, &nparts)
                             : launch_bwd<__nv_bfloat16>(a, fr, d, num_sms, st, &nparts);
  if (e != cudaSuccess || !dw) return e;
  rope_dw_kernel<<<2 * d / 32, dim3(32, 32), 0, st>>>(a.part, nparts, d, dq_w, dk_w);
  return cudaGetLastError();
}

}  // namespace tpmlp
