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
// What bounds it: forward and append of many 16-bit rows, memory, with the
// instruction rate close behind (512 values leave an SM about 90 cycles of its
// share of the copy rate).  The backward, neither bytes nor issue slots (60% of
// them active, 65% forward): each step is one chain of two sums of 16 values,
// shuffles, rsqrt and products, with four warps a scheduler to hide it.  f32
// rows lose more: a lane's 8 values are two 16-byte pieces, so each of a warp's
// accesses has gaps of 16 bytes: 2.1 times the L2 sectors that the rows have,
// three times the requests, 22% of the issue slots active.  A warp never
// works on two rows at once, so rows of fewer heads than it takes in a step
// leave lanes idle and pay the row's angles and addresses all the same.
// A head belongs to d / 16 lanes; a lane holds two 16-byte (bf16) chunks whose
// values are each other's rotation partners, so the rotation needs no shuffle
// and the norm three or four.  A warp walks rows, four heads at a time at
// d = 128, and takes a row's sines, cosines and addresses once.  Loads run
// several steps ahead, across rows, through a queue in shared memory
// (cp.async): each lane reads back only what it copied itself, so nothing but
// its own copies is waited for, and no registers are held by loads in flight.
//
// Measured on a GB300 (copy rate 6.68 TB/s), bf16, 32 + 8 heads of 128, norms:
// forward of 32768 rows 106 us, 6.4 TB/s; append of 16000 rows with 8 value
// heads 68 us, 5.8 TB/s (E4M3 cache: 79 us, 4.6 TB/s, with 16 divisions a lane
// and step); backward of 8192 rows 52 us, 4.8 TB/s (heads of 256, half
// rotated: 5.6 TB/s; 16 + 4 of them, all rotated: 4.9 TB/s).  f32, 4096 rows of
// 32 + 8 heads of 128: 41 us, 4.1 TB/s; backward 72 us, 3.5 TB/s.  8 + 1 heads
// of 128, bf16: 3.2 TB/s forward, 3.0 backward; 1 + 1 of 64: 0.8 and 0.5.  With
// the loads in registers instead of the queue the first three took 115, 78 and
// 58 us.
//
// Rounding.  Everything between a load and a store is f32.  The weight
// gradients are f32 sums: a lane's rows one after the other, then lanes, warps
// and blocks as trees or in order; an f64 addition a value would go through a
// slow pipe.  333 f32 rows: dx and the weight gradients together 1.3e-7 off the
// definition in 64 bits, 8e-8 for f32 arithmetic with the sums in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "allow_smem.h"
#include "qk_rope.h"
#include "vec.cuh"

namespace tpmlp {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// Steps that a lane's loads run ahead, and blocks of an SM: what fits shared
// memory (64 KB of queue a block forward, 96 KB backward) and the registers.
template <typename T>
struct Ahead {
  static constexpr int CHUNK = 8 * sizeof(T) / 16;              // 16-byte pieces of 8 values
  static constexpr int ROWS = sizeof(T) == 2 ? 8 : 4;           // forward and append: 2 chunks a step
  // backward: 4 chunks a step; heads of 256 values leave room for one step less
  static constexpr __host__ __device__ int bwd(int d) { return (sizeof(T) == 2 ? 6 : 3) - (d == 256 ? 1 : 0); }
};
// (rows to rows: two blocks, which may take 128 registers a thread and take 93
// to 102, are 8% faster than three of 80; the append is 2% slower with two: it
// has more latency to hide behind other warps)
constexpr int ROWS_BLOCKS[3] = {2, 3, 3}, BWD_BLOCKS = 2;

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t smem) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem)
               : "memory");
  return v;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 consecutive elements as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void get(float* f) const { Vec<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(&v), f); }
  __device__ void set(const float* f) { Vec<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(&v), f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
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

// A lane's queue slot (a shared-memory address): chunk c of a step lies 32
// lanes x 16 bytes behind the one before it, so a warp's accesses are
// contiguous.
template <typename T>
__device__ __forceinline__ void queue_load(uint32_t slot, int c, const T* g) {
#pragma unroll
  for (int i = 0; i < Ahead<T>::CHUNK; ++i)
    cp_async16(slot + (c * Ahead<T>::CHUNK + i) * 512, reinterpret_cast<const uint4*>(g) + i);
}
__device__ __forceinline__ void queue_get(uint32_t slot, int c, Raw8<__nv_bfloat16>& r) { r.v = lds16(slot + c * 512); }
__device__ __forceinline__ void queue_get(uint32_t slot, int c, Raw8<float>& r) {
  const uint4 x = lds16(slot + 2 * c * 512), y = lds16(slot + (2 * c + 1) * 512);
  r.a = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
  r.b = make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
}

// A warp's items are (row, share of its heads).  `left` steps remain of the
// current row, `h` is this lane's head: all row arithmetic happens once a row.
struct Walk {
  int64_t it, row;
  int left, h;
};
struct Items {
  int64_t count, stride;
  int splits, begin, end, step, groups, group;
  // Moves `w` to its item w.it or the first behind it that has heads; false at the end.
  __device__ __forceinline__ bool enter(Walk& w) const {
    for (; w.it < count; w.it += stride) {
      w.row = splits == 1 ? w.it : w.it / splits;
      const int h = begin + (splits == 1 ? 0 : (int)(w.it - w.row * splits) * groups);
      if (h < end) {
        w.left = (end - h + step - 1) / step;
        w.h = h + group;
        return true;
      }
    }
    w.left = 0;
    return false;
  }
};

// The norm weights of queries and keys as floats in shared memory.
template <typename T, int D>
__device__ __forceinline__ void stage_weights(float (&s_w)[2][D], const void* qw, const void* kw) {
  for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
    const T* w = static_cast<const T*>(i < D ? qw : kw);
    (&s_w[0][0])[i] = w ? (float)w[i < D ? i : i - D] : 1.0f;
  }
  __syncthreads();
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  Vec<float>::load(p, f);
  Vec<float>::load(p + 4, f + 4);
}

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

// The two chunks of unit u of a head of d values: the halves of the rotated
// part, or of what lies behind it, 8 values a unit, so that a warp's accesses
// are contiguous.  With pairs (j, j + rot/2) they are each other's partners,
// with neighbouring pairs each chunk holds four pairs.
__device__ __forceinline__ void unit_offsets(int u, int d, int rot, int& a, int& b) {
  const int v = u - rot / 16;
  a = v < 0 ? 8 * u : rot + 8 * v;
  b = v < 0 ? rot / 2 + 8 * u : (rot + d) / 2 + 8 * v;
}

// Rotates a lane's 16 values by its eight angles (sn = -sin for the inverse).
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

// The eight angles of unit u, which turns: of its partners, or four of the
// neighbours of each chunk; sign -1 for the inverse rotation.
__device__ __forceinline__ void unit_angles(const float2* cs_warp, int u, int rot, bool il, float sign, float* cs,
                                            float* sn) {
  const float2* at[2] = {cs_warp + (il ? 4 * u : 8 * u), cs_warp + (il ? rot / 4 + 4 * u : 8 * u + 4)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = *reinterpret_cast<const float4*>(at[i / 2] + 2 * (i % 2));
    cs[2 * i] = t.x;
    sn[2 * i] = sign * t.y;
    cs[2 * i + 1] = t.z;
    sn[2 * i + 1] = sign * t.w;
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
  const int past = a.past_lens ? a.past_lens[b] : 0;
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
__global__ void __launch_bounds__(THREADS, ROWS_BLOCKS[KIND]) rope_rows_kernel(const __grid_constant__ RopeArgs a,
                                                                         const __grid_constant__ RopeFreqs fr) {
  using HL = HeadLanes<D>;
  constexpr int S = Ahead<T>::ROWS, STEP = 2 * Ahead<T>::CHUNK * 512;  // bytes of a warp's step
  extern __shared__ __align__(16) uint4 s_queue[];
  __shared__ __align__(16) float2 s_cs[WARPS][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % HL::LANES, group = lane / HL::LANES;
  const bool active = u < HL::UNITS;
  const bool il = fr.interleaved != 0, norm = a.q_norm_w != nullptr || a.k_norm_w != nullptr;
  const int rot = fr.rot;
  int oa, ob;
  unit_offsets(active ? u : 0, D, rot, oa, ob);
  // Values behind the rotated part pass, whatever lies beside them; `whole`
  // spares the warp the question where there are none (6% of the forward).
  const bool whole = HL::UNITS == HL::LANES && rot == D;
  const bool turns = u < rot / 16;
  uint64_t turn[D / 64];
  load_turns<D>(fr, turn);
  const uint32_t queue = (uint32_t)__cvta_generic_to_shared(s_queue) + warp * S * STEP + lane * 16;
  __shared__ __align__(16) float s_w[2][D];

  Items items;
  items.count = a.rows * a.splits;
  items.stride = (int64_t)gridDim.x * WARPS;
  items.splits = a.splits;
  items.begin = KIND && !a.out ? a.nq : 0;  // an append without a query output skips the queries
  items.end = a.nq + a.nkv + (KIND ? a.nkv : 0);
  items.groups = HL::GROUPS;
  items.group = group;
  items.step = a.splits * HL::GROUPS;
  const int end = active ? items.end : 0;  // lanes without a unit never have work
  Walk ld, st;
  ld.it = (int64_t)blockIdx.x * WARPS + warp;
  bool more = items.enter(ld);
  st = ld;
  const T* src = static_cast<const T*>(a.in) + ld.row * a.ld_in;
  auto load = [&](uint32_t slot) {
    if (ld.left > 0) {
      if (ld.h < end) {
        queue_load<T>(slot, 0, src + (ld.h * D + oa));
        queue_load<T>(slot, 1, src + (ld.h * D + ob));
      }
      ld.h += items.step;
      if (--ld.left == 0) {
        ld.it += items.stride;
        if (items.enter(ld)) src = static_cast<const T*>(a.in) + ld.row * a.ld_in;
      }
    }
    cp_commit();
  };
  if (more) {
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(queue + i * STEP);
  }
  if (norm) stage_weights<T, D>(s_w, a.q_norm_w, a.k_norm_w);  // behind the first loads
  uint32_t slot = queue, fill = queue + (S - 1) * STEP;
  float cs[8], sn[8];
  while (more) {
    // ---- a row
    int64_t slot_off = 0;
    const int pos =
        KIND ? append_place(a, st.row, slot_off) : a.pos ? a.pos[st.row] : (int)(a.seq > 0 ? st.row % a.seq : st.row);
    if (slot_off >= 0) {
      if (rot) row_angles<D>(turn, rot / 2, pos, s_cs[warp]);
      if (turns) unit_angles(s_cs[warp], u, rot, il, 1.0f, cs, sn);
    }
    T* const out = static_cast<T*>(a.out) + st.row * a.ld_out;
    for (; st.left > 0; --st.left, st.h += items.step) {
      load(fill);
      cp_wait<S - 1>();
      const uint32_t now = slot;
      fill = slot;
      slot = slot == queue + (S - 1) * STEP ? queue : slot + STEP;
      if (KIND && slot_off < 0) continue;  // a row that is nobody's
      const int h = st.h;
      const bool work = h < end;
      const bool is_q = h < a.nq, is_v = KIND && h >= a.nq + a.nkv;
      Raw8<T> xa, xb;
      float fa[8], fb[8];
      xa.zero();
      xb.zero();
      if (work) {
        queue_get(now, 0, xa);
        queue_get(now, 1, xb);
      }
      if (KIND == 0 && a.save && work) {  // the values before the norm, for the backward pass
        T* sv = static_cast<T*>(a.save) + st.row * a.ld_save + h * D;
        xa.store(sv + oa);
        xb.store(sv + ob);
      }
      xa.get(fa);
      xb.get(fb);
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(fa[i], fa[i], fmaf(fb[i], fb[i], ss));
        ss = HL::sum(ss);
        if (is_q ? a.q_norm_w != nullptr : !is_v && a.k_norm_w != nullptr) {
          const float r = rsqrtf(ss * (1.0f / D) + a.eps);
          float wf[8];
          load8(&s_w[is_q ? 0 : 1][oa], wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) fa[i] *= r * wf[i];
          load8(&s_w[is_q ? 0 : 1][ob], wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) fb[i] *= r * wf[i];
        }
      }
      if (!work) continue;
      if (!is_v && (whole || turns)) rotate16(fa, fb, cs, sn, il);
      if (KIND == 0 || is_q) {
        xa.set(fa);
        xb.set(fb);
        xa.store(out + (h * D + oa));
        xb.store(out + (h * D + ob));
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
          if (isc) {
            const float sc = isc[g];
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
    st.it += items.stride;
    more = items.enter(st);
  }
  cp_wait<0>();
}

// Backward.  All rows' query heads are taken first, then their key heads, so
// that a lane holds its 16 columns of one weight gradient at a time in
// registers (a row's angles are computed in both passes); blocks leave their
// sums as partials, added in a fixed order by rope_dw_kernel, so the gradients
// are the same every run.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS) rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a,
                                                                       const __grid_constant__ RopeFreqs fr) {
  using HL = HeadLanes<D>;
  constexpr int S = Ahead<T>::bwd(D), STEP = 4 * Ahead<T>::CHUNK * 512;
  extern __shared__ __align__(16) uint4 s_queue[];
  __shared__ __align__(16) float2 s_cs[WARPS][D / 2];
  __shared__ float s_dw[WARPS][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % HL::LANES, group = lane / HL::LANES;
  const bool active = u < HL::UNITS;
  const bool il = fr.interleaved != 0;
  const int rot = fr.rot;
  int oa, ob;
  unit_offsets(active ? u : 0, D, rot, oa, ob);
  // (as in the forward)
  const bool whole = HL::UNITS == HL::LANES && rot == D;
  const bool turns = u < rot / 16;
  uint64_t turn[D / 64];
  load_turns<D>(fr, turn);
  const uint32_t queue = (uint32_t)__cvta_generic_to_shared(s_queue) + warp * S * STEP + lane * 16;
  __shared__ __align__(16) float s_w[2][D];
  if (a.q_norm_w || a.k_norm_w) stage_weights<T, D>(s_w, a.q_norm_w, a.k_norm_w);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const T* w = static_cast<const T*>(part ? a.k_norm_w : a.q_norm_w);
    float acc[16], cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    Items items;
    items.count = a.rows * a.splits;
    items.stride = (int64_t)gridDim.x * WARPS;
    items.splits = a.splits;
    items.begin = part ? a.nq : 0;
    items.end = part ? a.nq + a.nkv : a.nq;
    items.groups = HL::GROUPS;
    items.group = group;
    items.step = a.splits * HL::GROUPS;
    const int end = active ? items.end : 0;  // lanes without a unit never have work
    Walk ld, st;
    ld.it = (int64_t)blockIdx.x * WARPS + warp;
    bool more = items.enter(ld);
    st = ld;
    const T *src = nullptr, *srx = nullptr;
    auto aim = [&] {
      src = static_cast<const T*>(a.dout) + ld.row * a.ld_dout;
      srx = static_cast<const T*>(a.x) + ld.row * a.ld_x;
    };
    auto load = [&](uint32_t slot) {
      if (ld.left > 0) {
        if (ld.h < end) {
          const int ha = ld.h * D + oa, hb = ld.h * D + ob;
          queue_load<T>(slot, 0, src + ha);
          queue_load<T>(slot, 1, src + hb);
          if (w) {
            queue_load<T>(slot, 2, srx + ha);
            queue_load<T>(slot, 3, srx + hb);
          }
        }
        ld.h += items.step;
        if (--ld.left == 0) {
          ld.it += items.stride;
          if (items.enter(ld)) aim();
        }
      }
      cp_commit();
    };
    if (more) {
      aim();
#pragma unroll
      for (int i = 0; i < S - 1; ++i) load(queue + i * STEP);
    }
    uint32_t slot = queue, fill = queue + (S - 1) * STEP;
    while (more) {
      // ---- a row
      const int pos = a.pos ? a.pos[st.row] : (int)(a.seq > 0 ? st.row % a.seq : st.row);
      if (rot) row_angles<D>(turn, rot / 2, pos, s_cs[warp]);
      if (turns) unit_angles(s_cs[warp], u, rot, il, -1.0f, cs, sn);
      T* const dx = static_cast<T*>(a.dx) + st.row * a.ld_dx;
      for (; st.left > 0; --st.left, st.h += items.step) {
        load(fill);
        cp_wait<S - 1>();
        const uint32_t q = slot;
        fill = slot;
        slot = slot == queue + (S - 1) * STEP ? queue : slot + STEP;
        const int h = st.h;
        const bool work = h < end;
        Raw8<T> ra, rb;
        float fa[8], fb[8];
        ra.zero();
        rb.zero();
        if (work) {
          queue_get(q, 0, ra);
          queue_get(q, 1, rb);
        }
        ra.get(fa);
        rb.get(fb);
        if (whole || turns) rotate16(fa, fb, cs, sn, il);
        if (w) {
          float va[8], vb[8], wa[8], wb[8];
          ra.zero();
          rb.zero();
          if (work) {
            queue_get(q, 2, ra);
            queue_get(q, 3, rb);
          }
          ra.get(va);
          rb.get(vb);
          load8(&s_w[part][oa], wa);
          load8(&s_w[part][ob], wb);
          // both sums at once: sum x^2 and sum w g x = mean(w g xh) d / r
          float ss = 0.0f, dot = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            wa[i] *= fa[i];  // w g
            wb[i] *= fb[i];
            ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
            dot = fmaf(wa[i], va[i], fmaf(wb[i], vb[i], dot));
          }
          HL::sum2(ss, dot);
          // (idle lanes hold zeros, whose rsqrt is infinite where eps is 0)
          const float r = work ? rsqrtf(ss * (1.0f / D) + a.eps) : 0.0f;
          const float c = -dot * (1.0f / D) * r * r;  // dx = r w g + c xh
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            va[i] *= r;  // xh
            vb[i] *= r;
            acc[i] = fmaf(fa[i], va[i], acc[i]);
            acc[8 + i] = fmaf(fb[i], vb[i], acc[8 + i]);
            fa[i] = fmaf(r, wa[i], c * va[i]);
            fb[i] = fmaf(r, wb[i], c * vb[i]);
          }
        }
        if (!work) continue;
        ra.set(fa);
        rb.set(fb);
        ra.store(dx + (h * D + oa));
        rb.store(dx + (h * D + ob));
      }
      st.it += items.stride;
      more = items.enter(st);
    }
    cp_wait<0>();
    if (!a.part) continue;
    // lanes of the same unit, then the warps of the block in order
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = HL::LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (active && group == 0) s_dw[warp][(i < 8 ? oa : ob - 8) + i] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THREADS) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) v += s_dw[k][c];
      a.part[((int64_t)blockIdx.x * 2 + part) * D + c] = v;
    }
  }
}

// dw[c] = sum over blocks of part[block][c]: 32 columns a block, 32 rows of
// threads.  A programmatic launch: it may start once the backward kernel's
// blocks have exited, before their writes are visible, and waits here for
// those (the backward triggers nothing earlier).
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int nparts, int d,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;  // d is a multiple of 32
  float v = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 8
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

template <typename T>
constexpr int ROWS_QUEUE = WARPS * Ahead<T>::ROWS * 2 * Ahead<T>::CHUNK * 32 * 16;
template <typename T, int D>
constexpr int BWD_QUEUE = WARPS * Ahead<T>::bwd(D) * 4 * Ahead<T>::CHUNK * 32 * 16;

template <auto K, typename A>
cudaError_t launch_kernel(int64_t blocks, int queue, cudaStream_t st, const A& a, const RopeFreqs& fr) {
  const cudaError_t e = allow_smem<K>(queue);
  if (e != cudaSuccess) return e;
  K<<<(unsigned)blocks, THREADS, queue, st>>>(a, fr);
  return cudaGetLastError();
}

template <int KIND, typename T>
cudaError_t launch_rows(RopeArgs a, const RopeFreqs& fr, int d, int num_sms, cudaStream_t st) {
  const int heads = (KIND && !a.out ? 0 : a.nq) + a.nkv + (KIND ? a.nkv : 0);
  const int groups = d == 64 ? 8 : d == 128 ? 4 : 2;
  a.splits = head_splits(a.rows, heads, groups, num_sms);
  const int64_t items = a.rows * a.splits;
  int64_t blocks = (items + WARPS - 1) / WARPS;
  if (blocks > (int64_t)ROWS_BLOCKS[KIND] * num_sms) blocks = (int64_t)ROWS_BLOCKS[KIND] * num_sms;  // one wave
  switch (d) {
    case 64: return launch_kernel<rope_rows_kernel<T, 64, KIND>>(blocks, ROWS_QUEUE<T>, st, a, fr);
    case 128: return launch_kernel<rope_rows_kernel<T, 128, KIND>>(blocks, ROWS_QUEUE<T>, st, a, fr);
    case 192: return launch_kernel<rope_rows_kernel<T, 192, KIND>>(blocks, ROWS_QUEUE<T>, st, a, fr);
    case 256: return launch_kernel<rope_rows_kernel<T, 256, KIND>>(blocks, ROWS_QUEUE<T>, st, a, fr);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t launch_bwd(RopeBwdArgs a, const RopeFreqs& fr, int d, int num_sms, cudaStream_t st, int* blocks_out) {
  const int groups = d == 64 ? 8 : d == 128 ? 4 : 2;
  a.splits = head_splits(a.rows, a.nq + a.nkv, groups, num_sms);
  const int64_t items = a.rows * a.splits;
  int64_t blocks = (items + WARPS - 1) / WARPS;
  if (blocks > (int64_t)BWD_BLOCKS * num_sms) blocks = (int64_t)BWD_BLOCKS * num_sms;  // one wave
  if (blocks > ROPE_MAX_PARTS) blocks = ROPE_MAX_PARTS;
  *blocks_out = (int)blocks;
  switch (d) {
    case 64: return launch_kernel<rope_bwd_kernel<T, 64>>(blocks, BWD_QUEUE<T, 64>, st, a, fr);
    case 128: return launch_kernel<rope_bwd_kernel<T, 128>>(blocks, BWD_QUEUE<T, 128>, st, a, fr);
    case 192: return launch_kernel<rope_bwd_kernel<T, 192>>(blocks, BWD_QUEUE<T, 192>, st, a, fr);
    case 256: return launch_kernel<rope_bwd_kernel<T, 256>>(blocks, BWD_QUEUE<T, 256>, st, a, fr);
    default: return cudaErrorInvalidValue;
  }
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * d / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_dw_kernel, static_cast<const float*>(a.part), nparts, d, dq_w, dk_w);
}

}  // namespace tpmlp
