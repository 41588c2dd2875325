// Attention of one new token per sequence over a paged key/value cache.
//
//   s_t = scale q . k_t over the visible tokens t < len (with a window: the
//   last `window` tokens and the first `sinks`),  out = softmax(s) V,
//   lse = log sum exp s.  No visible token: out 0, lse -inf.  Scores that are
//   all -inf: out NaN, as 0 / 0 has it, lse -inf.
//
// What bounds it: reading the cache once.  A key head's query heads are worked
// on together, so a cache byte meets at most 32 of them: some 32 flops a byte
// in bf16, far below what even the mma.sync tensor path gives, which is why
// the products use m16n8k16 with the keys (and for P V the head dimension) as
// M and 8 query heads as N.  tcgen05 with 128 keys as M would hand scores and P
// through TMEM and shared memory for 8 columns of work: nothing to gain at up to
// 8 query heads a key head, where the kernel runs at 89 to 98% of the copy rate
// (d = 128, long caches; heads of 192 and 256 values 81 and 86%, E4M3 of 256
// 63%).  It would pay beyond: with 16 query heads a key head this kernel is at
// 71% (E4M3 57%), with 32 at 41% (33%), as each group of 8 reads and converts
// the tile on warps of its own and its chain of products, softmax and products
// is longer.
//
// The split.  The cache is cut into tiles of 64 or 128 tokens; the tiles of
// every (sequence, key head) laid end to end are divided evenly over two CTAs
// an SM, whatever the lengths are.  They are read on the device: each CTA scans
// them once.  A CTA walks its range; where a (sequence, key head) lies inside
// it, its result is written, and where one is shared with other CTAs, each
// leaves an unnormalised partial (weighted values, maximum, sum) in the
// workspace and the last to arrive joins them: in groups of about sqrt(parts),
// then the groups, so one CTA never reads hundreds of partials.  Nobody waits
// for another CTA, and partials are added in the order of the tokens, so the
// result does not depend on which came last.
//
// The pipe.  One warp fetches tiles by TMA (one box a page and operand, the
// swizzle making ldmatrix conflict-free) into a ring of 96 KB a CTA, 192 KB in
// flight on an SM; it reads block-table entries a batch of boxes ahead.  Four
// warps compute, each on its share of a tile's tokens for 8 query heads.  Two
// warpgroups of 128 registers a thread are launched and the fetching one gives
// 72 of them up: with 168 for all, heads of 256 values spilled and took 1.2 to
// 1.9 times as long.  Tokens that a window or the length hides are cleared in
// shared memory, only in the tiles that have some: masking the fragments put
// branches between the products (7% at d = 128 with E4M3).
//
// Measured on a GB300 (copy rate 6.68 TB/s): 64 sequences of up to 8192 tokens,
// 8 key heads of 128, 32 query heads, bf16: 153 us, 6.5 TB/s; 128 such with
// E4M3: 166 us, 6.2 TB/s, where the conversions of codes to f16 (two for four
// codes) keep the ALU half busy; one of 131072 tokens: 86 us, 6.2 TB/s, of
// which the start and the two-level join are about 8 us.  Tiles of
// 64 tokens took 168 us on the first: a tile costs a warp two waits and a chain
// of dependent steps whatever its size.  Heads of 192 and 256 values keep 64,
// where a ring of 128 would hold three operands or fewer (5 to 10% slower).
//
// Rounding.  Scores, maxima, sums and outputs are f32.  With a bf16 cache P is
// the sum of two bf16 values (16 bits), because a single one would add as much
// error as the final rounding of the output; the second product costs about
// 1%.  With an E4M3 cache, codes are converted to f16 exactly, q is brought to
// f16 after a power-of-two scale per head, and P is f16: its 2^-11 a weight,
// random in sign and averaged over the tokens, stays below the output's 2^-8,
// and a second f16 product would double the tensor work of a kernel that the
// conversions already hold up.  Weights are taken relative to 2^-15 of the
// maximum, so that all of f16's range is theirs: 2^-29 of the largest keeps 11
// bits and 2^-39 is not 0 (relative to the maximum itself, weights below 2^-25
// were lost from the product but not from the sum; the time is the same).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "allow_smem.h"
#include "kv_decode.h"
#include "ptx_sm103.cuh"
#include "tma_maps.cuh"
#include "f32x2.cuh"

namespace tpmlp {
namespace {

constexpr int NCW = 4;           // computing warps
constexpr int NTHR = 256;        // a warpgroup that computes and one whose first warp fetches
// Registers a thread: 128 at launch (two CTAs an SM); the computing warpgroup
// takes what the other gives up, 200 + 56 = 2 x 128.
constexpr int COMPUTE_REGS = 200, FETCH_REGS = 56;
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 100000000ull;

// Shape of the kernel for heads of D values, F8: E4M3 cache, HG: groups of 8
// query heads.  A warp works on one head group and its share of a tile's
// tokens, so its registers do not grow with the heads; NCW / HG warps share a
// head group's tokens.
template <int D, bool F8, int HG>
struct Cfg {
  static constexpr int HT = 8 * HG;                        // query heads of a CTA
  static constexpr int RING_BYTES = 96 * 1024;             // two CTAs an SM
  static constexpr int ROW = D * (F8 ? 1 : 2);             // bytes of a token's key or value
  static constexpr int BLOCK = ROW % 128 == 0 ? 128 : 64;  // bytes of a row that lie together (the swizzle's width)
  static constexpr int TK = D <= 128 ? 128 : 64;           // tokens of a tile
  static constexpr int SLOT = TK * ROW;                    // one operand of a tile
  // Every computing warp works on every tile, so each waits for every use of a
  // slot: a barrier's one-bit phase is never asked about two rounds ahead.
  static constexpr int N = RING_BYTES / SLOT;
  // Two head groups on one warp, so that a fragment is read and converted once
  // for both, took 3 to 14% longer at 16 query heads: the chain of a tile
  // (products, softmax, products) is then twice as long on each warp.
  static constexpr int KG = NCW / HG;                      // warps that share a tile's tokens
  static constexpr int KW = TK / KG;                       // tokens of a tile that a warp works on
  static constexpr int OD = 64;                            // columns of O joined at a time
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c1, int c3,
                                            int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %3, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c3), "r"(c4)
      : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 tile of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t movm(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Four E4M3 codes as two pairs of f16: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ void f16_of_e4m3(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory"); }
// The same barrier; true for every thread if any thread says so.
__device__ __forceinline__ bool bar_compute_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(NCW * 32)
      : "memory");
  return r != 0;
}

// Visible tokens of a sequence, as ranges of tiles: [0, sink_tiles) and
// [win_tile, ...), tile j of the sequence's list being tile(j).
template <int TK>
struct Seq {
  int len;         // tokens attended
  int lo;          // first token of the window (0 without one)
  int sinks;
  int sink_tiles;  // tiles that hold sinks and end before the window's first tile
  int win_tile;
  int tiles;       // tiles in the list, at least 1
  __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + win_tile; }
  __device__ __forceinline__ bool whole(int t0) const {
    return t0 + TK <= len && (t0 >= lo || t0 + TK <= sinks);
  }
  __device__ __forceinline__ bool sees(int t) const { return t < len && (t >= lo || t < sinks); }
};
template <int TK>
__device__ __forceinline__ Seq<TK> make_seq(const DecodeArgs& a, int b, bool report) {
  Seq<TK> s;
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t n = (int64_t)a.lens[b] + a.len_add;
  if (n > cap) {
    if (report) atomicOr(a.status, STATUS_BAD_INDEX);
    n = cap;
  }
  s.len = n < 0 ? 0 : (int)n;
  s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.sinks = s.lo > 0 ? min(a.sinks, s.lo) : 0;
  s.win_tile = s.lo / TK;
  s.sink_tiles = min((s.sinks + TK - 1) / TK, s.win_tile);
  s.tiles = s.sink_tiles + (s.len + TK - 1) / TK - s.win_tile;
  if (s.tiles < 1) s.tiles = 1;
  return s;
}

// A worker's place in the list of all (sequence, key head chunk, tile).
template <int TK>
struct Cursor {
  int64_t pos, end, base;  // tile index, end of the worker's range, first tile of sequence b
  int b;
  Seq<TK> s;
};

// Joins the partial results of one (sequence, key head chunk) whose tiles
// several CTAs had; called by the computing warps of each of them with their
// partial written.
struct JoinArgs {
  float* part;
  uint32_t *ctr_first, *ctr_last;  // arrival counts of the groups and of their leaders
  __nv_bfloat16* out;
  float* lse;
  int w_first, nparts, p_me, heads;
  float vscale;
};
template <int D, int HT>
__device__ __forceinline__ void join_parts(const JoinArgs& a, volatile int* s_last) {
  const int tid = threadIdx.x;
  const size_t part_sz = (size_t)HT * (D + 2);
  // groups of about sqrt(parts), then the groups' leaders
  int group = a.nparts;
  if (a.nparts > 8)
    for (group = 3; group * group < a.nparts;) ++group;
  const int ngroups = (a.nparts + group - 1) / group;
  for (int level = 0; level < 2; ++level) {
    const int p0 = level == 0 ? a.p_me / group * group : 0;
    const int pstep = level == 0 ? 1 : group;
    const int cnt = level == 0 ? min(group, a.nparts - p0) : ngroups;
    uint32_t* ctr = level == 0 ? a.ctr_first + 2 * (a.w_first + p0) + (p0 == 0) : a.ctr_last + a.w_first;
    if (cnt > 1) {
      bar_compute();
      if (tid == 0) {
        // the fences order the whole CTA's partial before the count and the
        // others' partials behind it (the barriers carry them)
        __threadfence();
        const uint32_t old = atomicAdd(ctr, 1u);
        __threadfence();
        *s_last = old == (uint32_t)cnt - 1;
        if (old == (uint32_t)cnt - 1) *ctr = 0;  // ready for the next launch
      }
      bar_compute();
      if (!*s_last) return;
    }
    const bool final_level = ngroups == 1 || level == 1;
    if (!final_level && cnt == 1) continue;  // a group of one stands for itself
    auto part_of = [&](int i) -> float* {
      const int p = p0 + i * pstep;
      return a.part + (size_t)(2 * (a.w_first + p) + (p == 0)) * part_sz;
    };
    // Each thread joins float4 columns by itself: maxima, sums and values of
    // eight parts in flight at once, added in the parts' order.
    // A pass covers whole heads, so that none is read again once it is written.
    constexpr int PER = HT * D / 4 / (NCW * 32), V = D == 192 ? 3 : PER >= 2 ? 2 : 1;
    static_assert(PER % V == 0 && V * NCW * 128 % D == 0, "passes of whole heads");
    for (int x0 = tid; x0 < HT * D / 4; x0 += V * NCW * 32) {
      float4 v[V];
      float mx[V], sum[V];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        mx[q] = -INFINITY;
        sum[q] = 0.0f;
      }
      for (int i0 = 0; i0 < cnt; i0 += 8) {
        float4 y[8][V];
        float m[8][V], l[8][V];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* pp = part_of(i0 + i < cnt ? i0 + i : i0);
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const int x = x0 + q * NCW * 32, h = 4 * x / D;
            m[i][q] = __ldcg(pp + (size_t)HT * D + h);
            l[i][q] = __ldcg(pp + (size_t)HT * D + HT + h);
            y[i][q] = __ldcg(reinterpret_cast<const float4*>(pp) + x);
          }
        }
#pragma unroll
        for (int q = 0; q < V; ++q) {
          float top = mx[q];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + i < cnt) top = fmaxf(top, m[i][q]);
          const float base = top == -INFINITY ? 0.0f : top;  // nothing visible: all weights 0
          const float f = ex2_fast(mx[q] - base);
          mx[q] = top;
          sum[q] *= f;
          v[q] = make_float4(v[q].x * f, v[q].y * f, v[q].z * f, v[q].w * f);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i0 + i < cnt) {
              const float w = ex2_fast(m[i][q] - base);
              sum[q] = fmaf(w, l[i][q], sum[q]);
              v[q].x = fmaf(w, y[i][q].x, v[q].x);
              v[q].y = fmaf(w, y[i][q].y, v[q].y);
              v[q].z = fmaf(w, y[i][q].z, v[q].z);
              v[q].w = fmaf(w, y[i][q].w, v[q].w);
            }
        }
      }
      float* lead = part_of(0);
      if (!final_level) bar_compute();  // every thread has read the leader's partial
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int x = x0 + q * NCW * 32, h = 4 * x / D, col = 4 * x % D;
        const float s = sum[q];
        if (final_level) {
          // (a sequence without tokens is one tile and never comes here)
          const float r = s > 0.0f ? a.vscale / s : NAN;
          if (h < a.heads) {
            *reinterpret_cast<uint2*>(a.out + (int64_t)h * D + col) =
                make_uint2(pack_bf16(v[q].x * r, v[q].y * r), pack_bf16(v[q].z * r, v[q].w * r));
            if (a.lse && col == 0)
              a.lse[h] = s == 0.0f ? -INFINITY : (mx[q] + log2f(s)) * 0.69314718055994531f;
          }
        } else {
          __stcg(reinterpret_cast<float4*>(lead) + x, v[q]);
          if (col == 0) {
            __stcg(lead + (size_t)HT * D + h, mx[q]);
            __stcg(lead + (size_t)HT * D + HT + h, s);
          }
        }
      }
    }
    if (final_level) return;
  }
}

// The segment the computing warps are at, kept in shared memory by one of
// their threads so that it costs the main loop no registers.
template <int TK>
struct Walk {
  Cursor<TK> c;
  int64_t T, G;
  int hc, j;   // key head chunk; first tile in the sequence's list
  int ntiles;  // tiles of the segment, 0 behind the last one
  int direct;  // the segment is the whole (sequence, key head chunk)
  int64_t item0, item1;
  __device__ __forceinline__ void set() {
    if (c.pos >= c.end) {
      ntiles = 0;
      return;
    }
    item0 = c.base + (int64_t)hc * c.s.tiles;
    item1 = item0 + c.s.tiles;
    const int64_t seg_end = item1 < c.end ? item1 : c.end;
    ntiles = (int)(seg_end - c.pos);
    direct = c.pos == item0 && seg_end == item1;
  }
  __device__ __forceinline__ void next(const DecodeArgs& a, int nhc) {
    j += ntiles;
    c.pos += ntiles;
    if (c.pos < c.end && j == c.s.tiles) {
      j = 0;
      if (++hc == nhc) {
        hc = 0;
        c.base += (int64_t)c.s.tiles * nhc;
        c.s = make_seq<TK>(a, ++c.b, false);
      }
    }
    set();
  }
};

template <int D, bool F8, int HG>
__global__ void __launch_bounds__(NTHR, 2)
    kv_decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using R = Cfg<D, F8, HG>;
  constexpr int TK = R::TK, KW = R::KW, KG = R::KG, HT = R::HT, OD = R::OD;
  constexpr int KT = KW / 16;          // a warp's tokens of a tile as m-tiles
  constexpr int KS = D / 16;           // k-steps of Q K^T
  constexpr int MT = D / 16;           // m-tiles of V^T P^T
  constexpr int ROWB = R::BLOCK;       // bytes of a block's row
  constexpr int NBLK = R::ROW / ROWB;  // blocks of a row in shared memory
  extern __shared__ __align__(1024) uint8_t ring_raw[];
  __shared__ __align__(8) uint64_t full[R::N], empty[R::N];
  __shared__ int s_abort, s_b, s_last;
  __shared__ Walk<TK> s_walks[2];  // the segment at hand and the next one
  __shared__ int64_t s_scan[NTHR / 32], s_base;
  __shared__ float s_m[KG][HT], s_l[KG][HT];
  __shared__ float s_inv[HT];
  __shared__ __align__(16) float s_o[KG * HT * (OD + 4)];  // the warps' outputs of OD columns

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ring_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring_s = smem_u32(ring);
  volatile int* abort_flag = &s_abort;

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < R::N; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NCW);
    }
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  // ---- the worker's range: prefix sums of the sequences' tiles
  const int per = (a.batch + NTHR - 1) / NTHR;
  const int b_lo = min(tid * per, a.batch), b_hi = min(b_lo + per, a.batch);
  int64_t sum = 0;
  for (int b = b_lo; b < b_hi; ++b) sum += make_seq<TK>(a, b, blockIdx.x == 0).tiles;
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - sum;
#pragma unroll
  for (int w = 0; w < NTHR / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int nhc = a.nkv * a.chunks;
  const int64_t T = total * nhc;
  // Four tiles a worker where there are few, as fewer partial results are then
  // joined.  Measured in today's tiles with 1, 2, 4 and 8 tiles a worker: one
  // sequence of 500 tokens and 8 key heads of 128: 8.5, 9.3, 8.4, 8.5 us; of
  // 2000 tokens: 12.0, 9.4, 10.8, 14.6; 500 tokens, heads of 256: 10.3, 11.2,
  // 12.8, 12.2; batches that fill the machine do not care.  But as many workers
  // as there are key heads of sequences: 69 sequences of 16 tokens, 2 key heads:
  // 6.6 us, 13 without this.
  const int64_t want = max((T + 3) / 4, (int64_t)a.batch * nhc);
  const int64_t G = want < a.workers ? want : a.workers;
  if ((int64_t)blockIdx.x >= G) return;
  Cursor<TK> c;
  c.pos = (int64_t)blockIdx.x * T / G;
  c.end = ((int64_t)blockIdx.x + 1) * T / G;
  if (c.pos >= before * nhc && c.pos < (before + sum) * nhc) {
    int64_t base = before * nhc;
    int b = b_lo;
    for (;;) {
      const int64_t next = base + (int64_t)make_seq<TK>(a, b, false).tiles * nhc;
      if (c.pos < next) break;
      base = next;
      ++b;
    }
    s_b = b;
    s_base = base;
  }
  __syncthreads();
  c.b = s_b;
  c.base = s_base;
  c.s = make_seq<TK>(a, c.b, false);

  if (tid == 0) {
    const int64_t rel = c.pos - c.base;
    Walk<TK> w;
    w.c = c;
    w.T = T;
    w.G = G;
    w.hc = (int)(rel / c.s.tiles);
    w.j = (int)(rel - (int64_t)w.hc * c.s.tiles);
    w.set();
    s_walks[0] = w;
  }
  __syncthreads();

  if (warp >= NCW) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FETCH_REGS));
    if (warp > NCW) return;
    // A batch is up to 32 boxes of consecutive tiles of one (sequence, key
    // head), a lane each: the next batch's table entries are read while this
    // one's are fetched, so no tile waits for its page's number.
    const int nbox = TK / a.box_tokens, per_batch = 32 / nbox;
    const int my_tile = lane / nbox, my_box = lane % nbox;
    const int box_bytes = a.box_tokens * D * (F8 ? 1 : 2);
    int64_t rel = c.pos - c.base;
    int hc = (int)(rel / c.s.tiles), j = (int)(rel - (int64_t)hc * c.s.tiles);
    struct Batch {
      int count, head, page, slot;  // tiles, key head; this lane's page (-1: not needed) and first slot in it
    };
    auto next_batch = [&]() -> Batch {
      Batch r{0, 0, -1, 0};
      if (c.pos >= c.end) return r;
      r.count = (int)min((int64_t)min(per_batch, c.s.tiles - j), c.end - c.pos);
      r.head = hc / a.chunks;
      const int t = c.s.tile(j + my_tile) * TK + my_box * a.box_tokens;
      if (my_tile < r.count && t < c.s.len && (t + a.box_tokens > c.s.lo || t < c.s.sinks)) {
        const int pi = t / a.page_size;
        r.slot = t - pi * a.page_size;
        r.page = a.table[(int64_t)c.b * a.ld_table + pi];
        if (r.page < 0 || r.page >= a.num_pages) {
          atomicOr(a.status, STATUS_BAD_INDEX);
          r.page = 0;
        }
      }
      c.pos += r.count;
      j += r.count;
      if (c.pos < c.end && j == c.s.tiles) {
        j = 0;
        if (++hc == nhc) {
          hc = 0;
          c.base += (int64_t)c.s.tiles * nhc;
          c.s = make_seq<TK>(a, ++c.b, false);
        }
      }
      return r;
    };
    uint32_t n = 0;  // fetches issued: K and V of tile 0, 1, ...
    bool ok = true;
    Batch cur = next_batch();
    while (ok && cur.count > 0) {
      const Batch nxt = next_batch();
      const unsigned need = __ballot_sync(0xffffffffu, cur.page >= 0);
      for (int i = 0; ok && i < cur.count; ++i) {
        const unsigned mine = (need >> (i * nbox)) & (nbox == 32 ? 0xffffffffu : (1u << nbox) - 1);
        const uint32_t bytes = (uint32_t)__popc(mine) * box_bytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t sl = n % R::N, round = n / R::N;
          ok = round == 0 || mbar_wait(&empty[sl], (round - 1) & 1, abort_flag, a.status, STATUS_TIMEOUT, WAIT_NS);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[sl], bytes);
          __syncwarp();
          if (my_tile == i && cur.page >= 0)
            tma_load_5d(ring_s + sl * R::SLOT + my_box * box_bytes, kv ? &vmap : &kmap, &full[sl], cur.slot, cur.head,
                        cur.page);
          ++n;
        }
      }
      cur = nxt;
    }
    // the CTA does not end before its copies have landed, whatever the others did
    int no_abort = 0;
    for (uint32_t i = n > (uint32_t)R::N ? n - R::N : 0; i < n; ++i)
      mbar_wait(&full[i % R::N], (i / R::N) & 1, &no_abort, a.status, STATUS_TIMEOUT, DRAIN_NS);
    return;
  }

  // -------------------------------------------------------------- computing warps
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(COMPUTE_REGS));
  const int hgrp = warp % HG, kgrp = warp / HG;  // the warp's head group and token share
  const int g8 = lane >> 2, c4 = lane & 3;       // row group and column pair of the mma fragments
  // Shared-memory offsets of the lane's ldmatrix rows (token 16 y + key of the
  // warp's share) with the swizzled chunk of the first pair; chunk pair p of a
  // block is that offset xor 32 p, as rows and blocks are multiples of 64 bytes
  // and chunk numbers differ in their upper bits only.
  const int bt = a.box_tokens;
  const uint32_t blk = (uint32_t)bt * ROWB;  // bytes from one block to the next
  const int bt_log2 = __ffs(bt) - 1;
  auto row_base = [&](int key) -> uint32_t {
    return (uint32_t)(key >> bt_log2) * (blk * NBLK) + (key & (bt - 1)) * ROWB;
  };
  const int k_key = lane & 15;  // K: matrices (keys 0-7, 8-15) x 2 chunks
  // V: the same with E4M3; bf16 (2 chunks) x (keys 0-7, 8-15)
  const int v_key = F8 ? k_key : (lane & 7) + ((lane >> 4) << 3);
  const uint32_t k_ch = (lane >> 4) ^ (ROWB == 64 ? (k_key >> 1) & 3 : k_key & 7);
  const uint32_t v_ch = (F8 ? lane >> 4 : (lane >> 3) & 1) ^ (ROWB == 64 ? (v_key >> 1) & 3 : v_key & 7);
  uint32_t k_off[KT], v_off[KT];
#pragma unroll
  for (int y = 0; y < KT; ++y) {
    k_off[y] = row_base(kgrp * KW + 16 * y + k_key) + (k_ch << 4);
    v_off[y] = row_base(kgrp * KW + 16 * y + v_key) + (v_ch << 4);
  }
  constexpr int PPB = ROWB / 32;  // chunk pairs of a block's row

  uint32_t nu = 0;  // ring uses so far
  bool ok = true;

  // A segment's queries as they are in memory, fetched before the join of the
  // segment in front of it (heads of up to 128 values: more would not fit the
  // registers).
  constexpr bool EARLY = D <= 128;
  uint32_t qr[KS][2];
  float kinv = 1.0f, vscale = 1.0f;  // E4M3: what the head's codes stand for
  auto fetch_q = [&](const Walk<TK>& w) {
    const int g = w.hc / a.chunks, h0 = (w.hc - g * a.chunks) * HT, heads = min(HT, a.hpg - h0);
    const int h = hgrp * 8 + g8;
    const __nv_bfloat16* q =
        static_cast<const __nv_bfloat16*>(a.q) + (int64_t)w.c.b * a.ld_q + (int64_t)(g * a.hpg + h0 + h) * D;
    if (F8 && a.k_inv_scale) kinv = a.k_inv_scale[g];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qr[k][0] = qr[k][1] = 0;
      if (h < heads) {
        if (F8) {
          const uint2 v = *reinterpret_cast<const uint2*>(q + 16 * k + 4 * c4);
          qr[k][0] = v.x;
          qr[k][1] = v.y;
        } else {
          qr[k][0] = *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c4);
          qr[k][1] = *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 + 2 * c4);
        }
      }
    }
  };
  int cur = 0;
  if (EARLY) fetch_q(s_walks[0]);

  for (;; cur ^= 1) {
    // ---- one segment: the worker's tiles of (sequence b, key head g, chunk)
    const Walk<TK>& s_walk = s_walks[cur];
    const int ntiles = s_walk.ntiles, j = s_walk.j;
    if (ntiles == 0) break;
    const Seq<TK> seq = s_walk.c.s;
    if (!EARLY) fetch_q(s_walk);
    if (F8 && a.v_inv_scale) vscale = a.v_inv_scale[s_walk.hc / a.chunks];
    if (tid == 0) {
      s_walks[cur ^ 1] = s_walk;
      s_walks[cur ^ 1].next(a, nhc);
    }
    uint32_t qf[KS][2];
    float qs[2];  // log2-domain scale of this lane's two score columns
    if (F8) {
      float mx = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(qr[k][i])), fabsf(bf_hi(qr[k][i]))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // q / 2^e with 2^e <= max|q| < 2^(e+1): exact in f16 down to 2^-14 of the largest
      int e = (int)(__float_as_uint(mx) >> 23) - 127;
      e = mx > 0.0f && mx < INFINITY ? max(-120, min(120, e)) : 0;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      const float mul = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) qf[k][i] = pack_f16(bf_lo(qr[k][i]) * inv, bf_hi(qr[k][i]) * inv);
      qs[0] = a.scale_log2 * kinv * __shfl_sync(0xffffffffu, mul, 8 * c4);
      qs[1] = a.scale_log2 * kinv * __shfl_sync(0xffffffffu, mul, 8 * c4 + 4);
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][0] = qr[k][0];
        qf[k][1] = qr[k][1];
      }
      qs[0] = qs[1] = a.scale_log2;
    }
    float o[MT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

    for (int it = 0; it < ntiles; ++it) {
      const int tile0 = seq.tile(j + it) * TK, t0 = tile0 + kgrp * KW;
      const bool whole = seq.whole(tile0);
      // ---- S^T = K Q^T
      uint32_t sl = nu % R::N;
      ok = mbar_wait(&full[sl], (nu / R::N) & 1, abort_flag, a.status, STATUS_TIMEOUT, WAIT_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float sc[KT][4];
#pragma unroll
      for (int y = 0; y < KT; ++y) sc[y][0] = sc[y][1] = sc[y][2] = sc[y][3] = 0.0f;
      const uint32_t kb = ring_s + sl * R::SLOT;
#pragma unroll
      for (int k = 0; k < (F8 ? KS / 2 : KS); ++k) {
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          uint32_t r[4];
          ldsm4(kb + (k / PPB) * blk + (k_off[y] ^ (32 * (k % PPB))), r);
          if (F8) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // chunk 2k + x
              uint32_t af[4];
              f16_of_e4m3(r[2 * x], af[0], af[2]);
              f16_of_e4m3(r[2 * x + 1], af[1], af[3]);
              mma16816<true>(sc[y], af, qf[(2 * k + x) % KS][0], qf[(2 * k + x) % KS][1]);
            }
          } else {
            mma16816<false>(sc[y], r, qf[k][0], qf[k][1]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
      ++nu;
      // ---- softmax
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[y][e] *= qs[e & 1];
      if (!whole) {
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (!seq.sees(t0 + 16 * y + 8 * x + g8)) sc[y][2 * x] = sc[y][2 * x + 1] = -INFINITY;
      }
      float mx[2] = {-INFINITY, -INFINITY}, alpha[2];
#pragma unroll
      for (int y = 0; y < KT; ++y) {
        mx[0] = fmax3(mx[0], sc[y][0], sc[y][2]);
        mx[1] = fmax3(mx[1], sc[y][1], sc[y][3]);
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], x));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], x));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (behind 2^20 a float's step is too wide to subtract 15 from)
        const float mn = fmaxf(m[e], F8 && fabsf(mx[e]) < 0x1p20f ? mx[e] - 15.0f : mx[e]);
        const float mu = mn == -INFINITY ? 0.0f : mn;  // nothing visible yet
        alpha[e] = ex2_fast(m[e] - mu);                // m = -inf: 0
        m[e] = mn;
        float add = 0.0f;
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          sc[y][e] = ex2_fast(sc[y][e] - mu);
          sc[y][2 + e] = ex2_fast(sc[y][2 + e] - mu);
          add += sc[y][e] + sc[y][2 + e];
        }
        l[e] = fmaf(l[e], alpha[e], add);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[1];
          o[i][2] *= alpha[0];
          o[i][3] *= alpha[1];
        }
      }
      uint32_t pf[KT][2], pl[KT][2];
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = sc[y][2 * x], p1 = sc[y][2 * x + 1];
          if (F8) {
            pf[y][x] = movm(pack_f16(p0, p1));
          } else {
            const uint32_t hi = pack_bf16(p0, p1);
            pf[y][x] = movm(hi);
            pl[y][x] = movm(pack_bf16(p0 - bf_lo(hi), p1 - bf_hi(hi)));
          }
        }
      // ---- O^T += V^T P^T
      sl = nu % R::N;
      ok = mbar_wait(&full[sl], (nu / R::N) & 1, abort_flag, a.status, STATUS_TIMEOUT, WAIT_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t vb = ring_s + sl * R::SLOT;
      if (!whole) {
        // Values of hidden tokens, NaN maybe, are made 0 where they lie (0 x NaN
        // would reach the sum): each warp clears those of its own tokens.
        constexpr int CH = R::ROW / 16;  // 16-byte chunks of a token
        for (int t = lane; t < KW; t += 32) {
          if (seq.sees(t0 + t)) continue;
          const uint32_t row = vb + row_base(kgrp * KW + t);
          for (int x = 0; x < CH; ++x) {
            const int ch = (x + lane) % CH;  // lanes start at different banks
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + (ch / (ROWB / 16)) * blk +
                                                                         (ch % (ROWB / 16)) * 16),
                         "r"(0)
                         : "memory");
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int y = 0; y < KT; ++y) {
#pragma unroll
        for (int i = 0; i < (F8 ? MT / 2 : MT); ++i) {
          uint32_t r[4];
          ldsm4t(vb + (i / PPB) * blk + (v_off[y] ^ (32 * (i % PPB))), r);
          if (F8) {  // 32 columns: matrices (keys 0-7, 8-15) x chunks (2i, 2i + 1)
            uint32_t ev[4], od[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f16_of_e4m3(__byte_perm(r[x], 0, 0x3120), ev[x], od[x]);
            }
            const uint32_t ea[4] = {ev[0], ev[2], ev[1], ev[3]}, oa[4] = {od[0], od[2], od[1], od[3]};
            mma16816<true>(o[(2 * i) % MT], ea, pf[y][0], pf[y][1]);
            mma16816<true>(o[(2 * i + 1) % MT], oa, pf[y][0], pf[y][1]);
          } else {  // 16 columns: matrices (chunks 2i, 2i + 1) x (keys 0-7, 8-15)
            mma16816<false>(o[i], r, pf[y][0], pf[y][1]);
            mma16816<false>(o[i], r, pl[y][0], pl[y][1]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
      ++nu;
    }

    // ---- join the warps that share a head group: common maximum, then the sums in warp order
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[e];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g8 == 0) {
        s_m[kgrp][hgrp * 8 + 2 * c4 + e] = m[e];
        s_l[kgrp][hgrp * 8 + 2 * c4 + e] = v;
      }
    }
    if (bar_compute_any(!ok)) return;  // a wait gave up: all four warps leave together
    if (EARLY && s_walks[cur ^ 1].ntiles) fetch_q(s_walks[cur ^ 1]);
    const size_t part_sz = (size_t)HT * (D + 2);
    const bool direct = s_walk.direct;
    const int hc = s_walk.hc, g = hc / a.chunks, h0 = (hc - g * a.chunks) * HT, heads = min(HT, a.hpg - h0), b = s_walk.c.b;
    const int64_t w_first = direct ? blockIdx.x : ((s_walk.item0 + 1) * s_walk.G + s_walk.T - 1) / s_walk.T - 1;
    float* my_part = a.part + (size_t)(2 * blockIdx.x + (blockIdx.x == w_first)) * part_sz;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (int64_t)b * a.ld_out + (int64_t)(g * a.hpg + h0) * D;
    float* lse = a.lse ? a.lse + (int64_t)b * a.nq + g * a.hpg + h0 : nullptr;
    float al[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = hgrp * 8 + 2 * c4 + e;
      float mx = s_m[0][h];
#pragma unroll
      for (int w = 1; w < KG; ++w) mx = fmaxf(mx, s_m[w][h]);
      al[e] = mx == -INFINITY ? 0.0f : ex2_fast(m[e] - mx);
    }
    // (max drops NaN: where every score of a warp is one its maximum stays -inf,
    // and its sum carries the NaN, so no sum is replaced by 0)
    if (tid < HT) {
      float mx = s_m[0][tid];
#pragma unroll
      for (int w = 1; w < KG; ++w) mx = fmaxf(mx, s_m[w][tid]);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < KG; ++w) s += s_l[w][tid] * ex2_fast(s_m[w][tid] - (mx == -INFINITY ? 0.0f : mx));
      if (direct) {
        s_inv[tid] = s > 0.0f ? vscale / s : seq.len > 0 ? NAN : 0.0f;
        if (lse && tid < heads) lse[tid] = s == 0.0f ? -INFINITY : (mx + log2f(s)) * 0.69314718055994531f;
      } else {
        __stcg(my_part + (size_t)HT * D + tid, mx);
        __stcg(my_part + (size_t)HT * D + HT + tid, s);
      }
    }
    constexpr int IP = OD / 16;  // m-tiles joined at a time
#pragma unroll
    for (int ps = 0; ps < D / OD; ++ps) {
#pragma unroll
      for (int ii = 0; ii < IP; ++ii) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = hgrp * 8 + 2 * c4 + (e & 1);
          // column of the m-tile's row, within the columns joined now
          const int col = F8 ? 32 * (ii / 2) + 16 * (e >> 1) + 2 * g8 + (ii & 1) : 16 * ii + g8 + 8 * (e >> 1);
          s_o[(kgrp * HT + h) * (OD + 4) + col] = o[ps * IP + ii][e] * al[e & 1];
        }
      }
      bar_compute();
      for (int x = tid; x < HT * OD / 4; x += NCW * 32) {
        const int h = x / (OD / 4), col = 4 * (x % (OD / 4));
        float4 v = *reinterpret_cast<const float4*>(&s_o[h * (OD + 4) + col]);
#pragma unroll
        for (int w = 1; w < KG; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(&s_o[(w * HT + h) * (OD + 4) + col]);
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        if (direct) {
          const float r = s_inv[h];
          if (h < heads)
            *reinterpret_cast<uint2*>(out + (int64_t)h * D + ps * OD + col) =
                make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
        } else {
          __stcg(reinterpret_cast<float4*>(my_part + (size_t)h * D + ps * OD + col), v);
        }
      }
      bar_compute();
    }

    if (!direct) {
      JoinArgs ja;
      ja.part = a.part;
      ja.ctr_first = a.counters;
      ja.ctr_last = a.counters + 2 * (int64_t)a.workers;
      ja.out = out;
      ja.lse = lse;
      ja.w_first = (int)w_first;
      ja.nparts = (int)((s_walk.item1 * s_walk.G + s_walk.T - 1) / s_walk.T - w_first);
      ja.p_me = (int)(blockIdx.x - w_first);
      ja.heads = heads;
      ja.vscale = vscale;
      join_parts<D, HT>(ja, &s_last);
    }
    bar_compute();  // everyone is done with this segment's walk
  }
}

template <int D, bool F8, int HG>
cudaError_t launch_one(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  constexpr int smem = Cfg<D, F8, HG>::N * Cfg<D, F8, HG>::SLOT + 1024;
  const cudaError_t e = allow_smem<kv_decode_kernel<D, F8, HG>>(smem);
  if (e != cudaSuccess) return e;
  kv_decode_kernel<D, F8, HG><<<a.workers, NTHR, smem, st>>>(a, km, vm);
  return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_h(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  switch (kv_decode_head_tile(a.hpg)) {
    case 8: return launch_one<D, F8, 1>(a, km, vm, st);
    case 16: return launch_one<D, F8, 2>(a, km, vm, st);
    default: return launch_one<D, F8, 4>(a, km, vm, st);
  }
}

template <int D>
cudaError_t launch_d(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, bool e4m3, cudaStream_t st) {
  return e4m3 ? launch_h<D, true>(a, km, vm, st) : launch_h<D, false>(a, km, vm, st);
}

}  // namespace

int kv_decode_tile(int d) { return d <= 128 ? 128 : 64; }  // Cfg::TK

int kv_decode_workers(int num_sms) { return 2 * num_sms; }

bool make_cache_map(CUtensorMap* m, const void* ptr, bool e4m3, int d, int page_size, int nkv, int64_t num_pages,
                    int64_t stride_page, int64_t stride_head, int64_t stride_slot, int box_tokens) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const uint64_t e = e4m3 ? 1 : 2;
  // {block of columns, slot, block, key head, page}: a box of all blocks lands
  // as [box_tokens][block] one behind the other (Cfg::BLOCK bytes a block's row)
  const uint64_t row = d * e, blk = row % 128 == 0 ? 128 : 64;
  cuuint64_t dims[5] = {blk / e, (cuuint64_t)page_size, row / blk, (cuuint64_t)nkv, (cuuint64_t)num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)stride_slot * e, blk, (cuuint64_t)stride_head * e, (cuuint64_t)stride_page * e};
  cuuint32_t box[5] = {(cuuint32_t)(blk / e), (cuuint32_t)box_tokens, (cuuint32_t)(row / blk), 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, blk == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv_decode(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int d, bool e4m3,
                             cudaStream_t st) {
  if (a.batch <= 0) return cudaSuccess;
  switch (d) {
    case 64: return launch_d<64>(a, km, vm, e4m3, st);
    case 128: return launch_d<128>(a, km, vm, e4m3, st);
    case 192: return launch_d<192>(a, km, vm, e4m3, st);
    case 256: return launch_d<256>(a, km, vm, e4m3, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tpmlp
