// Attention of one new token per sequence over a paged key/value cache.
//
//   s_t = scale q . k_t over the visible tokens t < len (with a window: the
//   last `window` tokens and the first `sinks`),  out = softmax(s) V,
//   lse = log sum exp s.  No visible token: out 0, lse -inf.
//
// What bounds it: reading the cache once.  A key head's query heads are worked
// on together, so a cache byte meets at most 16 of them: about 16 flops a byte
// in bf16, far below what even the mma.sync tensor path gives, which is why
// the products use m16n8k16 with the keys (and for P V the head dimension) as
// M and 8 query heads as N; a 128-row tcgen05 tile would be all padding.
//
// The split.  The cache is cut into tiles of 64 tokens; the tiles of every
// (sequence, key head) laid end to end are divided evenly over a fixed number
// of CTAs (two an SM), whatever the lengths are.  They are read on the device:
// each CTA scans them once.  A CTA walks its range; where a (sequence, key
// head) ends inside it, its result is written, and where one is shared with
// other CTAs, each leaves an unnormalised partial (sum, maximum, weighted
// values) in the workspace and the last to arrive joins them: in groups of 16,
// then the groups, so one CTA never reads hundreds of partials.  Nobody waits
// for another CTA, and partials are added in the order of the tokens, so the
// result does not depend on which came last.
//
// The pipe.  One warp fetches tiles by TMA (one box per page and operand, the
// swizzle making ldmatrix conflict-free) into a ring of 96 KB a CTA, which
// keeps 192 KB in flight on an SM; four warps compute, each on 16 tokens of a
// tile with its own running maximum and sum, joined at the end of a segment.
//
// Rounding.  Scores, maxima, sums and outputs are f32.  With a bf16 cache P is
// the sum of two bf16 values (16 bits), because a single one would add as much
// error as the final rounding of the output; the second product costs nothing
// that is not hidden behind the reads.  With an E4M3 cache, codes are converted
// to f16 exactly, q is brought to f16 after a power-of-two scale per head, and
// P is f16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv_decode.h"
#include "ptx_sm103.cuh"
#include "tma_maps.cuh"
#include "f32x2.cuh"

namespace tpmlp {
namespace {

constexpr int NCW = 4;          // computing warps
constexpr int NTHR = 32 * (NCW + 1);
constexpr int RING_BYTES = 96 * 1024;
constexpr int JOIN_GROUP = 16;  // partials one CTA joins at a time
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 100000000ull;

// Every computing warp works on every tile, so each waits for every use of a
// slot: a barrier's one-bit phase is never asked about two rounds ahead.
template <int D, bool F8>
struct Ring {
  static constexpr int ROW = D * (F8 ? 1 : 2);
  static constexpr int BLOCK = ROW % 128 == 0 ? 128 : 64;  // bytes of a row that lie together (the swizzle's width)
  static constexpr int TK = ROW <= 128 ? 128 : 64;  // tokens of a tile
  static constexpr int SLOT = TK * ROW;             // one operand of a tile
  static constexpr int N = RING_BYTES / SLOT;
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 tile of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t movm(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t lo16) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(lo16));
  return r;
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

template <int D, bool F8, int HT>
__global__ void __launch_bounds__(NTHR, (D * HT >= 4096 || (D == 192 && HT == 16)) ? 1 : 2)
    kv_decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using R = Ring<D, F8>;
  constexpr int TK = R::TK;
  constexpr int KW = TK / NCW;      // tokens of a tile that a warp works on
  constexpr int KT = KW / 16;       // as m-tiles
  constexpr int NT = HT / 8;        // n-tiles of 8 heads
  constexpr int KS = D / 16;        // k-steps of Q K^T
  constexpr int MT = D / 16;        // m-tiles of V^T P^T
  constexpr int ROWB = R::BLOCK;        // bytes of a block's row
  constexpr int NBLK = R::ROW / ROWB;   // blocks of a row in shared memory
  extern __shared__ __align__(1024) uint8_t ring_raw[];
  __shared__ __align__(8) uint64_t full[R::N], empty[R::N];
  __shared__ int s_abort;
  __shared__ int64_t s_scan[NTHR / 32 + 1];
  __shared__ int64_t s_base;
  __shared__ int s_b;
  __shared__ int s_last;
  __shared__ float s_m[NCW][HT], s_l[NCW][HT];
  __shared__ float s_mx[HT], s_inv[HT];
  __shared__ float s_w[32][HT], s_s[32][HT];
  constexpr int OD = 512 / HT;  // columns of O joined at a time: 8 KB, so that two CTAs fit an SM
  __shared__ __align__(16) float s_o[NCW][HT * (OD + 4)];

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
  // two tiles a worker where there are few: fewer partial results to join
  const int64_t want = (T + 1) / 2;
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

  if (warp == NCW) {
    // ------------------------------------------------------------ producer
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
  const int g8 = lane >> 2, c4 = lane & 3;  // row group and column pair of the mma fragments
  // shared-memory address parts of the lane's ldmatrix rows: token 16 y + key of the warp's
  const int bt = a.box_tokens;
  const uint32_t blk = (uint32_t)bt * ROWB;  // bytes from one block to the next
  auto row_base = [&](int key) -> uint32_t { return (uint32_t)(key / bt) * (blk * NBLK) + (key % bt) * ROWB; };
  const int k_key = lane & 15;  // K: matrices (keys 0-7, 8-15) x 2 chunks
  // V: the same with E4M3; bf16 (2 chunks) x (keys 0-7, 8-15)
  const int v_key = F8 ? k_key : (lane & 7) + ((lane >> 4) << 3);
  uint32_t k_row[KT], v_row[KT];
#pragma unroll
  for (int y = 0; y < KT; ++y) {
    k_row[y] = row_base(warp * KW + 16 * y + k_key);
    v_row[y] = row_base(warp * KW + 16 * y + v_key);
  }
  const uint32_t k_sw = ROWB == 64 ? (k_key >> 1) & 3 : k_key & 7, v_sw = ROWB == 64 ? (v_key >> 1) & 3 : v_key & 7;
  const uint32_t k_half = lane >> 4;  // chunk of the pair
  const uint32_t v_half = F8 ? lane >> 4 : (lane >> 3) & 1;
  constexpr int CPB = ROWB / 16;  // 16-byte chunks of a block's row
  // offset of 16-byte chunk 2 pair + half within a token's row
  auto chunk_off = [&](int pair, uint32_t half, uint32_t sw) -> uint32_t {
    return (uint32_t)(2 * pair / CPB) * blk + ((((uint32_t)(2 * pair % CPB) + half) ^ sw) << 4);
  };

  uint32_t qf[NT][KS][2];
  float qs[NT][2];  // log2-domain scale of this lane's two score columns
  float o[MT][NT][4];
  float m[NT][2], l[NT][2];

  uint32_t n = 0;  // ring uses so far
  bool ok = true;
  int64_t rel = c.pos - c.base;
  int hc = (int)(rel / c.s.tiles), j = (int)(rel - (int64_t)hc * c.s.tiles);

  while (ok && c.pos < c.end) {
    // ---- one segment: the worker's tiles of (sequence b, key head g, chunk)
    const int g = hc / a.chunks, h0 = (hc - g * a.chunks) * HT;
    const int heads = min(HT, a.hpg - h0);
    const int64_t item0 = c.base + (int64_t)hc * c.s.tiles, item1 = item0 + c.s.tiles;
    const int64_t seg_end = item1 < c.end ? item1 : c.end;
    const int64_t seg_begin = c.pos;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)c.b * a.ld_q + (int64_t)(g * a.hpg + h0) * D;
    const float kscale = a.scale_log2 * (F8 && a.k_inv_scale ? a.k_inv_scale[g] : 1.0f);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = t * 8 + g8;
      if (F8) {
        float mx = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint2 v = make_uint2(0, 0);
          if (h < heads) v = *reinterpret_cast<const uint2*>(q + (int64_t)h * D + 16 * k + 4 * c4);
          qf[t][k][0] = v.x;
          qf[t][k][1] = v.y;
          mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf_lo(v.x)), fabsf(bf_hi(v.x))), fmaxf(fabsf(bf_lo(v.y)), fabsf(bf_hi(v.y)))));
        }
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
          for (int i = 0; i < 2; ++i) qf[t][k][i] = pack_f16(bf_lo(qf[t][k][i]) * inv, bf_hi(qf[t][k][i]) * inv);
        qs[t][0] = kscale * __shfl_sync(0xffffffffu, mul, 8 * c4);
        qs[t][1] = kscale * __shfl_sync(0xffffffffu, mul, 8 * c4 + 4);
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            qf[t][k][i] = 0;
            if (h < heads) qf[t][k][i] = *reinterpret_cast<const uint32_t*>(q + (int64_t)h * D + 16 * k + 8 * i + 2 * c4);
          }
        qs[t][0] = qs[t][1] = kscale;
      }
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][e] = 0.0f;
    }

    for (; ok && c.pos < seg_end; ++c.pos, ++j) {
      const int tile0 = c.s.tile(j) * TK, t0 = tile0 + warp * KW;
      const bool whole = c.s.whole(tile0);
      // ---- S^T = K Q^T
      uint32_t sl = n % R::N;
      ok = mbar_wait(&full[sl], (n / R::N) & 1, abort_flag, a.status, STATUS_TIMEOUT, WAIT_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      float sc[KT][NT][4];
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[y][t][0] = sc[y][t][1] = sc[y][t][2] = sc[y][t][3] = 0.0f;
      const uint32_t kb = ring_s + sl * R::SLOT;
#pragma unroll
      for (int k = 0; k < (F8 ? KS / 2 : KS); ++k) {
        const uint32_t off = kb + chunk_off(k, k_half, k_sw);
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          uint32_t r[4];
          ldsm4(off + k_row[y], r);
          if (F8) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // chunk 2k + x
              const uint32_t af[4] = {f16x2_of_e4m3x2(r[2 * x]), f16x2_of_e4m3x2(r[2 * x + 1]),
                                      f16x2_of_e4m3x2(r[2 * x] >> 16), f16x2_of_e4m3x2(r[2 * x + 1] >> 16)};
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816<true>(sc[y][t], af, qf[t][(2 * k + x) % KS][0], qf[t][(2 * k + x) % KS][1]);
            }
          } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<false>(sc[y][t], r, qf[t][k][0], qf[t][k][1]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
      // ---- softmax
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[y][t][e] *= qs[t][e & 1];
      if (!whole) {
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (!c.s.sees(t0 + 16 * y + 8 * x + g8)) {
#pragma unroll
              for (int t = 0; t < NT; ++t) sc[y][t][2 * x] = sc[y][t][2 * x + 1] = -INFINITY;
            }
      }
      uint32_t pf[KT][NT][2], pl[KT][NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -INFINITY;
#pragma unroll
          for (int y = 0; y < KT; ++y) mx = fmax3(mx, sc[y][t][e], sc[y][t][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[t][e], mx);
          const float mu = mn == -INFINITY ? 0.0f : mn;  // nothing visible yet
          alpha[e] = ex2_fast(m[t][e] - mu);             // m = -inf: 0
          m[t][e] = mn;
          float sum = 0.0f;
#pragma unroll
          for (int y = 0; y < KT; ++y) {
            sc[y][t][e] = ex2_fast(sc[y][t][e] - mu);
            sc[y][t][2 + e] = ex2_fast(sc[y][t][2 + e] - mu);
            sum += sc[y][t][e] + sc[y][t][2 + e];
          }
          l[t][e] = fmaf(l[t][e], alpha[e], sum);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][t][0] *= alpha[0];
            o[i][t][1] *= alpha[1];
            o[i][t][2] *= alpha[0];
            o[i][t][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float p0 = sc[y][t][2 * x], p1 = sc[y][t][2 * x + 1];
            if (F8) {
              pf[y][t][x] = movm(pack_f16(p0, p1));
            } else {
              const uint32_t hi = pack_bf16(p0, p1);
              pf[y][t][x] = movm(hi);
              pl[y][t][x] = movm(pack_bf16(p0 - bf_lo(hi), p1 - bf_hi(hi)));
            }
          }
      }
      // ---- O^T += V^T P^T
      ++n;
      sl = n % R::N;
      ok = mbar_wait(&full[sl], (n / R::N) & 1, abort_flag, a.status, STATUS_TIMEOUT, WAIT_NS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t vb = ring_s + sl * R::SLOT;
#pragma unroll
      for (int y = 0; y < KT; ++y) {
        uint32_t mk0 = 0xffffffffu, mk1 = 0xffffffffu;  // values of unseen tokens, NaN maybe, become 0
        if (!whole) {
          const int t = t0 + 16 * y + 2 * c4;
          mk0 = (c.s.sees(t) ? 0xffffu : 0u) | (c.s.sees(t + 1) ? 0xffff0000u : 0u);
          mk1 = (c.s.sees(t + 8) ? 0xffffu : 0u) | (c.s.sees(t + 9) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int i = 0; i < (F8 ? MT / 2 : MT); ++i) {
          uint32_t r[4];
          ldsm4t(vb + v_row[y] + chunk_off(i, v_half, v_sw), r);
          if (F8) {  // 32 columns: matrices (keys 0-7, 8-15) x chunks (2i, 2i + 1)
            uint32_t ev[4], od[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t s = __byte_perm(r[x], 0, 0x3120);
              ev[x] = f16x2_of_e4m3x2(s);
              od[x] = f16x2_of_e4m3x2(s >> 16);
              if (!whole) {
                ev[x] &= x & 1 ? mk1 : mk0;
                od[x] &= x & 1 ? mk1 : mk0;
              }
            }
            const uint32_t ea[4] = {ev[0], ev[2], ev[1], ev[3]}, oa[4] = {od[0], od[2], od[1], od[3]};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816<true>(o[(2 * i) % MT][t], ea, pf[y][t][0], pf[y][t][1]);
              mma16816<true>(o[(2 * i + 1) % MT][t], oa, pf[y][t][0], pf[y][t][1]);
            }
          } else {  // 16 columns: matrices (chunks 2i, 2i + 1) x (keys 0-7, 8-15)
            if (!whole) {
              r[0] &= mk0;
              r[1] &= mk0;
              r[2] &= mk1;
              r[3] &= mk1;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816<false>(o[i][t], r, pf[y][t][0], pf[y][t][1]);
              mma16816<false>(o[i][t], r, pl[y][t][0], pl[y][t][1]);
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
      ++n;
    }

    // ---- join the four warps: common maximum, then the sums in warp order
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[t][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (g8 == 0) {
          s_m[warp][t * 8 + 2 * c4 + e] = m[t][e];
          s_l[warp][t * 8 + 2 * c4 + e] = v;
        }
      }
    if (bar_compute_any(!ok)) return;  // a wait gave up: all four warps leave together
    const bool direct = seg_begin == item0 && seg_end == item1;
    const int64_t w_first = direct ? blockIdx.x : ((item0 + 1) * G + T - 1) / T - 1;
    const int64_t w_last = direct ? blockIdx.x : (item1 * G + T - 1) / T - 1;
    const int nparts = (int)(w_last - w_first + 1);
    const int p_me = (int)(blockIdx.x - w_first);
    const size_t part_sz = (size_t)HT * (D + 2);
    float* my_part = a.part + (size_t)(2 * blockIdx.x + (p_me == 0)) * part_sz;
    const float vscale = F8 && a.v_inv_scale ? a.v_inv_scale[g] : 1.0f;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (int64_t)c.b * a.ld_out + (int64_t)(g * a.hpg + h0) * D;
    float* lse = a.lse ? a.lse + (int64_t)c.b * a.nq + g * a.hpg + h0 : nullptr;
    float al[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = t * 8 + 2 * c4 + e;
        float mx = s_m[0][h];
#pragma unroll
        for (int w = 1; w < NCW; ++w) mx = fmaxf(mx, s_m[w][h]);
        al[t][e] = mx == -INFINITY ? 0.0f : ex2_fast(m[t][e] - mx);
      }
    if (tid < HT) {
      float mx = s_m[0][tid];
#pragma unroll
      for (int w = 1; w < NCW; ++w) mx = fmaxf(mx, s_m[w][tid]);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < NCW; ++w) s += mx == -INFINITY ? 0.0f : s_l[w][tid] * ex2_fast(s_m[w][tid] - mx);
      if (direct) {
        s_inv[tid] = s > 0.0f ? vscale / s : (s == s ? 0.0f : s);
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
        const int i = ps * IP + ii;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = g8 + (e >> 1) * 8, h = t * 8 + 2 * c4 + (e & 1);
            // column of the m-tile's row, within the columns joined now
            const int col = F8 ? 32 * (ii / 2) + 16 * (e >> 1) + 2 * g8 + (ii & 1) : 16 * ii + row;
            s_o[warp][h * (OD + 4) + col] = o[i][t][e] * al[t][e & 1];
          }
      }
      bar_compute();
      for (int x = tid; x < HT * OD / 2; x += NCW * 32) {
        const int h = x / (OD / 2), col = 2 * (x % (OD / 2));
        float2 v = *reinterpret_cast<const float2*>(&s_o[0][h * (OD + 4) + col]);
#pragma unroll
        for (int w = 1; w < NCW; ++w) {
          const float2 y = *reinterpret_cast<const float2*>(&s_o[w][h * (OD + 4) + col]);
          v.x += y.x;
          v.y += y.y;
        }
        if (direct) {
          if (h < heads)
            *reinterpret_cast<uint32_t*>(out + (int64_t)h * D + ps * OD + col) = pack_bf16(v.x * s_inv[h], v.y * s_inv[h]);
        } else {
          __stcg(reinterpret_cast<float2*>(my_part + (size_t)h * D + ps * OD + col), v);
        }
      }
      bar_compute();
    }

    if (!direct) {
      // ---- the last CTA to arrive joins: groups of JOIN_GROUP, then the groups' leaders
      for (int level = 0; level < 2; ++level) {
        const int ngroups = (nparts + JOIN_GROUP - 1) / JOIN_GROUP;
        const int p0 = level == 0 ? p_me / JOIN_GROUP * JOIN_GROUP : 0;
        const int pstep = level == 0 ? 1 : JOIN_GROUP;
        const int cnt = level == 0 ? min(JOIN_GROUP, nparts - p0) : ngroups;
        const int64_t w_lead = w_first + p0;
        uint32_t* ctr = a.counters + (level == 0 ? 2 * w_lead + (p0 == 0) : 2 * (int64_t)a.workers + w_first);
        if (cnt > 1) {
          __threadfence();
          bar_compute();
          if (tid == 0) {
            const uint32_t old = atomicAdd(ctr, 1u);
            s_last = old == (uint32_t)cnt - 1;
            if (old == (uint32_t)cnt - 1) *ctr = 0;  // ready for the next launch
          }
          bar_compute();
          if (!s_last) break;
          __threadfence();
        }
        auto part_of = [&](int i) -> float* {
          const int p = p0 + i * pstep;
          return a.part + (size_t)(2 * (w_first + p) + (p == 0)) * part_sz;
        };
        const bool final_level = ngroups == 1 || level == 1;
        if (!final_level && cnt == 1) continue;  // a group of one stands for itself
        for (int x = tid; x < cnt * HT; x += NCW * 32) {
          const float* pp = part_of(x / HT) + (size_t)HT * D + x % HT;
          s_w[x / HT][x % HT] = __ldcg(pp);
          s_s[x / HT][x % HT] = __ldcg(pp + HT);
        }
        bar_compute();
        if (tid < HT) {
          float mx = -INFINITY;
          for (int i = 0; i < cnt; ++i) mx = fmaxf(mx, s_w[i][tid]);
          float s = 0.0f;
          for (int i = 0; i < cnt; ++i) {
            const float w = mx == -INFINITY ? 0.0f : ex2_fast(s_w[i][tid] - mx);
            s_w[i][tid] = w;
            s += w * s_s[i][tid];
          }
          s_mx[tid] = mx;
          s_inv[tid] = final_level ? (s > 0.0f ? vscale / s : (s == s ? 0.0f : s)) : s;
          if (final_level && lse && tid < heads) lse[tid] = s == 0.0f ? -INFINITY : (mx + log2f(s)) * 0.69314718055994531f;
        }
        bar_compute();
        float* lead = part_of(0);
        for (int x = tid; x < HT * D / 4; x += NCW * 32) {
          const int h = 4 * x / D, col = 4 * x % D;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int i0 = 0; i0 < cnt; i0 += 8) {
            float4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < cnt) y[i] = __ldcg(reinterpret_cast<const float4*>(part_of(i0 + i)) + x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < cnt) {
                const float w = s_w[i0 + i][h];
                v.x = fmaf(w, y[i].x, v.x);
                v.y = fmaf(w, y[i].y, v.y);
                v.z = fmaf(w, y[i].z, v.z);
                v.w = fmaf(w, y[i].w, v.w);
              }
          }
          if (final_level) {
            const float r = s_inv[h];
            if (h < heads)
              *reinterpret_cast<uint2*>(out + (int64_t)h * D + col) = make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
          } else {
            __stcg(reinterpret_cast<float4*>(lead) + x, v);
          }
        }
        if (!final_level && tid < HT) {
          __stcg(lead + (size_t)HT * D + tid, s_mx[tid]);
          __stcg(lead + (size_t)HT * D + HT + tid, s_inv[tid]);
        }
        bar_compute();
        if (final_level) break;
      }
    }
    // ---- next segment
    if (c.pos < c.end && j == c.s.tiles) {
      j = 0;
      if (++hc == nhc) {
        hc = 0;
        c.base += (int64_t)c.s.tiles * nhc;
        c.s = make_seq<TK>(a, ++c.b, false);
      }
    }
  }
}

template <int D, bool F8, int HT>
cudaError_t launch_one(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  constexpr int smem = Ring<D, F8>::N * Ring<D, F8>::SLOT + 1024;
  static const cudaError_t attr = cudaFuncSetAttribute(kv_decode_kernel<D, F8, HT>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (attr != cudaSuccess) return attr;
  kv_decode_kernel<D, F8, HT><<<a.workers, NTHR, smem, st>>>(a, km, vm);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, bool e4m3, cudaStream_t st) {
  const bool wide = kv_decode_head_tile(a.hpg) == 16;
  if (e4m3) return wide ? launch_one<D, true, 16>(a, km, vm, st) : launch_one<D, true, 8>(a, km, vm, st);
  return wide ? launch_one<D, false, 16>(a, km, vm, st) : launch_one<D, false, 8>(a, km, vm, st);
}

}  // namespace

int kv_decode_tile(int d, bool e4m3) { return d * (e4m3 ? 1 : 2) <= 128 ? 128 : 64; }  // Ring::TK

int kv_decode_workers(int d, int hpg, int num_sms) {
  const int ht = kv_decode_head_tile(hpg);
  return (d * ht >= 4096 || (d == 192 && ht == 16) ? 1 : 2) * num_sms;
}

bool make_cache_map(CUtensorMap* m, const void* ptr, bool e4m3, int d, int page_size, int nkv, int64_t num_pages,
                    int64_t stride_page, int64_t stride_head, int64_t stride_slot, int box_tokens) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const uint64_t e = e4m3 ? 1 : 2;
  // {block of columns, slot, block, key head, page}: a box of all blocks lands
  // as [box_tokens][block] one behind the other (Ring::BLOCK bytes a block's row)
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
