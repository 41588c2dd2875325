// Attention of sequences of different lengths on the sm_103a tensor cores:
// whole packed sequences, or new tokens over a paged cache that holds them.
// For the token at position p, over the tokens t that it sees (t <= p; with a
// window, p - t < window or t < sinks):
//   s_t = scale q . k_t,  lse = log sum exp s_t,  out = sum exp(s_t - lse) v_t
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "allow_smem.h"
#include "f32x2.cuh"
#include "ptx_sm103.cuh"
#include "tma_maps.cuh"
#include "varlen.cuh"

namespace tpmlp {
namespace {

constexpr int KB = 128;  // keys of a step
constexpr uint32_t SUB = 128 * 128;  // bytes of a [128 x 64] bf16 tile with the 128-byte swizzle
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 200000000ull;
constexpr float MOVE_LOG2 = 8.0f;  // the running maximum is moved when it is off by more than 2^8
constexpr int MIN_PART = 4;        // steps of a part at least

enum Source { PACKED = 0, PAGED = 1, PAGED_F8 = 2 };

template <int D, int SRC>
struct Cfg {
  static constexpr bool F8 = SRC == PAGED_F8;
  static constexpr int NT = D <= 128 ? 2 : 1;              // query tiles of a CTA
  static constexpr int EC = D % 128 == 0 ? 128 : 64;       // columns of a ring element
  static constexpr int NE = D / EC;                        // elements of an operand
  static constexpr uint32_t EB = EC / 64 * SUB;            // bytes of an element
  static constexpr uint32_t RB = EC * 128;                 // bytes of an element in E4M3 codes
  static constexpr uint32_t QT = D / 64 * SUB;             // bytes of a query tile
  static constexpr int NR = F8 ? (EC == 128 ? 2 : 4) : 0;  // code stages
  static constexpr int FIT = (int)((225 * 1024 - NT * QT - NR * RB) / EB);
  static constexpr int NST = FIT < 12 ? FIT : 12;          // ring stages
  static constexpr uint32_t SMEM = NT * QT + NST * EB + NR * RB + 1024;
  static constexpr int WGS = 1 + NT + (F8 ? 1 : 0);        // issuing, softmax a tile, converting
  static constexpr int THREADS = 128 * WGS;
  // registers a thread after the exchange (0: none takes place)
  static constexpr int SOFTMAX_REGS = WGS == 4 ? 192 : WGS == 3 ? (F8 ? 232 : 216) : 0;
  static constexpr int ISSUE_REGS = WGS == 4 ? 48 : 72;
  static constexpr int CONVERT_REGS = WGS == 4 ? 80 : 168;
  static constexpr int REGS = 128 * (NT * SOFTMAX_REGS + ISSUE_REGS + (F8 ? CONVERT_REGS : 0));
};

struct FwdParams {
  SeqRows seq;
  void* out;
  int64_t ld_out;
  float* lse;
  float* part;  // parts of split blocks, or null
  int nq, nkv, hpg;
  int ht, chunks;    // heads of a tile, tiles of heads a key head
  int tok;           // tokens of a tile
  int slots, heads;  // block slots, key heads times chunks
  int nsplit;
  bool by_length;
  float scale_log2;
  bool negate;
  int window, sinks;
  uint32_t* status;
  const int32_t* table;
  int64_t ld_table;
  int max_pages, page_size, box;
  int64_t num_pages;
  const float *k_inv_scale, *v_inv_scale;
};

// A block's list of steps: the tiles of 128 keys [0, sink_tiles) and [win_tile, ...).
struct Block {
  int b, i;         // b < 0: none
  int first, count, past;  // rows of the block (from `first` on), position of its first row
  int n, n_a;       // steps of the block and of its first tile
  int sink_tiles, win_tile;
  int lo, end, sink_end;  // keys that any row sees: [lo, end) and [0, sink_end)
  __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + win_tile; }
};

__device__ __forceinline__ void fill_block(Block* o, const SeqSpan& sp, int b, int i, int tok, int block_tok, int window,
                                           int sinks) {
  o->b = b;
  o->i = i;
  o->first = sp.first + i * block_tok;
  o->count = min(sp.count - i * block_tok, block_tok);
  o->past = sp.past + i * block_tok;
  if (sp.past < 0) {  // inactive: no keys
    o->past = -1;
    o->n = o->n_a = 0;
    o->sink_tiles = o->win_tile = o->lo = o->end = o->sink_end = 0;
    return;
  }
  o->end = o->past + o->count;
  o->lo = window > 0 ? max(0, o->past + 1 - window) : 0;
  o->sink_end = min(sinks, o->lo);
  o->win_tile = o->lo / KB;
  o->sink_tiles = min((o->sink_end + KB - 1) / KB, o->win_tile);
  const int end_a = o->past + min(o->count, tok);
  o->n = o->sink_tiles + (o->end + KB - 1) / KB - o->win_tile;
  o->n_a = o->sink_tiles + (end_a + KB - 1) / KB - o->win_tile;
}

// Steps of a part of a block of n steps that nsplit CTAs share.
__device__ __forceinline__ int part_steps(int n, int nsplit) {
  return nsplit == 1 ? n : max(MIN_PART, (n + nsplit - 1) / nsplit);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Two E4M3 codes (the low or high half of v) as bf16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_of_e4m3(uint32_t v, bool high) {
  uint32_t h;
  const uint16_t c = (uint16_t)(high ? v >> 16 : v);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return pack_bf16(f.x, f.y);
}

template <int D, int SRC>
__global__ void __launch_bounds__(Cfg<D, SRC>::THREADS, 1)
    var_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const FwdParams p) {
  using C = Cfg<D, SRC>;
  constexpr int NT = C::NT, NE = C::NE, EC = C::EC, NST = C::NST, NR = C::NR;
  constexpr bool F8 = C::F8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full, full[NST], empty[NST], raw_full[NR + 1], raw_empty[NR + 1], s_full[2],
      p_full[2][2], o_full[2], pv_done, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ Block blk;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + NT * C::QT;
  uint8_t* raw = ring + NST * C::EB;
  volatile int* abort_flag = &abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)(blockIdx.x % p.nsplit), unit = (int)(blockIdx.x / p.nsplit);
  const int rank = unit / p.heads, hd = unit % p.heads;
  const int g = hd / p.chunks, h0 = g * p.hpg + hd % p.chunks * p.ht;  // key head, first query head
  const int nh = min(p.ht, (g + 1) * p.hpg - h0);                      // query heads of the tile
  const int64_t cap = SRC == PACKED ? -1 : (int64_t)p.max_pages * p.page_size;
  const int block_tok = NT * p.tok;

  // ---- which block
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], F8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 4);
      mbar_init(&p_full[i][1], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&pv_done, 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  int2* sq = reinterpret_cast<int2*>(smem);  // until the first copy
  if (p.by_length || blockIdx.x == 0) {  // one CTA looks at every sequence, for the report
    bool bad = false;
    for (int b = threadIdx.x; b < p.seq.batch; b += blockDim.x) {
      const SeqSpan s = seq_span(p.seq, b, cap, &bad);
      if (p.by_length) sq[b] = make_int2(s.past, s.count);
    }
    if (bad) atomicOr(p.status, STATUS_BAD_INDEX);
    fence_proxy_async_smem();
  }
  if (p.by_length) __syncthreads();
  if (warp == 2) {
    int b, i = 0;
    if (p.by_length) {
      const int most = p.window > 0 ? (p.window + block_tok) / KB + 2 + (p.sinks + KB - 1) / KB : 0x7fffffff;
      find_by_length<KB>(sq, p.seq.batch, rank, block_tok, most, lane, &b, &i);
    } else {
      const int slot = p.slots - 1 - rank;
      b = find_slot(p.seq, slot, block_tok, lane);
      i = -1;  // below
    }
    if (lane == 0) {
      Block k;
      k.b = -1;
      k.n = 0;
      bool bad = false;
      if (b >= 0) {
        const SeqSpan s = seq_span(p.seq, b, cap, &bad);
        if (i < 0) i = p.slots - 1 - rank - slot_base(s.first, b, block_tok);
        if (i >= 0 && (int64_t)i * block_tok < s.count)
          fill_block(&k, s, b, i, p.tok, block_tok, p.window, p.sinks);
      }
      if (bad) atomicOr(p.status, STATUS_BAD_INDEX);
      blk = k;
    }
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  // this CTA's steps [j0, j0 + nk) of the block
  const int per = part_steps(blk.n, p.nsplit);
  const int j0 = split * per;
  const bool whole = per >= blk.n;
  const bool mine = blk.b >= 0 && (split == 0 || j0 < blk.n);
  const bool has_b = NT == 2 && blk.count > p.tok;
  const int nk_x[2] = {mine ? max(0, min(blk.n_a, j0 + per) - j0) : 0,
                       mine && has_b ? max(0, min(blk.n, j0 + per) - j0) : 0};
  const int nk = max(nk_x[0], nk_x[1]);
  // where a step's operands lie in the ring, in the order that they are used
  auto k_at = [&](int j) -> int { return (NT == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1) * NE; };
  auto v_at = [&](int j) -> int { return (NT == 2 ? 2 * j + 1 : j < nk - 1 ? 2 * j + 2 : 2 * nk - 1) * NE; };

  // Registers: what the issuing and converting warpgroups give up, the softmax
  // takes.  Every warp passes the exchange, with or without steps: an increase
  // waits until the others have given theirs up.
  if (warp < 4) {
  if constexpr (C::SOFTMAX_REGS > 0) regs_dec<C::ISSUE_REGS>();
  if (warp == 0 && nk > 0) {
    // -------------------------------------------------------------- producer
    constexpr int CB = EC / 64;  // 64-column boxes of an element's row
    const int boxes = SRC == PACKED ? 1 : KB / p.box;
    const int my_box = lane / CB, my_col = lane % CB;
    const bool issues = my_box < boxes;
    uint32_t armed = 0, par_armed = 0;  // by stage of the ring that copies land in
    constexpr int LST = F8 ? NR : NST;
    uint64_t *lfull = F8 ? raw_full : full, *lempty = F8 ? raw_empty : empty;
    bool ok = true;
    if (lane == 0) {
      const int tiles = has_b ? 2 : 1;
      mbar_arrive_expect_tx(&q_full, (uint32_t)(tiles * (D / 64) * p.ht * p.tok * 128));
      for (int x = 0; x < tiles; ++x)
        for (int t = 0; t < D / 64; ++t)
          tma_load_3d(smem + x * C::QT + t * SUB, &map_q, &q_full, 64 * t, h0, blk.first + x * p.tok);
    }
    __syncwarp();
    // page of this lane's box in a tile: num_pages (nothing is read, zeros land) where no row sees it
    auto page_of = [&](int tile) -> int {
      const int t = tile * KB + my_box * p.box;
      const bool seen = (t < blk.end && t + p.box > blk.lo) || t < blk.sink_end;
      if (!issues || !seen) return (int)p.num_pages;
      const int pi = t / p.page_size;
      int pg = -1;
      if (pi < p.max_pages) pg = p.table[(int64_t)blk.b * p.ld_table + pi];
      if (pg < 0 || pg >= p.num_pages) {
        atomicOr(p.status, STATUS_BAD_INDEX);
        pg = (int)p.num_pages;
      }
      return pg;
    };
    auto load = [&](int at, const CUtensorMap* map, int tile, int page) -> bool {
      for (int e = 0; e < NE; ++e, ++at) {
        const int s = at % LST;
        const uint32_t par = (uint32_t)((at / LST) & 1);
        if (!__all_sync(0xffffffffu, mbar_wait(&lempty[s], par ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS)))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&lfull[s], F8 ? C::RB : C::EB);
        __syncwarp();
        armed |= 1u << s;
        par_armed = (par_armed & ~(1u << s)) | (par << s);
        if (issues) {
          const int col = e * EC + my_col * 64;
          if constexpr (SRC == PACKED) {
            tma_load_3d(ring + s * C::EB + my_col * SUB, map, &lfull[s], col, g, blk.first - blk.i * block_tok + tile * KB);
          } else {
            const int t = tile * KB + my_box * p.box;
            uint8_t* dst = F8 ? raw + s * C::RB + my_col * (KB * 64) + my_box * p.box * 64
                              : ring + s * C::EB + my_col * SUB + my_box * p.box * 128;
            tma_load_4d(dst, map, &lfull[s], col, t % p.page_size, g, page);
          }
        }
      }
      return true;
    };
    int page_k = 0, page_v = 0, page_n = 0;
    if constexpr (SRC != PACKED) page_n = page_of(blk.tile(j0));
    for (int j = 0; ok && j < nk; ++j) {
      const int tile = blk.tile(j0 + j);
      page_k = page_n;
      if constexpr (SRC != PACKED)
        if (j + 1 < nk) page_n = page_of(blk.tile(j0 + j + 1));
      ok = load(k_at(j), &map_k, tile, page_k);
      if constexpr (NT == 2) {
        if (ok) ok = load(v_at(j), &map_v, tile, page_k);
      } else {  // the values one step behind
        if (ok && j > 0) ok = load(v_at(j - 1), &map_v, blk.tile(j0 + j - 1), page_v);
        page_v = page_k;
      }
    }
    if constexpr (NT == 1)
      if (ok) ok = load(v_at(nk - 1), &map_v, blk.tile(j0 + nk - 1), page_v);
    if (!ok || *abort_flag) {  // copies still in flight land on the barriers armed last
      int no_abort = 0;
      mbar_wait(&q_full, 0, &no_abort, p.status, 0u, DRAIN_NS);
      for (int s = 0; s < LST; ++s)
        if (armed & (1u << s)) mbar_wait(&lfull[s], (par_armed >> s) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 8);
    }
  } else if (warp == 1 && nk > 0) {
    // ---------------------------------------------------------------- issuer
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, KB, false, false);
    constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, EC, false, true);
    const uint64_t q_desc = sw128_desc(smem_u32(smem), 16, 1024);
    const uint64_t k_desc = sw128_desc(smem_u32(ring), 16, 1024);
    const uint64_t v_desc = sw128_desc(smem_u32(ring), SUB, 1024);
    auto wait_all = [&](uint64_t* bar, uint32_t par) -> int {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
    };
    auto wait_elems = [&](int at) -> int {
      int r = 1;
      for (int e = 0; r && e < NE; ++e) r = wait_all(&full[(at + e) % NST], (uint32_t)(((at + e) / NST) & 1));
      return r;
    };
    // S = Q_x K_j^T into score slot `slot`; frees the keys when asked to
    auto mma_s = [&](int x, int slot, int at, bool last) {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int s = (at + e) % NST;
        const uint64_t kb = desc_advance(k_desc, s * C::EB), qa = desc_advance(q_desc, x * C::QT + e * C::EB);
#pragma unroll
        for (int kk = 0; kk < EC / 16; ++kk)
          tc_mma_f16(tmem_base + slot * KB, desc_advance(qa, (kk >> 2) * SUB + (kk & 3) * 32),
                     desc_advance(kb, (kk >> 2) * SUB + (kk & 3) * 32), IDESC_S, e > 0 || kk > 0 ? 1u : 0u);
        if (last) tc_commit(&empty[s]);
      }
      tc_commit(&s_full[slot]);
    };
    // half of O_x += P V_j: keys 64 half .. 64 half + 63
    auto mma_pv = [&](int x, int slot, int at, int half, bool first, bool last) {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int s = (at + e) % NST;
        const uint64_t vb = desc_advance(v_desc, s * C::EB);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_f16_ts(tmem_base + 256 + x * D + e * EC, tmem_base + slot * KB + (half * 4 + kk) * 8,
                        desc_advance(vb, (half * 4 + kk) * 2048), IDESC_PV, !first || half > 0 || kk > 0 ? 1u : 0u);
        if (last && half == 1) tc_commit(&empty[s]);
      }
    };
    int ok = wait_all(&q_full, 0) && wait_elems(k_at(0));
    tc_fence_after();
    if constexpr (NT == 2) {
      if (ok && elect_one()) {
        if (nk_x[0] > 0) mma_s(0, 0, k_at(0), nk_x[1] == 0);
        if (nk_x[1] > 0) mma_s(1, 1, k_at(0), true);
      }
      __syncwarp();
      for (int j = 0; ok && j < nk; ++j) {
        if (!(ok = wait_elems(v_at(j)))) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (ok && j < nk_x[x]) {
            // the last tile that uses the step's operands frees them
            const bool last = x == 1 || j >= nk_x[1], lastn = x == 1 || j + 1 >= nk_x[1];
            for (int half = 0; ok && half < 2; ++half) {
              if (!(ok = wait_all(&p_full[x][half], j & 1))) break;
              tc_fence_after();
              if (elect_one()) {
                mma_pv(x, x, v_at(j), half, j == 0, last);
                if (half == 1 && j + 1 == nk_x[x]) tc_commit(&o_full[x]);
              }
              __syncwarp();
            }
            if (ok && j + 1 < nk_x[x]) {
              if (!(ok = wait_elems(k_at(j + 1)))) break;
              tc_fence_after();
              if (elect_one()) mma_s(x, x, k_at(j + 1), lastn);
              __syncwarp();
            }
          }
        }
      }
    } else {
      if (ok && elect_one()) mma_s(0, 0, k_at(0), true);
      __syncwarp();
      for (int j = 0; ok && j < nk; ++j) {
        const int slot = j & 1;
        if (j + 1 < nk) {
          if (!(ok = wait_elems(k_at(j + 1)))) break;
          tc_fence_after();
          if (elect_one()) mma_s(0, slot ^ 1, k_at(j + 1), true);
          __syncwarp();
        }
        if (!(ok = wait_elems(v_at(j)))) break;
        for (int half = 0; ok && half < 2; ++half) {
          if (!(ok = wait_all(&p_full[slot][half], (j >> 1) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            mma_pv(0, slot, v_at(j), half, j == 0, true);
            if (half == 1) tc_commit(j + 1 == nk ? &o_full[0] : &pv_done);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) tc_commit(&drain_bar);
    __syncwarp();
    int no_abort = 0;
    mbar_wait(&drain_bar, 0, &no_abort, p.status, STATUS_TIMEOUT, DRAIN_NS);
  }
  } else if (warp < 4 + 4 * NT) {
    // --------------------------------------------------------------- softmax
    if constexpr (C::SOFTMAX_REGS > 0) regs_inc<C::SOFTMAX_REGS>();
    const int x = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const int nkx = nk_x[x];
    const int tk = x * p.tok + r / p.ht, hh = r % p.ht;  // token in the block, head in the tile
    const bool stored = r < p.tok * p.ht && hh < nh && tk < blk.count;
    const int pos = blk.past + tk;
    const int pos_first = blk.past + x * p.tok, pos_last = blk.past + min(blk.count, (x + 1) * p.tok) - 1;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t t_o = tmem_base + lane_off + 256 + x * D;
    float scale_log2 = p.scale_log2, vscale = 1.0f;
    if constexpr (F8) {
      if (p.k_inv_scale) scale_log2 *= p.k_inv_scale[g];
      if (p.v_inv_scale) vscale = p.v_inv_scale[g];
    }
    float m_run = -INFINITY, l = 0.0f;
    int ok = nkx > 0;
    for (int j = 0; ok && j < nkx; ++j) {
      const int slot = NT == 2 ? x : j & 1;
      const uint32_t spar = (uint32_t)(NT == 2 ? j & 1 : (j >> 1) & 1);
      const uint32_t t_s = tmem_base + lane_off + slot * KB;
      const int t0 = blk.tile(j0 + j) * KB;
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[slot], spar, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
      if (!ok) break;
      tc_fence_after();
      // values that no row of the block sees: cleared, so that they count nothing whatever they are
      if (t0 + KB > blk.end || (t0 < blk.lo && t0 + KB > blk.sink_end)) {
        // (A wait for a ring stage is good for the next phase only: what was in
        // the stage before has landed, as the scores of this step and, with two
        // score slots, the products of the one before are complete.)
        if constexpr (NT == 1)
          if (j > 0)
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done, (uint32_t)((j - 1) & 1), abort_flag, p.status,
                                                   STATUS_TIMEOUT, WAIT_NS));
        const int at = v_at(j);
        const int t = t0 + r;
        const bool clear = t >= blk.end || (t < blk.lo && t >= blk.sink_end);
        for (int e = 0; ok && e < NE; ++e) {
          const int s = (at + e) % NST;
          ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (uint32_t)(((at + e) / NST) & 1), abort_flag, p.status,
                                                 STATUS_TIMEOUT, WAIT_NS));
          if (ok && clear) {
#pragma unroll
            for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(ring + s * C::EB + cb * SUB + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
      }
      uint32_t v[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
      tmem_ld_wait();
      if (p.negate) {
#pragma unroll
        for (int c = 0; c < 128; ++c) v[c] ^= 0x80000000u;
      }
      const bool masked = t0 + KB - 1 > pos_first ||
                          (p.window > 0 && pos_last - t0 >= p.window && t0 + KB > p.sinks);
      if (masked) {
        const int hi = pos - t0;                                    // keys c <= hi
        const int lo = p.window > 0 ? pos - p.window - t0 : -1;     // and c > lo
        const int sk = p.window > 0 ? p.sinks - t0 : 0;             // or c < sk
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > hi || (c <= lo && c >= sk)) v[c] = 0xff800000u;  // -inf
      }
      float mx[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float m = __uint_as_float(v[k]);
#pragma unroll
        for (int i = 1; i < 15; i += 2) m = fmax3(m, __uint_as_float(v[k + 8 * i]), __uint_as_float(v[k + 8 * i + 8]));
        mx[k] = fmaxf(m, __uint_as_float(v[k + 120]));
      }
      const float mb =
          fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7])) * scale_log2;
      const bool move = __any_sync(0xffffffffu, mb > m_run + MOVE_LOG2);
      float alpha = 1.0f;
      if (move) {
        const float m_new = fmaxf(m_run, mb);
        alpha = m_new == -INFINITY ? 1.0f : ex2_fast(m_run - m_new);  // 0 on the first step
        l *= alpha;
        m_run = m_new;
        if (j > 0) {
          if constexpr (NT == 1) {  // the products of the step before may still be running
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done, (uint32_t)((j - 1) & 1), abort_flag, p.status,
                                                   STATUS_TIMEOUT, WAIT_NS));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(t_o + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x16(t_o + 16 * c, o);
          }
        }
      }
      // P = 2^(s scale - m), a row that has seen nothing yet in the frame 0
      const float m_use = m_run == -INFINITY ? 0.0f : m_run;
      const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-m_use, -m_use);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const int c = half * 64 + i;
          float a0, a1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nm2), a0, a1);
          const float p0 = ex2_fast(a0), p1 = ex2_fast(a1);
          v[c] = __float_as_uint(p0);
          v[c + 1] = __float_as_uint(p1);
          w[i >> 1] = pack_bf16(p0, p1);
        }
        tmem_st_32x32b_x32(t_s + 32 * half, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[slot][half]);
      }
      uint64_t ps[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ps[k] = f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
#pragma unroll
      for (int c = 8; c < 128; c += 2)
        ps[(c >> 1) & 3] = f2_add(ps[(c >> 1) & 3], f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])));
      float s0, s1;
      f2_unpack(f2_add(f2_add(ps[0], ps[1]), f2_add(ps[2], ps[3])), s0, s1);
      l += s0 + s1;
    }
    if (mine && (x == 0 || has_b)) {
      const int64_t row = (int64_t)blk.first + tk;
      const int head = h0 + hh;
      if (nkx > 0 && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], 0, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
      const bool none = nkx == 0;  // nothing seen: zeros
      if ((none || ok) && whole) {
        tc_fence_after();
        const float inv = blk.past < 0 ? 0.0f : vscale / l;
        if (stored && p.lse) p.lse[row * p.nq + head] = none ? -INFINITY : (m_run + log2f(l)) * 0.69314718055994531f;
        const int64_t off = stored ? row * p.ld_out + (int64_t)head * D : -1;
        // the warp's rows, turned in its part of the tile's queries, which are no longer needed
        uint8_t* stg = smem + x * C::QT + q4 * (C::QT / 4);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (!none) {
            tmem_ld_32x32b_x32(t_o + 32 * c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (!none)
              w = make_uint4(pack_bf16(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                             pack_bf16(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                             pack_bf16(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                             pack_bf16(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
            *reinterpret_cast<uint4*>(stg + lane * (D * 2) + (((4 * c + k) ^ (lane & 7)) << 4)) = w;
          }
        }
        __syncwarp();
        constexpr int CH = D / 8;  // 16-byte pieces of a row
        uint8_t* out = static_cast<uint8_t*>(p.out);
#pragma unroll 4
        for (int u = lane; u < 32 * CH; u += 32) {
          const int rr = u / CH, c = u % CH;
          const int64_t to = __shfl_sync(0xffffffffu, off, rr);
          if (to >= 0)
            *reinterpret_cast<uint4*>(out + 2 * to + 16 * c) =
                *reinterpret_cast<const uint4*>(stg + rr * (D * 2) + ((c ^ (rr & 7)) << 4));
        }
      } else if (none || ok) {  // a part: weighted values, maximum and sum
        tc_fence_after();
        const int64_t slot_b = slot_base(blk.first - blk.i * block_tok, blk.b, block_tok) + blk.i;
        float* part = p.part + ((slot_b * p.heads + hd) * p.nsplit + split) * (NT * 128) * (D + 2);
        const int rr = x * 128 + r;
        if (stored) {
          part[(size_t)NT * 128 * D + rr] = m_run;
          part[(size_t)NT * 128 * (D + 1) + rr] = l;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (!none) {
            tmem_ld_32x32b_x32(t_o + 32 * c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (stored)
              *reinterpret_cast<uint4*>(part + (size_t)rr * D + 32 * c + 4 * k) =
                  none ? make_uint4(0, 0, 0, 0) : make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
    }
  } else {
    // ------------------------------------------------- E4M3 codes to bf16
    if constexpr (F8) regs_dec<C::CONVERT_REGS>();
    constexpr int NRX = F8 ? NR : 1;
    const int tid = threadIdx.x - 128 * (1 + NT);
    bool ok = true;
    for (int at = 0; F8 && ok && at < 2 * nk * NE; ++at) {
      const int rs = at % NRX, s = at % NST;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(&raw_full[rs], (uint32_t)((at / NRX) & 1), abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS) &&
                          mbar_wait(&empty[s], (uint32_t)((at / NST) & 1) ^ 1u, abort_flag, p.status, STATUS_TIMEOUT,
                                    WAIT_NS));
      if (!ok) break;
#pragma unroll
      for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = tid + 128 * k, piece = u & 3, row = u >> 2;
          const uint4 c = *reinterpret_cast<const uint4*>(raw + rs * C::RB + cb * (KB * 64) + row * 64 + piece * 16);
          uint8_t* dst = ring + s * C::EB + cb * SUB + row * 128;
          *reinterpret_cast<uint4*>(dst + (((2 * piece) ^ (row & 7)) << 4)) =
              make_uint4(bf16_of_e4m3(c.x, false), bf16_of_e4m3(c.x, true), bf16_of_e4m3(c.y, false),
                         bf16_of_e4m3(c.y, true));
          *reinterpret_cast<uint4*>(dst + (((2 * piece + 1) ^ (row & 7)) << 4)) =
              make_uint4(bf16_of_e4m3(c.z, false), bf16_of_e4m3(c.z, true), bf16_of_e4m3(c.w, false),
                         bf16_of_e4m3(c.w, true));
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&raw_empty[rs]);
        mbar_arrive(&full[s]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the parts of split blocks, a warp a row and head, in the parts' order.
template <int D>
__global__ void __launch_bounds__(256) var_join_kernel(const FwdParams p) {
  constexpr int NT = D <= 128 ? 2 : 1, V = D / 64;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (id >= p.seq.rows * p.nq) return;
  const int row = (int)(id / p.nq), head = (int)(id % p.nq);
  const int block_tok = NT * p.tok;
  const int b = find_row(p.seq, row, lane);
  bool bad = false;
  const SeqSpan s = seq_span(p.seq, b, (int64_t)p.max_pages * p.page_size, &bad);
  if (row < s.first || row - s.first >= s.count) return;
  const int i = (row - s.first) / block_tok, tk = row - s.first - i * block_tok;
  Block k;
  fill_block(&k, s, b, i, p.tok, block_tok, p.window, p.sinks);
  const int per = part_steps(k.n, p.nsplit);
  if (per >= k.n) return;  // not split
  const int parts = (k.n + per - 1) / per;
  const int g = head / p.hpg, hc = (head - g * p.hpg) / p.ht, hh = head - g * p.hpg - hc * p.ht;
  const int rr = tk / p.tok * 128 + tk % p.tok * p.ht + hh;
  const int hd = g * p.chunks + hc;
  const size_t size = (size_t)NT * 128 * (D + 2);
  const float* base = p.part + ((int64_t)(slot_base(s.first, b, block_tok) + i) * p.heads + hd) * p.nsplit * size;
  // all lanes look at the parts' maxima, 32 at a time
  float top = -INFINITY;
  for (int q = lane; q < parts; q += 32) top = fmaxf(top, __ldcg(base + q * size + (size_t)NT * 128 * D + rr));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.0f : top;
  float2 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float2(0.0f, 0.0f);
  float sum = 0.0f;
#pragma unroll 4
  for (int q = 0; q < parts; ++q) {
    const float* src = base + q * size;
    const float w = ex2_fast(__ldcg(src + (size_t)NT * 128 * D + rr) - ref);
    sum = fmaf(w, __ldcg(src + (size_t)NT * 128 * (D + 1) + rr), sum);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 y = __ldcg(reinterpret_cast<const float2*>(src + (size_t)rr * D) + lane + 32 * v);
      acc[v].x = fmaf(w, y.x, acc[v].x);
      acc[v].y = fmaf(w, y.y, acc[v].y);
    }
  }
  const float inv = (p.v_inv_scale ? p.v_inv_scale[g] : 1.0f) / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + (int64_t)row * p.ld_out + (int64_t)head * D);
#pragma unroll
  for (int v = 0; v < V; ++v) out[lane + 32 * v] = pack_bf16(acc[v].x * inv, acc[v].y * inv);
  if (p.lse && lane == 0) p.lse[id] = (top + log2f(sum)) * 0.69314718055994531f;
}

// {64 columns, box slots} of a cache {d, page_size, nkv, pages}; E4M3 codes lie unswizzled, 64 bytes a row.
bool map_cache(CUtensorMap* m, const void* ptr, const VarFwdArgs& a, int box_tokens) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t e = a.e4m3 ? 1 : 2;
  cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page_size, (cuuint64_t)a.nkv, (cuuint64_t)a.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)a.stride_slot * e, (cuuint64_t)a.stride_head * e, (cuuint64_t)a.stride_page * e};
  cuuint32_t box[4] = {64, (cuuint32_t)box_tokens, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             a.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int SRC>
cudaError_t launch_one(FwdParams& p, const VarFwdArgs& a, int num_sms, cudaStream_t st) {
  using C = Cfg<D, SRC>;
  static_assert(C::SMEM + 1400 <= 232448, "shared memory");
  const int block_tok = C::NT * p.tok;
  const int64_t slots = a.seq.rows / block_tok + a.seq.batch;
  const int64_t units = slots * p.heads;
  if (units > 0x7fffffff / 2) return cudaErrorInvalidConfiguration;
  p.slots = (int)slots;
  p.nsplit = 1;
  if (SRC != PACKED && a.part && units * 2 <= num_sms) {
    const int most = num_sms < VAR_MAX_PARTS ? num_sms : VAR_MAX_PARTS;
    const int64_t steps = ((int64_t)a.max_pages * a.page_size + KB - 1) / KB;
    const int64_t parts = (steps + MIN_PART - 1) / MIN_PART;
    p.nsplit = (int)(most / units < parts ? most / units : parts);
    if (p.nsplit < 1) p.nsplit = 1;
  }
  p.by_length = units > num_sms && a.seq.batch <= LPT_BATCH;
  CUtensorMap mq, mk, mv;
  bool ok = map3(&mq, a.q, D, a.nq, a.seq.rows, a.ld_q, p.ht, p.tok);
  if (SRC == PACKED) {
    ok = ok && map3(&mk, a.k, D, a.nkv, a.seq.rows, a.ld_k, 1, KB) && map3(&mv, a.v, D, a.nkv, a.seq.rows, a.ld_v, 1, KB);
  } else {
    for (p.box = KB; a.page_size % p.box;) p.box /= 2;  // ends at 8 at the latest
    ok = ok && map_cache(&mk, a.k_cache, a, p.box) && map_cache(&mv, a.v_cache, a, p.box);
  }
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<var_fwd_kernel<D, SRC>>(C::SMEM);
  if (e == cudaSuccess) e = check_regs<var_fwd_kernel<D, SRC>>(C::THREADS, C::SOFTMAX_REGS > 0 ? C::REGS : 0);
  if (e != cudaSuccess) return e;
  var_fwd_kernel<D, SRC><<<(unsigned)(units * p.nsplit), C::THREADS, C::SMEM, st>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  var_join_kernel<D><<<(unsigned)((a.seq.rows * a.nq + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(FwdParams& p, const VarFwdArgs& a, int num_sms, cudaStream_t st) {
  if (!a.paged) return launch_one<D, PACKED>(p, a, num_sms, st);
  return a.e4m3 ? launch_one<D, PAGED_F8>(p, a, num_sms, st) : launch_one<D, PAGED>(p, a, num_sms, st);
}

}  // namespace

cudaError_t launch_var_fwd(const VarFwdArgs& a, int num_sms, cudaStream_t st) {
  FwdParams p{};
  p.seq = a.seq;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.lse = a.lse;
  p.part = a.part;
  p.nq = a.nq;
  p.nkv = a.nkv;
  p.hpg = a.nq / a.nkv;
  p.ht = p.hpg < 128 ? p.hpg : 128;
  p.chunks = (p.hpg + p.ht - 1) / p.ht;
  p.tok = 128 / p.ht;
  p.heads = a.nkv * p.chunks;
  // a scale of 0 keeps hidden scores at -inf
  p.negate = a.scale < 0.0f;
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;
  if (p.scale_log2 < 1e-30f) p.scale_log2 = 1e-30f;
  p.window = a.window;
  p.sinks = a.sinks;
  p.status = a.status;
  p.table = a.table;
  p.ld_table = a.ld_table;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.num_pages = a.num_pages;
  p.k_inv_scale = a.k_inv_scale;
  p.v_inv_scale = a.v_inv_scale;
  switch (a.d) {
    case 64: return launch_d<64>(p, a, num_sms, st);
    case 128: return launch_d<128>(p, a, num_sms, st);
    case 192: return launch_d<192>(p, a, num_sms, st);
    case 256: return launch_d<256>(p, a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tpmlp
