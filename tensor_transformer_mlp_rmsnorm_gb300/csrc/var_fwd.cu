// Attention of sequences of different lengths on the sm_103a tensor cores:
// whole packed sequences, or new tokens over a paged cache that holds them.
// For the token at position p, over the tokens t that it sees (t <= p; with a
// window, p - t < window or t < sinks):
//   s_t = scale q . k_t,  lse = log sum exp s_t,  out = sum exp(s_t - lse) v_t
//
// Rows.  The query heads of a key head see the same keys, so a tile of 128 rows
// holds the heads of one key head by 128 / heads tokens, and every key that is
// read serves them all.  Heads of 64 and 128 have two tiles at work, whose
// softmaxes hide under each other's products; heads of 192 and 256 leave room
// for one, with two score buffers.  A step is 128 keys: the longest block whose
// scores fit tensor memory beside the sums.
//
// Numbers.  S and O are 32-bit sums in tensor memory, m and l are 32 bits.  The
// maximum that P = 2^(s - m) refers to is moved only when it is off by more than
// 2^8: P stays below 2^8, l and O in range, and O is seldom rescaled.  P is
// rounded once, to bf16, as the products want it, and l sums what was not
// rounded: outputs are off by 0.0022 of their norm, where rounding the result
// alone gives 0.0017.  Hidden scores are -inf before the maximum is taken, and
// values that no row of the block sees are cleared in shared memory, so what a
// block does not see counts nothing, whatever it holds.  A value that one row of
// a block sees and another does not has the weight 0 for the other: one that is
// not finite makes NaN of that.  Blocks have at most 256 tokens.  E4M3 codes
// become bf16 exactly; their scales go into the scores' scale and the result.
//
// Work.  One CTA an SM takes blocks (two tiles) by a static order, longest
// first: times of causal blocks differ 100-fold.  The next block's copies, then
// its scores, run under the end of the one before.  Few rows over a long cache
// are cut along the cache: each part leaves its weighted sums, maximum and sum,
// and a second kernel joins them in order, so repeats give the same bits.
//
// Measured (GB300; 1947 TFLOP/s and 6678 GB/s are its product and copy rates), in
// replays of a captured graph; calls in a row, under the power cap, take 1586, 1540,
// 126, 470, 74 and 171 us:
//   one sequence of 16384 tokens, 32 + 8 heads of 128   1497 us, 1469 TFLOP/s
//   2 x 2048 tokens behind 30000, the same heads        1432 us, 1451 TFLOP/s
//   64 tokens behind 131000, the same heads              117 us, 4.6 TB/s and 1170 TFLOP/s
//   4 x 1024 tokens behind 7000, E4M3                    466 us, 1106 TFLOP/s
//   19 sequences, 8192 tokens                             73 us,  569 TFLOP/s of pairs that are seen
//   48 x 5 tokens behind up to 8192, E4M3                170 us, 2.5 TB/s
// What bounds them.  Long: a step of two tiles takes some 2800 to 3300 cycles
// where its products need 2080, the rest is the way between the issuing warp and
// the softmax (a wait that is fulfilled costs 150 cycles, a load from tensor
// memory beside products 300).  Short sequences: a block of one to four steps
// pays some 7000 cycles for its result (5000) and the next one's start, in which
// the tensor cores rest, and up to half of a step's keys are hidden.  E4M3: 16384
// codes an operand are converted by 128 threads, about 1500 cycles, which few rows
// do not hide.
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
// For a whole block (2^30 keys take some 13 s), and for the scheduler's next one, which it
// may find behind 2^20 empty sequences.
constexpr uint64_t BLOCK_NS = 60000000000ull;
constexpr float MOVE_LOG2 = 8.0f;  // the running maximum is moved when it is off by more than 2^8
// In place of a scale of 0: the smallest number there is, which keeps hidden scores at -inf
// and makes less than 10^-6 of the largest others.
constexpr float NO_SCALE = 1.4e-45f;
// Steps of a part at least: 64 tokens behind 131000 take 117 us with 2, 4 and 8 alike; 16
// behind 484, whose four steps are too few to cut, 16.6 with 2 (cut), 17.8 with 4 (not cut,
// and a second kernel that finds nothing to join) and 15.5 with 8 (one kernel).
constexpr int MIN_PART = 4;
// And of one of a last turn's blocks: 13 prompts behind 300 tokens take 112 us with 4, 106
// with 12 and with 24; 4 x 1024 behind 7000 in E4M3 463, 463 and 459.
constexpr int TAIL_PART = 12;
// Steps in the time of a part's start and result: 13 prompts 106 us with 2, 5 and 12;
// 4 x 1024 in E4M3 464, 463 and 460.
constexpr int PART_STEPS = 5;

enum Source { PACKED = 0, PAGED = 1, PAGED_F8 = 2 };

// FEW: blocks of one tile of rows, for sequences of few rows over long caches:
// both tiles take turns at the steps, and the room of the second tile's queries
// goes to copies in flight.
template <int D, int SRC, bool FEW>
struct Cfg {
  static constexpr bool F8 = SRC == PAGED_F8;
  static constexpr int NT = D <= 128 ? 2 : 1;         // tiles in tensor memory
  static constexpr int QTILES = FEW ? 1 : NT;         // query tiles of a block
  static constexpr int EC = D % 128 == 0 ? 128 : 64;  // columns of a ring element
  static constexpr int NE = D / EC;                   // elements of an operand
  static constexpr uint32_t EB = EC / 64 * SUB;       // bytes of an element
  static constexpr uint32_t QT = D / 64 * SUB;        // bytes of a query tile
  // E4M3 codes land in the space of the bf16 rows that are made of them, or, where the
  // copies are what counts, in a ring of their own that is free again once they are read.
  static constexpr bool RAW_RING = F8 && FEW;
  static constexpr int NRAW = RAW_RING ? 3 * 128 / EC : 0;
  static constexpr uint32_t RAW = NRAW * EB / 2;
  // Results are turned in shared memory, 128 bytes of a row at a time, where there is
  // room: a store of 16 bytes in each of 32 rows takes some 250 cycles.
  static constexpr bool STAGED = D != 256;
  static constexpr uint32_t STAGE = STAGED ? QTILES * 4 * 4096 : 0;
  static constexpr int FIT = (int)((225 * 1024 - QTILES * QT - STAGE - RAW) / EB);
  static constexpr int NST = FIT < 12 ? FIT : 12;     // ring stages
  // A turn at a step waits for its values and the tile's next keys, up to four operands on.
  static_assert(NST >= (NT == 2 ? 4 : 2) * NE, "ring");
  static constexpr int LAND = RAW_RING ? NRAW : NST;  // stages that copies land in
  static constexpr uint32_t SMEM = QTILES * QT + NST * EB + RAW + STAGE + 1024;
  static constexpr int WGS = 1 + NT + (F8 ? 1 : 0);   // issuing, softmax a tile, converting
  static constexpr int THREADS = 128 * WGS;
  static constexpr int READERS = 2 + 4 * NT + (F8 ? 4 : 0);  // warps that a piece of work is handed to
  // registers a thread after the exchange (0: none takes place)
  static constexpr int SOFTMAX_REGS = WGS == 4 ? 184 : WGS == 3 ? (F8 ? 232 : 208) : 0;
  static constexpr int ISSUE_REGS = WGS == 4 ? 80 : F8 ? 72 : 88;
  static constexpr int CONVERT_REGS = WGS == 4 ? 64 : 168;
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
  Slots slots;
  int heads;  // block slots, key heads times chunks
  // Blocks in order (slots times heads): those from `tail` on are shared by
  // nsplit CTAs each, in parts of at least min_part steps.
  int units;         // blocks and parts
  int tail, nsplit, min_part;
  bool by_length;
  float scale_log2;
  bool negate;
  bool out_boxes;  // 32 rows of a tile are a box of out
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

// Steps of a part of a shared block of n steps.
__device__ __forceinline__ int part_steps(const FwdParams& p, int n) {
  return max(p.min_part, (n + p.nsplit - 1) / p.nsplit);
}

// Block `rank` of the order in which blocks are taken, by the lanes of one warp; false: none.
__device__ __forceinline__ bool find_block(const FwdParams& p, ByLength<KB>& order, int rank, int block_tok, int64_t cap,
                                           int lane, Block* k) {
  int b, i = -1;
  if (p.by_length) order.find(rank, lane, &b, &i);
  else b = find_slot(p.seq, p.slots, (int)p.slots.count - 1 - rank, lane);
  if (b < 0) return false;
  bool bad = false;  // reported elsewhere
  const SeqSpan s = seq_span(p.seq, b, cap, &bad);
  if (!p.by_length) i = (int)p.slots.count - 1 - rank - slot_base(p.slots, s.first, b);
  if (i < 0 || (int64_t)i * block_tok >= s.count) return false;
  fill_block(k, s, b, i, p.tok, block_tok, p.window, p.sinks);
  return true;
}
__device__ __forceinline__ void start_order(const FwdParams& p, ByLength<KB>& order, int block_tok, int64_t cap,
                                            int lane) {
  if (p.by_length)
    order.init(p.seq, cap, block_tok,
               p.window > 0 ? (p.window + block_tok) / KB + 2 + (p.sinks + KB - 1) / KB : 0x7fffffff, lane);
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

// A piece of work: a block, or a part of its steps.
struct Work : Block {
  int part;        // its place among the parts
  int g, h0, nh;   // key head, first query head, query heads
  int j0, nk;      // steps [j0, j0 + nk) of the block
  int na, nb;      // those of the first and the second tile
  bool whole;      // all steps of the block
  bool dual;       // one tile of rows: the two tiles take turns at its steps
};
constexpr int NONE = -2;  // Work::b behind the last piece

template <int D, int SRC, bool FEW>
__global__ void __launch_bounds__(Cfg<D, SRC, FEW>::THREADS, 1)
    var_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const FwdParams p) {
  using C = Cfg<D, SRC, FEW>;
  constexpr int NT = C::NT, NE = C::NE, EC = C::EC, NST = C::NST;
  constexpr bool F8 = C::F8, RAW_RING = C::RAW_RING;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], full[NST], empty[NST], raw_full[F8 ? C::LAND : 1], raw_empty[RAW_RING ? C::LAND : 1], s_full[2],
      p_full[2][2], o_full[2], pv_done, post, taken, work_full[2], work_empty[2], drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ Work work_sh[2];
  __shared__ float2 other[NT == 2 ? 128 : 1];  // second tile's maximum and sum
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + C::QTILES * C::QT;
  uint8_t* raw = ring + NST * C::EB;
  volatile int* abort_flag = &abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cap = SRC == PACKED ? -1 : (int64_t)p.max_pages * p.page_size;
  const int block_tok = C::QTILES * p.tok;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], F8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; F8 && i < C::LAND; ++i) {
      mbar_init(&raw_full[i], 1);
      if (RAW_RING) mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 4);
      mbar_init(&p_full[i][1], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&work_full[i], 1);
      mbar_init(&work_empty[i], C::READERS);
    }
    mbar_init(&pv_done, 1);
    mbar_init(&post, 4);
    mbar_init(&taken, 4);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    tma_prefetch_desc(&map_o);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
  };
  // The t-th piece of this CTA's work, in shared memory until it is given back;
  // null behind the last.
  auto next = [&](int t) -> const Work* {
    if (!__all_sync(0xffffffffu, mbar_wait(&work_full[t & 1], (uint32_t)((t >> 1) & 1), abort_flag, p.status,
                                           STATUS_TIMEOUT, BLOCK_NS)))
      return nullptr;
    return work_sh[t & 1].b == NONE ? nullptr : &work_sh[t & 1];
  };
  auto give_back = [&](int t) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[t & 1]);
  };
  // Where a step's operands lie in the ring, in the order that they are used,
  // from `base` on: the elements of the pieces before.
  auto k_at = [&](int base, const Work& w, int j) -> int {
    return base + (NT == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1) * NE;
  };
  auto v_at = [&](int base, const Work& w, int j) -> int {
    return base + (NT == 2 ? 2 * j + 1 : j < w.nk - 1 ? 2 * j + 2 : 2 * w.nk - 1) * NE;
  };

  // Registers: what the issuing and converting warpgroups give up, the softmax
  // takes.  Every warp passes the exchange, with or without work: an increase
  // waits until the others have given theirs up.
  if (warp < 4) {
    if constexpr (C::SOFTMAX_REGS > 0) regs_dec<C::ISSUE_REGS>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      constexpr int CB = EC / 64;  // 64-column boxes of an element's row
      const int boxes = SRC == PACKED ? 1 : KB / p.box;
      const int my_box = lane / CB, my_col = lane % CB;
      const bool issues = my_box < boxes;
      // E4M3 codes land in the upper half of the space of the bf16 rows that the same warp makes of them
      const int row0 = my_box * p.box;
      const uint32_t my_dst = RAW_RING ? my_col * (KB * 64) + row0 * 64
                              : my_col * SUB + (SRC == PACKED ? 0 : F8 ? row0 / 32 * 4096 + 2048 + row0 % 32 * 64 : row0 * 128);
      uint64_t *land = F8 ? raw_full : full, *room = RAW_RING ? raw_empty : empty;
      uint8_t* land_at = RAW_RING ? raw : ring;
      constexpr uint32_t LAND_BYTES = RAW_RING ? C::EB / 2 : C::EB;
      uint32_t armed = 0, par_armed = 0;  // by stage
      uint32_t q_a = 0, q_b = 0;          // pieces whose queries are in each tile
      bool ok = true;
      const Work* wp;
      for (int t = 0, base = 0; ok && (wp = next(t)); give_back(t++)) {
        const Work& w = *wp;
        const int g = w.g, h0 = w.h0;
        // Page of this lane's box in a step, asked for a step ahead and looked at when it is
        // used; num_pages (nothing is read, zeros land) where no row sees the box.
        const int no_page = (int)p.num_pages;
        bool seen = false;  // of the page that was asked for last
        auto look = [&](int j) -> int {
          const int at = w.tile(w.j0 + j) * KB + row0, pi = at / p.page_size;
          seen = issues && ((at < w.end && at + p.box > w.lo) || at < w.sink_end);
          if (!seen) return no_page;
          return pi < p.max_pages ? __ldg(p.table + (int64_t)w.b * p.ld_table + pi) : -1;
        };
        auto valid = [&](int page) -> int {
          if ((uint32_t)page < (uint32_t)no_page) return page;
          if (seen) atomicOr(p.status, STATUS_BAD_INDEX);
          return no_page;
        };
        auto load = [&](int at, const CUtensorMap* map, int j, int page) -> bool {
          const int tile = w.tile(w.j0 + j);
          for (int e = 0; e < NE; ++e, ++at) {
            const int s = at % C::LAND;
            const uint32_t par = (uint32_t)((at / C::LAND) & 1);
            if (!wait_all(&room[s], par ^ 1u)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&land[s], F8 ? C::EB / 2 : C::EB);
            __syncwarp();
            armed |= 1u << s;
            par_armed = (par_armed & ~(1u << s)) | (par << s);
            if (issues) {
              const int col = e * EC + my_col * 64;
              uint8_t* dst = land_at + s * LAND_BYTES + my_dst;
              if constexpr (SRC == PACKED) tma_load_3d(dst, map, &land[s], col, g, w.first - w.i * block_tok + tile * KB);
              else tma_load_4d(dst, map, &land[s], col, (tile * KB + row0) % p.page_size, g, page);
            }
          }
          return true;
        };
        int page = 0, page_n = 0, page_v = 0;
        if (w.nk > 0) {
          if constexpr (SRC != PACKED) {
            page = valid(look(0));
            if (w.nk > 1) page_n = look(1);
          }
          ok = load(k_at(base, w, 0), &map_k, 0, page);
          auto queries = [&](int x, uint32_t n) -> bool {
            if (!wait_all(&q_empty[x], (n & 1u) ^ 1u)) return false;
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full[x], (uint32_t)(D / 64 * p.ht * p.tok * 128));
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(smem + x * C::QT + c * SUB, &map_q, &q_full[x], 64 * c, h0, w.first + x * p.tok);
            }
            __syncwarp();
            return true;
          };
          if (ok && w.na > 0) ok = queries(0, q_a++);
          if (NT == 2 && ok && w.nb > 0 && !w.dual) ok = queries(1, q_b++);
        }
        for (int j = 0; ok && j < w.nk; ++j) {
          if (j > 0) {
            if constexpr (SRC != PACKED) {
              page = valid(page_n);
              if (j + 1 < w.nk) page_n = look(j + 1);
            }
            ok = load(k_at(base, w, j), &map_k, j, page);
          }
          if constexpr (NT == 2) {
            if (ok) ok = load(v_at(base, w, j), &map_v, j, page);
          } else {  // the values one step behind
            if (ok && j > 0) ok = load(v_at(base, w, j - 1), &map_v, j - 1, page_v);
            page_v = page;
          }
        }
        if constexpr (NT == 1)
          if (ok && w.nk > 0) ok = load(v_at(base, w, w.nk - 1), &map_v, w.nk - 1, page_v);
        base += 2 * w.nk * NE;
      }
      if (!ok || *abort_flag) {  // copies still in flight land on the barriers armed last
        int no_abort = 0;
        if (q_a) mbar_wait(&q_full[0], (q_a - 1) & 1u, &no_abort, p.status, 0u, DRAIN_NS);
        if (q_b) mbar_wait(&q_full[1], (q_b - 1) & 1u, &no_abort, p.status, 0u, DRAIN_NS);
        for (int s = 0; s < C::LAND; ++s)
          if (armed & (1u << s)) mbar_wait(&land[s], (par_armed >> s) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 8);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- issuer
      // A wait takes some 150 cycles although what it waits for is there: the
      // copies are waited for before the row groups, so that a tile's second
      // half of P V and its next scores are issued together.
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, KB, false, false);
      constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, EC, false, true);
      const uint64_t q_desc = sw128_desc(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = sw128_desc(smem_u32(ring), 16, 1024);
      const uint64_t v_desc = sw128_desc(smem_u32(ring), SUB, 1024);
      auto wait_elems = [&](int at) -> bool {
        bool r = true;
#pragma unroll
        for (int e = 0; e < NE; ++e) r = r && wait_all(&full[(at + e) % NST], (uint32_t)(((at + e) / NST) & 1));
        return r;
      };
      // S = Q K_j^T into score slot `slot`, with the queries of tile `qt`; the last user of a ring element frees it
      auto mma_s = [&](int qt, int slot, int at, bool last) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const int s = (at + e) % NST;
          const uint64_t kb = desc_advance(k_desc, s * C::EB), qa = desc_advance(q_desc, qt * C::QT + e * C::EB);
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
          if (half == 1 && last) tc_commit(&empty[s]);
        }
      };
      uint32_t q_a = 0, q_b = 0, steps_a = 0, steps_b = 0;  // queries and steps of each tile so far
      bool ok = true;
      const Work* wp;
      for (int t = 0, base = 0; ok && (wp = next(t)); give_back(t++)) {
        const Work& w = *wp;
        if constexpr (NT == 2) {
          const int na = w.na, nb = w.nb, nk = w.nk, most = max(na, nb);
          const bool dual = w.dual;
          // Elements of the ring that are there.  With two tiles of rows each one is waited
          // for in order, by the tile that comes first.  Turns at the steps go out of
          // order, and copies land out of order: each is waited for by the one that uses it.
          int seen = base;
          auto there = [&](int at) -> bool {
            if (!dual && at < seen) return true;
            if (!wait_elems(at)) return false;
            seen = at + NE;
            return true;
          };
          auto step = [&](int x, int i) -> int { return dual ? 2 * i + x : i; };
          auto put_s = [&](int x, int i) {
            const int mine = x ? nb : na, j = step(x, i);
            mma_s(x && !dual ? 1 : 0, x, k_at(base, w, j), dual || x == 1 || i >= nb);
            if (dual ? j == nk - 1 : i == mine - 1) tc_commit(&q_empty[x && !dual ? 1 : 0]);
          };
          auto first = [&](int x) -> bool {
            if (!there(k_at(base, w, step(x, 0)))) return false;
            tc_fence_after();
            if (elect_one()) put_s(x, 0);
            __syncwarp();
            return true;
          };
          // tile x's i-th step: O += P V, and the next step's scores
          auto turn = [&](int x, int i, uint32_t par) -> bool {
            const int mine = x ? nb : na, at = v_at(base, w, step(x, i));
            const bool more = i + 1 < mine, last = dual || x == 1 || i >= nb;
            if (!there(at) || (more && !there(k_at(base, w, step(x, i + 1))))) return false;
            if (!wait_all(&p_full[x][0], par)) return false;
            tc_fence_after();
            if (elect_one()) mma_pv(x, x, at, 0, i == 0, last);
            __syncwarp();
            if (!wait_all(&p_full[x][1], par)) return false;
            tc_fence_after();
            if (elect_one()) {
              mma_pv(x, x, at, 1, i == 0, last);
              if (more) put_s(x, i + 1);
              else tc_commit(&o_full[x]);
            }
            __syncwarp();
            return true;
          };
          if (na > 0) ok = wait_all(&q_full[0], q_a++ & 1u) && first(0);
          if (ok && nb > 0) ok = (dual || wait_all(&q_full[1], q_b++ & 1u)) && first(1);
#pragma unroll 1
          for (int i = 0; ok && i < most; ++i) {
            if (i < na) ok = turn(0, i, (steps_a + i) & 1u);
            if (ok && i < nb) ok = turn(1, i, (steps_b + i) & 1u);
          }
          steps_a += na;
          steps_b += nb;
        } else if (w.nk > 0) {
          auto scores = [&](int j) -> bool {
            const int at = k_at(base, w, j);
            if (!wait_elems(at)) return false;
            tc_fence_after();
            if (elect_one()) {
              mma_s(0, (steps_a + j) & 1, at, true);
              if (j == w.nk - 1) tc_commit(&q_empty[0]);
            }
            __syncwarp();
            return true;
          };
          ok = wait_all(&q_full[0], q_a++ & 1u) && scores(0);
          for (int j = 0; ok && j < w.nk; ++j) {
            const uint32_t n = steps_a + j;
            const int slot = n & 1, at = v_at(base, w, j);
            if (j + 1 < w.nk && !(ok = scores(j + 1))) break;
            if (!(ok = wait_elems(at))) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!(ok = wait_all(&p_full[slot][half], (n >> 1) & 1u))) break;
              tc_fence_after();
              if (elect_one()) {
                mma_pv(0, slot, at, half, j == 0, true);
                if (half == 1) {
                  tc_commit(&pv_done);
                  if (j + 1 == w.nk) tc_commit(&o_full[0]);
                }
              }
              __syncwarp();
            }
          }
          steps_a += w.nk;
        }
        base += 2 * w.nk * NE;
      }
      if (elect_one()) tc_commit(&drain_bar);
      __syncwarp();
      int no_abort = 0;
      mbar_wait(&drain_bar, 0, &no_abort, p.status, STATUS_TIMEOUT, DRAIN_NS);
    } else if (warp == 2) {
      // ----------------------------------------------------------- scheduler
      ByLength<KB> order;
      start_order(p, order, block_tok, cap, lane);
      bool ok = true;
      int t = 0;
      for (int k = 0; ok; ++k) {
        const int64_t u = snake(k, (int)blockIdx.x, (int)gridDim.x);
        const bool end = (int64_t)k * gridDim.x >= p.units;
        Work w;
        w.b = NONE;
        if (!end) {
          if (u >= p.units) continue;
          int unit = (int)u, split = 0;
          const bool shared = unit >= p.tail;
          w.part = unit - p.tail;
          if (shared) {
            split = w.part % p.nsplit;
            unit = p.tail + w.part / p.nsplit;
          }
          const int hd = unit % p.heads;
          w.g = hd / p.chunks;
          w.h0 = w.g * p.hpg + hd % p.chunks * p.ht;
          w.nh = min(p.ht, (w.g + 1) * p.hpg - w.h0);
          if (!find_block(p, order, unit / p.heads, block_tok, cap, lane, &w)) {
            // An empty slot is one of all key heads: on with the next slot.  (Sequences are not
            // passed over many at a time: the code for that cost 1 to 2% of every call.)
            k = max(k, (unit / p.heads + 1) * p.heads / (int)gridDim.x - 1);
            continue;
          }
          const int per = shared ? part_steps(p, w.n) : w.n;
          w.j0 = split * per;
          if (split > 0 && w.j0 >= w.n) continue;
          w.whole = per >= w.n;
          w.nk = min(w.n, w.j0 + per) - w.j0;
          w.dual = NT == 2 && (FEW || w.count <= p.tok) && w.nk > 1;
          if (w.dual) {
            w.na = (w.nk + 1) / 2;
            w.nb = w.nk / 2;
          } else {
            w.na = max(0, min(w.n_a, w.j0 + per) - w.j0);
            w.nb = NT == 2 && w.count > p.tok ? w.nk : 0;
          }
        }
        const int q = t & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&work_empty[q], (uint32_t)((t >> 1) & 1) ^ 1u, abort_flag, p.status,
                                               STATUS_TIMEOUT, BLOCK_NS));
        if (ok && lane == 0) {
          work_sh[q] = w;
          mbar_arrive(&work_full[q]);
        }
        __syncwarp();
        ++t;
        if (end) break;
      }
      report_bad(p.seq, cap, p.status, lane);
    }
  } else if (warp < 4 + 4 * NT) {
    // --------------------------------------------------------------- softmax
    if constexpr (C::SOFTMAX_REGS > 0) regs_inc<C::SOFTMAX_REGS>();
    const int x = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t t_o = tmem_base + lane_off + 256 + x * D;
    const int tok_r = r / p.ht, hh = r - tok_r * p.ht;  // token in the tile, head
    uint8_t* stg = raw + C::RAW + (FEW ? warp & 3 : warp - 4) * 4096;
    // before the warp's staging space is written: what a bulk copy reads there
    auto stage_free = [&]() {
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
    };
    uint32_t steps = 0, outs = 0, duals = 0;  // of this tile so far
    bool ok = true;
    const Work* wp;
    for (int t = 0, base = 0; ok && (wp = next(t)); give_back(t++)) {
      const Work& w = *wp;
      const int nkx = x ? w.nb : w.na;
      const int xt = w.dual ? 0 : x;         // tile of rows
      const int tk = xt * p.tok + tok_r;     // token in the block
      const bool stored = r < p.tok * p.ht && hh < w.nh && tk < w.count;
      const int pos = w.past + tk;
      const int pos_first = w.past + xt * p.tok, pos_last = w.past + min(w.count, (xt + 1) * p.tok) - 1;
      float scale_log2 = p.scale_log2, vscale = 1.0f;
      if constexpr (F8) {
        if (p.k_inv_scale) scale_log2 *= p.k_inv_scale[w.g];
        if (scale_log2 == 0.0f) scale_log2 = NO_SCALE;
        if (p.v_inv_scale) vscale = p.v_inv_scale[w.g];
      }
      float m_run = -INFINITY, l = 0.0f;
      for (int i = 0; ok && i < nkx; ++i) {
        const int j = w.dual ? 2 * i + x : i;
        const uint32_t n = steps + i;
        const int slot = NT == 2 ? x : n & 1;
        const uint32_t t_s = tmem_base + lane_off + slot * KB;
        const int t0 = w.tile(w.j0 + j) * KB;
        if (!(ok = wait_all(&s_full[slot], NT == 2 ? n & 1 : (n >> 1) & 1))) break;
        tc_fence_after();
        // values that no row of the block sees: cleared, so that they count nothing whatever they are
        if (t0 + KB > w.end || (t0 < w.lo && t0 + KB > w.sink_end)) {
          // (A wait for a ring stage is good for the next phase only: what was in
          // the stage before has landed, as the scores of this step and, with two
          // score slots, the products of the one before are complete.)
          if constexpr (NT == 1)
            if (n > 0) ok = wait_all(&pv_done, (n - 1) & 1u);
          const int at = v_at(base, w, j);
          const int tt = t0 + r;
          const bool clear = tt >= w.end || (tt < w.lo && tt >= w.sink_end);
          for (int e = 0; ok && e < NE; ++e) {
            const int s = (at + e) % NST;
            ok = wait_all(&full[s], (uint32_t)(((at + e) / NST) & 1));
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
        if (t0 + KB - 1 > pos_first || (p.window > 0 && pos_last - t0 >= p.window && t0 + KB > p.sinks)) {
          // What the row sees as bits, 32 columns a word: two instructions a column, and
          // none for the words that every row of the warp sees whole.
          const int hi = pos - t0 + 1;                                // keys c < hi
          const int lo = p.window > 0 ? pos + 1 - p.window - t0 : 0;  // and c >= lo
          const int sk = p.window > 0 ? p.sinks - t0 : 0;             // or c < sk
#pragma unroll
          for (int c0 = 0; c0 < KB; c0 += 32) {
            const uint32_t bits = below(hi - c0) & (~below(lo - c0) | below(sk - c0));
            if (__any_sync(0xffffffffu, bits != ~0u)) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits & (1u << c))) v[c0 + c] = 0xff800000u;  // -inf
            }
          }
        }
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float m = __uint_as_float(v[k]);
#pragma unroll
          for (int c = 1; c < 15; c += 2) m = fmax3(m, __uint_as_float(v[k + 8 * c]), __uint_as_float(v[k + 8 * c + 8]));
          mx[k] = fmaxf(m, __uint_as_float(v[k + 120]));
        }
        const float mb =
            fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7])) * scale_log2;
        // Lanes without a result have no say: their queries are other sequences', nobody's or
        // no copy's, and the frame that P is rounded in must not depend on those.
        const bool move = __any_sync(0xffffffffu, stored && mb > m_run + MOVE_LOG2);
        if (move) {
          const float m_new = fmaxf(m_run, mb);
          const float alpha = m_new == -INFINITY ? 1.0f : ex2_fast(m_run - m_new);  // 0 on the first step
          l *= alpha;
          m_run = m_new;
          if (i > 0) {
            if constexpr (NT == 1) {  // the products of the step before may still be running
              if (!(ok = wait_all(&pv_done, (n - 1) & 1u))) break;
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
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const int c = half * 64 + e;
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nm2), a0, a1);
            const float p0 = ex2_fast(a0), p1 = ex2_fast(a1);
            v[c] = __float_as_uint(p0);
            v[c + 1] = __float_as_uint(p1);
            pk[e >> 1] = pack_bf16(p0, p1);
          }
          tmem_st_32x32b_x32(t_s + 32 * half, pk);
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
      steps += nkx;
      base += 2 * w.nk * NE;
      if (!ok) break;
      if (nkx > 0) {
        if (!(ok = wait_all(&o_full[x], outs++ & 1u))) break;
        tc_fence_after();
      }
      // ---- the piece's result
      float fa = 1.0f, fb = 0.0f;  // weights of the two tiles' values
      if (NT == 2 && w.dual) {
        const uint32_t par = duals++ & 1u;
        if (x == 1) {  // the first tile's warps take the second's values too
          other[r] = make_float2(m_run, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&post);
          if (!(ok = wait_all(&taken, par))) break;
          tc_fence_after();
          continue;
        }
        if (!(ok = wait_all(&post, par))) break;
        tc_fence_after();
        const float2 o = other[r];
        const float top = fmaxf(m_run, o.x), ref = top == -INFINITY ? 0.0f : top;
        fa = ex2_fast(m_run - ref);
        fb = ex2_fast(o.x - ref);
        l = fa * l + fb * o.y;
        m_run = top;
      } else if (x == 1 && w.count <= p.tok) {
        continue;  // no second tile
      }
      const bool none = nkx == 0;  // nothing seen: zeros
      const float inv = none ? 0.0f : vscale / l;
      const int64_t row = (int64_t)w.first + tk;
      const int rr = xt * 128 + r;
      uint8_t* dst = nullptr;
      if (w.whole) {
        const int head = w.h0 + hh;
        if (stored) {
          if (p.lse) p.lse[row * p.nq + head] = none ? -INFINITY : (m_run + log2f(l)) * 0.69314718055994531f;
          dst = reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + (int64_t)head * D);
        }
        fa *= inv;
        fb *= inv;
      } else {  // a part: weighted values, maximum and sum
        float* part = p.part + (int64_t)w.part * (C::QTILES * 128) * (D + 2);
        if (stored) {
          part[(size_t)C::QTILES * 128 * D + rr] = m_run;
          part[(size_t)C::QTILES * 128 * (D + 1) + rr] = l;
          dst = reinterpret_cast<uint8_t*>(part + (size_t)rr * D);
        }
      }
      // A warp whose 32 rows are all results hands them to a bulk copy; the others' rows
      // of other sequences, or of nobody, lie between theirs in memory.
      if constexpr (C::STAGED) {
        if (w.whole && !(NT == 2 && w.dual)) {  // 64 columns at a time, the next ones on their way
          const bool bulk = p.out_boxes && __all_sync(0xffffffffu, stored);
          uint32_t o[64];
          tmem_ld_32x32b_x32(t_o, *reinterpret_cast<uint32_t(*)[32]>(o));
          tmem_ld_32x32b_x32(t_o + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t u[32];
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              u[e] = none ? 0u : pack_bf16(fa * __uint_as_float(o[2 * e]), fa * __uint_as_float(o[2 * e + 1]));
            if (c + 64 < D) {
              tmem_ld_32x32b_x32(t_o + c + 64, *reinterpret_cast<uint32_t(*)[32]>(o));
              tmem_ld_32x32b_x32(t_o + c + 96, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
            }
            stage_free();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                  make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
            if (bulk) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&map_o, stg, c, w.h0, w.first + xt * p.tok + q4 * 32 / p.ht);
                bulk_commit_group();
              }
              continue;
            }
            __syncwarp();
            const int64_t to = dst ? reinterpret_cast<int64_t>(dst) + 2 * c : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int y = 4 * k + lane / 8, piece = lane & 7;
              const int64_t at = __shfl_sync(0xffffffffu, to, y);
              const uint4 z = *reinterpret_cast<const uint4*>(stg + y * 128 + ((piece ^ (y & 7)) << 4));
              if (at) *reinterpret_cast<uint4*>(at + 16 * piece) = z;
            }
            __syncwarp();
          }
          continue;
        }
      }
      // 32 columns at a time: a load from tensor memory takes some 300 cycles beside
      // the other tile's products whatever its size
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(t_o + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(fa * __uint_as_float(o[e]));
        if (NT == 2 && w.dual) {
          uint32_t y[32];
          tmem_ld_32x32b_x32(t_o + D + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(fb, __uint_as_float(y[e]), __uint_as_float(o[e])));
        }
        int pieces = 8;  // 16-byte pieces of o
        if (w.whole) {
          pieces = 4;
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        }
        if constexpr (C::STAGED) {
          if (c == 0) stage_free();
          const int k0 = w.whole ? (c & 32) >> 3 : 0;  // piece of the 128 bytes
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < pieces)
              *reinterpret_cast<uint4*>(stg + lane * 128 + (((k0 + k) ^ (lane & 7)) << 4)) =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (w.whole && !(c & 32)) continue;  // not yet full
          __syncwarp();
          const int64_t to = reinterpret_cast<int64_t>(dst) + (w.whole ? 2 * (c - 32) : 4 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int y = 4 * k + lane / 8, piece = lane & 7;
            const int64_t at = __shfl_sync(0xffffffffu, dst ? to : 0, y);
            const uint4 u = *reinterpret_cast<const uint4*>(stg + y * 128 + ((piece ^ (y & 7)) << 4));
            if (at) *reinterpret_cast<uint4*>(at + 16 * piece) = u;
          }
          __syncwarp();
        } else if (dst) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < pieces)
              reinterpret_cast<uint4*>(dst + (w.whole ? 2 : 4) * c)[k] =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        __syncwarp();
      }
      if (NT == 2 && w.dual) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken);
      }
    }
    if (C::STAGED && lane == 0) bulk_wait_read_all();  // shared memory goes with the CTA
  } else {
    // ------------------------------------------------- E4M3 codes to bf16
    if constexpr (F8) {
      regs_dec<C::CONVERT_REGS>();
      const int cw = warp - 4 - 4 * NT;
      bool ok = true;
      const Work* wp;
      for (int t = 0, at = 0; ok && (wp = next(t)); give_back(t++)) {
        const int end = at + 2 * wp->nk * NE;
        for (; ok && at < end; ++at) {
          const int s = at % NST, rs = at % C::LAND;
          if (!(ok = wait_all(&raw_full[rs], (uint32_t)((at / C::LAND) & 1)))) break;
          // 32 rows of the tile; their codes in a ring of their own, or in the upper half of their space
          uint8_t* mine = ring + s * C::EB + cw * 4096;
          const uint8_t* codes = RAW_RING ? raw + rs * (C::EB / 2) + cw * 2048 : mine + 2048;
          uint4 c[EC / 64][4];
#pragma unroll
          for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              c[cb][k] = *reinterpret_cast<const uint4*>(codes + cb * (RAW_RING ? KB * 64 : SUB) + (lane + 32 * k) * 16);
          if (RAW_RING) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[rs]);
            if (!(ok = wait_all(&empty[s], (uint32_t)((at / NST) & 1) ^ 1u))) break;
          }
          __syncwarp();
#pragma unroll
          for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int piece = lane & 3, row = (lane >> 2) + 8 * k;
              uint8_t* dst = mine + cb * SUB + row * 128;
              const uint4 y = c[cb][k];
              *reinterpret_cast<uint4*>(dst + (((2 * piece) ^ (row & 7)) << 4)) =
                  make_uint4(bf16_of_e4m3(y.x, false), bf16_of_e4m3(y.x, true), bf16_of_e4m3(y.y, false),
                             bf16_of_e4m3(y.y, true));
              *reinterpret_cast<uint4*>(dst + (((2 * piece + 1) ^ (row & 7)) << 4)) =
                  make_uint4(bf16_of_e4m3(y.z, false), bf16_of_e4m3(y.z, true), bf16_of_e4m3(y.w, false),
                             bf16_of_e4m3(y.w, true));
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
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

// Joins the parts of shared blocks, a warp a row and head, in the parts' order.
template <int D>
__global__ void __launch_bounds__(256) var_join_kernel(const FwdParams p, int tiles) {
  constexpr int V = D / 64;
  const int lane = threadIdx.x & 31;
  const int block_tok = tiles * p.tok, at = (int)blockIdx.x / (16 * tiles);  // place among the shared blocks
  const int rr = (int)blockIdx.x % (16 * tiles) * 8 + (threadIdx.x >> 5), r = rr & 127;
  const int unit = p.tail + at, hd = unit % p.heads, g = hd / p.chunks;
  const int tk = (rr >> 7) * p.tok + r / p.ht, head = g * p.hpg + hd % p.chunks * p.ht + r % p.ht;
  if (r >= p.tok * p.ht || head >= (g + 1) * p.hpg) return;
  const int64_t cap = (int64_t)p.max_pages * p.page_size;
  ByLength<KB> order;
  start_order(p, order, block_tok, cap, lane);
  Block k;
  if (!find_block(p, order, unit / p.heads, block_tok, cap, lane, &k) || tk >= k.count) return;
  const int per = part_steps(p, k.n);
  if (per >= k.n) return;  // one CTA's
  const int parts = (k.n + per - 1) / per;
  const int64_t row = (int64_t)k.first + tk;
  const size_t size = (size_t)tiles * 128 * (D + 2);
  const float* base = p.part + (int64_t)at * p.nsplit * size;
  // all lanes look at the parts' maxima, 32 at a time
  float top = -INFINITY;
  for (int q = lane; q < parts; q += 32) top = fmaxf(top, __ldcg(base + q * size + (size_t)tiles * 128 * D + rr));
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
    const float w = ex2_fast(__ldcg(src + (size_t)tiles * 128 * D + rr) - ref);
    sum = fmaf(w, __ldcg(src + (size_t)tiles * 128 * (D + 1) + rr), sum);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 y = __ldcg(reinterpret_cast<const float2*>(src + (size_t)rr * D) + lane + 32 * v);
      acc[v].x = fmaf(w, y.x, acc[v].x);
      acc[v].y = fmaf(w, y.y, acc[v].y);
    }
  }
  const float inv = (p.v_inv_scale ? p.v_inv_scale[g] : 1.0f) / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + (int64_t)head * D);
#pragma unroll
  for (int v = 0; v < V; ++v) out[lane + 32 * v] = pack_bf16(acc[v].x * inv, acc[v].y * inv);
  if (p.lse && lane == 0) p.lse[row * p.nq + head] = (top + log2f(sum)) * 0.69314718055994531f;
}

// {64 columns, box slots} of a cache {d, page_size, nkv, pages}; E4M3 codes lie unswizzled, 64 bytes a row.
bool map_cache(CUtensorMap* m, const void* ptr, const VarFwdArgs& a, int box_tokens) {
  const cuuint64_t e = a.e4m3 ? 1 : 2;
  cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page_size, (cuuint64_t)a.nkv, (cuuint64_t)a.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)a.stride_slot * e, (cuuint64_t)a.stride_head * e, (cuuint64_t)a.stride_page * e};
  cuuint32_t box[4] = {64, (cuuint32_t)box_tokens, 1, 1};
  return encode_tiled(m, a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, ptr, dims, strides,
                      box, a.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int SRC, bool FEW>
cudaError_t launch_one(FwdParams& p, const VarFwdArgs& a, int num_sms, cudaStream_t st) {
  using C = Cfg<D, SRC, FEW>;
  static_assert(C::SMEM + 900 + (C::NT == 2 ? 1024 : 0) <= 232448, "shared memory");
  p.slots = make_slots(a.seq, C::QTILES * p.tok);
  const int64_t units = p.slots.count * p.heads;
  if (units > VAR_MAX_BLOCKS) return cudaErrorInvalidConfiguration;  // var_fits
  // Few blocks: all are shared.  Many: the CTAs take them in turns, and a last turn
  // with work for less than half of them shares out its blocks, which are the shortest.
  // What is counted are slots: the lengths are on the device, and with sequences of
  // different ones a last turn may be empty slots, with nothing to share.
  // (With more the parts' own time is what it costs: 48 x 5 tokens behind up to 8192 in
  // E4M3, 80 blocks left, 169 us without and 185 with.)  A part takes its steps and the
  // time of PART_STEPS more; the number of parts is the one that ends first.
  // 2 x 2048 tokens behind 30000 (512 blocks for 152 CTAs): 1651 us without, 1431 with;
  // 4 x 1024 behind 7000 in E4M3: 493 and 461.  More than one turn of parts has to be 5%
  // better by that count; without the margin 13 prompts take 106 us as with it.
  p.tail = (int)units;
  p.nsplit = 1;
  p.min_part = units > num_sms ? TAIL_PART : MIN_PART;
  if (SRC != PACKED && a.part) {
    const int64_t steps = ((int64_t)a.max_pages * a.page_size + KB - 1) / KB;
    const int64_t last = units % num_sms, left = units <= num_sms ? units : last * 2 <= num_sms ? last : 0;
    const int64_t room = a.part_floats / ((size_t)C::QTILES * 128 * (D + 2));  // parts
    const int64_t most = (steps + p.min_part - 1) / p.min_part;
    int64_t best = steps + PART_STEPS;
    for (int64_t n = 2; left > 0 && n <= most && n * left <= room; ++n) {
      const int64_t turns = (n * left + num_sms - 1) / num_sms, time = turns * ((steps + n - 1) / n + PART_STEPS);
      if (turns == 1 ? time < best : time * 20 < best * 19) {
        best = time;
        p.nsplit = (int)n;
      }
    }
    if (p.nsplit > 1) p.tail = (int)(units - left);
  }
  p.by_length = units > num_sms && a.seq.batch <= LPT_BATCH;
  p.units = (int)(p.tail + (units - p.tail) * p.nsplit);
  CUtensorMap mq, mk, mv, mo;
  p.out_boxes = 32 % p.ht == 0;
  bool ok = map3(&mo, a.out, D, a.nq, a.seq.rows, a.ld_out, p.out_boxes ? p.ht : 1, p.out_boxes ? 32 / p.ht : 32);
  ok = ok && map3(&mq, a.q, D, a.nq, a.seq.rows, a.ld_q, p.ht, p.tok);
  if (SRC == PACKED) {
    ok = ok && map3(&mk, a.k, D, a.nkv, a.seq.rows, a.ld_k, 1, KB) && map3(&mv, a.v, D, a.nkv, a.seq.rows, a.ld_v, 1, KB);
  } else {
    for (p.box = C::F8 ? 32 : KB; a.page_size % p.box;) p.box /= 2;  // ends at 8 at the latest
    ok = ok && map_cache(&mk, a.k_cache, a, p.box) && map_cache(&mv, a.v_cache, a, p.box);
  }
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<var_fwd_kernel<D, SRC, FEW>>(C::SMEM);
  if (e == cudaSuccess) e = check_regs<var_fwd_kernel<D, SRC, FEW>>(C::THREADS, C::SOFTMAX_REGS > 0 ? C::REGS : 0);
  if (e != cudaSuccess) return e;
  var_fwd_kernel<D, SRC, FEW><<<p.units < num_sms ? p.units : num_sms, C::THREADS, C::SMEM, st>>>(mq, mk, mv, mo, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  if (a.launches) ++*a.launches;
  var_join_kernel<D><<<(unsigned)((units - p.tail) * 16 * C::QTILES), 256, 0, st>>>(p, C::QTILES);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(FwdParams& p, const VarFwdArgs& a, int num_sms, cudaStream_t st) {
  if (!a.paged) return launch_one<D, PACKED, false>(p, a, num_sms, st);
  // sequences of at most one tile of rows on average
  constexpr bool CAN = D <= 128;
  if (CAN && a.seq.rows <= (int64_t)a.seq.batch * p.tok)
    return a.e4m3 ? launch_one<D, PAGED_F8, CAN>(p, a, num_sms, st) : launch_one<D, PAGED, CAN>(p, a, num_sms, st);
  return a.e4m3 ? launch_one<D, PAGED_F8, false>(p, a, num_sms, st) : launch_one<D, PAGED, false>(p, a, num_sms, st);
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
  p.negate = a.scale < 0.0f;
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;
  if (p.scale_log2 == 0.0f) p.scale_log2 = NO_SCALE;
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
