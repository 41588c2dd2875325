// Backward of causal attention over packed sequences on the sm_103a tensor
// cores.  With s = scale q . k, P = exp(s - lse), dP = dO V^T, D = sum_t P dP:
//   dS = scale P (dP - D),  dQ = dS K,  dK = sum over heads dS^T Q,  dV = P^T dO
//
// Three passes: var_bwd_prep_kernel takes lse and D = dO . O of each row and head;
// one kernel holds 128 rows of (token, head) and streams keys and values for dQ;
// one (two for heads of 192 and 256, whose accumulators do not fit together) holds
// 128 keys and values and streams the rows that see them for dK and dV.  So every
// gradient is summed in tensor memory by one CTA in a fixed order: no atomics, no
// partial sums in memory, the same bits every time, and the query heads of a key
// head add up on the way.  The price is S and dP computed twice: 7 products of
// which 5 are needed.  A kernel that keeps keys and adds dQ to memory in 32 bits
// would need an order among the CTAs for that.
//
// The scores lie as M = what stays, so that P and dS, rounded to bf16 in tensor
// memory, are the A operand of the second products as they are, and what streams
// by is read as B both ways, along D and along its rows.  P and dS are each rounded
// once (gradients off by 0.0024 of their norm, where rounding the results alone
// gives 0.0017); S, dP, the statistics and all sums have 32 bits.  Streamed rows
// that none of the block's sees are cleared, and hidden P and dS are 0: other
// sequences count nothing, whatever they hold.  Within a sequence a row that is
// not finite may make any gradient NaN (0 times it, and D of the rows that see it).
//
// Both row groups work on every step, each on half of the columns, while the
// tensor cores run the step's other products: dV and the next scores under dS, dK
// and the next dP under P.
//
// Measured (GB300; 1947 TFLOP/s is its product rate, flops count 5 products), in replays of
// a captured graph; calls in a row take 1435, 245 and 37 to 44 us:
//   one sequence of 8192 tokens, 32 + 8 heads of 128    1368 us, 1005 TFLOP/s (1407 with all 7)
//   19 sequences, 8192 tokens                            237 us,  440 TFLOP/s of pairs that are seen:
//     lse and D 26 (bytes), dQ 110, dK and dV 104
//   5 sequences, 333 tokens, 5 + 1 heads of 64            30 us, three launches' latencies
// What bounds them.  dK and dV: a step takes some 2950 cycles, its products 2560.
// dQ: a step takes some 2650 cycles where its products need 1540; one buffer for
// dP is all that tensor memory has left beside two for scores and dQ, so dP, the row
// groups' dS and the next dP follow one another.  Short sequences: a block of one to
// four steps pays some 4000 cycles for its first copies, its statistics and its
// result.  Heads of 192 and 256: steps of 64 keys, as 128 would not leave room for
// two in flight, pay the same chain for half the work (2 x 4096 tokens, 16 heads
// of 192 on 4 key heads: 1446 us, 357 TFLOP/s; of 128: 391 us, 879 TFLOP/s).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "allow_smem.h"
#include "f32x2.cuh"
#include "ptx_sm103.cuh"
#include "varlen.cuh"
#include "vec.cuh"

namespace tpmlp {
namespace {

// Registers a thread of the issuing warpgroup gives up and the row groups take:
// 88 + 2 x 208 = 3 x 168.
constexpr int ISSUE_REGS = 88, ROW_REGS = 208;
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 200000000ull;
// For a whole block (the largest that fits memory takes some 6 s), and for the scheduler's
// next one, which it may find behind 2^20 empty sequences.
constexpr uint64_t BLOCK_NS = 60000000000ull;

// What a CTA accumulates.  DQ: 128 rows of (token, head) stay, their keys and
// values stream by.  The others: 128 keys stay, the rows of (token, head) that
// see them stream by; DKV both gradients, DV and DK one.
enum Role { DQ = 0, DKV = 1, DV = 2, DK = 3 };

template <int D, int ROLE>
struct Cfg {
  static constexpr bool HAS_DP = ROLE != DV;                 // dP and dS are needed
  static constexpr bool HAS_PV = ROLE == DKV || ROLE == DV;  // P^T dO is accumulated
  static constexpr int KB = D <= 128 ? 128 : 64;             // streamed rows of a step
  static constexpr int HC = KB / 2;                          // columns of a row group
  static constexpr int EC = D % 128 == 0 ? 128 : 64;         // columns of a ring element
  static constexpr int NE = D / EC;                          // elements of a streamed operand
  static constexpr uint32_t SUB = KB * 128;                  // a [KB x 64] tile
  static constexpr uint32_t EB = EC / 64 * SUB;              // an element [KB x EC]
  static constexpr uint32_t RSUB = 128 * 128;                // a [128 x 64] tile
  static constexpr uint32_t RB = D / 64 * RSUB;              // a resident operand [128 x D]
  static constexpr int NRES = HAS_DP ? 2 : 1;
  // Score buffers.  DKV has none to spare in tensor memory (its products hide
  // the row work all the same), heads of 256 no room for a third step's rows.
  static constexpr int NS = ROLE == DKV || (D == 256 && HAS_DP) ? 1 : 2;
  // ring stages of the streamed operands, in steps
  static constexpr int S1 = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int S2 = D == 64 ? 4 : NS == 1 && D == 256 ? 1 : 2;
  static constexpr int N1 = S1 * NE, N2 = S2 * NE;
  static constexpr uint32_t T_DP = KB == 128 && ROLE != DKV ? 256 : 128;
  static constexpr uint32_t T_ACC = KB == 128 && ROLE != DKV ? 384 : 256;
  // DQ: blocks of so many steps, and those under a window of few keys, take D from
  // their own sums.  A single step's P and dP are still in registers then; more steps
  // are run over twice.
  static constexpr int EXACT = 128 / KB;
  static constexpr bool HELD = EXACT == 1;
  static constexpr uint32_t TILES = NRES * RB + (N1 + N2) * EB;
  static constexpr int READERS = ROLE == DQ ? 10 : 11;  // warps that a block is handed to
};

struct BwdParams {
  SeqRows seq;
  float2* stats;  // base-2 log-sum-exp and D of each row and head
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t ld_dq, ld_dk, ld_dv;
  int nq, nkv, hpg;
  int ht, chunks, tok;     // DQ: heads and tokens of a tile of 128 rows
  int sht, schunks, stok;  // the others: of a step
  Slots slots;
  int heads, units;
  bool by_length;
  float scale, scale_log2;
  int window, sinks;
  uint32_t* status;
};

struct BwdBlock {
  int b;                 // NONE: no more
  int g, h0, nh;         // key head, first query head, query heads
  int first, count;      // rows of the sequence
  int at, n, pre;        // first token of the block, steps, of which before the gradient's (DQ)
  int sink_tiles, win_tile, lo, end, sink_end;  // DQ: as in the forward, in tiles of KB keys
};
constexpr int NONE = -2;

// Shared memory behind the tiles.
template <int D, int ROLE>
struct Aux {
  using C = Cfg<D, ROLE>;
  uint64_t r_full, r_empty, full1[C::N1], empty1[C::N1], full2[C::N2], empty2[C::N2], s_full[2], p_full[2], dp_full,
      ds_full, stat_full[2], stat_empty[2], acc_full, sums[2], work_full[2], work_empty[2], drain;
  BwdBlock work[2];
  uint32_t tmem;
  int abort;
  alignas(16) float nlse2[2][ROLE == DQ ? 4 : C::KB];    // the streamed rows' statistics, negated
  alignas(16) float nd[2][ROLE == DQ ? 4 : C::KB];
  float2 row[ROLE == DQ ? 128 : 1];                      // DQ: sums of the rows that stay, and dref
  float row_ref[ROLE == DQ ? 128 : 1];
};

template <int D, int ROLE>
__global__ void __launch_bounds__(384, 1)
    var_bwd_kernel(const __grid_constant__ CUtensorMap map_r1, const __grid_constant__ CUtensorMap map_r2,
                   const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                   const BwdParams p) {
  using C = Cfg<D, ROLE>;
  constexpr int NE = C::NE, EC = C::EC, N1 = C::N1, N2 = C::N2, NS = C::NS, KB = C::KB, HC = C::HC;
  constexpr bool Q_STAYS = ROLE == DQ;
  // no other shared memory is declared, so this begins at a multiple of 1024
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring1 = smem + C::NRES * C::RB;
  uint8_t* ring2 = ring1 + N1 * C::EB;
  Aux<D, ROLE>& x = *reinterpret_cast<Aux<D, ROLE>*>(smem + C::TILES);
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_TIMEOUT);
    return;
  }
  volatile int* abort_flag = &x.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block_tok = Q_STAYS ? p.tok : 128;

  if (threadIdx.x == 0) {
    mbar_init(&x.r_full, 1);
    mbar_init(&x.r_empty, 1);
    for (int i = 0; i < N1; ++i) {
      mbar_init(&x.full1[i], 1);
      mbar_init(&x.empty1[i], 1);
    }
    for (int i = 0; i < N2; ++i) {
      mbar_init(&x.full2[i], 1);
      mbar_init(&x.empty2[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.s_full[i], 1);
      mbar_init(&x.p_full[i], 8);
      mbar_init(&x.stat_full[i], 1);
      mbar_init(&x.stat_empty[i], 8);
      mbar_init(&x.sums[i], 8);
      mbar_init(&x.work_full[i], 1);
      mbar_init(&x.work_empty[i], C::READERS);
    }
    mbar_init(&x.dp_full, 1);
    mbar_init(&x.ds_full, 8);
    mbar_init(&x.acc_full, 1);
    mbar_init(&x.drain, 1);
    x.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_r1);
    tma_prefetch_desc(&map_r2);
    tma_prefetch_desc(&map_x1);
    tma_prefetch_desc(&map_x2);
  }
  // Rows of a step that no copy fills: the products run over them, so they hold zeros.
  if (!Q_STAYS) {
    const int used = p.sht * p.stok;
    if (used < KB)
      for (int i = threadIdx.x; i < (N1 + N2) * (EC / 64) * (KB - used) * 8; i += blockDim.x) {
        const int c = i & 7, r = used + (i >> 3) % (KB - used), t = (i >> 3) / (KB - used);
        *reinterpret_cast<uint4*>(ring1 + t * C::SUB + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
      }
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(&x.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = x.tmem;
  // Step n of a block, n < pre: of the run before the gradient's
  auto tile_of = [](const BwdBlock& k, int n) -> int {
    const int j = n < k.pre ? n : n - k.pre;
    return j < k.sink_tiles ? j : j - k.sink_tiles + k.win_tile;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> int {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
  };
  // The t-th block of this CTA, in shared memory until it is given back; null behind the last.
  auto next = [&](int t) -> const BwdBlock* {
    if (!__all_sync(0xffffffffu, mbar_wait(&x.work_full[t & 1], (uint32_t)((t >> 1) & 1), abort_flag, p.status,
                                           STATUS_TIMEOUT, BLOCK_NS)))
      return nullptr;
    return x.work[t & 1].b == NONE ? nullptr : &x.work[t & 1];
  };
  auto give_back = [&](int t) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&x.work_empty[t & 1]);
  };
  // where dS goes: over the scores, with two score buffers; else over dP
  constexpr bool DS_OVER_S = NS == 2;
  auto ds_col = [&](int n) -> uint32_t { return DS_OVER_S ? (n & 1) * KB : C::T_DP; };
  auto s_col = [&](int n) -> uint32_t { return NS == 2 ? (n & 1) * KB : 0; };

  if (warp < 4) {
    regs_dec<ISSUE_REGS>();
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      uint32_t armed1 = 0, par1 = 0, armed2 = 0, par2 = 0;
      bool ok = true;
      const BwdBlock* kp;
      int t = 0;
      for (int c = 0; ok && (kp = next(t)); give_back(t++)) {
        const BwdBlock& k = *kp;
        if (lane == 0) {
          const uint32_t rows = Q_STAYS ? p.ht * p.tok : 128;
          const uint32_t bytes = (uint32_t)(Q_STAYS ? KB : p.sht * p.stok) * EC * 2;
          for (int n = 0; ok && n < k.n; ++n) {
            const int c1 = Q_STAYS ? k.g : k.h0 + n % p.schunks * p.sht;
            const int c2 = k.first + (Q_STAYS ? tile_of(k, n) * KB : k.at + n / p.schunks * p.stok);
            auto load = [&](uint64_t* fb, uint64_t* eb, uint8_t* ring, int stages, const CUtensorMap* map, uint32_t& armed,
                            uint32_t& pars) -> bool {
              for (int e = 0; e < NE; ++e) {
                const int at = (c + n) * NE + e, st = at % stages;
                const uint32_t par = (uint32_t)((at / stages) & 1);
                if (!mbar_wait(&eb[st], par ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS)) return false;
                mbar_arrive_expect_tx(&fb[st], bytes);
                armed |= 1u << st;
                pars = (pars & ~(1u << st)) | (par << st);
                for (int u = 0; u < EC / 64; ++u)
                  tma_load_3d(ring + st * C::EB + u * C::SUB, map, &fb[st], e * EC + 64 * u, c1, c2);
              }
              return true;
            };
            ok = load(x.full1, x.empty1, ring1, N1, &map_x1, armed1, par1);
            if (ok && n == 0) {
              ok = mbar_wait(&x.r_empty, (uint32_t)(t & 1) ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS);
              if (!ok) break;
              mbar_arrive_expect_tx(&x.r_full, C::NRES * (D / 64) * rows * 128);
              for (int o = 0; o < C::NRES; ++o)
                for (int u = 0; u < D / 64; ++u)
                  tma_load_3d(smem + o * C::RB + u * C::RSUB, o ? &map_r2 : &map_r1, &x.r_full, 64 * u,
                              Q_STAYS ? k.h0 : k.g, k.first + k.at);
            }
            ok = ok && load(x.full2, x.empty2, ring2, N2, &map_x2, armed2, par2);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        c += k.n;
      }
      if (lane == 0 && (!ok || *abort_flag)) {  // copies still in flight land on the barriers armed last
        int no_abort = 0;
        if (t > 0 || armed1) mbar_wait(&x.r_full, (uint32_t)((t > 0 ? t - 1 : 0) & 1), &no_abort, p.status, 0u, DRAIN_NS);
        for (int st = 0; st < N1; ++st)
          if (armed1 & (1u << st)) mbar_wait(&x.full1[st], (par1 >> st) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 16);
        for (int st = 0; st < N2; ++st)
          if (armed2 & (1u << st)) mbar_wait(&x.full2[st], (par2 >> st) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 16);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- issuer
      // A wait costs the tensor core a gap of some 150 cycles where nothing is
      // queued: there is one on the row groups a step and gradient, and the
      // copies are waited for before it.
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, KB, false, false);
      constexpr uint32_t IDESC_A = idesc_bf16_f32(128, EC, false, true);
      const uint64_t r_desc = sw128_desc(smem_u32(smem), 16, 1024);
      const uint64_t x1k = sw128_desc(smem_u32(ring1), 16, 1024), x2k = sw128_desc(smem_u32(ring2), 16, 1024);
      const uint64_t x1m = sw128_desc(smem_u32(ring1), C::SUB, 1024), x2m = sw128_desc(smem_u32(ring2), C::SUB, 1024);
      auto wait_elems = [&](uint64_t* bars, int stages, int n) -> int {
        int r = 1;
#pragma unroll
        for (int e = 0; e < NE; ++e)
          r = r && wait_all(&bars[(n * NE + e) % stages], (uint32_t)(((n * NE + e) / stages) & 1));
        return r;
      };
      // scores: resident operand `o` times the streamed one
      auto product = [&](int o, int stages, uint64_t xk, int n, uint32_t col) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const uint64_t b = desc_advance(xk, ((n * NE + e) % stages) * C::EB);
          const uint64_t a = desc_advance(r_desc, o * C::RB + e * (EC / 64) * C::RSUB);
#pragma unroll
          for (int kk = 0; kk < EC / 16; ++kk)
            tc_mma_f16(tmem_base + col, desc_advance(a, (kk >> 2) * C::RSUB + (kk & 3) * 32),
                       desc_advance(b, (kk >> 2) * C::SUB + (kk & 3) * 32), IDESC_S, e > 0 || kk > 0 ? 1u : 0u);
        }
      };
      // accumulator at `acc` += (bf16 rows, each row group's half at the start of
      // its half of the columns from `a_col` on) times the streamed operand
      auto accumulate = [&](int stages, uint64_t xm, int n, uint32_t a_col, uint32_t acc, bool first) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          const uint64_t b = desc_advance(xm, ((n * NE + e) % stages) * C::EB);
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk)
            tc_mma_f16_ts(tmem_base + acc + e * EC, tmem_base + a_col + kk / (HC / 16) * HC + kk % (HC / 16) * 8,
                          desc_advance(b, kk * 2048), IDESC_A, !first || kk > 0 ? 1u : 0u);
        }
      };
      auto release = [&](uint64_t* bars, int stages, int n) {
#pragma unroll
        for (int e = 0; e < NE; ++e) tc_commit(&bars[(n * NE + e) % stages]);
      };
      bool ok = true;
      const BwdBlock* kp;
      for (int t = 0, c = 0; ok && (kp = next(t)); give_back(t++)) {
        const int nk = kp->n, pre = kp->pre;
        // steps of this block; in the rings and barriers they count on from the blocks before
        auto put_s = [&](int n) {
          product(0, N1, x1k, c + n, s_col(c + n));
          tc_commit(&x.s_full[NS == 2 ? (c + n) & 1 : 0]);
          if (!C::HAS_DP) {
            release(x.empty1, N1, c + n);
            if (n + 1 == nk) tc_commit(&x.r_empty);
          }
        };
        auto put_dp = [&](int n) {  // the last product of the operands that stay
          product(1, N2, x2k, c + n, C::T_DP);
          tc_commit(&x.dp_full);
          if (!C::HAS_PV) release(x.empty2, N2, c + n);
          if (n + 1 == nk) tc_commit(&x.r_empty);
        };
        auto put_acc = [&](int n) {  // dS X1
          if (n >= pre) accumulate(N1, x1m, c + n, ds_col(c + n), C::T_ACC, n == pre);
          release(x.empty1, N1, c + n);
          if (n + 1 == nk) tc_commit(&x.acc_full);
        };
        auto put_pv = [&](int n) {  // P X2
          accumulate(N2, x2m, c + n, s_col(c + n), C::T_ACC + (ROLE == DKV ? D : 0), n == 0);
          release(x.empty2, N2, c + n);
          if (!C::HAS_DP && n + 1 == nk) tc_commit(&x.acc_full);
        };
        auto have1 = [&](int n) -> bool { return wait_elems(x.full1, N1, c + n); };
        auto have2 = [&](int n) -> bool { return wait_elems(x.full2, N2, c + n); };
        ok = have1(0) && wait_all(&x.r_full, (uint32_t)(t & 1));
        if (ok && C::HAS_DP) ok = have2(0);
        tc_fence_after();
        if (ok && elect_one()) {
          put_s(0);
          if (C::HAS_DP) put_dp(0);
        }
        __syncwarp();
        if (ok && NS == 2 && nk > 1 && (ok = have1(1))) {
          tc_fence_after();
          if (elect_one()) put_s(1);
          __syncwarp();
        }
#pragma unroll 1
        for (int n = 0; ok && n < nk; ++n) {
          const uint32_t par = (uint32_t)((c + n) & 1);
          const bool n1 = n + 1 < nk, n2 = n + 2 < nk;
          if constexpr (C::HAS_DP && !C::HAS_PV && NS == 2) {
            // dP_{n+1}, then dS_n X1 and S_{n+2} while the row groups turn dP_{n+1} into dS
            if (n1 && !(ok = have2(n + 1))) break;
            if (!(ok = wait_all(&x.ds_full, par))) break;
            tc_fence_after();
            if (elect_one()) {
              if (n1) put_dp(n + 1);
              put_acc(n);
            }
            __syncwarp();
            if (n2) {  // its rows come into the place of step n's
              if (!(ok = have1(n + 2))) break;
              tc_fence_after();
              if (elect_one()) put_s(n + 2);
              __syncwarp();
            }
          } else if constexpr (C::HAS_DP && !C::HAS_PV) {
            if (n1) {
              if (!(ok = have1(n + 1) && wait_all(&x.p_full[0], par))) break;  // the scores are read
              tc_fence_after();
              if (elect_one()) put_s(n + 1);
              __syncwarp();
            } else if (!(ok = wait_all(&x.p_full[0], par))) {  // every phase is seen
              break;
            }
            if (!(ok = wait_all(&x.ds_full, par))) break;
            tc_fence_after();
            if (elect_one()) put_acc(n);
            __syncwarp();
            if (n1) {
              if (!(ok = have2(n + 1))) break;
              tc_fence_after();
              if (elect_one()) put_dp(n + 1);
              __syncwarp();
            }
          } else if constexpr (C::HAS_DP) {
            // dV_n and S_{n+1} under the row groups' dS_n, dK_n and dP_{n+1} under their P_{n+1}
            if (n1 && !(ok = have1(n + 1))) break;
            if (!(ok = wait_all(&x.p_full[0], par))) break;
            tc_fence_after();
            if (elect_one()) {
              put_pv(n);
              if (n1) put_s(n + 1);
            }
            __syncwarp();
            if (n1 && !(ok = have2(n + 1))) break;
            if (!(ok = wait_all(&x.ds_full, par))) break;
            tc_fence_after();
            if (elect_one()) {
              put_acc(n);
              if (n1) put_dp(n + 1);
            }
            __syncwarp();
          } else {
            if (n2 && !(ok = have1(n + 2))) break;
            if (!(ok = have2(n) && wait_all(&x.p_full[(c + n) & 1], (uint32_t)(((c + n) >> 1) & 1)))) break;
            tc_fence_after();
            if (elect_one()) {
              put_pv(n);
              if (n2) put_s(n + 2);
            }
            __syncwarp();
          }
        }
        c += nk;
      }
      if (elect_one()) tc_commit(&x.drain);
      __syncwarp();
      int no_abort = 0;
      mbar_wait(&x.drain, 0, &no_abort, p.status, STATUS_TIMEOUT, DRAIN_NS);
    } else if (warp == 2) {
      // ---------------------------------------- statistics of the streamed rows
      bool ok = true;
      const BwdBlock* kp;
      for (int t = 0, c = 0; !Q_STAYS && ok && (kp = next(t)); give_back(t++)) {
        const BwdBlock& k = *kp;
        for (int n = 0; ok && n < k.n; ++n) {
          const int st = (c + n) & 1;
          const int tok0 = k.at + n / p.schunks * p.stok, hc = n % p.schunks * p.sht;
          float2 v[KB / 32];
#pragma unroll
          for (int q = 0; q < KB / 32; ++q) {
            const int r = lane + 32 * q, tk = tok0 + r / p.sht, hh = hc + r % p.sht;
            const bool valid = r < p.sht * p.stok && tk < k.end && hh < p.hpg;
            v[q] = valid ? __ldg(p.stats + (int64_t)(k.first + tk) * p.nq + k.h0 + hh) : make_float2(INFINITY, 0.0f);
          }
          if (!(ok = wait_all(&x.stat_empty[st], (uint32_t)(((c + n) >> 1) & 1) ^ 1u))) break;
#pragma unroll
          for (int q = 0; q < KB / 32; ++q) {
            x.nlse2[st][lane + 32 * q] = -v[q].x;
            x.nd[st][lane + 32 * q] = -v[q].y;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.stat_full[st]);
        }
        c += k.n;
      }
    } else {
      // ------------------------------------------------------------- scheduler
      ByLength<KB> order;
      if (p.by_length)
        order.init(p.seq, -1, block_tok,
                   p.window > 0 ? (p.window + block_tok) / KB + 2 + (Q_STAYS ? (p.sinks + KB - 1) / KB : 0) : 0x7fffffff,
                   lane);
      bool ok = true;
      int t = 0;
      for (int turn = 0; ok; ++turn) {
        const int64_t u = snake(turn, (int)blockIdx.x, (int)gridDim.x);
        const bool last = (int64_t)turn * gridDim.x >= p.units;
        BwdBlock k;
        k.b = NONE;
        if (!last) {
          if (u >= p.units) continue;
          const int rank = (int)u / p.heads, hd = (int)u % p.heads;
          k.g = Q_STAYS ? hd / p.chunks : hd;
          k.h0 = k.g * p.hpg + (Q_STAYS ? hd % p.chunks * p.ht : 0);
          k.nh = Q_STAYS ? min(p.ht, (k.g + 1) * p.hpg - k.h0) : p.hpg;
          int b, i = 0;
          if (p.by_length) {
            order.find(rank, lane, &b, &i);
          } else {
            b = find_slot(p.seq, p.slots, (int)p.slots.count - 1 - rank, lane);
            i = -1;  // below
          }
          if (b < 0) continue;
          bool bad = false;
          const SeqSpan s = seq_span(p.seq, b, -1, &bad);
          if (i < 0) i = (int)p.slots.count - 1 - rank - slot_base(p.slots, s.first, b);
          if (i < 0 || (int64_t)i * block_tok >= s.count) {
            turn = max(turn, (rank + 1) * p.heads / (int)gridDim.x - 1);  // empty for all key heads
            continue;
          }
          // key blocks from the first on are the long ones
          if (!Q_STAYS) i = (s.count - 1) / block_tok - i;
          k.b = b;
          k.first = s.first;
          k.count = s.count;
          k.at = i * block_tok;
          k.pre = 0;
          if (Q_STAYS) {
            k.end = min(k.at + block_tok, s.count);
            k.lo = p.window > 0 ? max(0, k.at + 1 - p.window) : 0;
            k.sink_end = min(p.sinks, k.lo);
            k.win_tile = k.lo / KB;
            k.sink_tiles = min((k.sink_end + KB - 1) / KB, k.win_tile);
            k.n = k.sink_tiles + (k.end + KB - 1) / KB - k.win_tile;
            // D = dO . O takes the output as it was rounded.  For tokens that see few
            // others D is as large as what it is taken from, and that rounding would be a
            // good part of a small gradient (dq off by 0.0026 of its norm where its own
            // rounding is 0.0017): there D = sum P dP.  It shrinks with the root of the
            // number of keys; behind 100 it is a tenth of the gradient's own rounding.
            if (k.n <= C::EXACT ? !C::HELD : p.window > 0 && p.window + p.sinks < 128) k.pre = k.n;
            k.n += k.pre;
          } else {
            // the tokens [at, end) see keys of the block
            const int end = min(k.at + block_tok, s.count) - 1;
            k.end = p.window > 0 && k.at >= p.sinks ? (int)min((int64_t)s.count, (int64_t)end + p.window) : s.count;
            k.lo = k.sink_end = k.win_tile = k.sink_tiles = 0;
            k.n = (k.end - k.at + p.stok - 1) / p.stok * p.schunks;
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&x.work_empty[t & 1], (uint32_t)((t >> 1) & 1) ^ 1u, abort_flag, p.status,
                                               STATUS_TIMEOUT, BLOCK_NS));
        if (ok && lane == 0) {
          x.work[t & 1] = k;
          mbar_arrive(&x.work_full[t & 1]);
        }
        __syncwarp();
        ++t;
        if (last) break;
      }
      report_bad(p.seq, -1, p.status, lane);
    }
  } else {
    regs_inc<ROW_REGS>();
    // ------------------------------------------------------------ row groups
    // Both work on every step, each on half of its columns: that halves the
    // time from scores to P and from dP to dS, which the products of the other
    // kind hide.
    const int grp = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the accumulators
    const int tid = grp * 128 + r;
    const uint32_t tl = tmem_base + ((uint32_t)(q4 * 32) << 16) + grp * HC;
    const int tok_r = Q_STAYS ? r / p.ht : r, hh = Q_STAYS ? r - tok_r * p.ht : 0;  // token or key of the row, head
    uint32_t pres = 0;
    int ok = 1;
    const BwdBlock* kp;
    for (int t = 0, done = 0; ok && (kp = next(t)); give_back(t++)) {
      const BwdBlock& blk = *kp;
      const int nk = blk.n, pre = blk.pre, h0 = blk.h0, g = blk.g;
      const int tk = blk.at + tok_r;
      const bool stored = tk < blk.count && (!Q_STAYS || (r < p.ht * p.tok && hh < blk.nh));
      const int64_t stat_at = (int64_t)(blk.first + tk) * p.nq + h0 + hh;
      float lse2 = 0.0f, dsum = 0.0f;
      // Over few keys: sum P, and sum P (dP - dref) with dref the dP of the first
      // key that the row sees: exact where it sees no other.
      const bool held = Q_STAYS && C::HELD && nk == 1, exact = held || pre > 0;
      float l = 0.0f, dref = 0.0f;
      if (Q_STAYS) {
        if (stored) {
          const float2 z = p.stats[stat_at];
          lse2 = z.x;
          if (!exact) dsum = z.y;
        }
      }
      auto add = [&](float pr, uint32_t d) {
        if (pr != 0.0f) {  // hidden values may be anything
          if (l == 0.0f) dref = __uint_as_float(d);
          l += pr;
          dsum = fmaf(pr, __uint_as_float(d) - dref, dsum);
        }
      };
      // The sums of both groups' halves: l becomes sum P, dsum becomes D.
      auto settle = [&]() -> bool {
        auto meet = [&](int i) -> bool {
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.sums[i]);
          return wait_all(&x.sums[i], pres & 1u);
        };
        if (grp == 1) {
          x.row[r] = make_float2(l, dsum);
          x.row_ref[r] = dref;
        }
        if (!meet(0)) return false;
        if (grp == 0) {
          const float2 o = x.row[r];
          const float ref = x.row_ref[r], all = l + o.x;
          const float d = l != 0.0f ? dref + (dsum + o.y + (o.x != 0.0f ? o.x * (ref - dref) : 0.0f)) / all
                                    : ref + (o.y + dsum) / all;
          x.row[r] = make_float2(all, d);
        }
        if (!meet(1)) return false;
        ++pres;
        l = x.row[r].x;
        dsum = x.row[r].y;
        lse2 += log2f(l);
        if (stored && grp == 0) p.stats[stat_at] = make_float2(lse2, dsum);
        return true;
      };
      for (int n = 0; n < nk; ++n) {
        const int N = done + n;  // as rings and barriers count
        const uint32_t par = (uint32_t)(N & 1), par2 = (uint32_t)((N >> 1) & 1);
        const int st = N & 1;
        if (Q_STAYS && pre && n == pre) {
          if (!(ok = settle())) break;
        }
        if (!Q_STAYS && !(ok = wait_all(&x.stat_full[st], par2))) break;
        if (!(ok = wait_all(&x.s_full[NS == 2 ? N & 1 : 0], NS == 2 ? par2 : par))) break;
        tc_fence_after();
        const uint32_t t_s = tl + s_col(N);
        uint32_t v[HC];
        tmem_ld_32x32b_x32(t_s, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld_wait();
        if constexpr (HC == 64) tmem_ld_32x32b_x32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        if (!C::HAS_PV && NS == 1) {  // the scores may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.p_full[0]);
        }
        // Streamed rows that none of ours sees (other sequences', or behind the end) are
        // cleared where a product sums over them.  A wait for a ring stage is good for the
        // next phase only: what was in the stage before has landed, as the scores of this
        // step are complete.
        constexpr int CPT = 8 * KB / 256;  // 16-byte pieces of a tile's row for each thread
        const int crow = tid % KB, cpart = tid / KB * CPT;
        bool masked;
        int t0 = 0, c_lo = 0, c_hi = 0;  // columns c_lo to c_hi - 1 of this group's are seen
        if (Q_STAYS) {
          const int tile0 = tile_of(blk, n) * KB;
          t0 = tile0 + grp * HC;
          const int last = blk.at + min(p.tok, blk.count - blk.at) - 1;
          masked = t0 + HC - 1 > blk.at || (p.window > 0 && last - t0 >= p.window && t0 + HC > p.sinks);
          if (tile0 + KB > blk.end || (tile0 < blk.lo && tile0 + KB > blk.sink_end)) {
            const int t = tile0 + crow;
            if (t >= blk.end || (t < blk.lo && t >= blk.sink_end))
              for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
                  for (int c = 0; c < CPT; ++c)
                    *reinterpret_cast<uint4*>(ring1 + ((N * NE + e) % N1) * C::EB + cb * C::SUB + crow * 128 +
                                              (cpart + c) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        } else {
          const int tok0 = blk.at + n / p.schunks * p.stok, hc = n % p.schunks * p.sht;
          // a key is seen by tokens without a gap, whose heads lie together: with more than one
          // chunk of heads a step has one token
          const int w = p.window > 0 && tk >= p.sinks ? min(p.window, 0x7fffff00) : 0x7fffff00;
          c_lo = min(max(tk - tok0, 0), p.stok) * p.sht - grp * HC;
          c_hi = min(max(min(min(blk.end - tok0, p.stok), tk - tok0 + w), 0) * p.sht,
                     p.schunks > 1 ? p.hpg - hc : KB) - grp * HC;
          const bool cut = tok0 + p.stok > blk.end || hc + p.sht > p.hpg;
          masked = cut || blk.at + 127 > tok0 ||
                   (p.window > 0 && tok0 + p.stok - 1 - blk.at >= p.window && blk.at + 128 > p.sinks);
          if (cut) {
            if (C::HAS_PV)
              for (int e = 0; ok && e < NE; ++e)
                ok = wait_all(&x.full2[(N * NE + e) % N2], (uint32_t)(((N * NE + e) / N2) & 1));
            if (!ok) break;
            if (crow < p.sht * p.stok && (tok0 + crow / p.sht >= blk.end || hc + crow % p.sht >= p.hpg))
              for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
                  for (int c = 0; c < CPT; ++c) {
                    const uint32_t o = cb * C::SUB + crow * 128 + (cpart + c) * 16;
                    if (C::HAS_DP) *reinterpret_cast<uint4*>(ring1 + ((N * NE + e) % N1) * C::EB + o) = make_uint4(0, 0, 0, 0);
                    if (C::HAS_PV) *reinterpret_cast<uint4*>(ring2 + ((N * NE + e) % N2) * C::EB + o) = make_uint4(0, 0, 0, 0);
                  }
            fence_proxy_async_smem();
          }
        }
        // P, 32 columns at a time
        uint32_t w[HC / 2];
#pragma unroll
        for (int hf = 0; hf < HC / 32; ++hf) {
          uint32_t* u = v + 32 * hf;
          if (hf == 1) tmem_ld_wait();
          const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
          if (Q_STAYS) {
            const uint64_t nl2 = f2_pack(-lse2, -lse2);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float a0, a1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sc2, nl2), a0, a1);
              u[c] = __float_as_uint(ex2_fast(a0));
              u[c + 1] = __float_as_uint(ex2_fast(a1));
            }
            if (masked) {
              const int t = t0 + 32 * hf;
              uint32_t bits = below(tk - t + 1);
              if (p.window > 0) bits &= ~below(tk - p.window - t + 1) | below(p.sinks - t);
              if (__any_sync(0xffffffffu, bits != ~0u)) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(bits & (1u << c))) u[c] = 0u;
              }
            }
          } else {
            const ulonglong2* sp = reinterpret_cast<const ulonglong2*>(x.nlse2[st] + grp * HC + 32 * hf);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const ulonglong2 z = sp[c >> 2];
              float a0, a1, a2, a3;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sc2, z.x), a0, a1);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(u[c + 2]), __uint_as_float(u[c + 3])), sc2, z.y), a2, a3);
              u[c] = __float_as_uint(ex2_fast(a0));
              u[c + 1] = __float_as_uint(ex2_fast(a1));
              u[c + 2] = __float_as_uint(ex2_fast(a2));
              u[c + 3] = __float_as_uint(ex2_fast(a3));
            }
            if (masked) {
              const uint32_t bits = below(c_hi - 32 * hf) & ~below(c_lo - 32 * hf);
              if (__any_sync(0xffffffffu, bits != ~0u)) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(bits & (1u << c))) u[c] = 0u;
              }
            }
          }
          if (C::HAS_PV) {
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              w[16 * hf + (c >> 1)] = pack_bf16(__uint_as_float(u[c]), __uint_as_float(u[c + 1]));
          }
        }
        if (C::HAS_PV) {  // over the group's scores
          if constexpr (HC == 64) tmem_st_32x32b_x32(t_s, w);
          else tmem_st_32x32b_x16(t_s, w);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.p_full[NS == 2 ? N & 1 : 0]);
        }
        if (C::HAS_DP) {
          if (!(ok = wait_all(&x.dp_full, par))) break;
          tc_fence_after();
          const uint32_t t_dp = tl + C::T_DP;
          uint32_t dd[HC];
          tmem_ld_32x32b_x32(t_dp, *reinterpret_cast<uint32_t(*)[32]>(dd));
          tmem_ld_wait();
          if constexpr (HC == 64) tmem_ld_32x32b_x32(t_dp + 32, *reinterpret_cast<uint32_t(*)[32]>(dd + 32));
          if (held) {
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < HC; ++c) add(__uint_as_float(v[c]), dd[c]);
            if (!(ok = settle())) break;
            const float inv = 1.0f / l;
#pragma unroll
            for (int c = 0; c < HC; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * inv);
          }
#pragma unroll
          for (int hf = 0; hf < HC / 32; ++hf) {
            uint32_t* d = dd + 32 * hf;
            if (hf == 1) tmem_ld_wait();
            if (Q_STAYS && n < pre) {  // the sums alone
#pragma unroll
              for (int c = 0; c < 32; ++c) add(__uint_as_float(v[32 * hf + c]), d[c]);
            } else {
              // P (dP - D); the scale comes in at the end
              const ulonglong2* dp = reinterpret_cast<const ulonglong2*>(x.nd[Q_STAYS ? 0 : st] + (Q_STAYS ? 0 : grp * HC + 32 * hf));
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const int cc = 32 * hf + c;
                ulonglong2 z;
                if (Q_STAYS) z.x = z.y = f2_pack(-dsum, -dsum);
                else z = dp[c >> 2];
                float e[4];
                f2_unpack(f2_mul(f2_pack(__uint_as_float(v[cc]), __uint_as_float(v[cc + 1])),
                                 f2_add(f2_pack(__uint_as_float(d[c]), __uint_as_float(d[c + 1])), z.x)), e[0], e[1]);
                f2_unpack(f2_mul(f2_pack(__uint_as_float(v[cc + 2]), __uint_as_float(v[cc + 3])),
                                 f2_add(f2_pack(__uint_as_float(d[c + 2]), __uint_as_float(d[c + 3])), z.y)), e[2], e[3]);
                if (masked) {  // 0 whatever dP is
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (v[cc + k] == 0u) e[k] = 0.0f;
                }
                w[cc >> 1] = pack_bf16(e[0], e[1]);
                w[(cc >> 1) + 1] = pack_bf16(e[2], e[3]);
              }
            }
          }
          if (!Q_STAYS || n >= pre) {
            if constexpr (HC == 64) tmem_st_32x32b_x32(tl + ds_col(N), w);
            else tmem_st_32x32b_x16(tl + ds_col(N), w);
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.ds_full);
        }
        if (!Q_STAYS) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&x.stat_empty[st]);
        }
      }
      done += nk;
      if (!ok || !(ok = wait_all(&x.acc_full, (uint32_t)(t & 1)))) break;
      tc_fence_after();
      // DKV: group 0 dV, group 1 dK; else each group half of the columns
      constexpr int W = ROLE == DKV ? D : D / 2;
      const uint32_t t_acc =
          tmem_base + ((uint32_t)(q4 * 32) << 16) + C::T_ACC + (ROLE == DKV ? (grp ? 0 : D) : grp * W);
      __nv_bfloat16* dst = nullptr;
      if (stored) {
        const int64_t row = blk.first + tk;
        if (Q_STAYS) dst = p.dq + row * p.ld_dq + (int64_t)(h0 + hh) * D + grp * W;
        else if (ROLE == DV || (ROLE == DKV && grp == 0)) dst = p.dv + row * p.ld_dv + (int64_t)g * D + (ROLE == DKV ? 0 : grp * W);
        else dst = p.dk + row * p.ld_dk + (int64_t)g * D + (ROLE == DKV ? 0 : grp * W);
      }
      int64_t row_at[4];  // of the four lanes that turn their pieces together
#pragma unroll
      for (int q = 0; q < 4; ++q) row_at[q] = __shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(dst), (lane & ~3) + q);
      const float fin = ROLE == DV || (ROLE == DKV && grp == 0) ? 1.0f : p.scale;
#pragma unroll 1
      for (int c = 0; c < W; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(t_acc + c, o);
        tmem_ld_wait();
        uint4 u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          u[q] = make_uint4(pack_bf16(__uint_as_float(o[8 * q]) * fin, __uint_as_float(o[8 * q + 1]) * fin),
                            pack_bf16(__uint_as_float(o[8 * q + 2]) * fin, __uint_as_float(o[8 * q + 3]) * fin),
                            pack_bf16(__uint_as_float(o[8 * q + 4]) * fin, __uint_as_float(o[8 * q + 5]) * fin),
                            pack_bf16(__uint_as_float(o[8 * q + 6]) * fin, __uint_as_float(o[8 * q + 7]) * fin));
        turn_pieces(u, lane);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (row_at[q]) *reinterpret_cast<uint4*>(row_at[q] + 2 * c + 16 * (lane & 3)) = u[q];
        __syncwarp();
      }
      // the accumulators may be overwritten: the next block's first product into them
      // waits for these warps' P or dS
      tc_fence_before();
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

// stats = (log2(e) lse, D = dO . O) of each row and head.  Bound by bytes: a
// warp a row, D / 8 lanes a head, two loads of 16 bytes a lane and turn.
template <int D>
__global__ void __launch_bounds__(256) var_bwd_prep_kernel(const VarBwdArgs a) {
  constexpr int LPR = D / 8, HPW = D == 192 ? 1 : 32 / LPR;  // lanes a head, heads a turn
  const int lane = threadIdx.x & 31;
  const int sub = HPW > 1 ? lane / LPR : 0, c = HPW > 1 ? lane % LPR : lane;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.seq.rows; row += (int64_t)gridDim.x * 8) {
    const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.dout) + row * a.ld_dout;
    const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(a.out) + row * a.ld_out;
#pragma unroll 4
    for (int h0 = 0; h0 < a.nq; h0 += HPW) {
      const int h = h0 + sub;
      float s = 0.0f;
      if (h < a.nq && c < LPR) {
        float x[8], y[8];
        Vec<__nv_bfloat16>::load(g + (int64_t)h * D + 8 * c, x);
        Vec<__nv_bfloat16>::load(o + (int64_t)h * D + 8 * c, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
      }
#pragma unroll
      for (int k = (HPW > 1 ? LPR : 32) / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if (c == 0 && h < a.nq) a.stats[row * a.nq + h] = make_float2(a.lse[row * a.nq + h] * 1.4426950408889634f, s);
    }
  }
}

template <int D, int ROLE>
cudaError_t launch_role(BwdParams p, const VarBwdArgs& a, int num_sms, cudaStream_t st) {
  using C = Cfg<D, ROLE>;
  constexpr int SMEM = (int)(C::TILES + sizeof(Aux<D, ROLE>));
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(C::NS * C::KB <= (int)C::T_DP || !C::HAS_DP, "tensor memory");
  static_assert(C::T_ACC + (ROLE == DKV ? 2 * D : D) <= 512, "tensor memory");
  const int block_tok = ROLE == DQ ? p.tok : 128;
  p.heads = ROLE == DQ ? a.nkv * p.chunks : a.nkv;
  p.schunks = (p.hpg + C::KB - 1) / C::KB;
  p.sht = (p.hpg + p.schunks - 1) / p.schunks;
  p.stok = C::KB / p.sht;
  p.slots = make_slots(a.seq, block_tok);
  const int64_t units = p.slots.count * p.heads;
  if (units > VAR_MAX_BLOCKS) return cudaErrorInvalidConfiguration;  // var_fits
  p.units = (int)units;
  p.by_length = units > num_sms && a.seq.batch <= LPT_BATCH;
  CUtensorMap r1, r2, x1, x2;
  const int64_t rows = a.seq.rows;
  const bool ok =
      ROLE == DQ ? map3(&r1, a.q, D, a.nq, rows, a.ld_q, p.ht, p.tok) && map3(&r2, a.dout, D, a.nq, rows, a.ld_dout, p.ht, p.tok) &&
                       map3(&x1, a.k, D, a.nkv, rows, a.ld_k, 1, C::KB) && map3(&x2, a.v, D, a.nkv, rows, a.ld_v, 1, C::KB)
                 : map3(&r1, a.k, D, a.nkv, rows, a.ld_k, 1, 128) && map3(&r2, a.v, D, a.nkv, rows, a.ld_v, 1, 128) &&
                       map3(&x1, a.q, D, a.nq, rows, a.ld_q, p.sht, p.stok) &&
                       map3(&x2, a.dout, D, a.nq, rows, a.ld_dout, p.sht, p.stok);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<var_bwd_kernel<D, ROLE>>(SMEM);
  if (e == cudaSuccess) e = check_regs<var_bwd_kernel<D, ROLE>>(384, 128 * (ISSUE_REGS + 2 * ROW_REGS));
  if (e != cudaSuccess) return e;
  var_bwd_kernel<D, ROLE><<<p.units < num_sms ? p.units : num_sms, 384, SMEM, st>>>(r1, r2, x1, x2, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const BwdParams& p, const VarBwdArgs& a, int num_sms, cudaStream_t st) {
  const int64_t want = (a.seq.rows + 7) / 8, most = 8LL * num_sms;
  var_bwd_prep_kernel<D><<<(unsigned)(want < most ? want : most), 256, 0, st>>>(a);
  if (a.launches) *a.launches += D <= 128 ? 2 : 3;
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_role<D, DQ>(p, a, num_sms, st);  // corrects the statistics that the others read
  if (e != cudaSuccess) return e;
  if constexpr (D <= 128) {
    return launch_role<D, DKV>(p, a, num_sms, st);
  } else {
    e = launch_role<D, DV>(p, a, num_sms, st);
    return e != cudaSuccess ? e : launch_role<D, DK>(p, a, num_sms, st);
  }
}

}  // namespace

cudaError_t launch_var_bwd(const VarBwdArgs& a, int num_sms, cudaStream_t st) {
  BwdParams p{};
  p.seq = a.seq;
  p.stats = a.stats;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.ld_dq = a.ld_dq;
  p.ld_dk = a.ld_dk;
  p.ld_dv = a.ld_dv;
  p.nq = a.nq;
  p.nkv = a.nkv;
  p.hpg = a.nq / a.nkv;
  p.ht = p.hpg < 128 ? p.hpg : 128;
  p.chunks = (p.hpg + p.ht - 1) / p.ht;
  p.tok = 128 / p.ht;
  p.scale = a.scale;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.window = a.window;
  p.sinks = a.sinks;
  p.status = a.status;
  switch (a.d) {
    case 64: return launch_d<64>(p, a, num_sms, st);
    case 128: return launch_d<128>(p, a, num_sms, st);
    case 192: return launch_d<192>(p, a, num_sms, st);
    case 256: return launch_d<256>(p, a, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tpmlp
