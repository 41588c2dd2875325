// Backward of causal attention over packed sequences on the sm_103a tensor
// cores.  With s = scale q . k, P = exp(s - lse), dP = dO V^T, D = sum_t P dP:
//   dS = scale P (dP - D),  dQ = dS K,  dK = sum over heads dS^T Q,  dV = P^T dO
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "allow_smem.h"
#include "f32x2.cuh"
#include "ptx_sm103.cuh"
#include "varlen.cuh"

namespace tpmlp {
namespace {

// Registers a thread of the issuing warpgroup gives up and the row groups take:
// 88 + 2 x 208 = 3 x 168.
constexpr int ISSUE_REGS = 88, ROW_REGS = 208;
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 200000000ull;

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
  static constexpr int S1 = D == 64 ? 4 : NS == 1 && D == 256 ? 2 : 3;
  static constexpr int S2 = D == 64 ? 4 : NS == 1 && D == 256 ? 1 : 2;
  static constexpr int N1 = S1 * NE, N2 = S2 * NE;
  // tensor memory: scores, dP, accumulators
  static constexpr uint32_t T_DP = KB == 128 && ROLE != DKV ? 256 : 128;
  static constexpr uint32_t T_ACC = KB == 128 && ROLE != DKV ? 384 : 256;
  static constexpr int TWICE = 256 / KB;
  static constexpr uint32_t TILES = NRES * RB + (N1 + N2) * EB;
};

struct BwdParams {
  SeqRows seq;
  const __nv_bfloat16 *out, *dout;
  int64_t ld_out, ld_dout;
  const float* lse;
  float2* stats;  // base-2 log-sum-exp and D of each row and head
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t ld_dq, ld_dk, ld_dv;
  int nq, nkv, hpg;
  int ht, chunks, tok;     // DQ: heads and tokens of a tile of 128 rows
  int sht, schunks, stok;  // the others: of a step
  Slots slots;
  int heads;
  bool by_length;
  float scale, scale_log2;
  int window, sinks;
  uint32_t* status;
};

struct BwdBlock {
  int b;                 // < 0: none
  int first, count;      // rows of the sequence
  int at, n;             // first token of the block, steps
  int sink_tiles, win_tile, lo, end, sink_end;  // DQ: as in the forward, in tiles of KB keys
};

// Shared memory behind the tiles.
template <int D, int ROLE>
struct Aux {
  using C = Cfg<D, ROLE>;
  uint64_t r_full, full1[C::N1], empty1[C::N1], full2[C::N2], empty2[C::N2], s_full[2], p_full[2], dp_full, ds_full,
      stat_full[2], stat_empty[2], acc_full, drain;
  BwdBlock blk;
  uint32_t tmem;
  int abort;
  alignas(16) float nlse2[2][ROLE == DQ ? 4 : C::KB];  // the streamed rows' statistics, negated
  alignas(16) float nd[2][ROLE == DQ ? 4 : C::KB];
  alignas(16) float4 row[ROLE == DQ ? 128 : 1];       // DQ: sums of the rows that stay
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
  const int rank = (int)(blockIdx.x / p.heads), hd = (int)(blockIdx.x % p.heads);
  const int g = Q_STAYS ? hd / p.chunks : hd;                             // key head
  const int h0 = Q_STAYS ? g * p.hpg + hd % p.chunks * p.ht : g * p.hpg;  // first query head
  const int nh = Q_STAYS ? min(p.ht, (g + 1) * p.hpg - h0) : p.hpg;
  const int block_tok = Q_STAYS ? p.tok : 128;

  if (threadIdx.x == 0) {
    mbar_init(&x.r_full, 1);
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
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < p.seq.batch; b += blockDim.x) seq_span(p.seq, b, -1, &bad);
    if (bad) atomicOr(p.status, STATUS_BAD_INDEX);
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
  if (warp == 2) {
    int b, i = 0;
    if (p.by_length) {
      const int most = p.window > 0 ? (p.window + block_tok) / KB + 2 + (Q_STAYS ? (p.sinks + KB - 1) / KB : 0) : 0x7fffffff;
      ByLength<KB> order;
      order.init(p.seq, -1, block_tok, most, lane);
      order.find(rank, lane, &b, &i);
    } else {
      b = find_slot(p.seq, p.slots, (int)p.slots.count - 1 - rank, lane);
      i = -1;  // below
    }
    if (lane == 0) {
      BwdBlock k;
      k.b = -1;
      k.n = 0;
      if (b >= 0) {
        bool bad = false;
        const SeqSpan s = seq_span(p.seq, b, -1, &bad);
        if (i < 0) i = (int)p.slots.count - 1 - rank - slot_base(p.slots, s.first, b);
        if (i >= 0 && (int64_t)i * block_tok < s.count) {
          // key blocks from the first on are the long ones
          if (!Q_STAYS) i = (s.count - 1) / block_tok - i;
          k.b = b;
          k.first = s.first;
          k.count = s.count;
          k.at = i * block_tok;
          if (Q_STAYS) {
            k.end = min(k.at + block_tok, s.count);
            k.lo = p.window > 0 ? max(0, k.at + 1 - p.window) : 0;
            k.sink_end = min(p.sinks, k.lo);
            k.win_tile = k.lo / KB;
            k.sink_tiles = min((k.sink_end + KB - 1) / KB, k.win_tile);
            k.n = k.sink_tiles + (k.end + KB - 1) / KB - k.win_tile;
          } else {
            // the tokens [at, end) see keys of the block
            const int last = min(k.at + block_tok, s.count) - 1;
            k.end = p.window > 0 && k.at >= p.sinks ? (int)min((int64_t)s.count, (int64_t)last + p.window) : s.count;
            k.lo = k.sink_end = k.win_tile = k.sink_tiles = 0;
            k.n = (k.end - k.at + p.stok - 1) / p.stok * p.schunks;
          }
        }
      }
      x.blk = k;
    }
  }
  if (warp == 1) {
    tmem_alloc(&x.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = x.tmem;
  const BwdBlock blk = x.blk;
  // DQ: D = dO . O takes the output as it was rounded.  For tokens that see few
  // others D is as large as what it is taken from, and that rounding would be a
  // good part of a small gradient (dq off by 0.0026 of its norm where its own
  // rounding is 0.0017).  Blocks of few steps run over their keys once more,
  // before, for D = sum P dP: with 256 keys or more the rounding is averaged out.
  const int pre = Q_STAYS && blk.n <= C::TWICE ? blk.n : 0;
  const int nk = blk.n + pre;
  auto tile_of = [&](int n) -> int {
    const int j = n < pre ? n : n - pre;
    return j < blk.sink_tiles ? j : j - blk.sink_tiles + blk.win_tile;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> int {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
  };
  // where dS goes: over the scores, with two score buffers; else over dP
  constexpr bool DS_OVER_S = NS == 2;
  auto ds_col = [&](int n) -> uint32_t { return DS_OVER_S ? (n & 1) * KB : C::T_DP; };
  auto s_col = [&](int n) -> uint32_t { return NS == 2 ? (n & 1) * KB : 0; };

  if (warp < 4) {
  regs_dec<ISSUE_REGS>();
  if (warp == 0 && nk > 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t armed[2] = {0, 0}, par_armed[2] = {0, 0};
      bool ok = true;
      const uint32_t rows = Q_STAYS ? p.ht * p.tok : 128;
      mbar_arrive_expect_tx(&x.r_full, C::NRES * (D / 64) * rows * 128);
      for (int o = 0; o < C::NRES; ++o)
        for (int t = 0; t < D / 64; ++t)
          tma_load_3d(smem + o * C::RB + t * C::RSUB, o ? &map_r2 : &map_r1, &x.r_full, 64 * t, Q_STAYS ? h0 : g,
                      blk.first + blk.at);
      const uint32_t bytes = (uint32_t)(Q_STAYS ? KB : p.sht * p.stok) * EC * 2;
      for (int n = 0; ok && n < nk; ++n) {
        const int c1 = Q_STAYS ? g : h0 + n % p.schunks * p.sht;
        const int c2 = blk.first + (Q_STAYS ? tile_of(n) * KB : blk.at + n / p.schunks * p.stok);
        for (int o = 0; ok && o < 2; ++o) {
          const int stages = o ? N2 : N1;
          uint64_t *fb = o ? x.full2 : x.full1, *eb = o ? x.empty2 : x.empty1;
          uint8_t* ring = o ? ring2 : ring1;
          for (int e = 0; e < NE; ++e) {
            const int at = n * NE + e, s = at % stages;
            const uint32_t par = (uint32_t)((at / stages) & 1);
            if (!mbar_wait(&eb[s], par ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&fb[s], bytes);
            armed[o] |= 1u << s;
            par_armed[o] = (par_armed[o] & ~(1u << s)) | (par << s);
            for (int t = 0; t < EC / 64; ++t)
              tma_load_3d(ring + s * C::EB + t * C::SUB, o ? &map_x2 : &map_x1, &fb[s], e * EC + 64 * t, c1, c2);
          }
        }
      }
      if (!ok || *abort_flag) {  // copies still in flight land on the barriers armed last
        int no_abort = 0;
        mbar_wait(&x.r_full, 0, &no_abort, p.status, 0u, DRAIN_NS);
        for (int o = 0; o < 2; ++o)
          for (int s = 0; s < (o ? N2 : N1); ++s)
            if (armed[o] & (1u << s))
              mbar_wait(o ? &x.full2[s] : &x.full1[s], (par_armed[o] >> s) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 16);
      }
    }
  } else if (warp == 1 && nk > 0) {
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
    auto accumulate = [&](int stages, uint64_t xm, int n, uint32_t a_col, uint32_t acc) {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const uint64_t b = desc_advance(xm, ((n * NE + e) % stages) * C::EB);
#pragma unroll
        for (int kk = 0; kk < KB / 16; ++kk)
          tc_mma_f16_ts(tmem_base + acc + e * EC, tmem_base + a_col + kk / (HC / 16) * HC + kk % (HC / 16) * 8,
                        desc_advance(b, kk * 2048), IDESC_A, n > pre || kk > 0 ? 1u : 0u);
      }
    };
    auto release = [&](uint64_t* bars, int stages, int n) {
#pragma unroll
      for (int e = 0; e < NE; ++e) tc_commit(&bars[(n * NE + e) % stages]);
    };
    auto put_s = [&](int n) {
      product(0, N1, x1k, n, s_col(n));
      tc_commit(&x.s_full[NS == 2 ? n & 1 : 0]);
      if (!C::HAS_DP) release(x.empty1, N1, n);
    };
    auto put_dp = [&](int n) {
      product(1, N2, x2k, n, C::T_DP);
      tc_commit(&x.dp_full);
      if (!C::HAS_PV) release(x.empty2, N2, n);
    };
    auto put_acc = [&](int n) {  // dS X1
      if (n >= pre) accumulate(N1, x1m, n, ds_col(n), C::T_ACC);
      release(x.empty1, N1, n);
      if (n + 1 == nk) tc_commit(&x.acc_full);
    };
    auto put_pv = [&](int n) {  // P X2
      accumulate(N2, x2m, n, s_col(n), C::T_ACC + (ROLE == DKV ? D : 0));
      release(x.empty2, N2, n);
      if (!C::HAS_DP && n + 1 == nk) tc_commit(&x.acc_full);
    };
    int ok = wait_all(&x.r_full, 0) && wait_elems(x.full1, N1, 0);
    if (ok && C::HAS_DP) ok = wait_elems(x.full2, N2, 0);
    tc_fence_after();
    if (ok && elect_one()) {
      put_s(0);
      if (C::HAS_DP) put_dp(0);
    }
    __syncwarp();
    if (ok && NS == 2 && nk > 1 && (ok = wait_elems(x.full1, N1, 1))) {
      tc_fence_after();
      if (elect_one()) put_s(1);
      __syncwarp();
    }
    for (int n = 0; ok && n < nk; ++n) {
      const uint32_t par = (uint32_t)(n & 1);
      const bool n1 = n + 1 < nk, n2 = n + 2 < nk;
      if constexpr (C::HAS_DP && !C::HAS_PV && NS == 2) {
        // dP_{n+1}, then dS_n X1 and S_{n+2} while the row groups turn dP_{n+1} into dS
        if (n1 && !(ok = wait_elems(x.full2, N2, n + 1))) break;
        if (!(ok = wait_all(&x.ds_full, par))) break;
        tc_fence_after();
        if (elect_one()) {
          if (n1) put_dp(n + 1);
          put_acc(n);
        }
        __syncwarp();
        if (n2) {  // its rows come into the place of step n - 1's
          if (!(ok = wait_elems(x.full1, N1, n + 2))) break;
          tc_fence_after();
          if (elect_one()) put_s(n + 2);
          __syncwarp();
        }
      } else if constexpr (C::HAS_DP && !C::HAS_PV) {
        if (n1) {
          if (!(ok = wait_elems(x.full1, N1, n + 1) && wait_all(&x.p_full[0], par))) break;  // the scores are read
          tc_fence_after();
          if (elect_one()) put_s(n + 1);
          __syncwarp();
        }
        if (!(ok = wait_all(&x.ds_full, par))) break;
        tc_fence_after();
        if (elect_one()) put_acc(n);
        __syncwarp();
        if (n1) {
          if (!(ok = wait_elems(x.full2, N2, n + 1))) break;
          tc_fence_after();
          if (elect_one()) put_dp(n + 1);
          __syncwarp();
        }
      } else if constexpr (C::HAS_DP) {
        // dV_n and S_{n+1} under the row groups' dS_n, dK_n and dP_{n+1} under their P_{n+1}
        if (n1 && !(ok = wait_elems(x.full1, N1, n + 1))) break;
        if (!(ok = wait_all(&x.p_full[0], par))) break;
        tc_fence_after();
        if (elect_one()) {
          put_pv(n);
          if (n1) put_s(n + 1);
        }
        __syncwarp();
        if (n1 && !(ok = wait_elems(x.full2, N2, n + 1))) break;
        if (!(ok = wait_all(&x.ds_full, par))) break;
        tc_fence_after();
        if (elect_one()) {
          put_acc(n);
          if (n1) put_dp(n + 1);
        }
        __syncwarp();
      } else {
        if (n2 && !(ok = wait_elems(x.full1, N1, n + 2))) break;
        if (!(ok = wait_elems(x.full2, N2, n) && wait_all(&x.p_full[n & 1], (uint32_t)((n >> 1) & 1)))) break;
        tc_fence_after();
        if (elect_one()) {
          put_pv(n);
          if (n2) put_s(n + 2);
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(&x.drain);
    __syncwarp();
    int no_abort = 0;
    mbar_wait(&x.drain, 0, &no_abort, p.status, STATUS_TIMEOUT, DRAIN_NS);
  } else if (warp == 2 && !Q_STAYS && nk > 0) {
    // ---------------------------------------- statistics of the streamed rows
    int ok = 1;
    for (int n = 0; ok && n < nk; ++n) {
      const int st = n & 1;
      const int tok0 = blk.at + n / p.schunks * p.stok, hc = n % p.schunks * p.sht;
      float2 v[KB / 32];
#pragma unroll
      for (int k = 0; k < KB / 32; ++k) {
        const int r = lane + 32 * k, tk = tok0 + r / p.sht, hh = hc + r % p.sht;
        const bool valid = r < p.sht * p.stok && tk < blk.end && hh < p.hpg;
        v[k] = valid ? __ldg(p.stats + (int64_t)(blk.first + tk) * p.nq + h0 + hh) : make_float2(INFINITY, 0.0f);
      }
      ok = wait_all(&x.stat_empty[st], (uint32_t)((n >> 1) & 1) ^ 1u);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < KB / 32; ++k) {
        x.nlse2[st][lane + 32 * k] = -v[k].x;
        x.nd[st][lane + 32 * k] = -v[k].y;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.stat_full[st]);
    }
  }
  } else if (regs_inc<ROW_REGS>(), nk > 0) {
    // ------------------------------------------------------------ row groups
    // Both work on every step, each on half of its columns: that halves the
    // time from scores to P and from dP to dS, which the products of the other
    // kind hide.
    const int grp = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the accumulators
    const int tid = grp * 128 + r;
    const uint32_t tl = tmem_base + ((uint32_t)(q4 * 32) << 16) + grp * HC;
    // DQ: this row's token and head; else its key
    const int tk = Q_STAYS ? blk.at + r / p.ht : blk.at + r;
    const int hh = Q_STAYS ? r % p.ht : 0;
    const bool stored = tk < blk.count && (!Q_STAYS || (r < p.ht * p.tok && hh < nh));
    const int64_t stat_at = (int64_t)(blk.first + tk) * p.nq + h0 + hh;
    const uint32_t magic = 65536u / (uint32_t)p.sht + 1u;  // c / sht = c magic >> 16 for c < 128
    float lse2 = 0.0f, dsum = 0.0f;
    if (Q_STAYS) {
      if (stored) lse2 = p.lse[stat_at] * 1.4426950408889634f;
      if (!pre) {
        // D = dO . O of 16 rows a warp, D / 8 lanes a row
        constexpr int LPR = D / 8, RPP = D == 192 ? 1 : 32 / LPR;
        for (int i = 0; i < 16; i += RPP) {
          const int rr = (warp - 4) * 16 + i + (RPP > 1 ? lane / LPR : 0);
          const int c = RPP > 1 ? lane % LPR : lane;
          const int t = blk.at + rr / p.ht, h = rr % p.ht;
          float s = 0.0f;
          if (t < blk.count && rr < p.ht * p.tok && h < nh && c < LPR) {
            const int64_t row = blk.first + t, col = (int64_t)(h0 + h) * D + 8 * c;
            const uint4 a = *reinterpret_cast<const uint4*>(p.dout + row * p.ld_dout + col);
            const uint4 o = *reinterpret_cast<const uint4*>(p.out + row * p.ld_out + col);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s = fmaf(__uint_as_float(aw[k] << 16), __uint_as_float(ow[k] << 16), s);
              s = fmaf(__uint_as_float(aw[k] & 0xffff0000u), __uint_as_float(ow[k] & 0xffff0000u), s);
            }
          }
#pragma unroll
          for (int o = (RPP > 1 ? LPR : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (c == 0) x.row[rr].x = s;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        dsum = x.row[r].x;
        if (stored && grp == 0) p.stats[stat_at] = make_float2(lse2, dsum);
      }
    }
    int ok = 1;
    // The first run over few keys: sum P, and sum P (dP - dref) with dref the
    // dP of the first key that the row sees: exact where it sees no other.
    float l = 0.0f, dref = 0.0f;
    for (int n = 0; n < nk; ++n) {
      const uint32_t par = (uint32_t)(n & 1), par2 = (uint32_t)((n >> 1) & 1);
      const int st = n & 1;
      if (Q_STAYS && pre && n == pre) {  // both groups' sums
        if (grp == 1) x.row[r] = make_float4(l, dsum, dref, 0.0f);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (grp == 0) {
          const float4 o = x.row[r];
          const float all = l + o.x;
          const float d = l != 0.0f ? dref + (dsum + o.y + (o.x != 0.0f ? o.x * (o.z - dref) : 0.0f)) / all
                                    : o.z + (o.y + dsum) / all;
          x.row[r] = make_float4(all, d, 0.0f, 0.0f);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        lse2 += log2f(x.row[r].x);
        dsum = x.row[r].y;
        if (stored && grp == 0) p.stats[stat_at] = make_float2(lse2, dsum);
      }
      if (!Q_STAYS && !(ok = wait_all(&x.stat_full[st], par2))) break;
      if (!(ok = wait_all(&x.s_full[NS == 2 ? n & 1 : 0], NS == 2 ? par2 : par))) break;
      tc_fence_after();
      const uint32_t t_s = tl + s_col(n);
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
      int t0 = 0, tok0 = 0, hc = 0;
      if (Q_STAYS) {
        const int tile0 = tile_of(n) * KB;
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
                  *reinterpret_cast<uint4*>(ring1 + ((n * NE + e) % N1) * C::EB + cb * C::SUB + crow * 128 +
                                            (cpart + c) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
      } else {
        tok0 = blk.at + n / p.schunks * p.stok;
        hc = n % p.schunks * p.sht;
        const bool cut = tok0 + p.stok > blk.end || hc + p.sht > p.hpg;
        masked = cut || blk.at + 127 > tok0 ||
                 (p.window > 0 && tok0 + p.stok - 1 - blk.at >= p.window && blk.at + 128 > p.sinks);
        if (cut) {
          if (C::HAS_PV)
            for (int e = 0; ok && e < NE; ++e)
              ok = wait_all(&x.full2[(n * NE + e) % N2], (uint32_t)(((n * NE + e) / N2) & 1));
          if (!ok) break;
          if (crow < p.sht * p.stok && (tok0 + crow / p.sht >= blk.end || hc + crow % p.sht >= p.hpg))
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                  const uint32_t o = cb * C::SUB + crow * 128 + (cpart + c) * 16;
                  if (C::HAS_DP) *reinterpret_cast<uint4*>(ring1 + ((n * NE + e) % N1) * C::EB + o) = make_uint4(0, 0, 0, 0);
                  if (C::HAS_PV) *reinterpret_cast<uint4*>(ring2 + ((n * NE + e) % N2) * C::EB + o) = make_uint4(0, 0, 0, 0);
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
            const int hi = tk - t, lo = p.window > 0 ? tk - p.window - t : -1, sk = p.window > 0 ? p.sinks - t : 0;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c > hi || (c <= lo && c >= sk)) u[c] = 0u;
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
            const bool sink = p.window == 0 || tk < p.sinks;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int cc = grp * HC + 32 * hf + c, dt = (int)((uint32_t)cc * magic >> 16), q = tok0 + dt;
              const bool seen = tk <= q && q < blk.end && hc + cc - dt * p.sht < p.hpg && (sink || q - tk < p.window);
              if (!seen) u[c] = 0u;
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
        if (lane == 0) mbar_arrive(&x.p_full[NS == 2 ? n & 1 : 0]);
      }
      if (C::HAS_DP) {
        if (!(ok = wait_all(&x.dp_full, par))) break;
        tc_fence_after();
        const uint32_t t_dp = tl + C::T_DP;
        uint32_t dd[HC];
        tmem_ld_32x32b_x32(t_dp, *reinterpret_cast<uint32_t(*)[32]>(dd));
        tmem_ld_wait();
        if constexpr (HC == 64) tmem_ld_32x32b_x32(t_dp + 32, *reinterpret_cast<uint32_t(*)[32]>(dd + 32));
#pragma unroll
        for (int hf = 0; hf < HC / 32; ++hf) {
          uint32_t* d = dd + 32 * hf;
          if (hf == 1) tmem_ld_wait();
          if (Q_STAYS && n < pre) {  // the sums alone
#pragma unroll
            for (int c = 0; c < 32; ++c)  // hidden values may be anything
              if (v[32 * hf + c] != 0u) {
                if (l == 0.0f) dref = __uint_as_float(d[c]);
                l += __uint_as_float(v[32 * hf + c]);
                dsum = fmaf(__uint_as_float(v[32 * hf + c]), __uint_as_float(d[c]) - dref, dsum);
              }
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
          if constexpr (HC == 64) tmem_st_32x32b_x32(tl + ds_col(n), w);
          else tmem_st_32x32b_x16(tl + ds_col(n), w);
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
    if (ok && (ok = wait_all(&x.acc_full, 0))) {
      tc_fence_after();
      // DKV: group 0 dV, group 1 dK; else each group half of the columns.  The warp's rows
      // are turned in shared memory, which nothing uses any more.
      constexpr int W = ROLE == DKV ? D : D / 2;
      const uint32_t t_acc =
          tmem_base + ((uint32_t)(q4 * 32) << 16) + C::T_ACC + (ROLE == DKV ? (grp ? 0 : D) : grp * W);
      __nv_bfloat16* dst;
      int64_t off;
      if (Q_STAYS) {
        dst = p.dq;
        off = (int64_t)(blk.first + tk) * p.ld_dq + (int64_t)(h0 + hh) * D + grp * W;
      } else if (ROLE == DV || (ROLE == DKV && grp == 0)) {
        dst = p.dv;
        off = (int64_t)(blk.first + tk) * p.ld_dv + (int64_t)g * D + (ROLE == DKV ? 0 : grp * W);
      } else {
        dst = p.dk;
        off = (int64_t)(blk.first + tk) * p.ld_dk + (int64_t)g * D + (ROLE == DKV ? 0 : grp * W);
      }
      if (!stored) off = -1;
      const float fin = ROLE == DV || (ROLE == DKV && grp == 0) ? 1.0f : p.scale;
      constexpr int PITCH = W * 2 + 16;
      uint8_t* stg = smem + (warp - 4) * (32 * PITCH);
#pragma unroll 1
      for (int c = 0; c < W / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(t_acc + 32 * c, o);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(stg + lane * PITCH + 64 * c + 16 * k) =
              make_uint4(pack_bf16(__uint_as_float(o[8 * k]) * fin, __uint_as_float(o[8 * k + 1]) * fin),
                         pack_bf16(__uint_as_float(o[8 * k + 2]) * fin, __uint_as_float(o[8 * k + 3]) * fin),
                         pack_bf16(__uint_as_float(o[8 * k + 4]) * fin, __uint_as_float(o[8 * k + 5]) * fin),
                         pack_bf16(__uint_as_float(o[8 * k + 6]) * fin, __uint_as_float(o[8 * k + 7]) * fin));
      }
      __syncwarp();
      constexpr int CH = W / 8;
#pragma unroll 4
      for (int u = lane; u < 32 * CH; u += 32) {
        const int rr = u / CH, c = u % CH;
        const int64_t to = __shfl_sync(0xffffffffu, off, rr);
        if (to >= 0) *reinterpret_cast<uint4*>(dst + to + 8 * c) = *reinterpret_cast<const uint4*>(stg + rr * PITCH + 16 * c);
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
  if (units > 0x7fffffff / 2) return cudaErrorInvalidConfiguration;
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
  var_bwd_kernel<D, ROLE><<<(unsigned)units, 384, SMEM, st>>>(r1, r2, x1, x2, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const BwdParams& p, const VarBwdArgs& a, int num_sms, cudaStream_t st) {
  cudaError_t e = launch_role<D, DQ>(p, a, num_sms, st);  // writes the statistics that the others read
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
  p.out = static_cast<const __nv_bfloat16*>(a.out);
  p.dout = static_cast<const __nv_bfloat16*>(a.dout);
  p.ld_out = a.ld_out;
  p.ld_dout = a.ld_dout;
  p.lse = a.lse;
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
