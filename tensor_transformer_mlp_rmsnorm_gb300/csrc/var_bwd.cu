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

constexpr int KB = 64;  // rows of a step
constexpr int TWICE = 4;  // DQ: blocks of 2 to TWICE steps run over their keys twice
constexpr uint64_t WAIT_NS = 1000000000ull, DRAIN_NS = 200000000ull;

// What a CTA accumulates.  DQ: 128 rows of (token, head) stay, their keys and
// values stream by.  The others: 128 keys stay, the rows of (token, head) that
// see them stream by; DKV both gradients, DV and DK one.
enum Role { DQ = 0, DKV = 1, DV = 2, DK = 3 };

template <int D, int ROLE>
struct Cfg {
  static constexpr bool HAS_DP = ROLE != DV;                   // dP and dS are needed
  static constexpr bool HAS_PV = ROLE == DKV || ROLE == DV;    // P^T dO is accumulated
  static constexpr int EC = D % 128 == 0 ? 128 : 64;           // columns of a ring element
  static constexpr int NE = D / EC;                            // elements of a streamed operand
  static constexpr uint32_t SUB = 64 * 128;                    // a [64 x 64] tile
  static constexpr uint32_t EB = EC / 64 * SUB;                // an element [64 x EC]
  static constexpr uint32_t RSUB = 128 * 128;                  // a [128 x 64] tile
  static constexpr uint32_t RB = D / 64 * RSUB;                // a resident operand [128 x D]
  static constexpr int NRES = HAS_DP ? 2 : 1;
  // stages of the streamed rows' statistics; heads of 256 leave little room
  static constexpr int NSTAT = ROLE == DQ ? 1 : D == 256 ? 2 : 4;
  static constexpr int FIT = (int)(((D == 256 ? 224 : 222) * 1024 - NRES * RB) / EB);
  // stages of the two streamed operands.  Two steps ahead needs three steps of
  // the first (scores, and dS times it at the end of the step).
  static constexpr int LOOK = FIT >= 5 * NE ? 2 : 1;
  static constexpr int CAP = FIT < 16 ? FIT : 16;
  static constexpr int N2 = LOOK == 2 ? (CAP / 2 / NE < 2 ? 2 * NE : CAP / 2 / NE * NE) : NE;
  static constexpr int N1 = (CAP - N2) / NE * NE;
  static constexpr uint32_t SMEM = NRES * RB + (N1 + N2) * EB + 1024;
  static_assert(N1 >= (LOOK + 1) * NE && N2 >= NE, "ring");
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
  int sht, schunks, stok;  // the others: of a step of 64 rows
  int slots, heads;
  bool by_length;
  float scale, scale_log2;
  int window, sinks;
  uint32_t* status;
};

struct BwdBlock {
  int b;                 // < 0: none
  int first, count;      // rows of the sequence
  int at, n;             // first token of the block, steps
  int sink_tiles, win_tile, lo, end, sink_end;  // DQ: as in the forward, in tiles of 64 keys
};

template <int D, int ROLE>
__global__ void __launch_bounds__(384, 1)
    var_bwd_kernel(const __grid_constant__ CUtensorMap map_r1, const __grid_constant__ CUtensorMap map_r2,
                   const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_x2,
                   const BwdParams p) {
  using C = Cfg<D, ROLE>;
  constexpr int NE = C::NE, EC = C::EC, N1 = C::N1, N2 = C::N2, LOOK = C::LOOK, NSTAT = C::NSTAT;
  constexpr bool Q_STAYS = ROLE == DQ;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t r_full, full1[N1], empty1[N1], full2[N2], empty2[N2], s_full[2], p_full[2], dp_full[2],
      ds_full[2], stat_full[NSTAT], stat_empty[NSTAT], acc_full, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ BwdBlock blk;
  __shared__ __align__(16) float2 s_stat[NSTAT][Q_STAYS ? 2 : KB];
  __shared__ __align__(16) int s_pos[NSTAT][Q_STAYS ? 4 : KB];
  __shared__ float2 s_row[Q_STAYS ? 128 : 1];  // sums of the rows that stay
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring1 = smem + C::NRES * C::RB;
  uint8_t* ring2 = ring1 + N1 * C::EB;
  volatile int* abort_flag = &abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x / p.heads), hd = (int)(blockIdx.x % p.heads);
  const int g = Q_STAYS ? hd / p.chunks : hd;                         // key head
  const int h0 = Q_STAYS ? g * p.hpg + hd % p.chunks * p.ht : g * p.hpg;  // first query head
  const int nh = Q_STAYS ? min(p.ht, (g + 1) * p.hpg - h0) : p.hpg;
  const int block_tok = Q_STAYS ? p.tok : 128;

  if (threadIdx.x == 0) {
    mbar_init(&r_full, 1);
    for (int i = 0; i < N1; ++i) {
      mbar_init(&full1[i], 1);
      mbar_init(&empty1[i], 1);
    }
    for (int i = 0; i < N2; ++i) {
      mbar_init(&full2[i], 1);
      mbar_init(&empty2[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&dp_full[i], 1);
      mbar_init(&ds_full[i], 4);
    }
    for (int i = 0; i < NSTAT; ++i) {
      mbar_init(&stat_full[i], 1);
      mbar_init(&stat_empty[i], 4);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_r1);
    tma_prefetch_desc(&map_r2);
    tma_prefetch_desc(&map_x1);
    tma_prefetch_desc(&map_x2);
  }
  int2* sq = reinterpret_cast<int2*>(smem);  // until the first copy
  if (p.by_length || blockIdx.x == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < p.seq.batch; b += blockDim.x) {
      const SeqSpan s = seq_span(p.seq, b, -1, &bad);
      if (p.by_length) sq[b] = make_int2(0, s.count);
    }
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
  if (p.by_length) __syncthreads();
  if (warp == 2) {
    int b, i = 0;
    if (p.by_length) {
      const int most = p.window > 0 ? (p.window + block_tok) / KB + 2 + (Q_STAYS ? (p.sinks + KB - 1) / KB : 0) : 0x7fffffff;
      find_by_length<KB>(sq, p.seq.batch, rank, block_tok, most, lane, &b, &i);
    } else {
      b = find_slot(p.seq, p.slots - 1 - rank, block_tok, lane);
      i = -1;  // below
    }
    if (lane == 0) {
      BwdBlock k;
      k.b = -1;
      k.n = 0;
      if (b >= 0) {
        bool bad = false;
        const SeqSpan s = seq_span(p.seq, b, -1, &bad);
        if (i < 0) i = p.slots - 1 - rank - slot_base(s.first, b, block_tok);
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
  // DQ: D = dO . O takes the output as it was rounded.  For tokens that see few
  // others D is as large as what it is taken from, and that rounding would be a
  // good part of a small gradient (dq off by 0.0026 of its norm where its own
  // rounding is 0.0017).  Blocks of few steps run over their keys once more,
  // before, for D = sum P dP: with 256 keys or more the rounding is averaged out.
  const int pre = Q_STAYS && blk.n > 1 && blk.n <= TWICE ? blk.n : 0;
  const int nk = blk.n + pre;
  constexpr uint32_t T_DP = 128, T_ACC = 256;  // score slots at 0 and 64, dP slots at 128 and 192
  auto tile_of = [&](int n) -> int {
    const int j = n < pre ? n : n - pre;
    return j < blk.sink_tiles ? j : j - blk.sink_tiles + blk.win_tile;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> int {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, p.status, STATUS_TIMEOUT, WAIT_NS));
  };

  if (warp == 0 && nk > 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t armed[2] = {0, 0}, par_armed[2] = {0, 0};
      bool ok = true;
      const uint32_t rows = Q_STAYS ? p.ht * p.tok : 128;
      mbar_arrive_expect_tx(&r_full, C::NRES * (D / 64) * rows * 128);
      for (int o = 0; o < C::NRES; ++o)
        for (int t = 0; t < D / 64; ++t)
          tma_load_3d(smem + o * C::RB + t * C::RSUB, o ? &map_r2 : &map_r1, &r_full, 64 * t, Q_STAYS ? h0 : g,
                      blk.first + blk.at);
      const uint32_t bytes = (uint32_t)(Q_STAYS ? KB : p.sht * p.stok) * EC * 2;
      for (int n = 0; ok && n < nk; ++n) {
        const int c1 = Q_STAYS ? g : h0 + n % p.schunks * p.sht;
        const int c2 = blk.first + (Q_STAYS ? tile_of(n) * KB : blk.at + n / p.schunks * p.stok);
        for (int o = 0; ok && o < 2; ++o) {
          const int stages = o ? N2 : N1;
          uint64_t *fb = o ? full2 : full1, *eb = o ? empty2 : empty1;
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
        mbar_wait(&r_full, 0, &no_abort, p.status, 0u, DRAIN_NS);
        for (int o = 0; o < 2; ++o)
          for (int s = 0; s < (o ? N2 : N1); ++s)
            if (armed[o] & (1u << s))
              mbar_wait(o ? &full2[s] : &full1[s], (par_armed[o] >> s) & 1u, &no_abort, p.status, 0u, DRAIN_NS / 16);
      }
    }
  } else if (warp == 1 && nk > 0) {
    // ---------------------------------------------------------------- issuer
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, KB, false, false);
    constexpr uint32_t IDESC_A = idesc_bf16_f32(128, EC, false, true);
    const uint64_t r_desc = sw128_desc(smem_u32(smem), 16, 1024);
    const uint64_t x1k = sw128_desc(smem_u32(ring1), 16, 1024), x2k = sw128_desc(smem_u32(ring2), 16, 1024);
    const uint64_t x1m = sw128_desc(smem_u32(ring1), C::SUB, 1024), x2m = sw128_desc(smem_u32(ring2), C::SUB, 1024);
    auto wait_elems = [&](uint64_t* bars, int stages, int n) -> int {
      int r = 1;
      for (int e = 0; r && e < NE; ++e)
        r = wait_all(&bars[(n * NE + e) % stages], (uint32_t)(((n * NE + e) / stages) & 1));
      return r;
    };
    // scores: resident operand `o` times the streamed one, 64 columns at `col`
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
    // accumulator at `acc` += (bf16 rows at `a_col`) times the streamed operand
    auto accumulate = [&](int stages, uint64_t xm, int n, uint32_t a_col, uint32_t acc) {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const uint64_t b = desc_advance(xm, ((n * NE + e) % stages) * C::EB);
#pragma unroll
        for (int kk = 0; kk < KB / 16; ++kk)
          tc_mma_f16_ts(tmem_base + acc + e * EC, tmem_base + a_col + kk * 8, desc_advance(b, kk * 2048), IDESC_A,
                        n > pre || kk > 0 ? 1u : 0u);
      }
    };
    auto release = [&](uint64_t* bars, int stages, int n) {
#pragma unroll
      for (int e = 0; e < NE; ++e) tc_commit(&bars[(n * NE + e) % stages]);
    };
    auto issue_s = [&](int n) -> int {
      if (!wait_elems(full1, N1, n)) return 0;
      tc_fence_after();
      if (elect_one()) {
        product(0, N1, x1k, n, (n & 1) * KB);
        tc_commit(&s_full[n & 1]);
        if (!C::HAS_DP) release(empty1, N1, n);
      }
      __syncwarp();
      return 1;
    };
    auto issue_dp = [&](int n) -> int {
      if (!C::HAS_DP) return 1;
      if (!wait_elems(full2, N2, n)) return 0;
      tc_fence_after();
      if (elect_one()) {
        product(1, N2, x2k, n, T_DP + (n & 1) * KB);
        tc_commit(&dp_full[n & 1]);
        if (!C::HAS_PV) release(empty2, N2, n);
      }
      __syncwarp();
      return 1;
    };
    int ok = wait_all(&r_full, 0);
    for (int n = 0; ok && n < LOOK && n < nk; ++n) ok = issue_s(n) && issue_dp(n);
    for (int n = 0; ok && n < nk; ++n) {
      const int slot = n & 1;
      const uint32_t par = (uint32_t)((n >> 1) & 1);
      if (LOOK == 1 && n + 1 < nk && !(ok = issue_s(n + 1) && issue_dp(n + 1))) break;
      // the scores have been read; with a product of its own, P is in their place
      if (!(ok = wait_all(&p_full[slot], par))) break;
      if (C::HAS_PV) {
        if (!C::HAS_DP && !(ok = wait_elems(full2, N2, n))) break;
        tc_fence_after();
        if (elect_one()) {
          accumulate(N2, x2m, n, slot * KB, T_ACC + (ROLE == DKV ? D : 0));
          release(empty2, N2, n);
          if (!C::HAS_DP && n + 1 == nk) tc_commit(&acc_full);
        }
        __syncwarp();
      }
      if (LOOK == 2 && n + 2 < nk && !(ok = issue_s(n + 2))) break;
      if (C::HAS_DP) {
        if (!(ok = wait_all(&ds_full[slot], par))) break;
        tc_fence_after();
        if (elect_one()) {
          if (n >= pre) accumulate(N1, x1m, n, T_DP + slot * KB, T_ACC);
          release(empty1, N1, n);
          if (n + 1 == nk) tc_commit(&acc_full);
        }
        __syncwarp();
        if (LOOK == 2 && n + 2 < nk && !(ok = issue_dp(n + 2))) break;
      }
    }
    if (elect_one()) tc_commit(&drain_bar);
    __syncwarp();
    int no_abort = 0;
    mbar_wait(&drain_bar, 0, &no_abort, p.status, STATUS_TIMEOUT, DRAIN_NS);
  } else if (warp == 2 && !Q_STAYS && nk > 0) {
    // --------------------------- statistics and positions of the streamed rows
    int ok = 1;
    for (int n = 0; ok && n < nk; ++n) {
      const int st = n % NSTAT;
      const int tok0 = blk.at + n / p.schunks * p.stok, hc = n % p.schunks * p.sht;
      float2 v[2];
      int pos[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = lane + 32 * k, tk = tok0 + r / p.sht, hh = hc + r % p.sht;
        const bool valid = r < p.sht * p.stok && tk < blk.end && hh < p.hpg;
        v[k] = valid ? __ldg(p.stats + (int64_t)(blk.first + tk) * p.nq + h0 + hh) : make_float2(INFINITY, 0.0f);
        pos[k] = valid ? tk : -1;
      }
      ok = wait_all(&stat_empty[st], (uint32_t)((n / NSTAT) & 1) ^ 1u);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s_stat[st][lane + 32 * k] = v[k];
        s_pos[st][lane + 32 * k] = pos[k];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[st]);
    }
  } else if (warp >= 4 && nk > 0) {
    // ------------------------------------------------------------ row groups
    const int grp = (warp - 4) >> 2;  // steps n with n & 1 == grp
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;     // row of the accumulators
    const uint32_t tl = tmem_base + ((uint32_t)(q4 * 32) << 16);
    const uint32_t t_s = tl + grp * KB, t_dp = tl + T_DP + grp * KB;
    // DQ: this row's token and head; else its key
    const int tk = Q_STAYS ? blk.at + r / p.ht : blk.at + r;
    const int hh = Q_STAYS ? r % p.ht : 0;
    const bool stored = tk < blk.count && (!Q_STAYS || (r < p.ht * p.tok && hh < nh));
    float lse2 = 0.0f, dsum = 0.0f;
    const bool one = Q_STAYS && nk == 1;  // every key that the rows see is in one step
    if (Q_STAYS) {
      const int64_t at = (int64_t)(blk.first + tk) * p.nq + h0 + hh;
      if (stored) lse2 = p.lse[at] * 1.4426950408889634f;
      if (!one && !pre) {
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
          if (c == 0) s_row[rr].x = s;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        dsum = s_row[r].x;
        if (stored && grp == 0) p.stats[at] = make_float2(lse2, dsum);
      }
    }
    int ok = 1;
    float l = 0.0f;  // of the steps before: sum P
    for (int n = grp; n < nk; n += 2) {
      if (Q_STAYS && pre && (n == pre || n == pre + 1)) {  // both groups' sums
        if (grp == 1) s_row[r] = make_float2(l, dsum);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (grp == 0) s_row[r] = make_float2(l + s_row[r].x, dsum + s_row[r].y);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        l = s_row[r].x;
        dsum = s_row[r].y / l;
        lse2 += log2f(l);
        if (stored && grp == 0) p.stats[(int64_t)(blk.first + tk) * p.nq + h0 + hh] = make_float2(lse2, dsum);
      }
      const uint32_t par = (uint32_t)((n >> 1) & 1);
      const int st = n % NSTAT;
      if (!Q_STAYS && !(ok = wait_all(&stat_full[st], (uint32_t)((n / NSTAT) & 1)))) break;
      if (!(ok = wait_all(&s_full[grp], par))) break;
      tc_fence_after();
      uint32_t v[64];
      tmem_ld_32x32b_x32(t_s, *reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_ld_32x32b_x32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      tmem_ld_wait();
      // Streamed rows that none of ours sees (other sequences', or behind the end) are
      // cleared where a product sums over them.  A wait for a ring stage is good for the
      // next phase only: what was in the stage before has landed, as the scores of this
      // step are complete.
      bool masked;
      if (Q_STAYS) {
        const int t0 = tile_of(n) * KB;
        const int last = blk.at + min(p.tok, blk.count - blk.at) - 1;
        masked = t0 + KB - 1 > blk.at || (p.window > 0 && last - t0 >= p.window && t0 + KB > p.sinks);
        if (t0 + KB > blk.end || (t0 < blk.lo && t0 + KB > blk.sink_end)) {
          const int t = t0 + (r & 63);
          if (t >= blk.end || (t < blk.lo && t >= blk.sink_end))
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  *reinterpret_cast<uint4*>(ring1 + ((n * NE + e) % N1) * C::EB + cb * C::SUB + (r & 63) * 128 +
                                            ((r >> 6) * 4 + c) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
      } else {
        const int tok0 = blk.at + n / p.schunks * p.stok, hc = n % p.schunks * p.sht;
        const bool cut = tok0 + p.stok > blk.end || hc + p.sht > p.hpg;
        masked = cut || blk.at + 127 > tok0 || (p.window > 0 && tok0 + p.stok - 1 - blk.at >= p.window && blk.at + 128 > p.sinks);
        if (cut) {
          if (C::HAS_PV)
            for (int e = 0; ok && e < NE; ++e)
              ok = wait_all(&full2[(n * NE + e) % N2], (uint32_t)(((n * NE + e) / N2) & 1));
          if (!ok) break;
          const int rr = r & 63;
          if (rr < p.sht * p.stok && (tok0 + rr / p.sht >= blk.end || hc + rr % p.sht >= p.hpg))
            for (int e = 0; e < NE; ++e)
#pragma unroll
              for (int cb = 0; cb < EC / 64; ++cb)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const uint32_t o = cb * C::SUB + rr * 128 + ((r >> 6) * 4 + c) * 16;
                  if (C::HAS_DP) *reinterpret_cast<uint4*>(ring1 + ((n * NE + e) % N1) * C::EB + o) = make_uint4(0, 0, 0, 0);
                  if (C::HAS_PV) *reinterpret_cast<uint4*>(ring2 + ((n * NE + e) % N2) * C::EB + o) = make_uint4(0, 0, 0, 0);
                }
          fence_proxy_async_smem();
        }
      }
      // P, in place of the scores
      if (Q_STAYS) {
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(-lse2, -lse2);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float a0, a1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nl2), a0, a1);
          v[c] = __float_as_uint(ex2_fast(a0));
          v[c + 1] = __float_as_uint(ex2_fast(a1));
        }
        if (masked) {
          const int t0 = tile_of(n) * KB;
          const int hi = tk - t0, lo = p.window > 0 ? tk - p.window - t0 : -1, sk = p.window > 0 ? p.sinks - t0 : 0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > hi || (c <= lo && c >= sk)) v[c] = 0u;
        }
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      } else {
        const float4* sp = reinterpret_cast<const float4*>(s_stat[st]);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float4 x = sp[c >> 1];
          v[c] = __float_as_uint(ex2_fast(fmaf(__uint_as_float(v[c]), p.scale_log2, -x.x)));
          v[c + 1] = __float_as_uint(ex2_fast(fmaf(__uint_as_float(v[c + 1]), p.scale_log2, -x.z)));
        }
        if (masked) {
          const int4* pp = reinterpret_cast<const int4*>(s_pos[st]);
          const bool sink = tk < p.sinks;
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const int4 x = pp[c >> 2];
            const int q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (tk > q[k] || (p.window > 0 && q[k] - tk >= p.window && !sink)) v[c + k] = 0u;
          }
        }
        if (C::HAS_PV) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) w[c >> 1] = pack_bf16(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
          tmem_st_32x32b_x32(t_s, w);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      }
      if (C::HAS_DP) {
        if (!(ok = wait_all(&dp_full[grp], par))) break;
        tc_fence_after();
        if (one) {
          // The softmax and D from the step itself: the gradient of a token that sees one or
          // two is close to 0, and the output's rounding in D would be all of it.
#pragma unroll
          for (int c = 0; c < 64; ++c) l += __uint_as_float(v[c]);
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = __float_as_uint(__fdiv_rn(__uint_as_float(v[c]), l));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t d[32];
            tmem_ld_32x32b_x32(t_dp + 32 * hf, d);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c)  // hidden values may be anything
              if (v[32 * hf + c] != 0u) dsum = fmaf(__uint_as_float(v[32 * hf + c]), __uint_as_float(d[c]), dsum);
          }
          lse2 += log2f(l);
          if (stored) p.stats[(int64_t)(blk.first + tk) * p.nq + h0 + hh] = make_float2(lse2, dsum);
        }
        if (Q_STAYS && n < pre) {  // the sums alone
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t d[32];
            tmem_ld_32x32b_x32(t_dp + 32 * hf, d);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c)  // hidden values may be anything
              if (v[32 * hf + c] != 0u) {
                l += __uint_as_float(v[32 * hf + c]);
                dsum = fmaf(__uint_as_float(v[32 * hf + c]), __uint_as_float(d[c]), dsum);
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ds_full[grp]);
          continue;
        }
        uint32_t w[32];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t d[32];
          tmem_ld_32x32b_x32(t_dp + 32 * hf, d);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const int cc = 32 * hf + c;
            uint64_t nd;
            if (Q_STAYS) {
              nd = f2_pack(-dsum, -dsum);
            } else {
              const float4 x = reinterpret_cast<const float4*>(s_stat[st])[cc >> 1];
              nd = f2_pack(-x.y, -x.w);
            }
            const uint64_t pv = f2_mul(f2_pack(__uint_as_float(v[cc]), __uint_as_float(v[cc + 1])), f2_pack(p.scale, p.scale));
            float d0, d1;
            f2_unpack(f2_mul(pv, f2_add(f2_pack(__uint_as_float(d[c]), __uint_as_float(d[c + 1])), nd)), d0, d1);
            if (masked) {  // 0 whatever dP is
              if (v[cc] == 0u) d0 = 0.0f;
              if (v[cc + 1] == 0u) d1 = 0.0f;
            }
            w[cc >> 1] = pack_bf16(d0, d1);
          }
        }
        tmem_st_32x32b_x32(t_dp, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[grp]);
      }
      if (!Q_STAYS) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&stat_empty[st]);
      }
    }
    if (ok && (ok = wait_all(&acc_full, 0))) {
      tc_fence_after();
      // DKV: group 0 dV, group 1 dK; else each group half of the columns.  The warp's rows
      // are turned in shared memory, which nothing uses any more.
      constexpr int W = ROLE == DKV ? D : D / 2;
      const uint32_t col = T_ACC + (ROLE == DKV ? (grp ? 0 : D) : grp * W);
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
      constexpr int PITCH = W * 2 + 16;
      uint8_t* stg = smem + (warp - 4) * (32 * PITCH);
#pragma unroll 1
      for (int c = 0; c < W / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tl + col + 32 * c, o);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(stg + lane * PITCH + 64 * c + 16 * k) =
              make_uint4(pack_bf16(__uint_as_float(o[8 * k]), __uint_as_float(o[8 * k + 1])),
                         pack_bf16(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3])),
                         pack_bf16(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5])),
                         pack_bf16(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7])));
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
  static_assert(C::SMEM + C::NSTAT * (ROLE == DQ ? 32 : KB * 12) + (ROLE == DQ ? 1024 : 0) + 500 <= 232448, "shared memory");
  const int block_tok = ROLE == DQ ? p.tok : 128;
  p.heads = ROLE == DQ ? a.nkv * p.chunks : a.nkv;
  const int64_t slots = a.seq.rows / block_tok + a.seq.batch, units = slots * p.heads;
  if (units > 0x7fffffff / 2) return cudaErrorInvalidConfiguration;
  p.slots = (int)slots;
  p.by_length = units > num_sms && a.seq.batch <= LPT_BATCH;
  CUtensorMap r1, r2, x1, x2;
  const int64_t rows = a.seq.rows;
  const bool ok =
      ROLE == DQ ? map3(&r1, a.q, D, a.nq, rows, a.ld_q, p.ht, p.tok) && map3(&r2, a.dout, D, a.nq, rows, a.ld_dout, p.ht, p.tok) &&
                       map3(&x1, a.k, D, a.nkv, rows, a.ld_k, 1, KB) && map3(&x2, a.v, D, a.nkv, rows, a.ld_v, 1, KB)
                 : map3(&r1, a.k, D, a.nkv, rows, a.ld_k, 1, 128) && map3(&r2, a.v, D, a.nkv, rows, a.ld_v, 1, 128) &&
                       map3(&x1, a.q, D, a.nq, rows, a.ld_q, p.sht, p.stok) &&
                       map3(&x2, a.dout, D, a.nq, rows, a.ld_dout, p.sht, p.stok);
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<var_bwd_kernel<D, ROLE>>(C::SMEM);
  if (e != cudaSuccess) return e;
  var_bwd_kernel<D, ROLE><<<(unsigned)units, 384, C::SMEM, st>>>(r1, r2, x1, x2, p);
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
  p.schunks = (p.hpg + KB - 1) / KB;
  p.sht = (p.hpg + p.schunks - 1) / p.schunks;
  p.stok = KB / p.sht;
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
