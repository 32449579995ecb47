// diff_bwd_tc.cu -- gradients of the differential softmax anchor's products, bf16,
// d = 128, on tcgen05/TMEM. With P_m recomputed from the saved log-sum-exp, dA
// and the row sums delta_m (diff_aux.cu):
//     W = P_1 - lambda P_2,  dS_1 = P_1 (dP - delta_1),  dS_2 = -lambda P_2 (dP - delta_2)
//     dV = W^T dA,  dK_m = scale dS_m^T Q_m,  dQ_m = scale dS_m K_m
// Two passes of one shape, so that every output has one owner and its sum one
// order (no atomics): 128 rows X, Y stand, blocks of 64 rows X', Y' stream by.
//     keys stand:    X, Y = K, V   X', Y' = Q, dA   S^T = K Q^T, dP^T = V dA^T;
//                    out dK = dS^T Q, dV = W^T dA
//     queries stand: X, Y = Q, dA  X', Y' = K, V    S = Q K^T, dP = dA V^T; out dQ = dS K
// Either recomputes the scores: 7/5 of the products of one pass over the pairs,
// against adding dQ into memory in an order that changes from run to run.
//
// 20 warps in five warpgroups: warp 0 TMA, warp 1 TMEM and the scores' MMAs, warp 3
// the products' MMAs, the others the weights: thread r of each of four warpgroups
// owns standing row r (its TMEM lane) and 16 of the block's 64 columns. The weights'
// loop is turned by half a step: round i makes dS of block i - 1 and P (and W) of
// block i from dP_{i-1} and S_i, so that it waits for no MMA that needs what the same
// round makes:
//     warp 1, round i:  S_i, dP_{i-1} in registers  ->  dP_i, S_{i+1}
//     warp 3, round i:  dS_{i-1}, W_i stored        ->  dX += dS_{i-1} X', dV += W_i Y'
// What one warp's MMAs need of the other's goes through the weights' barriers. dS goes
// to TMEM and W to shared memory, in bf16, as A operands (a weight is off by 2^-8 of
// itself at most, at random, as P is in the forward pass: 0.0029 of a gradient, relative
// L2, where its own rounding alone is 0.0017).
//
// dlambda_t = -dA_t . O_2[t] = -sum_s P_2 dP is a sum whose terms cancel, and a lambda shared
// by all tokens adds up tokens that cancel again, while the errors that O_2 brings from the
// forward pass's bf16 weights (0.0015 of a token's terms, at random) do not: of 302 training
// steps with any number of heads seven were off by more than 0.005, one by 0.024. The
// queries' side has P_2 and dP in fp32, so it adds what O_2 missed: with delta_2 = r . O_2,
// r the rounded dA,
//     sum_s P_2 dP = delta_2 + sum_s P_2 (dP - delta_2)
// where the last sum would be zero for an exact O_2, and an error of sum_s P_2 times it
// cancels. It is one addition per pair and map 2, on dS_2 before its rounding, and takes 35
// us of a training step of 8,190 tokens and 16 heads (3.40 -> 3.44 ms).
//
// 8,190 tokens of 16 heads: 2.4 to 2.5 ms for both sides, 550 to 570 TFLOP/s of
// the 10 d operations a pair that the gradients need; the steps there: MMAs behind elect.sync in uniform code
// 3.2 -> 2.8 ms, two warps of weights a scheduler -> four without a spilled register
// (16 columns a thread, dP's registers free before S's are read) 2.86 -> 2.26 ms. A
// spill is dear here: next to this shared memory L1 keeps a few KB.
// What bounds it: keys standing, the reads of shared memory. K and V are left operands
// there (dK and dV take half of TMEM), 6 KB an MMA of 48 cycles, and the statistics that
// each thread reads by column stand in line behind them: without those reads the pass
// would take 0.35 ms less, without the exponentials as much less. Queries standing: the
// weights' instructions (0.93 ms of it). Sending exponentials to the FMA pipe costs here.
// Few long tiles are cut along their stream over the CTAs of a cluster, which add up in
// the order of the cuts: 64 queries against 4,000 keys, 8 heads, 89 -> 60 us call after call.
#include <algorithm>

#include "diff_common.cuh"

namespace sva {
namespace {

constexpr int HD = 128;
constexpr int BR = 128, BS = 64;
constexpr int BOXR = 64 * BR * 2;  // [64 columns x 128 rows] bf16
constexpr int BOXS = 64 * BS * 2;  // [64 columns x 64 rows]
constexpr int STAGES = 4;
constexpr int STAGE_BYTES = 4 * BOXS;  // X', Y'
constexpr int STAT_BYTES = kStats * 64 * 4;
constexpr int WGS = 4;          // warpgroups that make weights, 16 of the block's columns each
constexpr int kWarps = 4 * WGS;  // each arrives once for its 32 rows
constexpr int NUM_THREADS = 128 * (1 + WGS);
constexpr int TMEM_COLS = 512;
// register split: 128 threads at 64 + 512 threads at 104 = 640 threads at 96
constexpr int kRegsProducer = 64, kRegsWeights = 104;
constexpr int COLS = BS / WGS;
// TMEM columns
constexpr int TM_S = 0;      // S_1, S_2: 64 each
constexpr int TM_DP = 128;   // dP
constexpr int TM_DS = 192;   // dS_1, dS_2 (bf16): 16 columns of each per warpgroup
constexpr int TM_ACC = 256;  // keys stand: dK, dV; queries stand: dQ
constexpr int TM_X = 384;    // queries stand: Q and dA as A operands, 64 each
constexpr int W_BYTES = BR * BS * 2;

struct Tail {
  uint64_t x_full;
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t s_full, dp_full;  // scores in TMEM
  uint64_t loaded;           // ... and in registers
  uint64_t ds_full;          // dS and W stored
  uint64_t ds_empty;         // ... and used
  uint64_t acc_done;
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
};
template <bool KV>
struct Layout {
  static constexpr int X_OFF = 0;  // keys stand: K, V, two boxes each
  static constexpr int RING = KV ? 4 * BOXR : 0;
  static constexpr int STAT = RING + STAGES * STAGE_BYTES;
  static constexpr int W_OFF = (STAT + (KV ? STAGES * STAT_BYTES : 0) + 1023) / 1024 * 1024;
  static constexpr int TAIL = W_OFF + (KV ? W_BYTES : 0);
  static constexpr size_t SMEM = 1024 + TAIL + sizeof(Tail);
  static_assert(SMEM <= kMaxSmem, "shared memory of one CTA");
};

// a whole warp's wait
__device__ __forceinline__ bool mma_wait(uint64_t* bar, int parity, volatile int* abort_flag,
                                         int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, WHERE_DIFF_BWD));
}

struct Maps {  // boxes of 128 standing rows of K and V; of 64 streamed rows of each
  CUtensorMap k_stand, v_stand, k, v, q, da;
};

template <bool KV>
__device__ __forceinline__ void bwd_tile(const Maps& maps, const sva_diff_args& a,
                                         const sva_diff_grads& g, const DiffBwdScratch& ws,
                                         const DiffBwdTile& u, float scale, int* status,
                                         uint8_t* smem_raw) {
  const CUtensorMap &map_x = maps.k_stand, &map_y = maps.v_stand;  // Q and dA stand in TMEM, loaded by threads
  const CUtensorMap &map_x2 = KV ? maps.q : maps.k, &map_y2 = KV ? maps.da : maps.v;
  using L = Layout<KV>;
  constexpr int NC = KV ? 2 * HD : HD;  // columns of the results
  constexpr int SUMS_AT = BR * (NC + 4);  // behind a share of the results: WGS sums a row
  static_assert((SUMS_AT + (KV ? 0 : WGS * BR)) * 4 <= L::TAIL - L::RING, "a share fits the ring's place");
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail* tl = reinterpret_cast<Tail*>(smem + L::TAIL);
  const int bh = u.bh, h = bh % a.H, b = bh / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int r0 = u.tile * BR;
  const int n_stat_tiles = (a.N + 63) / 64;
  // this CTA's blocks of the streamed side: [j0, j0 + n)
  const int n_all = KV ? (r0 < valid ? n_stat_tiles : 0) : (valid + BS - 1) / BS;
  const int j0 = u.cut * n_all / u.cuts, n = (u.cut + 1) * n_all / u.cuts - j0;
  const float scale_log2 = scale * kLog2e;
  const int warp = warp_uniform(warp_id()), lane = lane_id();
  const int wg = warp >> 2;

  if (threadIdx.x == 0) {
    mbar_init(&tl->x_full, KV ? 1 : kWarps);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tl->full[s], 1);
      mbar_init(&tl->empty[s], 1);
    }
    mbar_init(&tl->s_full, 1);
    mbar_init(&tl->dp_full, 1);
    mbar_init(&tl->loaded, kWarps);
    mbar_init(&tl->ds_full, kWarps);
    mbar_init(&tl->ds_empty, 1);
    mbar_init(&tl->acc_done, 1);
    mbar_init(&tl->drain[0], 1);
    mbar_init(&tl->drain[1], 1);
    tl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tl->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(tl->tmem_base);
  volatile int* abort_flag = &tl->abort_flag;

  if (wg == 0) {
    warpgroup_reg_dec<kRegsProducer>();
    if (warp == 0) {
      // ------------------------------------------------ TMA producer
      if (KV && n > 0 && lane == 0) {
        mbar_arrive_expect_tx(&tl->x_full, 4 * BOXR);
        tma_load_3d(&map_x, &tl->x_full, smem + L::X_OFF, h * HD, r0, b);
        tma_load_3d(&map_x, &tl->x_full, smem + L::X_OFF + BOXR, h * HD + 64, r0, b);
        tma_load_3d(&map_y, &tl->x_full, smem + L::X_OFF + 2 * BOXR, h * HD, r0, b);
        tma_load_3d(&map_y, &tl->x_full, smem + L::X_OFF + 3 * BOXR, h * HD + 64, r0, b);
      }
      __syncwarp();
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        const int st = j % STAGES;
        const bool w = mbar_wait(&tl->empty[st], ((j / STAGES) & 1) ^ 1, abort_flag, status,
                                 WHERE_DIFF_BWD);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* p = smem + L::RING + st * STAGE_BYTES;
          mbar_arrive_expect_tx(&tl->full[st], STAGE_BYTES + (KV ? STAT_BYTES : 0));
          tma_load_3d(&map_x2, &tl->full[st], p, h * HD, (j0 + j) * BS, b);
          tma_load_3d(&map_x2, &tl->full[st], p + BOXS, h * HD + 64, (j0 + j) * BS, b);
          tma_load_3d(&map_y2, &tl->full[st], p + 2 * BOXS, h * HD, (j0 + j) * BS, b);
          tma_load_3d(&map_y2, &tl->full[st], p + 3 * BOXS, h * HD + 64, (j0 + j) * BS, b);
          if (KV)
            bulk_load(smem + L::STAT + st * STAT_BYTES, ws.stats + stat_at(bh, n_stat_tiles, (j0 + j) * BS),
                      STAT_BYTES, &tl->full[st]);
        }
        __syncwarp();
        ++issued;
      }
      if (lane == 0) {
        if (KV && n > 0) (void)drain_wait(&tl->x_full, 0);
        if (!ok)
          for (int i = max(0, issued - STAGES); i < issued; ++i)
            (void)drain_wait(&tl->full[i % STAGES], (i / STAGES) & 1);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------ MMAs: scores
      constexpr uint32_t idesc_s = idesc_bf16_f32(BR, BS, false, false);  // X X'^T
      const uint32_t xd = warp_uniform(desc_lo(smem_u32(smem + L::X_OFF), 16));
      const uint32_t sk = warp_uniform(desc_lo(smem_u32(smem + L::RING), 16));
      // S_1, S_2 of the block in stage st: 64 of the 128 columns each
      auto issue_s = [&](int st) {
        const uint32_t bb = sk + static_cast<uint32_t>(st * (STAGE_BYTES >> 4));
        unrolled<HD / 16>([&](auto k) {
          constexpr int kk = decltype(k)::value, m = kk >> 2, e = kk & 3;
          const uint32_t d = tmem + TM_S + 64 * m;
          if (KV)
            umma_ss_at<m * BOXR + e * 32, m * BOXS + e * 32>(d, xd, bb, idesc_s, e != 0 ? 1u : 0u);
          else
            umma_ts_at<m * BOXS + e * 32>(d, tmem + TM_X + 8 * kk, bb, idesc_s, e != 0 ? 1u : 0u);
        });
        umma_commit(&tl->s_full);
      };
      auto issue_dp = [&](int st) {
        const uint32_t bb = sk + static_cast<uint32_t>(st * (STAGE_BYTES >> 4));
        unrolled<HD / 16>([&](auto k) {
          constexpr int kk = decltype(k)::value, m = kk >> 2, e = kk & 3;
          if (KV)
            umma_ss_at<(2 + m) * BOXR + e * 32, (2 + m) * BOXS + e * 32>(tmem + TM_DP, xd, bb, idesc_s,
                                                                         kk != 0 ? 1u : 0u);
          else
            umma_ts_at<(2 + m) * BOXS + e * 32>(tmem + TM_DP, tmem + TM_X + 64 + 8 * kk, bb, idesc_s,
                                                kk != 0 ? 1u : 0u);
        });
        umma_commit(&tl->dp_full);
      };
      // queries stand: the last block's rows of K behind the batch's last key
      // become zero, since a weight of zero times what lies there may be NaN
      auto stage_ready = [&](int j, int st) -> bool {
        if (!__all_sync(0xffffffffu, mbar_wait(&tl->full[st], (j / STAGES) & 1, abort_flag, status,
                                               WHERE_DIFF_BWD)))
          return false;
        const int left = valid - (j0 + j) * BS;
        if (!KV && left < BS && valid < Nk) {
          uint8_t* p = smem + L::RING + st * STAGE_BYTES;
          for (int i = left * 8 + lane; i < BS * 8; i += 32) {
            *reinterpret_cast<uint4*>(p + i * 16) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(p + BOXS + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      bool ok = n > 0 && mma_wait(&tl->x_full, 0, abort_flag, status) && stage_ready(0, 0);
      if (ok) {
        tc_fence_after();
        if (elect_one()) {
          issue_s(0);
          issue_dp(0);
        }
        __syncwarp();
      }
      int st = 0;  // stage of block i
      for (int i = 0; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        const int sn = st + 1 == STAGES ? 0 : st + 1;
        ok = (!more || stage_ready(i + 1, sn)) && mma_wait(&tl->loaded, i & 1, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (i >= 1) issue_dp(st);
          if (more) issue_s(sn);
        }
        __syncwarp();
        st = sn;
      }
      if (elect_one()) {
        umma_commit(&tl->drain[0]);
        (void)drain_wait(&tl->drain[0], 0);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------ MMAs: products
      constexpr uint32_t idesc_half = idesc_bf16_f32(BR, HD / 2, false, true);  // dS_m X'_m
      constexpr uint32_t idesc_full = idesc_bf16_f32(BR, HD, false, true);      // W Y'
      const uint32_t sm = warp_uniform(desc_lo(smem_u32(smem + L::RING), BOXS));
      const uint32_t wd = warp_uniform(desc_lo(smem_u32(smem + L::W_OFF), 16));
      bool ok = n > 0;
      int st = 0, sp = STAGES - 1;  // stages of blocks i and i - 1
      for (int i = 0; i <= n && ok; ++i) {
        ok = mma_wait(&tl->ds_full, i & 1, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (i >= 1) {  // dX += dS_{i-1} X', 16 rows of X' (a warpgroup's columns of dS) an MMA
            const uint32_t xb = sm + static_cast<uint32_t>(sp * (STAGE_BYTES >> 4));
            const uint32_t more = i != 1 ? 1u : 0u;
            unrolled<2 * BS / 16>([&](auto k) {
              constexpr int m = decltype(k)::value & 1, kk = decltype(k)::value >> 1;
              umma_ts_at<m * BOXS + kk * 2048>(tmem + TM_ACC + 64 * m, tmem + TM_DS + 16 * kk + 8 * m,
                                               xb, idesc_half, kk != 0 ? 1u : more);
            });
            umma_commit(&tl->empty[sp]);  // the stage's last use
          }
          if (KV && i < n) {  // dV += W_i Y'
            const uint32_t yb = sm + static_cast<uint32_t>(st * (STAGE_BYTES >> 4));
            const uint32_t more = i != 0 ? 1u : 0u;
            unrolled<BS / 16>([&](auto k) {
              constexpr int kk = decltype(k)::value;
              umma_ss_at<kk * 32, 2 * BOXS + kk * 2048>(tmem + TM_ACC + HD, wd, yb, idesc_full,
                                                        kk != 0 ? 1u : more);
            });
          }
          umma_commit(&tl->ds_empty);
        }
        __syncwarp();
        sp = st;
        st = st + 1 == STAGES ? 0 : st + 1;
      }
      if (elect_one()) {
        if (ok) umma_commit(&tl->acc_done);
        umma_commit(&tl->drain[1]);
        (void)drain_wait(&tl->drain[1], 0);
      }
      __syncwarp();
    }
  } else {
    warpgroup_reg_inc<kRegsWeights>();
    // ------------------------------------------------ weights, then the results
    const int part = wg - 1;  // this warpgroup's 16 of the block's 64 columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int row = r0 + r;
    const int n_rows = KV ? Nk : a.N;
    const uint64_t scale2 = f2pack(scale_log2, scale_log2);
    uint64_t nlse1 = 0, nlse2 = 0, nd1 = 0, nd2 = 0, nl = 0;  // queries stand: this row's
    uint64_t off2 = 0;  // and its sum of P_2 (dP - delta_2), with lambda in P_2 or not, see below
    if (!KV && n > 0) {
      // the first two warpgroups bring Q, the others dA, half of the columns each
      const bool in = row < a.N;
      const int64_t at = static_cast<int64_t>(b) * a.N + row;
      const __nv_bfloat16* src = part < 2 ? static_cast<const __nv_bfloat16*>(a.q) + at * a.ldq
                                          : static_cast<const __nv_bfloat16*>(ws.da) + at * a.H * HD;
      const uint4* p = reinterpret_cast<const uint4*>(src + h * HD + (part & 1) * 64);
      uint32_t x[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 w = in ? p[i] : make_uint4(0, 0, 0, 0);
        x[4 * i] = w.x; x[4 * i + 1] = w.y; x[4 * i + 2] = w.z; x[4 * i + 3] = w.w;
      }
      __syncwarp();  // rows behind the last query loaded nothing
      tmem_st32(lane_base + TM_X + 32 * part, x);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&tl->x_full);
      // rows behind the last query: their -infinity makes every weight zero
      const float* st = ws.stats + stat_at(bh, n_stat_tiles, min(row, n_stat_tiles * 64 - 1));
      const float f[5] = {in ? st[0] : -INFINITY, in ? st[64] : -INFINITY, st[128], st[192], st[256]};
      nlse1 = f2pack(f[0], f[0]);
      nlse2 = f2pack(f[1], f[1]);
      nd1 = f2pack(f[2], f[2]);
      nd2 = f2pack(f[3], f[3]);
      nl = f2pack(f[4], f[4]);
    }
    const uint64_t minus_one = f2pack(-1.f, -1.f);
    const bool raw = (a.flags & SVA_FLAG_LAMBDA_VALUE) != 0;  // else the last statistic is -1
    bool ok = true;
    // P_1 and, keys standing, -lambda P_2 of a block; queries standing the last factor comes
    // later: P_2, with a sigmoid's lambda in its exponent
    uint64_t p1[COLS / 2], q2[COLS / 2];
    const float* stat0 = reinterpret_cast<const float*>(smem + L::STAT) + COLS * part;
    const float* stat = stat0;  // block i's statistics; prev: block i - 1's
    const float* prev = stat0 + (STAGES - 1) * (STAT_BYTES / 4);
    int st = 0;
    uint32_t phase = 0;  // of full[st]
    for (int i = 0; i <= n && n > 0; ++i) {
      uint32_t d1[COLS / 2], d2[COLS / 2], wk[COLS / 2];
      // dS of the block before first, then this block's scores: fewer values in registers
      bool w = i == 0 || mbar_wait(&tl->dp_full, (i - 1) & 1, abort_flag, status, WHERE_DIFF_BWD);
      if (!__all_sync(0xffffffffu, w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (i > 0) {
        uint32_t dp[COLS];
        tmem_ld16(lane_base + TM_DP + COLS * part, dp);
        tmem_wait_ld();
        // queries stand: keys of block i - 1 that count, of this warpgroup's
        const int left = KV ? COLS : valid - (j0 + i - 1) * BS - COLS * part;
        auto make_ds = [&](auto all) {
          ulonglong2 g1, g2;  // two pairs of queries' statistics at a time
#pragma unroll
          for (int k = 0; k < COLS / 2; ++k) {
            if (KV) {
              if (k % 2 == 0) {
                g1 = *reinterpret_cast<const ulonglong2*>(prev + 128 + 2 * k);
                g2 = *reinterpret_cast<const ulonglong2*>(prev + 192 + 2 * k);
              }
              nd1 = k % 2 == 0 ? g1.x : g1.y;
              nd2 = k % 2 == 0 ? g2.x : g2.y;
            }
            float x0, x1, y0, y1;
            const uint64_t dpp = f2pack(__uint_as_float(dp[2 * k]), __uint_as_float(dp[2 * k + 1]));
            const uint64_t ds1 = mul_f2(p1[k], add_f2(dpp, nd1));
            uint64_t ds2 = mul_f2(q2[k], add_f2(dpp, nd2));
            if (!decltype(all)::value) {
              f2unpack(ds2, y0, y1);
              ds2 = f2pack(2 * k < left ? y0 : 0.f, 2 * k + 1 < left ? y1 : 0.f);
            }
            if (!KV) {
              off2 = add_f2(off2, ds2);
              ds2 = mul_f2(ds2, nl);
            }
            f2unpack(ds1, x0, x1);
            f2unpack(ds2, y0, y1);
            d1[k] = pack_bf16x2(x0, x1);
            d2[k] = pack_bf16x2(y0, y1);
            if (!decltype(all)::value)
              d1[k] &= (2 * k < left ? 0xFFFFu : 0u) | (2 * k + 1 < left ? 0xFFFF0000u : 0u);
          }
        };
        if (left < COLS)
          make_ds(Int<0>());
        else
          make_ds(Int<1>());
      }
      if (i < n) {
        // the stage's statistics landed before the scores were made of its rows, but
        // this thread has to see that copy itself
        w = !KV || mbar_wait(&tl->full[st], phase, abort_flag, status, WHERE_DIFF_BWD);
        w = w && mbar_wait(&tl->s_full, i & 1, abort_flag, status, WHERE_DIFF_BWD);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s1[COLS], s2[COLS];
        tmem_ld16(lane_base + TM_S + COLS * part, s1);
        tmem_ld16(lane_base + TM_S + 64 + COLS * part, s2);
        tmem_wait_ld();
        tc_fence_before();
        warp_arrive(&tl->loaded);
        ulonglong2 f1, f2, f3 = {minus_one, minus_one};
#pragma unroll
        for (int k = 0; k < COLS / 2; ++k) {
          if (KV) {
            if (k % 2 == 0) {
              f1 = *reinterpret_cast<const ulonglong2*>(stat + 2 * k);
              f2 = *reinterpret_cast<const ulonglong2*>(stat + 64 + 2 * k);
              if (raw) f3 = *reinterpret_cast<const ulonglong2*>(stat + 256 + 2 * k);
            }
            nlse1 = k % 2 == 0 ? f1.x : f1.y;
            nlse2 = k % 2 == 0 ? f2.x : f2.y;
            nl = k % 2 == 0 ? f3.x : f3.y;
          }
          float x0, x1, y0, y1;
          f2unpack(fma_f2(f2pack(__uint_as_float(s1[2 * k]), __uint_as_float(s1[2 * k + 1])), scale2,
                          nlse1), x0, x1);
          f2unpack(fma_f2(f2pack(__uint_as_float(s2[2 * k]), __uint_as_float(s2[2 * k + 1])), scale2,
                          nlse2), y0, y1);
          p1[k] = f2pack(ex2_mufu(x0), ex2_mufu(x1));
          q2[k] = f2pack(ex2_mufu(y0), ex2_mufu(y1));
          if (KV) {
            q2[k] = mul_f2(q2[k], nl);
            f2unpack(add_f2(p1[k], q2[k]), x0, x1);
            wk[k] = pack_bf16x2(x0, x1);
          }
        }
      }
      // the products of the round before have used dS and W
      w = i == 0 || mbar_wait(&tl->ds_empty, (i - 1) & 1, abort_flag, status, WHERE_DIFF_BWD);
      if (!__all_sync(0xffffffffu, w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (i > 0) {
        tmem_st8(lane_base + TM_DS + COLS * part, d1);
        tmem_st8(lane_base + TM_DS + COLS * part + COLS / 2, d2);
      }
      if (KV && i < n) {
        // row r of W, 128-byte swizzle: chunk c of the row at c ^ (r & 7)
        uint8_t* wrow = smem + L::W_OFF + r * 128;
#pragma unroll
        for (int c = 0; c < COLS / 8; ++c)
          *reinterpret_cast<uint4*>(wrow + (((COLS / 8 * part + c) ^ (r & 7)) << 4)) =
              make_uint4(wk[4 * c], wk[4 * c + 1], wk[4 * c + 2], wk[4 * c + 3]);
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&tl->ds_full);
      prev = stat;
      st = st + 1 == STAGES ? 0 : st + 1;
      phase ^= st == 0 ? 1u : 0u;
      stat = stat0 + st * (STAT_BYTES / 4);
    }
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&tl->acc_done, 0, abort_flag, status, WHERE_DIFF_BWD));
    tc_fence_after();
    if (!KV) {  // off2 of this warpgroup's columns, behind the place of dQ's shares
      float x0, x1;
      f2unpack(off2, x0, x1);
      reinterpret_cast<float*>(smem + L::RING)[SUMS_AT + part * BR + r] = x0 + x1;
    }
    // keys stand: half of dK or dV a warpgroup; queries stand: a quarter of dQ
    const int64_t at = static_cast<int64_t>(b) * n_rows + row;
    __nv_bfloat16* dst;
    constexpr int ncols = KV ? 64 : 32;
    if (KV)
      dst = (part < 2 ? static_cast<__nv_bfloat16*>(g.dk) + at * g.lddk
                      : static_cast<__nv_bfloat16*>(g.dv) + at * g.lddv) + (part & 1) * 64;
    else
      dst = static_cast<__nv_bfloat16*>(g.dq) + at * g.lddq + 32 * part;
    dst += h * HD;
    const int col0 = TM_ACC + ncols * part;
    const float f = KV && part >= 2 ? 1.0f : scale;
    const bool zero = n == 0 || (KV && row >= valid);
#pragma unroll 1
    for (int c = 0; c < ncols && ok; c += 32) {
      uint32_t o[32];
      if (n > 0) {
        tmem_ld32(lane_base + col0 + c, o);
        tmem_wait_ld();
      }
      if (u.cuts > 1) {  // a share of the sum: in fp32 to shared memory, the ring's place
        float* os = reinterpret_cast<float*>(smem + L::RING) + r * (NC + 4) + ncols * part + c;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(os + 4 * k) =
              zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : make_float4(f * __uint_as_float(o[4 * k]), f * __uint_as_float(o[4 * k + 1]),
                                 f * __uint_as_float(o[4 * k + 2]), f * __uint_as_float(o[4 * k + 3]));
      } else if (row < n_rows) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (!zero) {
            v.x = pack_bf16x2(f * __uint_as_float(o[8 * k]), f * __uint_as_float(o[8 * k + 1]));
            v.y = pack_bf16x2(f * __uint_as_float(o[8 * k + 2]), f * __uint_as_float(o[8 * k + 3]));
            v.z = pack_bf16x2(f * __uint_as_float(o[8 * k + 4]), f * __uint_as_float(o[8 * k + 5]));
            v.w = pack_bf16x2(f * __uint_as_float(o[8 * k + 6]), f * __uint_as_float(o[8 * k + 7]));
          }
          *reinterpret_cast<uint4*>(dst + c + 8 * k) = v;
        }
      }
      __syncwarp();  // the next round's tcgen05.ld wants the whole warp at once
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  // queries stand: dlambda of row `row`, its sums added up in the order of cuts and warpgroups
  auto finish_dlam = [&](const float* sums, int row) {
    float off = 0.f;
    for (int p = 0; p < u.cuts; ++p)
      for (int w = 0; w < WGS; ++w)
        off += u.cuts > 1 ? ld_cluster(sums + w * BR, static_cast<uint32_t>(p)) : sums[w * BR];
    float* dl = ws.dlam + static_cast<int64_t>(bh) * a.N + row;
    const float x = *dl - off;
    if (a.ldl == 0)
      *dl = x;
    else
      from_f32(static_cast<__nv_bfloat16*>(g.dlam) + (static_cast<int64_t>(b) * a.N + row) * g.lddl + h,
               x * dlambda_factor<__nv_bfloat16>(a, b, row, h));
  };
  const float* sums = reinterpret_cast<const float*>(smem + L::RING) + SUMS_AT + threadIdx.x;
  const bool sums_row = !KV && threadIdx.x < BR && r0 + static_cast<int>(threadIdx.x) < a.N;
  if (u.cuts == 1 && sums_row) finish_dlam(sums, r0 + static_cast<int>(threadIdx.x));
  if (u.cuts > 1) {
    // the cuts of a tile are a cluster; the first adds up the shares, in their order
    cluster_sync();
    if (u.cut == 0) {
      const int n_rows = KV ? Nk : a.N;
      const float* os = reinterpret_cast<const float*>(smem + L::RING);
      for (int i = threadIdx.x; i < BR * NC / 4; i += NUM_THREADS) {
        const int r = i / (NC / 4), c = (i % (NC / 4)) * 4, row = r0 + r;
        if (row >= n_rows) break;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < u.cuts; ++p) {
          const float4 y = ld_cluster4(os + r * (NC + 4) + c, static_cast<uint32_t>(p));
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        const int64_t at = static_cast<int64_t>(b) * n_rows + row;
        __nv_bfloat16* dst = !KV      ? static_cast<__nv_bfloat16*>(g.dq) + at * g.lddq
                             : c < HD ? static_cast<__nv_bfloat16*>(g.dk) + at * g.lddk
                                      : static_cast<__nv_bfloat16*>(g.dv) + at * g.lddv;
        store4(dst + h * HD + c % HD, x);
      }
      if (sums_row) finish_dlam(sums, r0 + static_cast<int>(threadIdx.x));
    }
    cluster_sync();  // nobody leaves while its shared memory is read
  }
}

// Both sides in one launch, the second filling the first's last wave.
__global__ void __launch_bounds__(NUM_THREADS, 1)
    diff_bwd_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ sva_diff_args a,
                       const __grid_constant__ sva_diff_grads g, DiffBwdScratch ws, DiffBwdGrid grid,
                       float scale, int* status) {
  extern __shared__ uint8_t smem_raw[];
  DiffBwdTile u;
  if (!diff_bwd_tile(grid, a.B * a.H, static_cast<int>(blockIdx.x), u)) return;
  if (u.keys_stand)
    bwd_tile<true>(maps, a, g, ws, u, scale, status, smem_raw);
  else
    bwd_tile<false>(maps, a, g, ws, u, scale, status, smem_raw);
}

}  // namespace

cudaError_t diff_bwd_bf16(const sva_diff_args& a, const sva_diff_grads& g, int* status,
                          void* scratch, cudaStream_t s) {
  const DiffBwdScratch ws = diff_bwd_scratch(a, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(HD / 2));
  const int D = a.H * a.d;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  Maps m;
  if (!diff_map(&m.k_stand, a.k, a.ldk, a.B, Nk, D, BR) ||
      !diff_map(&m.v_stand, a.v, a.ldv, a.B, Nk, D, BR) || !diff_map(&m.k, a.k, a.ldk, a.B, Nk, D, BS) ||
      !diff_map(&m.v, a.v, a.ldv, a.B, Nk, D, BS) || !diff_map(&m.q, a.q, a.ldq, a.B, a.N, D, BS) ||
      !diff_map(&m.da, ws.da, D, a.B, a.N, D, BS))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_max_smem<diff_bwd_tc_kernel>();
  if (e != cudaSuccess) return e;
  const DiffBwdGrid grid = diff_bwd_grid(a, BR, BS, 1);
  constexpr size_t smem = Layout<true>::SMEM > Layout<false>::SMEM ? Layout<true>::SMEM : Layout<false>::SMEM;
  return launch_clusters(diff_bwd_tc_kernel, grid.ctas(a.B * a.H), NUM_THREADS, smem, grid.cuts, s, m, a, g, ws,
                         grid, scale, status);
}

}  // namespace sva
