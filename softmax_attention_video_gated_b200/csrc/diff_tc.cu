// diff_tc.cu -- the gated differential softmax anchor, forward, bf16, d = 128, on
// tcgen05/TMEM: out = (P_1 V - lambda P_2 V) * sigmoid(G), the two maps' queries
// and keys being the halves of a head's columns.
//
// One CTA per 128-query tile of one (head, batch); 12 warps in three warpgroups:
//   WG0  warp 0: TMA for the Q tile, the 128-key K tiles, then the gate tile
//        into Q's buffer; warp 2: TMA for V; warp 3: residency of V_j and
//        K_{j+1}, and zeros in the rows of V behind a batch's last key (a weight
//        of zero times what lies there may be NaN); warp 1: TMEM and the MMAs.
//   WG1, WG2  softmax of map 1 and map 2: thread r owns query row r.
// TMEM: S_m at 256 m, O_m at 256 m + 128. S_m = Q_m K_m^T is one swizzle box of
// Q and K (64 of their 128 columns), P_m (bf16, unnormalised) goes over S_m's
// first 64 columns and is the A operand of O_m += P_m V, V being read by both.
// The MMA thread works on one map while the other's softmax runs. Running maximum
// in the log2 domain, moved only when it grows by more than 8 (p <= 2^8
// otherwise); l sums the unrounded p in fp32. Rounding p to bf16 for the product
// is off by half a step, 2^-8 of the weight, at most and at random: the result is off by
// 0.0026 (relative L2) where its own rounding alone is 0.0017. P in more bits would double
// its product.
// Where the maps nearly cancel that is 0.002 of each map's output, not of the difference.
// What bounds it: the chain of one map, S -> softmax -> P -> P V, whose S has one buffer
// that P lies over; tensor pipe and MUFU are both busy half of the time. 8,190 tokens of
// 16 heads (1,024 CTAs) take 870 to 890 us call after call, 940 TFLOP/s, 0.57 of the
// measured bf16 peak (850 alone, behind a pause). The softmax is the longer half of the
// chain: on a box and clock where it took 823 us, it took 595 without exponentials and 651
// with half of them, so a quarter runs on the FMA pipe (823 -> 772 there). Tried and slower
// than those 772: two warpgroups a map with half of the keys each (862), P reported in
// halves (795), the maximum begun on half of S (879).
// At the end both warpgroups read both maps' O (a TMEM lane quarter belongs to a
// warp's place in its warpgroup, so the two share it), half of the columns each,
// and combine them with lambda, the sums and the gate.
#include <algorithm>

#include "diff_common.cuh"

namespace sva {
namespace {

constexpr int HD = 128;
constexpr int BQ = kDiffTcRows, BKV = kDiffTcKeys;
constexpr int BOX = 128 * 128;  // [64 columns x 128 rows] bf16
constexpr int K_STAGES = 3, V_STAGES = 3;
constexpr int Q_OFF = 0;
constexpr int K_OFF = 2 * BOX;
constexpr int V_OFF = K_OFF + K_STAGES * 2 * BOX;
constexpr int TAIL_OFF = V_OFF + V_STAGES * 2 * BOX;
constexpr int NUM_THREADS = 384;
constexpr int TMEM_COLS = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// register split: 128 threads at 56 + 256 threads at 224 = 384 threads at 168
constexpr int kRegsProducer = 56, kRegsSoftmax = 224;

struct Tail {
  uint64_t q_full;
  uint64_t k_full[K_STAGES];
  uint64_t k_empty[K_STAGES];
  uint64_t v_full[V_STAGES];
  uint64_t v_empty[V_STAGES];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_done;
  uint64_t g_full;  // the gate tile, loaded into Q's buffer once Q is no longer read
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kSmem = 1024 + TAIL_OFF + sizeof(Tail);
static_assert(kSmem <= kMaxSmem, "shared memory of one CTA");

// A row's sum holds 2^8 a key at most. One beyond 2^100 has the number in it that the FMA pipe's
// exponential made of a NaN. Asked for where the sum is about to shrink and at the end: 8190
// tokens, 16 heads 871 -> 874 us; in every block 886.
__device__ __forceinline__ float keep_nan(float l) { return l < 0x1p100f ? l : NAN; }

__global__ void __launch_bounds__(NUM_THREADS, 1)
    diff_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_g,
                   const __grid_constant__ sva_diff_args a, float scale_log2, DiffWork wk,
                   int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Tail* tl = reinterpret_cast<Tail*>(smem + TAIL_OFF);
  const DiffUnit u = diff_unit(wk, static_cast<int>(blockIdx.x));
  const int q0 = u.q0, h = u.h, b = u.b;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  int kb0 = 0, nkv = (valid + BKV - 1) / BKV;
  if (u.part >= 0) {
    kb0 = u.part * nkv / wk.split;
    nkv = (u.part + 1) * nkv / wk.split - kb0;
  }
  const int warp = warp_uniform(warp_id()), lane = lane_id();
  const int wg = warp >> 2;

  if (threadIdx.x == 0) {
    mbar_init(&tl->q_full, 1);
    for (int s = 0; s < K_STAGES; ++s) {
      mbar_init(&tl->k_full[s], 1);
      mbar_init(&tl->k_empty[s], 1);
    }
    for (int s = 0; s < V_STAGES; ++s) {
      mbar_init(&tl->v_full[s], 1);
      mbar_init(&tl->v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tl->s_full[i], 1);
      mbar_init(&tl->p_full[i], 5);  // four warps, and warp 3: V_j, K_{j+1} resident
    }
    mbar_init(&tl->o_done, 1);
    mbar_init(&tl->g_full, 1);
    mbar_init(&tl->drain, 1);
    tl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tl->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(tl->tmem_base);
  volatile int* abort_flag = &tl->abort_flag;

  if (wg == 0) {
    warpgroup_reg_dec<kRegsProducer>();
    if (warp == 0) {
      // ------------------------------------------------ TMA producer: Q, K, the gate
      if (lane == 0) {
        mbar_arrive_expect_tx(&tl->q_full, 2 * BOX);
        tma_load_3d(&map_q, &tl->q_full, smem + Q_OFF, h * HD, q0, b);
        tma_load_3d(&map_q, &tl->q_full, smem + Q_OFF + BOX, h * HD + 64, q0, b);
      }
      __syncwarp();
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % K_STAGES;
        const bool w = mbar_wait(&tl->k_empty[st], ((j / K_STAGES) & 1) ^ 1, abort_flag, status,
                                 WHERE_DIFF);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* kt = smem + K_OFF + st * 2 * BOX;
          mbar_arrive_expect_tx(&tl->k_full[st], 2 * BOX);
          tma_load_3d(&map_k, &tl->k_full[st], kt, h * HD, (kb0 + j) * BKV, b);
          tma_load_3d(&map_k, &tl->k_full[st], kt + BOX, h * HD + 64, (kb0 + j) * BKV, b);
        }
        __syncwarp();
        ++issued;
      }
      const bool gated = a.gate != nullptr && u.part < 0 && nkv > 0;
      if (ok && gated) {
        // the commit that frees the last K stage covers the last reads of Q
        const bool w = mbar_wait(&tl->k_empty[(nkv - 1) % K_STAGES], ((nkv - 1) / K_STAGES) & 1,
                                 abort_flag, status, WHERE_DIFF);
        ok = __all_sync(0xffffffffu, w);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&tl->g_full, 2 * BOX);
          tma_load_3d(&map_g, &tl->g_full, smem + Q_OFF, h * HD, q0, b);
          tma_load_3d(&map_g, &tl->g_full, smem + Q_OFF + BOX, h * HD + 64, q0, b);
        }
        __syncwarp();
      }
      if (lane == 0) {
        (void)drain_wait(&tl->q_full, 0);
        if (ok && gated) (void)drain_wait(&tl->g_full, 0);
        if (!ok)
          for (int i = max(0, issued - K_STAGES); i < issued; ++i)
            (void)drain_wait(&tl->k_full[i % K_STAGES], (i / K_STAGES) & 1);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------ TMA producer: V
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % V_STAGES;
        const bool w = mbar_wait(&tl->v_empty[st], ((j / V_STAGES) & 1) ^ 1, abort_flag, status,
                                 WHERE_DIFF);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* vt = smem + V_OFF + st * 2 * BOX;
          mbar_arrive_expect_tx(&tl->v_full[st], 2 * BOX);
          tma_load_3d(&map_v, &tl->v_full[st], vt, h * HD, (kb0 + j) * BKV, b);
          tma_load_3d(&map_v, &tl->v_full[st], vt + BOX, h * HD + 64, (kb0 + j) * BKV, b);
        }
        __syncwarp();
        ++issued;
      }
      if (lane == 0 && !ok)
        for (int i = max(0, issued - V_STAGES); i < issued; ++i)
          (void)drain_wait(&tl->v_full[i % V_STAGES], (i / V_STAGES) & 1);
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------ residency of V_j and K_{j+1}
      // one arrival per map and block; it waits for that phase to complete
      // before the next block, so it never arrives twice in one phase
      for (int j = 0; j < nkv; ++j) {
        bool w = mbar_wait(&tl->v_full[j % V_STAGES], (j / V_STAGES) & 1, abort_flag, status,
                           WHERE_DIFF);
        if (j + 1 < nkv)
          w = w && mbar_wait(&tl->k_full[(j + 1) % K_STAGES], ((j + 1) / K_STAGES) & 1, abort_flag,
                             status, WHERE_DIFF);
        if (!__all_sync(0xffffffffu, w)) break;
        const int left = valid - (kb0 + j) * BKV;
        if (left < BKV && valid < Nk) {
          // rows behind the batch's last key (behind Nk the copy filled zeros);
          // a row's 128 bytes of a box stay together under the swizzle
          uint8_t* vt = smem + V_OFF + (j % V_STAGES) * 2 * BOX;
          for (int i = left * 8 + lane; i < BKV * 8; i += 32) {
            *reinterpret_cast<uint4*>(vt + i * 16) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(vt + BOX + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(&tl->p_full[0]);
          mbar_arrive(&tl->p_full[1]);
        }
        __syncwarp();
        bool wp = mbar_wait(&tl->p_full[0], j & 1, abort_flag, status, WHERE_DIFF);
        wp = wp && mbar_wait(&tl->p_full[1], j & 1, abort_flag, status, WHERE_DIFF);
        if (!__all_sync(0xffffffffu, wp)) break;
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(BQ, BKV, false, false);  // Q, K: K-major
      constexpr uint32_t idesc_o = idesc_bf16_f32(BQ, HD, false, true);    // P (TMEM), V: MN-major
      bool ok = __all_sync(0xffffffffu, mbar_wait(&tl->q_full, 0, abort_flag, status, WHERE_DIFF));
      const uint64_t qd0 = smem_desc(smem_u32(smem + Q_OFF), 16, 1024);
      const uint64_t kd0 = smem_desc(smem_u32(smem + K_OFF), 16, 1024);
      const uint64_t vd0 = smem_desc(smem_u32(smem + V_OFF), BOX, 1024);
      auto issue_s = [&](int m, int kst) {
        const uint64_t qb = qd0 + static_cast<uint64_t>(m * (BOX >> 4));
        const uint64_t kb = kd0 + static_cast<uint64_t>((kst * 2 + m) * (BOX >> 4));
#pragma unroll
        for (int kk = 0; kk < HD / 2 / 16; ++kk)
          umma_ss(tmem + m * 256, qb + (kk * 32 >> 4), kb + (kk * 32 >> 4), idesc_s,
                  kk != 0 ? 1u : 0u);
        umma_commit(&tl->s_full[m]);
      };
      auto issue_pv = [&](int m, int vst, bool first) {
        const uint64_t vb = vd0 + static_cast<uint64_t>(vst * (2 * BOX >> 4));
        const uint32_t p_tmem = tmem + m * 256;
#pragma unroll
        for (int kk = 0; kk < BKV / 16; ++kk)
          umma_ts(p_tmem + 128, p_tmem + kk * 8, vb + static_cast<uint32_t>(kk * 2048 >> 4), idesc_o,
                  (kk != 0 || !first) ? 1u : 0u);
      };
      if (ok && nkv > 0) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&tl->k_full[0], 0, abort_flag, status, WHERE_DIFF));
        if (ok) {
          tc_fence_after();
          if (elect_one()) {
            issue_s(0, 0);
            issue_s(1, 0);
            umma_commit(&tl->k_empty[0]);
          }
          __syncwarp();
        }
      }
      int vst = 0, kn = 1 % K_STAGES;  // stages of V_j and K_{j+1}
      for (int j = 0; j < nkv && ok; ++j) {
        const bool more = j + 1 < nkv;
        for (int m = 0; m < 2; ++m) {
          const bool w = mbar_wait(&tl->p_full[m], j & 1, abort_flag, status, WHERE_DIFF);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            issue_pv(m, vst, j == 0);
            if (m == 1) umma_commit(&tl->v_empty[vst]);
            if (more) {
              issue_s(m, kn);
              if (m == 1) umma_commit(&tl->k_empty[kn]);
            }
          }
          __syncwarp();
        }
        vst = vst + 1 == V_STAGES ? 0 : vst + 1;
        kn = kn + 1 == K_STAGES ? 0 : kn + 1;
      }
      if (elect_one()) {
        if (ok) umma_commit(&tl->o_done);
        umma_commit(&tl->drain);
        (void)drain_wait(&tl->drain, 0);
      }
      __syncwarp();
    }
  } else {
    warpgroup_reg_inc<kRegsSoftmax>();
    // ------------------------------------------------ softmax (WG1: map 1, WG2: map 2)
    const int mp = wg - 1;
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t s_col = tmem + lane_base + mp * 256;
    const uint32_t o_col = s_col + 128;
    float m = -INFINITY;  // running (possibly stale) maximum of the scaled logits, log2 units
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      const bool w = mbar_wait(&tl->s_full[mp], j & 1, abort_flag, status, WHERE_DIFF);
      if (!__all_sync(0xffffffffu, w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t v[4][32];
      tmem_ld32(s_col, v[0]);
      tmem_ld32(s_col + 32, v[1]);
      tmem_ld32(s_col + 64, v[2]);
      tmem_ld32(s_col + 96, v[3]);
      tmem_wait_ld();
      float s[BKV];
#pragma unroll
      for (int i = 0; i < BKV; ++i) s[i] = __uint_as_float(v[i >> 5][i & 31]);
      const int left = valid - (kb0 + j) * BKV;  // keys of this block that count
      if (left < BKV) {
#pragma unroll
        for (int i = 0; i < BKV; ++i)
          if (i >= left) s[i] = -INFINITY;
      }
      // row maximum: eight chains of three-input max over the 128 keys
      float mx8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mx8[k] = max3_f(s[k], s[k + 8], s[k + 16]);
#pragma unroll
      for (int base = 24; base + 16 <= BKV - 8; base += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = max3_f(mx8[k], s[base + k], s[base + 8 + k]);
#pragma unroll
      for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], s[BKV - 8 + k]);
      const float mx = fmaxf(max3_f(max3_f(mx8[0], mx8[1], mx8[2]),
                                    max3_f(mx8[3], mx8[4], mx8[5]), mx8[6]),
                             mx8[7]) *
                       scale_log2;
      const bool grow = mx > m + kRescaleThreshold;
      float factor = 1.f;
      if (grow) {
        factor = (m == -INFINITY) ? 0.f : ex2_mufu(m - mx);
        m = mx;
      }
      // O of this map is complete up to block j-1 here: the commit that reported
      // S_j also covers P_{j-1} V_{j-1}
      if (j > 0 && __any_sync(0xffffffffu, grow)) {
        l = keep_nan(l);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
          tmem_st32(o_col + c, o);
        }
      }
      l *= factor;
      // x = s * scale - m and the row sum on packed pairs
      const uint64_t scale2 = f2pack(scale_log2, scale_log2), negm2 = f2pack(-m, -m);
      uint64_t acc2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc2[i] = f2pack(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float x0, x1;
          f2unpack(fma_f2(f2pack(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), scale2, negm2), x0, x1);
          float p0, p1;
          // a quarter on the FMA pipe: 8190 tokens, 16 heads 823 -> 772 us (an eighth: 804,
          // half: 793)
          if (i % 4 == 3) {
            ex2_poly2(x0, x1, p0, p1);
          } else {
            p0 = ex2_mufu(x0);
            p1 = ex2_mufu(x1);
          }
          acc2[i & 3] = add_f2(acc2[i & 3], f2pack(p0, p1));
          pk[i] = pack_bf16x2(p0, p1);
        }
        tmem_st16(s_col + 16 * c, pk);
      }
      tmem_wait_st();
      {
        float u0, u1;
        f2unpack(add_f2(add_f2(acc2[0], acc2[1]), add_f2(acc2[2], acc2[3])), u0, u1);
        l += u0 + u1;
      }
      tc_fence_before();
      warp_arrive(&tl->p_full[mp]);
    }
    l = keep_nan(l);
    if (ok && nkv > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&tl->o_done, 0, abort_flag, status, WHERE_DIFF));
    tc_fence_after();
    const int t = q0 + r;
    if (ok && u.part >= 0) {
      float* po = diff_part(wk, HD, u.su, u.part, mp);
      if (nkv > 0) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_wait_ld();
          if (t < a.N) {
            float4* dst = reinterpret_cast<float4*>(po + r * HD + c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
          __syncwarp();  // the next tcgen05.ld wants the whole warp at once
        }
      }
      *reinterpret_cast<float2*>(po + BQ * HD + 2 * r) = make_float2(m, l);
    } else if (u.part < 0) {
      // every softmax thread comes here, an aborted one too: the barrier counts them all
      // sums for the other warpgroup, in the first K stage (no longer read: o_done
      // covers every MMA)
      float* sums = reinterpret_cast<float*>(smem + K_OFF);
      sums[mp * BQ + r] = l;
      named_barrier_sync(1, 256);
      const float l1 = sums[r], l2 = sums[BQ + r];
      const float i1 = inverse_sum(l1), i2 = inverse_sum(l2);
      const bool gated = a.gate != nullptr && nkv > 0;
      if (ok && gated)
        ok = __all_sync(0xffffffffu, mbar_wait(&tl->g_full, 0, abort_flag, status, WHERE_DIFF));
      const bool row_ok = t < a.N;
      const int64_t row = static_cast<int64_t>(b) * a.N + t;
      const float lam = row_ok ? lambda_of<__nv_bfloat16>(a, b, t, h) : 0.f;
      if (row_ok && ok) finish_lse(a, mp, b, h, t, m, l);
      __syncwarp();  // the next tcgen05.ld wants the whole warp at once
#pragma unroll 1
      for (int c = mp * 64; c < mp * 64 + 64 && ok; c += 32) {
        uint32_t o1[32], o2[32];
        if (nkv > 0) {
          tmem_ld32(tmem + lane_base + 128 + c, o1);
          tmem_ld32(tmem + lane_base + 384 + c, o2);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o1[i] = o2[i] = 0u;
        }
        if (a.o1 != nullptr) {
          // The saved rows leave 128 bytes each, through the K stages: a row a lane would
          // write 16 bytes of 32 rows at a time (one row a lane: 8190 tokens, 16 heads, 100 us
          // more than without them; now 11 us).
          float* box = reinterpret_cast<float*>(smem + K_OFF + 4096) + (mp * 4 + q) * 2 * 32 * 36;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            *reinterpret_cast<float4*>(box + lane * 36 + 4 * k) = make_float4(
                __uint_as_float(o1[4 * k]) * i1, __uint_as_float(o1[4 * k + 1]) * i1,
                __uint_as_float(o1[4 * k + 2]) * i1, __uint_as_float(o1[4 * k + 3]) * i1);
            *reinterpret_cast<float4*>(box + (32 + lane) * 36 + 4 * k) = make_float4(
                __uint_as_float(o2[4 * k]) * i2, __uint_as_float(o2[4 * k + 1]) * i2,
                __uint_as_float(o2[4 * k + 2]) * i2, __uint_as_float(o2[4 * k + 3]) * i2);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + (lane >> 3), tt = q0 + q * 32 + rr;
            if (tt < a.N) {
              const int64_t at = (static_cast<int64_t>(b) * a.N + tt) * a.H * HD + h * HD + c + 4 * (lane & 7);
              store4(a.o1 + at, *reinterpret_cast<const float4*>(box + rr * 36 + 4 * (lane & 7)));
              store4(a.o2 + at, *reinterpret_cast<const float4*>(box + (32 + rr) * 36 + 4 * (lane & 7)));
            }
          }
          __syncwarp();
        }
        if (row_ok) {
          const uint8_t* grow = smem + Q_OFF + (c >> 6) * BOX + r * 128;
          __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + row * a.ldo + h * HD + c;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] = __uint_as_float(o1[8 * k + e]) * i1;
              y[e] = __uint_as_float(o2[8 * k + e]) * i2;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(-lam, y[e], x[e]);
            if (gated) {
              // row r of the gate tile, 128-byte swizzle: chunk i of the row at i ^ (r & 7)
              const int chunk = ((c & 63) >> 3) + k;
              const uint4 gv = *reinterpret_cast<const uint4*>(grow + ((chunk ^ (r & 7)) << 4));
              const float gg[8] = {bf16lo_to_f32(gv.x), bf16hi_to_f32(gv.x), bf16lo_to_f32(gv.y),
                                   bf16hi_to_f32(gv.y), bf16lo_to_f32(gv.z), bf16hi_to_f32(gv.z),
                                   bf16lo_to_f32(gv.w), bf16hi_to_f32(gv.w)};
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] *= __fdividef(1.0f, 1.0f + __expf(-gg[e]));
            }
            uint4 ov;
            ov.x = pack_bf16x2(y[0], y[1]);
            ov.y = pack_bf16x2(y[2], y[3]);
            ov.z = pack_bf16x2(y[4], y[5]);
            ov.w = pack_bf16x2(y[6], y[7]);
            *reinterpret_cast<uint4*>(op + 8 * k) = ov;
          }
        }
        __syncwarp();  // as above
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

cudaError_t diff_fwd_bf16(const sva_diff_args& a, int* status, void* scratch, cudaStream_t s) {
  const int D = a.H * a.d;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  CUtensorMap mq, mk, mv, mg;
  if (!diff_map(&mq, a.q, a.ldq, a.B, a.N, D, 128) || !diff_map(&mk, a.k, a.ldk, a.B, Nk, D, 128) ||
      !diff_map(&mv, a.v, a.ldv, a.B, Nk, D, 128))
    return cudaErrorInvalidValue;
  mg = mq;
  if (a.gate != nullptr && !diff_map(&mg, a.gate, a.ldg, a.B, a.N, D, 128))
    return cudaErrorInvalidValue;
  const DiffPlan p = diff_plan(a.B, a.N, a.H, a.d, a.n_keys, a.dtype);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(HD / 2));
  cudaError_t e = allow_max_smem<diff_tc_kernel>();
  if (e != cudaSuccess) return e;
  diff_tc_kernel<<<p.grid(), NUM_THREADS, kSmem, s>>>(mq, mk, mv, mg, a, scale * kLog2e,
                                                      diff_work(p, a.H, scratch), status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return diff_merge(a, p, scratch, s);
}

}  // namespace sva
