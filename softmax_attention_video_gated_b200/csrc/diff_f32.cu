// diff_f32.cu -- the differential softmax anchor in fp32, forward and backward.
//
// Products on the tensor cores with both operands split in two tf32 parts, a = a_hi
// + a_lo (11 + 11 bits), a b = a_hi b_hi + (a_hi b_lo + a_lo b_hi) + O(2^-22 a b):
// three MMAs of 16 x 8 x 8, 170 fp32 multiply-adds a cycle and SM where the CUDA
// cores have 128, and a sixteenth of their instructions (the CUDA-core form of
// these kernels reached 30% of that rate, bound by operand loads and few warps).
// The tensor core cuts its sums off (towards minus infinity) instead of rounding
// them, half a step of bias per MMA, so a chain is kept short: the large and the
// small products are summed apart, over 64 to 128 channels or 16 rows, and added
// to the running fp32 sums by the CUDA cores.
//
// Forward: 64 query rows a CTA, 16 a warp; keys 16 at a time, both maps' scores,
// one online softmax each, and O_m += P_m V with V's fragments read once for both.
// Backward: the query-stationary and the key-stationary products are the same
// computation with the two sides exchanged, S^T = K Q^T, dP^T = V dA^T, so one
// kernel does both; each output has one owner and no atomics are needed. Both maps
// share dP, and dV needs one product of the combined weights W = P_1 - lambda P_2.
// Scores leave the MMA in the layout that the next one takes as its left operand,
// up to an exchange of the summed index that the right operand follows: P, W and
// dS stay in registers.
// 777 tokens, two batches, 4 heads of 128: forward 115 us and 22 for the merge of its
// five parts, backward 276 us, 35 TFLOP/s in fp32; the tensor pipe is busy 39 to 42% of
// the time, behind the operands' splitting and two warps a scheduler. Parts that fit the
// machine at once join in a cluster instead: 1,024 tokens, 4 heads of 64, 51 us in all
// (2 us more with a merge; past one resident wave the clusters' waits made it slower).
// Few long tiles of the backward pass are cut along their stream over a cluster: 64
// queries against 4,000 keys, 8 heads of 128, 435 -> 198 us.
#include <algorithm>

#include "diff_common.cuh"

namespace sva {
namespace {

// x = hi + lo, each with 11 significant bits: hi is x rounded, lo what that left, cut
// off behind a factor of 1 + 2^-11.5 that stands for the mean half step (rounding its
// bits as hi's would turn a NaN into a zero; as it is the NaN stays in lo)
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  lo = __float_as_uint((x - __uint_as_float(hi)) * 1.00034527f) & 0xFFFFE000u;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
struct FragA {
  uint32_t hi[4], lo[4];
};
struct FragB {
  uint32_t hi[2], lo[2];
};
// sums of one tile: the large products, the small ones
struct Sum {
  float big[4], small[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) big[i] = small[i] = 0.f;
  }
  __device__ __forceinline__ float at(int i) const { return big[i] + small[i]; }
};

// x += a b and y += c d, their MMAs in turn: one that adds to the same sum follows
// three others, about its latency
__device__ __forceinline__ void add2(Sum& x, const FragA& a, const FragB& b, Sum& y, const FragA& c,
                                     const FragB& d) {
  mma(x.small, a.lo, b.hi);
  mma(y.small, c.lo, d.hi);
  mma(x.big, a.hi, b.hi);
  mma(y.big, c.hi, d.hi);
  mma(x.small, a.hi, b.lo);
  mma(y.small, c.hi, d.lo);
}

// A lane's place in a 16 x 8 tile: rows g and g + 8; as a result the columns 2 t and
// 2 t + 1, as a left operand the summed indexes t and t + 4.
struct Lane {
  int g, t;
  __device__ __forceinline__ Lane() : g(lane_id() >> 2), t(lane_id() & 3) {}
};

// left operand of rows [r, r + 16), columns [k, k + 8) from split rows of stride L
template <int L>
__device__ __forceinline__ void frag_a(FragA& f, const uint32_t* hi, const uint32_t* lo, int r, int k,
                                       Lane ln) {
  const int at = (r + ln.g) * L + k + ln.t;
  f.hi[0] = hi[at]; f.hi[1] = hi[at + 8 * L]; f.hi[2] = hi[at + 4]; f.hi[3] = hi[at + 8 * L + 4];
  f.lo[0] = lo[at]; f.lo[1] = lo[at + 8 * L]; f.lo[2] = lo[at + 4]; f.lo[3] = lo[at + 8 * L + 4];
}
// right operand: rows n..n+7 of x as columns, summed over their columns [k, k + 8)
template <int L>
__device__ __forceinline__ void frag_dot(FragB& f, const float* x, int n, int k, Lane ln) {
  const float* p = x + (n + ln.g) * L + k + ln.t;
  split(p[0], f.hi[0], f.lo[0]);
  split(p[4], f.hi[1], f.lo[1]);
}
// right operand: columns [n, n + 8) of x, summed over its rows k..k+7 in the order
// that frag_mix's left operand takes them
template <int L>
__device__ __forceinline__ void frag_rows(FragB& f, const float* x, int k, int n, Lane ln) {
  const float* p = x + (k + 2 * ln.t) * L + n + ln.g;
  split(p[0], f.hi[0], f.lo[0]);
  split(p[L], f.hi[1], f.lo[1]);
}
// a tile of weights (result layout) as the left operand of a sum over its columns:
// the columns 2 t and 2 t + 1 take the places t and t + 4
__device__ __forceinline__ void frag_mix(FragA& f, const float (&c)[4]) {
  split(c[0], f.hi[0], f.lo[0]);
  split(c[2], f.hi[1], f.lo[1]);
  split(c[1], f.hi[2], f.lo[2]);
  split(c[3], f.hi[3], f.lo[3]);
}

// Rows [r0, r0 + R) of a [B, n, ld] activation's head columns to shared memory (row
// stride D + 4), in the background; rows at or behind `valid` are zero.
template <int R, int D>
__device__ __forceinline__ void load_rows(float* dst, const void* src, int64_t ld, int64_t b, int n,
                                          int col, int r0, int valid) {
#pragma unroll 4
  for (int i = threadIdx.x; i < R * D / 4; i += blockDim.x) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const bool in = r0 + r < valid;
    copy16_upto(dst + r * (D + 4) + c,
                static_cast<const float*>(src) + (b * n + (in ? r0 + r : 0)) * ld + col + c, in ? 16 : 0);
  }
}
// the same, split
template <int R, int D>
__device__ __forceinline__ void load_split(uint32_t* hi, uint32_t* lo, const void* src, int64_t ld,
                                           int64_t b, int n, int col, int r0, int valid) {
#pragma unroll 2
  for (int i = threadIdx.x; i < R * D / 4; i += blockDim.x) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < valid) v = load4(static_cast<const float*>(src) + (b * n + r0 + r) * ld + col + c);
    uint4 h, l;
    split(v.x, h.x, l.x);
    split(v.y, h.y, l.y);
    split(v.z, h.z, l.z);
    split(v.w, h.w, l.w);
    *reinterpret_cast<uint4*>(hi + r * (D + 4) + c) = h;
    *reinterpret_cast<uint4*>(lo + r * (D + 4) + c) = l;
  }
}

// a row's four lanes
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// s[n] = rows [r, r + 16) of the split x, columns [k0, k0 + K), times rows c + 8 n of y
template <int K, int L>
__device__ __forceinline__ void scores(float (&s)[2][4], const uint32_t* hi, const uint32_t* lo,
                                       const float* y, int r, int c, int k0, Lane ln) {
  Sum acc[2];
  acc[0].clear();
  acc[1].clear();
#pragma unroll 4
  for (int k = 0; k < K; k += 8) {
    FragA a;
    FragB b[2];
    frag_a<L>(a, hi, lo, r, k0 + k, ln);
    frag_dot<L>(b[0], y, c, k0 + k, ln);
    frag_dot<L>(b[1], y, c + 8, k0 + k, ln);
    add2(acc[0], a, b[0], acc[1], a, b[1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = acc[n].at(i);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int FR = kDiffF32Rows;  // 4 warps
static_assert(4 * FR + 2 * FR * 9 <= 4 * 16 * (64 + 4), "sums and weights fit the tiles' place");

template <int D>
constexpr size_t fwd_smem() {
  return static_cast<size_t>(2 * FR + 4 * diff_f32_keys(D)) * (D + 4) * sizeof(float);
}

// The join of key parts as a call, for heads of 128: inlined, its registers make the key
// loop spill 76 bytes (2 x 777 tokens, 4 heads: 136 us inlined, 132 as a call; 4,096 tokens,
// where nothing joins: 1,204 and 1,196). Heads of 64 inline it: 55 us so, 57 as a call
// (1,024 tokens, 4 heads).
template <int D, int L>
__device__ __noinline__ void cluster_join(const sva_diff_args& a, const DiffUnit& u, int split,
                                          const float* os, const float* mls, float* w) {
  cluster_finish<float, FR, D, L>(a, u, split, os, mls, w);
}

template <int D>
__global__ void __launch_bounds__(128, 2)
    diff_fwd_kernel(const __grid_constant__ sva_diff_args a, float scale_log2, DiffWork wk) {
  constexpr int M = D / 2, L = D + 4, NT = D / 8, FK = diff_f32_keys(D);
  extern __shared__ __align__(16) float sm[];
  uint32_t* qhi = reinterpret_cast<uint32_t*>(sm);
  uint32_t* qlo = qhi + FR * L;
  float* ring = sm + 2 * FR * L;  // two stages of K and V
  const Lane ln;
  const int r = warp_id() * 16;
  const DiffUnit u = diff_unit(wk, static_cast<int>(blockIdx.x));
  const int h = u.h, b = u.b;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int nkb = (valid + FK - 1) / FK;
  const int kb0 = u.part < 0 ? 0 : static_cast<int>(static_cast<int64_t>(u.part) * nkb / wk.split);
  const int kb1 = u.part < 0 ? nkb : static_cast<int>((u.part + 1LL) * nkb / wk.split);
  load_split<FR, D>(qhi, qlo, a.q, a.ldq, b, a.N, h * D, u.q0, a.N);
  float o[2][NT][4];
  float m[2][2], l[2][2];  // [map][row g, g + 8]
#pragma unroll
  for (int mp = 0; mp < 2; ++mp) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[mp][n][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) { m[mp][i] = -INFINITY; l[mp][i] = 0.f; }
  }
  auto fetch = [&](int kb) {
    if (kb >= kb1) return;
    float* st = ring + (kb & 1) * 2 * FK * L;
    load_rows<FK, D>(st, a.k, a.ldk, b, Nk, h * D, kb * FK, valid);
    load_rows<FK, D>(st + FK * L, a.v, a.ldv, b, Nk, h * D, kb * FK, valid);
  };
  fetch(kb0);
  for (int kb = kb0; kb < kb1; ++kb) {
    copy_wait_all();
    __syncthreads();  // the block is here, and nobody reads the other stage any more
    fetch(kb + 1);
    const float* ks = ring + (kb & 1) * 2 * FK * L;
    const float* vs = ks + FK * L;
#pragma unroll 1
    for (int c = 0; c < FK; c += 16) {
      const int left = valid - kb * FK - c;  // keys of these 16 that count
      if (left <= 0) break;
      FragA p[2][2];  // [map][8 keys]
#pragma unroll
      for (int mp = 0; mp < 2; ++mp) {
        float s[2][4];
        scores<M, L>(s, qhi, qlo, ks, r, c, mp * M, ln);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[n][i] = n * 8 + 2 * ln.t + (i & 1) < left ? s[n][i] * scale_log2 : -INFINITY;
            top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
          }
        bool grew = false;
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // one of the keys counts at least, so the new maximum is finite
          const float mx = fmaxf(m[mp][i], row_max(top[i]));
          f[i] = exp2f(m[mp][i] - mx);
          grew = grew || mx != m[mp][i];
          m[mp][i] = mx;
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[n][i] = exp2f(s[n][i] - m[mp][i >> 1]);
            sum[i >> 1] += s[n][i];
          }
          frag_mix(p[mp][n], s[n]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) l[mp][i] = fmaf(l[mp][i], f[i], row_sum(sum[i]));
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mp][n][i] *= f[i >> 1];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        FragB v[2];
        frag_rows<L>(v[0], vs, c, n * 8, ln);
        frag_rows<L>(v[1], vs, c + 8, n * 8, ln);
        Sum acc[2];
        acc[0].clear();
        acc[1].clear();
        add2(acc[0], p[0][0], v[0], acc[1], p[1][0], v[0]);
        add2(acc[0], p[0][1], v[1], acc[1], p[1][1], v[1]);
#pragma unroll
        for (int mp = 0; mp < 2; ++mp)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mp][n][i] += acc[mp].at(i);
      }
    }
  }
  // rows g and g + 8, columns 8 n + 2 t and + 1; a whole unit's end takes four
  // columns a thread, so the outputs go through shared memory
  __syncthreads();
  float* os = sm;  // [2 maps][FR][L]: Q's place and more
#pragma unroll
  for (int mp = 0; mp < 2; ++mp)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(os + (mp * FR + r + ln.g + 8 * i) * L + 8 * n + 2 * ln.t) =
            make_float2(o[mp][n][2 * i], o[mp][n][2 * i + 1]);
  float* mls = sm + 2 * FR * L;  // [2 maps][FR][2]
  if (ln.t == 0)
#pragma unroll
    for (int mp = 0; mp < 2; ++mp)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(mls + 2 * (mp * FR + r + ln.g + 8 * i)) =
            make_float2(m[mp][i], l[mp][i]);
  if (wk.cluster) {
    if constexpr (D == 128)
      cluster_join<D, L>(a, u, wk.split, os, mls, mls + 4 * FR);
    else
      cluster_finish<float, FR, D, L>(a, u, wk.split, os, mls, mls + 4 * FR);
    return;
  }
  __syncwarp();  // a warp's rows are its own
  const int lane = lane_id();
  for (int i = lane; i < 16 * D / 4; i += 32) {
    const int rr = r + i / (D / 4), c = (i % (D / 4)) * 4, t = u.q0 + rr;
    if (t >= a.N) break;
    const float4 x = *reinterpret_cast<const float4*>(os + rr * L + c);
    const float4 y = *reinterpret_cast<const float4*>(os + (FR + rr) * L + c);
    const float2 ml1 = *reinterpret_cast<const float2*>(mls + 2 * rr);
    const float2 ml2 = *reinterpret_cast<const float2*>(mls + 2 * (FR + rr));
    if (u.part >= 0) {
      float* p1 = diff_part(wk, D, u.su, u.part, 0);
      float* p2 = diff_part(wk, D, u.su, u.part, 1);
      *reinterpret_cast<float4*>(p1 + rr * D + c) = x;
      *reinterpret_cast<float4*>(p2 + rr * D + c) = y;
      if (c == 0) {
        *reinterpret_cast<float2*>(p1 + FR * D + 2 * rr) = ml1;
        *reinterpret_cast<float2*>(p2 + FR * D + 2 * rr) = ml2;
      }
    } else {
      finish4<float>(a, b, h, t, c, x, y, ml1.y, ml2.y, lambda_of<float>(a, b, t, h));
      if (c < 8) finish_lse(a, c / 4, b, h, t, c == 0 ? ml1.x : ml2.x, c == 0 ? ml1.y : ml2.y);
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// standing and streamed rows of a tile. 8 warps: 16 standing rows by a quarter of the
// streamed ones each; the quarters' sums join at the end. Two stages of streamed rows.
constexpr int BR = 32, BS = 64;

template <int D>
constexpr size_t bwd_smem() {
  return (static_cast<size_t>(4 * BR + 4 * BS) * (D + 4) + 2 * kStats * 64) * sizeof(float);
}

// acc[n] += w (16 rows x 16 streamed ones) times columns n0 + 8 n of x's rows c..c+15
template <int NT, int L>
__device__ __forceinline__ void mix(float (&acc)[NT][4], const FragA (&w)[2], const float* x, int c,
                                    int n0, Lane ln) {
#pragma unroll
  for (int n = 0; n < NT; n += 2) {
    Sum s[2];
    s[0].clear();
    s[1].clear();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      FragB v[2];
      frag_rows<L>(v[0], x, c + 8 * k, n0 + n * 8, ln);
      frag_rows<L>(v[1], x, c + 8 * k, n0 + n * 8 + 8, ln);
      add2(s[0], w[k], v[0], s[1], w[k], v[1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n + j][i] += s[j].at(i);
  }
}

// KV = false: query rows stand (X = Q, Y = dA), keys stream (X' = K, Y' = V), out dQ.
// KV = true: key rows stand (X = K, Y = V), queries stream (X' = Q, Y' = dA), out dK, dV.
template <int D, bool KV>
__device__ __forceinline__ void bwd_tile(const sva_diff_args& a, const sva_diff_grads& g,
                                         const DiffBwdScratch& ws, float scale, const DiffBwdTile& u,
                                         float* sm) {
  constexpr int M = D / 2, L = D + 4, NT = D / 8;
  uint32_t* xhi = reinterpret_cast<uint32_t*>(sm);
  uint32_t* xlo = xhi + BR * L;
  uint32_t* yhi = xlo + BR * L;
  uint32_t* ylo = yhi + BR * L;
  float* ring = sm + 4 * BR * L;                    // two stages of X', Y'
  float* stats = ring + 4 * BS * L;                 // and, KV, of the queries' statistics [5][64]
  const Lane ln;
  const int r = (warp_id() & 1) * 16, quarter = warp_id() >> 1;
  const int bh = u.bh, h = bh % a.H, b = bh / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int r0 = u.tile * BR;
  const float scale_log2 = scale * kLog2e;
  const int64_t D_all = static_cast<int64_t>(a.H) * D;
  const int n_stat_tiles = (a.N + 63) / 64;
  float rs[2][kStats] = {};  // queries stand: statistics of rows g, g + 8
  if (KV) {
    load_split<BR, D>(xhi, xlo, a.k, a.ldk, b, Nk, h * D, r0, valid);
    load_split<BR, D>(yhi, ylo, a.v, a.ldv, b, Nk, h * D, r0, valid);
  } else {
    load_split<BR, D>(xhi, xlo, a.q, a.ldq, b, a.N, h * D, r0, a.N);
    load_split<BR, D>(yhi, ylo, ws.da, D_all, b, a.N, h * D, r0, a.N);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < kStats; ++k)
        rs[i][k] = ws.stats[stat_at(bh, n_stat_tiles, r0 + r + ln.g + 8 * i) + 64 * k];
  }
  // this CTA's rows of the streamed side: [first, stream)
  const int all = KV ? (r0 < valid ? a.N : 0) : valid, blocks = (all + BS - 1) / BS;
  const int first = u.cut * blocks / u.cuts * BS;
  const int stream = min(all, (u.cut + 1) * blocks / u.cuts * BS);
  float acc[NT][4];             // dQ or dK
  float accv[KV ? NT : 1][4];   // dV
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[n][i] = 0.f;
      if (KV) accv[KV ? n : 0][i] = 0.f;
    }
  auto fetch = [&](int s0) {
    if (s0 >= stream) return;
    const int st = (s0 / BS) & 1;
    float* x2 = ring + st * 2 * BS * L;
    float* y2 = x2 + BS * L;
    if (KV) {
      load_rows<BS, D>(x2, a.q, a.ldq, b, a.N, h * D, s0, a.N);
      load_rows<BS, D>(y2, ws.da, D_all, b, a.N, h * D, s0, a.N);
      for (int i = threadIdx.x * 4; i < kStats * 64; i += blockDim.x * 4)
        copy16(stats + st * kStats * 64 + i, ws.stats + stat_at(bh, n_stat_tiles, s0) + i);
      __syncwarp();  // some lanes of a warp copied; its MMAs want all
    } else {
      load_rows<BS, D>(x2, a.k, a.ldk, b, Nk, h * D, s0, valid);
      load_rows<BS, D>(y2, a.v, a.ldv, b, Nk, h * D, s0, valid);
    }
  };
  fetch(first);
  for (int s0 = first; s0 < stream; s0 += BS) {
    copy_wait_all();
    __syncthreads();  // the block is here, and nobody reads the other stage any more
    fetch(s0 + BS);
    const int st = (s0 / BS) & 1;
    const float* x2 = ring + st * 2 * BS * L;
    const float* y2 = x2 + BS * L;
    const float* stat = stats + st * kStats * 64;
    const int c = quarter * 16;
    if (s0 + c < stream) {
      float p1[2][4], p2[2][4];
      scores<M, L>(p1, xhi, xlo, x2, r, c, 0, ln);
      scores<M, L>(p2, xhi, xlo, x2, r, c, M, ln);
      FragA w[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cc = c + n * 8 + 2 * ln.t + (i & 1);
          const bool ok = (KV ? r0 + r + ln.g + 8 * (i >> 1) : s0 + cc) < valid;
          const float n1 = KV ? stat[cc] : rs[i >> 1][0], n2 = KV ? stat[64 + cc] : rs[i >> 1][1];
          const float nl = KV ? stat[256 + cc] : rs[i >> 1][4];
          p1[n][i] = ok ? exp2f(fmaf(p1[n][i], scale_log2, n1)) : 0.f;
          p2[n][i] = ok ? nl * exp2f(fmaf(p2[n][i], scale_log2, n2)) : 0.f;
          wv[i] = p1[n][i] + p2[n][i];
        }
        if (KV) frag_mix(w[n], wv);
      }
      if constexpr (KV) mix<NT, L>(accv, w, y2, c, 0, ln);
      float dp[2][4];
      scores<D, L>(dp, yhi, ylo, y2, r, c, 0, ln);
#pragma unroll
      for (int mp = 0; mp < 2; ++mp) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float ds[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int cc = c + n * 8 + 2 * ln.t + (i & 1);
            const float nd = KV ? stat[(2 + mp) * 64 + cc] : rs[i >> 1][2 + mp];
            ds[i] = (mp == 0 ? p1[n][i] : p2[n][i]) * (dp[n][i] + nd);
          }
          frag_mix(w[n], ds);
        }
        // dS_1 mixes the first map's half of the columns, dS_2 the second's
        mix<NT / 2, L>(reinterpret_cast<float(&)[NT / 2][4]>(acc[mp * NT / 2]), w, x2, c, mp * M, ln);
      }
    }
  }
  // the other quarters' sums to the first, through the tiles' place, in their order
  copy_wait_all();
  __syncthreads();
  constexpr int OUT = KV ? 2 * NT : NT;
  float4* js = reinterpret_cast<float4*>(sm) + (warp_id() & 1) * 32 * OUT + lane_id();
  for (int turn = 1; turn < 4; ++turn) {
    if (quarter == turn) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        js[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        if constexpr (KV)
          js[(NT + n) * 32] = make_float4(accv[n][0], accv[n][1], accv[n][2], accv[n][3]);
      }
    }
    __syncthreads();
    if (quarter == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 j = js[n * 32];
        acc[n][0] += j.x; acc[n][1] += j.y; acc[n][2] += j.z; acc[n][3] += j.w;
        if constexpr (KV) {
          const float4 jv = js[(NT + n) * 32];
          accv[n][0] += jv.x; accv[n][1] += jv.y; accv[n][2] += jv.z; accv[n][3] += jv.w;
        }
      }
    }
    __syncthreads();
  }
  if (u.cuts > 1) {
    // the cuts of a tile are a cluster; the first adds up their sums, in their order
    if (quarter == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        js[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        if constexpr (KV)
          js[(NT + n) * 32] = make_float4(accv[n][0], accv[n][1], accv[n][2], accv[n][3]);
      }
    }
    cluster_sync();
    if (u.cut == 0 && quarter == 0) {
      for (int p = 1; p < u.cuts; ++p) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 j = ld_cluster4(reinterpret_cast<const float*>(js + n * 32), static_cast<uint32_t>(p));
          acc[n][0] += j.x; acc[n][1] += j.y; acc[n][2] += j.z; acc[n][3] += j.w;
          if constexpr (KV) {
            const float4 jv =
                ld_cluster4(reinterpret_cast<const float*>(js + (NT + n) * 32), static_cast<uint32_t>(p));
            accv[n][0] += jv.x; accv[n][1] += jv.y; accv[n][2] += jv.z; accv[n][3] += jv.w;
          }
        }
      }
    }
    cluster_sync();  // nobody leaves while its shared memory is read
    if (u.cut != 0) return;
  }
  if (quarter != 0) return;
  const int n_rows = KV ? Nk : a.N;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = r0 + r + ln.g + 8 * i;
      if (rr >= n_rows) continue;
      const int64_t row = static_cast<int64_t>(b) * n_rows + rr;
      const int col = h * D + 8 * n + 2 * ln.t;
      if constexpr (KV) {
        // rows behind the last key are zero, also where a query's values are no numbers
        const bool in = rr < valid;
        *reinterpret_cast<float2*>(static_cast<float*>(g.dk) + row * g.lddk + col) =
            make_float2(in ? scale * acc[n][2 * i] : 0.f, in ? scale * acc[n][2 * i + 1] : 0.f);
        *reinterpret_cast<float2*>(static_cast<float*>(g.dv) + row * g.lddv + col) =
            make_float2(in ? accv[n][2 * i] : 0.f, in ? accv[n][2 * i + 1] : 0.f);
      } else {
        *reinterpret_cast<float2*>(static_cast<float*>(g.dq) + row * g.lddq + col) =
            make_float2(scale * acc[n][2 * i], scale * acc[n][2 * i + 1]);
      }
    }
  }
}

// Both sides in one launch, the second filling the first's last wave.
template <int D>
__global__ void __launch_bounds__(256)
    diff_bwd_kernel(const __grid_constant__ sva_diff_args a, const __grid_constant__ sva_diff_grads g,
                    DiffBwdScratch ws, float scale, DiffBwdGrid grid) {
  extern __shared__ __align__(16) float sm[];
  DiffBwdTile u;
  if (!diff_bwd_tile(grid, a.B * a.H, static_cast<int>(blockIdx.x), u)) return;
  if (u.keys_stand)
    bwd_tile<D, true>(a, g, ws, scale, u, sm);
  else
    bwd_tile<D, false>(a, g, ws, scale, u, sm);
}

template <int D>
cudaError_t fwd(const sva_diff_args& a, void* scratch, cudaStream_t s) {
  const DiffPlan p = diff_plan(a.B, a.N, a.H, a.d, a.n_keys, a.dtype);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  cudaError_t e = allow_max_smem<diff_fwd_kernel<D>>();
  if (e != cudaSuccess) return e;
  e = launch_clusters(diff_fwd_kernel<D>, p.grid(), 128, fwd_smem<D>(), p.cluster ? p.split : 1, s, a,
                      scale * kLog2e, diff_work(p, a.H, scratch));
  if (e != cudaSuccess) return e;
  return diff_merge(a, p, scratch, s);
}

template <int D>
cudaError_t bwd(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  const DiffBwdScratch ws = diff_bwd_scratch(a, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  constexpr int smem = static_cast<int>(bwd_smem<D>());
  static_assert(smem <= kMaxSmem, "shared memory of one CTA");
  const cudaError_t e = allow_max_smem<diff_bwd_kernel<D>>();
  if (e != cudaSuccess) return e;
  const DiffBwdGrid grid = diff_bwd_grid(a, BR, BS, 1);
  return launch_clusters(diff_bwd_kernel<D>, grid.ctas(a.B * a.H), 256, smem, grid.cuts, s, a, g, ws, scale, grid);
}

}  // namespace

cudaError_t diff_fwd_f32(const sva_diff_args& a, void* scratch, cudaStream_t s) {
  return a.d == 64 ? fwd<64>(a, scratch, s) : fwd<128>(a, scratch, s);
}

cudaError_t diff_bwd_f32(const sva_diff_args& a, const sva_diff_grads& g, void* scratch,
                         cudaStream_t s) {
  return a.d == 64 ? bwd<64>(a, g, scratch, s) : bwd<128>(a, g, scratch, s);
}

}  // namespace sva
