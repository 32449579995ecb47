// diff_f32.cu -- the differential softmax anchor in fp32 on the CUDA cores,
// forward and backward.
//
// Forward per query tile: both maps' scores of a key block, one online softmax
// per map (running maximum and sum in registers), and O_m += P_m V with the
// block's V read once for both. Backward: the query-stationary and the
// key-stationary products are the same computation with the two sides
// exchanged, S^T = K Q^T, dP^T = V dA^T, so one kernel does both; each output
// has one owner and no atomics are needed. Both maps share dP, and dV needs one
// product of the combined weights W = P_1 - lambda P_2.
#include <algorithm>
#include <math.h>

#include "diff_common.cuh"

namespace sva {
namespace {

// Rows [r0, r0 + R) of a [B, n, ld] activation's head columns to shared memory
// (fp32, row stride D + 4); rows at or behind `valid` are zero.
template <int R, int D>
__device__ __forceinline__ void load_rows(float* dst, const void* src, int64_t ld, int64_t b, int n,
                                          int col, int r0, int valid) {
  for (int i = threadIdx.x; i < R * D / 4; i += blockDim.x) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < valid) v = load4(static_cast<const float*>(src) + (b * n + r0 + r) * ld + col + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
  }
}

// acc[i][j] = sum_k a[ty*RI + i][k] b[tx + 16 j][k], k < K (row strides LA, LB).
// The even and the odd k are summed apart, so that a packed fp32 pair takes both.
template <int RI, int RJ, int K, int LA, int LB>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int tx, int ty,
                                         float (&acc)[RI][RJ]) {
  uint64_t p[RI][RJ];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < RJ; ++j) p[i][j] = 0;
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    ulonglong2 av[RI], bv[RJ];
#pragma unroll
    for (int i = 0; i < RI; ++i)
      av[i] = *reinterpret_cast<const ulonglong2*>(a + (ty * RI + i) * LA + k);
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      bv[j] = *reinterpret_cast<const ulonglong2*>(b + (tx + 16 * j) * LB + k);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        p[i][j] = fma_f2(av[i].x, bv[j].x, p[i][j]);
        p[i][j] = fma_f2(av[i].y, bv[j].y, p[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      float lo, hi;
      f2unpack(p[i][j], lo, hi);
      acc[i][j] = lo + hi;
    }
}

// acc[i][2 j + e] += sum_k p[ty*RI + i][k] x[k][64 j + 4 tx + 2 e, + 1], k < K: pairs of columns
template <int RI, int RJ, int K, int LP, int LX>
__device__ __forceinline__ void mix_tile(const float* p, const float* x, int tx, int ty,
                                         uint64_t (&acc)[RI][2 * RJ]) {
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 pv[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) pv[i] = *reinterpret_cast<const float4*>(p + (ty * RI + i) * LP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const ulonglong2 xv = *reinterpret_cast<const ulonglong2*>(x + (k + kk) * LX + 64 * j + 4 * tx);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float w = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
          const uint64_t w2 = f2pack(w, w);
          acc[i][2 * j] = fma_f2(w2, xv.x, acc[i][2 * j]);
          acc[i][2 * j + 1] = fma_f2(w2, xv.y, acc[i][2 * j + 1]);
        }
      }
    }
  }
}
__device__ __forceinline__ float4 quad(uint64_t a, uint64_t b) {
  float4 v;
  f2unpack(a, v.x, v.y);
  f2unpack(b, v.z, v.w);
  return v;
}

__device__ __forceinline__ float row_max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// query rows and keys of a tile: 128 threads, 4 x 4 scores of a map each
constexpr int FR = kDiffF32Rows, FK = kDiffF32Keys;

template <int D>
constexpr size_t fwd_smem() {
  return (static_cast<size_t>(FR + 2 * FK) * (D + 4) + 2 * FR * (FK + 4)) * sizeof(float);
}

template <int D>
__global__ void __launch_bounds__(128) diff_fwd_kernel(const sva_diff_args a, float scale_log2,
                                                       DiffWork wk) {
  constexpr int M = D / 2, L = D + 4, LP = FK + 4, RJ = D / 64;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;
  float* ks = qs + FR * L;
  float* vs = ks + FK * L;
  float* ps = vs + FK * L;  // [2][FR][LP]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const DiffUnit u = diff_unit(wk, static_cast<int>(blockIdx.x));
  const int h = u.h, b = u.b;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int nkb = (valid + FK - 1) / FK;
  const int kb0 = u.part < 0 ? 0 : u.part * nkb / wk.split;
  const int kb1 = u.part < 0 ? nkb : (u.part + 1) * nkb / wk.split;
  const int q0 = u.q0;
  load_rows<FR, D>(qs, a.q, a.ldq, b, a.N, h * D, q0, a.N);
  uint64_t o[2][4][2 * RJ] = {};
  float m[2][4], l[2][4];
#pragma unroll
  for (int mm = 0; mm < 2; ++mm)
#pragma unroll
    for (int i = 0; i < 4; ++i) { m[mm][i] = -INFINITY; l[mm][i] = 0.f; }
  for (int kb = kb0; kb < kb1; ++kb) {
    __syncthreads();
    load_rows<FK, D>(ks, a.k, a.ldk, b, Nk, h * D, kb * FK, valid);
    load_rows<FK, D>(vs, a.v, a.ldv, b, Nk, h * D, kb * FK, valid);
    __syncthreads();
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      float s[4][FK / 16];
      dot_tile<4, FK / 16, M, L, L>(qs + mm * M, ks + mm * M, tx, ty, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < FK / 16; ++j) {
          s[i][j] = kb * FK + tx + 16 * j < valid ? s[i][j] * scale_log2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
        // a block holds one valid key at least, so the new maximum is finite
        const float mx = fmaxf(m[mm][i], row_max16(top));
        const float f = exp2f(m[mm][i] - mx);
        m[mm][i] = mx;
        float* pr = ps + (mm * FR + ty * 4 + i) * LP;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < FK / 16; ++j) {
          const float p = exp2f(s[i][j] - mx);
          pr[tx + 16 * j] = p;
          sum += p;
        }
        l[mm][i] = fmaf(l[mm][i], f, row_sum16(sum));
#pragma unroll
        for (int e = 0; e < 2 * RJ; ++e) o[mm][i][e] = mul_f2(o[mm][i][e], f2pack(f, f));
      }
    }
    // a row of P is written and read by the same half warp
    __syncwarp();
    mix_tile<4, RJ, FK, LP, L>(ps, vs, tx, ty, o[0]);
    mix_tile<4, RJ, FK, LP, L>(ps + FR * LP, vs, tx, ty, o[1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = q0 + ty * 4 + i;
    if (t >= a.N) continue;
    if (u.part >= 0) {
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        float* po = diff_part(wk, D, u.su, u.part, mm);
        const int r = ty * 4 + i;
#pragma unroll
        for (int j = 0; j < RJ; ++j)
          *reinterpret_cast<float4*>(po + r * D + 64 * j + 4 * tx) =
              quad(o[mm][i][2 * j], o[mm][i][2 * j + 1]);
        if (tx == 0)
          *reinterpret_cast<float2*>(po + FR * D + 2 * r) = make_float2(m[mm][i], l[mm][i]);
      }
      continue;
    }
    const float lam = lambda_of<float>(a, b, t, h);
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      finish4<float>(a, b, h, t, 64 * j + 4 * tx,
                 quad(o[0][i][2 * j], o[0][i][2 * j + 1]), quad(o[1][i][2 * j], o[1][i][2 * j + 1]),
                 l[0][i], l[1][i], lam);
    if (tx < 2) finish_lse(a, tx, b, h, t, tx == 0 ? m[0][i] : m[1][i], tx == 0 ? l[0][i] : l[1][i]);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// standing and streamed rows of a tile: 256 threads, 4 x 4 scores of a map each
constexpr int BR = 64, BS = 64;

template <int D>
constexpr size_t bwd_smem() {
  return (static_cast<size_t>(2 * BR + 2 * BS) * (D + 4) + 3 * BR * (BS + 4) + 5 * BR) *
         sizeof(float);
}

// KV = false: query rows stand (X = Q, Y = dA), keys stream (X' = K, Y' = V), out dQ.
// KV = true: key rows stand (X = K, Y = V), queries stream (X' = Q, Y' = dA), out dK, dV.
template <int D, bool KV>
__global__ void __launch_bounds__(256) diff_bwd_kernel(const sva_diff_args a,
                                                       const sva_diff_grads g, DiffBwdScratch ws,
                                                       float scale) {
  constexpr int M = D / 2, L = D + 4, LP = BS + 4, RJ = D / 64;
  constexpr int ST = KV ? BS : BR;  // queries whose statistics a tile needs
  extern __shared__ __align__(16) float sm[];
  float* xs = sm;
  float* ys = xs + BR * L;
  float* x2 = ys + BR * L;
  float* y2 = x2 + BS * L;
  float* wsm = y2 + BS * L;        // [3][BR][LP]: dS_1, dS_2, W
  float* stat = wsm + 3 * BR * LP; // [5][ST]: -lse_m log2 e, -delta_m, -lambda
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int h = blockIdx.y % a.H, b = blockIdx.y / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int r0 = blockIdx.x * BR;
  const float scale_log2 = scale * kLog2e;
  const int64_t D_all = static_cast<int64_t>(a.H) * D;
  auto load_stats = [&](int q0) {
    // q0 is a multiple of 32, so a tile's statistics are one run of a 64-query tile
    for (int i = threadIdx.x; i < kStats * ST; i += blockDim.x) {
      const int k = i / ST, c = i % ST;
      stat[i] = ws.stats[stat_at(static_cast<int>(blockIdx.y), (a.N + 63) / 64, q0 + c) + k * 64];
    }
  };
  if (KV) {
    load_rows<BR, D>(xs, a.k, a.ldk, b, Nk, h * D, r0, valid);
    load_rows<BR, D>(ys, a.v, a.ldv, b, Nk, h * D, r0, valid);
  } else {
    load_rows<BR, D>(xs, a.q, a.ldq, b, a.N, h * D, r0, a.N);
    load_rows<BR, D>(ys, ws.da, D_all, b, a.N, h * D, r0, a.N);
    load_stats(r0);
  }
  const int stream = KV ? (r0 < valid ? a.N : 0) : valid;
  uint64_t acc[4][2 * RJ] = {};            // dQ or dK: columns 64 j + 4 tx + e of the head
  uint64_t accv[KV ? 4 : 1][2 * RJ] = {};  // dV
  for (int s0 = 0; s0 < stream; s0 += BS) {
    __syncthreads();
    if (KV) {
      load_rows<BS, D>(x2, a.q, a.ldq, b, a.N, h * D, s0, a.N);
      load_rows<BS, D>(y2, ws.da, D_all, b, a.N, h * D, s0, a.N);
      load_stats(s0);
    } else {
      load_rows<BS, D>(x2, a.k, a.ldk, b, Nk, h * D, s0, valid);
      load_rows<BS, D>(y2, a.v, a.ldv, b, Nk, h * D, s0, valid);
    }
    __syncthreads();
    float s1[4][BS / 16], s2[4][BS / 16], dp[4][BS / 16];
    dot_tile<4, BS / 16, M, L, L>(xs, x2, tx, ty, s1);
    dot_tile<4, BS / 16, M, L, L>(xs + M, x2 + M, tx, ty, s2);
    dot_tile<4, BS / 16, D, L, L>(ys, y2, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < BS / 16; ++j) {
        const int rr = ty * 4 + i, cc = tx + 16 * j;
        const int qi = KV ? cc : rr;
        const bool ok = (KV ? r0 + rr : s0 + cc) < valid;
        const float p1 = ok ? exp2f(fmaf(s1[i][j], scale_log2, stat[qi])) : 0.f;
        const float p2 =
            ok ? stat[4 * ST + qi] * exp2f(fmaf(s2[i][j], scale_log2, stat[ST + qi])) : 0.f;
        wsm[rr * LP + cc] = p1 * (dp[i][j] + stat[2 * ST + qi]);
        wsm[(BR + rr) * LP + cc] = p2 * (dp[i][j] + stat[3 * ST + qi]);
        if (KV) wsm[(2 * BR + rr) * LP + cc] = p1 + p2;
      }
    __syncwarp();  // a row of W and dS is written and read by the same half warp
    // dS_1 mixes the first map's half of the columns, dS_2 the second's
    if (RJ == 2) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint64_t half[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) half[i][e] = acc[i][2 * (RJ - 1) * m + e];
        mix_tile<4, 1, BS, LP, L>(wsm + m * BR * LP, x2 + m * M, tx, ty, half);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[i][2 * (RJ - 1) * m + e] = half[i][e];
      }
    } else {  // d = 64: columns 4 tx + e; the first eight threads' belong to map 1
      uint64_t one[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) one[i][e] = acc[i][e];
      mix_tile<4, 1, BS, LP, L>(wsm + (tx >= 8 ? BR * LP : 0), x2, tx, ty, one);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[i][e] = one[i][e];
    }
    if constexpr (KV) mix_tile<4, RJ, BS, LP, L>(wsm + 2 * BR * LP, y2, tx, ty, accv);
  }
  const int n_rows = KV ? Nk : a.N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= n_rows) continue;
    const int64_t row = static_cast<int64_t>(b) * n_rows + r;
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      const int col = h * D + 64 * j + 4 * tx;
      const float4 x = quad(acc[i][2 * j], acc[i][2 * j + 1]);
      const float4 v = make_float4(scale * x.x, scale * x.y, scale * x.z, scale * x.w);
      if constexpr (KV) {
        store4(static_cast<float*>(g.dk) + row * g.lddk + col, v);
        store4(static_cast<float*>(g.dv) + row * g.lddv + col,
               quad(accv[i][2 * j], accv[i][2 * j + 1]));
      } else {
        store4(static_cast<float*>(g.dq) + row * g.lddq + col, v);
      }
    }
  }
}

template <int D>
cudaError_t fwd(const sva_diff_args& a, void* scratch, cudaStream_t s) {
  const DiffPlan p = diff_plan(a.B, a.N, a.H, a.d, a.n_keys, a.dtype);
  const DiffWork wk = diff_work(p, a.H, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  cudaError_t e = allow_max_smem<diff_fwd_kernel<D>>();
  if (e != cudaSuccess) return e;
  diff_fwd_kernel<D><<<p.grid(), 128, fwd_smem<D>(), s>>>(a, scale * kLog2e, wk);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return diff_merge(a, p, scratch, s);
}

template <int D>
cudaError_t bwd(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  const DiffBwdScratch ws = diff_bwd_scratch(a, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const unsigned bh = static_cast<unsigned>(a.B * a.H);
  const int smem = static_cast<int>(bwd_smem<D>());
  cudaError_t e;
  if ((e = allow_max_smem<diff_bwd_kernel<D, false>>()) != cudaSuccess ||
      (e = allow_max_smem<diff_bwd_kernel<D, true>>()) != cudaSuccess)
    return e;
  diff_bwd_kernel<D, false><<<dim3(static_cast<unsigned>((a.N + BR - 1) / BR), bh), 256, smem, s>>>(a, g, ws, scale);
  diff_bwd_kernel<D, true><<<dim3(static_cast<unsigned>((Nk + BR - 1) / BR), bh), 256, smem, s>>>(a, g, ws, scale);
  return cudaGetLastError();
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
