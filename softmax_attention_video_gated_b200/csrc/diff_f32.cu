// diff_f32.cu -- the differential softmax anchor on the CUDA cores, forward and
// backward, plus the kernels around the attention core that both types share
// (the merge of a key split, the backward pass's preparation).
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

#include "common.cuh"
#include "internal.h"

namespace sva {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

__device__ __forceinline__ float sigmoid_f(float x) { return 1.0f / (1.0f + expf(-x)); }

__device__ __forceinline__ int key_count(const int32_t* key_lens, int b, int Nk) {
  return key_lens == nullptr ? Nk : max(0, min(Nk, key_lens[b]));
}

// lambda of token t (batch b, head h)
template <typename T>
__device__ __forceinline__ float lambda_of(const sva_diff_args& a, int b, int64_t t, int h) {
  const T* p = static_cast<const T*>(a.lam);
  const float x = to_f32(a.ldl == 0 ? p[h] : p[(static_cast<int64_t>(b) * a.N + t) * a.ldl + h]);
  return (a.flags & SVA_FLAG_LAMBDA_VALUE) ? x : sigmoid_f(x);
}

// Rows [r0, r0 + R) of a [B, n, ld] activation's head columns to shared memory
// (fp32, row stride D + 4); rows at or behind `valid` are zero.
template <typename T, int R, int D>
__device__ __forceinline__ void load_rows(float* dst, const void* src, int64_t ld, int64_t b, int n,
                                          int col, int r0, int valid) {
  for (int i = threadIdx.x; i < R * D / 4; i += blockDim.x) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < valid) v = load4(static_cast<const T*>(src) + (b * n + r0 + r) * ld + col + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
  }
}

// acc[i][j] += sum_k a[ty*RI + i][k0 + k] b[tx + 16 j][k0 + k], k < K (row strides LA, LB)
template <int RI, int RJ, int K, int LA, int LB>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int tx, int ty,
                                         float (&acc)[RI][RJ]) {
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    float4 av[RI], bv[RJ];
#pragma unroll
    for (int i = 0; i < RI; ++i) av[i] = *reinterpret_cast<const float4*>(a + (ty * RI + i) * LA + k);
#pragma unroll
    for (int j = 0; j < RJ; ++j) bv[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LB + k);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        acc[i][j] = fmaf(av[i].x, bv[j].x, acc[i][j]);
        acc[i][j] = fmaf(av[i].y, bv[j].y, acc[i][j]);
        acc[i][j] = fmaf(av[i].z, bv[j].z, acc[i][j]);
        acc[i][j] = fmaf(av[i].w, bv[j].w, acc[i][j]);
      }
  }
}

// acc[i][4 j + e] += sum_k p[ty*RI + i][k] x[k][c0 + 64 j + 4 tx + e], k < K
template <int RI, int RJ, int K, int LP, int LX>
__device__ __forceinline__ void mix_tile(const float* p, const float* x, int tx, int ty,
                                         float (&acc)[RI][4 * RJ]) {
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 pv[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) pv[i] = *reinterpret_cast<const float4*>(p + (ty * RI + i) * LP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const float4 xv = *reinterpret_cast<const float4*>(x + (k + kk) * LX + 64 * j + 4 * tx);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const float w = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
          acc[i][4 * j] = fmaf(w, xv.x, acc[i][4 * j]);
          acc[i][4 * j + 1] = fmaf(w, xv.y, acc[i][4 * j + 1]);
          acc[i][4 * j + 2] = fmaf(w, xv.z, acc[i][4 * j + 2]);
          acc[i][4 * j + 3] = fmaf(w, xv.w, acc[i][4 * j + 3]);
        }
      }
    }
  }
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

// Scratch of a split call: per part, map, batch, head and query the
// unnormalised output, then (max in log2 units, sum).
struct DiffParts {
  float* o;      // [split][2][B*H][N][d]
  float2* ml;    // [split][2][B*H][N]
};

// One query row's end: both maps normalised, lambda, gate, stores, saved tensors.
// o1, o2: this thread's four columns [c, c + 4) of the head (unnormalised).
template <typename T>
__device__ __forceinline__ void finish4(const sva_diff_args& a, int b, int h, int64_t t, int c,
                                        float4 o1, float4 o2, float l1, float l2, float lam) {
  const float i1 = l1 > 0.f ? 1.0f / l1 : 0.f, i2 = l2 > 0.f ? 1.0f / l2 : 0.f;
  o1 = make_float4(o1.x * i1, o1.y * i1, o1.z * i1, o1.w * i1);
  o2 = make_float4(o2.x * i2, o2.y * i2, o2.z * i2, o2.w * i2);
  const int64_t row = static_cast<int64_t>(b) * a.N + t;
  const int col = h * a.d + c;
  if (a.o1 != nullptr) {
    const int64_t at = row * a.H * a.d + col;
    store4(a.o1 + at, o1);
    store4(a.o2 + at, o2);
  }
  float4 y = make_float4(fmaf(-lam, o2.x, o1.x), fmaf(-lam, o2.y, o1.y), fmaf(-lam, o2.z, o1.z),
                         fmaf(-lam, o2.w, o1.w));
  if (a.gate != nullptr) {
    const float4 g = load4(static_cast<const T*>(a.gate) + row * a.ldg + col);
    y = make_float4(y.x * sigmoid_f(g.x), y.y * sigmoid_f(g.y), y.z * sigmoid_f(g.z),
                    y.w * sigmoid_f(g.w));
  }
  store4(static_cast<T*>(a.out) + row * a.ldo + col, y);
}

__device__ __forceinline__ void finish_lse(const sva_diff_args& a, int m, int b, int h, int64_t t,
                                           float mx, float l) {
  if (a.lse != nullptr)
    a.lse[((static_cast<int64_t>(m) * a.B + b) * a.H + h) * a.N + t] =
        l > 0.f ? (mx + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int FR = 32, FK = 32;  // query rows and keys of a tile: 128 threads, 4 x 2 scores each

template <int D>
constexpr size_t fwd_smem() {
  return (static_cast<size_t>(FR + 2 * FK) * (D + 4) + 2 * FR * (FK + 4)) * sizeof(float);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) diff_fwd_kernel(const sva_diff_args a, float scale_log2,
                                                       int n_qtiles, int split, DiffParts parts) {
  constexpr int M = D / 2, L = D + 4, LP = FK + 4, RJ = D / 64;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;
  float* ks = qs + FR * L;
  float* vs = ks + FK * L;
  float* ps = vs + FK * L;  // [2][FR][LP]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int qt = blockIdx.x % n_qtiles, part = blockIdx.x / n_qtiles;
  const int h = blockIdx.y % a.H, b = blockIdx.y / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int nkb = (valid + FK - 1) / FK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(part) * nkb / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * nkb / split);
  const int q0 = qt * FR;
  load_rows<T, FR, D>(qs, a.q, a.ldq, b, a.N, h * D, q0, a.N);
  float o[2][4][4 * RJ] = {};
  float m[2][4], l[2][4];
#pragma unroll
  for (int mm = 0; mm < 2; ++mm)
#pragma unroll
    for (int i = 0; i < 4; ++i) { m[mm][i] = -INFINITY; l[mm][i] = 0.f; }
  for (int kb = kb0; kb < kb1; ++kb) {
    __syncthreads();
    load_rows<T, FK, D>(ks, a.k, a.ldk, b, Nk, h * D, kb * FK, valid);
    load_rows<T, FK, D>(vs, a.v, a.ldv, b, Nk, h * D, kb * FK, valid);
    __syncthreads();
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      float s[4][2] = {};
      dot_tile<4, 2, M, L, L>(qs + mm * M, ks + mm * M, tx, ty, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s[i][j] = kb * FK + tx + 16 * j < valid ? s[i][j] * scale_log2 : -INFINITY;
        // a block holds one valid key at least, so the new maximum is finite
        const float mx = fmaxf(m[mm][i], row_max16(fmaxf(s[i][0], s[i][1])));
        const float f = exp2f(m[mm][i] - mx);
        m[mm][i] = mx;
        const float p0 = exp2f(s[i][0] - mx), p1 = exp2f(s[i][1] - mx);
        l[mm][i] = fmaf(l[mm][i], f, row_sum16(p0 + p1));
#pragma unroll
        for (int e = 0; e < 4 * RJ; ++e) o[mm][i][e] *= f;
        float* pr = ps + (mm * FR + ty * 4 + i) * LP;
        pr[tx] = p0;
        pr[tx + 16] = p1;
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
    if (split > 1) {
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        const int64_t at = ((static_cast<int64_t>(part) * 2 + mm) * a.B * a.H + blockIdx.y) * a.N + t;
#pragma unroll
        for (int j = 0; j < RJ; ++j)
          *reinterpret_cast<float4*>(parts.o + at * D + 64 * j + 4 * tx) =
              make_float4(o[mm][i][4 * j], o[mm][i][4 * j + 1], o[mm][i][4 * j + 2], o[mm][i][4 * j + 3]);
        if (tx == 0) parts.ml[at] = make_float2(m[mm][i], l[mm][i]);
      }
      continue;
    }
    const float lam = lambda_of<T>(a, b, t, h);
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      finish4<T>(a, b, h, t, 64 * j + 4 * tx,
                 make_float4(o[0][i][4 * j], o[0][i][4 * j + 1], o[0][i][4 * j + 2], o[0][i][4 * j + 3]),
                 make_float4(o[1][i][4 * j], o[1][i][4 * j + 1], o[1][i][4 * j + 2], o[1][i][4 * j + 3]),
                 l[0][i], l[1][i], lam);
    if (tx < 2) finish_lse(a, tx, b, h, t, tx == 0 ? m[0][i] : m[1][i], tx == 0 ? l[0][i] : l[1][i]);
  }
}

// Joins the parts of a split call: per map, with M the largest part maximum and
// w_p = 2^(m_p - M), O = sum w_p O_p and l = sum w_p l_p. One warp per query row.
template <typename T>
__global__ void __launch_bounds__(256) diff_merge_kernel(const sva_diff_args a, int split,
                                                         DiffParts parts) {
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.N;
  if (wid >= rows) return;
  const int64_t t = wid % a.N;
  const int bh = static_cast<int>(wid / a.N), h = bh % a.H, b = bh / a.H;
  float4 o[2];
  float mx[2], l[2];
#pragma unroll
  for (int mm = 0; mm < 2; ++mm) {
    mx[mm] = -INFINITY;
    for (int p = 0; p < split; ++p) mx[mm] = fmaxf(mx[mm], parts.ml[(p * 2 + mm) * rows + wid].x);
    o[mm] = make_float4(0.f, 0.f, 0.f, 0.f);
    l[mm] = 0.f;
    for (int p = 0; p < split; ++p) {
      const int64_t at = (p * 2 + mm) * rows + wid;
      const float2 ml = parts.ml[at];
      const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mx[mm]);
      if (w > 0.f && 4 * lane < a.d) {
        const float4 x = *reinterpret_cast<const float4*>(parts.o + at * a.d + 4 * lane);
        o[mm].x = fmaf(w, x.x, o[mm].x);
        o[mm].y = fmaf(w, x.y, o[mm].y);
        o[mm].z = fmaf(w, x.z, o[mm].z);
        o[mm].w = fmaf(w, x.w, o[mm].w);
      }
      l[mm] = fmaf(w, ml.y, l[mm]);
    }
  }
  if (4 * lane < a.d)
    finish4<T>(a, b, h, t, 4 * lane, o[0], o[1], l[0], l[1], lambda_of<T>(a, b, t, h));
  if (lane == 0) {
    finish_lse(a, 0, b, h, t, mx[0], l[0]);
    finish_lse(a, 1, b, h, t, mx[1], l[1]);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

struct DiffBwdScratch {
  void* da;      // [B, N, D] in dtype
  float* stats;  // [B*H][tiles of 64 queries][5][64]: -lse_m log2 e, delta_m, -lambda
  float* dlam;   // [B*H][N]: dlambda per token, where one lambda is shared by all
};
constexpr int kStats = 5;
__device__ __forceinline__ int64_t stat_at(int bh, int n_tiles, int t) {
  return (static_cast<int64_t>(bh) * n_tiles + (t >> 6)) * (kStats * 64) + (t & 63);
}

__device__ __forceinline__ float4 round4(float4 v, const float*) { return v; }
__device__ __forceinline__ float4 round4(float4 v, const __nv_bfloat16*) {
  const uint32_t a = pack_bf16x2(v.x, v.y), b = pack_bf16x2(v.z, v.w);
  return make_float4(bf16lo_to_f32(a), bf16hi_to_f32(a), bf16lo_to_f32(b), bf16hi_to_f32(b));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// dA = dout sigmoid(G) (kept in dtype for the products that follow), dG, the
// row sums delta_m = dA . O_m and dlambda = -delta_2. One warp per (token,
// head), the tokens rounded up to whole tiles of 64: those behind the last
// get a weight of zero. delta_m is made of the rounded dA, as dP is, so that
// dP - delta_m cancels where a map sits on one key; dlambda is a result of its
// own and is made of the unrounded one.
template <typename T>
__global__ void __launch_bounds__(256) diff_prep_kernel(const sva_diff_args a,
                                                        const sva_diff_grads g, DiffBwdScratch ws) {
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tiles = (a.N + 63) / 64;
  const int h = static_cast<int>(wid % a.H);
  const int64_t prow = wid / a.H;
  const int b = static_cast<int>(prow / (n_tiles * 64)), t = static_cast<int>(prow % (n_tiles * 64));
  if (b >= a.B) return;
  const int bh = b * a.H + h;
  float* st = ws.stats + stat_at(bh, n_tiles, t);
  if (t >= a.N) {
    if (lane < kStats) st[lane * 64] = lane < 2 ? -INFINITY : 0.f;
    return;
  }
  const int64_t row = static_cast<int64_t>(b) * a.N + t;
  const float lam = lambda_of<T>(a, b, t, h);
  float d1 = 0.f, d2 = 0.f, dl = 0.f;
  if (4 * lane < a.d) {
    const int col = h * a.d + 4 * lane;
    const int64_t at = row * a.H * a.d + col;
    const float4 o1 = load4<float>(a.o1 + at);
    const float4 o2 = load4<float>(a.o2 + at);
    float4 da = load4(static_cast<const T*>(g.dout) + row * g.lddo + col);
    if (a.gate != nullptr) {
      const float4 x = load4(static_cast<const T*>(a.gate) + row * a.ldg + col);
      const float4 s = make_float4(sigmoid_f(x.x), sigmoid_f(x.y), sigmoid_f(x.z), sigmoid_f(x.w));
      const float4 dg = make_float4(da.x * fmaf(-lam, o2.x, o1.x) * s.x * (1.f - s.x),
                                    da.y * fmaf(-lam, o2.y, o1.y) * s.y * (1.f - s.y),
                                    da.z * fmaf(-lam, o2.z, o1.z) * s.z * (1.f - s.z),
                                    da.w * fmaf(-lam, o2.w, o1.w) * s.w * (1.f - s.w));
      store4(static_cast<T*>(g.dgate) + row * g.lddg + col, dg);
      da = make_float4(da.x * s.x, da.y * s.y, da.z * s.z, da.w * s.w);
    }
    dl = -dot4(da, o2);
    da = round4(da, static_cast<const T*>(nullptr));
    store4(static_cast<T*>(ws.da) + at, da);
    d1 = dot4(da, o1);
    d2 = dot4(da, o2);
  }
  d1 = warp_sum(d1);
  d2 = warp_sum(d2);
  dl = warp_sum(dl);
  if (lane < 2) {
    // an empty row's -infinity stays: its weights come out as 2^-inf = 0
    const float lse = a.lse[(static_cast<int64_t>(lane) * a.B * a.H + bh) * a.N + t];
    st[lane * 64] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    st[(2 + lane) * 64] = lane == 0 ? d1 : d2;
  }
  if (lane == 2) st[4 * 64] = -lam;
  if (lane == 0) {
    if (a.ldl != 0) {
      const float f = (a.flags & SVA_FLAG_LAMBDA_VALUE) ? 1.f : lam * (1.f - lam);
      from_f32(static_cast<T*>(g.dlam) + row * g.lddl + h, dl * f);
    } else {
      ws.dlam[static_cast<int64_t>(bh) * a.N + t] = dl;
    }
  }
}

// dlam of a lambda shared by all tokens: one block per head
template <typename T>
__global__ void __launch_bounds__(1024) diff_dlam_kernel(const sva_diff_args a,
                                                         const sva_diff_grads g,
                                                         DiffBwdScratch ws) {
  __shared__ float part[32];
  const int h = blockIdx.x;
  float s = 0.f;
  for (int b = 0; b < a.B; ++b) {
    const float* p = ws.dlam + (static_cast<int64_t>(b) * a.H + h) * a.N;
    for (int t = threadIdx.x; t < a.N; t += blockDim.x) s += p[t];
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = part[threadIdx.x];
    s = warp_sum(s);
    if (threadIdx.x == 0) {
      const float lam = lambda_of<T>(a, 0, 0, h);
      const float f = (a.flags & SVA_FLAG_LAMBDA_VALUE) ? 1.f : lam * (1.f - lam);
      from_f32(static_cast<T*>(g.dlam) + h, s * f);
    }
  }
}

constexpr int BR = 64, BS = 32;  // stationary rows and streamed rows of a tile: 256 threads

template <int D>
constexpr size_t bwd_smem() {
  return (static_cast<size_t>(2 * BR + 2 * BS) * (D + 4) + 3 * BR * (BS + 4) + 5 * BR) *
         sizeof(float);
}

// KV = false: query rows stand (X = Q, Y = dA), keys stream (X' = K, Y' = V), out dQ.
// KV = true: key rows stand (X = K, Y = V), queries stream (X' = Q, Y' = dA), out dK, dV.
template <typename T, int D, bool KV>
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
  float* stat = wsm + 3 * BR * LP; // [5][ST]: nlse_1, nlse_2, delta_1, delta_2, -lambda
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
    load_rows<T, BR, D>(xs, a.k, a.ldk, b, Nk, h * D, r0, valid);
    load_rows<T, BR, D>(ys, a.v, a.ldv, b, Nk, h * D, r0, valid);
  } else {
    load_rows<T, BR, D>(xs, a.q, a.ldq, b, a.N, h * D, r0, a.N);
    load_rows<T, BR, D>(ys, ws.da, D_all, b, a.N, h * D, r0, a.N);
    load_stats(r0);
  }
  const int stream = KV ? (r0 < valid ? a.N : 0) : valid;
  float acc[4][4 * RJ] = {};             // dQ or dK: columns 64 j + 4 tx + e of the head
  float accv[KV ? 4 : 1][4 * RJ] = {};   // dV
  for (int s0 = 0; s0 < stream; s0 += BS) {
    __syncthreads();
    if (KV) {
      load_rows<T, BS, D>(x2, a.q, a.ldq, b, a.N, h * D, s0, a.N);
      load_rows<T, BS, D>(y2, ws.da, D_all, b, a.N, h * D, s0, a.N);
      load_stats(s0);
    } else {
      load_rows<T, BS, D>(x2, a.k, a.ldk, b, Nk, h * D, s0, valid);
      load_rows<T, BS, D>(y2, a.v, a.ldv, b, Nk, h * D, s0, valid);
    }
    __syncthreads();
    float s1[4][2] = {}, s2[4][2] = {}, dp[4][2] = {};
    dot_tile<4, 2, M, L, L>(xs, x2, tx, ty, s1);
    dot_tile<4, 2, M, L, L>(xs + M, x2 + M, tx, ty, s2);
    dot_tile<4, 2, D, L, L>(ys, y2, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rr = ty * 4 + i, cc = tx + 16 * j;
        const int qi = KV ? cc : rr;
        const bool ok = (KV ? r0 + rr : s0 + cc) < valid;
        const float p1 = ok ? exp2f(fmaf(s1[i][j], scale_log2, stat[qi])) : 0.f;
        const float p2 =
            ok ? stat[4 * ST + qi] * exp2f(fmaf(s2[i][j], scale_log2, stat[ST + qi])) : 0.f;
        wsm[rr * LP + cc] = p1 * (dp[i][j] - stat[2 * ST + qi]);
        wsm[(BR + rr) * LP + cc] = p2 * (dp[i][j] - stat[3 * ST + qi]);
        if (KV) wsm[(2 * BR + rr) * LP + cc] = p1 + p2;
      }
    __syncwarp();  // a row of W and dS is written and read by the same half warp
    // dS_1 mixes the first map's half of the columns, dS_2 the second's
    if (RJ == 2) {
      float half[4][4] = {};
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) half[i][e] = acc[i][4 * (RJ - 1) * m + e];
        mix_tile<4, 1, BS, LP, L>(wsm + m * BR * LP, x2 + m * M, tx, ty, half);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][4 * (RJ - 1) * m + e] = half[i][e];
      }
    } else {  // d = 64: columns 4 tx + e; the first eight threads' belong to map 1
      float one[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) one[i][e] = acc[i][e];
      mix_tile<4, 1, BS, LP, L>(wsm + (tx >= 8 ? BR * LP : 0), x2, tx, ty, one);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = one[i][e];
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
      const float4 v = make_float4(scale * acc[i][4 * j], scale * acc[i][4 * j + 1],
                                   scale * acc[i][4 * j + 2], scale * acc[i][4 * j + 3]);
      if constexpr (KV) {
        store4(static_cast<T*>(g.dk) + row * g.lddk + col, v);
        store4(static_cast<T*>(g.dv) + row * g.lddv + col,
               make_float4(accv[i][4 * j], accv[i][4 * j + 1], accv[i][4 * j + 2], accv[i][4 * j + 3]));
      } else {
        store4(static_cast<T*>(g.dq) + row * g.lddq + col, v);
      }
    }
  }
}

DiffParts parts_of(const DiffPlan& p, const sva_diff_args& a, void* scratch) {
  DiffParts x;
  x.o = static_cast<float*>(scratch);
  x.ml = reinterpret_cast<float2*>(
      x.o + static_cast<size_t>(p.split) * 2 * a.B * a.H * a.N * a.d);
  return x;
}

DiffBwdScratch scratch_of(const sva_diff_args& a, void* scratch) {
  const DiffBwdPlan p = diff_bwd_plan(a.B, a.N, a.H, a.d, a.dtype);
  char* base = static_cast<char*>(scratch);
  return {base, reinterpret_cast<float*>(base + p.stats_off),
          reinterpret_cast<float*>(base + p.dlam_off)};
}

template <typename T, int D>
cudaError_t fwd(const sva_diff_args& a, void* scratch, cudaStream_t s) {
  const DiffPlan p = diff_plan(a.B, a.N, a.H, a.d, a.n_keys, a.dtype);
  const DiffParts parts = parts_of(p, a, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  auto kern = diff_fwd_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(fwd_smem<D>()));
  if (e != cudaSuccess) return e;
  kern<<<dim3(static_cast<unsigned>(p.n_qtiles) * p.split, static_cast<unsigned>(a.B * a.H)), 128,
         fwd_smem<D>(), s>>>(a, scale * kLog2e, p.n_qtiles, p.split, parts);
  if ((e = cudaGetLastError()) != cudaSuccess || p.split == 1) return e;
  const int64_t threads = static_cast<int64_t>(a.B) * a.H * a.N * 32;
  diff_merge_kernel<T><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, s>>>(a, p.split, parts);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  const DiffBwdScratch ws = scratch_of(a, scratch);
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const unsigned bh = static_cast<unsigned>(a.B * a.H);
  const int64_t threads = static_cast<int64_t>(a.B) * ((a.N + 63) / 64 * 64) * a.H * 32;
  diff_prep_kernel<T><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, s>>>(a, g, ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.ldl == 0) diff_dlam_kernel<T><<<static_cast<unsigned>(a.H), 1024, 0, s>>>(a, g, ws);
  auto kq = diff_bwd_kernel<T, D, false>;
  auto kk = diff_bwd_kernel<T, D, true>;
  const int smem = static_cast<int>(bwd_smem<D>());
  if ((e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  kq<<<dim3(static_cast<unsigned>((a.N + BR - 1) / BR), bh), 256, smem, s>>>(a, g, ws, scale);
  kk<<<dim3(static_cast<unsigned>((Nk + BR - 1) / BR), bh), 256, smem, s>>>(a, g, ws, scale);
  return cudaGetLastError();
}

}  // namespace

DiffPlan diff_plan(int B, int N, int H, int d, int n_keys, sva_dtype_t dt) {
  DiffPlan p;
  p.rows = FR;
  p.keys = FK;
  const int Nk = n_keys > 0 ? n_keys : N;
  p.n_qtiles = (N + p.rows - 1) / p.rows;
  p.n_kblocks = (Nk + p.keys - 1) / p.keys;
  const int64_t units = static_cast<int64_t>(p.n_qtiles) * B * H;
  const int64_t slots = 2 * static_cast<int64_t>(std::max(1, device_sm_count()));
  p.split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(slots / units, p.n_kblocks / 4)));
  if (p.split > 1)
    p.partial_bytes = static_cast<size_t>(p.split) * 2 * B * H * N * (static_cast<size_t>(d) + 2) * sizeof(float);
  return p;
}

DiffBwdPlan diff_bwd_plan(int B, int N, int H, int d, sva_dtype_t dt) {
  DiffBwdPlan p;
  const size_t rows = static_cast<size_t>(B) * N;
  const size_t tiles = static_cast<size_t>(B) * H * ((static_cast<size_t>(N) + 63) / 64);
  p.stats_off = align_up(rows * H * d * (dt == SVA_BF16 ? 2 : 4), 256);
  p.dlam_off = p.stats_off + tiles * kStats * 64 * sizeof(float);
  p.total = p.dlam_off + rows * H * sizeof(float);
  return p;
}

cudaError_t diff_fwd_f32(const sva_diff_args& a, int* status, void* scratch, cudaStream_t s) {
  (void)status;
  if (a.dtype == SVA_BF16) return fwd<__nv_bfloat16, 128>(a, scratch, s);
  return a.d == 64 ? fwd<float, 64>(a, scratch, s) : fwd<float, 128>(a, scratch, s);
}

cudaError_t diff_bwd_f32(const sva_diff_args& a, const sva_diff_grads& g, int* status,
                         void* scratch, cudaStream_t s) {
  (void)status;
  if (a.dtype == SVA_BF16) return bwd<__nv_bfloat16, 128>(a, g, scratch, s);
  return a.d == 64 ? bwd<float, 64>(a, g, scratch, s) : bwd<float, 128>(a, g, scratch, s);
}

}  // namespace sva
