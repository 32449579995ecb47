// diff_common.cuh -- what the kernels of the differential softmax anchor share:
// element access, lambda and key counts, the end of a query row, and the layout
// of the backward pass's scratch.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace sva {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Two exponentials 2^x on the FMA pipe, for x <= 126 or so: 2^n 2^f with n = x rounded
// (by adding 1.5 * 2^23) and f in [-1/2, 1/2], 2^f by the degree-4 polynomial of least
// relative error there (2.6e-6, fitted by weighted least squares). The MUFU unit makes
// 16 a cycle and SM, and two maps take twice the exponentials of one per product with
// V: a kernel that is bound by them gives a share to this form.
__device__ __forceinline__ void ex2_poly2(float x0, float x1, float& p0, float& p1) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-126.f));  // a NaN ends as the largest number
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-126.f));
  const uint64_t x = f2pack(x0, x1);
  const uint64_t t = add_f2(x, f2pack(12582912.f, 12582912.f));
  const uint64_t n = add_f2(t, f2pack(-12582912.f, -12582912.f));
  const uint64_t f = fma_f2(n, f2pack(-1.f, -1.f), x);
  uint64_t q = fma_f2(f, f2pack(0.00957010185f, 0.00957010185f), f2pack(0.0559178618f, 0.0559178618f));
  q = fma_f2(f, q, f2pack(0.240247448f, 0.240247448f));
  q = fma_f2(f, q, f2pack(0.693121815f, 0.693121815f));
  q = fma_f2(f, q, f2pack(0.999999261f, 0.999999261f));
  float t0, t1, q0, q1;
  f2unpack(t, t0, t1);
  f2unpack(q, q0, q1);
  p0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  p1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

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

// fp32 to a few units in the last place: the gate meets fp32 results too
__device__ __forceinline__ float sigmoid_f(float x) { return 1.0f / (1.0f + expf(-x)); }

__device__ __forceinline__ int key_count(const int32_t* key_lens, int b, int Nk) {
  return key_lens == nullptr ? Nk : max(0, min(Nk, key_lens[b]));
}

// lam of token t (batch b, head h), and the lambda that it stands for
template <typename T>
__device__ __forceinline__ float lambda_arg(const sva_diff_args& a, int b, int64_t t, int h) {
  const T* p = static_cast<const T*>(a.lam);
  return to_f32(a.ldl == 0 ? p[h] : p[(static_cast<int64_t>(b) * a.N + t) * a.ldl + h]);
}
template <typename T>
__device__ __forceinline__ float lambda_of(const sva_diff_args& a, int b, int64_t t, int h) {
  const float x = lambda_arg<T>(a, b, t, h);
  return (a.flags & SVA_FLAG_LAMBDA_VALUE) ? x : sigmoid_f(x);
}

// What dlambda's sum is multiplied by in the end, 1 for lambda as a value: the sum for a
// sigmoid's lambda carries the factor lambda already (dsigma = lambda (1 - lambda)), and
// 1 - sigma(x) is sigma(-x), which keeps its digits where lambda is next to 1.
template <typename T>
__device__ __forceinline__ float dlambda_factor(const sva_diff_args& a, int b, int64_t t, int h) {
  return (a.flags & SVA_FLAG_LAMBDA_VALUE) ? 1.f : sigmoid_f(-lambda_arg<T>(a, b, t, h));
}

// 1 / l of a row's sum. Without a key l is zero, and so is the row; with keys it is 2^-8 at
// least (the running maximum's threshold), or not a number where a score was none.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }

// One query row's end: both maps normalised, lambda, gate, stores, saved tensors.
// o1, o2: this thread's four columns [c, c + 4) of the head (unnormalised).
template <typename T>
__device__ __forceinline__ void finish4(const sva_diff_args& a, int b, int h, int64_t t, int c,
                                        float4 o1, float4 o2, float l1, float l2, float lam) {
  const float i1 = inverse_sum(l1), i2 = inverse_sum(l2);
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
        l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
}

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

// Tensor map of a bf16 activation [B, N, D] (row stride ld): boxes of 64
// columns (one 128-byte swizzle row) x `rows` tokens; what lies outside is zero.
inline bool diff_map(CUtensorMap* m, const void* base, int64_t ld, int B, int N, int D, int rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(N),
                            static_cast<uint64_t>(B)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2,
                               static_cast<uint64_t>(ld) * 2 * static_cast<uint64_t>(N)};
  const uint32_t box[3] = {64, static_cast<uint32_t>(rows), 1};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

// Work of one forward launch: units (query tile, head, batch), tiles fastest.
// The first n_full run whole, one CTA each; the rest, the last partial wave, are
// cut `split` ways along the key blocks, and every part leaves both maps'
// unnormalised output and (running maximum in log2 units, sum) per row.
struct DiffWork {
  int n_qtiles, H, rows, n_full, split;
  bool cluster;    // a unit's parts are a cluster and join there
  float* partial;  // [unit][part][map][rows x d O | rows x (m, l)]
};
__host__ __device__ inline DiffWork diff_work(const DiffPlan& p, int H, void* scratch) {
  return {p.n_qtiles, H, p.rows, p.n_full, p.split, p.cluster, static_cast<float*>(scratch)};
}
struct DiffUnit {
  int q0, h, b, part, su;  // part < 0: the unit runs whole
};
__device__ __forceinline__ DiffUnit diff_unit(const DiffWork& wk, int cta) {
  DiffUnit u;
  int unit = cta;
  u.part = -1;
  u.su = 0;
  if (cta >= wk.n_full) {
    u.su = (cta - wk.n_full) / wk.split;
    u.part = (cta - wk.n_full) % wk.split;
    unit = wk.n_full + u.su;
  }
  u.q0 = (unit % wk.n_qtiles) * wk.rows;
  u.h = (unit / wk.n_qtiles) % wk.H;
  u.b = unit / wk.n_qtiles / wk.H;
  return u;
}
__device__ __forceinline__ float* diff_part(const DiffWork& wk, int d, int su, int part, int map) {
  return wk.partial +
         ((static_cast<int64_t>(su) * wk.split + part) * 2 + map) * wk.rows * (d + 2);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A backward CTA's tile: cut `cut` of `cuts` of its stream.
struct DiffBwdTile {
  int tile, bh, cut, cuts;
  bool keys_stand;
};
// false: the CTA only fills up a cluster
__device__ __forceinline__ bool diff_bwd_tile(const DiffBwdGrid& grid, int heads, int cta, DiffBwdTile& u) {
  const int n_first = grid.first * heads * grid.cuts;
  const bool in_first = cta < n_first;
  u.keys_stand = in_first == grid.keys_first;
  u.cuts = in_first ? grid.cuts : 1;
  u.cut = in_first ? cta % grid.cuts : 0;
  const int unit = in_first ? cta / grid.cuts : cta - n_first;
  const int tiles = in_first ? grid.first : grid.second;
  u.tile = unit % tiles;
  u.bh = unit / tiles;
  return u.bh < heads;
}

// The end of a unit whose key parts are the CTAs of one cluster: every CTA has its part's
// outputs (unnormalised) in os [2 maps][ROWS][L] and (maximum, sum) in mls [2][ROWS][2], and
// joins a share of the rows, reading the others' over distributed shared memory in the order
// of the parts. w: room for 2 * ROWS * (8 + 1) floats. All threads of the CTA, which must
// have written os and mls before.
template <typename T, int ROWS, int D, int L>
__device__ __forceinline__ void cluster_finish(const sva_diff_args& a, const DiffUnit& u, int split,
                                               const float* os, const float* mls, float* w) {
  cluster_sync();
  const int r0 = ROWS * u.part / split, rows = ROWS * (u.part + 1) / split - r0;
  for (int i = threadIdx.x; i < 2 * rows; i += blockDim.x) {
    const int mp = i / rows, r = r0 + i % rows;
    float2 ml[8];
    float mx = -INFINITY;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      ml[p] = make_float2(-INFINITY, 0.f);
      if (p < split) ml[p] = ld_cluster2(mls + 2 * (mp * ROWS + r), static_cast<uint32_t>(p));
      mx = fmaxf(mx, ml[p].x);
    }
    float l = 0.f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      // a part without keys has a weight of zero, and its outputs are zero; one whose scores
      // are not numbers has no maximum either, but its sum and outputs are none, and stay so
      const float wp = ml[p].x == -INFINITY ? 0.f : exp2f(ml[p].x - mx);
      l = fmaf(wp, ml[p].y, l);
      w[(mp * ROWS + r) * 9 + p] = wp;
    }
    w[(mp * ROWS + r) * 9 + 8] = l;
    const int t = u.q0 + r;
    if (t < a.N) finish_lse(a, mp, u.b, u.h, t, mx, l);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D / 4; i += blockDim.x) {
    const int r = r0 + i / (D / 4), c = (i % (D / 4)) * 4, t = u.q0 + r;
    if (t >= a.N) break;
    const float *w1 = w + r * 9, *w2 = w + (ROWS + r) * 9;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int p = 0; p < split; ++p) {
      const float4 o1 = ld_cluster4(os + r * L + c, static_cast<uint32_t>(p));
      const float4 o2 = ld_cluster4(os + (ROWS + r) * L + c, static_cast<uint32_t>(p));
      x = make_float4(fmaf(w1[p], o1.x, x.x), fmaf(w1[p], o1.y, x.y), fmaf(w1[p], o1.z, x.z), fmaf(w1[p], o1.w, x.w));
      y = make_float4(fmaf(w2[p], o2.x, y.x), fmaf(w2[p], o2.y, y.y), fmaf(w2[p], o2.z, y.z), fmaf(w2[p], o2.w, y.w));
    }
    finish4<T>(a, u.b, u.h, t, c, x, y, w1[8], w2[8], lambda_of<T>(a, u.b, t, u.h));
  }
  cluster_sync();  // nobody leaves while its shared memory is read
}

}  // namespace
}  // namespace sva
