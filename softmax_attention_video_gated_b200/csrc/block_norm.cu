// block_norm.cu -- the norms around a block, fused with the block's gate, the
// residual scale and the residual update, forward and backward.
//
// Forward, per token row: h' = a h + g_b (N(o) w_post); u = N(h') w_pre (1 + s_b)
// + t_b, N the RMS or layer norm over D. Backward, with x^ the normalised row,
// r its reciprocal deviation and y the gradient behind the norm:
//     N'(y) = r (y - x^ mean(y x^) [- mean(y)])
//     dh' = dh_out + N'(du w_pre (1 + s_b)),  dh = a dh'
//     do  = N'(dh' g_b w_post)
// The sums over tokens need three column sums only, sum du, sum du h'^ and
// sum dh' o^ per batch: every weight's gradient is one of them times a vector.
//
// All of it is memory traffic: 12 bytes per value forward in bf16 (o, h in; h',
// u out), 18 backward. A group of W warps owns a row: each lane holds chunks
// of 8 consecutive values, so all loads are 16 bytes wide, a row is read once
// and both norms run on registers. A group keeps its per-channel factors in
// registers (g_b w_post, w_pre (1 + s_b), t_b: one batch per group) and walks
// over several rows, so the factors cost nothing per row; the column sums stay
// in registers too and leave once per group, summed by a second kernel in a
// fixed order.
#include <algorithm>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace sva {
namespace {

constexpr int kMaxSums = 3;  // column sums of the backward pass

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[8]);

// n: values of the row left at p (the chunk is read whole when n >= 8)
template <>
__device__ __forceinline__ void load8<float>(const float* p, int n, float (&f)[8]) {
  if (n >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.f;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, int n, float (&f)[8]) {
  if (n >= 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16lo_to_f32(v.x); f[1] = bf16hi_to_f32(v.x);
    f[2] = bf16lo_to_f32(v.y); f[3] = bf16hi_to_f32(v.y);
    f[4] = bf16lo_to_f32(v.z); f[5] = bf16hi_to_f32(v.z);
    f[6] = bf16lo_to_f32(v.w); f[7] = bf16hi_to_f32(v.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? __bfloat162float(p[i]) : 0.f;
  }
}

__device__ __forceinline__ void store8(float* p, int n, const float (&f)[8]) {
  if (n >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, const float (&f)[8]) {
  if (n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16(f[i]);
  }
}

// Sums of two values over the W warps of a group. `slot` alternates, so one
// barrier per sum is enough: a warp writes a slot again only after the barrier
// of the sum in between, which every warp reaches after reading the slot.
template <int W>
__device__ __forceinline__ float2 group_sum(float2 v, float2 (*part)[W], int& slot, int warp_in,
                                            int bar) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (W == 1) return v;
  if (lane_id() == 0) part[slot][warp_in] = v;
  named_barrier_sync(bar, 32 * W);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float2 p = part[slot][w];
    s.x += p.x;
    s.y += p.y;
  }
  slot ^= 1;
  return s;
}

// Rows of one launch: every batch is cut into `units` runs of `per` rows, one
// group of warps each.
struct RowRuns {
  int units, per;
  int64_t total;  // B * units
};

template <typename T, int W, int NV>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256)
    norm_fwd_kernel(const sva_block_norm_args a, RowRuns rr) {
  constexpr int G = 32 * W;                          // threads of a group
  constexpr int GROUPS = W >= 8 ? 1 : 8 / W;
  __shared__ float2 part[GROUPS][2][W];
  const int g = threadIdx.x / G, tg = threadIdx.x % G;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * GROUPS + g;
  if (unit >= rr.total) return;
  const int b = static_cast<int>(unit / rr.units), ub = static_cast<int>(unit % rr.units);
  const int t0 = ub * rr.per, t1 = min(a.N, t0 + rr.per);
  const bool post = a.o != nullptr, pre = a.u != nullptr;
  const bool layer = a.kind == SVA_NORM_LAYER;
  int slot = 0;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  float gw[NV][8], ws[NV][8], sh[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + tg) * 8, n = a.D - c;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) { gw[i][e] = 1.f; ws[i][e] = 1.f; sh[i][e] = 0.f; }
    if (a.w_post != nullptr) load8(static_cast<const T*>(a.w_post) + c, n, gw[i]);
    if (a.gate != nullptr) {
      load8(static_cast<const T*>(a.gate) + b * a.ldgate + c, n, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[i][e] *= x[e];
    }
    if (a.w_pre != nullptr) load8(static_cast<const T*>(a.w_pre) + c, n, ws[i]);
    if (a.scale != nullptr) {
      load8(static_cast<const T*>(a.scale) + b * a.ldscale + c, n, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ws[i][e] *= 1.f + x[e];
    }
    if (a.shift != nullptr) load8(static_cast<const T*>(a.shift) + b * a.ldshift + c, n, sh[i]);
  }
  // mean and reciprocal deviation of a row; x becomes the normalised row
  auto normalise = [&](float (&x)[NV][8]) -> float2 {
    float mean = 0.f;
    float s = 0.f;
    if (layer) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[i][e];
      mean = group_sum<W>(make_float2(s, 0.f), part[g], slot, tg >> 5, 1 + g).x * inv_d;
      // the values behind the row's end stay zero, so they count for nothing
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = a.D - (i * G + tg) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = e < n ? x[i][e] - mean : 0.f;
      }
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[i][e], x[i][e], s);
    const float var = group_sum<W>(make_float2(s, 0.f), part[g], slot, tg >> 5, 1 + g).x * inv_d;
    const float r = 1.0f / sqrtf(var + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= r;
    return make_float2(mean, r);
  };
  for (int t = t0; t < t1; ++t) {
    const int64_t row = static_cast<int64_t>(b) * a.N + t;
    float h[NV][8], x[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + tg) * 8, n = a.D - c;
      load8(a.h + row * a.ldh + c, n, h[i]);
      if (post) load8(static_cast<const T*>(a.o) + row * a.ldo + c, n, x[i]);
    }
    float2 so = make_float2(0.f, 0.f), sp = so;
    if (post) {
      so = normalise(x);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + tg) * 8, n = a.D - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = fmaf(gw[i][e], x[i][e], a.res_scale * h[i][e]);
        store8(a.h_out + row * a.ldho + c, n, h[i]);
      }
    }
    if (pre) {
      sp = normalise(h);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + tg) * 8, n = a.D - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = fmaf(h[i][e], ws[i][e], sh[i][e]);
        store8(static_cast<T*>(a.u) + row * a.ldu + c, n, h[i]);
      }
    }
    if (a.stats != nullptr && tg == 0)
      *reinterpret_cast<float4*>(a.stats + row * 4) = make_float4(so.x, so.y, sp.x, sp.y);
  }
}

template <typename T, int W, int NV>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256)
    norm_bwd_kernel(const sva_block_norm_args a, const sva_block_norm_grads gr, RowRuns rr,
                    float* partial) {
  constexpr int G = 32 * W;
  constexpr int GROUPS = W >= 8 ? 1 : 8 / W;
  __shared__ float2 part[GROUPS][2][W];
  const int g = threadIdx.x / G, tg = threadIdx.x % G;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * GROUPS + g;
  if (unit >= rr.total) return;
  const int b = static_cast<int>(unit / rr.units), ub = static_cast<int>(unit % rr.units);
  const int t0 = ub * rr.per, t1 = min(a.N, t0 + rr.per);
  const bool post = a.o != nullptr, pre = a.u != nullptr;
  const bool layer = a.kind == SVA_NORM_LAYER;
  const float* hsrc = post ? a.h_out : a.h;
  const int64_t ldhs = post ? a.ldho : a.ldh;
  int slot = 0;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  float gw[NV][8], ws[NV][8], sum_du[NV][8], sum_dux[NV][8], sum_do[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + tg) * 8, n = a.D - c;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gw[i][e] = 1.f; ws[i][e] = 1.f;
      sum_du[i][e] = 0.f; sum_dux[i][e] = 0.f; sum_do[i][e] = 0.f;
    }
    if (a.w_post != nullptr) load8(static_cast<const T*>(a.w_post) + c, n, gw[i]);
    if (a.gate != nullptr) {
      load8(static_cast<const T*>(a.gate) + b * a.ldgate + c, n, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[i][e] *= x[e];
    }
    if (a.w_pre != nullptr) load8(static_cast<const T*>(a.w_pre) + c, n, ws[i]);
    if (a.scale != nullptr) {
      load8(static_cast<const T*>(a.scale) + b * a.ldscale + c, n, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) ws[i][e] *= 1.f + x[e];
    }
  }
  for (int t = t0; t < t1; ++t) {
    const int64_t row = static_cast<int64_t>(b) * a.N + t;
    const float4 st = *reinterpret_cast<const float4*>(a.stats + row * 4);
    float dh[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + tg) * 8, n = a.D - c;
      if (gr.dh_out != nullptr) {
        load8(gr.dh_out + row * gr.lddho + c, n, dh[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[i][e] = 0.f;
      }
    }
    float on[NV][8];
    if (post) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + tg) * 8, n = a.D - c;
        load8(static_cast<const T*>(a.o) + row * a.ldo + c, n, on[i]);
      }
    }
    if (pre) {
      float x[NV][8], y[NV][8];
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + tg) * 8, n = a.D - c;
        load8(hsrc + row * ldhs + c, n, x[i]);
        load8(static_cast<const T*>(gr.du) + row * gr.lddu + c, n, y[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] = (x[i][e] - st.z) * st.w;
          sum_du[i][e] += y[i][e];
          sum_dux[i][e] = fmaf(y[i][e], x[i][e], sum_dux[i][e]);
          y[i][e] *= ws[i][e];
          s.x = fmaf(y[i][e], x[i][e], s.x);  // y is zero behind the row's end
          s.y += y[i][e];
        }
      }
      s = group_sum<W>(s, part[g], slot, tg >> 5, 1 + g);
      const float m1 = s.x * inv_d, m0 = layer ? s.y * inv_d : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dh[i][e] = fmaf(st.w, y[i][e] - m0 - x[i][e] * m1, dh[i][e]);
    }
    if (post) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = a.D - (i * G + tg) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          on[i][e] = (on[i][e] - st.x) * st.y;
          const float y = e < n ? dh[i][e] * gw[i][e] : 0.f;
          s.x = fmaf(y, on[i][e], s.x);
          s.y += y;
        }
      }
      s = group_sum<W>(s, part[g], slot, tg >> 5, 1 + g);
      const float m1 = s.x * inv_d, m0 = layer ? s.y * inv_d : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + tg) * 8, n = a.D - c;
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum_do[i][e] = fmaf(dh[i][e], on[i][e], sum_do[i][e]);
          d[e] = st.y * (dh[i][e] * gw[i][e] - m0 - on[i][e] * m1);
          dh[i][e] *= a.res_scale;
        }
        store8(static_cast<T*>(gr.d_o) + row * gr.lddo + c, n, d);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + tg) * 8, n = a.D - c;
      store8(gr.dh + row * gr.lddh + c, n, dh[i]);
    }
  }
  if (partial == nullptr) return;
  float* p = partial + unit * kMaxSums * a.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + tg) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e >= a.D) break;
      if (pre) {
        p[c + e] = sum_du[i][e];
        p[a.D + c + e] = sum_dux[i][e];
      }
      if (post) p[2 * a.D + c + e] = sum_do[i][e];
    }
  }
}

// The groups' column sums to the gradients: 32 columns per block, the units of
// a batch spread over 8 rows of threads and joined in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256)
    norm_sums_kernel(const sva_block_norm_args a, const sva_block_norm_grads gr, RowRuns rr,
                     const float* partial) {
  __shared__ float red[kMaxSums][8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const bool ok = c < a.D;
  const bool post = a.o != nullptr, pre = a.u != nullptr;
  const float wp = ok && a.w_pre != nullptr ? static_cast<float>(static_cast<const T*>(a.w_pre)[c]) : 1.f;
  const float wq = ok && a.w_post != nullptr ? static_cast<float>(static_cast<const T*>(a.w_post)[c]) : 1.f;
  float dwp = 0.f, dwq = 0.f;
  for (int b = 0; b < a.B; ++b) {
    float s[kMaxSums] = {0.f, 0.f, 0.f};
    if (ok) {
      for (int u = ty; u < rr.units; u += 8) {
        const float* p = partial + (static_cast<int64_t>(b) * rr.units + u) * kMaxSums * a.D + c;
        if (pre) {
          s[0] += p[0];
          s[1] += p[a.D];
        }
        if (post) s[2] += p[2 * a.D];
      }
    }
#pragma unroll
    for (int k = 0; k < kMaxSums; ++k) red[k][ty][tx] = s[k];
    __syncthreads();
    if (ty == 0 && ok) {
#pragma unroll
      for (int k = 0; k < kMaxSums; ++k) {
        s[k] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s[k] += red[k][w][tx];
      }
      const int64_t at = static_cast<int64_t>(b) * a.D + c;
      if (gr.dshift != nullptr) gr.dshift[at] = s[0];
      if (gr.dscale != nullptr) gr.dscale[at] = s[1] * wp;
      if (gr.dgate != nullptr) gr.dgate[at] = s[2] * wq;
      const float sc = a.scale != nullptr
                           ? 1.f + static_cast<float>(static_cast<const T*>(a.scale)[b * a.ldscale + c])
                           : 1.f;
      const float gt = a.gate != nullptr
                           ? static_cast<float>(static_cast<const T*>(a.gate)[b * a.ldgate + c])
                           : 1.f;
      dwp = fmaf(s[1], sc, dwp);
      dwq = fmaf(s[2], gt, dwq);
    }
    __syncthreads();
  }
  if (ty == 0 && ok) {
    if (gr.dw_pre != nullptr) gr.dw_pre[c] = dwp;
    if (gr.dw_post != nullptr) gr.dw_post[c] = dwq;
  }
}

// Runs of rows: about `groups_per_sm` groups per SM, at least one row each.
RowRuns row_runs(int B, int N, int groups_per_sm) {
  const int64_t want = static_cast<int64_t>(std::max(1, device_sm_count())) * groups_per_sm;
  RowRuns r;
  const int64_t units = std::min<int64_t>(N, std::max<int64_t>(1, want / B));
  r.per = static_cast<int>((N + units - 1) / units);
  r.units = (N + r.per - 1) / r.per;
  r.total = static_cast<int64_t>(B) * r.units;
  return r;
}

// warps of a row's group: one chunk of 8 values per lane up to 4,096 channels, two above
int group_warps(int D) {
  int w = 1;
  while (w < 16 && 256 * w < D) w *= 2;
  return w;
}

int groups_per_cta(int w) { return w >= 8 ? 1 : 8 / w; }
// two 256-thread CTAs of groups per SM, one CTA of 512 threads
int groups_per_sm(int w) { return w >= 8 ? (w > 8 ? 2 : 3) : 3 * (8 / w); }

template <typename T, int W, int NV>
cudaError_t launch_fwd(const sva_block_norm_args& a, cudaStream_t s) {
  const RowRuns rr = row_runs(a.B, a.N, groups_per_sm(W));
  const int gc = groups_per_cta(W);
  norm_fwd_kernel<T, W, NV><<<static_cast<unsigned>((rr.total + gc - 1) / gc), W > 8 ? 32 * W : 256, 0, s>>>(a, rr);
  return cudaGetLastError();
}

template <typename T, int W, int NV>
cudaError_t launch_bwd(const sva_block_norm_args& a, const sva_block_norm_grads& g, float* partial,
                       cudaStream_t s) {
  const RowRuns rr = row_runs(a.B, a.N, groups_per_sm(W));
  const int gc = groups_per_cta(W);
  norm_bwd_kernel<T, W, NV><<<static_cast<unsigned>((rr.total + gc - 1) / gc), W > 8 ? 32 * W : 256, 0, s>>>(
      a, g, rr, partial);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || partial == nullptr) return e;
  norm_sums_kernel<T><<<(a.D + 31) / 32, 256, 0, s>>>(a, g, rr, partial);
  return cudaGetLastError();
}

#define SVA_NORM_DISPATCH(fn, T, ...)                  \
  switch (group_warps(a.D)) {                          \
    case 1: return fn<T, 1, 1>(__VA_ARGS__);           \
    case 2: return fn<T, 2, 1>(__VA_ARGS__);           \
    case 4: return fn<T, 4, 1>(__VA_ARGS__);           \
    case 8: return fn<T, 8, 1>(__VA_ARGS__);           \
    default:                                           \
      if (a.D <= 4096) return fn<T, 16, 1>(__VA_ARGS__); \
      return fn<T, 16, 2>(__VA_ARGS__);                \
  }

}  // namespace

size_t block_norm_partial_bytes(int B, int N, int D) {
  const RowRuns rr = row_runs(B, N, groups_per_sm(group_warps(D)));
  return static_cast<size_t>(rr.total) * kMaxSums * D * sizeof(float);
}

cudaError_t block_norm_fwd(const sva_block_norm_args& a, cudaStream_t s) {
  if (a.dtype == SVA_BF16) {
    SVA_NORM_DISPATCH(launch_fwd, __nv_bfloat16, a, s)
  }
  SVA_NORM_DISPATCH(launch_fwd, float, a, s)
}

cudaError_t block_norm_bwd(const sva_block_norm_args& a, const sva_block_norm_grads& g,
                           void* scratch, cudaStream_t s) {
  const bool sums = g.dw_post != nullptr || g.dgate != nullptr || g.dw_pre != nullptr ||
                    g.dscale != nullptr || g.dshift != nullptr;
  float* partial = sums ? static_cast<float*>(scratch) : nullptr;
  if (a.dtype == SVA_BF16) {
    SVA_NORM_DISPATCH(launch_bwd, __nv_bfloat16, a, g, partial, s)
  }
  SVA_NORM_DISPATCH(launch_bwd, float, a, g, partial, s)
}

}  // namespace sva
