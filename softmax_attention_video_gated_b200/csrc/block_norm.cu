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
// u out), 18 backward. A group of W warps owns a row, as few as hold it with NQ
// = 4 quads of 4 consecutive values a thread (the sums' shuffles and barriers
// cost a warp the same whatever it holds: 8 values a thread took 453 instructions
// per warp and row and were bound by issuing them); quads are 128 values apart per
// warp, so every access is one coalesced run. A warp copies its own values of the
// next rows into its own place in shared memory (cp.async, no barrier: no other
// warp reads them), `stages` rows ahead, so that loads stay in flight while the
// group reduces. A row is read once and both norms run on registers. A CTA's
// groups share one batch, and with it the per-channel factors in shared memory
// (g_b w_post, w_pre (1 + s_b), t_b). The column sums stay in registers over a
// CTA's rows, leave once per CTA, and are summed by a second kernel in a fixed
// order.
// 16,380 rows of 2,048 channels in bf16 (402 MB forward, 604 MB backward): 75 us a call
// forward, 5.4 TB/s, 0.82 of the measured copy rate; forward and backward 188, the backward
// kernel 94 alone and 10 for the sums. Above 6,144 channels a backward row leaves room for
// one stage, and its loads are waited for: 8,192 channels 3.7 TB/s where 6,144 reach 5.5.
// The backward pass keeps 48 sums and a row a thread in registers: at 128 of them it
// spilled, and next to this much shared memory L1 holds no spills (180 us).
#include <algorithm>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace sva {
namespace {

constexpr int kMaxSums = 3;     // column sums of the backward pass
constexpr int kMaxWarps = 16;   // of a row's group
constexpr int kMaxStages = 6;

__device__ __forceinline__ float4 widen(float4 v) { return v; }
__device__ __forceinline__ float4 widen(uint2 v) {
  return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
}
template <typename T>
struct Quad {
  using type = float4;
};
template <>
struct Quad<__nv_bfloat16> {
  using type = uint2;
};
template <typename T>
using quad_t = typename Quad<T>::type;

// a quad at p, n of its values inside the row (the others are zero)
template <typename T>
__device__ __forceinline__ float4 load4n(const T* p, int n) {
  if (n >= 4) return widen(*reinterpret_cast<const quad_t<T>*>(p));
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = i < n ? static_cast<float>(p[i]) : 0.f;
  return make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4n(float* p, int n, float4 v) {
  if (n >= 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = f[i];
  }
}
__device__ __forceinline__ void store4n(__nv_bfloat16* p, int n, float4 v) {
  if (n >= 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  } else {
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = __float2bfloat16(f[i]);
  }
}

// until at most `stages` - 1 later rows are still on their way
__device__ __forceinline__ void copy_wait(int stages) {
  switch (stages) {
    case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}

#define SVA_EACH(i) _Pragma("unroll") for (int i = 0; i < NQ; ++i)

// Four values as two packed pairs: one instruction for two of them, each rounded
// as its scalar counterpart.
__device__ __forceinline__ uint64_t lo2(float4 a) { return f2pack(a.x, a.y); }
__device__ __forceinline__ uint64_t hi2(float4 a) { return f2pack(a.z, a.w); }
__device__ __forceinline__ uint64_t both(float a) { return f2pack(a, a); }
__device__ __forceinline__ float4 join4(uint64_t lo, uint64_t hi) {
  float4 r;
  f2unpack(lo, r.x, r.y);
  f2unpack(hi, r.z, r.w);
  return r;
}
__device__ __forceinline__ float4 operator*(float4 a, float4 b) {
  return join4(mul_f2(lo2(a), lo2(b)), mul_f2(hi2(a), hi2(b)));
}
__device__ __forceinline__ float4 operator*(float4 a, float b) {
  return join4(mul_f2(lo2(a), both(b)), mul_f2(hi2(a), both(b)));
}
__device__ __forceinline__ float4 operator+(float4 a, float4 b) {
  return join4(add_f2(lo2(a), lo2(b)), add_f2(hi2(a), hi2(b)));
}
__device__ __forceinline__ float4 operator-(float4 a, float b) {
  return join4(add_f2(lo2(a), both(-b)), add_f2(hi2(a), both(-b)));
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return join4(fma_f2(lo2(a), lo2(b), lo2(c)), fma_f2(hi2(a), hi2(b), hi2(c)));
}
__device__ __forceinline__ float4 fma4(float a, float4 b, float4 c) {
  return join4(fma_f2(both(a), lo2(b), lo2(c)), fma_f2(both(a), hi2(b), hi2(c)));
}
// running sums in two pairs, joined at the end
struct Acc {
  uint64_t lo = 0, hi = 0;
  __device__ __forceinline__ void dot(float4 a, float4 b) {
    lo = fma_f2(lo2(a), lo2(b), lo);
    hi = fma_f2(hi2(a), hi2(b), hi);
  }
  __device__ __forceinline__ void add(float4 a) {
    lo = add_f2(lo2(a), lo);
    hi = add_f2(hi2(a), hi);
  }
  __device__ __forceinline__ float total() const {
    float x, y;
    f2unpack(add_f2(lo, hi), x, y);
    return x + y;
  }
};
__device__ __forceinline__ float sum4(float4 a) { return (a.x + a.y) + (a.z + a.w); }
// the first n values, zero behind them
__device__ __forceinline__ float4 keep4(float4 a, int n) {
  return make_float4(n > 0 ? a.x : 0.f, n > 1 ? a.y : 0.f, n > 2 ? a.z : 0.f, n > 3 ? a.w : 0.f);
}
__device__ __forceinline__ float4 all4(float x) { return make_float4(x, x, x, x); }

// A group of W warps: sums over it, with one barrier each. `slot` alternates: a
// warp writes a slot again only after the barrier of the sum in between, which
// every warp reaches after reading the slot. The warps' parts are read back as
// whole vectors (those of missing warps are zero): a loop over W loads one after
// the other was a quarter of a row's time.
struct GroupSums {
  float part[2][2][kMaxWarps];  // [slot][value][warp]
};
struct Group {
  GroupSums* sums;
  int W, warp_in, bar, slot;
  __device__ __forceinline__ void init(int tg) {
    for (int i = tg; i < 4 * kMaxWarps; i += 32 * W) (&sums->part[0][0][0])[i] = 0.f;
    if (W > 1) named_barrier_sync(bar, 32 * W);
  }
  __device__ __forceinline__ float joined(int value) const {
    const float4* p = reinterpret_cast<const float4*>(sums->part[slot][value]);
    float s = sum4(p[0]);
    if (W > 4) s += sum4(p[1]);
    if (W > 8) s += sum4(p[2]) + sum4(p[3]);
    return s;
  }
  __device__ __forceinline__ float2 sum(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (W == 1) return v;
    // all lanes hold the sum and write it: bar.sync wants the whole warp at once
    sums->part[slot][0][warp_in] = v.x;
    sums->part[slot][1][warp_in] = v.y;
    named_barrier_sync(bar, 32 * W);
    v = make_float2(joined(0), joined(1));
    slot ^= 1;
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (W == 1) return v;
    sums->part[slot][0][warp_in] = v;
    named_barrier_sync(bar, 32 * W);
    v = joined(0);
    slot ^= 1;
    return v;
  }
};

// Rows of one launch: `units` CTAs of `groups` groups of W warps share a batch, the
// groups taking its rows in turn.
struct RowRuns {
  int W, groups, stages, units;
  int64_t total;  // B * units
};

// A thread's place in its group's rows: a warp owns NQ * 128 values in one run, a
// thread a quad of each 128, so that all its offsets are constants.
template <int NQ>
struct Place {
  int c0, D;  // its first column, the row's values
  bool full;  // the warp's run lies inside the row
  __device__ __forceinline__ Place(int tg, int D_) : c0((tg >> 5) * NQ * 128 + (tg & 31) * 4), D(D_) {
    full = (tg >> 5) * NQ * 128 + NQ * 128 <= D_;
  }
  __device__ __forceinline__ int left(int i) const { return D - c0 - i * 128; }
};

// the per-channel factors of a batch into shared memory: g w_post, w_pre (1 + s), t
template <typename T, int NQ>
__device__ __forceinline__ void load_factors(const sva_block_norm_args& a, int b, int width, float* gw,
                                             float* ws, float* sh) {
  const T* wq = static_cast<const T*>(a.w_post);
  const T* wp = static_cast<const T*>(a.w_pre);
  for (int c = threadIdx.x * 4; c < width; c += blockDim.x * 4) {
    const int n = a.D - c;
    float4 x = wq != nullptr ? load4n(wq + c, n) : all4(1.f);
    if (a.gate != nullptr) x = x * load4n(static_cast<const T*>(a.gate) + b * a.ldgate + c, n);
    *reinterpret_cast<float4*>(gw + c) = x;
    x = wp != nullptr ? load4n(wp + c, n) : all4(1.f);
    if (a.scale != nullptr)
      x = x * (load4n(static_cast<const T*>(a.scale) + b * a.ldscale + c, n) + all4(1.f));
    *reinterpret_cast<float4*>(ws + c) = x;
    if (sh != nullptr)
      *reinterpret_cast<float4*>(sh + c) =
          a.shift != nullptr ? load4n(static_cast<const T*>(a.shift) + b * a.ldshift + c, n) : all4(0.f);
  }
}

// Staged values of one row in shared memory: [quad i][thread] of each array, so
// that a warp's accesses are one run. A warp copies what its own lanes read, 16
// bytes a copy: an fp32 quad each, or two lanes' bf16 quads (8-byte copies go
// through the few KB of L1 that the ring leaves and waited there: 3.6 TB/s).
template <int NQ>
__device__ __forceinline__ void stage_row(char* st, const float* row, const Place<NQ>& at) {
  char* dst = st + at.c0 * 4;
  const float* src = row + at.c0;
  if (at.full) {
    SVA_EACH(i) copy16(dst + i * 512, src + i * 128);
  } else {
    // behind the row's end nothing is read; the address stays inside it
    SVA_EACH(i) copy16_upto(dst + i * 512, at.left(i) > 0 ? src + i * 128 : row, at.left(i) * 4);
  }
}
template <int NQ>
__device__ __forceinline__ void stage_row(char* st, const __nv_bfloat16* row, const Place<NQ>& at) {
  const int lane = lane_id(), c = at.c0 + lane * 4;  // twice as far into the warp's run
  if (NQ == 1 && lane >= 16) return;
  char* dst = st + c * 2;
  const __nv_bfloat16* src = row + c;
#pragma unroll
  for (int i = 0; i < (NQ + 1) / 2; ++i) {
    const int left = at.D - c - i * 256;
    if (at.full)
      copy16(dst + i * 512, src + i * 256);
    else
      copy16_upto(dst + i * 512, left > 0 ? src + i * 256 : row, left * 2);
  }
}
template <typename T, int NQ>
__device__ __forceinline__ void staged(const char* st, const Place<NQ>& at, float4 (&x)[NQ]) {
  const quad_t<T>* src = reinterpret_cast<const quad_t<T>*>(st) + at.c0 / 4;
  SVA_EACH(i) x[i] = widen(src[i * 32]);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
// p: this thread's first quad of the row
template <typename T, int NQ>
__device__ __forceinline__ void store_row(T* p, const Place<NQ>& at, const float4 (&x)[NQ]) {
  if (at.full) {
    SVA_EACH(i) store4(p + i * 128, x[i]);
  } else {
    SVA_EACH(i) store4n(p + i * 128, at.left(i), x[i]);
  }
}

template <typename T, int NQ, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 3 : 1)
    norm_fwd_kernel(const __grid_constant__ sva_block_norm_args a, RowRuns rr) {
  extern __shared__ __align__(16) char dyn[];
  GroupSums* gsums = reinterpret_cast<GroupSums*>(dyn);
  const int G = 32 * rr.W;
  const int g = threadIdx.x / G;
  const int tg = static_cast<int>(threadIdx.x) - g * G;
  const Place<NQ> at(tg, a.D);
  const int b = static_cast<int>(blockIdx.x) / rr.units, ub = static_cast<int>(blockIdx.x) % rr.units;
  const bool post = a.o != nullptr, pre = a.u != nullptr;
  const bool layer = a.kind == SVA_NORM_LAYER;
  Group grp{&gsums[g], rr.W, tg >> 5, 1 + g, 0};
  grp.init(tg);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int width = NQ * G * 4;
  float* gw = reinterpret_cast<float*>(gsums + rr.groups);
  float* ws = gw + width;
  float* sh = ws + width;
  // a stage: h, then o
  const int h_bytes = width * 4, stage_bytes = h_bytes + (post ? width * static_cast<int>(sizeof(T)) : 0);
  char* ring = reinterpret_cast<char*>(sh + width) + g * rr.stages * stage_bytes;
  const int base = b * a.N;  // rows are numbered over all batches
  // neighbours in time are neighbours in memory: runs of rows of their own, a CTA each,
  // kept 1,776 streams open at once and 402 MB took 80 us
  uint32_t t = base + ub * rr.groups + g;
  const uint32_t end = base + a.N, step = rr.units * rr.groups;
  uint32_t tf = t;
  int sf = 0;  // the next row to fetch and its stage
  auto fetch = [&]() {
    if (tf < end) {
      char* st = ring + sf * stage_bytes;
      const int64_t row = tf;
      stage_row(st, a.h + row * a.ldh, at);
      if (post) stage_row(st + h_bytes, static_cast<const T*>(a.o) + row * a.ldo, at);
    }
    copy_commit();
    tf += step;
    sf = sf + 1 == rr.stages ? 0 : sf + 1;
  };
  for (int s = 0; s < rr.stages; ++s) fetch();
  load_factors<T, NQ>(a, b, width, gw, ws, sh);
  __syncthreads();
  // mean and reciprocal deviation of a row; x becomes the normalised row
  auto normalise = [&](float4 (&x)[NQ]) -> float2 {
    float mean = 0.f;
    if (layer) {
      Acc s;
      SVA_EACH(i) s.add(x[i]);
      mean = grp.sum(s.total()) * inv_d;
      SVA_EACH(i) {
        x[i] = x[i] - mean;
        // the values behind the row's end stay zero, so they count for nothing
        if (!at.full) x[i] = keep4(x[i], at.left(i));
      }
    }
    Acc s;
    SVA_EACH(i) s.dot(x[i], x[i]);
    const float r = rsqrtf(grp.sum(s.total()) * inv_d + a.eps);
    SVA_EACH(i) x[i] = x[i] * r;
    return make_float2(mean, r);
  };
  for (int st = 0; t < end; t += step) {
    const int64_t row = t;
    float4 h[NQ], x[NQ];
    copy_wait(rr.stages);
    __syncwarp();
    const char* stage = ring + st * stage_bytes;
    st = st + 1 == rr.stages ? 0 : st + 1;
    staged<float, NQ>(stage, at, h);
    if (post) staged<T, NQ>(stage + h_bytes, at, x);
    float2 so = make_float2(0.f, 0.f), sp = so;
    if (post)
      so = normalise(x);
    else
      sp = normalise(h);
    __syncwarp();  // the warp has the stage's values in use: its place is free
    fetch();
    if (post) {
      SVA_EACH(i) {
        const float4 w = *reinterpret_cast<const float4*>(gw + at.c0 + i * 128);
        h[i] = fma4(w, x[i], h[i] * a.res_scale);
      }
      store_row(a.h_out + row * a.ldho + at.c0, at, h);
      if (pre) sp = normalise(h);
    }
    if (pre) {
      SVA_EACH(i) {
        const float4 w = *reinterpret_cast<const float4*>(ws + at.c0 + i * 128);
        const float4 z = *reinterpret_cast<const float4*>(sh + at.c0 + i * 128);
        h[i] = fma4(h[i], w, z);
      }
      store_row(static_cast<T*>(a.u) + row * a.ldu + at.c0, at, h);
    }
    if (a.stats != nullptr && tg == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(so.x, so.y, sp.x, sp.y);
  }
}

template <typename T, int NQ, int MAXT>
__global__ void __launch_bounds__(MAXT)
    norm_bwd_kernel(const __grid_constant__ sva_block_norm_args a,
                    const __grid_constant__ sva_block_norm_grads gr, RowRuns rr, float* partial,
                    int* done, int* status) {
  extern __shared__ __align__(16) char dyn[];
  GroupSums* gsums = reinterpret_cast<GroupSums*>(dyn);
  if (blockIdx.x == 0) {  // words that the host and the sums' kernel read later
    if (threadIdx.x < SVA_STATUS_BYTES / 4) status[threadIdx.x] = 0;
    if (partial != nullptr)
      for (int i = threadIdx.x; i < (a.D + 31) / 32; i += blockDim.x) done[i] = 0;
  }
  const int G = 32 * rr.W;
  const int g = threadIdx.x / G;
  const int tg = static_cast<int>(threadIdx.x) - g * G;
  const Place<NQ> at(tg, a.D);
  const int b = static_cast<int>(blockIdx.x) / rr.units, ub = static_cast<int>(blockIdx.x) % rr.units;
  const bool post = a.o != nullptr, pre = a.u != nullptr, upstream = gr.dh_out != nullptr;
  const bool layer = a.kind == SVA_NORM_LAYER;
  Group grp{&gsums[g], rr.W, tg >> 5, 1 + g, 0};
  grp.init(tg);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int width = NQ * G * 4;
  float* gw = reinterpret_cast<float*>(gsums + rr.groups);
  float* ws = gw + width;
  // a stage: dh_out, h', du, o, those that the call has
  const int f_bytes = width * 4, t_bytes = width * static_cast<int>(sizeof(T));
  const int at_h = upstream ? f_bytes : 0, at_du = at_h + (pre ? f_bytes : 0),
            at_o = at_du + (pre ? t_bytes : 0), stage_bytes = at_o + (post ? t_bytes : 0);
  char* ring = reinterpret_cast<char*>(ws + width) + g * rr.stages * stage_bytes;
  const int64_t ldhs = post ? a.ldho : a.ldh;
  const float* hsrc = post ? a.h_out : a.h;
  const int base = b * a.N;  // rows are numbered over all batches; addresses are made of the
  uint32_t t = base + ub * rr.groups + g;  // number each time, which costs less than six pointers kept
  const uint32_t end = base + a.N, step = rr.units * rr.groups;
  uint32_t tf = t;
  int sf = 0;
  auto fetch = [&]() {
    if (tf < end) {
      char* st = ring + sf * stage_bytes;
      const int64_t row = tf;
      if (upstream) stage_row(st, gr.dh_out + row * gr.lddho, at);
      if (pre) {
        stage_row(st + at_h, hsrc + row * ldhs, at);
        stage_row(st + at_du, static_cast<const T*>(gr.du) + row * gr.lddu, at);
      }
      if (post) stage_row(st + at_o, static_cast<const T*>(a.o) + row * a.ldo, at);
    }
    copy_commit();
    tf += step;
    sf = sf + 1 == rr.stages ? 0 : sf + 1;
  };
  for (int s = 0; s < rr.stages; ++s) fetch();
  load_factors<T, NQ>(a, b, width, gw, ws, nullptr);
  __syncthreads();
  float4 sum_du[NQ], sum_dux[NQ], sum_do[NQ];
  SVA_EACH(i) sum_du[i] = sum_dux[i] = sum_do[i] = all4(0.f);
  const float4* stats = reinterpret_cast<const float4*>(a.stats);
  float4 st_next = t < end ? stats[t] : all4(0.f);
  for (int st = 0; t < end; t += step) {
    const int64_t row = t;
    const float4 st4 = st_next;
    if (t + step < end) st_next = stats[t + step];
    float4 dh[NQ], y[NQ];
    copy_wait(rr.stages);
    __syncwarp();
    const char* stage = ring + st * stage_bytes;
    st = st + 1 == rr.stages ? 0 : st + 1;
    // read late, so that fewer values are in registers at once
    auto load_dh = [&]() {
      if (upstream) {
        staged<float, NQ>(stage, at, dh);
      } else {
        SVA_EACH(i) dh[i] = all4(0.f);
      }
    };
    if (!pre) load_dh();
    if (pre) {
      float4 x[NQ];
      staged<float, NQ>(stage + at_h, at, x);
      staged<T, NQ>(stage + at_du, at, y);
      Acc sx, sy;
      SVA_EACH(i) {
        const float4 w = *reinterpret_cast<const float4*>(ws + at.c0 + i * 128);
        x[i] = (x[i] - st4.z) * st4.w;
        sum_du[i] = sum_du[i] + y[i];
        sum_dux[i] = fma4(y[i], x[i], sum_dux[i]);
        y[i] = y[i] * w;  // zero behind the row's end
        sx.dot(y[i], x[i]);
        sy.add(y[i]);
      }
      const float2 s = layer ? grp.sum(make_float2(sx.total(), sy.total()))
                             : make_float2(grp.sum(sx.total()), 0.f);
      const float m1 = -s.x * inv_d, m0 = s.y * inv_d;
      load_dh();
      SVA_EACH(i) dh[i] = fma4(st4.w, fma4(m1, x[i], y[i] - m0), dh[i]);
    }
    if (post) {
      float4 on[NQ];
      staged<T, NQ>(stage + at_o, at, on);
      Acc sx, sy;
      SVA_EACH(i) {
        const float4 w = *reinterpret_cast<const float4*>(gw + at.c0 + i * 128);
        on[i] = (on[i] - st4.x) * st4.y;
        y[i] = dh[i] * w;
        if (!at.full) y[i] = keep4(y[i], at.left(i));
        sx.dot(y[i], on[i]);
        sy.add(y[i]);
      }
      const float2 s = layer ? grp.sum(make_float2(sx.total(), sy.total()))
                             : make_float2(grp.sum(sx.total()), 0.f);
      const float m1 = -s.x * inv_d, m0 = s.y * inv_d;
      SVA_EACH(i) {
        sum_do[i] = fma4(dh[i], on[i], sum_do[i]);
        on[i] = fma4(m1, on[i], y[i] - m0) * st4.y;
        dh[i] = dh[i] * a.res_scale;
      }
      store_row(static_cast<T*>(gr.d_o) + row * gr.lddo + at.c0, at, on);
    }
    __syncwarp();  // the warp has the stage's values in use: its place is free
    fetch();
    store_row(gr.dh + row * gr.lddh + at.c0, at, dh);
  }
  if (partial == nullptr) return;
  // the groups' sums join in the ring (no copy is in flight: the last wait left
  // only empty ones), in the order of the groups, and leave as one part
  float* join = ws + width;
  for (int turn = 0; turn < rr.groups; ++turn) {
    __syncthreads();
    if (turn != g) continue;
    SVA_EACH(i) {
      float4* p = reinterpret_cast<float4*>(join + at.c0 + i * 128);
      const int w4 = width / 4;
      p[0] = turn == 0 ? sum_du[i] : p[0] + sum_du[i];
      p[w4] = turn == 0 ? sum_dux[i] : p[w4] + sum_dux[i];
      p[2 * w4] = turn == 0 ? sum_do[i] : p[2 * w4] + sum_do[i];
    }
  }
  __syncthreads();
  const int ldp = (a.D + 3) / 4 * 4;  // rows of partial are whole quads
  float* p = partial + static_cast<int64_t>(blockIdx.x) * kMaxSums * ldp;
  for (int c = threadIdx.x * 4; c < ldp; c += blockDim.x * 4)
#pragma unroll
    for (int k = 0; k < kMaxSums; ++k)
      if (k < 2 ? pre : post)
        *reinterpret_cast<float4*>(p + k * ldp + c) = *reinterpret_cast<const float4*>(join + k * width + c);
}

// The CTAs' column sums to the gradients. A block takes 32 columns of one batch,
// its units spread over 32 rows of threads and joined in a fixed order; the last
// block of a column range to finish adds up the batches, in their order, whichever
// block it is. Launched ahead of the backward kernel's end, it waits for it here.
constexpr int kSumRows = 32;

// 256 threads: 8 quads x 32 rows; the sum over the rows, in threads 0 to 7
__device__ __forceinline__ float4 rows_sum(float4 v, float4 (*red)[8]) {
#pragma unroll
  for (int o = 8; o <= 16; o <<= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  const int lane = lane_id();
  __syncthreads();
  if (lane < 8) red[warp_id()][lane] = v;
  __syncthreads();
  v = all4(0.f);
  if (threadIdx.x < 8)
#pragma unroll
    for (int w = 0; w < 8; ++w) v = v + red[w][threadIdx.x];
  return v;
}

template <typename T>
__global__ void __launch_bounds__(256)
    norm_sums_kernel(const __grid_constant__ sva_block_norm_args a,
                     const __grid_constant__ sva_block_norm_grads gr, int units,
                     const float* partial, float* wsum, int* done) {
  __shared__ float4 red[8][8];
  __shared__ int last;
  const int q = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + q * 4, b = blockIdx.y;
  const int ldp = (a.D + 3) / 4 * 4;
  const bool ok = c < a.D, first = threadIdx.x < 8 && ok;
  const bool post = a.o != nullptr, pre = a.u != nullptr;
  const int n = a.D - c;
  // the factors of the sums, read while the backward kernel still runs
  float4 wp = all4(1.f), wq = wp, sc = wp, gt = wp;
  if (first) {
    if (a.w_pre != nullptr) wp = load4n(static_cast<const T*>(a.w_pre) + c, n);
    if (a.w_post != nullptr) wq = load4n(static_cast<const T*>(a.w_post) + c, n);
    if (a.scale != nullptr) sc = sc + load4n(static_cast<const T*>(a.scale) + b * a.ldscale + c, n);
    if (a.gate != nullptr) gt = load4n(static_cast<const T*>(a.gate) + b * a.ldgate + c, n);
  }
  cudaGridDependencySynchronize();
  float4 s[kMaxSums] = {all4(0.f), all4(0.f), all4(0.f)};
  if (ok) {
    for (int u = ty; u < units; u += kSumRows) {
      const float* p = partial + (static_cast<int64_t>(b) * units + u) * kMaxSums * ldp + c;
#pragma unroll
      for (int k = 0; k < kMaxSums; ++k)
        if (k < 2 ? pre : post) s[k] = s[k] + *reinterpret_cast<const float4*>(p + k * ldp);
    }
  }
#pragma unroll
  for (int k = 0; k < kMaxSums; ++k) s[k] = rows_sum(s[k], red);
  auto put = [&](float* p, float4 v) {  // rows of D floats need not be 16-byte aligned
    const float f[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < min(4, n); ++i) p[i] = f[i];
  };
  const int64_t at = static_cast<int64_t>(b) * a.D + c;
  if (first) {
    if (gr.dshift != nullptr) put(gr.dshift + at, s[0]);
    if (gr.dscale != nullptr) put(gr.dscale + at, s[1] * wp);
    if (gr.dgate != nullptr) put(gr.dgate + at, s[2] * wq);
  }
  if (gr.dw_pre == nullptr && gr.dw_post == nullptr) return;
  if (first) {
    float4* w = reinterpret_cast<float4*>(wsum + static_cast<int64_t>(b) * 2 * ldp + c);
    w[0] = s[1] * sc;
    w[ldp / 4] = s[2] * gt;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(done + blockIdx.x, 1) == a.B - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  s[0] = s[1] = all4(0.f);
  if (ok) {
    for (int bb = ty; bb < a.B; bb += kSumRows) {
      const float* p = wsum + static_cast<int64_t>(bb) * 2 * ldp + c;
      s[0] = s[0] + __ldcg(reinterpret_cast<const float4*>(p));
      s[1] = s[1] + __ldcg(reinterpret_cast<const float4*>(p + ldp));
    }
  }
  s[0] = rows_sum(s[0], red);
  s[1] = rows_sum(s[1], red);
  if (first) {
    if (gr.dw_pre != nullptr) put(gr.dw_pre + c, s[0]);
    if (gr.dw_post != nullptr) put(gr.dw_post + c, s[1]);
  }
}

constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024;  // the latter per CTA

int quads(int D) { return D <= 128 ? 1 : D <= 256 ? 2 : 4; }

// Launch shape. A CTA holds `groups` groups (8 warps where a row needs fewer),
// each with its factors once per CTA and `stages` rows a group. CTAs an SM: what
// registers (at most `warps` warps) and two stages a group leave. A batch is cut
// into units so that few CTAs are left over in the last wave: a wave costs its
// rows and about two more for the factors and the sums.
RowRuns row_runs(int B, int N, int D, int cta_warps, int warps, int factors, int bytes_per_value) {
  RowRuns r;
  const int nq = quads(D);
  r.W = (D + 128 * nq - 1) / (128 * nq);
  r.groups = std::max(1, cta_warps / r.W);
  const int width = nq * 128 * r.W;
  const int fixed = width * 4 * factors + r.groups * static_cast<int>(sizeof(GroupSums)), stage = r.groups * width * bytes_per_value;
  int per_sm = std::max(1, warps / (r.W * r.groups));
  auto room = [&](int n) { return kSmemPerSm / n - kSmemReserved - fixed; };
  while (per_sm > 1 && 2 * stage > room(per_sm)) --per_sm;
  r.stages = std::max(1, std::min(kMaxStages, room(per_sm) / stage));
  const int64_t slots = static_cast<int64_t>(std::max(1, device_sm_count())) * per_sm;
  int64_t best = INT64_MAX, rows = 1;
  for (int64_t w = 1; w <= 4; ++w) {
    const int64_t most = (static_cast<int64_t>(N) + r.groups - 1) / r.groups;
    const int64_t u = std::max<int64_t>(1, std::min(most, w * slots / B));
    const int64_t per_group = (most + u - 1) / u;
    const int64_t cost = (u * B + slots - 1) / slots * (per_group + 2);
    if (cost < best) {
      best = cost;
      rows = per_group;
      r.units = static_cast<int>(u);
    }
  }
  r.total = static_cast<int64_t>(B) * r.units;
  r.stages = static_cast<int>(std::min<int64_t>(r.stages, rows));
  return r;
}

// values a thread copies, bytes each: h and o; dh_out, h', du and o
RowRuns fwd_runs(const sva_block_norm_args& a) {
  const int e = a.dtype == SVA_BF16 ? 2 : 4;
  return row_runs(a.B, a.N, a.D, 8, 24, 3, 4 + (a.o != nullptr ? e : 0));
}
// by sizes and type alone, whichever of the arrays a call has
RowRuns bwd_runs(int B, int N, int D, int e) { return row_runs(B, N, D, 12, 12, 2, 8 + 2 * e); }

template <auto K>
cudaError_t launch(const RowRuns& rr, int smem, cudaStream_t s, void** args) {
  const cudaError_t e = allow_max_smem<K>();
  if (e != cudaSuccess) return e;
  return cudaLaunchKernel(reinterpret_cast<const void*>(K), dim3(static_cast<unsigned>(rr.total)),
                          dim3(static_cast<unsigned>(32 * rr.W * rr.groups)), args,
                          static_cast<size_t>(smem), s);
}

template <typename T>
cudaError_t launch_fwd(sva_block_norm_args a, cudaStream_t s) {
  RowRuns rr = fwd_runs(a);
  const int nq = quads(a.D), width = nq * 128 * rr.W;
  const int bytes = 4 + (a.o != nullptr ? static_cast<int>(sizeof(T)) : 0);
  const int smem = rr.groups * static_cast<int>(sizeof(GroupSums)) + width * 12 +
                   rr.groups * rr.stages * width * bytes;
  void* args[] = {&a, &rr};
  if (nq == 1) return launch<norm_fwd_kernel<T, 1, 256>>(rr, smem, s, args);
  if (nq == 2) return launch<norm_fwd_kernel<T, 2, 256>>(rr, smem, s, args);
  if (rr.W <= 8) return launch<norm_fwd_kernel<T, 4, 256>>(rr, smem, s, args);
  return launch<norm_fwd_kernel<T, 4, 512>>(rr, smem, s, args);
}

// Scratch of a backward call: the CTAs' column sums, the batches' weighted sums,
// and a counter per 32 columns.
struct Scratch {
  float *partial, *wsum;
  int* done;
  size_t bytes;
};
Scratch scratch_of(int B, int N, int D, char* base) {
  const size_t ldp = static_cast<size_t>(D + 3) / 4 * 4;
  const int64_t ctas = std::max(bwd_runs(B, N, D, 2).total, bwd_runs(B, N, D, 4).total);
  const size_t at_w = static_cast<size_t>(ctas) * kMaxSums * ldp * sizeof(float);
  const size_t at_done = at_w + static_cast<size_t>(B) * 2 * ldp * sizeof(float);
  return {reinterpret_cast<float*>(base), reinterpret_cast<float*>(base + at_w),
          reinterpret_cast<int*>(base + at_done), at_done + static_cast<size_t>(D + 31) / 32 * sizeof(int)};
}

template <typename T>
cudaError_t launch_bwd(sva_block_norm_args a, sva_block_norm_grads g, bool sums, int* status,
                       char* scratch, cudaStream_t s) {
  const int e = static_cast<int>(sizeof(T));
  RowRuns rr = bwd_runs(a.B, a.N, a.D, e);
  const int nq = quads(a.D), width = nq * 128 * rr.W;
  const int bytes = (g.dh_out != nullptr ? 4 : 0) + (a.u != nullptr ? 4 + e : 0) +
                    (a.o != nullptr ? e : 0);
  // the ring also holds the groups' joined sums at the end
  const int smem = rr.groups * static_cast<int>(sizeof(GroupSums)) + width * 8 +
                   std::max(rr.groups * rr.stages * width * bytes, width * 4 * kMaxSums);
  const Scratch sc = scratch_of(a.B, a.N, a.D, scratch);
  float* partial = sums ? sc.partial : nullptr;
  int* done = sc.done;
  void* args[] = {&a, &g, &rr, &partial, &done, &status};
  cudaError_t err;
  if (nq == 1)
    err = launch<norm_bwd_kernel<T, 1, 384>>(rr, smem, s, args);
  else if (nq == 2)
    err = launch<norm_bwd_kernel<T, 2, 384>>(rr, smem, s, args);
  else if (rr.W <= 12)
    err = launch<norm_bwd_kernel<T, 4, 384>>(rr, smem, s, args);
  else
    err = launch<norm_bwd_kernel<T, 4, 512>>(rr, smem, s, args);
  if (err != cudaSuccess || !sums) return err;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.D + 31) / 32), static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_sums_kernel<T>, a, g, rr.units,
                            static_cast<const float*>(partial), sc.wsum, done);
}

}  // namespace

size_t block_norm_scratch_bytes(int B, int N, int D) { return scratch_of(B, N, D, nullptr).bytes; }

cudaError_t block_norm_fwd(const sva_block_norm_args& a, cudaStream_t s) {
  return a.dtype == SVA_BF16 ? launch_fwd<__nv_bfloat16>(a, s) : launch_fwd<float>(a, s);
}

cudaError_t block_norm_bwd(const sva_block_norm_args& a, const sva_block_norm_grads& g, int* status,
                           void* scratch, cudaStream_t s) {
  const bool sums = g.dw_post != nullptr || g.dgate != nullptr || g.dw_pre != nullptr ||
                    g.dscale != nullptr || g.dshift != nullptr;
  char* base = static_cast<char*>(scratch);
  return a.dtype == SVA_BF16 ? launch_bwd<__nv_bfloat16>(a, g, sums, status, base, s)
                             : launch_bwd<float>(a, g, sums, status, base, s);
}

}  // namespace sva
