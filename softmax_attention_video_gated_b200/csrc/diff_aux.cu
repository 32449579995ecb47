// diff_aux.cu -- around the differential anchor's attention core, for both types:
// the launch plans, the merge of a key split, and the backward pass's
// preparation. All of it is memory traffic.
#include <algorithm>

#include "diff_common.cuh"

namespace sva {
namespace {

// Joins the parts of split units: per map, with M the largest part maximum and
// w_p = 2^(m_p - M), O = sum w_p O_p and l = sum w_p l_p. One warp per query row.
template <typename T>
__global__ void __launch_bounds__(256) diff_merge_kernel(const sva_diff_args a, DiffWork wk,
                                                         int n_split_units) {
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<int64_t>(n_split_units) * wk.rows) return;
  const int su = static_cast<int>(wid / wk.rows), r = static_cast<int>(wid % wk.rows);
  const DiffUnit u = diff_unit(wk, wk.n_full + su * wk.split);
  const int t = u.q0 + r;
  if (t >= a.N) return;
  float4 o[2];
  float mx[2], l[2];
#pragma unroll
  for (int mm = 0; mm < 2; ++mm) {
    // a lane per part (the plan makes 32 at most) for the weights
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < wk.split)
      ml = *reinterpret_cast<const float2*>(diff_part(wk, a.d, su, lane, mm) + wk.rows * a.d + 2 * r);
    mx[mm] = warp_max(ml.x);
    // a part has no keys where its sum is zero; one whose scores are not numbers has a maximum
    // of -infinity too, and must not be lost: a part with keys has a weight above zero
    const float w = ml.y == 0.f ? 0.f : fmaxf(exp2f(ml.x - mx[mm]), 0x1p-126f);
    l[mm] = warp_sum(w * ml.y);
    o[mm] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = 0; p < wk.split; ++p) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (4 * lane < a.d)
        x = *reinterpret_cast<const float4*>(diff_part(wk, a.d, su, p, mm) + r * a.d + 4 * lane);
      // a part without keys has not written its O: whatever is there does not count
      const float wp = __shfl_sync(0xffffffffu, w, p);
      o[mm].x = fmaf(wp, wp != 0.f ? x.x : 0.f, o[mm].x);
      o[mm].y = fmaf(wp, wp != 0.f ? x.y : 0.f, o[mm].y);
      o[mm].z = fmaf(wp, wp != 0.f ? x.z : 0.f, o[mm].z);
      o[mm].w = fmaf(wp, wp != 0.f ? x.w : 0.f, o[mm].w);
    }
  }
  if (4 * lane < a.d)
    finish4<T>(a, u.b, u.h, t, 4 * lane, o[0], o[1], l[0], l[1], lambda_of<T>(a, u.b, t, u.h));
  if (lane == 0) {
    finish_lse(a, 0, u.b, u.h, t, mx[0], l[0]);
    finish_lse(a, 1, u.b, u.h, t, mx[1], l[1]);
  }
}

// the gate's sigmoid s and 1 - s, which keeps its digits where s is next to 1: with e = exp(-|x|)
// one of them is 1 / (1 + e), the other e / (1 + e). bf16 results do not see the last bits of
// a division.
struct Sigmoid {
  float s, rest;
};
template <typename T>
__device__ __forceinline__ Sigmoid prep_sigmoid(float x) {
  const float e = sizeof(T) == 2 ? __expf(-fabsf(x)) : expf(-fabsf(x));
  const float r = sizeof(T) == 2 ? __fdividef(1.0f, 1.0f + e) : 1.0f / (1.0f + e);
  return x >= 0.f ? Sigmoid{r, e * r} : Sigmoid{e * r, r};
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// dA = dout sigmoid(G) (kept in dtype for the products that follow), dG, the row
// sums delta_m = dA . O_m and dlambda = -delta_2. Half a warp a token and head, Q
// quads a lane, so that the sums' shuffles are shared by two tokens; a block's warps
// are eight heads that stand beside each other in memory. The tokens are rounded up
// to whole tiles of 64: those behind the last get a weight of zero. 8,190 tokens of 16
// heads of 128, bf16 (270 MB): 50 us; a warp a token 83 us, bound by its instructions.
// delta_m is made
// of the rounded dA, as dP is, so that dP - delta_m cancels where a map sits on one
// key; dlambda is a result of its own and is made of the unrounded one (for the bf16 tiles
// it goes to scratch, where the gradients' kernel adds what the forward pass's bf16 weights
// left out of O_2).
template <typename T, int Q>
__global__ void __launch_bounds__(256)
    diff_prep_kernel(const __grid_constant__ sva_diff_args a, const __grid_constant__ sva_diff_grads g,
                     DiffBwdScratch ws, int* status) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < SVA_STATUS_BYTES / 4)
    status[threadIdx.x] = 0;  // for the kernel behind
  const int lane = lane_id(), l16 = lane & 15;
  const int h = static_cast<int>(blockIdx.y) * 8 + warp_id(), b = static_cast<int>(blockIdx.z);
  if (h >= a.H) return;
  const int bh = b * a.H + h;
  const int t = static_cast<int>(blockIdx.x) * 2 + (lane >> 4);
  const bool in = t < a.N;
  const int64_t row = static_cast<int64_t>(b) * a.N + (in ? t : 0);  // the rounded-up tokens read one
  const int64_t D = static_cast<int64_t>(a.H) * a.d;
  const int col = h * a.d + 4 * l16;  // quads 64 columns apart
  float4 o1[Q], o2[Q], d[Q], gx[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    o1[i] = load4<float>(a.o1 + row * D + col + 64 * i);
    o2[i] = load4<float>(a.o2 + row * D + col + 64 * i);
    d[i] = load4(static_cast<const T*>(g.dout) + row * g.lddo + col + 64 * i);
    if (a.gate != nullptr) gx[i] = load4(static_cast<const T*>(a.gate) + row * a.ldg + col + 64 * i);
  }
  const float lam = lambda_of<T>(a, b, in ? t : 0, h);
  float lse = -INFINITY;
  if (l16 < 2 && in) lse = a.lse[(static_cast<int64_t>(l16) * a.B * a.H + bh) * a.N + t];
  float dl = 0.f, d1 = 0.f, d2 = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    if (a.gate != nullptr) {
      const Sigmoid sx = prep_sigmoid<T>(gx[i].x), sy = prep_sigmoid<T>(gx[i].y),
                    sz = prep_sigmoid<T>(gx[i].z), sw = prep_sigmoid<T>(gx[i].w);
      const float4 y = make_float4(d[i].x * sx.s, d[i].y * sy.s, d[i].z * sz.s, d[i].w * sw.s);
      if (in)
        store4(static_cast<T*>(g.dgate) + row * g.lddg + col + 64 * i,
               make_float4(y.x * fmaf(-lam, o2[i].x, o1[i].x) * sx.rest,
                           y.y * fmaf(-lam, o2[i].y, o1[i].y) * sy.rest,
                           y.z * fmaf(-lam, o2[i].z, o1[i].z) * sz.rest,
                           y.w * fmaf(-lam, o2[i].w, o1[i].w) * sw.rest));
      d[i] = y;
    }
    dl -= dot4(d[i], o2[i]);
    d[i] = round4(d[i], static_cast<const T*>(nullptr));
    if (in) store4(static_cast<T*>(ws.da) + row * D + col + 64 * i, d[i]);
    d1 += dot4(d[i], o1[i]);
    d2 += dot4(d[i], o2[i]);
  }
  d1 = half_sum(d1);
  d2 = half_sum(d2);
  dl = half_sum(dl);
  if (l16 < kStats) {
    // an empty row's -infinity stays, a rounded-up token has it: their weights come
    // out as 2^-inf = 0
    float v = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    // a sigmoid's lambda is positive and goes into the second map's exponent
    const bool raw = (a.flags & SVA_FLAG_LAMBDA_VALUE) != 0;
    if (l16 == 1 && !raw) v += log2f(lam);
    if (l16 >= 2) v = !in ? 0.f : l16 == 2 ? -d1 : l16 == 3 ? -d2 : raw ? -lam : -1.f;
    ws.stats[stat_at(bh, (a.N + 63) / 64, t) + l16 * 64] = v;
  }
  if (l16 == 0 && in) {
    if ((a.flags & SVA_FLAG_LAMBDA_VALUE) == 0) dl *= lam;
    if (a.ldl != 0 && !diff_dlam_later(a))
      from_f32(static_cast<T*>(g.dlam) + row * g.lddl + h, dl * dlambda_factor<T>(a, b, t, h));
    else
      ws.dlam[static_cast<int64_t>(bh) * a.N + t] = dl;
  }
}

// dlam of a lambda shared by all tokens: one block per head adds the tokens'
template <typename T>
__global__ void __launch_bounds__(1024) diff_dlam_kernel(const __grid_constant__ sva_diff_args a,
                                                         const __grid_constant__ sva_diff_grads g,
                                                         DiffBwdScratch ws) {
  __shared__ float part[32];
  const int h = blockIdx.x;
  float s = 0.f;
  for (int b = 0; b < a.B; ++b) {
    const float* p = ws.dlam + (static_cast<int64_t>(b) * a.H + h) * a.N;
#pragma unroll 8
    for (int t = threadIdx.x; t < a.N; t += 1024) s += p[t];
  }
  s = warp_sum(s);
  if (lane_id() == 0) part[warp_id()] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = warp_sum(part[threadIdx.x]);
  if (threadIdx.x != 0) return;
  from_f32(static_cast<T*>(g.dlam) + h, s * dlambda_factor<T>(a, 0, 0, h));
}

template <typename T>
cudaError_t prepare(const sva_diff_args& a, const sva_diff_grads& g, const DiffBwdScratch& ws,
                    int* status, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.N + 63) / 64 * 32), static_cast<unsigned>((a.H + 7) / 8),
                  static_cast<unsigned>(a.B));
  constexpr bool kHalf = sizeof(T) == 4;  // fp32 heads may be of 64
  if (kHalf && a.d == 64)
    diff_prep_kernel<T, kHalf ? 1 : 2><<<grid, 256, 0, s>>>(a, g, ws, status);
  else
    diff_prep_kernel<T, 2><<<grid, 256, 0, s>>>(a, g, ws, status);
  return cudaGetLastError();
}

}  // namespace

DiffPlan diff_plan(int B, int N, int H, int d, int n_keys, sva_dtype_t dt) {
  DiffPlan p;
  if (N <= kDiffFewRows) return p;  // no tiles, no scratch
  const bool tc = dt == SVA_BF16;
  p.rows = tc ? kDiffTcRows : kDiffF32Rows;
  const int keys = tc ? kDiffTcKeys : diff_f32_keys(d);
  const int Nk = n_keys > 0 ? n_keys : N;
  p.n_qtiles = static_cast<int>((N + static_cast<int64_t>(p.rows) - 1) / p.rows);
  const int64_t nkb = (Nk + static_cast<int64_t>(keys) - 1) / keys;
  const int64_t units = static_cast<int64_t>(p.n_qtiles) * B * H;
  const int64_t slots = static_cast<int64_t>(std::max(1, device_sm_count())) * (tc ? 1 : 2);
  p.n_full = static_cast<int>(units);
  // The last wave's units, cut s ways, take waves(s) x (their key blocks + 2
  // blocks' time for a CTA's start and end), and two more such times for writing
  // the parts and for the merge. Cut them where that saves a fifth of the wave at
  // least.
  const int64_t tail = units % slots;
  int64_t best = nkb + 2;
  const int64_t most = best * 4 / 5;
  for (int64_t sp = 2; tail > 0 && sp <= std::min<int64_t>(nkb, 32); ++sp) {
    const int64_t cost = (tail * sp + slots - 1) / slots * ((nkb + sp - 1) / sp + 2) + 2;
    if (cost < best && cost <= most) {
      best = cost;
      p.split = static_cast<int>(sp);
    }
  }
  // fp32, nothing but that wave: parts that are all resident at once can be a cluster and
  // join in it, in one block's time (1,024 tokens, 4 heads of 64: 47 us and 11 for the
  // merge -> 52; clusters that wait for a second wave lose more than the merge costs).
  // Clusters of eight leave some SMs of a GPC over.
  for (int64_t sp = 2; !tc && units < slots && sp <= std::min<int64_t>(nkb, 8); sp *= 2) {
    const int64_t cost = (nkb + sp - 1) / sp + 2 + 1;
    if (units * sp <= (sp == 8 ? slots * 7 / 8 : slots) && cost < best && cost <= most) {
      best = cost;
      p.split = static_cast<int>(sp);
      p.cluster = true;
    }
  }
  if (p.cluster) {
    p.n_full = 0;
    p.n_split_units = static_cast<int>(units);
    return p;
  }
  if (p.split > 1) {
    p.n_split_units = static_cast<int>(tail);
    p.n_full = static_cast<int>(units - tail);
    p.partial_bytes = static_cast<size_t>(tail) * p.split * 2 * p.rows *
                      (static_cast<size_t>(d) + 2) * sizeof(float);
  }
  return p;
}

cudaError_t diff_merge(const sva_diff_args& a, const DiffPlan& p, void* scratch, cudaStream_t s) {
  if (p.n_split_units == 0 || p.cluster) return cudaSuccess;
  const DiffWork wk = diff_work(p, a.H, scratch);
  const int64_t threads = static_cast<int64_t>(p.n_split_units) * p.rows * 32;
  const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
  if (a.dtype == SVA_BF16)
    diff_merge_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, wk, p.n_split_units);
  else
    diff_merge_kernel<float><<<grid, 256, 0, s>>>(a, wk, p.n_split_units);
  return cudaGetLastError();
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

DiffBwdGrid diff_bwd_grid(const sva_diff_args& a, int rows, int streamed, int ctas_per_sm) {
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int key_tiles = (Nk + rows - 1) / rows, query_tiles = (a.N + rows - 1) / rows;
  DiffBwdGrid r;
  r.keys_first = a.N >= Nk;
  r.first = r.keys_first ? key_tiles : query_tiles;
  r.second = r.keys_first ? query_tiles : key_tiles;
  // four blocks a cut at least
  const int64_t blocks = (std::max(a.N, Nk) + streamed - 1) / streamed;
  const int64_t ctas = static_cast<int64_t>(r.first) * a.B * a.H;
  const int64_t slots = static_cast<int64_t>(std::max(1, device_sm_count())) * ctas_per_sm;
  while (r.cuts < 8 && ctas * r.cuts * 2 <= slots && blocks >= 8 * r.cuts) r.cuts *= 2;
  return r;
}

DiffBwdScratch diff_bwd_scratch(const sva_diff_args& a, void* scratch) {
  const DiffBwdPlan p = diff_bwd_plan(a.B, a.N, a.H, a.d, a.dtype);
  char* base = static_cast<char*>(scratch);
  return {base, reinterpret_cast<float*>(base + p.stats_off),
          reinterpret_cast<float*>(base + p.dlam_off)};
}

cudaError_t diff_bwd(const sva_diff_args& a, const sva_diff_grads& g, int* status, void* scratch,
                     cudaStream_t s) {
  const bool tc = a.dtype == SVA_BF16;
  const DiffBwdScratch ws = diff_bwd_scratch(a, scratch);
  cudaError_t e = tc ? prepare<__nv_bfloat16>(a, g, ws, status, s) : prepare<float>(a, g, ws, status, s);
  if (e != cudaSuccess) return e;
  e = a.N <= kDiffFewRows ? diff_bwd_few(a, g, scratch, s)
      : tc                ? diff_bwd_bf16(a, g, status, scratch, s)
                          : diff_bwd_f32(a, g, scratch, s);
  if (e != cudaSuccess || a.ldl != 0) return e;
  if (tc)
    diff_dlam_kernel<__nv_bfloat16><<<static_cast<unsigned>(a.H), 1024, 0, s>>>(a, g, ws);
  else
    diff_dlam_kernel<float><<<static_cast<unsigned>(a.H), 1024, 0, s>>>(a, g, ws);
  return cudaGetLastError();
}

}  // namespace sva
