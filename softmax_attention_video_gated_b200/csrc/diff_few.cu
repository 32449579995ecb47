// diff_few.cu -- the differential softmax anchor for a handful of queries (single
// tokens against a long sequence of keys), forward and backward, both types, on the
// CUDA cores.
//
// The work is one read of K and V: a key's row is 16 bytes a lane (LPK lanes a
// key, the first half of them map 1's columns), so a warp takes 32 / LPK keys at
// a time and UNROLL of them a step, all loads ahead of the arithmetic. A lane's
// columns of V belong to both maps; the half rows swap their weights by shuffle.
// One online softmax per map and subgroup. The keys of a (batch, head) are cut
// over the CTAs of a cluster, which join their sums in rank 0 over distributed
// shared memory: one launch, no scratch, one order of summation.
// 8,190 keys, 16 heads of 128, two batches, one query each (134 MB, 20.5 us at the
// measured copy rate): 30 us with a cold L2, 4.5 TB/s, in one launch; the tile kernel,
// one valid row in 128, and its merge took 51 us. From five queries on the tile kernel
// is taken: a lane here holds both maps' outputs of every row.
// Backward the same read of K and V makes all of it: a key's dK and dV rows are its
// own, dQ is summed like the forward outputs. One query each of 4 batches against 19,000
// keys, 16 heads, bf16 (1.24 GB): 228 us with the preparation, where a tile of queries
// took 917, all keys one after another; fp32 485 us against 4,590.
#include <algorithm>

#include "diff_common.cuh"

namespace sva {
namespace {

constexpr int WARPS = 8;

template <typename T>
__device__ __forceinline__ void widen16(uint4 x, float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void widen16<float>(uint4 x, float (&f)[4]) {
  f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y);
  f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
}
template <>
__device__ __forceinline__ void widen16<__nv_bfloat16>(uint4 x, float (&f)[8]) {
  f[0] = bf16lo_to_f32(x.x); f[1] = bf16hi_to_f32(x.x);
  f[2] = bf16lo_to_f32(x.y); f[3] = bf16hi_to_f32(x.y);
  f[4] = bf16lo_to_f32(x.z); f[5] = bf16hi_to_f32(x.z);
  f[6] = bf16lo_to_f32(x.w); f[7] = bf16hi_to_f32(x.w);
}

// keys a subgroup has in flight, K and V
constexpr int few_unroll(int rows) { return rows == 1 ? 8 : 4; }

template <int D, int R>
struct FewSmem {
  // a subgroup's and then the CTA's state: per row and map the output (unnormalised),
  // maximum (log2 units) and sum
  static constexpr int STATE = R * 2 * (D + 2);
};

template <typename T, int D, int R>
__global__ void __launch_bounds__(32 * WARPS)
    diff_few_kernel(const __grid_constant__ sva_diff_args a, float scale_log2, int cluster,
                    int* status) {
  constexpr int UNROLL = few_unroll(R);
  if (blockIdx.x == 0 && threadIdx.x < SVA_STATUS_BYTES / 4) status[threadIdx.x] = 0;
  constexpr int V = 16 / sizeof(T);       // values a lane
  constexpr int LPK = D / V;              // lanes a key
  constexpr int SUBS = WARPS * 32 / LPK;  // subgroups of the CTA, a key each
  constexpr int STATE = FewSmem<D, R>::STATE;
  extern __shared__ __align__(16) float sm[];  // [SUBS][STATE], then the CTA's [STATE]
  float* mine = sm + SUBS * STATE;
  const int bh = static_cast<int>(blockIdx.x) / cluster, rank = static_cast<int>(blockIdx.x) % cluster;
  const int h = bh % a.H, b = bh / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int k0 = static_cast<int>(static_cast<int64_t>(valid) * rank / cluster);
  const int k1 = static_cast<int>(static_cast<int64_t>(valid) * (rank + 1) / cluster);
  const int lane = lane_id(), in_key = lane % LPK, sub = threadIdx.x / LPK;
  const bool second = in_key >= LPK / 2;
  const int col = h * D + in_key * V;
  float q[R][V], o1[R][V], o2[R][V], m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < a.N)
      x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                          (static_cast<int64_t>(b) * a.N + r) * a.ldq + col);
    widen16<T>(x, q[r]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      q[r][e] *= scale_log2;
      o1[r][e] = o2[r][e] = 0.f;
    }
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  const T* kp = static_cast<const T*>(a.k) + static_cast<int64_t>(b) * Nk * a.ldk + col;
  const T* vp = static_cast<const T*>(a.v) + static_cast<int64_t>(b) * Nk * a.ldv + col;
  for (int base = k0 + sub; base - sub < k1; base += SUBS * UNROLL) {
    uint4 kx[UNROLL], vx[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int key = base + u * SUBS;
      kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
      if (key < k1) {
        kx[u] = __ldcs(reinterpret_cast<const uint4*>(kp + key * a.ldk));
        vx[u] = __ldcs(reinterpret_cast<const uint4*>(vp + key * a.ldv));
      }
    }
    float s[R][UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float kf[V];
      widen16<T>(kx[u], kf);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r][u] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) s[r][u] = fmaf(q[r][e], kf[e], s[r][u]);
      }
    }
#pragma unroll
    for (int o = LPK / 4; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) s[r][u] += __shfl_xor_sync(0xffffffffu, s[r][u], o);
    float p[R][UNROLL], p2[R][UNROLL];  // weights of the maps 1 and 2
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mx = m[r];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (base + u * SUBS >= k1) s[r][u] = -INFINITY;
        mx = fmaxf(mx, s[r][u]);
      }
      // without a key so far mx is -infinity; 0 in its place keeps the weights zero
      const float at = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f(m[r] - at);
      m[r] = mx;
      l[r] *= f;
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        p[r][u] = exp2f(s[r][u] - at);
        l[r] += p[r][u];
        const float other = __shfl_xor_sync(0xffffffffu, p[r][u], LPK / 2);
        p2[r][u] = second ? p[r][u] : other;
        if (second) p[r][u] = other;
      }
      const float fo = __shfl_xor_sync(0xffffffffu, f, LPK / 2);
      const float f1 = second ? fo : f, f2 = second ? f : fo;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        o1[r][e] *= f1;
        o2[r][e] *= f2;
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float vf[V];
      widen16<T>(vx[u], vf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o1[r][e] = fmaf(p[r][u], vf[e], o1[r][e]);
          o2[r][e] = fmaf(p2[r][u], vf[e], o2[r][e]);
        }
    }
  }
  // subgroup states: [r][map][D] outputs, then [r][map] maxima and sums
  float* st = sm + sub * STATE;
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      *reinterpret_cast<float4*>(st + (r * 2) * D + in_key * V + e) =
          make_float4(o1[r][e], o1[r][e + 1], o1[r][e + 2], o1[r][e + 3]);
      *reinterpret_cast<float4*>(st + (r * 2 + 1) * D + in_key * V + e) =
          make_float4(o2[r][e], o2[r][e + 1], o2[r][e + 2], o2[r][e + 3]);
    }
    if (in_key == 0 || in_key == LPK / 2) {
      st[R * 2 * D + r * 2 + (second ? 1 : 0)] = m[r];
      st[R * 2 * D + R * 2 + r * 2 + (second ? 1 : 0)] = l[r];
    }
  }
  __syncthreads();
  // joins n states, read through `get`, into `out`; one thread per (row, map, column)
  auto join = [&](int n, auto get, float* out) {
    for (int i = threadIdx.x; i < R * 2 * D; i += 32 * WARPS) {
      const int rm = i / D;
      float mx = -INFINITY;
      for (int k = 0; k < n; ++k) mx = fmaxf(mx, get(k, R * 2 * D + rm));
      float o = 0.f, sum = 0.f;
      for (int k = 0; k < n; ++k) {
        const float mk = get(k, R * 2 * D + rm);
        const float w = mk == -INFINITY ? 0.f : exp2f(mk - mx);
        o = fmaf(w, get(k, i), o);
        sum = fmaf(w, get(k, R * 2 * D + R * 2 + rm), sum);
      }
      out[i] = o;
      if (i % D == 0) {
        out[R * 2 * D + rm] = mx;
        out[R * 2 * D + R * 2 + rm] = sum;
      }
    }
  };
  join(SUBS, [&](int k, int i) { return sm[k * STATE + i]; }, mine);
  if (cluster > 1) {
    cluster_sync();
    if (rank == 0)
      join(cluster, [&](int k, int i) { return ld_cluster(mine + i, static_cast<uint32_t>(k)); }, sm);
    cluster_sync();  // the others' shared memory has been read
    if (rank != 0) return;
    mine = sm;
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < R * D / 4; i += 32 * WARPS) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    if (r >= a.N) break;
    const float* ml = mine + R * 2 * D + r * 2;
    const float4 x = *reinterpret_cast<const float4*>(mine + r * 2 * D + c);
    const float4 y = *reinterpret_cast<const float4*>(mine + (r * 2 + 1) * D + c);
    finish4<T>(a, b, h, r, c, x, y, ml[R * 2], ml[R * 2 + 1], lambda_of<T>(a, b, r, h));
    if (c < 8) finish_lse(a, c / 4, b, h, r, ml[c / 4], ml[R * 2 + c / 4]);
  }
}

template <typename T>
__device__ __forceinline__ uint4 narrow16(const float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ uint4 narrow16<float>(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 narrow16<__nv_bfloat16>(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(32 * WARPS)
    diff_few_bwd_kernel(const __grid_constant__ sva_diff_args a, const __grid_constant__ sva_diff_grads g,
                        DiffBwdScratch ws, float scale, int cluster) {
  constexpr int UNROLL = few_unroll(R) / 2;
  constexpr int V = 16 / sizeof(T), LPK = D / V, SUBS = WARPS * 32 / LPK;
  extern __shared__ __align__(16) float sm[];  // [SUBS][R * D], then the CTA's [R * D]
  float* mine = sm + SUBS * R * D;
  const int bh = static_cast<int>(blockIdx.x) / cluster, rank = static_cast<int>(blockIdx.x) % cluster;
  const int h = bh % a.H, b = bh / a.H;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  const int valid = key_count(a.key_lens, b, Nk);
  const int k0 = static_cast<int>(static_cast<int64_t>(Nk) * rank / cluster);
  const int k1 = static_cast<int>(static_cast<int64_t>(Nk) * (rank + 1) / cluster);
  const int in_key = lane_id() % LPK, sub = threadIdx.x / LPK;
  const bool second = in_key >= LPK / 2;
  const int col = h * D + in_key * V;
  const float scale_log2 = scale * kLog2e;
  // the rows' queries (in log2 units) and dA, and this lane's map's statistics
  float q[R][V], da[R][V], dq[R][V], nlse[R], nd[R], nl[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    const bool in = r < a.N;
    if (in) {
      const int64_t row = static_cast<int64_t>(b) * a.N + r;
      x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + row * a.ldq + col);
      y = *reinterpret_cast<const uint4*>(static_cast<const T*>(ws.da) + row * a.H * D + col);
    }
    widen16<T>(x, q[r]);
    widen16<T>(y, da[r]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      q[r][e] *= scale_log2;
      dq[r][e] = 0.f;
    }
    const float* st = ws.stats + stat_at(bh, 1, r);  // one tile of 64 holds them
    nlse[r] = in ? st[second ? 64 : 0] : -INFINITY;
    nd[r] = in ? st[second ? 192 : 128] : 0.f;
    nl[r] = second && in ? st[256] : 1.f;
  }
  const int64_t krow0 = static_cast<int64_t>(b) * Nk;
  const T* kp = static_cast<const T*>(a.k) + krow0 * a.ldk + col;
  const T* vp = static_cast<const T*>(a.v) + krow0 * a.ldv + col;
  T* dkp = static_cast<T*>(g.dk) + krow0 * g.lddk + col;
  T* dvp = static_cast<T*>(g.dv) + krow0 * g.lddv + col;
  for (int base = k0 + sub; base - sub < k1; base += SUBS * UNROLL) {
    uint4 kx[UNROLL], vx[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int key = base + u * SUBS;
      kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
      if (key < k1 && key < valid) {  // what lies behind counts for nothing
        kx[u] = __ldcs(reinterpret_cast<const uint4*>(kp + key * a.ldk));
        vx[u] = __ldcs(reinterpret_cast<const uint4*>(vp + key * a.ldv));
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int key = base + u * SUBS;
      float kf[V], vf[V], s[R], dp[R];
      widen16<T>(kx[u], kf);
      widen16<T>(vx[u], vf);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = dp[r] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[r] = fmaf(q[r][e], kf[e], s[r]);
          dp[r] = fmaf(da[r][e], vf[e], dp[r]);
        }
      }
#pragma unroll
      for (int o = LPK / 4; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
          dp[r] += __shfl_xor_sync(0xffffffffu, dp[r], o);
        }
      float dk[V], dv[V];
#pragma unroll
      for (int e = 0; e < V; ++e) dk[e] = dv[e] = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        dp[r] += __shfl_xor_sync(0xffffffffu, dp[r], LPK / 2);  // over all columns of V
        // this map's weight: P_1, or -lambda P_2
        const float p = key < valid ? nl[r] * exp2f(s[r] + nlse[r]) : 0.f;
        const float w = p + __shfl_xor_sync(0xffffffffu, p, LPK / 2);
        // q is in log2 units
        const float ds = key < valid ? p * (dp[r] + nd[r]) : 0.f, dsq = ds * 0.6931471805599453f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dk[e] = fmaf(dsq, q[r][e], dk[e]);
          dv[e] = fmaf(w, da[r][e], dv[e]);
          dq[r][e] = fmaf(ds, kf[e], dq[r][e]);
        }
      }
      if (key < k1) {
        // zeros behind the last key, also where q or dA is not a number
        uint4* dko = reinterpret_cast<uint4*>(dkp + key * g.lddk);
        uint4* dvo = reinterpret_cast<uint4*>(dvp + key * g.lddv);
        const bool in = key < valid;
        *dko = in ? narrow16<T>(dk) : make_uint4(0, 0, 0, 0);
        *dvo = in ? narrow16<T>(dv) : make_uint4(0, 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < V; ++e) sm[(sub * R + r) * D + in_key * V + e] = dq[r][e];
  __syncthreads();
  for (int i = threadIdx.x; i < R * D; i += 32 * WARPS) {
    float x = 0.f;
    for (int k = 0; k < SUBS; ++k) x += sm[k * R * D + i];
    mine[i] = x;
  }
  if (cluster > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank == 0)
    for (int i = threadIdx.x; i < R * D; i += 32 * WARPS) {
      const int r = i / D;
      if (r >= a.N) break;
      float x = 0.f;
      for (int k = 0; k < cluster; ++k) x += cluster > 1 ? ld_cluster(mine + i, static_cast<uint32_t>(k)) : mine[i];
      from_f32(static_cast<T*>(g.dq) + (static_cast<int64_t>(b) * a.N + r) * g.lddq + h * D + i % D, scale * x);
    }
  if (cluster > 1) cluster_sync();  // the others' shared memory has been read
}

template <typename T, int D, int R>
cudaError_t launch(const sva_diff_args& a, int* status, cudaStream_t s) {
  constexpr int SUBS = WARPS * 32 / (D * static_cast<int>(sizeof(T)) / 16);
  constexpr size_t smem = (SUBS + 1) * static_cast<size_t>(FewSmem<D, R>::STATE) * sizeof(float);
  cudaError_t e = allow_max_smem<diff_few_kernel<T, D, R>>();
  if (e != cudaSuccess) return e;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  int cluster = 1;  // two steps of every subgroup at least
  while (cluster < 8 && Nk > cluster * SUBS * few_unroll(R) * 2) cluster *= 2;
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  return launch_clusters(diff_few_kernel<T, D, R>, static_cast<unsigned>(a.B * a.H * cluster), 32 * WARPS,
                         smem, cluster, s, a, scale * kLog2e, cluster, status);
}

template <typename T, int D, int R>
cudaError_t launch_bwd(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  constexpr int SUBS = WARPS * 32 / (D * static_cast<int>(sizeof(T)) / 16);
  const cudaError_t e = allow_max_smem<diff_few_bwd_kernel<T, D, R>>();
  if (e != cudaSuccess) return e;
  const int Nk = a.n_keys > 0 ? a.n_keys : a.N;
  int cluster = 1;
  while (cluster < 8 && Nk > cluster * SUBS * few_unroll(R)) cluster *= 2;
  const float scale = a.scale != 0.f ? a.scale : 1.0f / sqrtf(static_cast<float>(D / 2));
  return launch_clusters(diff_few_bwd_kernel<T, D, R>, static_cast<unsigned>(a.B * a.H * cluster), 32 * WARPS,
                         (SUBS + 1) * static_cast<size_t>(R * D) * sizeof(float), cluster, s, a, g,
                         diff_bwd_scratch(a, scratch), scale, cluster);
}

template <typename T, int D>
cudaError_t bwd_by_rows(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  return a.N == 1   ? launch_bwd<T, D, 1>(a, g, scratch, s)
         : a.N == 2 ? launch_bwd<T, D, 2>(a, g, scratch, s)
                    : launch_bwd<T, D, 4>(a, g, scratch, s);
}

template <typename T, int D>
cudaError_t by_rows(const sva_diff_args& a, int* status, cudaStream_t s) {
  return a.N == 1   ? launch<T, D, 1>(a, status, s)
         : a.N == 2 ? launch<T, D, 2>(a, status, s)
                    : launch<T, D, 4>(a, status, s);
}

}  // namespace

cudaError_t diff_fwd_few(const sva_diff_args& a, int* status, cudaStream_t s) {
  if (a.dtype == SVA_BF16) return by_rows<__nv_bfloat16, 128>(a, status, s);
  return a.d == 64 ? by_rows<float, 64>(a, status, s) : by_rows<float, 128>(a, status, s);
}

cudaError_t diff_bwd_few(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s) {
  if (a.dtype == SVA_BF16) return bwd_by_rows<__nv_bfloat16, 128>(a, g, scratch, s);
  return a.d == 64 ? bwd_by_rows<float, 64>(a, g, scratch, s) : bwd_by_rows<float, 128>(a, g, scratch, s);
}

}  // namespace sva
