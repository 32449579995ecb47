// internal.h -- host-side interface between the C ABI layer and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/sva.h"

namespace sva {

// Launch bracketing for the stack's optional per-launch CUDA-event profile.
struct Prof {
  cudaEvent_t* events = nullptr;  // 2 * capacity
  int capacity = 0;
  int* kinds = nullptr;           // host, capacity
  int count = 0;
  int launches = 0;  // kernels launched (a scope may launch more than one)
  int cur_kind = SVA_KERNEL_OTHER;
  void before(cudaStream_t s, int kind) {
    cur_kind = kind;
    if (events != nullptr && count < capacity) cudaEventRecord(events[2 * count], s);
  }
  void after(cudaStream_t s) {
    if (events != nullptr && count < capacity) {
      cudaEventRecord(events[2 * count + 1], s);
      if (kinds != nullptr) kinds[count] = cur_kind;
    }
    ++count;
    ++launches;
  }
  void extra_launch() { ++launches; }  // a second kernel inside one scope
};

struct ProfScope {
  Prof* p;
  cudaStream_t s;
  ProfScope(Prof* p_, cudaStream_t s_, int kind) : p(p_), s(s_) {
    if (p) p->before(s, kind);
  }
  ~ProfScope() {
    if (p) p->after(s);
  }
};

// ---------------------------------------------------------------- utilities
// Records the CUDA error's text for sva_last_cuda_error and returns SVA_ERR_CUDA.
sva_status_t cuda_fail(cudaError_t e);
// Host-side validation of an attention call (null and misaligned pointers,
// row strides, sizes, eps / scale, supported head sizes). need_kv: k, v (and
// the write gate) are read; need_qgo: q, gate, out (and the residual) are used.
sva_status_t check_attn(const sva_attn_args* a, bool linear, bool need_kv = true,
                        bool need_qgo = true);
int device_sm_count();
int device_index();
bool encode_tmap(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                 const uint64_t* dims, const uint64_t* strides_bytes /* rank-1 */,
                 const uint32_t* box, CUtensorMapSwizzle swizzle);

// Lets kernel K have as much shared memory as a CTA can take, once per device.
constexpr int kMaxSmem = 227 * 1024;
template <auto K>
cudaError_t allow_max_smem() {
  static std::atomic<bool> done[64];
  const int d = device_index();
  if (d >= 0 && d < 64 && done[d].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess && d >= 0 && d < 64) done[d].store(true, std::memory_order_relaxed);
  return e;
}

// One launch with clusters of `cluster` CTAs (1: without).
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem, int cluster,
                            cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

constexpr size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------- projections
enum GemmEpi { EPI_STORE = 0, EPI_RESIDUAL = 1 };

struct GemmArgs {
  const void* a = nullptr;  int64_t lda = 0;   // [M, K]
  const void* b = nullptr;  int64_t ldb = 0;   // [N, K]
  // optional second weight: output columns n >= n_split take row n - n_split
  // of b2 ([N - n_split, K], row stride ldb) instead of row n of b; n_split is
  // a multiple of 256 (the tile width of the tensor-core path)
  const void* b2 = nullptr; int64_t n_split = 0;
  int64_t M = 0, N = 0, K = 0;
  int epi = EPI_STORE;
  void* c = nullptr;        int64_t ldc = 0;   // EPI_STORE: [M, N] output
  int relu_cols = 0;
  float* h = nullptr;       int64_t ldh = 0;   // EPI_RESIDUAL: fp32 stream
  void* h_copy = nullptr;   int64_t ldhc = 0;  // EPI_RESIDUAL: optional copy
  // EPI_RESIDUAL, bf16: 0 = the copy is rounded to nearest; otherwise it is
  // rounded without bias (pack_bf16x2_unbiased), the random bits hashed from
  // this seed, the row and the column pair (deterministic)
  uint32_t copy_dither = 0;
  int* status = nullptr;
};

cudaError_t gemm_bf16(const GemmArgs& g, cudaStream_t s);
cudaError_t gemm_f32(const GemmArgs& g, cudaStream_t s);
cudaError_t transpose_2d(const void* src, void* dst, int64_t rows, int64_t cols, sva_dtype_t dt,
                         cudaStream_t s);  // dst[c][r] = src[r][c]

// ---------------------------------------------------------------- linear attention
// Scratch of one linear-attention call (offsets from the scratch base):
// fp32 per-chunk partial states, then (fp32 path only) the reduced state.
struct LinearPlan {
  int tiles_per_chunk = 0;  // 128-token tiles per state chunk (bf16) / tokens per chunk (f32)
  int n_chunks = 0;
  size_t partial_off = 0, state_off = 0, total = 0;
};
LinearPlan linear_plan(int B, int N, int H, int d, sva_dtype_t dt);
// Gated linear attention. With state_out, only the state pass runs and the
// fp32 state [B*H][d*d + d] (S row-major d_k x d_v, then z) is written there;
// with state_in, the state pass is skipped and the read-out uses that state;
// with neither, the fused layer.
cudaError_t linear_bf16(const sva_attn_args& a, int* status, void* scratch, cudaStream_t s,
                        Prof* prof, float* state_out = nullptr, const float* state_in = nullptr);
cudaError_t linear_f32(const sva_attn_args& a, int* status, void* scratch, cudaStream_t s,
                       Prof* prof, float* state_out = nullptr, const float* state_in = nullptr);

// ---------------------------------------------------------------- softmax anchor
// Anchor launch plan: units of 512 queries (one CTA pair each), key blocks,
// and the split of the last wave's units along the keys (partial_bytes of
// scratch for their parts).
struct AnchorPlan {
  int n_qunits = 0, nkv_total = 0, n_full = 0, n_split_units = 0, split = 0;
  size_t partial_bytes = 0;
};
AnchorPlan anchor_plan(int B, int N, int H, int n_keys);
cudaError_t anchor_bf16(const sva_attn_args& a, int* status, void* scratch, cudaStream_t s,
                        Prof* prof = nullptr);
cudaError_t anchor_f32(const sva_attn_args& a, int* status, cudaStream_t s);

// ---------------------------------------------------------------- differential anchor
constexpr int kDiffTcRows = 128, kDiffTcKeys = 128;  // bf16: query rows and keys of a tile
constexpr int kDiffF32Rows = 64;
constexpr int diff_f32_keys(int d) { return d > 64 ? 16 : 32; }  // two stages of K and V, two CTAs an SM
// Units (query tile, head, batch) of a forward call; those of the last partial
// wave may be cut `split` ways along the keys, with parts in scratch.
struct DiffPlan {
  int rows = 0, n_qtiles = 0, n_full = 0, n_split_units = 0, split = 1;
  bool cluster = false;  // every unit is split, its parts are a cluster and join there: no scratch
  size_t partial_bytes = 0;
  unsigned grid() const { return static_cast<unsigned>(n_full + n_split_units * split); }
};
// At most this many queries a batch go to the kernel that reads K and V once. 16 heads, B = 1, us
// forward/gradients, that kernel and a tile of queries with the merge of its parts (bf16; the
// tile's do not depend on N):
//     keys    N = 1    2        3, 4      tile
//     300     12/14    14/16    18/27     20/18
//     2,000   16/23    23/27    41/47     27/49
//     8,190   31/49    45/63    88/125    39/119
// fp32: 43/80, 59/106, 80/131 against 160/534 at 8,190 keys. Three and four rows in bf16 are
// slower forward behind 2,000 keys; they stay here for their unrounded weights.
constexpr int kDiffFewRows = 4;
// (it waits for nothing, reports nothing and writes the status words itself)
cudaError_t diff_fwd_few(const sva_diff_args& a, int* status, cudaStream_t s);
DiffPlan diff_plan(int B, int N, int H, int d, int n_keys, sva_dtype_t dt);
cudaError_t diff_fwd_f32(const sva_diff_args& a, void* scratch, cudaStream_t s);
cudaError_t diff_fwd_bf16(const sva_diff_args& a, int* status, void* scratch, cudaStream_t s);
cudaError_t diff_merge(const sva_diff_args& a, const DiffPlan& p, void* scratch, cudaStream_t s);
// Scratch of a backward call: dA (dtype, [B*N, D]), then the queries' statistics
// (per batch, head and 64-query tile) and dlambda per token (fp32).
struct DiffBwdPlan {
  size_t stats_off = 0, dlam_off = 0, total = 0;
};
struct DiffBwdScratch {
  void* da;      // [B, N, D] in dtype
  // [B*H][tiles of 64 queries][5][64]: -lse_1 log2 e, -lse_2 log2 e + log2 lambda,
  // -delta_m, -1; with lambda given as a value the second without it, the last -lambda
  float* stats;
  // [B*H][N]: -dA . O_2 per token (times a sigmoid's lambda), where one lambda is shared by
  // all or the gradients' kernel corrects it
  float* dlam;
};
// bf16 tiles: O_2 was made of bf16 weights
__host__ __device__ inline bool diff_dlam_later(const sva_diff_args& a) {
  return a.dtype == SVA_BF16 && a.N > kDiffFewRows;
}
// One launch of the backward tiles: `first` tiles a (batch, head) of the side whose
// tiles take longer (their streamed side is the longer one), each cut `cuts` ways along
// that stream where there are too few of them, the cuts being a cluster; then the
// other side's tiles.
struct DiffBwdGrid {
  int first = 0, second = 0, cuts = 1;
  bool keys_first = true;  // the first side's tiles are keys (dK, dV), else queries (dQ)
  unsigned ctas(int heads) const {
    return static_cast<unsigned>((first * cuts + (second + cuts - 1) / cuts * cuts) * heads);
  }
};
DiffBwdGrid diff_bwd_grid(const sva_diff_args& a, int rows, int streamed, int ctas_per_sm);
DiffBwdPlan diff_bwd_plan(int B, int N, int H, int d, sva_dtype_t dt);
DiffBwdScratch diff_bwd_scratch(const sva_diff_args& a, void* scratch);
cudaError_t diff_bwd(const sva_diff_args& a, const sva_diff_grads& g, int* status, void* scratch,
                     cudaStream_t s);
cudaError_t diff_bwd_few(const sva_diff_args& a, const sva_diff_grads& g, void* scratch, cudaStream_t s);
cudaError_t diff_bwd_f32(const sva_diff_args& a, const sva_diff_grads& g, void* scratch,
                         cudaStream_t s);
cudaError_t diff_bwd_bf16(const sva_diff_args& a, const sva_diff_grads& g, int* status,
                          void* scratch, cudaStream_t s);

// ---------------------------------------------------------------- block norms
size_t block_norm_scratch_bytes(int B, int N, int D);
cudaError_t block_norm_fwd(const sva_block_norm_args& a, cudaStream_t s);
cudaError_t block_norm_bwd(const sva_block_norm_args& a, const sva_block_norm_grads& g, int* status,
                           void* scratch, cudaStream_t s);

// ---------------------------------------------------------------- router
cudaError_t route(const float* h, const void* const* keys, const void* const* summaries,
                  int n_blocks, void* u, float* alpha, int64_t rows, int D, sva_dtype_t dt,
                  cudaStream_t s);

// ---------------------------------------------------------------- misc
cudaError_t selftest_wait(int* status, unsigned timeout_us, cudaStream_t s);
cudaError_t cast_f32(const float* src, void* dst, int64_t n, sva_dtype_t dt, cudaStream_t s);
cudaError_t upcast_to_f32(const void* src, float* dst, int64_t n, sva_dtype_t dt, cudaStream_t s);
cudaError_t sub_inplace(const float* a, float* out, int64_t n, cudaStream_t s);  // out = a - out

}  // namespace sva
