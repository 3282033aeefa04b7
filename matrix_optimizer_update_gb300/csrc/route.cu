// route.cu - tokens to experts and back (include/dmuon.h, "Tokens to experts
// and back"): a stable counting sort of the assignments by expert, the copy of
// token rows into expert order, the weighted sum of expert rows per token, and
// the gradients of both.
#include <cuda_bf16.h>

#include <algorithm>

#include "dmuon.h"
#include "follow.cuh"
#include "internal.h"

namespace dmuon {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxTop = 64;
constexpr int kMaxExperts = 4096;
constexpr int64_t kMaxAssignments = int64_t(1) << 30;

// ------------------------------------------------------------------ sort
// Stable counting sort. A block owns a contiguous run of assignments and each of
// its 8 warps a contiguous part of it; a warp takes 32 assignments at a time and
// finds those of equal expert with one match per round, so the order within an
// expert is the order of the assignments whatever the blocks' timing.
constexpr int kSortWarps = 8;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr int kSortRun = 2048;      // assignments per block while there are few
constexpr int kSortMaxBlocks = 1024;

struct SortParams {
  const int64_t* ids;
  int64_t n;
  int32_t experts;
  int32_t run;        // assignments per block, a multiple of kSortThreads
  int32_t blocks;
  int32_t* dest;
  int32_t* source;
  int32_t* offsets;
  int32_t* counts;    // [blocks][experts]: a block's assignments per expert, then its first rows
};

__device__ __forceinline__ int expert_of(const SortParams& p, int64_t i) {
  if (i >= p.n) return -1;
  const int64_t e = p.ids[i];
  return (e >= 0 && e < p.experts) ? static_cast<int>(e) : -1;
}

// Each warp's assignments per expert into hist[warp][experts].
__device__ __forceinline__ void warp_counts(const SortParams& p, int* hist, int64_t first, int per_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < kSortWarps * p.experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  int* mine = hist + warp * p.experts;
  for (int r = 0; r < per_warp; r += 32) {
    const int e = expert_of(p, first + r + lane);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && (same & ((1u << lane) - 1u)) == 0u) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) route_count_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int hist[];
  follow();
  const int per_warp = p.run / kSortWarps;
  warp_counts(p, hist, int64_t(blockIdx.x) * p.run + int64_t(threadIdx.x >> 5) * per_warp, per_warp);
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) {
    int c = 0;
    for (int w = 0; w < kSortWarps; ++w) c += hist[w * p.experts + e];
    p.counts[int64_t(blockIdx.x) * p.experts + e] = c;
  }
}

// Exclusive sum over the block's threads (kSortThreads of them); *total receives the sum of all.
__device__ __forceinline__ int block_exclusive(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSortWarps; ++w) {
    const int c = scratch[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// One block: the counts become each block's first row per expert, and offsets the experts' first rows.
__global__ void __launch_bounds__(kSortThreads) route_scan_kernel(const __grid_constant__ SortParams p) {
  __shared__ int scratch[kSortWarps];
  follow();
  int base = 0;
  for (int e0 = 0; e0 < p.experts; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    int mine = 0;
    if (e < p.experts)
      for (int b = 0; b < p.blocks; ++b) mine += p.counts[int64_t(b) * p.experts + e];
    int total;
    int at = base + block_exclusive(mine, scratch, &total);
    if (e < p.experts) {
      p.offsets[e] = at;
      for (int b = 0; b < p.blocks; ++b) {
        int* c = &p.counts[int64_t(b) * p.experts + e];
        const int k = *c;
        *c = at;
        at += k;
      }
    }
    base += total;
  }
  if (threadIdx.x == 0) p.offsets[p.experts] = base;
}

// Rows of the block's assignments. ONE: a single block has all of them and makes the offsets itself.
template <bool ONE>
__global__ void __launch_bounds__(kSortThreads) route_place_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int hist[];
  __shared__ int scratch[kSortWarps];
  follow();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_warp = p.run / kSortWarps;
  const int64_t first = int64_t(blockIdx.x) * p.run + int64_t(warp) * per_warp;
  warp_counts(p, hist, first, per_warp);
  int rows = 0;  // rows in use
  if (ONE) {
    for (int e0 = 0; e0 < p.experts; e0 += kSortThreads) {
      const int e = e0 + threadIdx.x;
      int mine = 0;
      if (e < p.experts)
        for (int w = 0; w < kSortWarps; ++w) mine += hist[w * p.experts + e];
      int total;
      int at = rows + block_exclusive(mine, scratch, &total);
      if (e < p.experts) {
        p.offsets[e] = at;
        for (int w = 0; w < kSortWarps; ++w) {
          const int k = hist[w * p.experts + e];
          hist[w * p.experts + e] = at;
          at += k;
        }
      }
      rows += total;
    }
    if (threadIdx.x == 0) p.offsets[p.experts] = rows;
  } else {
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) {
      int at = p.counts[int64_t(blockIdx.x) * p.experts + e];
      for (int w = 0; w < kSortWarps; ++w) {
        const int k = hist[w * p.experts + e];
        hist[w * p.experts + e] = at;
        at += k;
      }
    }
    rows = p.offsets[p.experts];
  }
  __syncthreads();
  int* mine = hist + warp * p.experts;
  for (int r = 0; r < per_warp; r += 32) {
    const int64_t i = first + r + lane;
    const int e = expert_of(p, i);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int row = e >= 0 ? mine[e] + rank : -1;
    __syncwarp();
    if (e >= 0 && rank == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i < p.n) {
      p.dest[i] = row;
      if (row >= 0) p.source[row] = static_cast<int32_t>(i);
      if (i >= rows) p.source[i] = -1;
    }
  }
}

int64_t sort_blocks(int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>((n + kSortRun - 1) / kSortRun, kSortMaxBlocks));
}

// ------------------------------------------------------------------ rows
// A row moves in pieces of V elements: 16 bytes where every row starts on 16 bytes and is a whole
// number of them, else one element.
template <typename T, int V>
struct alignas(V == 1 ? sizeof(T) : 16) Packed {
  T v[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) {
  return __float2bfloat16_rn(x);
}

struct RowParams {
  const void* in;      // x (dispatch), ys (combine, combine_backward)
  const void* dy;      // combine_backward
  void* out;           // xs, y, dys
  const float* weights;
  float* dweights;
  const int32_t* dest;
  const int32_t* source;
  int64_t tokens;
  int64_t ld;          // row pitch of the tokens' side
  int32_t top;
  int32_t pieces;      // per row
};

constexpr int kRowThreads = 256;

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) route_dispatch_kernel(const __grid_constant__ RowParams p) {
  using P = Packed<T, V>;
  follow();
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(p.in) + t * p.ld;
  const int64_t dim = int64_t(p.pieces) * V;
  for (int c = blockIdx.y * kRowThreads + threadIdx.x; c < p.pieces; c += gridDim.y * kRowThreads) {
    const P v = *reinterpret_cast<const P*>(x + int64_t(c) * V);
    for (int k = 0; k < p.top; ++k) {
      const int64_t i = t * p.top + k;
      const int row = p.dest[i];
      if (row >= 0) *reinterpret_cast<P*>(static_cast<T*>(p.out) + row * dim + int64_t(c) * V) = v;
      if (p.source[i] < 0) {
        P zero;
#pragma unroll
        for (int j = 0; j < V; ++j) zero.v[j] = from_f<T>(0.f);
        *reinterpret_cast<P*>(static_cast<T*>(p.out) + i * dim + int64_t(c) * V) = zero;
      }
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) route_combine_kernel(const __grid_constant__ RowParams p) {
  using P = Packed<T, V>;
  follow();
  const int64_t t = blockIdx.x;
  T* y = static_cast<T*>(p.out) + t * p.ld;
  const int64_t dim = int64_t(p.pieces) * V;
  for (int c = blockIdx.y * kRowThreads + threadIdx.x; c < p.pieces; c += gridDim.y * kRowThreads) {
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.f;
    for (int k = 0; k < p.top; ++k) {
      const int64_t i = t * p.top + k;
      const int row = p.dest[i];
      if (row < 0) continue;
      const float w = p.weights != nullptr ? p.weights[i] : 1.f;
      const P v = *reinterpret_cast<const P*>(static_cast<const T*>(p.in) + row * dim + int64_t(c) * V);
#pragma unroll
      for (int j = 0; j < V; ++j) sum[j] = fmaf(w, to_f(v.v[j]), sum[j]);
    }
    P o;
#pragma unroll
    for (int j = 0; j < V; ++j) o.v[j] = from_f<T>(sum[j]);
    *reinterpret_cast<P*>(y + int64_t(c) * V) = o;
  }
}

// One warp per assignment: dys = w * dy and the dot product for dw in one pass over the row.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) route_combine_backward_kernel(const __grid_constant__ RowParams p) {
  using P = Packed<T, V>;
  follow();
  const int lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (i >= p.tokens * p.top) return;
  const int64_t dim = int64_t(p.pieces) * V;
  const int row = p.dest[i];
  if (p.source[i] < 0) {
    P zero;
#pragma unroll
    for (int j = 0; j < V; ++j) zero.v[j] = from_f<T>(0.f);
    for (int c = lane; c < p.pieces; c += 32)
      *reinterpret_cast<P*>(static_cast<T*>(p.out) + i * dim + int64_t(c) * V) = zero;
  }
  if (row < 0) {
    if (lane == 0) p.dweights[i] = 0.f;
    return;
  }
  const float w = p.weights[i];
  const T* dy = static_cast<const T*>(p.dy) + (i / p.top) * p.ld;
  const T* ys = static_cast<const T*>(p.in) + row * dim;
  T* dys = static_cast<T*>(p.out) + row * dim;
  float dot = 0.f;
  for (int c = lane; c < p.pieces; c += 32) {
    const P a = *reinterpret_cast<const P*>(dy + int64_t(c) * V);
    const P b = *reinterpret_cast<const P*>(ys + int64_t(c) * V);
    P o;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = to_f(a.v[j]);
      dot = fmaf(d, to_f(b.v[j]), dot);
      o.v[j] = from_f<T>(w * d);
    }
    *reinterpret_cast<P*>(dys + int64_t(c) * V) = o;
  }
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (lane == 0) p.dweights[i] = dot;
}

// ------------------------------------------------------------------ host
dmuon_status refuse(const char* msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

dmuon_status check_sizes(int64_t tokens, int32_t top) {
  if (tokens < 0 || top < 1 || top > kMaxTop) return refuse("tokens must be >= 0 and top between 1 and 64");
  if (tokens > kMaxAssignments / top) return refuse("tokens * top must be at most 2^30");
  return DMUON_OK;
}

dmuon_status check_rows(int64_t tokens, int32_t top, int64_t dim, int32_t dtype, int64_t ld) {
  dmuon_status st = check_sizes(tokens, top);
  if (st != DMUON_OK) return st;
  if (dim < 1 || dim > (int64_t(1) << 24)) return refuse("dim must be between 1 and 2^24");
  if (dtype != DMUON_F32 && dtype != DMUON_BF16)
    return set_last_error(DMUON_ERR_UNSUPPORTED, "dtype must be DMUON_F32 or DMUON_BF16");
  if (ld < dim) return refuse("a row pitch is shorter than dim");
  return DMUON_OK;
}

dmuon_status done(cudaError_t e) {
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  return set_last_error(DMUON_OK, "");
}

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

enum RowOp { kDispatch, kCombine, kCombineBackward };

template <typename T, int V>
cudaError_t launch_rows(RowOp op, RowParams& p, int64_t dim, cudaStream_t s) {
  p.pieces = static_cast<int32_t>(dim / V);
  if (op == kCombineBackward) {
    const int64_t blocks = (p.tokens * p.top + kRowThreads / 32 - 1) / (kRowThreads / 32);
    return launch_follow(route_combine_backward_kernel<T, V>, dim3(static_cast<unsigned>(blocks)), kRowThreads, 0, s, 1,
                         p);
  }
  const unsigned parts = static_cast<unsigned>(std::min<int64_t>((p.pieces + kRowThreads - 1) / kRowThreads, 65535));
  return launch_follow(op == kDispatch ? route_dispatch_kernel<T, V> : route_combine_kernel<T, V>,
                       dim3(static_cast<unsigned>(p.tokens), parts), kRowThreads, 0, s, 1, p);
}

dmuon_status run_rows(RowOp op, RowParams p, int64_t dim, int32_t dtype, void* stream) {
  const size_t es = dtype == DMUON_BF16 ? 2 : 4;
  const bool vec = (dim * es) % 16 == 0 && (p.ld * es) % 16 == 0 && !misaligned(p.in, 16) && !misaligned(p.out, 16) &&
                   !misaligned(p.dy, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == DMUON_BF16) return done(vec ? launch_rows<bf16, 8>(op, p, dim, s) : launch_rows<bf16, 1>(op, p, dim, s));
  return done(vec ? launch_rows<float, 4>(op, p, dim, s) : launch_rows<float, 1>(op, p, dim, s));
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" dmuon_status dmuon_route_workspace_bytes(int64_t tokens, int32_t top, int32_t experts, size_t* bytes) {
  if (bytes == nullptr) return refuse("NULL argument");
  dmuon_status st = check_sizes(tokens, top);
  if (st != DMUON_OK) return st;
  if (experts < 1 || experts > kMaxExperts) return refuse("experts must be between 1 and 4096");
  *bytes = static_cast<size_t>(sort_blocks(tokens * top) * experts) * sizeof(int32_t);
  return set_last_error(DMUON_OK, "");
}

extern "C" dmuon_status dmuon_route_sort(const int64_t* expert_ids, int64_t tokens, int32_t top, int32_t experts,
                                         int32_t* dest, int32_t* source, int32_t* offsets, void* d_workspace,
                                         size_t bytes, void* stream) {
  size_t need = 0;
  dmuon_status st = dmuon_route_workspace_bytes(tokens, top, experts, &need);
  if (st != DMUON_OK) return st;
  const int64_t n = tokens * top;
  if (offsets == nullptr || (n > 0 && (expert_ids == nullptr || dest == nullptr || source == nullptr)))
    return refuse("NULL pointer argument");
  if (d_workspace == nullptr || misaligned(d_workspace, 256) || bytes < need)
    return set_last_error(DMUON_ERR_WORKSPACE, "workspace is NULL, too small or not 256-byte aligned");
  if (misaligned(expert_ids, 8) || misaligned(dest, 4) || misaligned(source, 4) || misaligned(offsets, 4))
    return refuse("an index pointer is not aligned to its elements");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  SortParams p;
  p.ids = expert_ids;
  p.n = n;
  p.experts = experts;
  p.blocks = static_cast<int32_t>(sort_blocks(n));
  const int64_t per = (n + p.blocks - 1) / p.blocks;
  p.run = static_cast<int32_t>(std::max<int64_t>(1, (per + kSortThreads - 1) / kSortThreads) * kSortThreads);
  p.dest = dest;
  p.source = source;
  p.offsets = offsets;
  p.counts = static_cast<int32_t*>(d_workspace);
  const size_t smem = sizeof(int) * kSortWarps * experts;
  if (smem > 48 * 1024) {
    for (auto* k : {route_count_kernel, route_place_kernel<true>, route_place_kernel<false>}) {
      const cudaError_t e =
          cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
    }
  }
  if (p.blocks == 1) {
    return done(launch_follow(route_place_kernel<true>, dim3(1), kSortThreads, smem, s, 1, p));
  }
  cudaError_t e = launch_follow(route_count_kernel, dim3(p.blocks), kSortThreads, smem, s, 1, p);
  if (e == cudaSuccess) e = launch_follow(route_scan_kernel, dim3(1), kSortThreads, 0, s, 1, p);
  if (e == cudaSuccess) e = launch_follow(route_place_kernel<false>, dim3(p.blocks), kSortThreads, smem, s, 1, p);
  return done(e);
}

extern "C" dmuon_status dmuon_route_dispatch(const void* x, int64_t ld_x, const int32_t* dest, const int32_t* source,
                                             int64_t tokens, int32_t top, int64_t dim, int32_t dtype, void* xs,
                                             void* stream) {
  dmuon_status st = check_rows(tokens, top, dim, dtype, ld_x);
  if (st != DMUON_OK) return st;
  if (tokens == 0) return set_last_error(DMUON_OK, "");
  if (x == nullptr || dest == nullptr || source == nullptr || xs == nullptr) return refuse("NULL pointer argument");
  RowParams p{};
  p.in = x;
  p.out = xs;
  p.dest = dest;
  p.source = source;
  p.tokens = tokens;
  p.ld = ld_x;
  p.top = top;
  return run_rows(kDispatch, p, dim, dtype, stream);
}

extern "C" dmuon_status dmuon_route_combine(const void* ys, const float* weights, const int32_t* dest, int64_t tokens,
                                            int32_t top, int64_t dim, int32_t dtype, void* y, int64_t ld_y,
                                            void* stream) {
  dmuon_status st = check_rows(tokens, top, dim, dtype, ld_y);
  if (st != DMUON_OK) return st;
  if (tokens == 0) return set_last_error(DMUON_OK, "");
  if (ys == nullptr || dest == nullptr || y == nullptr) return refuse("NULL pointer argument");
  RowParams p{};
  p.in = ys;
  p.out = y;
  p.weights = weights;
  p.dest = dest;
  p.tokens = tokens;
  p.ld = ld_y;
  p.top = top;
  return run_rows(kCombine, p, dim, dtype, stream);
}

extern "C" dmuon_status dmuon_route_combine_backward(const void* dy, int64_t ld_dy, const void* ys,
                                                     const float* weights, const int32_t* dest, const int32_t* source,
                                                     int64_t tokens, int32_t top, int64_t dim, int32_t dtype, void* dys,
                                                     float* dweights, void* stream) {
  dmuon_status st = check_rows(tokens, top, dim, dtype, ld_dy);
  if (st != DMUON_OK) return st;
  if (tokens == 0) return set_last_error(DMUON_OK, "");
  if (dy == nullptr || ys == nullptr || weights == nullptr || dest == nullptr || source == nullptr || dys == nullptr ||
      dweights == nullptr)
    return refuse("NULL pointer argument");
  RowParams p{};
  p.in = ys;
  p.dy = dy;
  p.out = dys;
  p.weights = weights;
  p.dweights = dweights;
  p.dest = dest;
  p.source = source;
  p.tokens = tokens;
  p.ld = ld_dy;
  p.top = top;
  return run_rows(kCombineBackward, p, dim, dtype, stream);
}
