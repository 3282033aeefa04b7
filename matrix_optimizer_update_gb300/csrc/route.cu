// route.cu - tokens to experts and back (include/dmuon.h, "Tokens to experts and
// back"; the expert matrices of mixture-of-experts models are what "DMuon: Efficient
// Distributed Muon Training with Near-Adam Overhead" balances over owners): a stable counting sort of the assignments by expert, the copy of
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
// Stable counting sort. A block owns a contiguous run of assignments and each of its warps a contiguous part of
// it; a warp takes 32 assignments at a time and finds those of equal expert with one match per round, so the
// order within an expert is the order of the assignments whatever the blocks' timing. A warp reads 256 ids
// before it looks at the first and keeps what it found of them: the sort takes the latency of one round of
// loads, eight dependent updates of the counts and the sums over the warps.
//
// Up to 65536 assignments are one launch: a block of as many warps as they fill, or a cluster of up to 8
// blocks that read each other's counts from shared memory. More take three: counts, sums over the blocks, rows.
// (32768 assignments to 64 experts: 16 us against 28 in three launches; 131072 to 128: 39 against 31.)
constexpr int kSortBatch = 8;       // rounds of 32 a warp holds at a time
constexpr int kSortHeld = 32 * kSortBatch;
constexpr int kSortMaxBlocks = 1024;
constexpr int kSortCluster = 8;     // blocks of a cluster
// Warps per block at most: 32, or 8 where 32 counts per expert would not fit in shared memory (132 or 144 KB).
constexpr int kManyExperts = 1024, kMaxWarps = 32, kManyExpertsWarps = 8;
int sort_warps(int experts) { return experts <= kManyExperts ? kMaxWarps : kManyExpertsWarps; }
// The most shared memory a sort asks for: the counts of each warp and the block's own.
constexpr size_t kSortSmem =
    sizeof(int) * std::max((kMaxWarps + 1) * kManyExperts, (kManyExpertsWarps + 1) * kMaxExperts);

struct SortParams {
  const int64_t* ids;
  int64_t n;
  int32_t experts;
  int32_t per_warp;   // assignments per warp, a multiple of kSortHeld
  int32_t blocks;
  int32_t* dest;
  int32_t* source;
  int32_t* offsets;
  int32_t* counts;    // [blocks][experts]: a block's assignments per expert, then its first rows
};

// 256 assignments of a warp: their experts (-1: dropped), and each one's place among the warp's of its expert;
// mine[expert] counts them.
__device__ __forceinline__ void count_batch(const SortParams& p, int64_t first, int lane, int* mine,
                                            int (&e)[kSortBatch], int (&place)[kSortBatch]) {
  int64_t id[kSortBatch];
#pragma unroll
  for (int r = 0; r < kSortBatch; ++r) {
    const int64_t i = first + r * 32 + lane;
    id[r] = i < p.n ? p.ids[i] : -1;
  }
  unsigned same[kSortBatch];
#pragma unroll
  for (int r = 0; r < kSortBatch; ++r) {
    e[r] = id[r] >= 0 && id[r] < p.experts ? static_cast<int>(id[r]) : -1;
    same[r] = __match_any_sync(0xffffffffu, e[r]);
  }
#pragma unroll
  for (int r = 0; r < kSortBatch; ++r) {
    const int before = e[r] >= 0 ? mine[e[r]] : 0;
    const int rank = __popc(same[r] & ((1u << lane) - 1u));
    place[r] = before + rank;
    __syncwarp();
    if (e[r] >= 0 && rank == 0) mine[e[r]] = before + __popc(same[r]);
    __syncwarp();
  }
}

// Each warp's assignments per expert into hist[warp][experts]; e and place hold the last batch's.
__device__ __forceinline__ void warp_counts(const SortParams& p, int* hist, int64_t first, int (&e)[kSortBatch],
                                            int (&place)[kSortBatch]) {
  for (int j = threadIdx.x; j < int(blockDim.x >> 5) * p.experts; j += blockDim.x) hist[j] = 0;
  __syncthreads();
  for (int at = 0; at < p.per_warp; at += kSortHeld)
    count_batch(p, first + at, threadIdx.x & 31, hist + (threadIdx.x >> 5) * p.experts, e, place);
  __syncthreads();
}

__global__ void __launch_bounds__(1024) route_count_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int hist[];
  follow();
  const int warps = blockDim.x >> 5;
  int e[kSortBatch], place[kSortBatch];
  warp_counts(p, hist, (int64_t(blockIdx.x) * warps + (threadIdx.x >> 5)) * p.per_warp, e, place);
  for (int j = threadIdx.x; j < p.experts; j += blockDim.x) {
    int c = 0;
    for (int w = 0; w < warps; ++w) c += hist[w * p.experts + j];
    p.counts[int64_t(blockIdx.x) * p.experts + j] = c;
  }
}

// Exclusive sum over the block's threads; *total receives the sum of all.
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
  for (int w = 0; w < int(blockDim.x >> 5); ++w) {
    const int c = scratch[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// One block: the counts become each block's first row per expert, and offsets the experts' first rows.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) route_scan_kernel(const __grid_constant__ SortParams p) {
  __shared__ int scratch[32];
  follow();
  int base = 0;
  for (int e0 = 0; e0 < p.experts; e0 += kScanThreads) {
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

__device__ __forceinline__ int cluster_load(const int* mine, unsigned rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Rows of the block's assignments. ALL: the launch is one cluster (of gridDim.x blocks) that has all of them and
// makes the offsets itself; else the blocks' first rows are in p.counts.
template <bool ALL>
__global__ void __launch_bounds__(1024) route_place_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int hist[];  // [warps][experts], then (ALL) the block's own counts [experts]
  __shared__ int scratch[32];
  follow();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t first = (int64_t(blockIdx.x) * warps + warp) * p.per_warp;
  int e[kSortBatch], place[kSortBatch];
  warp_counts(p, hist, first, e, place);
  int* own = hist + warps * p.experts;
  if (ALL) {
    for (int x = threadIdx.x; x < p.experts; x += blockDim.x) {
      int mine = 0;
      for (int w = 0; w < warps; ++w) mine += hist[w * p.experts + x];
      own[x] = mine;
    }
    if (gridDim.x > 1) cluster_barrier();
    else __syncthreads();
  }
  int rows = 0;  // rows in use
  for (int e0 = 0; e0 < p.experts; e0 += blockDim.x) {
    const int x = e0 + threadIdx.x;
    int at = 0;
    if (ALL) {
      int before = 0, mine = 0, total;  // of the blocks before this one, of all
      if (x < p.experts)
        for (unsigned b = 0; b < gridDim.x; ++b) {
          const int c = gridDim.x > 1 ? cluster_load(&own[x], b) : own[x];
          before += b < blockIdx.x ? c : 0;
          mine += c;
        }
      const int start = rows + block_exclusive(mine, scratch, &total);
      if (x < p.experts && blockIdx.x == 0) p.offsets[x] = start;
      at = start + before;
      rows += total;
    } else if (x < p.experts) {
      at = p.counts[int64_t(blockIdx.x) * p.experts + x];
    }
    if (x < p.experts) {
      for (int w0 = 0; w0 < warps; w0 += 8) {  // the warps' first rows; 8 reads in flight, then 8 writes
        int k[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) k[u] = w0 + u < warps ? hist[(w0 + u) * p.experts + x] : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (w0 + u < warps) hist[(w0 + u) * p.experts + x] = at;
          at += k[u];
        }
      }
    }
  }
  if (!ALL) rows = p.offsets[p.experts];
  else if (threadIdx.x == 0 && blockIdx.x == 0) p.offsets[p.experts] = rows;
  __syncthreads();
  int* mine = hist + warp * p.experts;
  const bool held = p.per_warp == kSortHeld;  // else the batches are gone through again, the rows in place of counts
  for (int a = 0; a < p.per_warp; a += kSortHeld) {
    if (!held) count_batch(p, first + a, lane, mine, e, place);
#pragma unroll
    for (int r = 0; r < kSortBatch; ++r) {
      const int64_t i = first + a + r * 32 + lane;
      if (i >= p.n) break;
      const int row = e[r] < 0 ? -1 : held ? mine[e[r]] + place[r] : place[r];
      p.dest[i] = row;
      if (row >= 0) p.source[row] = static_cast<int32_t>(i);
      if (i >= rows) p.source[i] = -1;
    }
  }
  if (ALL && gridDim.x > 1) cluster_barrier();  // no block leaves while others read its counts
}

int64_t sort_blocks(int64_t n, int experts) {
  const int64_t run = int64_t(sort_warps(experts)) * kSortHeld;
  return std::max<int64_t>(1, std::min<int64_t>((n + run - 1) / run, kSortMaxBlocks));
}

cudaError_t launch_sort(SortParams& p, cudaStream_t s) {
  const int most = sort_warps(p.experts);
  const int64_t held = (p.n + kSortHeld - 1) / kSortHeld;  // batches of 256
  const bool all = held <= int64_t(kSortCluster) * most;
  int warps = most;
  if (all) {
    p.blocks = static_cast<int32_t>(std::min<int64_t>(kSortCluster, std::max<int64_t>(1, (held + most - 1) / most)));
    if (p.blocks == 1) warps = static_cast<int>(std::max<int64_t>(1, held));
  }
  const int64_t total = int64_t(p.blocks) * warps;
  p.per_warp = static_cast<int32_t>(std::max<int64_t>(1, (held + total - 1) / total) * kSortHeld);
  const size_t smem = sizeof(int) * (warps + 1) * p.experts;
  cudaError_t e = cudaSuccess;
  // Beside the static arrays, 40 KB are within the 48 KB that a launch has without asking. The limit is a property of
  // the kernel, not of the launch: every call sets the same, for threads that sort at the same time.
  if (smem > 40 * 1024) {
    for (auto* k : {route_count_kernel, route_place_kernel<true>, route_place_kernel<false>})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSortSmem));
    if (e != cudaSuccess) return e;
  }
  if (all) return launch_follow(route_place_kernel<true>, dim3(p.blocks), warps * 32, smem, s, p.blocks, p);
  e = launch_follow(route_count_kernel, dim3(p.blocks), warps * 32, smem, s, 1, p);
  if (e == cudaSuccess) e = launch_follow(route_scan_kernel, dim3(1), kScanThreads, 0, s, 1, p);
  if (e == cudaSuccess) e = launch_follow(route_place_kernel<false>, dim3(p.blocks), warps * 32, smem, s, 1, p);
  return e;
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

// All three move rows and are bound by memory: a row is read once and written once per side, in pieces of 16
// bytes, a block of 256 threads (combine_backward: a warp) to a row's pieces. 16384 tokens to 8 experts each,
// 4096 wide, bf16: dispatch 178 us (6.8 TB/s of 1.21 GB), combine 196 us (6.2), combine_backward 331 us (6.9 of
// 2.28 GB); the copy rate is 6.67.
//
// Assignments whose rows a thread reads at a time: their loads are in flight together.
constexpr int kAtOnce = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) route_dispatch_kernel(const __grid_constant__ RowParams p) {
  using P = Packed<T, V>;
  follow();
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(p.in) + t * p.ld;
  const int64_t dim = int64_t(p.pieces) * V;
  T* xs = static_cast<T*>(p.out);
  P zero;
#pragma unroll
  for (int j = 0; j < V; ++j) zero.v[j] = from_f<T>(0.f);
  for (int c = blockIdx.y * kRowThreads + threadIdx.x; c < p.pieces; c += gridDim.y * kRowThreads) {
    const int64_t at = int64_t(c) * V;
    const P v = *reinterpret_cast<const P*>(x + at);
    for (int k0 = 0; k0 < p.top; k0 += kAtOnce) {
      int row[kAtOnce];
      bool unused[kAtOnce];  // row i of xs is not in use
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t i = t * p.top + k0 + u;
        row[u] = k0 + u < p.top ? p.dest[i] : -1;
        unused[u] = k0 + u < p.top && p.source[i] < 0;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (row[u] >= 0) *reinterpret_cast<P*>(xs + row[u] * dim + at) = v;
        if (unused[u]) *reinterpret_cast<P*>(xs + (t * p.top + k0 + u) * dim + at) = zero;
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
    const T* ys = static_cast<const T*>(p.in) + int64_t(c) * V;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.f;
    for (int k0 = 0; k0 < p.top; k0 += kAtOnce) {
      int row[kAtOnce];
      float w[kAtOnce];
      P v[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t i = t * p.top + k0 + u;
        row[u] = k0 + u < p.top ? p.dest[i] : -1;
        w[u] = p.weights != nullptr && k0 + u < p.top ? p.weights[i] : 1.f;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (row[u] >= 0) v[u] = *reinterpret_cast<const P*>(ys + row[u] * dim);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (row[u] < 0) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = fmaf(w[u], to_f(v[u].v[j]), sum[j]);
      }
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
  *bytes = static_cast<size_t>(sort_blocks(tokens * top, experts) * experts) * sizeof(int32_t);
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
  p.blocks = static_cast<int32_t>(sort_blocks(n, experts));
  p.dest = dest;
  p.source = source;
  p.offsets = offsets;
  p.counts = static_cast<int32_t*>(d_workspace);
  return done(launch_sort(p, s));
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
