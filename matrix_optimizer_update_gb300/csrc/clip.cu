// clip.cu - the global norm of many gradient tensors, and their clipping (include/dmuon.h,
// "The global gradient norm, and clipping").
//
//   norm = sqrt(sum over all tensors of x^2);  out = x * min(1, max_norm / norm)
//
// Bound by memory: the norm reads every gradient once, the clipping reads it again (nothing can be
// written before everything has been read) and writes it.
//
// The tensors' table travels in the launch's parameters, so that nothing is copied to the device and a
// captured call carries its own. A tensor is cut into units of whole 16-byte vectors; unit u of a launch
// belongs to block u mod the grid, whatever the blocks' timing, and each block sums its units in their
// order: the norm is the same from call to call.
//
// Up to 512 KB are one launch: a cluster of 8 blocks holds all of it in registers, joins its sums through shared
// memory, and writes it back scaled. The host, which is what small sets wait for, pays for a launch less: four fp32
// matrices of 128 x 256 take 17 us a call for 22 in two launches. On the GPU it takes as long as the two up to
// 256 KB (10 us replayed from a graph) and 2 us more beyond (12.3 for 10.3).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "dmuon.h"
#include "follow.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dmuon {
namespace {

using bf16 = __nv_bfloat16;

// Few and large blocks: each block of the clipping pass adds up all blocks' sums in 64 bits, of which an SM does two
// or so a cycle. (8 blocks of 256 threads to an SM took 8 us more.)
constexpr int kThreads = 1024;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxBlocks = 512;
constexpr size_t kWorkspace = kMaxBlocks * sizeof(double);
constexpr int kMostTensors = 1024;  // per launch: 28 bytes each of the 32764 that parameters may take
constexpr int kFlight = 4;          // vectors a thread has in flight

// Tensors of one launch. Bit 0 of `in` marks bf16 (elements are 2 or 4 bytes apart, so that it is free).
template <int N>
struct Table {
  uint64_t in[N];
  uint64_t out[N];
  int64_t count[N];
  int32_t first[N + 1];  // first unit of each tensor; [tensors]: units
  int32_t tensors;
  int32_t per_unit;      // vectors per unit, a multiple of kThreads
};

// One tensor as it lies in memory: elements before the first 16-byte boundary, whole vectors, the rest.
struct Lie {
  int32_t head, tail;
  int64_t vectors;
};

__host__ __device__ __forceinline__ Lie lie_of(uint64_t address, int64_t count, bool half) {
  const int size = half ? 1 : 2, each = half ? 3 : 2;  // logarithms
  Lie l;
  const int64_t before = static_cast<int64_t>((16 - (address & 15)) & 15) >> size;
  l.head = static_cast<int32_t>(before < count ? before : count);
  l.vectors = (count - l.head) >> each;
  l.tail = static_cast<int32_t>(count - l.head - (l.vectors << each));
  return l;
}

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int unit) {
  int lo = 0, hi = t.tensors - 1;  // the last tensor that starts at or before the unit
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ float2 pair_of(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// A thread's sum of squares. Squares of a vector are added up in fp32 where all that counts of them is well
// inside its range (the vector's sum between 2^-100 and 2^100), in 64 bits where it is not: gradients of 1e-30
// or 1e30, infinities and NaN. Those of a unit are then added to a sum in 64 bits.
struct Squares {
  float near = 0.f;
  double sum = 0.0;
  __device__ __forceinline__ void one(float x) { sum += static_cast<double>(x) * x; }
  __device__ __forceinline__ void vector(const uint4& v, bool half) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s = 0.f;
    if (half) {
      float r = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = pair_of(w[k]);
        s = fmaf(f.x, f.x, s);
        r = fmaf(f.y, f.y, r);
      }
      s += r;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) s = fmaf(__uint_as_float(w[k]), __uint_as_float(w[k]), s);
    }
    if (s >= 0x1p-100f && s <= 0x1p100f) {
      near += s;
    } else if (((w[0] | w[1] | w[2] | w[3]) & (half ? 0x7fff7fffu : 0x7fffffffu)) != 0u) {  // not all zeros
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (half) {
          const float2 f = pair_of(w[k]);
          one(f.x);
          one(f.y);
        } else {
          one(__uint_as_float(w[k]));
        }
      }
    }
  }
  __device__ __forceinline__ void unit_done() {
    sum += static_cast<double>(near);
    near = 0.f;
  }
};

// The block's sum of one value per thread, in a fixed order; the first warp gets it.
__device__ __forceinline__ double block_sum(double v, double* red) {
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  static_assert(kThreads == 32 * 32, "a lane to a warp");
  if (threadIdx.x < 32) {
    v = red[threadIdx.x];
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// This thread's element of a tensor outside its whole vectors, if it has one.
struct Loose {
  uint64_t from, to;
  bool there;
  __device__ __forceinline__ float value(bool half) const {
    return half ? __bfloat162float(*reinterpret_cast<const bf16*>(from)) : *reinterpret_cast<const float*>(from);
  }
  __device__ __forceinline__ void scale(bool half, float s) const {
    if (half) {
      const bf16 x = *reinterpret_cast<const bf16*>(from);
      *reinterpret_cast<bf16*>(to) = s == 1.f ? x : __float2bfloat16_rn(__bfloat162float(x) * s);
    } else {
      const float x = *reinterpret_cast<const float*>(from);
      *reinterpret_cast<float*>(to) = s == 1.f ? x : x * s;
    }
  }
};
template <int N>
__device__ __forceinline__ Loose loose_of(const Table<N>& t, int i, const Lie& l, int thread, int size) {
  Loose e;
  e.there = thread < l.head + l.tail;
  const int64_t at = thread < l.head ? thread : t.count[i] - l.tail + (thread - l.head);
  e.from = (t.in[i] & ~uint64_t(1)) + at * size;
  e.to = t.out[i] + at * size;
  return e;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_kernel(const __grid_constant__ Table<N> t, double* partial, int first) {
  __shared__ double red[kThreads / 32];
  follow();
  Squares q;
  for (int u = blockIdx.x; u < t.first[t.tensors]; u += gridDim.x) {
    const int i = tensor_of(t, u);
    const bool half = (t.in[i] & 1u) != 0;
    const uint64_t at = t.in[i] & ~uint64_t(1);
    const Lie l = lie_of(at, t.count[i], half);
    const int64_t v0 = int64_t(u - t.first[i]) * t.per_unit;
    const int64_t v1 = min(v0 + t.per_unit, l.vectors);
    const uint4* body = reinterpret_cast<const uint4*>(at + l.head * (half ? 2 : 4));
    for (int64_t v = v0 + threadIdx.x; v < v1; v += kFlight * kThreads) {
      uint4 x[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        x[k] = v + k * kThreads < v1 ? load_once(body + v + k * kThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) q.vector(x[k], half);
    }
    const Loose e = loose_of(t, i, l, threadIdx.x, half ? 2 : 4);
    if (v0 == 0 && e.there) q.one(e.value(half));
    q.unit_done();
  }
  const double sum = block_sum(q.sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = first ? sum : partial[blockIdx.x] + sum;
}

// The norm from the blocks' sums, in the first warp.
__device__ __forceinline__ double norm_of(const double* partial, int blocks) {
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += 32) s += partial[b];
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return sqrt(s);
}

// What gradients of that norm are multiplied by. (A norm that is not finite clips nothing: the caller sees it. So it
// is the fp32 number which the caller gets that decides, where the one in 64 bits may still be finite.)
__device__ __forceinline__ float scale_of(double norm, float max_norm) {
  const bool clip = norm > static_cast<double>(max_norm) && static_cast<float>(norm) < INFINITY;
  return clip ? static_cast<float>(static_cast<double>(max_norm) / norm) : 1.f;
}

__global__ void __launch_bounds__(32) norm_done_kernel(const double* partial, int blocks, float* norm) {
  follow();
  const double n = norm_of(partial, blocks);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

__device__ __forceinline__ uint4 scaled(const uint4& v, bool half, float s) {
  uint4 o;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (half) {
      const float2 f = pair_of(w[k]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * s, f.y * s);
      r[k] = reinterpret_cast<const uint32_t&>(h);
    } else {
      r[k] = __float_as_uint(__uint_as_float(w[k]) * s);
    }
  }
  o.x = r[0], o.y = r[1], o.z = r[2], o.w = r[3];
  return o;
}

__device__ __forceinline__ void store_vector(uint64_t to, const uint4& v, bool half) {
  if ((to & 15) == 0) {  // the result lies as the gradient does
    __stcs(reinterpret_cast<uint4*>(to), v);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (half) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      reinterpret_cast<uint16_t*>(to)[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) reinterpret_cast<uint32_t*>(to)[e] = w[e];
  }
}

// The last units first: they are what the norm's pass left in L2.
template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) clip_kernel(const __grid_constant__ Table<N> t, const double* partial,
                                                        int blocks, float max_norm, float* norm) {
  __shared__ float scale;
  follow();
  if (threadIdx.x < 32) {
    const double total = norm_of(partial, blocks);
    if (threadIdx.x == 0) {
      if (norm != nullptr && blockIdx.x == 0) *norm = static_cast<float>(total);
      scale = scale_of(total, max_norm);
    }
  }
  __syncthreads();
  const float s = scale;
  for (int u = t.first[t.tensors] - 1 - static_cast<int>(blockIdx.x); u >= 0; u -= gridDim.x) {
    const int i = tensor_of(t, u);
    const bool half = (t.in[i] & 1u) != 0;
    const uint64_t at = t.in[i] & ~uint64_t(1), to = t.out[i];
    if (s == 1.f && at == to) continue;
    const int size = half ? 2 : 4;
    const Lie l = lie_of(at, t.count[i], half);
    const int64_t v0 = int64_t(u - t.first[i]) * t.per_unit;
    const int64_t v1 = min(v0 + t.per_unit, l.vectors);
    const uint4* body = reinterpret_cast<const uint4*>(at + l.head * size);
    const uint64_t body_to = to + l.head * size;
    for (int64_t v = v0 + threadIdx.x; v < v1; v += kFlight * kThreads) {
      uint4 x[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (v + k * kThreads < v1) x[k] = load_once(body + v + k * kThreads);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        if (v + k * kThreads >= v1) break;
        const uint4 o = s == 1.f ? x[k] : scaled(x[k], half, s);
        const uint64_t a = body_to + (v + k * kThreads) * 16;
        store_vector(a, o, half);
      }
    }
    const Loose e = loose_of(t, i, l, threadIdx.x, size);
    if (v0 == 0 && e.there) e.scale(half, s);
  }
}

// ------------------------------------------------------------------ few elements
constexpr int kCluster = 8;
constexpr int kGroup = 256;                        // threads that have a unit at a time, a vector each
constexpr int kGroups = kThreads / kGroup;
constexpr int kHold = 4;                           // units a thread holds a vector of
constexpr int kFewUnits = kCluster * kGroups * kHold;  // of kGroup vectors: 512 KB

template <int N>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ Table<N> t, int clipped, float max_norm,
                                                                  float* norm) {
  __shared__ double red[kThreads / 32];
  __shared__ double sums[kCluster];
  __shared__ float factor;
  follow();
  const int thread = threadIdx.x % kGroup, group = blockIdx.x * kGroups + threadIdx.x / kGroup;
  const int units = t.first[t.tensors];
  uint4 x[kHold];
  float loose[kHold];
  unsigned halves = 0u;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    x[k] = make_uint4(0, 0, 0, 0);
    loose[k] = 0.f;
    const int u = k * kCluster * kGroups + group;
    if (u >= units) continue;
    const int i = tensor_of(t, u);
    const bool half = (t.in[i] & 1u) != 0;
    const uint64_t at = t.in[i] & ~uint64_t(1);
    const Lie l = lie_of(at, t.count[i], half);
    const int64_t v = int64_t(u - t.first[i]) * kGroup + thread;
    if (v < l.vectors) x[k] = load_once(reinterpret_cast<const uint4*>(at + l.head * (half ? 2 : 4)) + v);
    const Loose e = loose_of(t, i, l, thread, half ? 2 : 4);
    if (v < kGroup && e.there) loose[k] = e.value(half);
    halves |= static_cast<unsigned>(half) << k;
  }
  Squares q;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    q.vector(x[k], (halves >> k & 1u) != 0);
    if (loose[k] != 0.f) q.one(loose[k]);
  }
  // A warp's sum: in fp32 where none of its threads has anything in 64 bits, of which it would be 32 times as many.
  double s;
  if (__any_sync(0xffffffffu, q.sum != 0.0)) {
    s = q.sum + static_cast<double>(q.near);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  } else {
    for (int d = 16; d > 0; d >>= 1) q.near += __shfl_xor_sync(0xffffffffu, q.near, d);
    s = static_cast<double>(q.near);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  ptx::cluster_sync();  // every block is there to be written to
  if (threadIdx.x < 32) {
    s = red[threadIdx.x];
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (threadIdx.x < kCluster) {
      const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sums[ptx::cluster_ctarank()]), threadIdx.x);
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(s) : "memory");
    }
  }
  __syncthreads();
  ptx::cluster_sync();
  if (threadIdx.x == 0) {
    double all = sums[0];
    for (int b = 1; b < kCluster; ++b) all += sums[b];
    const double total = sqrt(all);
    if (blockIdx.x == 0) *norm = static_cast<float>(total);
    factor = scale_of(total, max_norm);
  }
  if (!clipped) return;
  __syncthreads();
  const float scale = factor;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int u = k * kCluster * kGroups + group;
    if (u >= units) break;
    const int i = tensor_of(t, u);
    const bool half = (t.in[i] & 1u) != 0;
    const uint64_t at = t.in[i] & ~uint64_t(1);
    if (scale == 1.f && at == t.out[i]) continue;
    const int size = half ? 2 : 4;
    const Lie l = lie_of(at, t.count[i], half);
    const int64_t v = int64_t(u - t.first[i]) * kGroup + thread;
    if (v < l.vectors) store_vector(t.out[i] + l.head * size + v * 16, scale == 1.f ? x[k] : scaled(x[k], half, scale), half);
    const Loose e = loose_of(t, i, l, thread, size);
    if (v < kGroup && e.there) e.scale(half, scale);
  }
}

dmuon_status refuse(const char* msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

dmuon_status done(cudaError_t e) {
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  return set_last_error(DMUON_OK, "");
}

struct Call {
  const void* const* grads;
  void* const* out;   // nullptr: the norm alone
  const int64_t* counts;
  const int32_t* dtypes;
  int32_t n;
  float max_norm;
  float* norm;
  double* partial;
  int blocks;         // of every launch
  int32_t per_unit;
  cudaStream_t stream;
};

int64_t units_of(const Call& c, int i, int32_t per_unit) {
  const Lie l = lie_of(reinterpret_cast<uint64_t>(c.grads[i]), c.counts[i], c.dtypes[i] == DMUON_BF16);
  return std::max<int64_t>(1, (l.vectors + per_unit - 1) / per_unit);
}

// Tensors from..to of the call, those that are empty left out.
template <int N>
void fill(Table<N>& t, const Call& c, int from, int to, bool clip) {
  t.tensors = 0;
  t.per_unit = c.per_unit;
  int64_t units = 0;
  for (int i = from; i < to; ++i) {
    if (c.counts[i] == 0) continue;
    t.in[t.tensors] = reinterpret_cast<uint64_t>(c.grads[i]) | (c.dtypes[i] == DMUON_BF16 ? 1u : 0u);
    t.out[t.tensors] = clip ? reinterpret_cast<uint64_t>(c.out[i]) : 0;
    t.count[t.tensors] = c.counts[i];
    t.first[t.tensors++] = static_cast<int32_t>(units);
    units += units_of(c, i, c.per_unit);
  }
  t.first[t.tensors] = static_cast<int32_t>(units);
}

// One of the call's two passes over them.
template <int N>
cudaError_t launch(const Call& c, int from, int to, bool clip, bool first) {
  Table<N> t;
  fill(t, c, from, to, clip);
  if (clip)
    return launch_follow(clip_kernel<N>, dim3(c.blocks), kThreads, 0, c.stream, 1, t, static_cast<const double*>(c.partial),
                         c.blocks, c.max_norm, first ? c.norm : nullptr);
  return launch_follow(norm_kernel<N>, dim3(c.blocks), kThreads, 0, c.stream, 1, t, c.partial, static_cast<int>(first));
}

template <int N>
cudaError_t launch_few(Call c, bool clip) {
  Table<N> t;
  c.per_unit = kGroup;
  fill(t, c, 0, c.n, clip);
  return launch_follow(few_kernel<N>, dim3(kCluster), kThreads, 0, c.stream, kCluster, t, static_cast<int>(clip),
                       c.max_norm, c.norm);
}

// Small tables have launches of their own, as larger parameters take longer to launch.
cudaError_t pass(const Call& c, bool clip) {
  cudaError_t e = cudaSuccess;
  for (int from = 0; (from < c.n || from == 0) && e == cudaSuccess; from += kMostTensors) {
    const int to = std::min(c.n, from + kMostTensors), n = to - from;
    e = n <= 16    ? launch<16>(c, from, to, clip, from == 0)
        : n <= 128 ? launch<128>(c, from, to, clip, from == 0)
                   : launch<kMostTensors>(c, from, to, clip, from == 0);
  }
  return e;
}

struct Range {
  uint64_t begin, end;
  bool out;
};

// Whether a result lies over another tensor's gradient or result. (A tensor's own place is fine.)
bool overlap(const Call& c, std::vector<Range>& r) {
  for (int i = 0; i < c.n; ++i) {
    const uint64_t bytes = static_cast<uint64_t>(c.counts[i]) * (c.dtypes[i] == DMUON_BF16 ? 2 : 4);
    if (bytes == 0) continue;
    const uint64_t in = reinterpret_cast<uint64_t>(c.grads[i]), out = reinterpret_cast<uint64_t>(c.out[i]);
    r.push_back({out, out + bytes, true});
    if (in != out) r.push_back({in, in + bytes, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uint64_t outs = 0, ins = 0;  // how far those before reach
  for (const Range& x : r) {
    if (x.begin < outs || (x.out && x.begin < ins)) return true;
    uint64_t& reach = x.out ? outs : ins;
    reach = std::max(reach, x.end);
  }
  return false;
}

dmuon_status run(Call c, void* d_workspace, size_t bytes, void* stream, bool clip) {
  if (c.n < 0 || c.n > (1 << 20)) return refuse("n must be between 0 and 2^20");
  if (c.norm == nullptr || (reinterpret_cast<uintptr_t>(c.norm) & 3) != 0)
    return refuse("norm is NULL or not 4-byte aligned");
  if (c.n > 0 && (c.grads == nullptr || c.counts == nullptr || c.dtypes == nullptr || (clip && c.out == nullptr)))
    return refuse("NULL pointer argument");
  if (d_workspace == nullptr || (reinterpret_cast<uintptr_t>(d_workspace) & 255) != 0 || bytes < kWorkspace)
    return set_last_error(DMUON_ERR_WORKSPACE, "workspace is NULL, too small or not 256-byte aligned");
  if (clip && !(c.max_norm >= 0.f)) return refuse("max_norm must not be negative or NaN");
  int64_t vectors = 0;
  for (int i = 0; i < c.n; ++i) {
    if (c.dtypes[i] != DMUON_F32 && c.dtypes[i] != DMUON_BF16)
      return set_last_error(DMUON_ERR_UNSUPPORTED, "dtypes must be DMUON_F32 or DMUON_BF16");
    if (c.counts[i] < 0 || c.counts[i] > (int64_t(1) << 40)) return refuse("a count is negative or above 2^40");
    if (c.counts[i] == 0) continue;
    const uintptr_t mask = c.dtypes[i] == DMUON_BF16 ? 1 : 3;
    if (c.grads[i] == nullptr || (reinterpret_cast<uintptr_t>(c.grads[i]) & mask) != 0)
      return refuse("a gradient is NULL or not aligned to its elements");
    if (clip && (c.out[i] == nullptr || (reinterpret_cast<uintptr_t>(c.out[i]) & mask) != 0))
      return refuse("a result is NULL or not aligned to its elements");
    vectors += c.counts[i] / (c.dtypes[i] == DMUON_BF16 ? 8 : 4) + 1;
  }
  if (vectors > (int64_t(1) << 42)) return refuse("the tensors have too many elements");
  if (clip) {
    bool bad = false;
    try {
      std::vector<Range> r;
      r.reserve(2 * static_cast<size_t>(c.n));
      bad = overlap(c, r);
    } catch (...) {
      return refuse("out of host memory");
    }
    if (bad) return refuse("a result overlaps another tensor of the call");
  }
  c.partial = static_cast<double*>(d_workspace);
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  if (c.n <= 128 && vectors - c.n <= kFewUnits * kGroup) {  // too many to count otherwise
    int64_t units = 0;
    for (int i = 0; i < c.n; ++i)
      if (c.counts[i] > 0) units += units_of(c, i, kGroup);
    if (units <= kFewUnits) return done(c.n <= 16 ? launch_few<16>(c, clip) : launch_few<128>(c, clip));
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return done(e);
  // Units of 1 to 16 vectors a thread: as large as leaves every block several, as their start costs a search and a
  // partly filled round of loads.
  const int64_t most = std::min(kMaxBlocks, kBlocksPerSm * sms);
  int64_t turns = 1;
  while (turns < 16 && vectors / (kThreads * turns) > 8 * most) turns *= 2;
  while (vectors / (kThreads * turns) > (int64_t(1) << 29)) turns *= 2;  // unit numbers stay within 32 bits
  c.per_unit = static_cast<int32_t>(kThreads * turns);
  c.blocks = 1;
  for (int from = 0; from < c.n; from += kMostTensors) {
    int64_t units = 0;
    for (int i = from; i < std::min(c.n, from + kMostTensors); ++i)
      if (c.counts[i] > 0) units += units_of(c, i, c.per_unit);
    c.blocks = static_cast<int>(std::max<int64_t>(c.blocks, std::min(units, most)));
  }
  e = pass(c, false);
  if (e != cudaSuccess) return done(e);
  if (clip) return done(pass(c, true));
  return done(launch_follow(norm_done_kernel, dim3(1), 32, 0, c.stream, 1, static_cast<const double*>(c.partial),
                            c.blocks, c.norm));
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" dmuon_status dmuon_clip_workspace_bytes(size_t* bytes) {
  if (bytes == nullptr) return refuse("NULL argument");
  *bytes = kWorkspace;
  return set_last_error(DMUON_OK, "");
}

extern "C" dmuon_status dmuon_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                                        int32_t n, float* norm, void* d_workspace, size_t bytes, void* stream) {
  Call c{};
  c.grads = grads;
  c.counts = counts;
  c.dtypes = dtypes;
  c.n = n;
  c.norm = norm;
  return run(c, d_workspace, bytes, stream, false);
}

extern "C" dmuon_status dmuon_grad_clip(const void* const* grads, void* const* out, const int64_t* counts,
                                        const int32_t* dtypes, int32_t n, float max_norm, float* norm,
                                        void* d_workspace, size_t bytes, void* stream) {
  Call c{};
  c.grads = grads;
  c.out = out;
  c.counts = counts;
  c.dtypes = dtypes;
  c.n = n;
  c.max_norm = max_norm;
  c.norm = norm;
  return run(c, d_workspace, bytes, stream, true);
}
