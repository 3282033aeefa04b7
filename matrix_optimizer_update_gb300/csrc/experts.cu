// experts.cu - a mixture's experts for a few tokens (include/dmuon.h, "A mixture's experts for a few
// tokens"): from the router's ids and weights to the layer's output, in two launches.
//
//   h[i] = silu(G_e x_t) * U_e x_t   (without a gate: silu(U_e x_t))     i = t*top + k, e = ids[i]
//   y[t] = sum_k weights[i] * D_e h[i]
//
// Bound by reading the matrices of the experts that the tokens reach, once: a token's products are 1 flop
// for each byte read, 64 tokens' on 64 experts 8.
//
// A block takes 16 rows of an expert's matrix at a time (8 of gate and the same 8 of up) and all of the
// expert's tokens. Its 8 warps share K: each reads 64-byte pieces of the rows, 16 bytes a lane, straight
// into the registers that mma.sync takes as its A operand, and the tokens' pieces of the same columns as B.
// A product's sum may run over K in any order, so the lanes' 8 consecutive elements stand for whatever K
// indices the instruction gives its lanes: no shared memory, no barrier and no transposition between
// memory and tensor cores, and a block's whole 16 rows are in flight at once.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "dmuon.h"
#include "follow.cuh"
#include "internal.h"

namespace dmuon {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxTop = 64;
constexpr int kMaxExperts = 4096;
constexpr int kMaxAssignments = 4096;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;    // rows of a unit
constexpr int kStep = 32;    // K of a warp's step: 4 lanes of 8 elements
constexpr int kFlight = 8;   // steps in flight

struct ExpertsParams {
  const int64_t* ids;
  const float* weights;
  const bf16* x;
  int64_t ld_x;
  const bf16* up;
  const bf16* gate;    // or nullptr
  const bf16* down;
  bf16* h;             // [2][assignments][ld_h]: h as the sum of two bf16
  int64_t ld_h;
  float* part;         // [assignments][dim]: D_e h, not yet weighted
  unsigned* arrived;   // per block of 16 entries of y: experts that are done
  bf16* y;
  int64_t ld_y;
  int32_t tokens, top, experts, n;  // n = tokens * top
  int32_t dim, inner;
};

// What a block knows of the routing: each assignment's expert, and the experts in use in ascending order.
struct Routing {
  int16_t expert[kMaxAssignments];
  int16_t active[kMaxAssignments];
  uint32_t used[kMaxExperts / 32];
  int actives;
};

__device__ __forceinline__ void read_routing(const ExpertsParams& p, Routing& r) {
  for (int w = threadIdx.x; w < kMaxExperts / 32; w += kThreads) r.used[w] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int64_t id = p.ids[i];
    const bool in = id >= 0 && id < p.experts;
    r.expert[i] = in ? static_cast<int16_t>(id) : int16_t(-1);
    if (in) atomicOr(&r.used[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    constexpr int kEach = kMaxExperts / 32 / 32;  // words per lane
    int mine = 0;
    for (int k = 0; k < kEach; ++k) mine += __popc(r.used[threadIdx.x * kEach + k]);
    int before = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (threadIdx.x >= d) before += o;
    }
    if (threadIdx.x == 31) r.actives = before;
    before -= mine;
    for (int k = 0; k < kEach; ++k) {
      uint32_t w = r.used[threadIdx.x * kEach + k];
      while (w != 0u) {
        r.active[before++] = static_cast<int16_t>((threadIdx.x * kEach + k) * 32 + __ffs(w) - 1);
        w &= w - 1u;
      }
    }
  }
  __syncthreads();
}

// The assignments of an expert, in order, to list; by one warp. Returns how many.
__device__ __forceinline__ int list_of(const Routing& r, int n, int expert, int16_t* list, int lane) {
  int count = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const bool on = i0 + lane < n && r.expert[i0 + lane] == expert;
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (on) list[count + __popc(b & ((1u << lane) - 1u))] = static_cast<int16_t>(i0 + lane);
    count += __popc(b);
  }
  return count;
}

__device__ __forceinline__ uint4 load_weights(const bf16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 8 elements from column k of a row of `dim`, zeros past its end. VEC: dim is a multiple of 8 and rows start on 16 bytes.
template <bool VEC, bool WEIGHTS>
__device__ __forceinline__ uint4 piece(const bf16* row, int k, int dim) {
  if (VEC) {
    if (k >= dim) return make_uint4(0, 0, 0, 0);
    if (WEIGHTS) return load_weights(row + k);
    return *reinterpret_cast<const uint4*>(row + k);
  }
  uint32_t w[4] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < dim) w[e >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[k + e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

enum Phase { kGated, kUngated, kDown };

// Tiles of 8 assignments at a time: TILES.
template <int PHASE, int TILES, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) experts_kernel(const __grid_constant__ ExpertsParams p) {
  __shared__ Routing r;
  __shared__ int16_t list[kMaxAssignments];
  __shared__ int count;
  __shared__ float sums[kWarps][TILES][4][32];
  __shared__ unsigned last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // The down products' launch is set up while the up products' still runs: what it reads before follow() was
  // there before that launch began.
  if (PHASE != kDown) {
    follow();
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < (p.dim + kRows - 1) / kRows; i += gridDim.x * kThreads)
      p.arrived[i] = 0u;
  }
  read_routing(p, r);
  const int K = PHASE == kDown ? p.inner : p.dim;
  const int rows = PHASE == kDown ? p.dim : p.inner;  // of a matrix
  constexpr int kOut = PHASE == kGated ? 8 : 16;      // rows of the result per unit
  const int blocks = (rows + kOut - 1) / kOut;
  const int units = r.actives * blocks;
  if (PHASE == kDown) {
    if (units == 0) {
      follow();
      for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < int64_t(p.tokens) * p.dim; i += gridDim.x * kThreads)
        p.y[i / p.dim * p.ld_y + i % p.dim] = __float2bfloat16_rn(0.f);
      return;
    }
  }
  const int steps = (K + kStep - 1) / kStep;
  int before = -1;
  bool waited = PHASE != kDown;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = r.active[u / blocks], b = u % blocks;
    const int o0 = min(b * kOut + g, rows - 1), o1 = min(b * kOut + g + 8, rows - 1);
    const int64_t matrix = int64_t(e) * rows;
    const bf16 *row0, *row1;
    if (PHASE == kGated) {
      row0 = p.gate + (matrix + o0) * K;
      row1 = p.up + (matrix + o0) * K;
    } else {
      const bf16* w = PHASE == kDown ? p.down : p.up;
      row0 = w + (matrix + o0) * K;
      row1 = w + (matrix + o1) * K;
    }
    uint4 a[kFlight][2];
    auto fetch = [&](int s0) {
#pragma unroll
      for (int s = 0; s < kFlight; ++s) {
        const int k = (s0 + s * kWarps) * kStep + 8 * c;
        a[s][0] = piece<VEC, true>(row0, k, K);
        a[s][1] = piece<VEC, true>(row1, k, K);
      }
    };
    fetch(warp);
    if (e != before) {
      if (warp == 0) {
        const int n = list_of(r, p.n, e, list, lane);
        if (lane == 0) count = n;
      }
      before = e;
      __syncthreads();
    }
    if (!waited) {
      follow();
      waited = true;
    }
    for (int j0 = 0; j0 < count; j0 += 8 * TILES) {
      const int tiles = min(TILES, (count - j0 + 7) / 8);
      float acc[TILES][4] = {};
      int row[TILES];  // of x or h, of the column that this lane brings
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int j = j0 + t * 8 + g;
        row[t] = j < count ? (PHASE == kDown ? list[j] : list[j] / p.top) : -1;
      }
      if (j0 > 0) fetch(warp);
      for (int s0 = warp; s0 < steps; s0 += kWarps * kFlight) {
        if (s0 != warp) fetch(s0);
#pragma unroll
        for (int s = 0; s < kFlight; ++s) {
          const int k = (s0 + s * kWarps) * kStep + 8 * c;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            if (t >= tiles) break;
            uint4 v = make_uint4(0, 0, 0, 0), w = v;
            if (row[t] >= 0) {
              if (PHASE == kDown) {
                v = piece<VEC, false>(p.h + row[t] * p.ld_h, k, K);
                w = piece<VEC, false>(p.h + (p.n + row[t]) * p.ld_h, k, K);
              } else {
                v = piece<VEC, false>(p.x + row[t] * p.ld_x, k, K);
              }
            }
            mma(acc[t], a[s][0].x, a[s][1].x, a[s][0].y, a[s][1].y, v.x, v.y);
            mma(acc[t], a[s][0].z, a[s][1].z, a[s][0].w, a[s][1].w, v.z, v.w);
            if (PHASE == kDown) {
              mma(acc[t], a[s][0].x, a[s][1].x, a[s][0].y, a[s][1].y, w.x, w.y);
              mma(acc[t], a[s][0].z, a[s][1].z, a[s][0].w, a[s][1].w, w.z, w.w);
            }
          }
        }
      }
      // the warps' sums joined; sums[.][t][v][l] is row l / 4 (+ 8 for v >= 2), column 2 * (l % 4) + v % 2
#pragma unroll
      for (int t = 0; t < TILES; ++t)
        if (t < tiles)
#pragma unroll
          for (int v = 0; v < 4; ++v) sums[warp][t][v][lane] = acc[t][v];
      __syncthreads();
      constexpr int kEach = PHASE == kGated ? 2 : 4;
      for (int i = threadIdx.x; i < tiles * kEach * 32; i += kThreads) {
        const int l = i & 31, v = (i >> 5) % kEach, t = (i >> 5) / kEach;
        const int j = j0 + t * 8 + 2 * (l & 3) + (v & 1);
        const int o = b * kOut + (l >> 2) + (v >= 2 ? 8 : 0);
        if (j >= count || o >= rows) continue;
        float s = 0.f, s1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          s += sums[w][t][v][l];
          if (PHASE == kGated) s1 += sums[w][t][v + 2][l];
        }
        if (PHASE == kDown) {
          p.part[int64_t(list[j]) * p.dim + o] = s;
        } else {
          const float f = s / (1.f + expf(-s)) * (PHASE == kGated ? s1 : 1.f);
          // as the sum of two bf16: rounded to one, h would double the squared error of y, whose own rounding is as large
          const bf16 high = __float2bfloat16_rn(f);
          const float rest = fabsf(__bfloat162float(high)) < INFINITY ? f - __bfloat162float(high) : 0.f;
          p.h[list[j] * p.ld_h + o] = high;
          p.h[(p.n + list[j]) * p.ld_h + o] = __float2bfloat16_rn(rest);
        }
      }
      __syncthreads();
    }
    if (PHASE == kDown) {
      // the last expert's block to be done with these 16 entries of y adds them up, in the order of k
      if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(&p.arrived[b], 1u) == static_cast<unsigned>(r.actives - 1);
      }
      __syncthreads();
      if (last != 0u) {
        __threadfence();
        for (int i = threadIdx.x; i < p.tokens * kRows; i += kThreads) {
          const int t = i / kRows, o = b * kRows + i % kRows;
          if (o >= p.dim) continue;
          float s = 0.f;
          for (int k = 0; k < p.top; ++k) {
            const int q = t * p.top + k;
            if (r.expert[q] >= 0) s = fmaf(p.weights[q], __ldcg(&p.part[int64_t(q) * p.dim + o]), s);
          }
          p.y[t * p.ld_y + o] = __float2bfloat16_rn(s);
        }
      }
      __syncthreads();
    }
  }
  if (!waited) follow();
}

dmuon_status refuse(const char* msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int64_t pitch_h(int64_t inner) { return (inner + 7) / 8 * 8; }

dmuon_status check_sizes(int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner) {
  if (top < 1 || top > kMaxTop) return refuse("top must be between 1 and 64");
  if (tokens < 0 || tokens * top > kMaxAssignments || tokens > kMaxAssignments)
    return refuse("tokens * top must be between 0 and 4096 (for more: sort, dispatch, the experts' products, combine)");
  if (experts < 1 || experts > kMaxExperts) return refuse("experts must be between 1 and 4096");
  if (dim < 1 || dim > kMaxDim || inner < 1 || inner > kMaxDim) return refuse("dim and inner must be between 1 and 2^20");
  return DMUON_OK;
}

struct Workspace {
  size_t h, part, arrived, bytes;
};

Workspace workspace_of(int64_t n, int64_t dim, int64_t inner) {
  Workspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  w.h = take(2 * 2 * n * pitch_h(inner));
  w.part = take(4 * n * dim);
  w.arrived = take(4 * ((dim + kRows - 1) / kRows));
  w.bytes = at;
  return w;
}

template <int PHASE, int TILES>
cudaError_t launch(const ExpertsParams& p, bool vec, int grid, cudaStream_t s) {
  return vec ? launch_follow(experts_kernel<PHASE, TILES, true>, dim3(grid), kThreads, 0, s, 1, p)
             : launch_follow(experts_kernel<PHASE, TILES, false>, dim3(grid), kThreads, 0, s, 1, p);
}

template <int PHASE>
cudaError_t launch_tiles(const ExpertsParams& p, bool vec, int sms, cudaStream_t s) {
  const int rows = PHASE == kDown ? p.dim : p.inner, out = PHASE == kGated ? 8 : 16;
  const int64_t units = int64_t(std::min(p.experts, p.n)) * ((rows + out - 1) / out);
  const int grid = static_cast<int>(std::min<int64_t>(units, 2 * sms));
  // as many columns as an expert may get where no token names it twice
  if (p.tokens <= 8) return launch<PHASE, 1>(p, vec, grid, s);
  if (p.tokens <= 16) return launch<PHASE, 2>(p, vec, grid, s);
  return launch<PHASE, 4>(p, vec, grid, s);
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" dmuon_status dmuon_experts_workspace_bytes(int64_t tokens, int32_t top, int32_t experts, int64_t dim,
                                                      int64_t inner, size_t* bytes) {
  if (bytes == nullptr) return refuse("NULL argument");
  dmuon_status st = check_sizes(tokens, top, experts, dim, inner);
  if (st != DMUON_OK) return st;
  *bytes = workspace_of(tokens * top, dim, inner).bytes;
  return set_last_error(DMUON_OK, "");
}

extern "C" dmuon_status dmuon_experts_forward(const void* x, int64_t ld_x, const int64_t* expert_ids, const float* weights,
                                              int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner,
                                              const void* up, const void* gate, const void* down, void* y, int64_t ld_y,
                                              void* d_workspace, size_t bytes, void* stream) {
  dmuon_status st = check_sizes(tokens, top, experts, dim, inner);
  if (st != DMUON_OK) return st;
  if (tokens == 0) return set_last_error(DMUON_OK, "");
  if (x == nullptr || expert_ids == nullptr || weights == nullptr || up == nullptr || down == nullptr || y == nullptr)
    return refuse("NULL pointer argument");
  if (misaligned(expert_ids, 8) || misaligned(weights, 4) || misaligned(x, 2) || misaligned(up, 2) ||
      misaligned(gate, 2) || misaligned(down, 2) || misaligned(y, 2))
    return refuse("a pointer is not aligned to its elements");
  if (ld_x < dim || ld_y < dim || ld_x > (int64_t(1) << 32) || ld_y > (int64_t(1) << 32))
    return refuse("a row pitch is shorter than dim or above 2^32");
  const Workspace w = workspace_of(tokens * top, dim, inner);
  if (d_workspace == nullptr || misaligned(d_workspace, 256) || bytes < w.bytes)
    return set_last_error(DMUON_ERR_WORKSPACE, "workspace is NULL, too small or not 256-byte aligned");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  ExpertsParams p{};
  char* ws = static_cast<char*>(d_workspace);
  p.ids = expert_ids;
  p.weights = weights;
  p.x = static_cast<const bf16*>(x);
  p.ld_x = ld_x;
  p.up = static_cast<const bf16*>(up);
  p.gate = static_cast<const bf16*>(gate);
  p.down = static_cast<const bf16*>(down);
  p.h = reinterpret_cast<bf16*>(ws + w.h);
  p.ld_h = pitch_h(inner);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.arrived = reinterpret_cast<unsigned*>(ws + w.arrived);
  p.y = static_cast<bf16*>(y);
  p.ld_y = ld_y;
  p.tokens = static_cast<int32_t>(tokens);
  p.top = top;
  p.experts = experts;
  p.n = static_cast<int32_t>(tokens * top);
  p.dim = static_cast<int32_t>(dim);
  p.inner = static_cast<int32_t>(inner);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // rows that are whole 16-byte pieces are read so, others element by element
  const bool vec_up = dim % 8 == 0 && ld_x % 8 == 0 && !misaligned(x, 16) && !misaligned(up, 16) && !misaligned(gate, 16);
  const bool vec_down = inner % 8 == 0 && !misaligned(down, 16);
  e = gate != nullptr ? launch_tiles<kGated>(p, vec_up, sms, s) : launch_tiles<kUngated>(p, vec_up, sms, s);
  if (e == cudaSuccess) e = launch_tiles<kDown>(p, vec_down, sms, s);
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  return set_last_error(DMUON_OK, "");
}
