// experts.cu - a mixture's experts for a few tokens (include/dmuon.h, "A mixture's experts for a few
// tokens"): from the router's ids and weights to the layer's output, in two launches.
//
//   h[i] = silu(G_e x_t) * U_e x_t   (without a gate: silu(U_e x_t))     i = t*top + k, e = ids[i]
//   y[t] = sum_k weights[i] * D_e h[i]
//
// Bound by reading the matrices of the experts that the tokens reach, once: a token's products are 1 flop
// for each byte read, 64 tokens' on 64 experts 8.
//
// Rows that are whole 16-byte pieces stream through shared memory: one block per SM, whose ninth warp keeps three or four
// stages of 64 rows by 256 columns on their way by TMA, with the same columns of the expert's tokens, whatever the eight others do. A block owns a contiguous run of the row blocks
// of all experts in use, expert by expert, so that each has the same to read to one row block (16 rows of a matrix: 8
// of gate and the same 8 of up, or 16), and takes up to four of them together, which read the expert's tokens once.
// The eight warps share K. A product's sum may run over K in any order, so that a lane's 16 bytes of a row stand for
// whatever K indices mma.sync gives that lane, for the matrix and the tokens alike: nothing is transposed. mma.sync, as tcgen05 would pad a few tokens' products to 128
// rows that have to be in shared memory in full: the tensor pipe is at a few percent here either way.
// Down's matrices start to stream while the products before still run.
//
// Other rows are read element by element (experts_plain_kernel), every warp straight from memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include <cudaTypedefs.h>

#include "dmuon.h"
#include "follow.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dmuon {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxTop = 64;
constexpr int kMaxExperts = 4096;
constexpr int kMaxAssignments = 2048;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;    // rows of a unit
constexpr int kStep = 32;    // K of a warp's step: 4 lanes of 8 elements
constexpr int kCostRead = 8, kCostTile = 2;
// Streaming
constexpr int kTogether = 4;                     // row blocks taken together
constexpr int kChunk = 64;                       // columns of a TMA box, 128 bytes
constexpr int kBoxBytes = 8 * 2 * kChunk;        // of 8 rows
constexpr int kStageK = 4 * kChunk;              // a step of 32 for each warp
constexpr int kMatrixBytes = 2 * kTogether * 4 * kBoxBytes;
constexpr int kColumnPitch = 2 * kStageK + 16;   // of an assignment's columns: the next one's banks are 16 bytes on
constexpr int kMaxStages = 4;
constexpr int kStreamThreads = kThreads + 32;
constexpr int64_t kWaitNs = 2000000000LL;

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
  unsigned* status;
};

// ... and the matrices as rows of K: gate or down, and up.
struct StreamParams {
  ExpertsParams e;
  CUtensorMap w[2];
};

// What a block knows of the routing: the experts in use in ascending order, and each one's assignments.
struct Routing {
  int16_t active[kMaxAssignments];
  int16_t begin[kMaxAssignments + 1];  // of an expert's assignments in list
  int16_t list[kMaxAssignments];
  int actives;
};
// ... and what it needs to find that out.
struct RoutingScratch {
  int count[kMaxExperts];
  int16_t expert[kMaxAssignments];
};

__device__ __forceinline__ void read_routing(const ExpertsParams& p, Routing& r, RoutingScratch& s) {
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) s.count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
    const int64_t id = p.ids[i];
    const bool in = id >= 0 && id < p.experts;
    s.expert[i] = in ? static_cast<int16_t>(id) : int16_t(-1);
    if (in) atomicAdd(&s.count[id], 1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int actives = 0, at = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + threadIdx.x, n = e < p.experts ? s.count[e] : 0;
      const unsigned used = __ballot_sync(0xffffffffu, n > 0);
      if (used == 0u) continue;
      int before = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (threadIdx.x >= d) before += o;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      if (n > 0) {
        const int place = actives + __popc(used & ((1u << threadIdx.x) - 1u));
        r.active[place] = static_cast<int16_t>(e);
        r.begin[place] = static_cast<int16_t>(at + before - n);
        s.count[e] = at + before - n;
      }
      actives += __popc(used);
      at += all;
    }
    if (threadIdx.x == 0) {
      r.actives = actives;
      r.begin[actives] = static_cast<int16_t>(at);
    }
  }
  __syncthreads();
  // (an expert's assignments in any order: none of their products depends on it)
  for (int i = threadIdx.x; i < p.n; i += blockDim.x)
    if (s.expert[i] >= 0) r.list[atomicAdd(&s.count[s.expert[i]], 1)] = static_cast<int16_t>(i);
  __syncthreads();
}

// 8 elements from column k of a row of `dim`, zeros past its end.
__device__ __forceinline__ uint4 piece(const bf16* row, int k, int dim) {
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

// A product's result: D h of an assignment, or its h from the products with up and gate.
template <int PHASE>
__device__ __forceinline__ void result(const ExpertsParams& p, int assignment, int o, float s, float up) {
  if (PHASE == kDown) {
    p.part[int64_t(assignment) * p.dim + o] = s;
    return;
  }
  const float f = s / (1.f + expf(-s)) * (PHASE == kGated ? up : 1.f);
  // as the sum of two bf16: rounded to one, h would double the squared error of y, whose own rounding is as large
  const bf16 high = __float2bfloat16_rn(f);
  const float rest = fabsf(__bfloat162float(high)) < INFINITY ? f - __bfloat162float(high) : 0.f;
  p.h[assignment * p.ld_h + o] = high;
  p.h[(p.n + assignment) * p.ld_h + o] = __float2bfloat16_rn(rest);
}

// Entries b * 16 .. of y once every expert is done with them: the assignments' products added up in the order of k.
__device__ __forceinline__ void combine(const ExpertsParams& p, int b, int thread) {
  for (int i = thread; i < p.tokens * kRows; i += kThreads) {
    const int t = i / kRows, o = b * kRows + i % kRows;
    if (o >= p.dim) continue;
    float s = 0.f;
    for (int k = 0; k < p.top; ++k) {
      const int q = t * p.top + k;
      const int64_t id = p.ids[q];
      if (id >= 0 && id < p.experts) s = fmaf(p.weights[q], __ldcg(&p.part[int64_t(q) * p.dim + o]), s);
    }
    p.y[t * p.ld_y + o] = __float2bfloat16_rn(s);
  }
}

// y where no expert is named at all, by kThreads of each block.
__device__ __forceinline__ void clear(const ExpertsParams& p) {
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < int64_t(p.tokens) * p.dim;
       i += int64_t(gridDim.x) * kThreads)
    p.y[i / p.dim * p.ld_y + i % p.dim] = __float2bfloat16_rn(0.f);
}

// The first launch clears what the second counts in, and the status.
__device__ __forceinline__ void start(const ExpertsParams& p) {
  const int first = blockIdx.x * blockDim.x + threadIdx.x;
  if (first == 0) *p.status = 0u;
  for (int i = first; i < (p.dim + kRows - 1) / kRows; i += gridDim.x * blockDim.x) p.arrived[i] = 0u;
}

// ------------------------------------------------------------------ element by element
template <int TILES>
struct PlainShared {
  union {
    RoutingScratch scratch;
    float sums[kWarps][TILES][4][32];
  };
  Routing r;
  unsigned last;
};

// Tiles of 8 assignments at a time: TILES.
template <int PHASE, int TILES>
__global__ void __launch_bounds__(kThreads, 2) experts_plain_kernel(const __grid_constant__ ExpertsParams p) {
  extern __shared__ uint8_t raw[];
  PlainShared<TILES>& sh = *reinterpret_cast<PlainShared<TILES>*>(raw);
  const Routing& r = sh.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // The down products' launch is set up while the up products' still runs: what it reads before follow() was
  // there before that launch began.
  if (PHASE != kDown) {
    follow();
    start(p);
  }
  read_routing(p, sh.r, sh.scratch);
  const int K = PHASE == kDown ? p.inner : p.dim;
  const int rows = PHASE == kDown ? p.dim : p.inner;  // of a matrix
  constexpr int kOut = PHASE == kGated ? 8 : 16;      // rows of the result per unit
  const int blocks = (rows + kOut - 1) / kOut;
  const int units = r.actives * blocks;
  if (PHASE == kDown) {
    follow();
    if (units == 0) clear(p);
  }
  const int steps = (K + kStep - 1) / kStep;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = u / blocks, b = u % blocks;
    const int16_t* list = r.list + r.begin[i];
    const int count = r.begin[i + 1] - r.begin[i];
    const int o0 = min(b * kOut + g, rows - 1), o1 = min(b * kOut + g + 8, rows - 1);
    const int64_t matrix = int64_t(r.active[i]) * rows;
    const bf16* w = PHASE == kDown ? p.down : PHASE == kGated ? p.gate : p.up;
    const bf16* row0 = w + (matrix + o0) * K;
    const bf16* row1 = PHASE == kGated ? p.up + (matrix + o0) * K : w + (matrix + o1) * K;
    for (int j0 = 0; j0 < count; j0 += 8 * TILES) {
      const int tiles = min(TILES, (count - j0 + 7) / 8);
      float acc[TILES][4] = {};
      const bf16* col[TILES];  // of x or h, the row that this lane brings; nullptr: none
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int j = j0 + t * 8 + g;
        col[t] = nullptr;
        if (j < count) col[t] = PHASE == kDown ? p.h + list[j] * p.ld_h : p.x + (list[j] / p.top) * p.ld_x;
      }
      for (int s = warp; s < steps; s += kWarps) {
        const int k = s * kStep + 8 * c;
        const uint4 a0 = piece(row0, k, K), a1 = piece(row1, k, K);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (t >= tiles) break;
#pragma unroll
          for (int q = 0; q < (PHASE == kDown ? 2 : 1); ++q) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (col[t] != nullptr) v = piece(col[t] + q * p.n * p.ld_h, k, K);
            mma(acc[t], a0.x, a1.x, a0.y, a1.y, v.x, v.y);
            mma(acc[t], a0.z, a1.z, a0.w, a1.w, v.z, v.w);
          }
        }
      }
      // the warps' sums joined; sums[.][t][v][l] is row l / 4 (+ 8 for v >= 2), column 2 * (l % 4) + v % 2
#pragma unroll
      for (int t = 0; t < TILES; ++t)
        if (t < tiles)
#pragma unroll
          for (int v = 0; v < 4; ++v) sh.sums[warp][t][v][lane] = acc[t][v];
      __syncthreads();
      constexpr int kEach = PHASE == kGated ? 2 : 4;
      for (int n = threadIdx.x; n < tiles * kEach * 32; n += kThreads) {
        const int l = n & 31, v = (n >> 5) % kEach, t = (n >> 5) / kEach;
        const int j = j0 + t * 8 + 2 * (l & 3) + (v & 1);
        const int o = b * kOut + (l >> 2) + (v >= 2 ? 8 : 0);
        if (j >= count || o >= rows) continue;
        float s = 0.f, s1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          s += sh.sums[w][t][v][l];
          if (PHASE == kGated) s1 += sh.sums[w][t][v + 2][l];
        }
        result<PHASE>(p, list[j], o, s, s1);
      }
      __syncthreads();
    }
    if (PHASE == kDown) {
      // the last expert's block to be done with these 16 entries of y adds them up
      if (threadIdx.x == 0) {
        __threadfence();
        sh.last = atomicAdd(&p.arrived[b], 1u) == static_cast<unsigned>(r.actives - 1);
      }
      __syncthreads();
      if (sh.last != 0u) {
        __threadfence();
        combine(p, b, threadIdx.x);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ streaming
// A stage holds 64 rows by 256 columns of matrices and the same columns of the assignments' rows, which of h are two.
struct StreamShared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort_flag;
  int from, to;                    // the block's row blocks
  unsigned last[kTogether];
  Routing r;
  float sums[kWarps][kTogether][4][32];
};
constexpr int kRoom = 227 * 1024 - 1024 - static_cast<int>(sizeof(StreamShared));
__host__ __device__ constexpr int stage_bytes(int tiles, bool down) {
  return (kMatrixBytes + (down ? 2 : 1) * tiles * 8 * kColumnPitch + 1023) / 1024 * 1024;
}
__host__ __device__ constexpr int stages_of(int tiles, bool down) {
  return kRoom / stage_bytes(tiles, down) < kMaxStages ? kRoom / stage_bytes(tiles, down) : kMaxStages;
}
__host__ __device__ constexpr size_t stream_smem(int tiles, bool down) {
  return 1024 + stages_of(tiles, down) * stage_bytes(tiles, down) + sizeof(StreamShared);
}
static_assert(stages_of(4, true) >= 3 && sizeof(RoutingScratch) <= 3 * kMatrixBytes, "one block's shared memory");

// What a row block of an expert takes: reading it, and the products with its assignments, 8 at a time. (Measured: a
// block's time by the number of assignments, 64 rows by 2048: see the launch.)
__device__ __forceinline__ int cost_of(int assignments) { return kCostRead + (assignments + 7) / 8 * kCostTile; }

// Cuts the row blocks of all experts in use into one run for each block of the grid, of equal cost. By one warp.
__device__ __forceinline__ int cut(const Routing& r, int blocks, int64_t part, int64_t parts, int lane) {
  int64_t total = 0;
  for (int i0 = 0; i0 < r.actives; i0 += 32) {
    const int i = i0 + lane;
    total += __reduce_add_sync(0xffffffffu, i < r.actives ? cost_of(r.begin[i + 1] - r.begin[i]) : 0);
  }
  int64_t want = total * blocks * part / parts;  // cost before the cut
  for (int i0 = 0; i0 < r.actives; i0 += 32) {
    const int i = i0 + lane, mine = i < r.actives ? cost_of(r.begin[i + 1] - r.begin[i]) : 0;
    int before = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    const int64_t all = int64_t(__shfl_sync(0xffffffffu, before, 31)) * blocks;
    if (want > all) {
      want -= all;
      continue;
    }
    // the lane whose expert the cut falls into: the first that reaches it
    const unsigned reach = __ballot_sync(0xffffffffu, i < r.actives && int64_t(before) * blocks >= want);
    const int l = __ffs(reach) - 1;
    const int64_t rest = want - int64_t(before - mine) * blocks;
    const int block = mine > 0 ? static_cast<int>((rest + mine - 1) / mine) : 0;
    return (i0 + l) * blocks + __shfl_sync(0xffffffffu, block, l);
  }
  return r.actives * blocks;
}

// A block's run of row blocks, as many at a time as one expert has in it, at most kTogether.
struct Job {
  int unit, end, blocks;
  int active, first, rows;  // the expert's place among those in use, its first row block, how many
  __device__ __forceinline__ bool next() {
    unit += rows;
    if (unit >= end) return false;
    active = unit / blocks;
    first = unit - active * blocks;
    rows = min(min(kTogether, blocks - first), end - unit);
    return true;
  }
};

// The stages that a block fills, one after another: its jobs, 8 * TILES assignments at a time, 256 columns at a time.
template <int TILES>
struct Fills {
  Job job;
  const Routing* r;
  int nk, assignments, j0, kb;
  __device__ __forceinline__ bool next() {
    if (job.rows > 0) {
      if (++kb < nk) return true;
      kb = 0;
      if ((j0 += 8 * TILES) < assignments) return true;
    }
    if (!job.next()) return false;
    assignments = r->begin[job.active + 1] - r->begin[job.active];
    j0 = kb = 0;
    return true;
  }
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void tma_load_2d(void* dst, const void* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// `bytes` (a multiple of 16) from global to shared memory, both on 16 bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

template <int PHASE, int TILES>
__global__ void __launch_bounds__(kStreamThreads, 1) experts_stream_kernel(const __grid_constant__ StreamParams sp) {
  constexpr bool down = PHASE == kDown;
  constexpr int kStages = stages_of(TILES, down), kStageBytes = stage_bytes(TILES, down), kParts = down ? 2 : 1;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  StreamShared& sh = *reinterpret_cast<StreamShared*>(base + kStages * kStageBytes);
  const ExpertsParams& p = sp.e;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abortf = &sh.abort_flag;
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      ptx::mbar_init(&sh.full[k], 1);
      ptx::mbar_init(&sh.empty[k], kWarps);
    }
    sh.abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&sp.w[0]);
    if (PHASE == kGated) ptx::prefetch_tmap(&sp.w[1]);
  }
  // The down products' launch is set up while the up products' still runs: what it reads before follow() was
  // there before that launch began.
  if (!down) {
    follow();
    start(p);
  }
  read_routing(p, sh.r, *reinterpret_cast<RoutingScratch*>(base));
  const int K = down ? p.inner : p.dim;
  const int rows = down ? p.dim : p.inner;
  constexpr int kOut = PHASE == kGated ? 8 : 16;
  const int blocks = (rows + kOut - 1) / kOut;
  if (warp < 2) {
    const int at = cut(sh.r, blocks, blockIdx.x + warp, gridDim.x, lane);
    if (lane == 0) (warp == 0 ? sh.from : sh.to) = at;
  }
  ptx::fence_proxy_async_shared();  // the scratch's place is the ring's
  __syncthreads();
  const int nk = (K + kStageK - 1) / kStageK;
  Job job;
  job.unit = sh.from;
  job.end = sh.to;
  job.blocks = blocks;
  job.rows = 0;
  uint32_t stage = 0, phase = 0;

  if (warp == kWarps) {
    // ---------------------------------------------------------- loads
    uint32_t fills = 0;
    Fills<TILES> f;
    f.job = job;
    f.r = &sh.r;
    f.nk = nk;
    // A stage's matrices: a box of 8 rows by 64 columns each lane. Gated, groups 0..3 are gate's rows and 4..7 up's; else
    // the 16 rows of a row block are two groups.
    const int group = lane >> 2, chunk = lane & 3, half = PHASE == kGated ? group & 3 : group;
    const CUtensorMap* map = PHASE == kGated && group >= 4 ? &sp.w[1] : &sp.w[0];
    auto matrices = [&](const Fills<TILES>& f, uint32_t stage) {
      const int x = f.kb * kStageK, wide = min(kStageK, K - x), chunks = (wide + kChunk - 1) / kChunk;
      const int columns = min(8 * TILES, f.assignments - f.j0);
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * f.job.rows * chunks * kBoxBytes + kParts * columns * 2 * wide);
      __syncwarp();
      if (half < (PHASE == kGated ? f.job.rows : 2 * f.job.rows) && chunk < chunks)
        tma_load_2d(base + stage * kStageBytes + (group * 4 + chunk) * kBoxBytes, map, &sh.full[stage], x + chunk * kChunk,
                    sh.r.active[f.job.active] * rows + f.job.first * kOut + 8 * half);
    };
    // ... and the assignments' columns: a row each lane, of h in two parts.
    auto columns = [&](const Fills<TILES>& f, uint32_t stage) {
      if (lane >= min(8 * TILES, f.assignments - f.j0)) return;
      const int x = f.kb * kStageK, wide = min(kStageK, K - x);
      const int i = sh.r.list[sh.r.begin[f.job.active] + f.j0 + lane];
      const bf16* row = (down ? p.h + i * p.ld_h : p.x + (i / p.top) * p.ld_x) + x;
      uint8_t* at = base + stage * kStageBytes + kMatrixBytes + lane * kColumnPitch;
      for (int q = 0; q < kParts; ++q)
        bulk_load(at + q * 8 * TILES * kColumnPitch, row + q * p.n * p.ld_h, 2 * wide, &sh.full[stage]);
    };
    // the first stages' matrices need not wait for the launch before, which makes h
    const Fills<TILES> first = f;
    bool more = true;
    while (fills < kStages && (more = f.next())) matrices(f, fills++);
    if (down) follow();
    Fills<TILES> again = first;
    for (uint32_t k = 0; k < fills; ++k) {
      again.next();
      columns(again, k);
    }
    // from the first stage on again, each once its last load has been used
    while (more && (more = f.next())) {
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sh.empty[stage], phase, abortf, p.status, kWaitNs))) break;
      matrices(f, stage);
      columns(f, stage);
      ++fills;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // nothing is in flight once every stage that was filled is full
    for (uint32_t k = 0; k < kStages; ++k)
      if (fills > k) {
        int zero = 0;
        ptx::mbar_wait(&sh.full[k], ((fills - 1u - k) / kStages) & 1u, &zero, p.status, kWaitNs);
      }
    return;
  }

  // ------------------------------------------------------------ products
  if (down) {
    follow();
    if (sh.r.actives == 0) clear(p);
  }
  const int g = lane >> 2, c = lane & 3;
  // this warp's 32 columns of a stage: pieces 2c + (warp & 1) of chunk warp / 2, which no two lanes of a quarter warp
  // have in the same banks, of the swizzled rows as of the assignments' columns
  const uint32_t at = (warp >> 1) * kBoxBytes + g * 128 + (((2 * c + (warp & 1)) ^ g) << 4);
  const uint32_t of_column = kMatrixBytes + g * kColumnPitch + (warp >> 1) * 128 + ((2 * c + (warp & 1)) << 4);
  bool alive = true;
  while (job.next()) {
    const int16_t* list = sh.r.list + sh.r.begin[job.active];
    const int count = sh.r.begin[job.active + 1] - sh.r.begin[job.active];
    for (int j0 = 0; j0 < count; j0 += 8 * TILES) {
      const int tiles = min(TILES, (count - j0 + 7) / 8);
      float acc[kTogether][TILES][4] = {};
      for (int kb = 0; kb < nk; ++kb) {
        // (after a wait that ran out of time a warp only keeps the others' barriers company)
        if (alive) alive = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.full[stage], phase, abortf, p.status, kWaitNs));
        if (alive && kb * kStageK + (warp >> 1) * kChunk < K) {
          const uint8_t* s = base + stage * kStageBytes;
          // zeros for what the matrix has past its last column: there, and in columns of no assignment, the stage
          // holds what an earlier one left
          const bool inside = kb * kStageK + (warp >> 1) * kChunk + 16 * c + 8 * (warp & 1) < K;
          uint4 v[kParts][TILES];
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int t = 0; t < TILES; ++t)
              v[q][t] = inside && j0 + t * 8 + g < count
                            ? *reinterpret_cast<const uint4*>(s + of_column + (q * TILES + t) * 8 * kColumnPitch)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kTogether; ++i) {
            if (i >= job.rows) break;
            const uint4 a0 = *reinterpret_cast<const uint4*>(s + at + (PHASE == kGated ? i : 2 * i) * 4 * kBoxBytes);
            const uint4 a1 =
                *reinterpret_cast<const uint4*>(s + at + (PHASE == kGated ? i + 4 : 2 * i + 1) * 4 * kBoxBytes);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              if (t >= tiles) break;
#pragma unroll
              for (int q = 0; q < kParts; ++q) {
                mma(acc[i][t], a0.x, a1.x, a0.y, a1.y, v[q][t].x, v[q][t].y);
                mma(acc[i][t], a0.z, a1.z, a0.w, a1.w, v[q][t].z, v[q][t].w);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.empty[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the warps' sums joined; sums[.][i][v][l] is row l / 4 (+ 8 for v >= 2), column 2 * (l % 4) + v % 2
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        if (t >= tiles) break;
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) sh.sums[warp][i][k][lane] = acc[i][t][k];
        consumers_sync();
        constexpr int kEach = PHASE == kGated ? 2 : 4;
        for (int n = threadIdx.x; n < job.rows * kEach * 32; n += kThreads) {
          const int l = n & 31, k = (n >> 5) % kEach, i = (n >> 5) / kEach;
          const int j = j0 + t * 8 + 2 * (l & 3) + (k & 1);
          const int o = (job.first + i) * kOut + (l >> 2) + (k >= 2 ? 8 : 0);
          if (j >= count || o >= rows) continue;
          float s = 0.f, s1 = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            s += sh.sums[w][i][k][l];
            if (PHASE == kGated) s1 += sh.sums[w][i][k + 2][l];
          }
          result<PHASE>(p, list[j], o, s, s1);
        }
        consumers_sync();
      }
    }
    if (down) {
      // the last expert's block to be done with 16 entries of y adds them up
      if (threadIdx.x < job.rows) {
        __threadfence();
        sh.last[threadIdx.x] = atomicAdd(&p.arrived[job.first + threadIdx.x], 1u) == static_cast<unsigned>(sh.r.actives - 1);
      }
      consumers_sync();
      for (int i = 0; i < job.rows; ++i)
        if (sh.last[i] != 0u) {
          __threadfence();
          combine(p, job.first + i, threadIdx.x);
        }
      consumers_sync();
    }
  }
}

dmuon_status refuse(const char* msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int64_t pitch_h(int64_t inner) { return (inner + 7) / 8 * 8; }

dmuon_status check_sizes(int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner) {
  if (top < 1 || top > kMaxTop) return refuse("top must be between 1 and 64");
  if (tokens < 0 || tokens * top > kMaxAssignments || tokens > kMaxAssignments)
    return refuse("tokens * top must be between 0 and 2048 (for more: sort, dispatch, the experts' products, combine)");
  if (experts < 1 || experts > kMaxExperts) return refuse("experts must be between 1 and 4096");
  if (dim < 1 || dim > kMaxDim || inner < 1 || inner > kMaxDim) return refuse("dim and inner must be between 1 and 2^20");
  if (experts * std::max(dim, inner) > (int64_t(1) << 30)) return refuse("experts * dim and experts * inner must not be above 2^30");
  return DMUON_OK;
}

struct Workspace {
  size_t status, h, part, arrived, bytes;
};

Workspace workspace_of(int64_t n, int64_t dim, int64_t inner) {
  Workspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  w.status = take(4);
  w.h = take(2 * 2 * n * pitch_h(inner));
  w.part = take(4 * n * dim);
  w.arrived = take(4 * ((dim + kRows - 1) / kRows));
  w.bytes = at;
  return w;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Matrices as rows of K, in boxes of 8 rows by 64 columns; past the last column or row a box has zeros.
cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t K, int64_t rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
  const cuuint32_t box[2] = {kChunk, 8}, one[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int PHASE, int TILES>
cudaError_t launch(const ExpertsParams& p, bool stream, int sms, cudaStream_t s) {
  const int rows = PHASE == kDown ? p.dim : p.inner, K = PHASE == kDown ? p.inner : p.dim;
  const int out = PHASE == kGated ? 8 : 16;
  const int64_t units = int64_t(std::min(p.experts, p.n)) * ((rows + out - 1) / out);
  cudaError_t e;
  if (!stream) {
    e = cudaFuncSetAttribute(experts_plain_kernel<PHASE, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(PlainShared<TILES>)));
    if (e != cudaSuccess) return e;
    return launch_follow(experts_plain_kernel<PHASE, TILES>, dim3(static_cast<unsigned>(std::min<int64_t>(units, 2 * sms))),
                         kThreads, sizeof(PlainShared<TILES>), s, 1, p);
  }
  constexpr size_t smem = stream_smem(TILES, PHASE == kDown);
  StreamParams sp;
  sp.e = p;
  const bf16* w = PHASE == kGated ? p.gate : PHASE == kUngated ? p.up : p.down;
  e = map_rows(&sp.w[0], w, K, int64_t(p.experts) * rows);
  if (e == cudaSuccess) e = map_rows(&sp.w[1], PHASE == kGated ? p.up : w, K, int64_t(p.experts) * rows);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(experts_stream_kernel<PHASE, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_follow(experts_stream_kernel<PHASE, TILES>, dim3(static_cast<unsigned>(std::min<int64_t>(units, sms))),
                       kStreamThreads, smem, s, 1, sp);
}

template <int PHASE>
cudaError_t launch_tiles(const ExpertsParams& p, bool stream, int sms, cudaStream_t s) {
  // as many columns as an expert may get where no token names it twice
  if (p.tokens <= 8) return launch<PHASE, 1>(p, stream, sms, s);
  if (p.tokens <= 16) return launch<PHASE, 2>(p, stream, sms, s);
  return launch<PHASE, 4>(p, stream, sms, s);
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
  p.status = reinterpret_cast<unsigned*>(ws + w.status);
  p.y = static_cast<bf16*>(y);
  p.ld_y = ld_y;
  p.tokens = static_cast<int32_t>(tokens);
  p.top = top;
  p.experts = experts;
  p.n = static_cast<int32_t>(tokens * top);
  p.dim = static_cast<int32_t>(dim);
  p.inner = static_cast<int32_t>(inner);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // rows that are whole 16-byte pieces stream, others are read element by element
  const bool vec_up = dim % 8 == 0 && ld_x % 8 == 0 && !misaligned(x, 16) && !misaligned(up, 16) && !misaligned(gate, 16);
  const bool vec_down = inner % 8 == 0 && !misaligned(down, 16);
  e = gate != nullptr ? launch_tiles<kGated>(p, vec_up, sms, s) : launch_tiles<kUngated>(p, vec_up, sms, s);
  if (e == cudaSuccess) e = launch_tiles<kDown>(p, vec_down, sms, s);
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  return set_last_error(DMUON_OK, "");
}

extern "C" dmuon_status dmuon_experts_read_device_status(const void* d_workspace, void* stream, uint32_t* bits) {
  if (d_workspace == nullptr || bits == nullptr) return refuse("NULL argument");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, d_workspace, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return set_last_error(DMUON_ERR_CUDA, cudaGetErrorString(e));
  *bits = word;
  return set_last_error(DMUON_OK, "");
}
