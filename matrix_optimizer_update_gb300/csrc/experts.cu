// experts.cu - a mixture's experts for a few tokens (include/dmuon.h, "A mixture's experts for a few
// tokens"): from the router's ids and weights to the layer's output, in three launches.
//
//   h[i] = silu(G_e x_t) * U_e x_t   (without a gate: silu(U_e x_t))     i = t*top + k, e = ids[i]
//   y[t] = sum_k weights[i] * D_e h[i]
//
// Bound by reading the matrices of the experts that the tokens reach, once: a token's products are 1 flop
// for each byte read, 64 tokens' on 64 experts 8.
//
// Rows that are whole 16-byte pieces stream through shared memory: one block per SM, whose ninth warp keeps six
// stages of 64 rows by 256 columns on their way by TMA, whatever the eight others do. (Every warp loading its own
// rows straight into registers took 48 us for one token to 8 of 64, 2048 x 1408, and 454 for 64 tokens; this takes 34.4
// and 198, of which the matrices at the copy rate are 20 and 164.)
//
// A block owns a contiguous run of the row blocks of all experts in use, expert by expert, of the same cost to one
// row block (16 rows of a matrix: 8 of gate and the same 8 of up, or 16), and takes up to four of them together, which
// read the expert's tokens once. Four warps have the even stages and four the odd, each 64 of the columns. Down's
// blocks start to read the routing while the products before still run; to have them beside up's on an SM, with half
// its shared memory each, took 36.5 us in place of 35.1, and 81 in place of 72 for 7 tokens without a gate.
//
// A product's sum may run over K in any order, so that a lane's 16 bytes of a row stand for whatever K indices
// mma.sync gives that lane, for the matrix and the tokens alike: nothing is transposed. mma.sync, as tcgen05 wants the
// tokens' rows, gathered anew for each expert, in shared memory in a layout of its own: with 64 tokens the tensor pipe
// is at 13 % (up) and 23 % (down) of its cycles, and up to 8 assignments to an expert cost no more than one.
//
// Other rows are read element by element (experts_plain_kernel), every warp straight from memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
constexpr int kStep = 32;    // K of a warp's step: 4 lanes of 8 elements
// Streaming
constexpr int kMostTiles = 3;  // of 8 assignments in a pass: with four, what a lane holds no longer fits its registers
constexpr int kTogether = 4;                     // row blocks taken together
constexpr int kChunk = 64;                       // columns of a TMA box, 128 bytes
constexpr int kBoxBytes = 8 * 2 * kChunk;        // of 8 rows
constexpr int kStageK = 4 * kChunk;              // a chunk for each of four warps
constexpr int kStageBytes = 2 * kTogether * 4 * kBoxBytes;
constexpr int kStages = 6;                       // even: four warps have the even ones, four the odd
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
  bf16* h;             // [assignments][ld_h / 8][2][8]: h as the sum of two bf16, eight of the first, then of the second
  int64_t ld_h;
  float* part;         // [assignments][dim]: D_e h, not yet weighted
  bf16* y;
  int64_t ld_y;
  int32_t tokens, top, experts, n;  // n = tokens * top
  int32_t dim, inner;
  unsigned* status;
};

// ... and the matrices as rows of K (gate or down, and up), in boxes of 1, 2 and 4 row blocks.
struct StreamParams {
  ExpertsParams e;
  CUtensorMap boxes[2][3];
  uint64_t share;  // 2^64 / the grid, rounded up (not used where that is one)
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
  bf16* h = p.h + assignment * 2 * p.ld_h + (o >> 3) * 16 + (o & 7);
  h[0] = high;
  h[8] = __float2bfloat16_rn(rest);
}

// y: the assignments' products added up in the order of k, each once its weight has been multiplied in fp32.
__global__ void __launch_bounds__(kThreads) experts_combine_kernel(const __grid_constant__ ExpertsParams p) {
  follow();
  const int64_t all = int64_t(p.tokens) * p.dim;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < all; i += int64_t(gridDim.x) * kThreads) {
    const int64_t t = i / p.dim;
    const int o = static_cast<int>(i - t * p.dim);
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < p.top; ++k) {
      const int64_t q = t * p.top + k, id = p.ids[q];
      if (id >= 0 && id < p.experts) s = fmaf(p.weights[q], p.part[q * p.dim + o], s);
    }
    p.y[t * p.ld_y + o] = __float2bfloat16_rn(s);
  }
}

// ------------------------------------------------------------------ element by element
constexpr int kPlainTiles = 2;  // tiles of 8 assignments at a time
struct PlainShared {
  union {
    RoutingScratch scratch;
    float sums[kWarps][kPlainTiles][4][32];
  };
  Routing r;
};

template <int PHASE>
__global__ void __launch_bounds__(kThreads, 2) experts_plain_kernel(const __grid_constant__ ExpertsParams p) {
  extern __shared__ uint8_t raw[];
  PlainShared& sh = *reinterpret_cast<PlainShared*>(raw);
  const Routing& r = sh.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  // The down products' launch is set up while the up products' still runs: what it reads before follow() was
  // there before that launch began.
  if (PHASE != kDown) {
    follow();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  }
  read_routing(p, sh.r, sh.scratch);
  const int K = PHASE == kDown ? p.inner : p.dim;
  const int rows = PHASE == kDown ? p.dim : p.inner;  // of a matrix
  constexpr int kOut = PHASE == kGated ? 8 : 16;      // rows of the result per unit
  const int blocks = (rows + kOut - 1) / kOut;
  const int units = r.actives * blocks;
  if (PHASE == kDown) follow();
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
    for (int j0 = 0; j0 < count; j0 += 8 * kPlainTiles) {
      const int tiles = min(kPlainTiles, (count - j0 + 7) / 8);
      float acc[kPlainTiles][4] = {};
      const bf16* col[kPlainTiles];  // of x or h, the row that this lane brings; nullptr: none
#pragma unroll
      for (int t = 0; t < kPlainTiles; ++t) {
        const int j = j0 + t * 8 + g;
        col[t] = nullptr;
        if (j < count) col[t] = PHASE == kDown ? p.h + list[j] * 2 * p.ld_h : p.x + (list[j] / p.top) * p.ld_x;
      }
      for (int s = warp; s < steps; s += kWarps) {
        const int k = s * kStep + 8 * c;
        const uint4 a0 = piece(row0, k, K), a1 = piece(row1, k, K);
#pragma unroll
        for (int t = 0; t < kPlainTiles; ++t) {
          if (t >= tiles) break;
#pragma unroll
          for (int q = 0; q < (PHASE == kDown ? 2 : 1); ++q) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (col[t] != nullptr) v = PHASE == kDown ? piece(col[t] + 2 * k + 8 * q, 0, K - k) : piece(col[t], k, K);
            mma(acc[t], a0.x, a1.x, a0.y, a1.y, v.x, v.y);
            mma(acc[t], a0.z, a1.z, a0.w, a1.w, v.z, v.w);
          }
        }
      }
      // the warps' sums joined; sums[.][t][v][l] is row l / 4 (+ 8 for v >= 2), column 2 * (l % 4) + v % 2
#pragma unroll
      for (int t = 0; t < kPlainTiles; ++t)
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
  }
}

// ------------------------------------------------------------------ streaming
struct StreamShared {
  uint64_t full[kStages], empty[kStages];
  int abort_flag;
  int from, to;                    // the block's row blocks
  Routing r;
  float sums[kWarps][kTogether][4][32];
};
constexpr size_t kStreamSmem = 1024 + kStages * kStageBytes + sizeof(StreamShared);
static_assert(kStreamSmem <= 227 * 1024 && sizeof(RoutingScratch) <= kStages * kStageBytes, "one block's shared memory");

// What a row block of an expert takes, to within some percent: the time of 64 rows by 2048 (gated), and of 64 by 1408
// (down), for 1, 8, 16, 24 and 32 assignments to each of 64 experts, was 117, 119, 126, 136 and 217 us, and 61, 64, 79,
// 100 and 152 us. (Past 24 there is a second pass, whose matrices come out of L2.) With experts of many sizes the small
// ones' blocks leave bandwidth to the others': 64 tokens to 8 of 64 unequally liked take 249 us with costs of 8 + 2 for
// each tile, 205 with costs in proportion to those times, 199 with these.
template <bool DOWN>
__device__ __forceinline__ int cost_of(int assignments) {
  const int tiles = (assignments + 7) / 8, passes = (tiles + kMostTiles - 1) / kMostTiles;
  return DOWN ? 8 * passes + 4 * tiles : 16 * passes + 3 * tiles;
}

// Cuts the row blocks of all experts in use into one run for each block of the grid, of equal cost: where number `part`
// starts. `share` is 2^64 / the grid, rounded up, for grids of more than one. By one warp. (Divisions in 64 bits took
// 0.3 us before each launch's first load.)
template <bool DOWN>
__device__ __forceinline__ int cut(const Routing& r, int blocks, unsigned part, uint64_t share, int lane) {
  if (part == 0 || part == gridDim.x) return part == 0 ? 0 : r.actives * blocks;
  unsigned total = 0;
  for (int i0 = 0; i0 < r.actives; i0 += 32) {
    const int i = i0 + lane;
    total += __reduce_add_sync(0xffffffffu, i < r.actives ? cost_of<DOWN>(r.begin[i + 1] - r.begin[i]) : 0);
  }
  // cost before the cut (total * blocks is below 2^33)
  int64_t want = static_cast<int64_t>(__umul64hi(uint64_t(total) * blocks * part, share));
  for (int i0 = 0; i0 < r.actives; i0 += 32) {
    const int i = i0 + lane, mine = i < r.actives ? cost_of<DOWN>(r.begin[i + 1] - r.begin[i]) : 0;
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
    const unsigned rest = static_cast<unsigned>(want - int64_t(before - mine) * blocks);  // on that lane, mine * blocks at most
    const int block = mine > 0 ? static_cast<int>((rest + mine - 1u) / static_cast<unsigned>(mine)) : 0;
    return (i0 + l) * blocks + __shfl_sync(0xffffffffu, block, l);
  }
  return r.actives * blocks;
}

// A block's run of row blocks, those of an expert in jobs of at most kTogether.
struct Job {
  int unit, end, blocks;
  int active, first, rows;  // the expert's place among those in use, its first row block, how many
  __device__ __forceinline__ bool next() {
    unit += rows;
    if (unit >= end) return false;
    active = unit / blocks;
    first = unit - active * blocks;
    // what the run has of this expert in as few jobs as possible, of about the same size
    const int left = min(blocks - first, end - unit), jobs = (left + kTogether - 1) / kTogether;
    rows = (left + jobs - 1) / jobs;
    return true;
  }
};

// What a block does, one after another: its jobs, 8 * MOST assignments at a time.
template <int MOST>
struct Passes {
  Job job;
  const Routing* r;
  int assignments, j0;
  __device__ __forceinline__ bool next() {
    if (job.rows > 0 && (j0 += 8 * MOST) < assignments) return true;
    if (!job.next()) return false;
    assignments = r->begin[job.active + 1] - r->begin[job.active];
    j0 = 0;
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

// Where a warp of the products is: its next stage.
struct Ring {
  uint8_t* base;
  uint32_t stage, phase;
  bool alive;
};

// 32 bytes, on 32 bytes.
__device__ __forceinline__ void load_32(uint4& a, uint4& b, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}

// Stages (of its own) that a warp's pieces of the assignments are fetched ahead of their use, and what a lane holds of
// them: of x 16 columns to a tile and stage, of h the same twice.
__host__ __device__ constexpr int ahead(int tiles) { return tiles == 1 ? 3 : 1; }
template <int PHASE>
struct Pieces {
  static constexpr int kParts = PHASE == kDown ? 2 : 1;
  uint4 v[3][2][kParts];        // [stages ahead * tiles][which 8 columns][part]
  const bf16* col[kMostTiles];  // rows of x or h, from this lane's first column; nullptr: none

  // `left` columns of the row are left from col on.
  template <int T>
  __device__ __forceinline__ void fetch(int d, int kb, int left) {
    const int k = kb * kStageK;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4(&w)[kParts] = v[d * T + t][half];
        const bool in = col[t] != nullptr && k + 8 * half < left;
#pragma unroll
        for (int q = 0; q < kParts; ++q) w[q] = make_uint4(0, 0, 0, 0);
        if (in) {
          if (PHASE == kDown) load_32(w[0], w[kParts - 1], col[t] + 2 * (k + 8 * half));
          else w[0] = *reinterpret_cast<const uint4*>(col[t] + k + 8 * half);
        }
      }
  }

  // A pass's first ones, from K block kb on.
  template <int T>
  __device__ __forceinline__ void start(const ExpertsParams& p, const int16_t* list, int assignments, int kb, int column,
                                        int left) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int j = t * 8 + g;
      col[t] = nullptr;
      if (j < assignments)
        col[t] = PHASE == kDown ? p.h + list[j] * 2 * p.ld_h + 2 * column : p.x + (list[j] / p.top) * p.ld_x + column;
    }
#pragma unroll
    for (int d = 0; d < ahead(T); ++d) fetch<T>(d, kb + 2 * d, left);
  }
};

// One pass with T tiles of 8 assignments: `assignments` from list on, the row blocks of the job; this warp has every
// other K block from kb on. `then` is called once the matrices have been multiplied, before the sums are joined.
template <int PHASE, int T, class Then>
__device__ __forceinline__ void products(const ExpertsParams& p, StreamShared& sh, Ring& ring, Pieces<PHASE>& x, const Job& job,
                                         const int16_t* list, int assignments, int kb, int K, int rows, int left, uint32_t at,
                                         Then&& then) {
  constexpr int kParts = Pieces<PHASE>::kParts, kAhead = ahead(T), kOut = PHASE == kGated ? 8 : 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nk = (K + kStageK - 1) / kStageK;
  float acc[kTogether][T][4] = {};
  for (; kb < nk; kb += 2 * kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int now = kb + 2 * d;
      if (now >= nk) break;
      // (after a wait that ran out of time a warp only keeps the others' barriers company)
      if (ring.alive)
        ring.alive = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.full[ring.stage], ring.phase, &sh.abort_flag, p.status, kWaitNs));
      // (a stage has room for all row blocks: what it holds of those that the job has not is multiplied and not used)
      if (ring.alive && now * kStageK + (warp & 3) * kChunk < K) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* s = ring.base + ring.stage * kStageBytes + (at ^ (half << 4));
#pragma unroll
          for (int i0 = 0; i0 < kTogether; i0 += 2) {
            uint4 a[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              a[i][0] = *reinterpret_cast<const uint4*>(s + (PHASE == kGated ? i0 + i : 2 * (i0 + i)) * kBoxBytes);
              a[i][1] = *reinterpret_cast<const uint4*>(s + (PHASE == kGated ? i0 + i + 4 : 2 * (i0 + i) + 1) * kBoxBytes);
            }
#pragma unroll
            for (int q = 0; q < kParts; ++q)
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const uint4& v = x.v[d * T + t][half][q];
                    if (part == 0) mma(acc[i0 + i][t], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, v.x, v.y);
                    else mma(acc[i0 + i][t], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, v.z, v.w);
                  }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.empty[ring.stage]);
      if ((ring.stage += 2) >= kStages) {
        ring.stage -= kStages;
        ring.phase ^= 1u;
      }
      if (now + 2 * kAhead < nk) x.template fetch<T>(d, now + 2 * kAhead, left);
    }
  }
  then();
  // the warps' sums joined; sums[.][i][v][l] is row l / 4 (+ 8 for v >= 2), column 2 * (l % 4) + v % 2
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sh.sums[warp][i][k][lane] = acc[i][t][k];
    consumers_sync();
    constexpr int kEach = PHASE == kGated ? 2 : 4;
    for (int n = threadIdx.x; n < job.rows * kEach * 32; n += kThreads) {
      const int l = n & 31, k = (n >> 5) % kEach, i = (n >> 5) / kEach;
      const int j = t * 8 + 2 * (l & 3) + (k & 1);
      const int o = (job.first + i) * kOut + (l >> 2) + (k >= 2 ? 8 : 0);
      if (j >= assignments || o >= rows) continue;
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

template <int PHASE, int MOST>
__global__ void __launch_bounds__(kStreamThreads, 1) experts_stream_kernel(const __grid_constant__ StreamParams sp) {
  constexpr bool down = PHASE == kDown;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  StreamShared& sh = *reinterpret_cast<StreamShared*>(base + kStages * kStageBytes);
  const ExpertsParams& p = sp.e;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abortf = &sh.abort_flag;
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      ptx::mbar_init(&sh.full[k], 1);
      ptx::mbar_init(&sh.empty[k], kWarps / 2);
    }
    sh.abort_flag = 0;
    ptx::fence_mbar_init();
    for (int k = 0; k < 3; ++k) {
      ptx::prefetch_tmap(&sp.boxes[0][k]);
      if (PHASE == kGated) ptx::prefetch_tmap(&sp.boxes[1][k]);
    }
  }
  // The down products' launch is set up while the up products' still runs: what it reads before follow() was
  // there before that launch began.
  if (!down) {
    follow();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  }
  read_routing(p, sh.r, *reinterpret_cast<RoutingScratch*>(base));
  const int K = down ? p.inner : p.dim;
  const int rows = down ? p.dim : p.inner;
  constexpr int kOut = PHASE == kGated ? 8 : 16;
  const int blocks = (rows + kOut - 1) / kOut;
  if (warp < 2) {
    const int at = cut<down>(sh.r, blocks, blockIdx.x + warp, sp.share, lane);
    if (lane == 0) (warp == 0 ? sh.from : sh.to) = at;
  }
  ptx::fence_proxy_async_shared();  // the scratch's place is the ring's
  __syncthreads();
  const int nk = (K + kStageK - 1) / kStageK;
  Passes<MOST> pass;
  pass.job.unit = sh.from;
  pass.job.end = sh.to;
  pass.job.blocks = blocks;
  pass.job.rows = 0;
  pass.r = &sh.r;
  uint32_t stage = 0, phase = 0;

  if (warp == kWarps) {
    // ---------------------------------------------------------- loads
    // A stage: for each chunk of 64 columns 64 rows (gated, 32 of gate and then 32 of up). A lane to a chunk and kind,
    // and for three row blocks another to the third.
    uint32_t fills = 0;
    constexpr int kKinds = PHASE == kGated ? 2 : 1;
    bool ok = true;
    while (ok && pass.next()) {
      const Job& job = pass.job;
      const int y = sh.r.active[job.active] * rows + job.first * kOut;
      for (int kb = 0; kb < nk; ++kb) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh.empty[stage], phase ^ 1u, abortf, p.status, kWaitNs));
        if (!ok) break;
        const int x = kb * kStageK, chunks = min(4, (K - x + kChunk - 1) / kChunk);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * job.rows * chunks * kBoxBytes);
        __syncwarp();
        uint8_t* at = base + stage * kStageBytes;
        const int chunk = lane & 3, kind = (lane >> 2) % kKinds, third = lane / (4 * kKinds);
        if (chunk < chunks && third <= (job.rows == 3)) {
          const int size = third != 0 ? 0 : job.rows == kTogether ? 2 : job.rows >= 2 ? 1 : 0;
          constexpr int kBoxRows = PHASE == kGated ? 8 : 16;  // of a row block
          tma_load_2d(at + chunk * 8 * kBoxBytes + kind * 4 * kBoxBytes + 2 * third * (kBoxRows / 8) * kBoxBytes,
                      &sp.boxes[kind][size], &sh.full[stage], x + chunk * kChunk, y + 2 * third * kBoxRows);
        }
        ++fills;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
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
  if (down) follow();
  const int g = lane >> 2, c = lane & 3;
  // This warp's 64 columns of a stage: of chunk warp % 4 this lane has pieces 2c and 2c + 1, one after the other: 32
  // bytes of an assignment's row, and of the swizzled rows no two lanes of a quarter warp have the same banks.
  const uint32_t at = (warp & 3) * 8 * kBoxBytes + g * 128 + (((2 * c) ^ g) << 4);
  const int column = (warp & 3) * kChunk + 16 * c, columns_left = K - column;
  Ring ring = {base, static_cast<uint32_t>(warp >> 2), 0u, true};
  Pieces<PHASE> x;
  // The assignments' pieces come straight from L2, some stages before their use; a pass's first ones are sent for before
  // the sums of the pass before are joined. Each number of tiles has a loop of its own, without branches.
  int kb = warp >> 2;  // this warp's first K block of the pass
  auto start = [&](const Passes<MOST>& s, int kb) {
    const int16_t* list = sh.r.list + sh.r.begin[s.job.active] + s.j0;
    const int n = s.assignments - s.j0;
    if (MOST == 1 || n <= 8) x.template start<1>(p, list, n, kb, column, columns_left);
    else if (n <= 16) x.template start<2>(p, list, n, kb, column, columns_left);
    else x.template start<3>(p, list, n, kb, column, columns_left);
  };
  bool more = pass.next();
  if (more) start(pass, kb);
  while (more) {
    Passes<MOST> after = pass;
    more = after.next();
    const int kb_after = kb ^ (nk & 1);
    auto then = [&]() {
      if (more) start(after, kb_after);
    };
    const int16_t* list = sh.r.list + sh.r.begin[pass.job.active] + pass.j0;
    const int n = pass.assignments - pass.j0;
    auto run = [&](auto tiles) {
      products<PHASE, decltype(tiles)::value>(p, sh, ring, x, pass.job, list, n, kb, K, rows, columns_left, at, then);
    };
    if (MOST == 1 || n <= 8) run(std::integral_constant<int, 1>());
    else if (n <= 16) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 3>());
    pass = after;
    kb = kb_after;
  }
}

dmuon_status refuse(const char* msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int64_t pitch_h(int64_t inner) { return (inner + 7) / 8 * 8; }

dmuon_status check_sizes(int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner) {
  if (top < 1 || top > kMaxTop) return refuse("top must be between 1 and 64");
  if (tokens < 0 || tokens > kMaxAssignments || tokens * top > kMaxAssignments)
    return refuse("tokens * top must be between 0 and 2048 (for more: sort, dispatch, the experts' products, combine)");
  if (experts < 1 || experts > kMaxExperts) return refuse("experts must be between 1 and 4096");
  if (dim < 1 || dim > kMaxDim || inner < 1 || inner > kMaxDim) return refuse("dim and inner must be between 1 and 2^20");
  if (experts * std::max(dim, inner) > (int64_t(1) << 30)) return refuse("experts * dim and experts * inner must not be above 2^30");
  return DMUON_OK;
}

struct Workspace {
  size_t status, h, part, bytes;
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

// Matrices as rows of K, in boxes of so many rows by 64 columns; past the last column or row a box has zeros.
cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
  const cuuint32_t box[2] = {kChunk, (cuuint32_t)box_rows}, one[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int PHASE>
cudaError_t launch(const ExpertsParams& p, bool stream, int sms, cudaStream_t s) {
  const int rows = PHASE == kDown ? p.dim : p.inner, K = PHASE == kDown ? p.inner : p.dim;
  const int out = PHASE == kGated ? 8 : 16;
  const int64_t units = int64_t(std::min(p.experts, p.n)) * ((rows + out - 1) / out);
  cudaError_t e;
  auto shared = [](auto* kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  };
  if (!stream) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(units, 2 * sms)));
    if ((e = shared(experts_plain_kernel<PHASE>, sizeof(PlainShared))) != cudaSuccess) return e;
    return launch_follow(experts_plain_kernel<PHASE>, grid, kThreads, sizeof(PlainShared), s, 1, p);
  }
  StreamParams sp;
  sp.e = p;
  const bf16* w = PHASE == kGated ? p.gate : PHASE == kUngated ? p.up : p.down;
  e = cudaSuccess;
  for (int kind = 0; kind < (PHASE == kGated ? 2 : 1) && e == cudaSuccess; ++kind) {
    const bf16* m = kind == 0 ? w : p.up;
    for (int size = 0; size < 3 && e == cudaSuccess; ++size)
      e = map_rows(&sp.boxes[kind][size], m, K, int64_t(p.experts) * rows, out << size);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(units, sms)));
  sp.share = ~uint64_t(0) / grid.x + 1;
  // where no expert gets more than 8 assignments unless a token names it twice, the loops for more are left out
  auto* kernel = p.tokens <= 8 ? experts_stream_kernel<PHASE, 1> : experts_stream_kernel<PHASE, kMostTiles>;
  if ((e = shared(kernel, kStreamSmem)) != cudaSuccess) return e;
  return launch_follow(kernel, grid, kStreamThreads, kStreamSmem, s, 1, sp);
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
  e = gate != nullptr ? launch<kGated>(p, vec_up, sms, s) : launch<kUngated>(p, vec_up, sms, s);
  if (e == cudaSuccess) e = launch<kDown>(p, vec_down, sms, s);
  const int64_t blocks = (tokens * dim + kThreads - 1) / kThreads;
  if (e == cudaSuccess)
    e = launch_follow(experts_combine_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 8 * sms))), kThreads, 0, s,
                      1, p);
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
