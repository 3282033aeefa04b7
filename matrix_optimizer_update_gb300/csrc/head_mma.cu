// head_mma.cu - the products of the head's losses on the tensor cores:
// 256 x 256 output tiles on pairs of SMs (two-SM UMMA, tcgen05 cta_group::2),
// operands staged by TMA, fp32 accumulators in TMEM.
//
// Three launches share the pipeline and differ in operands and epilogue:
//  logits  z = H W^T, tile 256 tokens x 256 vocabulary entries. The epilogue
//          keeps, per token and 128 entries, the largest logit and the sum of
//          exponentials below it (one pass over z, joined later by rescaling),
//          and takes out the logits the loss asks for: z itself is never stored.
//  dz      the same product for one piece of the vocabulary; the epilogue turns
//          it into the loss's gradient with respect to z, in bf16.
//  grads   both gradients of a piece: dH += dz W (K = the piece's entries) and
//          dW = dz^T H (K = the tokens), one list of tiles.
// With many tokens each is bound by the tensor cores (a pair's tile moves 32 KB of operands per SM for 4.2
// MFLOP), and in long runs by the power limit. 2048 tokens x 32000 x 2048, alone: logits 145 us (1.85 PFLOP/s),
// dz 152 us (1.77), grads 271 to 278 us (1.93 to 1.98).
// With up to 128 tokens each is bound by reading W or writing dW. 64 tokens x 128000 x 4096: logits 165 us
// (6.35 TB/s), dz 170 us, dW alone 152 us, dH alone 168 us, both 345 us (6.1 TB/s).
//
// Roles in a CTA: warp 0 loads (and, in the leader, claims tiles from a counter
// and hands them to its peer), warp 1 issues the MMAs (leader only), warps 2 to
// 9 drain the accumulators, of which there are two, so that one tile's epilogue
// runs under the next tile's products. All waits are bounded (ptx.cuh).
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cudaTypedefs.h>

#include "follow.cuh"
#include "head.h"
#include "head_dot.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dmuon {
namespace head {
namespace {

constexpr int kTile = 256;                     // rows and columns of a pair's tile
constexpr int kStep = 64;                      // K per stage
constexpr uint32_t kHalf = 128 * kStep * 2;    // a CTA's 128 rows (or columns) of an operand, one stage
constexpr int kRingBytes = 6 * 2 * kHalf;      // operand stages: 6 of 32 KB, or more of fewer rows
constexpr int kThinGradStages = 5;             // gradients of few tokens: 5, and wide boxes in the sixth's place
constexpr int kMaxStages = 16;
constexpr int kThin = 128;                     // up to so many tokens, they are the N side of the products
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kBox = 32 * 64;                  // staging box of a TMA store: 32 rows of 64 bytes
constexpr int kWideBox = 32 * 128;             // ... of 128 bytes (gradients of few tokens)
constexpr int kRing = 8;
constexpr uint32_t kRingReaders = 2 + 2 * kEpiWarps;
constexpr uint32_t kTmemCols = 2 * kTile;
constexpr int64_t kWaitNs = 2000000000LL;
constexpr float kLog2e = 1.4426950408889634f;

// The thin forms of logits and dz turn the product round: vocabulary entries are the M side and the tokens
// the N side, padded to 32. With 77 tokens the M = 256 side of the other form is two thirds empty, and the
// launch is bound by products of zeros; turned round it is bound by reading W.
enum Mode { kLogits, kDz, kGrads, kThinLogits, kThinDz, kThinGrads };

struct Params {
  CUtensorMap a[2], b[2];  // [1]: the second kind of tile of a grads launch (dW)
  CUtensorMap out[2];      // dz; dH (bf16) or its fp32 sums; dW
  // tiles
  int32_t items;
  int32_t rows, cols;      // logits, dz: tiles along the tokens and the vocabulary
  int32_t nk;              // K stages per tile
  // grads: dH tiles come first (the longer ones), `slices` parts of K each, then dW tiles
  int32_t dh_items, dh_rows, dh_nk, slices, slice_nk;
  int32_t dim_tiles;
  int32_t thin_n;          // tokens padded to 32 when they are the N side, else 0
  int32_t thin_h;          // thin logits, dz: vocabulary entries per tile
  int32_t low;             // thin dz, grads: rows from dz's first parts to the second, 0: there are none
  int32_t dw_rows;         // grads: tokens per stage of dW
  int32_t stages, stage_bytes, a_bytes;  // thin logits, dz: a stage holds a_bytes of A, then B
  int32_t chunked;         // dim is a multiple of 64: one copy brings two 64-column blocks
  int32_t dh_direct;       // dH is complete: store bf16; else add into fp32 sums
  int32_t first;           // ... of which this is the first piece (store, not add)
  float* dh_acc;           // thin: the fp32 sums, pitch acc_ld
  int64_t acc_ld;
  float gscale;            // factor of the gradients beside *gmax
  float zscale;            // of the logits: 1 / temperature and what truncation takes
  float* gmax;             // largest finite |grad|: dz holds gradients relative to it
  LogitParams l;
  unsigned* sched;         // [0] tiles claimed, [1] CTAs done; both zero between launches
  unsigned* status;
};

struct Shared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t mma_done;
  uint64_t ring_full[kRing];
  uint64_t ring_empty[kRing];
  int ring[kRing];
  uint32_t tmem;
  int abort_flag;
  float red[kEpiWarps];
};
static_assert(sizeof(Shared) <= 1024, "barriers must fit their 1 KB");

// What thin dz needs of its tokens, in shared memory.
struct ThinTokens {
  float g[kThin];      // gradient relative to the largest, 0 for a token that does not count
  float lse[kThin];
};

// Instruction descriptor as ptx::idesc_bf16, with A MN-major too (bit 15).
__device__ __forceinline__ uint32_t idesc(int n, bool a_mn, bool b_mn) {
  return ptx::idesc_bf16(kTile, n, b_mn) | (a_mn ? (1u << 15) : 0u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(x) * 2^32, to be multiplied by kLow: the product may lie below 2^-126, where ex2 itself gives 0.
// Gradients of entries far down the tail, which sums may still be made of.
constexpr float kLow = 1.f / 4294967296.f;
__device__ __forceinline__ float exp_high(float x) { return ex2(fmaf(x, kLog2e, 32.f)); }

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_2d(const void* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// Arrive on an mbarrier of either CTA of the pair (cluster address). What it orders are this thread's own
// reads (a ring slot, TMEM) before the arrival, for which the scope of the CTA is enough; with the scope of the
// cluster the arrival waits for every store in flight, which took 2300 of the 5900 cycles of a dW tile.
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A 32-bit store to the peer's shared memory that counts its 4 bytes on a barrier there. (A plain store and an
// arrival that releases it at cluster scope wait for everything the thread has in flight.)
__device__ __forceinline__ void store_async_peer(uint32_t addr, int v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
               "r"(bar)
               : "memory");
}

// Adds a staged fp32 box to global memory, element by element.
__device__ __forceinline__ void tma_add_3d(const void* map, const void* src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(ptx::smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Staging boxes have 64-byte rows; piece c of row r sits at piece c ^ ((r >> 1) & 3) (64-byte swizzle).
__device__ __forceinline__ uint4* piece(uint8_t* box, int r, int c) {
  return reinterpret_cast<uint4*>(box + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Boxes with 128-byte rows: piece c of row r at piece c ^ (r & 7) (128-byte swizzle).
__device__ __forceinline__ uint4* wide_piece(uint8_t* box, int r, int c) {
  return reinterpret_cast<uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
}

// 8 consecutive values, scaled, as bf16.
__device__ __forceinline__ uint4 rounded(const float (&v)[32], int at, float scale) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(v[at + 2 * e] * scale, v[at + 2 * e + 1] * scale);
  return u;
}

struct Where {
  int kind;        // grads: 0 = dH, 1 = dW
  int row, col;    // tile coordinates
  int slice;
  int k0, nk;      // K stages
};

// Tiles of logits and dz: bands of 8 token blocks, the vocabulary within a band, so that the 76 pairs at
// work share the band's H (8 x 256 rows) and about ten blocks of W.
constexpr int kBand = 8;

template <int MODE>
__device__ __forceinline__ Where where_is(const Params& p, int w) {
  Where x;
  x.kind = 0;
  x.slice = 0;
  x.k0 = 0;
  if (MODE == kThinLogits || MODE == kThinDz) {
    x.row = 0;
    x.col = w;
    x.nk = p.nk;
  } else if (MODE == kLogits || MODE == kDz) {
    const int band = w / (kBand * p.cols);
    const int r = w - band * kBand * p.cols;
    const int high = min(kBand, p.rows - band * kBand);
    x.col = r / high;
    x.row = band * kBand + r - x.col * high;
    x.nk = p.nk;
  } else if (w < p.dh_items) {
    const int per = p.dh_rows * p.dim_tiles;
    x.slice = w / per;
    const int r = w - x.slice * per;
    x.row = r / p.dim_tiles;             // thin: always 0
    x.col = r - x.row * p.dim_tiles;
    x.k0 = x.slice * p.slice_nk;
    x.nk = min(p.slice_nk, p.dh_nk - x.k0);
  } else {
    const int r = w - p.dh_items;
    x.kind = 1;
    x.row = r / p.dim_tiles;
    x.col = r - x.row * p.dim_tiles;
    x.nk = p.nk;
  }
  return x;
}

// ------------------------------------------------------------------ what the loss wants of a row
// The wanted entries of one token inside its 128 columns, in ascending order: next() is the id of the
// next one, or INT_MAX.
struct Cursor {
  const int32_t* ids;
  const float* q;
  int pos, n, id;
  __device__ __forceinline__ void start(const Wanted& w, int64_t t, bool in, int first) {
    pos = n = 0;
    id = INT_MAX;
    if (!in) return;
    if (w.targets != nullptr) {
      const int64_t y = w.targets[t];
      if (y >= first && y < w.vocab) id = static_cast<int>(y);
      return;
    }
    ids = w.ids + t * w.top;
    q = w.q + t * w.top;
    n = w.count[t];
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ids[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    pos = lo;
    if (pos < n) id = ids[pos];
  }
};

// Whether a token has a loss at all.
__device__ __forceinline__ bool counts(const Wanted& w, int64_t t) {
  return w.targets != nullptr ? w.targets[t] >= 0 && w.targets[t] < w.vocab : w.count[t] > 0;
}

// Cross entropy's backward pass: the logits of this warp's targets (lane: token t, its target id) before `end`, in
// fp32 FMAs, to picked. By whole warps, before the wait for the tile's product: one target per token in the
// whole vocabulary, so few to a tile, and a launch of its own costs more (77 tokens: 128 against 116 us). Where
// they lie together they go by fours, as a trip to memory takes longer than what is fetched (243 tokens x 15031 x
// 3928, both passes: one by one 190 us, this way 166).
__device__ __forceinline__ void target_logits(const LogitParams& p, int id, int64_t t, int end, int lane) {
  if (p.want.targets == nullptr || p.loss != nullptr) return;  // a list's are formed where it is sorted
  unsigned more = __ballot_sync(0xffffffffu, id < end);
  while (more != 0u) {
    int L = 0;
    int64_t ts[4], ids[4];
    unsigned mine = 0u;
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // past the last one, that again
      if (more != 0u) L = __ffs(more) - 1;
      more &= more - 1u;
      ts[n] = __shfl_sync(0xffffffffu, t, L);
      ids[n] = __shfl_sync(0xffffffffu, id, L);
      if (lane == L) mine |= 1u << n;
    }
    float z[4];
    dot_parts<4>(p.in, ts, ids, lane, 32, z);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      z[n] = warp_sum(z[n]) * p.in.scale;
      if ((mine >> n & 1u) != 0u) p.picked[t] = z[n];
    }
  }
}

// p - share of a likely entry. From its logit: lse is rounded (by up to 1e-6 at 16 to 32) and z is, so that of a token
// predicted with near certainty p keeps no digit of 1 - p, and must at least not be above 1, where the gradient would
// push the target down. From the token's loss, which keeps them: p of the target is exp(-loss).
__device__ __forceinline__ float above(const LogitParams& p, float known, float lse, float share) {
  if (p.loss != nullptr) return expm1f(-known);
  return (known > lse ? 1.f : expf(known - lse)) - share;
}

// 32 x 32 values in shared memory, rows turned so that neither rows nor columns conflict.
__device__ __forceinline__ float& cell(float* sm, int row, int col) { return sm[row * 32 + (col ^ row)]; }

// Visits the entries of this lane's cursor before `end`, whose values are row `lane` of sm (column: id - first):
// visit(value, share, known, pos, again), `known` the logit of a likely entry (the token's loss, where the call has
// those), `again` when the entry before had the same id. A lane's entries may be many:
// frequent words lie together in many vocabularies. (With the values left in registers, where an entry takes a
// compare for each of 32, and one after another over a warp's tokens, both passes over 48 lists of 68 entries against
// 9328 x 1616 take 300 us; this way 81, and 74 with what follows.)
//
// Four entries are loaded together: a load of one each is a chain of trips to the L2, for the shared memory that
// the tiles take leaves an L1 too small for the warps' lists (242 lists of 39 against 9800 x 1056: 92 -> 77 us).
template <bool WITH_LOGIT, class Visit>
__device__ __forceinline__ void walk(const LogitParams& p, int64_t t, Cursor& c, int first, int end, float* sm,
                                     int lane, Visit&& visit) {
  const Wanted& w = p.want;
  const float* known = p.loss != nullptr ? p.loss : p.picked;
  int last = -1;
  while (c.id < end) {
    int id[5];
    float q[4], z[4];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const bool in = c.pos + j < c.n;
      id[j] = in ? c.ids[c.pos + j] : INT_MAX;
      if (j < 4) q[j] = in ? c.q[c.pos + j] : 1.f;  // a target's share
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      z[j] = WITH_LOGIT && (j == 0 || c.pos + j < c.n) && q[j] >= kSure ? known[t * w.top + c.pos + j] : 0.f;
    const int pos = c.pos;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c.id < end) {
        visit(cell(sm, lane, c.id - first), q[j], z[j], pos + j, c.id == last);
        last = c.id;
        c.id = id[j + 1];
        ++c.pos;
      }
  }
}

// The wanted entries of this lane's token among its 32 values v (entries from `first`).
template <bool WITH_LOGIT, class Visit>
__device__ __forceinline__ void wanted_of_row(const LogitParams& p, int64_t t, Cursor& c, int first, float (&v)[32],
                                              float* sm, int lane, Visit&& visit) {
#pragma unroll
  for (int k = 0; k < 32; ++k) cell(sm, lane, k) = v[k];
  walk<WITH_LOGIT>(p, t, c, first, first + 32, sm, lane, visit);
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = cell(sm, lane, k);
}

// One warp's part of a logits tile: 32 tokens, 128 entries from j0. `wait` returns false when the CTA gave up.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_logits(const LogitParams& p, float zscale, int64_t t, int j0, uint32_t tbase,
                                             int lane, float* sm, Wait&& wait, Free&& free) {
  const bool in = t < p.tokens;
  Cursor c;
  c.start(p.want, t, in, j0);
  if (!wait()) return false;
  ptx::tc_fence_after();
  float peak = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    const int jc = j0 + ch * 32;
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + ch * 32, v);
    if (ch == 3) free();
    if (jc >= p.vocab) continue;
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] *= zscale;
    if (jc + 32 > p.vocab) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (jc + k >= p.vocab) v[k] = -INFINITY;
    }
    if (__any_sync(0xffffffffu, c.id < jc + 32))
      wanted_of_row<false>(p, t, c, jc, v, sm, lane, [&](float& x, float share, float, int pos, bool again) {
        if (again) return;  // entries that share an id have one logit, with the first of them
        if (!(share >= kSure)) p.picked[t * p.want.top + pos] = x;
        x = -INFINITY;
      });
    float top = v[0];
#pragma unroll
    for (int k = 1; k < 32; ++k) top = fmaxf(top, v[k]);
    top = fmaxf(peak, top);
    const float from = top == -INFINITY ? 0.f : top;  // nothing yet: every exponential is 0
    float s[4] = {};
#pragma unroll
    for (int k = 0; k < 32; ++k) s[k & 3] += ex2((v[k] - from) * kLog2e);
    sum = sum * ex2((peak - from) * kLog2e) + ((s[0] + s[1]) + (s[2] + s[3]));
    peak = top;
  }
  if (in && j0 < p.vocab) p.parts[int64_t(j0 / kGroup) * p.tokens + t] = Part{peak, sum};
  return true;
}

// One warp's part of a dz tile. Row t's gradient relative to the largest: g (p - wanted), rounded to bf16
// as the operand of the gradients' products (the only rounding of dz).
template <class Wait, class Free>
__device__ __forceinline__ bool drain_dz(const Params& P, float gmax, int64_t t, int64_t t0, int j0, uint32_t tbase,
                                         int lane, uint8_t* stg, uint32_t& nbox, Wait&& wait, Free&& free) {
  const LogitParams& p = P.l;
  const bool in = t < p.tokens;
  Cursor c;
  c.start(p.want, t, in, j0);
  float g = 0.f, lse = 0.f;
  if (in) {
    lse = p.lse[t];
    g = counts(p.want, t) ? p.grad[t] / gmax : 0.f;
    if (g == 0.f) c.id = INT_MAX;  // zeros, whatever z is
  }
  target_logits(p, c.id, t, min(j0 + 128, p.vocab), lane);
  const float g_low = g * kLow;
  if (!wait()) return false;
  ptx::tc_fence_after();
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    const int jc = j0 + ch * 32;
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + ch * 32, v);
    if (ch == 3) free();
    // a row that does not count, and entries past the vocabulary, give exact zeros whatever z is
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float e = g_low * exp_high(fmaf(v[k], P.zscale, -lse));
      v[k] = g == 0.f ? 0.f : e;
    }
    if (jc + 32 > p.vocab) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (jc + k >= p.vocab) v[k] = 0.f;
    }
    if (__any_sync(0xffffffffu, c.id < jc + 32)) {
      if (lane == 0) ptx::bulk_wait_read<0>();  // both boxes' place
      __syncwarp();
      wanted_of_row<true>(p, t, c, jc, v, reinterpret_cast<float*>(stg), lane,
                          [&](float& x, float share, float z, int, bool again) {
                            x = share >= kSure && !again ? g * above(p, z, lse, share) : x - g * share;
                          });
    }
    uint8_t* box = stg + (nbox & 1u) * kBox;
    if (lane == 0) ptx::bulk_wait_read<1>();  // the store that last read this box is done with it
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) *piece(box, lane, q) = rounded(v, q * 8, 1.f);
    ptx::fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (t0 < p.tokens) ptx::tma_store_2d(&P.out[0], box, jc - p.v0, static_cast<int>(t0));
      ptx::bulk_commit();
    }
    ++nbox;
  }
  return true;
}

// ------------------------------------------------------------------ thin epilogues: lane = vocabulary entry, column = token
// Reduces 32 columns over the 32 lanes by halving: lane j ends with column j's result, in 31 exchanges.
template <class Op>
__device__ __forceinline__ float columns(const float (&v)[32], int lane, Op op) {
  float r[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const bool up = (lane & 16) != 0;
    r[k] = op(up ? v[k + 16] : v[k], __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + 16], 16));
  }
#pragma unroll
  for (int s = 8; s > 0; s >>= 1)
#pragma unroll
    for (int k = 0; k < s; ++k) {
      const bool up = (lane & s) != 0;
      r[k] = op(up ? r[k + s] : r[k], __shfl_xor_sync(0xffffffffu, up ? r[k] : r[k + s], s));
    }
  return r[0];
}

// The wanted entries of 32 tokens (lane: token, cursor c) among the warp's vocabulary entries [first, end): the
// lanes' columns go through shared memory, where each lane walks its own token's row.
template <bool WITH_LOGIT, class Visit>
__device__ __forceinline__ void wanted_of_tokens(const LogitParams& p, int64_t t, Cursor& c, int first, int end,
                                                 float (&v)[32], float* sm, int lane, Visit&& visit) {
  if (!__any_sync(0xffffffffu, c.id < end)) return;
#pragma unroll
  for (int k = 0; k < 32; ++k) cell(sm, k, lane) = v[k];
  __syncwarp();
  walk<WITH_LOGIT>(p, t, c, first, end, sm, lane, visit);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = cell(sm, k, lane);
  __syncwarp();  // before the next block's values
}

// One warp's part of a thin logits tile: 32 entries from `first` (those before `end` are this tile's), the
// blocks of 32 tokens that are its half's.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_thin_logits(const Params& P, int first, int end, int group, int half,
                                                  uint32_t tbase, int lane, float* sm, Wait&& wait, Free&& free) {
  const LogitParams& p = P.l;
  const int blocks = P.thin_n / 32;
  Cursor c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = (half + 2 * i) * 32 + lane;
    c[i].start(p.want, t, t < p.tokens && first < end, first);
  }
  if (!wait()) return false;
  ptx::tc_fence_after();
  const int v0 = first + lane;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int b = half + 2 * i;
    if (b >= blocks) {
      if (b < 2) free();  // this half has no tokens
      break;
    }
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + b * 32, v);
    if (b + 2 >= blocks) free();
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = v0 < end ? v[k] * P.zscale : -INFINITY;
    const int64_t t = b * 32 + lane;
    wanted_of_tokens<false>(p, t, c[i], first, end, v, sm, lane,
                            [&](float& x, float share, float, int pos, bool again) {
                              if (again) return;
                              if (!(share >= kSure)) p.picked[t * p.want.top + pos] = x;
                              x = -INFINITY;
                            });
    const float peak = columns(v, lane, [](float x, float y) { return fmaxf(x, y); });
    const float from = peak == -INFINITY ? 0.f : peak;
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = ex2((v[k] - __shfl_sync(0xffffffffu, from, k)) * kLog2e);
    const float sum = columns(v, lane, [](float x, float y) { return x + y; });
    if (t < p.tokens) p.parts[t * (P.items * 8) + group] = Part{peak, sum};
  }
  return true;
}

// One warp's part of a thin dz tile; dz[t][v - v0] as in the other form.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_thin_dz(const Params& P, const ThinTokens& tk, int first, int end, int half,
                                              uint32_t tbase, int lane, float* sm, Wait&& wait, Free&& free) {
  const LogitParams& p = P.l;
  const int blocks = P.thin_n / 32;
  Cursor c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = (half + 2 * i) * 32 + lane;
    c[i].start(p.want, t, t < p.tokens && first < end && tk.g[t] != 0.f, first);
  }
#pragma unroll 1  // one copy of its code: a short launch waits for its instructions, too
  for (int i = 0; i < 2; ++i)
    target_logits(p, i == 0 ? c[0].id : c[1].id, (half + 2 * i) * 32 + lane, end, lane);
  if (!wait()) return false;
  ptx::tc_fence_after();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int b = half + 2 * i;
    if (b >= blocks) {
      if (b < 2) free();  // this half has no tokens
      break;
    }
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + b * 32, v);
    if (b + 2 >= blocks) free();
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float g = tk.g[b * 32 + k];
      const float e = g * kLow * exp_high(fmaf(v[k], P.zscale, -tk.lse[b * 32 + k]));
      v[k] = g == 0.f ? 0.f : e;
    }
    const int t = b * 32 + lane;
    wanted_of_tokens<true>(p, t, c[i], first, end, v, sm, lane,
                           [&](float& x, float share, float z, int, bool again) {
                             const float g = tk.g[t];
                             x = share >= kSure && !again ? g * above(p, z, tk.lse[t], share) : x - g * share;
                           });
    // By way of shared memory, so that a lane stores 16 bytes: with 2 bytes a lane the number of stores shows in the
    // launch's time (both passes over 77 tokens x 50257 x 1024: 103 us, this way 99.7; with the tokens that there are not left
    // out, 103 again). `first` and the tiles' ends
    // are multiples of 8 from the piece's start; past its last entry lies room of dz that nothing reads.
    bf16* at = reinterpret_cast<bf16*>(sm);
    const int row = lane >> 2, col = (lane & 3) * 8;
    auto store = [&](bf16* out) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = row + 8 * j;
        if (b * 32 + k < p.tokens && first + col < end)
          *reinterpret_cast<uint4*>(out + (b * 32 + k) * p.ld_dz + col) =
              *reinterpret_cast<const uint4*>(at + k * 32 + col);
      }
      __syncwarp();
    };
    bf16* out = p.dz + (first - p.v0);
#pragma unroll
    for (int k = 0; k < 32; ++k) at[k * 32 + lane] = __float2bfloat16_rn(v[k]);
    store(out);
    if (P.low != 0) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        at[k * 32 + lane] = __float2bfloat16_rn(v[k] - __bfloat162float(__float2bfloat16_rn(v[k])));
      store(out + P.low * p.ld_dz);
    }
  }
  return true;
}

// One warp's part of a thin dH tile: 32 columns of dH (lane) by the tokens, into the slice's fp32 sums.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_thin_dh(const Params& P, const Where& x, int d0, int half, uint32_t tbase,
                                              int lane, Wait&& wait, Free&& free) {
  if (!wait()) return false;
  ptx::tc_fence_after();
  const int d = d0 + lane;
  float* acc = P.dh_acc + int64_t(x.slice) * P.l.tokens * P.acc_ld + d;
  if (half >= P.thin_n / 32) free();  // this half has no tokens
  for (int b = half; b < P.thin_n / 32; b += 2) {
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + b * 32, v);
    if (P.low != 0) {  // the second parts' columns
      float u[32];
      ptx::tmem_ld_32x32b_x32(tbase + P.thin_n + b * 32, u);
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] += u[k];
    }
    if (b + 2 >= P.thin_n / 32) free();
    if (d < P.l.in.dim) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (b * 32 + k < P.l.tokens) {
          float* o = acc + int64_t(b * 32 + k) * P.acc_ld;
          *o = P.first ? v[k] : *o + v[k];
        }
    }
  }
  return true;
}

// One warp's part of a gradient tile: 32 rows from r0, 128 columns from d0.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_grads(const Params& P, const Where& x, float scale, int64_t r0, int64_t r_lim, int d0,
                                            uint32_t tbase, int lane, uint8_t* stg, uint32_t& nbox, Wait&& wait, Free&& free) {
  const bool sums = x.kind == 0 && !P.dh_direct;
  if (!wait()) return false;
  ptx::tc_fence_after();
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    const int dc = d0 + ch * 32;
    float v[32];
    ptx::tmem_ld_32x32b_x32(tbase + ch * 32, v);
    if (ch == 3) free();
    const bool in = r0 < r_lim && dc < P.l.in.dim;
    if (sums) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* box = stg + (nbox & 1u) * kBox;
        if (lane == 0) ptx::bulk_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = h * 16 + q * 4;
          *reinterpret_cast<float4*>(piece(box, lane, q)) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          const int d = dc + h * 16;
          if (in && d < P.l.in.dim) {
            if (P.first) ptx::tma_store_3d(&P.out[0], box, d, static_cast<int>(r0), x.slice);
            else tma_add_3d(&P.out[0], box, d, static_cast<int>(r0), x.slice);
          }
          ptx::bulk_commit();
        }
        ++nbox;
      }
    } else {
      uint8_t* box = stg + (nbox & 1u) * kBox;
      if (lane == 0) ptx::bulk_wait_read<1>();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) *piece(box, lane, q) = rounded(v, q * 8, scale);
      ptx::fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (in) ptx::tma_store_2d(&P.out[x.kind], box, dc, static_cast<int>(r0));
        ptx::bulk_commit();
      }
      ++nbox;
    }
  }
  return true;
}

// The same for dW of few tokens, whose product is one or two K stages, so that the epilogue sets the pace: two
// stores of 64 columns, from a box each, which the next tile finds free again. v0: first row; v_lim: past the last.
template <class Wait, class Free>
__device__ __forceinline__ bool drain_thin_dw(const Params& P, float scale, int v0, int v_lim, int d0, uint32_t tbase, int lane,
                                              uint8_t* stg, Wait&& wait, Free&& free) {
  if (!wait()) return false;
  ptx::tc_fence_after();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint8_t* box = stg + h * kWideBox;
    if (lane == 0) ptx::bulk_wait_read<1>();  // the last tile's store from this box is done with it
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      float v[32];
      ptx::tmem_ld_32x32b_x32(tbase + (2 * h + ch) * 32, v);
      if (h == 1 && ch == 1) free();
#pragma unroll
      for (int q = 0; q < 4; ++q) *wide_piece(box, lane, ch * 4 + q) = rounded(v, q * 8, scale);
    }
    ptx::fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (v0 < v_lim && d0 + 64 * h < P.l.in.dim) ptx::tma_store_2d(&P.out[1], box, d0 + 64 * h, v0);
      ptx::bulk_commit();
    }
  }
  return true;
}

// ------------------------------------------------------------------ the kernel
__device__ __forceinline__ bool take(Shared* sh, uint32_t j, int& w, uint32_t lead_empty, volatile int* abortf,
                                     const Params& p, bool arm = false) {
  const uint32_t slot = j % kRing;
  if (!ptx::mbar_wait_cluster(&sh->ring_full[slot], (j / kRing) & 1u, abortf, p.status, kWaitNs)) return false;
  w = *reinterpret_cast<volatile int*>(&sh->ring[slot]);
  if (arm) ptx::mbar_arrive_expect_tx(&sh->ring_full[slot], 4);
  arrive_pair(lead_empty + slot * static_cast<uint32_t>(sizeof(uint64_t)));
  return true;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) head_pair_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr bool thin = MODE == kThinLogits || MODE == kThinDz;
  constexpr bool grads = MODE == kGrads || MODE == kThinGrads;
  constexpr int ring_bytes = MODE == kThinGrads ? kThinGradStages * 2 * kHalf : kRingBytes;
  constexpr int box_bytes = MODE == kThinGrads ? kWideBox : kBox;
  Shared* sh = reinterpret_cast<Shared*>(base + ring_bytes);
  uint8_t* boxes = base + ring_bytes + 1024;
  ThinTokens& tk = *reinterpret_cast<ThinTokens*>(boxes + kEpiWarps * 2 * kBox);  // thin dz only
  // operand ring: fixed at compile time but for the thin logits and dz, whose stages hold fewer rows
  const uint32_t stages = thin ? p.stages : ring_bytes / (2 * kHalf);
  const uint32_t stage_bytes = thin ? p.stage_bytes : 2 * kHalf;
  const uint32_t a_bytes = thin ? p.a_bytes : kHalf;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abortf = &sh->abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < (grads ? 2 : 1); ++i) {
      ptx::prefetch_tmap(&p.a[i]);
      ptx::prefetch_tmap(&p.b[i]);
    }
    for (int s = 0; s < kMaxStages; ++s) {
      ptx::mbar_init(&sh->full[s], 1);
      ptx::mbar_init(&sh->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&sh->tfull[a], 1);
      ptx::mbar_init(&sh->tempty[a], 2 * kEpiWarps);
    }
    ptx::mbar_init(&sh->mma_done, 1);
    for (int k = 0; k < kRing; ++k) {
      ptx::mbar_init(&sh->ring_full[k], 1);
      ptx::mbar_init(&sh->ring_empty[k], kRingReaders);
    }
    sh->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&sh->tmem, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem;
  // Set up while the kernel before still runs: the first stages of W on their way to L2 (a hint: nothing is read
  // before that kernel is done, and what it may write to W passes through L2). 1 to 2 % of a call with few tokens.
  if ((MODE == kThinLogits || MODE == kThinDz) && threadIdx.x == 0) {
    const int row = p.l.v0 + static_cast<int>(blockIdx.x >> 1) * p.thin_h + rank * (p.thin_h / 2);
    for (int kb = 0; kb < min(p.nk, 16); ++kb) tma_prefetch_2d(&p.b[0], kb * kStep, row);
  }
  // After the kernel that sorts the lists, which lets this one start once everything before it is done, only the
  // epilogue has to wait for it: loads and products of the first tile run beside it.
  if (!p.l.after_lists || warp >= 2) follow(MODE != kLogits && MODE != kThinLogits);
  const uint32_t lead_empty = ptx::mapa_shared(ptx::smem_u32(&sh->ring_empty[0]), 0);

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- loads
      const uint32_t lead_full = ptx::mapa_shared(ptx::smem_u32(&sh->full[0]), 0);
      uint32_t stage = 0, phase = 0, fills = 0;
      auto load_tile = [&](int w) -> bool {
        const Where x = where_is<MODE>(p, w);
        const bool turned = MODE == kThinGrads && x.kind == 0;  // dH^T = W^T dz^T
        const int row = x.row * kTile + rank * 128, col = x.col * kTile + rank * 128;
        // dH^T's N side: half of the tokens each, or rank 0 their dz's first parts and rank 1 the second
        const bool twofold = MODE == kThinGrads && p.low != 0;
        const uint32_t dw_block = MODE == kThinGrads ? p.dw_rows * 128 : kHalf / 2;  // 64 columns of a stage of dW
        const uint32_t bytes = thin       ? stage_bytes
                               : turned   ? kHalf + p.thin_n * (twofold ? 128 : 64)
                               : x.kind == 1 ? 4 * dw_block
                                             : 2 * kHalf;
        for (int kb = 0; kb < x.nk; ++kb) {
          if (!ptx::mbar_wait_cluster(&sh->empty[stage], phase ^ 1u, abortf, p.status, kWaitNs)) return false;
          if (leader) ptx::mbar_arrive_expect_tx(&sh->full[stage], 2 * bytes);
          const uint32_t fb = lead_full + stage * static_cast<uint32_t>(sizeof(uint64_t));
          uint8_t* a = base + stage * stage_bytes;
          uint8_t* b = a + a_bytes;
          const int k = (x.k0 + kb) * kStep;
          if (thin) {  // W and H, K-major: thin_h / 2 and thin_n / 2 rows of 64
            tma_load_2d_pair(a, &p.b[0], fb, k, p.l.v0 + x.col * p.thin_h + rank * (p.thin_h / 2));
            tma_load_2d_pair(b, &p.a[0], fb, k, rank * (p.thin_n / 2));
          } else if (!grads) {  // both K-major: 128 rows of 64
            tma_load_2d_pair(a, &p.a[0], fb, k, row);
            tma_load_2d_pair(b, &p.b[0], fb, k, p.l.v0 + col);
          } else {
            uint8_t* wide = turned ? a : b;                                     // W or H, MN-major
            const CUtensorMap* mw = &p.b[x.kind];
            // dW of twofold dz: K is the tokens twice, one stage each. (What the first stage's box has of the second
            // parts meets rows of zeros: those of H past its last token.)
            const int kr = x.kind == 0 ? k + p.l.v0 : twofold ? 0 : k;
            const int kz = twofold ? kb * p.low : k;
            if (turned) tma_load_2d_pair(b, &p.a[0], fb, k, rank * (twofold ? p.low : p.thin_n / 2));  // dz, K-major
            else if (x.kind == 0) tma_load_2d_pair(a, &p.a[0], fb, k, row);  // dz, K-major
            else ptx::tma_load_3d_pair(a, &p.a[1], fb, 0, kz, row / 64);     // dz, two blocks of 64 columns
            if (p.chunked) {
              ptx::tma_load_3d_pair(wide, mw, fb, 0, kr, col / 64);
            } else {
              tma_load_2d_pair(wide, mw, fb, col, kr);
              tma_load_2d_pair(wide + (x.kind == 1 ? dw_block : kHalf / 2), mw, fb, col + 64, kr);
            }
          }
          ++fills;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        return true;
      };
      if (leader) {
        const uint32_t peer_ring = ptx::mapa_shared(ptx::smem_u32(&sh->ring[0]), 1);
        const uint32_t peer_full = ptx::mapa_shared(ptx::smem_u32(&sh->ring_full[0]), 1);
        // The first tile is the pair's own number, the others are claimed in the order of the list.
        auto claim = [&]() -> int {
          const unsigned w = (gridDim.x >> 1) + atomicAdd(p.sched, 1u);
          return w < static_cast<unsigned>(p.items) ? static_cast<int>(w) : -1;
        };
        int w = static_cast<int>(blockIdx.x >> 1);
        for (uint32_t j = 0;; ++j) {
          const uint32_t slot = j % kRing;
          if (!ptx::mbar_wait_cluster(&sh->ring_empty[slot], ((j / kRing) & 1u) ^ 1u, abortf, p.status, kWaitNs)) break;
          sh->ring[slot] = w;
          store_async_peer(peer_ring + slot * 4u, w, peer_full + slot * static_cast<uint32_t>(sizeof(uint64_t)));
          ptx::mbar_arrive(&sh->ring_full[slot]);
          if (w < 0) break;
          const int next = claim();  // its latency hides under this tile's loads
          if (!load_tile(w)) break;
          w = next;
        }
        // the leader's full barriers count both CTAs' bytes: nothing is in flight once they complete
        for (uint32_t s = 0; s < stages; ++s) {
          if (fills > s) {
            const uint32_t n = (fills - 1u - s) / stages + 1u;
            int zero = 0;
            ptx::mbar_wait_cluster(&sh->full[s], (n - 1u) & 1u, &zero, p.status, kWaitNs);
          }
        }
      } else {
        // the ring's barriers here complete on the leader's 4 bytes: this thread arms each for its next use before
        // it hands the slot back
        for (int k = 0; k < kRing; ++k) ptx::mbar_arrive_expect_tx(&sh->ring_full[k], 4);
        for (uint32_t j = 0;; ++j) {
          int w;
          if (!take(sh, j, w, lead_empty, abortf, p, true) || w < 0) break;
          if (!load_tile(w)) break;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------- products
      uint32_t stage = 0, phase = 0, local = 0;
      bool ok = true;
      for (int w; ok && take(sh, local, w, lead_empty, abortf, p) && w >= 0; ++local) {
        const Where x = where_is<MODE>(p, w);
        const bool turned = MODE == kThinGrads && x.kind == 0;
        const bool a_mn = MODE == kThinGrads || (MODE == kGrads && x.kind == 1);
        const bool b_mn = grads && !turned;
        const uint32_t id = idesc(thin ? p.thin_n : turned ? p.thin_n * (p.low != 0 ? 2 : 1) : kTile, a_mn, b_mn);
        const uint32_t acc = local & 1u;
        if (!ptx::mbar_wait_cluster(&sh->tempty[acc], ((local >> 1) & 1u) ^ 1u, abortf, p.status, kWaitNs)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + acc * kTile;
        // Descriptors of stage 0; a stage or 16 columns of K further is an addition to the address field (in 16
        // bytes). K-major: 16 columns further in the swizzled rows; MN-major: 16 rows of 128 bytes further, the
        // operand's second 64-element block `block` on. One thread issues everything, so what it computes per
        // MMA counts: built anew each time, the four descriptors of a stage took 285 of its 512 cycles.
        const bool few = MODE == kThinGrads && x.kind == 1;  // a stage may have fewer than 64 of K
        const uint32_t block = few ? p.dw_rows * 128 : kHalf / 2, steps = few ? p.dw_rows / 16 : kStep / 16;
        const uint32_t s0 = ptx::smem_u32(base);
        const uint64_t a_desc = a_mn ? ptx::sw128_desc(s0, block, 1024) : ptx::sw128_desc(s0, 16, 1024);
        const uint64_t b_desc =
            b_mn ? ptx::sw128_desc(s0 + a_bytes, block, 1024) : ptx::sw128_desc(s0 + a_bytes, 16, 1024);
        const uint32_t a_step = a_mn ? 2048 / 16 : 32 / 16, b_step = b_mn ? 2048 / 16 : 32 / 16;
        for (int kb = 0; kb < x.nk; ++kb) {
          if (!ptx::mbar_wait_cluster(&sh->full[stage], phase, abortf, p.status, kWaitNs)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t a0 = a_desc + stage * (stage_bytes / 16), b0 = b_desc + stage * (stage_bytes / 16);
#pragma unroll
          for (uint32_t kk = 0; kk < kStep / 16; ++kk)
            if (kk < steps)
              ptx::umma_f16_pair(d, a0 + kk * a_step, b0 + kk * b_step, id, (kb | kk) != 0 ? 1u : 0u);
          ptx::umma_commit_pair(&sh->empty[stage], 0x3);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::umma_commit_pair(&sh->tfull[acc], 0x3);
      }
      ptx::umma_commit_pair(&sh->mma_done, 0x1);
      int zero = 0;
      ptx::mbar_wait(&sh->mma_done, 0, &zero, p.status, kWaitNs);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lead_tempty = ptx::mapa_shared(ptx::smem_u32(&sh->tempty[0]), 0);
    uint8_t* stg = boxes + (warp - 2) * (2 * box_bytes);
    float* sm = reinterpret_cast<float*>(stg);  // logits and thin dz: 32 x 32 values in the place of boxes
    static_assert(2 * kBox == 32 * 32 * 4, "a warp's two boxes");
    float gmax = 1.f;
    if (MODE == kDz || MODE == kThinDz) {  // under the first tile's products
      float m = 0.f;
      for (int64_t t = threadIdx.x - 64; t < p.l.tokens; t += kEpiWarps * 32)
        if (counts(p.l.want, t)) {
          const float g = fabsf(p.l.grad[t]);
          if (g < INFINITY) m = fmaxf(m, g);  // the others' gradients are relative to it, and finite
        }
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (lane == 0) sh->red[warp - 2] = m;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int k = 0; k < kEpiWarps; ++k) gmax = k == 0 ? sh->red[0] : fmaxf(gmax, sh->red[k]);
      if (gmax == 0.f) gmax = 1.f;
      if (blockIdx.x == 0 && threadIdx.x == 64) *p.gmax = gmax;
    }
    if (MODE == kThinDz) {
      const int t = threadIdx.x - 64;
      if (t < kThin) {
        float g = 0.f, lse = 0.f;
        if (t < p.l.tokens) {
          lse = p.l.lse[t];
          if (counts(p.l.want, t)) g = p.l.grad[t] / gmax;
        }
        tk.g[t] = g;
        tk.lse[t] = lse;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    const float scale = grads ? *p.gmax * p.gscale : 1.f;
    uint32_t nbox = 0;
    for (uint32_t local = 0;; ++local) {
      int w = -2;
      if (lane == 0 && !take(sh, local, w, lead_empty, abortf, p)) w = -2;
      w = __shfl_sync(0xffffffffu, w, 0);
      if (w < 0) break;
      const Where x = where_is<MODE>(p, w);
      const uint32_t acc = local & 1u;
      const int64_t r0 = int64_t(x.row) * kTile + rank * 128 + q * 32;
      const int c0 = x.col * kTile + half * 128;
      const uint32_t tbase = tmem + acc * kTile + half * 128 + (static_cast<uint32_t>(q * 32) << 16);
      auto wait = [&]() {
        return ptx::mbar_wait_cluster(&sh->tfull[acc], (local >> 1) & 1u, abortf, p.status, kWaitNs);
      };
      auto free = [&]() {  // the accumulator has been read
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(lead_tempty + acc * static_cast<uint32_t>(sizeof(uint64_t)));
      };
      bool ok;
      if (thin) {
        const int base_v = p.l.v0 + x.col * p.thin_h + rank * (p.thin_h / 2);
        const int last = min(min(base_v + p.thin_h / 2, p.l.v0 + p.l.width), base_v + q * 32 + 32);
        const uint32_t rows = tmem + acc * kTile + (static_cast<uint32_t>(q * 32) << 16);
        if (MODE == kThinLogits)
          ok = drain_thin_logits(p, base_v + q * 32, last, (x.col * 2 + rank) * 4 + q, half, rows, lane, sm, wait,
                                 free);
        else
          ok = drain_thin_dz(p, tk, base_v + q * 32, last, half, rows, lane, sm, wait, free);
      } else if (MODE == kThinGrads && x.kind == 0) {
        const uint32_t rows = tmem + acc * kTile + (static_cast<uint32_t>(q * 32) << 16);
        ok = drain_thin_dh(p, x, x.col * kTile + rank * 128 + q * 32, half, rows, lane, wait, free);
      } else if (MODE == kLogits) {
        ok = drain_logits(p.l, p.zscale, r0 + lane, c0, tbase, lane, sm, wait, free);
      } else if (MODE == kDz) {
        ok = drain_dz(p, gmax, r0 + lane, r0, p.l.v0 + c0, tbase, lane, stg, nbox, wait, free);
      } else if (MODE == kThinGrads) {
        ok = drain_thin_dw(p, scale, p.l.v0 + static_cast<int>(r0), p.l.vocab, c0, tbase, lane, stg, wait, free);
      } else {
        const int64_t row = r0 + (x.kind == 1 ? p.l.v0 : 0);
        ok = drain_grads(p, x, scale, row, x.kind == 1 ? p.l.vocab : p.l.tokens, c0, tbase, lane, stg, nbox, wait, free);
      }
      if (!ok) break;
    }
    ptx::bulk_wait_all();
  }

  __syncthreads();
  if (threadIdx.x == 0) {
    // every claim precedes its CTA's arrival here; the last CTA leaves both words zero for the next launch
    __threadfence();
    if (atomicAdd(p.sched + 1, 1u) == gridDim.x - 1) {
      p.sched[0] = 0u;
      p.sched[1] = 0u;
    }
  }
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ host
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

cudaError_t encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz) {
  auto fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = fn(m, type, rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Row-major bf16 rows x cols in boxes of box_rows x box_cols. Reads past either edge give zeros.
cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols,
                     int box_rows, CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dims, strides, box, swz);
}

// The same matrix as [block of 64 columns][row][64 columns], so that one box brings box_rows rows of two blocks,
// each a block of 128-byte rows as the MN-major operand wants them. cols must be a multiple of 64.
cudaError_t map_blocks(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 2};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t map_operand_mn(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld,
                           int box_rows = kStep) {
  return cols % 64 == 0 ? map_blocks(m, base, cols, rows, ld, box_rows)
                        : map_rows(m, base, cols, rows, ld, 64, box_rows);
}

int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

static_assert(kTwofold <= kStep && kTwofold <= kThin && 2 * kTwofold <= kTile, "a stage of dW, the N side of dH^T");
int32_t low_rows(int64_t tokens) { return tokens <= kTwofold ? static_cast<int32_t>(tokens) : 0; }

template <int MODE>
cudaError_t launch_pairs(const Params& p, int pairs, cudaStream_t s) {
  // (gradients of few tokens: one stage less and boxes twice as large, the same total)
  static_assert(2 * kHalf == kEpiWarps * 2 * (kWideBox - kBox), "both layouts fill the same shared memory");
  const size_t smem =
      1024 + kRingBytes + 1024 + kEpiWarps * 2 * kBox + (MODE == kThinDz ? sizeof(ThinTokens) : 0);
  cudaError_t e = cudaFuncSetAttribute(head_pair_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_follow(head_pair_kernel<MODE>, dim3(2 * std::min(pairs, p.items)), kThreads, smem, s, 2, p);
}

// A launch over `entries` of the vocabulary (from p.v0): tiles, operand maps and words of the workspace.
cudaError_t logit_launch(Params& P, const LogitParams& p, const Pipe& pipe) {
  std::memset(&P, 0, sizeof(P));
  P.l = p;
  P.zscale = static_cast<float>(p.in.scale * (1.0 + kTruncated * p.in.dim));
  P.nk = cdiv(p.in.dim, kStep);
  P.sched = pipe.sched;
  P.status = pipe.status;
  P.gmax = pipe.gmax;
  int w_rows = 128, h_rows = 128;
  if (thin_tokens(p.tokens)) {
    const Thin x = thin_tiles(p.width, pipe.pairs);
    P.thin_n = cdiv(p.tokens, 32) * 32;
    P.thin_h = x.height;
    P.low = low_rows(p.tokens);
    P.rows = 1;
    P.cols = P.items = x.tiles;
    w_rows = P.thin_h / 2;
    h_rows = P.thin_n / 2;
    P.a_bytes = w_rows * kStep * 2;
    P.stage_bytes = P.a_bytes + h_rows * kStep * 2;
    P.stages = std::min(kMaxStages, kRingBytes / P.stage_bytes);
  } else {
    P.rows = cdiv(p.tokens, kTile);
    P.cols = cdiv(p.width, kTile);
    P.items = P.rows * P.cols;
  }
  cudaError_t e = map_rows(&P.a[0], p.in.hidden, p.in.dim, p.tokens, p.in.ld_hidden, kStep, h_rows);
  if (e == cudaSuccess) e = map_rows(&P.b[0], p.in.weight, p.in.dim, p.vocab, p.in.ld_weight, kStep, w_rows);
  return e;
}

}  // namespace

bool thin_tokens(int64_t tokens) { return tokens <= kThin; }

// Heights of at most 256 that spread the entries evenly over whole rounds of the pairs: 32000 entries on 76
// pairs make two rounds of 216 rather than 125 tiles of 256, of which the second round has 49.
Thin thin_tiles(int64_t entries, int pairs) {
  const int rounds = cdiv(entries, int64_t(kTile) * pairs);
  Thin x;
  x.height = std::max(16, cdiv(cdiv(entries, int64_t(rounds) * pairs), 16) * 16);
  x.tiles = cdiv(entries, x.height);
  return x;
}

int logit_groups(int64_t tokens, int64_t vocab, int pairs) {
  return thin_tokens(tokens) ? thin_tiles(vocab, pairs).tiles * 8 : cdiv(vocab, kGroup);
}

cudaError_t launch_logits(const LogitParams& p, const Pipe& pipe, cudaStream_t s) {
  Params P;
  const cudaError_t e = logit_launch(P, p, pipe);
  if (e != cudaSuccess) return e;
  return P.thin_n != 0 ? launch_pairs<kThinLogits>(P, pipe.pairs, s) : launch_pairs<kLogits>(P, pipe.pairs, s);
}

cudaError_t launch_dz(const LogitParams& p, const Pipe& pipe, cudaStream_t s) {
  Params P;
  cudaError_t e = logit_launch(P, p, pipe);
  if (e == cudaSuccess && P.thin_n == 0)
    e = map_rows(&P.out[0], p.dz, p.ld_dz, p.tokens, p.ld_dz, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (e != cudaSuccess) return e;
  return P.thin_n != 0 ? launch_pairs<kThinDz>(P, pipe.pairs, s) : launch_pairs<kDz>(P, pipe.pairs, s);
}

// K is cut where whole dH tiles would keep a few pairs busy after all others are done: until a slice's K
// is no longer than the launch's work per pair. Each slice has sums of its own, joined by the rounding
// kernel in a fixed order.
Slices dh_slices(int64_t tokens, int64_t dim, int64_t width, bool dweight, int pairs) {
  const int64_t tiles = int64_t(cdiv(tokens, kTile)) * cdiv(dim, kTile);
  const int64_t nk = cdiv(width, kStep);
  // a tile of dW takes the time of 4 stages at least: it writes 128 KB
  const int64_t dw =
      dweight ? int64_t(cdiv(width, kTile)) * cdiv(dim, kTile) * std::max(4, cdiv(tokens, kStep)) : 0;
  const int64_t fair = std::max<int64_t>(16, cdiv(tiles * nk + dw, pairs));
  int64_t count = cdiv(nk, fair);
  if (!dweight && tiles < pairs) count = std::min<int64_t>(count, pairs / tiles);  // one round of the pairs
  Slices x;
  x.nk = cdiv(nk, count);
  x.count = cdiv(nk, x.nk);
  return x;
}

cudaError_t launch_grads(const GradParams& p, const Pipe& pipe, cudaStream_t s) {
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.l.tokens = p.tokens;
  P.l.vocab = p.v0 + p.width;
  P.l.in.dim = p.dim;
  P.l.v0 = p.v0;
  P.dim_tiles = cdiv(p.dim, kTile);
  P.thin_n = thin_tokens(p.tokens) ? cdiv(p.tokens, 32) * 32 : 0;
  P.low = low_rows(p.tokens);
  const int64_t dz_rows = p.tokens + P.low;
  P.chunked = p.dim % 64 == 0;
  P.gscale = p.gscale;
  P.gmax = pipe.gmax;
  P.sched = pipe.sched;
  P.status = pipe.status;
  cudaError_t e = cudaSuccess;
  const int64_t acc_ld = acc_pitch(p.dim);
  if (p.dhidden != nullptr || p.dh_acc != nullptr) {
    P.dh_rows = cdiv(p.tokens, kTile);
    P.dh_nk = cdiv(p.width, kStep);
    P.slice_nk = p.slices.nk;
    P.slices = cdiv(P.dh_nk, P.slice_nk);
    P.dh_items = P.dh_rows * P.dim_tiles * P.slices;
    P.dh_direct = p.dhidden != nullptr;
    P.first = p.first;
    P.dh_acc = p.dh_acc;
    P.acc_ld = acc_ld;
    e = map_rows(&P.a[0], p.dz, p.width, dz_rows, p.ld_dz, kStep,
                 P.low != 0 ? P.thin_n : P.thin_n != 0 ? P.thin_n / 2 : 128);
    if (e == cudaSuccess) e = map_operand_mn(&P.b[0], p.weight, p.dim, p.vocab, p.ld_weight);
    if (e == cudaSuccess && P.dh_direct) {
      e = map_rows(&P.out[0], p.dhidden, p.dim, p.tokens, p.ld_dhidden, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    } else if (e == cudaSuccess && P.thin_n == 0) {
      const cuuint64_t dims[3] = {(cuuint64_t)p.dim, (cuuint64_t)p.tokens, (cuuint64_t)p.slices.count};
      const cuuint64_t strides[2] = {(cuuint64_t)acc_ld * 4, (cuuint64_t)acc_ld * 4 * p.tokens};
      const cuuint32_t box[3] = {16, 32, 1};
      e = encode(&P.out[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.dh_acc, 3, dims, strides, box,
                 CU_TENSOR_MAP_SWIZZLE_64B);
    }
  }
  if (e != cudaSuccess) return e;
  P.items = P.dh_items;
  if (p.dweight != nullptr) {
    P.items += cdiv(p.width, kTile) * P.dim_tiles;
    P.nk = P.low != 0 ? 2 : cdiv(p.tokens, kStep);
    // no more zeros than the MMA's 16 of K asks for: they are written and read all the same
    P.dw_rows = P.low != 0 ? cdiv(p.tokens, 16) * 16 : kStep;
    e = map_blocks(&P.a[1], p.dz, p.ld_dz, dz_rows, p.ld_dz, P.dw_rows);
    if (e == cudaSuccess) e = map_operand_mn(&P.b[1], p.hidden, p.dim, p.tokens, p.ld_hidden, P.dw_rows);
    if (e == cudaSuccess)
      e = P.thin_n != 0 ? map_rows(&P.out[1], p.dweight, p.dim, p.vocab, p.ld_dweight, 64, 32)
                        : map_rows(&P.out[1], p.dweight, p.dim, p.vocab, p.ld_dweight, 32, 32,
                                   CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;
  }
  return P.thin_n != 0 ? launch_pairs<kThinGrads>(P, pipe.pairs, s) : launch_pairs<kGrads>(P, pipe.pairs, s);
}

}  // namespace head
}  // namespace dmuon
