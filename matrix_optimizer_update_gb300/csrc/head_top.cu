// head_top.cu - the largest logits of each token, with their ids: the alternatives that a scoring call returns.
//
// The logits of one piece of the vocabulary lie in memory, and each group's largest is known. A token's `held`
// largest entries, in the order (logit descending, id ascending), lie in the `held` first groups in the order
// (largest logit descending, group ascending): of an entry in another group, each of those groups has one that comes
// before it. So a block per token reads the groups' peaks, and of the logits only those groups'.
//
// Logits come from the tensor cores in fp32, off by about 1e-6 of themselves; alternatives nearer to each other than
// that would change places with the way the product is cut. `top` + kSpare entries are held, and where neighbours are
// too near to tell, their products are formed again with compensated sums, which decide the order.
#include <algorithm>
#include <climits>
#include <cmath>

#include "follow.cuh"
#include "head.h"
#include "head_dot.cuh"

namespace dmuon {
namespace head {
namespace {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kRanked = 512;       // so many candidates are put in order by counting
constexpr int kStagedGroups = 4096;  // so many groups' peaks are kept in shared memory

// Unsigned numbers in the order of the floats (NaN above or below all others, by its sign).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) != 0 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) != 0 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  return (u >> 63) != 0 ? ~u : u | (uint64_t(1) << 63);
}

struct TopShared {
  int red[2][kTopWarps];
  int wanted[kHeld];        // groups
  int groups, candidates;
  uint64_t sorted[kHeld + 1];
  int cluster[kHeld + 1];   // first place of those it cannot be told from
  uint64_t exact[kHeld + 1];
};

// The sum over the block; `turn` alternates between calls, so that one barrier is enough.
__device__ __forceinline__ int block_count(TopShared& sh, int n, int& turn) {
  n = __reduce_add_sync(0xffffffffu, n);
  int* red = sh.red[turn & 1];
  ++turn;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) all += red[w];
  return all;
}

// The largest number that at least `want` keys reach (all keys are at least 0; there are at least `want`), found bit
// by bit; `count(limit)` says how many of this thread's keys reach a limit. Stops where exactly `want` do.
template <typename T, class Count>
__device__ __forceinline__ T threshold(TopShared& sh, int want, int& turn, Count&& count) {
  T at = 0;
  for (int bit = static_cast<int>(sizeof(T)) * 8 - 1; bit >= 0; --bit) {
    const T next = at | (T(1) << bit);
    const int n = block_count(sh, count(next), turn);
    if (n >= want) at = next;
    if (n == want) break;
  }
  return at;
}

__device__ __forceinline__ void two_sum(float& sum, float& rest, float x) {
  const float s = sum + x, b = s - sum;
  rest += (sum - (s - b)) + (x - b);
  sum = s;
}

// A logit (unscaled) by one warp: products of bf16 are exact in fp32, their sums are compensated.
__device__ __forceinline__ double exact_dot(const DotParams& d, int64_t t, int64_t v, int lane) {
  float sum = 0.f, rest = 0.f;
  const bf16 *h = d.hidden + t * d.ld_hidden, *w = d.weight + v * d.ld_weight;
  const int whole = d.dim / 8;
#pragma unroll 2
  for (int c = lane; c < whole; c += 32) {
    const uint4 a = *reinterpret_cast<const uint4*>(h + 8 * c), b = *reinterpret_cast<const uint4*>(w + 8 * c);
    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162*>(&a),
                         *y = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(x[k]), g = __bfloat1622float2(y[k]);
      two_sum(sum, rest, f.x * g.x);
      two_sum(sum, rest, f.y * g.y);
    }
  }
  for (int k = 8 * whole + lane; k < d.dim; k += 32) two_sum(sum, rest, __bfloat162float(h[k]) * __bfloat162float(w[k]));
  double s = static_cast<double>(sum) + static_cast<double>(rest);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__global__ void __launch_bounds__(kTopThreads) top_kernel(const __grid_constant__ TopParams p) {
  extern __shared__ __align__(8) uint8_t dynamic[];
  __shared__ TopShared sh;
  uint32_t* peaks = reinterpret_cast<uint32_t*>(dynamic);   // the groups', then
  uint64_t* cand = reinterpret_cast<uint64_t*>(dynamic);    // (logit, ~id) of the candidates
  follow();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int held = p.top + kSpare;
  int turn = 0;

  // ---------------------------------------------------------- the groups with the largest peaks
  const Part* parts = p.parts + t * p.token_step;
  const bool staged = p.groups <= kStagedGroups;
  auto peak_of = [&](int g) { return staged ? peaks[g] : order_of(parts[g * p.group_step].peak); };
  if (staged)
    for (int g = tid; g < p.groups; g += kTopThreads) peaks[g] = order_of(parts[g * p.group_step].peak);
  if (tid == 0) sh.groups = sh.candidates = 0;
  __syncthreads();
  uint32_t least = 0;      // logits below it are not among the largest
  int up_to = INT_MAX;     // of groups whose peak is `least`, those before
  if (p.groups > held) {
    least = threshold<uint32_t>(sh, held, turn, [&](uint32_t limit) {
      int n = 0;
      for (int g = tid; g < p.groups; g += kTopThreads) n += peak_of(g) >= limit;
      return n;
    });
    int above = 0, level = 0;
    for (int g = tid; g < p.groups; g += kTopThreads) {
      above += peak_of(g) > least;
      level += peak_of(g) == least;
    }
    above = block_count(sh, above, turn);
    level = block_count(sh, level, turn);
    if (above + level > held) {
      // the first of the groups that share the last peak: `up_to` counts how many numbers may be too high
      const uint32_t below = threshold<uint32_t>(sh, held - above, turn, [&](uint32_t limit) {
        int n = 0;
        for (int g = tid; g < p.groups; g += kTopThreads)
          n += peak_of(g) == least && ~static_cast<uint32_t>(g) >= limit;
        return n;
      });
      up_to = static_cast<int>(~below);  // groups 0 .. up_to
    }
  }
  for (int g = tid; g < p.groups; g += kTopThreads) {
    const uint32_t k = peak_of(g);
    if (k > least || (k == least && g <= up_to)) {
      const int at = atomicAdd(&sh.groups, 1);
      if (at < held) sh.wanted[at] = g;
    }
  }
  __syncthreads();

  // ---------------------------------------------------------- their entries, and the list so far
  const int64_t y = p.targets != nullptr ? p.targets[t] : -1;
  const int per = p.thin_h != 0 ? 32 : kGroup, wanted = min(sh.groups, held);
  auto add = [&](float z, int id) {
    cand[atomicAdd(&sh.candidates, 1)] = (static_cast<uint64_t>(order_of(z)) << 32) | (~static_cast<uint32_t>(id));
  };
  for (int i = tid; i < wanted * per; i += kTopThreads) {
    const int g = sh.wanted[i / per];
    int id, end = p.v0 + p.width;
    if (p.thin_h != 0) {  // tile g / 8, half g / 4 % 2, 32 entries from g % 4 * 32
      const int first = p.v0 + (g >> 3) * p.thin_h + ((g >> 2) & 1) * (p.thin_h / 2);
      end = min(end, first + p.thin_h / 2);
      id = first + (g & 3) * 32 + i % per;
    } else {
      id = p.v0 + g * kGroup + i % per;
    }
    if (id >= end || id == y) continue;
    const float z = p.z[t * p.ld_z + (id - p.v0)];
    if (order_of(z) >= least) add(z, id);
  }
  if (!p.first)
    for (int i = tid; i < held; i += kTopThreads)
      if (p.list_id[t * kHeld + i] >= 0) add(p.list_z[t * kHeld + i], p.list_id[t * kHeld + i]);
  // the groups' peaks leave the target out: its logit goes in by itself
  if (tid == 0 && y >= p.v0 && y < p.v0 + p.width) add(p.z[t * p.ld_z + (y - p.v0)], static_cast<int>(y));
  __syncthreads();
  int n = sh.candidates;

  // ---------------------------------------------------------- the first of them, in order
  const int keep = min(n, held);
  uint64_t reach = 0;
  if (n > kRanked)
    reach = threshold<uint64_t>(sh, keep, turn, [&](uint64_t limit) {
      int m = 0;
      for (int i = tid; i < n; i += kTopThreads) m += cand[i] >= limit;
      return m;
    });
  for (int i = tid; i < n; i += kTopThreads) {
    const uint64_t mine = cand[i];
    if (mine < reach) continue;
    int place = 0;
    for (int j = 0; j < n; ++j) place += cand[j] > mine;
    if (place < keep) sh.sorted[place] = mine;
  }
  __syncthreads();
  if (!p.last) {
    for (int i = tid; i < held; i += kTopThreads) {
      p.list_z[t * kHeld + i] = i < keep ? value_of(static_cast<uint32_t>(sh.sorted[i] >> 32)) : 0.f;
      p.list_id[t * kHeld + i] = i < keep ? static_cast<int>(~static_cast<uint32_t>(sh.sorted[i])) : -1;
    }
    return;
  }

  // ---------------------------------------------------------- neighbours too near to tell
  auto z_at = [&](int i) { return value_of(static_cast<uint32_t>(sh.sorted[i] >> 32)); };
  auto id_at = [&](int i) { return static_cast<int>(~static_cast<uint32_t>(sh.sorted[i])); };
  if (tid == 0) {
    // what the products may be off by: 2^-14 of the logits up to 16384 dims, in proportion above (header: 2e-9 * dim)
    const float part = 0x1p-14f * fmaxf(1.f, p.dot.dim / 16384.f);
    for (int i = 0; i < keep; ++i) {
      const float a = i > 0 ? z_at(i - 1) : 0.f, b = z_at(i);
      const bool apart = i == 0 || a - b > part * (p.dot.scale + fabsf(a));
      sh.cluster[i] = apart ? i : sh.cluster[i - 1];
    }
  }
  __syncthreads();
  auto shared = [&](int i) {
    const int c = sh.cluster[i];
    return c < p.top && (c != i || (i + 1 < keep && sh.cluster[i + 1] == c));
  };
  for (int i = warp; i < keep; i += kTopWarps)
    if (shared(i)) {
      const double z = exact_dot(p.dot, t, id_at(i), lane);
      if (lane == 0) sh.exact[i] = order_of(z + 0.0);
    }
  __syncthreads();
  if (tid < keep) {
    int place = tid;
    const int c = sh.cluster[tid];
    if (shared(tid)) {
      place = c;
      for (int j = c; j < keep && sh.cluster[j] == c; ++j)
        place += sh.exact[j] > sh.exact[tid] || (sh.exact[j] == sh.exact[tid] && id_at(j) < id_at(tid));
    }
    if (place < p.top) {
      const int id = id_at(tid);
      p.top_ids[t * p.top + place] = id;
      p.top_logp[t * p.top + place] = id == y ? p.logp[t] : z_at(tid) - p.lse[t];
    }
  }
  for (int i = keep + tid; i < p.top; i += kTopThreads) {
    p.top_ids[t * p.top + i] = -1;
    p.top_logp[t * p.top + i] = -INFINITY;
  }
}

}  // namespace

cudaError_t launch_top(const TopParams& p, cudaStream_t s) {
  const int held = p.top + kSpare, per = p.thin_h != 0 ? 32 : kGroup;
  const size_t staged = sizeof(uint32_t) * std::min(p.groups, kStagedGroups);
  const size_t smem = std::max(staged, sizeof(uint64_t) * (held * per + held + 1));
  constexpr size_t most = sizeof(uint64_t) * (kHeld * kGroup + kHeld + 1);
  static_assert(most >= sizeof(uint32_t) * kStagedGroups && most + sizeof(TopShared) < 48 * 1024, "no opt-in needed");
  return launch_follow(top_kernel, dim3(static_cast<unsigned>(p.tokens)), kTopThreads, smem, s, 1, p);
}

}  // namespace head
}  // namespace dmuon
