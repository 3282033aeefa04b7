// head_top.cu - the largest logits of each token, with their ids: the alternatives that a scoring call returns.
//
// The logits of one piece of the vocabulary lie in memory, and each group's largest is known. A token's `held`
// largest entries, in the order (logit descending, id ascending), lie in the `held` first groups in the order
// (largest logit descending, group ascending): of an entry in another group, each of those groups has one that comes
// before it. So of the logits only those groups' are read.
//
// Logits come from the tensor cores in fp32, off by about 1e-6 of themselves; alternatives nearer to each other than
// that would change places with the way the product is cut. `top` + kSpare entries are held, and where neighbours are
// too near to tell, their products are formed again with compensated sums, which decide the order.
//
// A warp per token: the search for the last of `held` peaks is a count over the warp for each bit that they differ in,
// without a barrier. (A block per token took 105 us for 4093 tokens x 32768 entries, 15 us for one token.)
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "head.h"
#include "head_dot.cuh"
#include "head_score.cuh"

namespace dmuon {
namespace head {
namespace {

constexpr int kTopWarps = 8;
constexpr int kCandidates = 256;  // that a warp has room for

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
  uint64_t cand[kCandidates];     // (logit, ~id)
  uint64_t sorted[kHeld];
  uint64_t exact[kHeld];
  int wanted[kHeld];              // groups
};

// The largest number that at least `want` of the warp's numbers reach (they lie between low and high, and there are
// so many); `count(limit)` says how many of this lane's reach a limit. Stops where exactly `want` do.
template <typename T, class Count>
__device__ __forceinline__ T threshold(int want, T low, T high, Count&& count) {
  const T differ = low ^ high;
  if (differ == 0) return high;
  int bit = sizeof(T) == 8 ? 63 - __clzll(static_cast<long long>(differ)) : 31 - __clz(static_cast<int>(differ));
  T at = bit + 1 < static_cast<int>(sizeof(T)) * 8 ? high >> (bit + 1) << (bit + 1) : 0;  // what they share
  for (; bit >= 0; --bit) {
    const T next = at | (T(1) << bit);
    const int n = __reduce_add_sync(0xffffffffu, count(next));
    if (n >= want) at = next;
    if (n == want) break;
  }
  return at;
}

// Leaves the first `held` of n candidates, in any order.
__device__ __forceinline__ int compress(TopShared& sh, int n, int held, int lane) {
  if (n <= held) return n;
  __syncwarp();
  uint64_t mine[kCandidates / 32];
#pragma unroll
  for (int k = 0; k < kCandidates / 32; ++k) mine[k] = k * 32 + lane < n ? sh.cand[k * 32 + lane] : 0;
  const uint64_t least = threshold<uint64_t>(held, 0, ~uint64_t(0), [&](uint64_t limit) {
    int c = 0;
#pragma unroll
    for (int k = 0; k < kCandidates / 32; ++k) c += mine[k] >= limit;
    return c;
  });
  __syncwarp();
  int at = 0;
#pragma unroll
  for (int k = 0; k < kCandidates / 32; ++k) {
    const bool on = mine[k] >= least && mine[k] != 0;
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (on) sh.cand[at + __popc(b & ((1u << lane) - 1u))] = mine[k];
    at += __popc(b);
  }
  __syncwarp();
  return at;
}

__device__ __forceinline__ void two_sum(float& sum, float& rest, float x) {
  const float s = sum + x, b = s - sum;
  rest += (sum - (s - b)) + (x - b);
  sum = s;
}

// A logit (unscaled) by one warp: products of bf16 are exact in fp32, their sums are compensated. Four rounds of loads
// are in flight, as the trip to memory is what it takes.
__device__ __forceinline__ double exact_dot(const DotParams& d, int64_t t, int64_t v, int lane) {
  float sum = 0.f, rest = 0.f;
  const bf16 *h = d.hidden + t * d.ld_hidden, *w = d.weight + v * d.ld_weight;
  const int whole = d.dim / 8;
  for (int c0 = lane; c0 < whole; c0 += 4 * 32) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = c0 + 32 * u < whole;
      a[u] = in ? *reinterpret_cast<const uint4*>(h + 8 * (c0 + 32 * u)) : make_uint4(0, 0, 0, 0);
      b[u] = in ? *reinterpret_cast<const uint4*>(w + 8 * (c0 + 32 * u)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162*>(&a[u]),
                           *y = reinterpret_cast<const __nv_bfloat162*>(&b[u]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(x[k]), g = __bfloat1622float2(y[k]);
        two_sum(sum, rest, f.x * g.x);
        two_sum(sum, rest, f.y * g.y);
      }
    }
  }
  for (int k = 8 * whole + lane; k < d.dim; k += 32) two_sum(sum, rest, __bfloat162float(h[k]) * __bfloat162float(w[k]));
  double s = static_cast<double>(sum) + static_cast<double>(rest);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The first `held` of n keys in the order (key descending, number ascending): take(place, number, key) for each, by
// ascending number. Returns how many. KEYS: n is at most 32 * KEYS, and the keys are held in registers; 0: any n,
// read again each time. read(i) gives a key for i < n; keys of 0 are not there.
template <int KEYS, class Read, class Take>
__device__ __forceinline__ int pick(int n, int held, int lane, Read&& read, Take&& take) {
  const int turns = KEYS != 0 ? KEYS : (n + 31) / 32;
  uint32_t key[KEYS != 0 ? KEYS : 1] = {};
  auto at = [&](int k) { return KEYS != 0 ? key[k] : k * 32 + lane < n ? read(k * 32 + lane) : 0u; };
  uint32_t low = 0xffffffffu, high = 0u;
  int there = 0;
#pragma unroll
  for (int k = 0; k < turns; ++k) {
    const uint32_t v = k * 32 + lane < n ? read(k * 32 + lane) : 0u;
    if (KEYS != 0) key[k] = v;
    if (v != 0u) low = min(low, v);
    high = max(high, v);
    there += v != 0u;
  }
  uint32_t least = 1u;  // keys above it are among the first, and of those at it the first `level`
  int level = held;
  if (__reduce_add_sync(0xffffffffu, there) > held) {
    least = threshold<uint32_t>(held, __reduce_min_sync(0xffffffffu, low), __reduce_max_sync(0xffffffffu, high),
                                [&](uint32_t limit) {
                                  int c = 0;
#pragma unroll
                                  for (int k = 0; k < turns; ++k) c += at(k) >= limit;
                                  return c;
                                });
    int above = 0;
#pragma unroll
    for (int k = 0; k < turns; ++k) above += at(k) > least;
    level = held - __reduce_add_sync(0xffffffffu, above);
  }
  int taken = 0;
#pragma unroll
  for (int k = 0; k < turns; ++k) {
    const uint32_t v = at(k);
    const unsigned same = __ballot_sync(0xffffffffu, v == least);
    const bool on = v > least || (v == least && __popc(same & ((1u << lane) - 1u)) < level);
    level -= __popc(same);
    const unsigned w = __ballot_sync(0xffffffffu, on);
    if (on) take(taken + __popc(w & ((1u << lane) - 1u)), k * 32 + lane, v);
    taken += __popc(w);
  }
  return taken;
}

// A group's key: its peak in order, above 0 (where only a NaN would lie).
__device__ __forceinline__ uint32_t peak_of(const TopParams& p, int64_t t, int g) {
  return max(order_of(p.parts[t * p.token_step + g * p.group_step].peak), 1u);
}

// A token's alternatives among the entries of `wanted` groups, whose peaks are at least `least`, the target and the
// list so far. `scored` returns once the token's log sum and probability are there.
template <class Scored>
__device__ __forceinline__ void top_of(const TopParams& p, int64_t t, int lane, TopShared& sh, int wanted, uint32_t least,
                                       Scored&& scored) {
  const int held = p.top + kSpare;
  // ---------------------------------------------------------- their entries, the target, and the list so far
  const int64_t y = p.targets != nullptr ? p.targets[t] : -1;
  const float* z = p.z + t * p.ld_z;
  int n = 0;
  auto add = [&](bool on, float v, int id) {
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (on)
      sh.cand[n + __popc(b & ((1u << lane) - 1u))] =
          (static_cast<uint64_t>(order_of(v)) << 32) | (~static_cast<uint32_t>(id));
    n += __popc(b);
  };
  constexpr int kBatch = 4;  // groups whose loads are in flight together
  for (int i0 = 0; i0 < wanted; i0 += kBatch) {
    float4 v[kBatch];
    int id[kBatch], end[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      id[u] = end[u] = 0;
      if (i0 + u >= wanted) continue;
      const int g = sh.wanted[i0 + u];
      end[u] = p.v0 + p.width;
      if (p.thin_h != 0) {  // tile g / 8, half g / 4 % 2, 32 entries from g % 4 * 32
        const int first = p.v0 + (g >> 3) * p.thin_h + ((g >> 2) & 1) * (p.thin_h / 2);
        end[u] = min(end[u], first + p.thin_h / 2);
        id[u] = first + (g & 3) * 32 + lane;
        if (id[u] < end[u]) v[u].x = z[id[u] - p.v0];
      } else {  // four entries a lane; past the last group's the row goes on to a multiple of 256
        id[u] = p.v0 + g * kGroup + 4 * lane;
        v[u] = *reinterpret_cast<const float4*>(z + (id[u] - p.v0));
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i0 + u >= wanted) break;
      if (n > kCandidates - kGroup) n = compress(sh, n, held, lane);
      const float w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k > 0 && p.thin_h != 0) break;
        add(id[u] + k < end[u] && id[u] + k != y && order_of(w[k]) >= least, w[k], id[u] + k);
      }
    }
  }
  if (n > kCandidates - kHeld - 1) n = compress(sh, n, held, lane);
  // the groups' peaks leave the target out: its logit goes in by itself
  const bool here = y >= p.v0 && y < p.v0 + p.width;
  if (here) add(lane == 0, z[y - p.v0], static_cast<int>(y));
  if (!p.first)
    for (int i = lane; i - lane < held; i += 32) {
      const int id = i < held ? p.list_id[t * kHeld + i] : -1;
      add(id >= 0, id >= 0 ? p.list_z[t * kHeld + i] : 0.f, id);
    }
  __syncwarp();

  // ---------------------------------------------------------- the first of them, in order
  const int keep = min(n, held);
  for (int i = lane; i < n; i += 32) {
    const uint64_t mine = sh.cand[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += sh.cand[j] > mine;
    if (place < keep) sh.sorted[place] = mine;
  }
  __syncwarp();
  auto z_at = [&](int i) { return value_of(static_cast<uint32_t>(sh.sorted[i] >> 32)); };
  auto id_at = [&](int i) { return static_cast<int>(~static_cast<uint32_t>(sh.sorted[i])); };
  if (!p.last) {
    for (int i = lane; i < held; i += 32) {
      p.list_z[t * kHeld + i] = i < keep ? z_at(i) : 0.f;
      p.list_id[t * kHeld + i] = i < keep ? id_at(i) : -1;
    }
    return;
  }

  // ---------------------------------------------------------- neighbours too near to tell
  // What two products may be off by against each other: at most 2.2e-9 * dim of the largest partial sum of each, which
  // is their logit and some standard deviations of the rest; twice that (at 4096 dims 5e-4 at a logit of 12), and
  // no less than what fp32 sums of 512 terms have.
  const float part = 6e-9f * fmaxf(512.f, static_cast<float>(p.dot.dim));
  uint64_t starts = 0;  // places whose entry is surely below the one before
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 32 * h + lane;
    bool apart = true;
    if (i > 0 && i < keep) {
      const float a = z_at(i - 1), b = z_at(i);
      apart = a - b > part * (8.f * p.dot.scale + fabsf(a));
    }
    starts |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, apart)) << (32 * h);
  }
  // entry i shares its place where it or the next one is not a start; its run begins at the last start up to it
  auto begin = [&](int i) { return 63 - __clzll(static_cast<long long>(starts & ((uint64_t(2) << i) - 1))); };
  auto shared = [&](int i) { return begin(i) < p.top && (~(starts >> i) & (i + 1 < keep ? 3 : 1)) != 0; };
  for (int i = 0; i < keep; ++i)
    if (shared(i)) {
      const double d = exact_dot(p.dot, t, id_at(i), lane);
      if (lane == 0) sh.exact[i] = order_of(d + 0.0);
    }
  __syncwarp();
  scored();
  const float lse = p.lse[t], logp = p.logp[t];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 32 * h + lane;
    if (i >= keep) continue;
    int place = i;
    const int id = id_at(i);
    if (shared(i)) {
      place = begin(i);
      for (int j = place; j < keep && begin(j) == begin(i); ++j)
        place += sh.exact[j] > sh.exact[i] || (sh.exact[j] == sh.exact[i] && id_at(j) < id);
    }
    if (place < p.top) {
      p.top_ids[t * p.top + place] = id;
      p.top_logp[t * p.top + place] = id == y ? logp : z_at(i) - lse;
    }
  }
  for (int i = keep + lane; i < p.top; i += 32) {
    p.top_ids[t * p.top + i] = -1;
    p.top_logp[t * p.top + i] = -INFINITY;
  }
}

template <int KEYS>
__global__ void __launch_bounds__(32 * kTopWarps) top_kernel(const __grid_constant__ TopParams p) {
  __shared__ TopShared all[kTopWarps];
  follow();
  const int lane = threadIdx.x & 31;
  TopShared& sh = all[threadIdx.x >> 5];
  const int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  uint32_t least = 0xffffffffu;
  const int wanted = pick<KEYS>(p.groups, p.top + kSpare, lane, [&](int g) { return peak_of(p, t, g); },
                                [&](int place, int g, uint32_t key) {
                                  sh.wanted[place] = g;
                                  least = min(least, key);
                                });
  least = __reduce_min_sync(0xffffffffu, least);
  __syncwarp();
  top_of(p, t, lane, sh, wanted, p.groups > wanted ? least : 0u, [] {});
}

// Few tokens: a block each. Eight warps find the first groups, each of an eighth of them, and the first warp of those
// and the alternatives; meanwhile eight others join the groups' sums.
constexpr int kJoinThreads = 256;  // as where no alternatives are asked for: the same sums
template <int KEYS>
__global__ void __launch_bounds__(32 * kTopWarps + kJoinThreads) score_top_kernel(const __grid_constant__ ScoreParams r,
                                                                                  const __grid_constant__ TopParams p) {
  __shared__ TopShared sh;
  __shared__ ScoreShared<1, kJoinThreads> rows;
  __shared__ uint32_t first_key[kTopWarps * kHeld];
  __shared__ int first_group[kTopWarps * kHeld];
  follow();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= kTopWarps) {
    score_rows<1, kJoinThreads>(r, t, threadIdx.x - 32 * kTopWarps, rows, [] { asm volatile("bar.sync 1, 256;" ::: "memory"); });
    __syncthreads();
    return;
  }
  const int held = p.top + kSpare, share = (p.groups + kTopWarps - 1) / kTopWarps;
  const int begin = min(warp * share, p.groups), n = min(share, p.groups - begin);
  for (int i = lane; i < kHeld; i += 32) first_key[warp * kHeld + i] = 0u;
  __syncwarp();
  pick<KEYS>(n, held, lane, [&](int i) { return peak_of(p, t, begin + i); },
             [&](int place, int i, uint32_t key) {
               first_key[warp * kHeld + place] = key;
               first_group[warp * kHeld + place] = begin + i;
             });
  asm volatile("bar.sync 2, 256;" ::: "memory");
  if (warp == 0) {
    uint32_t least = 0xffffffffu;
    const int wanted = pick<kTopWarps * kHeld / 32>(kTopWarps * kHeld, held, lane, [&](int i) { return first_key[i]; },
                                                    [&](int place, int i, uint32_t key) {
                                                      sh.wanted[place] = first_group[i];
                                                      least = min(least, key);
                                                    });
    least = __reduce_min_sync(0xffffffffu, least);
    __syncwarp();
    top_of(p, t, lane, sh, wanted, p.groups > wanted ? least : 0u, [] { __syncthreads(); });
  } else {
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_top(const TopParams& p, cudaStream_t s) {
  // as many warps to a block as leave each SM one: the tokens of a block lie next to each other in the groups' sums
  const int warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kTopWarps, p.tokens / 128)));
  const dim3 grid(static_cast<unsigned>((p.tokens + warps - 1) / warps));
  if (p.groups <= 256) return launch_follow(top_kernel<8>, grid, 32 * warps, 0, s, 1, p);
  if (p.groups <= 1024) return launch_follow(top_kernel<32>, grid, 32 * warps, 0, s, 1, p);
  return launch_follow(top_kernel<0>, grid, 32 * warps, 0, s, 1, p);
}

cudaError_t launch_score_top(const ScoreParams& r, const TopParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.tokens));
  const int threads = 32 * kTopWarps + kJoinThreads;
  if (p.groups <= 256 * kTopWarps) return launch_follow(score_top_kernel<8>, grid, threads, 0, s, 1, r, p);
  if (p.groups <= 1024 * kTopWarps) return launch_follow(score_top_kernel<32>, grid, threads, 0, s, 1, r, p);
  return launch_follow(score_top_kernel<0>, grid, threads, 0, s, 1, r, p);
}

}  // namespace head
}  // namespace dmuon
