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
// without a barrier. (A block per token took 105 us for 4093 tokens x 32768 entries, 15 us for one token.) What bounds
// it is one warp's way through its instructions and trips to memory. 20 alternatives of 512 tokens, beside their log
// probabilities alone: 23 us more with 32000 entries, 42 with 128000, of which writing the logits is 10 and 39 at the
// copy rate; 61 tokens: 8 with 50257 entries, 15 with 128000.
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
__device__ __forceinline__ double value_of(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) != 0 ? k & ~(uint64_t(1) << 63) : ~k));
}

// An entry as a number that is the larger the earlier it comes: by logit, then by id from the lowest.
__device__ __forceinline__ uint64_t candidate(float z, int id) {
  return (static_cast<uint64_t>(order_of(z)) << 32) | (~static_cast<uint32_t>(id));
}

struct TopShared {
  uint64_t cand[kCandidates];     // (logit, ~id)
  uint64_t sorted[kHeld];
  uint64_t exact[kHeld];
  int ids[kMaxAlternatives];      // the results
  float values[kMaxAlternatives];
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

// A logit (unscaled) by one warp.
__device__ __forceinline__ double exact_dot(const DotParams& d, int64_t t, int64_t v, int lane) {
  return warp_sum(exact_part<4>(d, t, v, lane, 32)).value();
}

// The largest entries in order, as (logit, ~id), and what is done about neighbours too near to tell.
struct Order {
  const uint64_t* sorted;
  uint64_t* dots;  // exact logits of those that share a run
  int keep, top;

  __device__ __forceinline__ float z(int i) const { return value_of(static_cast<uint32_t>(sorted[i] >> 32)); }
  __device__ __forceinline__ int id(int i) const { return static_cast<int>(~static_cast<uint32_t>(sorted[i])); }

  // The places whose entry is surely below the one before, as bits; by one warp.
  __device__ __forceinline__ uint64_t starts(const TopParams& p, int64_t t, int lane) const {
    // What two products may be off by against each other: at most 2.2e-9 * dim of the largest partial sum of each, which
    // is at most half of the products' absolute values and of the logit. Those are known of one entry, the target where
    // there is one; the others' rows may have twice as much. And no less than 8 / temperature and the logit, twice
    // over, and what fp32 sums of 512 terms have. (At 4096 dims of order 1 and weights of 0.02 1.2e-3 at a logit of 12.)
    const float dim = fmaxf(512.f, static_cast<float>(p.dot.dim)), size = p.sizes[t];
    uint64_t bits = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 32 * h + lane;
      bool apart = true;
      if (i > 0 && i < keep) {
        const float a = z(i - 1), b = z(i);
        apart = a - b > dim * fmaxf(6e-9f * (8.f * p.dot.scale + fabsf(a)), 4.4e-9f * (size + fabsf(a))) &&
                size < INFINITY;
      }
      bits |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, apart)) << (32 * h);
    }
    return bits;
  }
  // The run that entry i belongs to begins at the last start up to it.
  static __device__ __forceinline__ int run(uint64_t starts, int i) {
    return 63 - __clzll(static_cast<long long>(starts & ((uint64_t(2) << i) - 1)));
  }
  // Whether it is not alone there, and the run matters.
  __device__ __forceinline__ bool shared(uint64_t starts, int i) const {
    return run(starts, i) < top && (~(starts >> i) & (i + 1 < keep ? 3 : 1)) != 0;
  }
  // The logits of such entries, of every step-th, by a warp each: `first` is this warp's number of `step`.
  __device__ __forceinline__ void exact_dots(const TopParams& p, int64_t t, uint64_t starts, int first, int step,
                                             int lane) const {
#pragma unroll 1
    for (int h = 0; h < keep; h += 32) {
      const int mine = h + lane;
      unsigned todo = __ballot_sync(0xffffffffu, mine < keep && mine % step == first && shared(starts, mine));
      for (; todo != 0u; todo &= todo - 1u) {
        const int i = h + __ffs(todo) - 1;
        const double d = exact_dot(p.dot, t, id(i), lane);
        if (lane == 0) dots[i] = order_of(d + 0.0);
      }
    }
  }
  // The results, by one warp; ids and values are its shared memory. What entries of a run have is formed from their exact
  // logits, and values follow their order to the last digit: lse and the target's log probability are rounded by themselves.
  __device__ __forceinline__ void results(const TopParams& p, int64_t t, int64_t y, uint64_t starts, int* ids, float* values,
                                          int lane) const {
    const float lse = p.lse[t], logp = p.logp[t];
    if (lane < top) {  // fewer entries than asked for: not finite
      ids[lane] = -1;
      values[lane] = -INFINITY;
    }
    __syncwarp();
#pragma unroll 1
    for (int i = lane; i < keep; i += 32) {
      int place = i;
      const int mine = id(i);
      float value = z(i) - lse;
      if (shared(starts, i)) {
        const int begin = run(starts, i);
        place = begin;
        for (int j = begin; j < keep && run(starts, j) == begin; ++j)
          place += dots[j] > dots[i] || (dots[j] == dots[i] && id(j) < mine);
        value = static_cast<float>(value_of(dots[i]) * p.dot.scale - lse);
      }
      if (place < top) {
        ids[place] = mine;
        values[place] = mine == y ? logp : value;
      }
    }
    __syncwarp();
    const bool in = lane < top;
    const int mine = in ? ids[lane] : -1;
    float value = in ? values[lane] : 0.f;
    const unsigned hit = __ballot_sync(0xffffffffu, in && y >= 0 && mine == y);
    const float pivot = __shfl_sync(0xffffffffu, value, hit != 0u ? __ffs(hit) - 1 : 0);
    if (hit != 0u && mine >= 0) value = (1u << lane) < hit ? fmaxf(value, pivot) : fminf(value, pivot);
    for (int d = 1; d < 32; d <<= 1) {
      const float before = __shfl_up_sync(0xffffffffu, value, d);
      if (lane >= d) value = fminf(value, before);
    }
    if (in) {
      p.top_ids[t * top + lane] = mine;
      p.top_logp[t * top + lane] = value;
    }
  }
};

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
    if (!__any_sync(0xffffffffu, v >= least)) continue;
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
// list so far; by one warp.
__device__ __forceinline__ void top_of(const TopParams& p, int64_t t, int lane, TopShared& sh, int wanted, uint32_t least) {
  const int held = p.top + kSpare;
  // ---------------------------------------------------------- their entries, the target, and the list so far
  const int64_t y = p.targets != nullptr ? p.targets[t] : -1;
  const float* z = p.z + t * p.ld_z;
  int n = 0;
  const int target = y >= p.v0 && y < p.v0 + p.width ? static_cast<int>(y) : -1;
  // This lane's first entry of a group, and where those of its part of the vocabulary end.
  auto first_of = [&](int g, int& end) {
    end = p.v0 + p.width;
    if (p.thin_h == 0) return p.v0 + g * kGroup + 4 * lane;
    const int first = p.v0 + (g >> 3) * p.thin_h + ((g >> 2) & 1) * (p.thin_h / 2);  // tile g / 8, half g / 4 % 2
    end = min(end, first + p.thin_h / 2);
    return first + (g & 3) * 32 + lane;
  };
  constexpr int kBatch = 8;  // groups whose loads are in flight together: a bit for each of 4 entries in a word
  for (int i0 = 0; i0 < wanted; i0 += kBatch) {
    float4 v[kBatch];
    int id[kBatch], end[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      id[u] = end[u] = 0;
      if (i0 + u >= wanted) continue;
      id[u] = first_of(sh.wanted[i0 + u], end[u]);
      if (p.thin_h == 0) {  // four entries a lane; past the last group's the row goes on to a multiple of 256
        v[u] = *reinterpret_cast<const float4*>(z + (id[u] - p.v0));
      } else {
        if (id[u] < end[u]) v[u].x = z[id[u] - p.v0];
        end[u] = min(end[u], id[u] + 1);
      }
    }
    // Which of them count, a bit each (without a branch: lanes that part and meet again for each of four conditions
    // took 85 cycles an entry), and where this lane's come to lie: one sum over the warp for the batch.
    unsigned on = 0u;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned in = id[u] + k < end[u], other = id[u] + k != target, high = order_of(w[k]) >= least;
        on |= (in & other & high) << (4 * u + k);
      }
    }
    int before = __popc(on);
    const int mine = before;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += o;
    }
    const int more = __shfl_sync(0xffffffffu, before, 31);
    before -= mine;
    // (a batch may have more than there is room for, where many entries are equal: then a part at a time)
    for (int done = 0; done < more;) {
      if (n + more - done > kCandidates) n = compress(sh, n, held, lane);
      const int now = min(more - done, kCandidates - n);
      int place = before - done;
      for (unsigned rest = on; rest != 0u; rest &= rest - 1u, ++place) {  // few: their values are loaded again
        const int b = __ffs(rest) - 1;
        int unused;
        const int entry = first_of(sh.wanted[i0 + (b >> 2)], unused) + (b & 3);
        if (place >= 0 && place < now) sh.cand[n + place] = candidate(z[entry - p.v0], entry);
      }
      n += now;
      done += now;
      __syncwarp();
    }
  }
  if (n > kCandidates - kHeld - 1) n = compress(sh, n, held, lane);
  // the groups' peaks leave the target out: its logit goes in by itself
  if (target >= 0) {
    if (lane == 0) sh.cand[n] = candidate(z[target - p.v0], target);
    ++n;
  }
  if (!p.first)
    for (int i = lane; i - lane < held; i += 32) {
      const int id = i < held ? p.list_id[t * kHeld + i] : -1;
      const unsigned b = __ballot_sync(0xffffffffu, id >= 0);
      if (id >= 0) sh.cand[n + __popc(b & ((1u << lane) - 1u))] = candidate(p.list_z[t * kHeld + i], id);
      n += __popc(b);
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
  const Order o = {sh.sorted, sh.exact, keep, p.top};
  if (!p.last) {
    for (int i = lane; i < held; i += 32) {
      p.list_z[t * kHeld + i] = i < keep ? o.z(i) : 0.f;
      p.list_id[t * kHeld + i] = i < keep ? o.id(i) : -1;
    }
    return;
  }
  const uint64_t starts = o.starts(p, t, lane);
  o.exact_dots(p, t, starts, 0, 1, lane);
  __syncwarp();
  o.results(p, t, y, starts, sh.ids, sh.values, lane);
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
  top_of(p, t, lane, sh, wanted, p.groups > wanted ? least : 0u);
}

// ------------------------------------------------------------------ few tokens
// A block each: eight warps find the alternatives together, eight others join the groups' sums meanwhile. What a
// short launch like this takes are trips to memory and its instructions' way to the SM, so that the groups' number may
// be up to kMoreGroups above what is needed (a search for exactly the first `held` takes twice the rounds), their
// entries are loaded by all warps at once, and loops are not unrolled without need.
constexpr int kJoinThreads = 256;  // as where no alternatives are asked for: the same sums
constexpr int kFindThreads = 32 * kTopWarps;
constexpr int kMoreGroups = 24;
constexpr int kFewCandidates = (kHeld + kMoreGroups) * 32 + kHeld + 1;
constexpr int kRanked = 512;  // so many candidates are put in order by counting

struct FindShared {
  int red[2][kTopWarps];
  uint32_t low, high;
  int groups, candidates;
  int wanted[kHeld + kMoreGroups];
  uint64_t cand[kFewCandidates];
  uint64_t sorted[kHeld], exact[kHeld];
  uint64_t starts;
  int ids[kMaxAlternatives];
  float values[kMaxAlternatives];
};

__device__ __forceinline__ void find_sync() { asm volatile("bar.sync 2, 256;" ::: "memory"); }

// The sum over the finders; `turn` alternates between calls, so that one barrier is enough.
__device__ __forceinline__ int find_count(FindShared& sh, int n, int& turn) {
  n = __reduce_add_sync(0xffffffffu, n);
  int* red = sh.red[turn & 1];
  ++turn;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
  find_sync();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) all += red[w];
  return all;
}

// As threshold(), over the finders, and content with up to `more` above `want`.
template <typename T, class Count>
__device__ __forceinline__ T find_threshold(FindShared& sh, int want, int more, T low, T high, int& turn, Count&& count) {
  const T differ = low ^ high;
  if (differ == 0) return high;
  int bit = sizeof(T) == 8 ? 63 - __clzll(static_cast<long long>(differ)) : 31 - __clz(static_cast<int>(differ));
  T at = bit + 1 < static_cast<int>(sizeof(T)) * 8 ? high >> (bit + 1) << (bit + 1) : 0;
#pragma unroll 1
  for (; bit >= 0; --bit) {
    const T next = at | (T(1) << bit);
    const int n = find_count(sh, count(next), turn);
    if (n >= want) at = next;
    if (n >= want && n <= want + more) break;
  }
  return at;
}

// Where the groups' peaks are held: up to kInRegisters to a finder in its registers, up to kInShared in all in shared
// memory, else they are read again each time. (Read again, one token x 262144 x 256 took 13 us more, 128 tokens 17; from
// shared memory 48 us and 83. 36 and 53 are the log probabilities alone.)
enum Keys { kRead, kRegisters, kShared };
constexpr int kInRegisters = 8;
constexpr int kInShared = 40 * 1024;

template <Keys KEYS>
__device__ __forceinline__ void find(const TopParams& p, int64_t t, FindShared& sh, uint32_t* keys) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, held = p.top + kSpare;
  int turn = 0;
  const int64_t y = p.targets != nullptr ? p.targets[t] : -1;
  const int turns = KEYS == kRegisters ? kInRegisters : (p.groups + kFindThreads - 1) / kFindThreads;
  auto read = [&](int g) {
    return g < p.groups ? max(order_of(p.parts[t * p.token_step + g * p.group_step].peak), 1u) : 0u;
  };
  uint32_t key[KEYS == kRegisters ? kInRegisters : 1] = {};
  auto at = [&](int k) {
    const int g = k * kFindThreads + tid;
    return KEYS == kRegisters ? key[k] : KEYS == kRead ? read(g) : g < p.groups ? keys[g] : 0u;
  };
  if (tid == 0) {
    sh.low = 0xffffffffu;
    sh.high = 0u;
    sh.groups = sh.candidates = 0;
  }
  uint32_t low = 0xffffffffu, high = 0u;
#pragma unroll
  for (int k = 0; k < turns; ++k) {
    const uint32_t v = read(k * kFindThreads + tid);
    if (KEYS == kRegisters) key[k] = v;
    if (KEYS == kShared && v != 0u) keys[k * kFindThreads + tid] = v;  // (which this thread alone reads)
    if (v != 0u) low = min(low, v);
    high = max(high, v);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  find_sync();
  if (lane == 0) {
    atomicMin(&sh.low, low);
    atomicMax(&sh.high, high);
  }
  find_sync();
  uint32_t least = 1u;         // of the groups; logits below it are not among the largest
  uint32_t up_to = 0xffffffffu;  // of groups whose peak is `least`, those up to this one
  if (p.groups > held + kMoreGroups) {
    least = find_threshold<uint32_t>(sh, held, kMoreGroups, sh.low, sh.high, turn, [&](uint32_t limit) {
      int n = 0;
#pragma unroll
      for (int k = 0; k < turns; ++k) n += at(k) >= limit;
      return n;
    });
    int above = 0, level = 0;
#pragma unroll
    for (int k = 0; k < turns; ++k) {
      above += at(k) > least;
      level += at(k) == least;
    }
    above = find_count(sh, above, turn);
    level = find_count(sh, level, turn);
    if (above + level > held + kMoreGroups) {  // many share it: the first of them by number
      const uint32_t first = find_threshold<uint32_t>(sh, held - above, 0, 0u, 0xffffffffu, turn, [&](uint32_t limit) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < turns; ++k) n += at(k) == least && ~static_cast<uint32_t>(k * kFindThreads + tid) >= limit;
        return n;
      });
      up_to = ~first;
    }
  }
#pragma unroll
  for (int k = 0; k < turns; ++k) {
    const uint32_t v = at(k), g = k * kFindThreads + tid;
    if (v > least || (v == least && g <= up_to)) sh.wanted[atomicAdd(&sh.groups, 1)] = static_cast<int>(g);
  }
  find_sync();

  // ---------------------------------------------------------- their entries, the target, and the list so far
  const int wanted = sh.groups;
  if (p.groups <= wanted) least = 0u;
  const float* z = p.z + t * p.ld_z;
  auto add = [&](bool on, float v, int id) {
    const unsigned b = __ballot_sync(0xffffffffu, on);
    if (b == 0u) return;
    int n = 0;
    if (lane == 0) n = atomicAdd(&sh.candidates, __popc(b));
    n = __shfl_sync(0xffffffffu, n, 0);
    if (on)
      sh.cand[n + __popc(b & ((1u << lane) - 1u))] = candidate(v, id);
  };
#pragma unroll 4
  for (int i = warp; i < wanted; i += kTopWarps) {  // tile g / 8, half g / 4 % 2, 32 entries from g % 4 * 32
    const int g = sh.wanted[i];
    const int first = p.v0 + (g >> 3) * p.thin_h + ((g >> 2) & 1) * (p.thin_h / 2);
    const int id = first + (g & 3) * 32 + lane;
    const bool in = id < min(p.v0 + p.width, first + p.thin_h / 2) && id != y;
    const float v = in ? z[id - p.v0] : 0.f;
    add(in && order_of(v) >= least, v, id);
  }
  // the groups' peaks leave the target out: its logit goes in by itself
  if (warp == 0 && y >= p.v0 && y < p.v0 + p.width) add(lane == 0, z[y - p.v0], static_cast<int>(y));
  if (warp == 1 && !p.first)
    for (int i = lane; i - lane < held; i += 32) {
      const int id = i < held ? p.list_id[t * kHeld + i] : -1;
      add(id >= 0, id >= 0 ? p.list_z[t * kHeld + i] : 0.f, id);
    }
  find_sync();

  // ---------------------------------------------------------- the first of them, in order
  const int n = sh.candidates, keep = min(n, held);
  uint64_t reach = 0;
  if (n > kRanked)
    reach = find_threshold<uint64_t>(sh, keep, 0, uint64_t(0), ~uint64_t(0), turn, [&](uint64_t limit) {
      int c = 0;
      for (int i = tid; i < n; i += kFindThreads) c += sh.cand[i] >= limit;
      return c;
    });
  for (int i = tid; i < n; i += kFindThreads) {
    const uint64_t mine = sh.cand[i];
    if (mine < reach) continue;
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) place += sh.cand[j] > mine;
    if (place < keep) sh.sorted[place] = mine;
  }
  __syncthreads();  // and the joined sums are there
  const Order o = {sh.sorted, sh.exact, keep, p.top};
  if (warp == 0) {
    const uint64_t starts = o.starts(p, t, lane);
    if (lane == 0) sh.starts = starts;
  }
  find_sync();
  o.exact_dots(p, t, sh.starts, warp, kTopWarps, lane);
  find_sync();
  if (warp == 0) o.results(p, t, y, sh.starts, sh.ids, sh.values, lane);
}

template <Keys KEYS>
__global__ void __launch_bounds__(kFindThreads + kJoinThreads) score_top_kernel(const __grid_constant__ ScoreParams r,
                                                                                const __grid_constant__ TopParams p) {
  __shared__ FindShared sh;
  __shared__ ScoreShared<1, kJoinThreads> rows;
  extern __shared__ uint32_t keys[];
  follow();
  if (threadIdx.x >= kFindThreads) {
    score_rows<1, kJoinThreads>(r, blockIdx.x, threadIdx.x - kFindThreads, rows,
                                [] { asm volatile("bar.sync 1, 256;" ::: "memory"); });
    __syncthreads();
    return;
  }
  find<KEYS>(p, blockIdx.x, sh, keys);
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
  const int threads = kFindThreads + kJoinThreads;
  if (p.groups <= kInRegisters * kFindThreads)
    return launch_follow(score_top_kernel<kRegisters>, grid, threads, 0, s, 1, r, p);
  if (p.groups > kInShared) return launch_follow(score_top_kernel<kRead>, grid, threads, 0, s, 1, r, p);
  const cudaError_t e = cudaFuncSetAttribute(score_top_kernel<kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kInShared * static_cast<int>(sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  return launch_follow(score_top_kernel<kShared>, grid, threads, sizeof(uint32_t) * p.groups, s, 1, r, p);
}

}  // namespace head
}  // namespace dmuon
