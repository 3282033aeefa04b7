// head_score.cuh - a token's log probability, entropy and log sum from its groups' sums.
//
// Groups' sums are joined with the entropy's beside them: of sum = sum exp(z - peak) and
// folded = sum exp(z - peak) (z - peak), the entropy is log(sum) - folded / sum, both terms positive. The peak's own 1 is
// left out of sum throughout (rest = sum - 1, and log(sum) is log1p(rest)): where one entry is nearly sure, all digits of
// the entropy are the others'. (With it inside, one entry 18 above 499 others was off by 2e-4.) The target's
// share comes apart from the others', so that a sure token's log probability and entropy keep their digits: of those,
// the relative error is the absolute one of the target's logit less the others' peak, which in fp32 is 1e-6 at 16 to
// 32. So that logit has twice the digits, and of the distance a second part is kept. (24 single tokens x 123366 x 1120
// were off by up to 2.1e-6 with the logit in fp32, by up to 3.1e-7 so; one token x 32000 x 2048 takes 34.9 us for 33.6.)
#pragma once

#include <cmath>

#include "head.h"
#include "head_dot.cuh"

namespace dmuon {
namespace head {

struct Folded {
  float peak = -INFINITY, rest = 0.f, fold = 0.f;  // (without a peak rest is 0, or NaN to pass on)
  // exp(-infinity) times a distance of -infinity is nothing
  static __device__ __forceinline__ float finite(float d) { return fmaxf(d, -1e4f); }
  __device__ __forceinline__ void join(float peak2, float rest2, float fold2) {
    const float m = fmaxf(peak, peak2);
    if (!(m > -INFINITY)) {  // neither has a number
      rest += rest2;
      fold += fold2;
      return;
    }
    const float a = peak - m, b = peak2 - m, ea = expf(a), eb = expf(b), all = 1.f + rest, all2 = 1.f + rest2;
    fold = ea * fmaf(all, finite(a), fold) + eb * fmaf(all2, finite(b), fold2);
    if (a == 0.f) rest = rest + (b == 0.f ? all2 : all2 * eb);
    else rest = rest2 + all * ea;
    peak = m;
  }
};

// What a second part is where the first is infinite.
__device__ __forceinline__ float finite(float x) { return fabsf(x) < INFINITY ? x : 0.f; }

template <int kTokens, int kThreads>
struct ScoreShared {
  float peak[kThreads / 32][kTokens], rest[kThreads / 32][kTokens], fold[kThreads / 32][kTokens];
  Twice dot[kThreads / 32];
  float size[kThreads / 32];
};

// kTokens tokens from t0 on (1 or 8) by kThreads threads, `thread` among them; `sync` is their barrier.
template <int kTokens, int kThreads, class Sync>
__device__ __forceinline__ void score_rows(const ScoreParams& p, int64_t t0, int thread, ScoreShared<kTokens, kThreads>& sh,
                                           Sync&& sync) {
  constexpr int kLanes = kThreads / kTokens;
  constexpr int kWarps = kThreads / 32;
  static_assert(kTokens == 1 || kTokens == kWarps, "a warp per token, or all of them");
  const int lane = thread & 31, warp = thread >> 5;
  {
    const int64_t t = t0 + thread % kTokens;
    Folded f;
    if (t < p.tokens) {
      const int64_t at = t * p.token_step;
      for (int g = thread / kTokens; g < p.groups; g += 4 * kLanes) {
        Part q[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t i = at + (g + u * kLanes) * p.group_step;
          const bool in = g + u * kLanes < p.groups;
          q[u] = in ? p.parts[i] : Part{-INFINITY, 0.f};
          w[u] = in ? p.folds[i] : 0.f;
        }
        const float m = fmaxf(fmaxf(q[0].peak, q[1].peak), fmaxf(q[2].peak, q[3].peak));
        if (!(m > -INFINITY)) {
          f.join(-INFINITY, q[0].sum + q[1].sum + q[2].sum + q[3].sum, w[0] + w[1] + w[2] + w[3]);
          continue;
        }
        float rest = 0.f, fold = 0.f;
        int ones = -1;  // one is the peak's own
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float d = q[u].peak - m, e = expf(d), all = 1.f + q[u].sum;
          if (d == 0.f) ++ones, rest += q[u].sum;
          else rest = fmaf(all, e, rest);
          fold = fmaf(fmaf(all, Folded::finite(d), w[u]), e, fold);
        }
        f.join(m, rest + static_cast<float>(ones), fold);
      }
    }
    for (int d = 16; d >= kTokens; d >>= 1) {
      const float p2 = __shfl_xor_sync(0xffffffffu, f.peak, d), s2 = __shfl_xor_sync(0xffffffffu, f.rest, d),
                  f2 = __shfl_xor_sync(0xffffffffu, f.fold, d);
      f.join(p2, s2, f2);
    }
    if (lane < kTokens) {
      sh.peak[warp][lane] = f.peak;
      sh.rest[warp][lane] = f.rest;
      sh.fold[warp][lane] = f.fold;
    }
  }
  // from here a warp per token
  const int64_t t = t0 + (kTokens == 1 ? 0 : warp);
  Twice dot = {0.f, 0.f};
  float size = 0.f;  // the sum of the products' absolute values
  int64_t y = -1;
  if (t < p.tokens) {
    if (p.targets != nullptr) {
      y = p.targets[t];
      if (y >= p.vocab) y = -1;
    }
    // where sizes are asked for, a token without a target has those of some entry
    const int64_t v = y >= 0 || p.sizes == nullptr ? y : t % p.vocab;
    // (two rounds are all of 4096 dims for a block, and less code to fetch for one token: 0.4 us)
    if (v >= 0) {
      dot = warp_sum(kTokens == 1 ? exact_part<2, true>(p.dot, t, v, thread, kThreads, &size)
                                  : exact_part<4, true>(p.dot, t, v, lane, 32, &size));
      size = warp_sum(size);
    }
  }
  if (lane == 0) {
    sh.dot[warp] = dot;
    sh.size[warp] = size;
  }
  sync();
  const int mine = kTokens == 1 ? 0 : warp;
  if (warp >= kTokens || t >= p.tokens || lane != 0) return;
  Folded f;
  for (int w = 0; w < kWarps; ++w) f.join(sh.peak[w][mine], sh.rest[w][mine], sh.fold[w][mine]);
  float lse, logp = 0.f, entropy;
  if (y < 0) {
    const float log_sum = log1pf(f.rest);
    lse = f.peak + log_sum;
    entropy = f.peak > -INFINITY ? log_sum - f.fold / (1.f + f.rest) : NAN;
  } else {
    if (kTokens == 1)
      for (int w = 1; w < kWarps; ++w) dot.add(sh.dot[w]);
    // the scaled logit z + rest, and its distance d + low from the others' peak
    const float sum = dot.sum + finite(dot.rest), z = sum * p.scale,
                rest = finite(fmaf(sum, p.scale, -z) + fmaf(sum, p.scale_low, finite(dot.rest - (sum - dot.sum)) * p.scale));
    Twice distance = {f.peak, 0.f};
    distance.add(-z);
    const float d = distance.sum, low = finite(distance.rest - rest);
    const float e = expf(d) * (1.f + low), others = 1.f + f.rest, ratio = others * e;  // their share to the target's
    if (ratio < 1.f) {
      logp = -log1pf(ratio);
      lse = z + (rest - logp);
      entropy = -logp - e * fmaf(others, Folded::finite(d), f.fold) / (1.f + ratio);
    } else {
      const float hit = expf(-d) * (1.f - low), rest = f.rest + hit, log_sum = log1pf(rest);
      lse = f.peak + log_sum;
      logp = -(d + (low + log_sum));
      entropy = log_sum - fmaf(hit, Folded::finite(-d), f.fold) / (1.f + rest);
    }
  }
  if (p.sizes != nullptr) {
    if (kTokens == 1)
      for (int w = 1; w < kWarps; ++w) size += sh.size[w];
    p.sizes[t] = size * p.scale;
  }
  p.lse[t] = lse;
  p.logp[t] = logp;
  p.entropy[t] = entropy < 0.f ? 0.f : entropy;  // off by a rounding where one entry has it all
}

}  // namespace head
}  // namespace dmuon
