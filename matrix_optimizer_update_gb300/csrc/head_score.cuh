// head_score.cuh - a token's log probability, entropy and log sum from its groups' sums.
//
// Groups' sums are joined with the entropy's beside them: of sum = sum exp(z - peak) and
// folded = sum exp(z - peak) (z - peak), the entropy is log(sum) - folded / sum, both terms positive. The target's
// share comes apart from the others', so that a sure token's log probability and entropy keep their digits.
#pragma once

#include <cmath>

#include "head.h"
#include "head_dot.cuh"

namespace dmuon {
namespace head {

struct Folded {
  float peak = -INFINITY, sum = 0.f, fold = 0.f;
  // exp(-infinity) times a distance of -infinity is nothing
  static __device__ __forceinline__ float finite(float d) { return fmaxf(d, -1e4f); }
  __device__ __forceinline__ void join(float peak2, float sum2, float fold2) {
    const float m = fmaxf(peak, peak2);
    if (!(m > -INFINITY)) {  // neither has a number: zeros, or NaN to pass on
      sum += sum2;
      fold += fold2;
      return;
    }
    const float a = peak - m, b = peak2 - m, ea = expf(a), eb = expf(b);
    fold = ea * fmaf(sum, finite(a), fold) + eb * fmaf(sum2, finite(b), fold2);
    sum = sum * ea + sum2 * eb;
    peak = m;
  }
};

template <int kTokens, int kThreads>
struct ScoreShared {
  float peak[kThreads / 32][kTokens], sum[kThreads / 32][kTokens], fold[kThreads / 32][kTokens], dot[kThreads / 32];
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
        float s = 0.f, fold = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float d = q[u].peak - m, e = expf(d);
          s = fmaf(q[u].sum, e, s);
          fold = fmaf(fmaf(q[u].sum, Folded::finite(d), w[u]), e, fold);
        }
        f.join(m, s, fold);
      }
    }
    for (int d = 16; d >= kTokens; d >>= 1) {
      const float p2 = __shfl_xor_sync(0xffffffffu, f.peak, d), s2 = __shfl_xor_sync(0xffffffffu, f.sum, d),
                  f2 = __shfl_xor_sync(0xffffffffu, f.fold, d);
      f.join(p2, s2, f2);
    }
    if (lane < kTokens) {
      sh.peak[warp][lane] = f.peak;
      sh.sum[warp][lane] = f.sum;
      sh.fold[warp][lane] = f.fold;
    }
  }
  // from here a warp per token
  const int64_t t = t0 + (kTokens == 1 ? 0 : warp);
  float z = 0.f;
  int64_t y = -1;
  if (p.targets != nullptr && t < p.tokens) {
    y = p.targets[t];
    if (y >= p.vocab) y = -1;
    if (y >= 0) {
      float part[1];
      dot_parts<1>(p.dot, {t}, {y}, kTokens == 1 ? thread : lane, kTokens == 1 ? kThreads : 32, part);
      z = warp_sum(part[0]);
    }
  }
  if (lane == 0) sh.dot[warp] = z;
  sync();
  const int mine = kTokens == 1 ? 0 : warp;
  if (warp >= kTokens || t >= p.tokens || lane != 0) return;
  Folded f;
  for (int w = 0; w < kWarps; ++w) f.join(sh.peak[w][mine], sh.sum[w][mine], sh.fold[w][mine]);
  float lse, logp = 0.f, entropy;
  if (y < 0) {
    lse = f.peak + logf(f.sum);
    entropy = logf(f.sum) - f.fold / f.sum;
  } else {
    if (kTokens == 1)
      for (int w = 1; w < kWarps; ++w) z += sh.dot[w];
    z *= p.dot.scale;
    p.picked[t] = z;
    const float d = f.peak - z, e = expf(d), ratio = f.sum * e;  // the others' share to the target's
    if (ratio < 1.f) {
      logp = -log1pf(ratio);
      lse = z - logp;
      entropy = -logp - e * fmaf(f.sum, Folded::finite(d), f.fold) / (1.f + ratio);
    } else {
      const float hit = expf(-d), sum = f.sum + hit;
      lse = f.peak + logf(sum);
      logp = z - lse;
      entropy = logf(sum) - fmaf(hit, Folded::finite(-d), f.fold) / sum;
    }
  }
  p.lse[t] = lse;
  p.logp[t] = logp;
  p.entropy[t] = entropy < 0.f ? 0.f : entropy;  // off by a rounding where one entry has it all
}

}  // namespace head
}  // namespace dmuon
