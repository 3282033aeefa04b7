// head_rows.cu - the per-token work of the head's losses beside the products:
// the teacher's list sorted and turned into probabilities, and the groups'
// partial sums joined into the loss.
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "head.h"
#include "head_dot.cuh"
#include "head_score.cuh"

namespace dmuon {
namespace head {
namespace {

constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------------ teacher
// One block per token, a thread per entry. Each entry of the list finds its place in the order by id by counting the
// entries before it (no sorting network: with 128 entries 128 compares and one barrier against 28 barriers),
// then a softmax over the entries that count, and the logits of the likeliest ones, two at a time to a warp.
// Entries that do not count come last, with id vocab. Bound by latency: 4096 lists of 128 entries take 36 us
// (58 us with a sorting network), 16 lists of 8 take 7.5 us, most of it the launch and the first reads of W.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) teacher_kernel(const __grid_constant__ TeacherParams p) {
  __shared__ uint64_t key[kThreads];
  __shared__ int id[kThreads];
  __shared__ float lg[kThreads];
  __shared__ float red[3][kThreads / 32];
  follow();
  const int64_t t = blockIdx.x;
  const int k = threadIdx.x, lane = k & 31, warp = k >> 5;
  constexpr int warps = kThreads / 32;
  int my = p.vocab;
  float l = kNegInf;
  if (k < p.top) {
    const int64_t v = p.ids[t * p.top + k];
    const float x = p.logits[t * p.top + k];
    if (v >= 0 && v < p.vocab && x != kNegInf) {
      my = static_cast<int>(v);
      l = x;
    }
  }
  // by id, and entries of equal id by their logits' bits, so that the result does not depend on the order
  // they came in
  const uint64_t mine = (static_cast<uint64_t>(my) << 32) | __float_as_uint(l);
  key[k] = mine;
  __syncthreads();
  if (k < p.top) {
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < p.top; ++j) place += key[j] < mine || (key[j] == mine && j < k);
    id[place] = my;
    lg[place] = l;
  }
  __syncthreads();
  const bool on = k < p.top && id[k] < p.vocab;
  l = on ? lg[k] : kNegInf;
  auto block = [&](float v, int slot, bool max) {
    for (int d = 16; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, d);
      v = max ? fmaxf(v, o) : v + o;
    }
    if (lane == 0) red[slot][warp] = v;
    __syncthreads();
    v = red[slot][0];
    for (int w = 1; w < warps; ++w) v = max ? fmaxf(v, red[slot][w]) : v + red[slot][w];
    return v;
  };
  // a NaN logit makes its whole row NaN through the sum
  const float best = block(l, 0, true);
  const float e = on ? expf((l - best) * p.scale) : 0.f;
  const float sum = block(e, 1, false);
  const float q = on ? e / sum : 0.f;
  if (k < p.top) lg[k] = q;
  const float ent = block(q > 0.f ? q * logf(q) : q, 2, false);
  const int count = __syncthreads_count(on);
  if (k < p.top) {
    p.out_ids[t * p.top + k] = id[k];
    p.out_q[t * p.top + k] = q;
  }
  if (k == 0) {
    p.out_count[t] = count;
    p.out_entropy[t] = ent;
  }
  // lane j looks at entries j, j + 32, ...; warp w takes the pairs w, w + warps, ... of the likely ones
  int seen = 0;
  for (int e0 = 0; e0 < count; e0 += 32) {
    unsigned likely = __ballot_sync(0xffffffffu, e0 + lane < count && lg[e0 + lane] >= kSure);
    while (likely != 0u) {
      const int a = e0 + __ffs(likely) - 1;
      likely &= likely - 1u;
      const int b = likely != 0u ? e0 + __ffs(likely) - 1 : a;
      likely &= likely - 1u;
      if (seen++ % warps != warp) continue;
      float z[2];
      dot_parts<2>(p.dot, {t, t}, {id[a], id[b]}, lane, 32, z);
      z[0] = warp_sum(z[0]);
      z[1] = warp_sum(z[1]);
      if (lane == 0) {
        p.picked[t * p.top + a] = z[0] * p.dot.scale;
        p.picked[t * p.top + b] = z[1] * p.dot.scale;
      }
    }
  }
}

// ------------------------------------------------------------------ rows
// The sum over the vocabulary is kept in two shares, of the wanted entries and of all others, so that a loss
// that is small beside the logits is formed from their ratio (log1p) and not as a difference.
//
// A block takes kTokens tokens: 8 where the groups' sums lie token by token (8 threads read a 64-byte piece
// of each group), 1 where the tokens are few and each has its groups' sums in a row. Four sums are joined at
// a time, so that their loads are in flight together. 4096 tokens x 1000 groups: 19 us (42 us with a token to a
// block and a sum at a time); 77 tokens: 6 us, a launch and three dependent reads.
constexpr int kRowThreads = 256;

__device__ __forceinline__ void join(float& peak, float& sum, float peak2, float sum2) {
  const float m = fmaxf(peak, peak2);
  if (!(m > kNegInf)) {  // neither has a number: zeros, or NaN to pass on
    sum += sum2;
    return;
  }
  sum = sum * expf(peak - m) + sum2 * expf(peak2 - m);
  peak = m;
}

template <int kTokens>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowParams p) {
  constexpr int kLanes = kRowThreads / kTokens;  // threads that share a token's groups
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float s_peak[kWarps][kTokens], s_sum[kWarps][kTokens], s_dot[kWarps];
  follow();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  {
    const int64_t t = int64_t(blockIdx.x) * kTokens + threadIdx.x % kTokens;
    float peak = kNegInf, sum = 0.f;
    if (t < p.tokens) {
      const Part* parts = p.parts + t * p.token_step;
      for (int g = threadIdx.x / kTokens; g < p.groups; g += 4 * kLanes) {
        Part q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          q[u] = g + u * kLanes < p.groups ? parts[(g + u * kLanes) * p.group_step] : Part{kNegInf, 0.f};
        const float m = fmaxf(fmaxf(q[0].peak, q[1].peak), fmaxf(q[2].peak, q[3].peak));
        if (!(m > kNegInf)) {  // (a group of nothing but NaN may have NaN for its peak)
          sum += q[0].sum + q[1].sum + q[2].sum + q[3].sum;
          continue;
        }
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) s += q[u].sum * expf(q[u].peak - m);
        join(peak, sum, m, s);
      }
    }
    for (int d = 16; d >= kTokens; d >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, peak, d), s2 = __shfl_xor_sync(0xffffffffu, sum, d);
      join(peak, sum, m2, s2);
    }
    if (lane < kTokens) {
      s_peak[warp][lane] = peak;
      s_sum[warp][lane] = sum;
    }
  }
  // from here a warp per token
  const int64_t t = int64_t(blockIdx.x) * kTokens + (kTokens == 1 ? 0 : warp);
  const bool xent = p.want.targets != nullptr;
  float z = 0.f;
  int64_t y = -1;
  if (xent && t < p.tokens) {
    y = p.want.targets[t];
    if (y >= p.vocab) y = -1;
    if (y >= 0) {
      float part[1];
      dot_parts<1>(p.dot, {t}, {y}, kTokens == 1 ? threadIdx.x : lane, kTokens == 1 ? kRowThreads : 32, part);
      z = warp_sum(part[0]);
    }
  }
  if (lane == 0) s_dot[warp] = z;
  __syncthreads();
  const int mine = kTokens == 1 ? 0 : warp;
  if (warp >= kTokens || t >= p.tokens) return;
  float peak = s_peak[0][mine], sum = s_sum[0][mine];
  for (int w = 1; w < kWarps; ++w) join(peak, sum, s_peak[w][mine], s_sum[w][mine]);
  // peak, sum: the others. Now the wanted entries.
  float hit_peak = kNegInf, hit = 0.f, dot = 0.f;
  int n;
  if (xent) {
    n = y >= 0;
    if (kTokens == 1)
      for (int w = 1; w < kWarps; ++w) z += s_dot[w];
    hit_peak = z * p.dot.scale;
    hit = 1.f;
  } else {
    n = p.want.count[t];
    const float* zs = p.picked + t * p.want.top;
    const int32_t* id = p.want.ids + t * p.want.top;
    const float* q = p.want.q + t * p.want.top;
    // entries that share an id: the first of them has the logit, and counts once
    auto first_of = [&](int k) {
      while (k > 0 && id[k - 1] == id[k]) --k;
      return k;
    };
    for (int k = lane; k < n; k += 32) hit_peak = fmaxf(hit_peak, zs[first_of(k)]);
    for (int d = 16; d > 0; d >>= 1) hit_peak = fmaxf(hit_peak, __shfl_xor_sync(0xffffffffu, hit_peak, d));
    for (int k = lane; k < n; k += 32) {
      const int f = first_of(k);
      const float above = zs[f] - hit_peak;
      if (f == k) hit += expf(above);
      dot = fmaf(q[k], above, dot);
    }
    hit = warp_sum(hit);
    dot = warp_sum(dot);
  }
  if (lane != 0) return;
  if (n == 0) {
    p.lse[t] = peak + logf(sum);
    p.loss[t] = 0.f;
    return;
  }
  const float lse_hit = hit_peak + logf(hit);
  const float ratio = sum * expf(peak - hit_peak) / hit;
  float lse, rest;  // rest = lse - lse_hit
  if (ratio < 1.f) {
    rest = log1pf(ratio);
    lse = lse_hit + rest;
  } else {
    lse = peak + logf(sum + hit * expf(hit_peak - peak));
    rest = lse - lse_hit;
  }
  p.lse[t] = lse;
  if (xent) {
    p.loss[t] = rest;
  } else {
    // sum_k q log q - q (z - hit_peak) + log(hit): the divergence within the list; rest: of the list's share
    const float within = p.entropy[t] - dot + logf(hit);
    p.loss[t] = (within + rest) * p.temperature * p.temperature;
  }
}

// ------------------------------------------------------------------ scores
template <int kTokens>
__global__ void __launch_bounds__(kRowThreads) score_rows_kernel(const __grid_constant__ ScoreParams p) {
  __shared__ ScoreShared<kTokens, kRowThreads> sh;
  follow();
  score_rows<kTokens, kRowThreads>(p, int64_t(blockIdx.x) * kTokens, threadIdx.x, sh, [] { __syncthreads(); });
}

// The slices of dH's sums joined in order, scaled and rounded: 4 elements per thread and step. Bound by reading
// the sums: 4096 x 2048, one slice, 12.3 us (4.1 TB/s).
__global__ void __launch_bounds__(256) round_kernel(const float* acc, int slices, int64_t tokens, int32_t dim,
                                                    int64_t pitch, float gscale, const float* gmax, bf16* out,
                                                    int64_t ld) {
  follow();
  const float scale = gscale * *gmax;
  const int64_t n = tokens * (pitch / 4), slice = tokens * pitch;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = i / (pitch / 4);
    const int d = static_cast<int>(i - t * (pitch / 4)) * 4;
    const float* a = acc + t * pitch + d;
    float4 v = *reinterpret_cast<const float4*>(a);
    for (int s = 1; s < slices; ++s) {
      const float4 o = *reinterpret_cast<const float4*>(a + s * slice);
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    bf16* q = out + t * ld + d;
    if (d + 4 <= dim) {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x * scale, v.y * scale),
                             __floats2bfloat162_rn(v.z * scale, v.w * scale)};
      *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(h);
    } else {
      const float x[4] = {v.x, v.y, v.z, v.w};
      for (int k = 0; d + k < dim; ++k) q[k] = __float2bfloat16_rn(x[k] * scale);
    }
  }
}

}  // namespace

cudaError_t launch_teacher(const TeacherParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.tokens));
  if (p.top <= 128) return launch_follow(teacher_kernel<128>, grid, 128, 0, s, 1, p);
  static_assert(kMaxTop <= 256, "a thread per entry");
  return launch_follow(teacher_kernel<256>, grid, 256, 0, s, 1, p);
}

cudaError_t launch_rows(const RowParams& p, cudaStream_t s) {
  if (p.group_step == 1)
    return launch_follow(rows_kernel<1>, dim3(static_cast<unsigned>(p.tokens)), kRowThreads, 0, s, 1, p);
  return launch_follow(rows_kernel<8>, dim3(static_cast<unsigned>((p.tokens + 7) / 8)), kRowThreads, 0, s, 1, p);
}

cudaError_t launch_score_rows(const ScoreParams& p, cudaStream_t s) {
  if (p.group_step == 1)
    return launch_follow(score_rows_kernel<1>, dim3(static_cast<unsigned>(p.tokens)), kRowThreads, 0, s, 1, p);
  return launch_follow(score_rows_kernel<8>, dim3(static_cast<unsigned>((p.tokens + 7) / 8)), kRowThreads, 0, s, 1, p);
}

cudaError_t launch_round(const float* acc, int slices, int64_t tokens, int32_t dim, float gscale, const float* gmax,
                         bf16* out, int64_t ld_out, cudaStream_t s) {
  const int64_t pitch = acc_pitch(dim), n = tokens * (pitch / 4);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 152 * 8));
  return launch_follow(round_kernel, dim3(blocks), 256, 0, s, 1, acc, slices, tokens, dim, pitch, gscale, gmax, out,
                       ld_out);
}

}  // namespace head
}  // namespace dmuon
