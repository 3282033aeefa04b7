// head_rows.cu - the per-token work of the head's losses beside the products:
// the teacher's list sorted and turned into probabilities, and the groups'
// partial sums joined into the loss.
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "head.h"

namespace dmuon {
namespace head {
namespace {

constexpr float kNegInf = -INFINITY;

// One thread's part (thread `at` of `of`) of the logit of (t, v): 8 elements at a time, the last few one by one.
__device__ __forceinline__ float dot_part(const DotParams& d, int64_t t, int64_t v, int at, int of) {
  const bf16* h = d.hidden + t * d.ld_hidden;
  const bf16* w = d.weight + v * d.ld_weight;
  const int whole = d.dim / 8;
  float s = 0.f;
  for (int c = at; c < whole; c += of) {
    const uint4 a = *reinterpret_cast<const uint4*>(h + 8 * c), b = *reinterpret_cast<const uint4*>(w + 8 * c);
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&a);
    const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(x[k]), g = __bfloat1622float2(y[k]);
      s = fmaf(f.x, g.x, s);
      s = fmaf(f.y, g.y, s);
    }
  }
  for (int k = 8 * whole + at; k < d.dim; k += of) s = fmaf(__bfloat162float(h[k]), __bfloat162float(w[k]), s);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// One warp per token.
__global__ void __launch_bounds__(256) targets_kernel(const __grid_constant__ DotParams d, const int64_t* targets,
                                                      int64_t tokens, int32_t vocab, float* picked) {
  follow();
  const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const int64_t y = targets[t];
  if (y < 0 || y >= vocab) return;
  const float z = warp_sum(dot_part(d, t, y, threadIdx.x & 31, 32)) * d.scale;
  if ((threadIdx.x & 31) == 0) picked[t] = z;
}

// ------------------------------------------------------------------ teacher
// One block per token, one thread per entry of a list padded to a power of two
// (at most 256): a bitonic sort by id in shared memory, then the softmax over
// the entries that count. Entries that do not count sort last, with id vocab.
__global__ void teacher_kernel(const __grid_constant__ TeacherParams p) {
  extern __shared__ unsigned char raw[];
  const int n = blockDim.x;
  int* id = reinterpret_cast<int*>(raw);
  float* lg = reinterpret_cast<float*>(id + n);
  __shared__ float red[8];
  follow();
  const int64_t t = blockIdx.x;
  const int k = threadIdx.x;
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
  id[k] = my;
  lg[k] = l;
  __syncthreads();
  for (int size = 2; size <= n; size <<= 1) {
    for (int d = size >> 1; d > 0; d >>= 1) {
      const int o = k ^ d;
      if (o > k) {
        const bool up = (k & size) == 0;
        const int a = id[k], b = id[o];
        // entries of equal id keep an order of their own (by logit), so that the result does not
        // depend on the order they came in
        const bool swap = up ? (a > b || (a == b && lg[k] > lg[o])) : (a < b || (a == b && lg[k] < lg[o]));
        if (swap) {
          id[k] = b;
          id[o] = a;
          const float x = lg[k];
          lg[k] = lg[o];
          lg[o] = x;
        }
      }
      __syncthreads();
    }
  }
  const int lane = k & 31, warp = k >> 5, warps = (n + 31) >> 5;
  auto reduce = [&](float v, bool max) {
    for (int d = 16; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, d);
      v = max ? fmaxf(v, o) : v + o;
    }
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < warps; ++w) v = max ? fmaxf(v, red[w]) : v + red[w];
    __syncthreads();
    return v;
  };
  const bool on = id[k] < p.vocab;
  l = lg[k];
  // a NaN logit makes its whole row NaN through the sum
  const float best = reduce(on ? l : kNegInf, true);
  const float e = on ? expf((l - best) * p.scale) : 0.f;
  const float sum = reduce(e, false);
  const float q = on ? e / sum : 0.f;
  const float ent = reduce(q > 0.f ? q * logf(q) : q, false);
  const float count = reduce(on ? 1.f : 0.f, false);
  if (k < p.top) {
    p.out_ids[t * p.top + k] = id[k];
    p.out_q[t * p.top + k] = q;
  }
  if (k == 0) {
    p.out_count[t] = static_cast<int>(count);
    p.out_entropy[t] = ent;
  }
  // the logits of the likeliest entries, a warp for each
  lg[k] = q;
  __syncthreads();
  int seen = 0;
  for (int e = 0; e < static_cast<int>(count); ++e) {
    if (!(lg[e] >= kSure)) continue;
    if (seen++ % warps != warp) continue;
    const float z = warp_sum(dot_part(p.dot, t, id[e], lane, 32)) * p.dot.scale;
    if (lane == 0) p.picked[t * p.top + e] = z;
  }
}

// ------------------------------------------------------------------ rows
// One block per token. The sum over the vocabulary is kept in two shares, of
// the wanted entries and of all others, so that a loss that is small beside
// the logits is formed from their ratio (log1p) and not as a difference.
constexpr int kRowThreads = 128;

__device__ __forceinline__ void join(float& peak, float& sum, float peak2, float sum2) {
  const float m = fmaxf(peak, peak2);
  if (m == kNegInf) return;  // neither has anything
  sum = sum * expf(peak - m) + sum2 * expf(peak2 - m);
  peak = m;
}

__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowParams p) {
  __shared__ float s_peak[kRowThreads / 32], s_sum[kRowThreads / 32], s_dot[kRowThreads / 32];
  follow();
  const int64_t t = blockIdx.x;
  float peak = kNegInf, sum = 0.f;
  for (int g = threadIdx.x; g < p.groups; g += kRowThreads) {
    const Part q = p.parts[int64_t(g) * p.tokens + t];
    join(peak, sum, q.peak, q.sum);
  }
  for (int d = 16; d > 0; d >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, peak, d), s2 = __shfl_xor_sync(0xffffffffu, sum, d);
    join(peak, sum, m2, s2);
  }
  if ((threadIdx.x & 31) == 0) {
    s_peak[threadIdx.x >> 5] = peak;
    s_sum[threadIdx.x >> 5] = sum;
  }
  float z = 0.f;
  int64_t y = -1;
  if (p.want.targets != nullptr) {
    y = p.want.targets[t];
    if (y >= p.vocab) y = -1;
    if (y >= 0) z = warp_sum(dot_part(p.dot, t, y, threadIdx.x, kRowThreads));
    if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5] = z;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  for (int w = 1; w < kRowThreads / 32; ++w) join(peak, sum, s_peak[w], s_sum[w]);
  // peak, sum: the others (warp 0 has them in every lane). Now the wanted entries.
  float hit_peak = kNegInf, hit = 0.f, dot = 0.f;
  int n;
  if (p.want.targets != nullptr) {
    n = y >= 0;
    z = s_dot[0];
    for (int w = 1; w < kRowThreads / 32; ++w) z += s_dot[w];
    hit_peak = z * p.dot.scale;
    hit = 1.f;
  } else {
    n = p.want.count[t];
    const float* zs = p.picked + t * p.want.top;
    const int32_t* id = p.want.ids + t * p.want.top;
    const float* q = p.want.q + t * p.want.top;
    const int lane = threadIdx.x;
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
  if (threadIdx.x != 0) return;
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
  if (p.want.targets != nullptr) {
    p.loss[t] = rest;
  } else {
    // sum_k q log q - q (z - hit_peak) + log(hit): the divergence within the list; rest: of the list's share
    const float within = p.entropy[t] - dot + logf(hit);
    p.loss[t] = (within + rest) * p.temperature * p.temperature;
  }
}

// The slices of dH's sums joined in order, scaled and rounded: 4 elements per thread and step.
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
  int n = 32;
  while (n < p.top) n <<= 1;
  return launch_follow(teacher_kernel, dim3(static_cast<unsigned>(p.tokens)), n, 8 * n, s, 1, p);
}

cudaError_t launch_targets(const DotParams& d, const int64_t* targets, int64_t tokens, int32_t vocab, float* picked,
                           cudaStream_t s) {
  return launch_follow(targets_kernel, dim3(static_cast<unsigned>((tokens + 7) / 8)), 256, 0, s, 1, d, targets, tokens,
                       vocab, picked);
}

cudaError_t launch_rows(const RowParams& p, cudaStream_t s) {
  return launch_follow(rows_kernel, dim3(static_cast<unsigned>(p.tokens)), kRowThreads, 0, s, 1, p);
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
