// head_dot.cuh - logits formed in fp32 FMAs (see kSure in head.h), or with twice the digits.
#pragma once

#include <cmath>

#include "head.h"

namespace dmuon {
namespace head {

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(x[k]), g = __bfloat1622float2(y[k]);
    s = fmaf(f.x, g.x, s);
    s = fmaf(f.y, g.y, s);
  }
  return s;
}

// One thread's part (thread `at` of `of`) of N logits (t[n], v[n]), their loads in flight together: 8 elements
// at a time, the last few one by one.
template <int N>
__device__ __forceinline__ void dot_parts(const DotParams& d, const int64_t (&t)[N], const int64_t (&v)[N], int at,
                                          int of, float (&s)[N]) {
  const int whole = d.dim / 8;
#pragma unroll
  for (int n = 0; n < N; ++n) s[n] = 0.f;
#pragma unroll 2
  for (int c = at; c < whole; c += of) {
    uint4 a[N], b[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      a[n] = *reinterpret_cast<const uint4*>(d.hidden + t[n] * d.ld_hidden + 8 * c);
      b[n] = *reinterpret_cast<const uint4*>(d.weight + v[n] * d.ld_weight + 8 * c);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] = dot8(a[n], b[n], s[n]);
  }
  for (int k = 8 * whole + at; k < d.dim; k += of)
#pragma unroll
    for (int n = 0; n < N; ++n)
      s[n] = fmaf(__bfloat162float(d.hidden[t[n] * d.ld_hidden + k]),
                  __bfloat162float(d.weight[v[n] * d.ld_weight + k]), s[n]);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// A sum with twice fp32's digits (Knuth's two-sum: what each addition rounds away is added up beside it). In 64 bits the
// same takes longer: an SM adds two or so of those a cycle.
struct Twice {
  float sum, rest;
  __device__ __forceinline__ void add(float x) {
    const float s = sum + x, b = s - sum;
    rest += (sum - (s - b)) + (x - b);
    sum = s;
  }
  __device__ __forceinline__ void add(const Twice& o) {
    add(o.sum);
    rest += o.rest;
  }
  __device__ __forceinline__ double value() const {  // (of a sum that is infinite the rest is NaN)
    return static_cast<double>(sum) + (fabsf(rest) < INFINITY ? static_cast<double>(rest) : 0.0);
  }
};
__device__ __forceinline__ Twice warp_sum(Twice v) {
  for (int d = 16; d > 0; d >>= 1) {
    Twice o;
    o.sum = __shfl_xor_sync(0xffffffffu, v.sum, d);
    o.rest = __shfl_xor_sync(0xffffffffu, v.rest, d);
    v.add(o);
  }
  return v;
}

// One thread's part of a logit with twice fp32's digits: products of bf16 are exact in fp32, their sums are compensated.
// FLIGHT rounds of loads are in flight, as the trip to memory is what it takes. With SIZE, size gets the sum of the
// products' absolute values, too.
template <int FLIGHT, bool SIZE = false>
__device__ __forceinline__ Twice exact_part(const DotParams& d, int64_t t, int64_t v, int at, int of,
                                            float* size = nullptr) {
  Twice s = {0.f, 0.f};
  float all = 0.f;
  const bf16 *h = d.hidden + t * d.ld_hidden, *w = d.weight + v * d.ld_weight;
  auto add = [&](float product) {
    s.add(product);
    if (SIZE) all += fabsf(product);
  };
  const int whole = d.dim / 8;
  for (int c0 = at; c0 < whole; c0 += FLIGHT * of) {
    uint4 a[FLIGHT], b[FLIGHT];
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const bool in = c0 + of * u < whole;
      a[u] = in ? *reinterpret_cast<const uint4*>(h + 8 * (c0 + of * u)) : make_uint4(0, 0, 0, 0);
      b[u] = in ? *reinterpret_cast<const uint4*>(w + 8 * (c0 + of * u)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162*>(&a[u]),
                           *y = reinterpret_cast<const __nv_bfloat162*>(&b[u]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(x[k]), g = __bfloat1622float2(y[k]);
        add(f.x * g.x);
        add(f.y * g.y);
      }
    }
  }
  for (int k = 8 * whole + at; k < d.dim; k += of) add(__bfloat162float(h[k]) * __bfloat162float(w[k]));
  if (SIZE) *size = all;
  return s;
}

}  // namespace head
}  // namespace dmuon
