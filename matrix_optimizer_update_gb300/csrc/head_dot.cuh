// head_dot.cuh - logits formed in fp32 FMAs (see kSure in head.h).
#pragma once

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

}  // namespace head
}  // namespace dmuon
