// head_simple.cu - the products of the head's losses on the fp32 units: 64 x 128
// output tiles, 256 threads with 4 x 8 outputs each, K 16 at a time. The plain
// form of each kernel; every size and pitch goes element by element.
#include <cmath>

#include "head.h"

namespace dmuon {
namespace head {
namespace {

constexpr int kM = 64, kN = 128, kK = 16;
constexpr int kThreads = 256;

struct Tile {
  float a[kK][kM + 4];
  float b[kK][kN + 4];
  float c[kM][kN + 1];
};

// C[m][n] = sum_k A[m][k] B[n][k] for one tile; A and B bf16 with any strides, rows past m_lim / n_lim read as 0.
__device__ void product(Tile& s, const bf16* A, int64_t sam, int64_t sak, int64_t m0, int64_t m_lim, const bf16* B,
                        int64_t sbn, int64_t sbk, int64_t n0, int64_t n_lim, int64_t kdim) {
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  float acc[4][8] = {};
  for (int64_t k0 = 0; k0 < kdim; k0 += kK) {
    for (int e = tid; e < kM * kK; e += kThreads) {
      // neighbouring threads read neighbouring elements of the contiguous direction
      const int k = sak == 1 ? e % kK : e / kM, m = sak == 1 ? e / kK : e % kM;
      const bool in = m0 + m < m_lim && k0 + k < kdim;
      s.a[k][m] = in ? __bfloat162float(A[(m0 + m) * sam + (k0 + k) * sak]) : 0.f;
    }
    for (int e = tid; e < kN * kK; e += kThreads) {
      const int k = sbk == 1 ? e % kK : e / kN, n = sbk == 1 ? e / kK : e % kN;
      const bool in = n0 + n < n_lim && k0 + k < kdim;
      s.b[k][n] = in ? __bfloat162float(B[(n0 + n) * sbn + (k0 + k) * sbk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      float a[4], b[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = s.a[k][tr * 4 + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = s.b[k][tc + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s.c[tr * 4 + i][tc + 16 * j] = acc[i][j];
  __syncthreads();
}

// BACKWARD false: the group's share of the softmax sum and the wanted logits. true: dz.
template <bool BACKWARD>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitParams p) {
  extern __shared__ float4 raw[];
  Tile& s = *reinterpret_cast<Tile*>(raw);
  const int64_t m0 = int64_t(blockIdx.y) * kM;
  const int64_t n0 = (BACKWARD ? p.v0 : 0) + int64_t(blockIdx.x) * kN;
  const int64_t n_end = BACKWARD ? p.v0 + p.width : p.vocab;
  product(s, p.hidden, p.ld_hidden, 1, m0, p.tokens, p.weight, p.ld_weight, 1, n0, n_end, p.dim);
  const int r = threadIdx.x;
  const int64_t t = m0 + r;
  if (r >= kM || t >= p.tokens) return;
  const int cols = static_cast<int>(min(int64_t(kN), n_end - n0));
  for (int j = 0; j < cols; ++j) s.c[r][j] *= p.scale;
  const Wanted& w = p.want;
  if (!BACKWARD) {
    if (w.targets != nullptr) {
      const int64_t y = w.targets[t];
      if (y >= n0 && y < n0 + cols) {
        p.picked[t] = s.c[r][y - n0];
        s.c[r][y - n0] = -INFINITY;
      }
    } else {
      const int n = w.count[t];
      for (int k = 0; k < n; ++k) {
        const int v = w.ids[t * w.top + k];
        if (v >= n0 && v < n0 + cols) p.picked[t * w.top + k] = s.c[r][v - n0];
      }
      for (int k = 0; k < n; ++k) {
        const int v = w.ids[t * w.top + k];
        if (v >= n0 && v < n0 + cols) s.c[r][v - n0] = -INFINITY;
      }
    }
    Part part = {-INFINITY, 0.f};
    for (int j = 0; j < cols; ++j) part.peak = fmaxf(part.peak, s.c[r][j]);
    if (part.peak != -INFINITY)
      for (int j = 0; j < cols; ++j) part.sum += expf(s.c[r][j] - part.peak);
    p.parts[int64_t(blockIdx.x) * p.tokens + t] = part;
  } else {
    const float lse = p.lse[t];
    float g = p.grad[t];
    if (w.targets != nullptr) {
      const int64_t y = w.targets[t];
      if (y < 0 || y >= w.vocab) g = 0.f;
      for (int j = 0; j < cols; ++j) {
        float d = expf(s.c[r][j] - lse);
        if (n0 + j == y) d -= 1.f;
        s.c[r][j] = g == 0.f ? 0.f : g * d;
      }
    } else {
      const int n = w.count[t];
      g = n == 0 ? 0.f : g / p.scale;
      for (int j = 0; j < cols; ++j) s.c[r][j] = expf(s.c[r][j] - lse);
      for (int k = 0; k < n; ++k) {
        const int v = w.ids[t * w.top + k];
        if (v >= n0 && v < n0 + cols) s.c[r][v - n0] -= w.q[t * w.top + k];
      }
      for (int j = 0; j < cols; ++j) s.c[r][j] = g == 0.f ? 0.f : g * s.c[r][j];
    }
    for (int j = 0; j < cols; ++j) p.dz[t * p.ld_dz + (n0 - p.v0) + j] = __float2bfloat16_rn(s.c[r][j]);
  }
}

__global__ void __launch_bounds__(kThreads) dhidden_kernel(const __grid_constant__ GradParams p) {
  extern __shared__ float4 raw[];
  Tile& s = *reinterpret_cast<Tile*>(raw);
  const int64_t m0 = int64_t(blockIdx.y) * kM, n0 = int64_t(blockIdx.x) * kN;
  product(s, p.dz, p.ld_dz, 1, m0, p.tokens, p.weight + p.v0 * p.ld_weight, 1, p.ld_weight, n0, p.dim, p.width);
  for (int e = threadIdx.x; e < kM * kN; e += kThreads) {
    const int64_t t = m0 + e / kN, d = n0 + e % kN;
    if (t >= p.tokens || d >= p.dim) continue;
    float* o = p.dh_acc + t * p.dim + d;
    *o = s.c[e / kN][e % kN] + (p.first ? 0.f : *o);
  }
}

__global__ void __launch_bounds__(kThreads) dweight_kernel(const __grid_constant__ GradParams p) {
  extern __shared__ float4 raw[];
  Tile& s = *reinterpret_cast<Tile*>(raw);
  const int64_t m0 = int64_t(blockIdx.y) * kM, n0 = int64_t(blockIdx.x) * kN;
  product(s, p.dz, 1, p.ld_dz, m0, p.width, p.hidden, 1, p.ld_hidden, n0, p.dim, p.tokens);
  for (int e = threadIdx.x; e < kM * kN; e += kThreads) {
    const int64_t v = m0 + e / kN, d = n0 + e % kN;
    if (v < p.width && d < p.dim)
      p.dweight[(p.v0 + v) * p.ld_dweight + d] = __float2bfloat16_rn(s.c[e / kN][e % kN]);
  }
}

template <typename K, typename P>
cudaError_t launch(K kernel, const P& p, int64_t m, int64_t n, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Tile));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((n + kN - 1) / kN), static_cast<unsigned>((m + kM - 1) / kM));
  kernel<<<grid, kThreads, sizeof(Tile), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits(const LogitParams& p, cudaStream_t s) {
  return launch(logits_kernel<false>, p, p.tokens, p.vocab, s);
}
cudaError_t launch_dz(const LogitParams& p, cudaStream_t s) {
  return launch(logits_kernel<true>, p, p.tokens, p.width, s);
}
cudaError_t launch_grads(const GradParams& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.dh_acc != nullptr) e = launch(dhidden_kernel, p, p.tokens, p.dim, s);
  if (e == cudaSuccess && p.dweight != nullptr) e = launch(dweight_kernel, p, p.width, p.dim, s);
  return e;
}

}  // namespace head
}  // namespace dmuon
