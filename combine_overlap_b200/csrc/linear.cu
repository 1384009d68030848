// linear.cu -- the linear layer (moe_linear) and its gradients: products with bias,
// activation and residual in the epilogue (include/moe.h states the formulas).
#include "kernels.h"
#include "combine.cuh"

#include <math.h>

namespace moe {

__device__ __forceinline__ float act_f32(int act, float u) {
  switch (act) {
    case 1: return fmaxf(u, 0.0f);
    case 2: return u / (1.0f + expf(-u));
    case 3: return 0.5f * u * (1.0f + erff(u * 0.70710678f));
  }
  return u;
}

__device__ __forceinline__ float dact_f32(int act, float u) {
  switch (act) {
    case 1: return u > 0.0f ? 1.0f : 0.0f;
    case 2: {
      const float p = 1.0f / (1.0f + expf(-u));
      return p * (1.0f + u * (1.0f - p));
    }
    case 3: return 0.5f * (1.0f + erff(u * 0.70710678f)) + u * expf(-0.5f * u * u) * 0.39894228f;
  }
  return 1.0f;
}

// An operand of a product: element (i, j) at p[i * si + j * sj], bf16 or fp32.
struct Operand {
  const void* p;
  long si, sj;
  int f32;
};

__device__ __forceinline__ float load_op(const Operand& o, long i, long j) {
  const long at = i * o.si + j * o.sj;
  return o.f32 ? static_cast<const float*>(o.p)[at]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(o.p)[at]);
}

// C[m][n] = epilogue( sum_k A(m, k) B(k, n) ): 64 x 64 tiles, 16-deep steps, 4 x 4
// sums per thread in fp32.  For any sizes, strides and types.
__global__ void __launch_bounds__(256) gemm_simple_kernel(Operand A, Operand B, int M, int N, int K,
                                                          const LinearEpi ep) {
  pdl_trigger();
  pdl_wait();
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int kk = A.sj == 1 ? i & 15 : i >> 6, mm = A.sj == 1 ? i >> 4 : i & 63;
      sa[kk][mm] = (m0 + mm < M && k0 + kk < K) ? load_op(A, m0 + mm, k0 + kk) : 0.0f;
      const int kb = B.sj == 1 ? i >> 6 : i & 15, nn = B.sj == 1 ? i & 63 : i >> 4;
      sb[kb][nn] = (n0 + nn < N && k0 + kb < K) ? load_op(B, k0 + kb, n0 + nn) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[i] = sa[kk][ty * 4 + i]; b[i] = sb[kk][tx * 4 + i]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= M || n >= N) continue;
      const size_t at = (size_t)m * N + n;
      float u = acc[i][j] + (ep.bias ? ep.bias[n] : 0.0f);
      if (ep.pre) static_cast<__nv_bfloat16*>(ep.pre)[at] = __float2bfloat16(u);
      float v = act_f32(ep.act, u);
      if (ep.residual)
        v += ep.out_f32 ? static_cast<const float*>(ep.residual)[at]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(ep.residual)[at]);
      if (ep.out_f32) static_cast<float*>(ep.out)[at] = v;
      else static_cast<__nv_bfloat16*>(ep.out)[at] = __float2bfloat16(v);
    }
  }
}

static cudaError_t gemm_simple(const Operand& A, const Operand& B, int M, int N, int K, const LinearEpi& ep,
                               cudaStream_t s) {
  return launch_pdl(gemm_simple_kernel, dim3(cdiv(M, 64), cdiv(N, 64)), dim3(256), 0, s, A, B, M, N, K, ep);
}

// du = dout * act'(pre), and per block of rows the column sums of du.
__global__ void __launch_bounds__(256) dact_kernel(const void* __restrict__ dout, int f32,
                                                   const __nv_bfloat16* __restrict__ pre, int act, int M,
                                                   int N, int rows, float* __restrict__ du,
                                                   float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float sum = 0.0f;
  for (int m = blockIdx.y * rows; m < min(M, (int)(blockIdx.y + 1) * rows); ++m) {
    const size_t at = (size_t)m * N + n;
    float v = f32 ? static_cast<const float*>(dout)[at]
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(dout)[at]);
    if (act) v *= dact_f32(act, __bfloat162float(pre[at]));
    du[at] = v;
    sum += v;
  }
  part[(size_t)blockIdx.y * N + n] = sum;
}

__global__ void __launch_bounds__(256) dbias_kernel(const float* __restrict__ part, int nblk, int N,
                                                    float* __restrict__ dbias) {
  pdl_trigger();
  pdl_wait();
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float sum = 0.0f;
  for (int b = 0; b < nblk; ++b) sum += part[(size_t)b * N + n];
  dbias[n] = sum;
}

constexpr int DACT_ROWS = 128;

size_t linear_ws_bytes(int M, int K, int N) {
  (void)M; (void)K; (void)N;
  return 0;
}

size_t linear_bwd_ws_bytes(int M, int K, int N) {
  (void)K;
  return (size_t)M * N * 4 + (size_t)cdiv(M, DACT_ROWS) * N * 4 + 256;
}

cudaError_t launch_linear(const LinearArgs& a, void* ws, cudaStream_t s) {
  (void)ws;
  return gemm_simple({a.x, a.K, 1, 0}, {a.W, a.N, 1, 0}, a.M, a.N, a.K, a.ep, s);
}

cudaError_t launch_linear_bwd(const LinearBwdArgs& a, void* ws, cudaStream_t s) {
  float* du = static_cast<float*>(ws);
  float* part = du + (size_t)a.M * a.N;
  const int nblk = cdiv(a.M, DACT_ROWS);
  cudaError_t e = launch_pdl(dact_kernel, dim3(cdiv(a.N, 256), nblk), dim3(256), 0, s, a.dout, a.dout_f32,
                             static_cast<const __nv_bfloat16*>(a.pre), a.act, a.M, a.N, DACT_ROWS, du, part);
  if (e != cudaSuccess) return e;
  if (a.dbias) {
    e = launch_pdl(dbias_kernel, dim3(cdiv(a.N, 256)), dim3(256), 0, s, (const float*)part, nblk, a.N, a.dbias);
    if (e != cudaSuccess) return e;
  }
  LinearEpi ep = {};
  if (a.dx) {
    ep.out = a.dx;
    e = gemm_simple({du, a.N, 1, 1}, {a.W, 1, a.N, 0}, a.M, a.K, a.N, ep, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dW) {
    ep.out = a.dW;
    ep.out_f32 = a.dW_f32;
    e = gemm_simple({a.x, 1, a.K, 0}, {du, a.N, 1, 1}, a.K, a.N, a.M, ep, s);
  }
  return e;
}

}  // namespace moe
