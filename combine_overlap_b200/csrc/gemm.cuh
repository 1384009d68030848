// gemm.cuh -- what the linear layer's tensor-core product (gemm.cu) takes.
#pragma once

#include "kernels.h"

namespace moe {

// C [M][N] = epilogue( sum over B's planes p and over k of A(m, k) B_p(k, n) ).
// An operand is `planes` bf16 matrices, `plane` bytes apart, of rows `ld` bytes apart
// (multiples of 16; base 16-byte aligned):
//   A: [M][K] (k contiguous) or, a_mn set, [K][M] (m contiguous); its first plane counts
//   B: [K][N] (n contiguous, b_mn set) or [N][K] (k contiguous; one plane)
// Planes are the bf16 terms of an operand of more than 8 bits; each stage of the
// operand ring holds all of them, so A is read once for all.
struct GemmOperand {
  const void* p;
  size_t ld, plane;
  int planes;
};

// Partial column sums [nblk][N] and where their sums go: done beside the join of slices.
struct ColumnSums {
  const float* part;
  int nblk, N;
  float* out;                    // null: none
};

struct GemmProblem {
  GemmOperand A, B;
  int a_mn, b_mn;
  int M, N, K;
  LinearEpi ep;
  void* ws;                      // gemm_ws_bytes(M, N) for slices of the reduction, or null;
                                 // with an output alone (no bias, activation, residual, pre)
  ColumnSums* sums;              // done if the reduction is cut into slices (out is then cleared), or null
};

// 32 columns' sums by a block of W warps: each every W-th row of partial sums.
template <int W>
__device__ __forceinline__ void column_sums(const ColumnSums& c, int block, float (*sh)[33]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = block * 32 + lane;
  float sum = 0.0f;
  if (n < c.N) {
#pragma unroll 8
    for (int b = w; b < c.nblk; b += W) sum += c.part[(size_t)b * c.N + n];
  }
  sh[w][lane] = sum;
  __syncthreads();
  if (w == 0 && n < c.N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += sh[i][lane];
    c.out[n] = s;
  }
}

// The current device and its SMs (asked of the driver once per device).
cudaError_t device_of(int* dev, int* sms);

size_t gemm_ws_bytes(int M, int N);
int gemm_slices(int M, int N);
cudaError_t launch_gemm(const GemmProblem& p, cudaStream_t s);

__device__ __forceinline__ float act_f32(int act, float u) {
  switch (act) {
    case 1: return u < 0.0f ? 0.0f : u;   // a NaN stays one
    case 2: return __fdividef(u, 1.0f + __expf(-u));
    case 3: return 0.5f * u * (1.0f + erff(u * 0.70710678f));
  }
  return u;
}

}  // namespace moe
