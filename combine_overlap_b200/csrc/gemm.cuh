// gemm.cuh -- what the linear layer's tensor-core product (gemm.cu) takes.
#pragma once

#include "kernels.h"

namespace moe {

// C [M][N] = epilogue( sum over planes p and over k of A_p(m, k) B_p(k, n) ), an operand of one
// plane standing in for all of them.
// An operand is `planes` bf16 matrices, `plane` bytes apart, of rows `ld` bytes apart
// (multiples of 16; base 16-byte aligned):
//   A: [M][K] (k contiguous) or, a_mn set, [K][M] (m contiguous; one plane)
//   B: [K][N] (n contiguous, b_mn set) or [N][K] (k contiguous; one plane)
// Planes are the bf16 terms of an operand of more than 8 bits.  Each stage of the operand ring
// holds all of them, so the other operand is read once for all.  A has two at the most, where k
// is contiguous in both, and B then one.
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

// p = 1 / (1 + exp(-u)) and q = 1 - p, each within a few steps of itself: the exponential is
// that of -|u|, so nothing overflows or cancels (__fdividef is good to 2 steps for 1 .. 2).
struct Sigmoid { float p, q; };
__device__ __forceinline__ Sigmoid sigmoid_f32(float u) {
  const float e = expf(-fabsf(u)), r = __fdividef(1.0f, 1.0f + e), s = e * r;
  return u >= 0.0f ? Sigmoid{r, s} : Sigmoid{s, r};
}

// The normal distribution P(u) of GELU, and e = exp(-u^2 / 2).  For fp32 results by erfc: the
// usual 1 + erf loses bits of the result from u = -0.5 on, and all of them at -5.5.  For bf16
// results by Hastings' form, P(-a) = e poly(t) with t = 1 / (1 + 0.35 a), whose coefficients were
// fitted here (least largest relative error over a = 0 .. 13.6: 3.1e-7): it keeps the tail as
// well.  8192 x 2048 x 1408 with GELU to bf16: 58 us, as with erf; 69 by erfc.  To fp32: 115 us,
// 90 with erf, and 91 with SiLU, 79 with the fast exponential.
struct Normal { float P, e; };
template <bool EXACT>
__device__ __forceinline__ Normal normal_f32(float u) {
  if (EXACT) return {0.5f * erfcf(u * -0.70710678f), expf(-0.5f * u * u)};
  const float e = __expf(-0.5f * u * u), t = __fdividef(1.0f, fmaf(0.35f, fabsf(u), 1.0f));
  float p = 0.048942413f;
  p = fmaf(p, t, -0.20211914f);
  p = fmaf(p, t, 0.24064058f);
  p = fmaf(p, t, -0.017023224f);
  p = fmaf(p, t, 0.15596138f);
  p = fmaf(p, t, 0.13335513f);
  p = fmaf(p, t, 0.14027034f);
  p = fmaf(p, t, -2.7315136e-5f) * e;
  return {u < 0.0f ? p : 1.0f - p, e};
}

// f32: for an fp32 output.  bf16 ones take SiLU from the fast exponential, whose error of
// |u| 2^-24 is far below their rounding.
__device__ __forceinline__ float act_f32(int act, float u, bool f32) {
  switch (act) {
    case 1: return u < 0.0f ? 0.0f : u;   // a NaN stays one
    case 2: return f32 ? u * sigmoid_f32(u).p : __fdividef(u, 1.0f + __expf(-u));
    case 3: return u * (f32 ? normal_f32<true>(u).P : normal_f32<false>(u).P);
  }
  return u;
}

}  // namespace moe
