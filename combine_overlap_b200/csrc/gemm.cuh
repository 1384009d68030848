// gemm.cuh -- what the linear layer's tensor-core product (gemm.cu) takes.
#pragma once

#include "kernels.h"

namespace moe {

// C [M][N] = epilogue( sum over planes pa, pb and over k of A_pa(m, k) B_pb(k, n) ).
// An operand is `planes` bf16 matrices, `plane` bytes apart, of rows `ld` bytes apart
// (a multiple of 16; base 16-byte aligned):
//   A: [M][K] (k contiguous) or, a_mn set, [K][M] (m contiguous)
//   B: [K][N] (n contiguous, b_mn set) or [N][K] (k contiguous)
// Planes are the bf16 terms of an operand of more than 8 bits; each stage of the
// operand ring holds all of them, so the other operand is read once for all.
struct GemmOperand {
  const void* p;
  size_t ld, plane;
  int planes;
};

struct GemmProblem {
  GemmOperand A, B;
  int a_mn, b_mn;
  int M, N, K;
  LinearEpi ep;
};

cudaError_t launch_gemm(const GemmProblem& p, cudaStream_t s);

__device__ __forceinline__ float act_f32(int act, float u) {
  switch (act) {
    case 1: return fmaxf(u, 0.0f);
    case 2: return u / (1.0f + expf(-u));
    case 3: return 0.5f * u * (1.0f + erff(u * 0.70710678f));
  }
  return u;
}

// Up to four consecutive outputs of row m from column n on: bias, pre-activation,
// activation, residual, one rounding.  `vec`: N is a multiple of 4.
__device__ __forceinline__ void epilogue4(const LinearEpi& ep, int N, int m, int n, float4 v, bool vec) {
  const size_t at = (size_t)m * N + n;
  float u[4] = {v.x, v.y, v.z, v.w};
  if (vec) {
    if (ep.bias) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(ep.bias + n));
      u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
    }
    if (ep.pre) {
      const __nv_bfloat162 p0 = __floats2bfloat162_rn(u[0], u[1]), p1 = __floats2bfloat162_rn(u[2], u[3]);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(ep.pre) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
    }
    if (ep.act) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = act_f32(ep.act, u[i]);
    }
    if (ep.out_f32) {
      if (ep.residual) {
        const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(ep.residual) + at);
        u[0] += r.x; u[1] += r.y; u[2] += r.z; u[3] += r.w;
      }
      *reinterpret_cast<float4*>(static_cast<float*>(ep.out) + at) = make_float4(u[0], u[1], u[2], u[3]);
    } else {
      if (ep.residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(ep.residual) + at);
        u[0] += __uint_as_float(r.x << 16); u[1] += __uint_as_float(r.x & 0xffff0000u);
        u[2] += __uint_as_float(r.y << 16); u[3] += __uint_as_float(r.y & 0xffff0000u);
      }
      const __nv_bfloat162 p0 = __floats2bfloat162_rn(u[0], u[1]), p1 = __floats2bfloat162_rn(u[2], u[3]);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(ep.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= N) break;
    float x = u[i] + (ep.bias ? ep.bias[n + i] : 0.0f);
    if (ep.pre) static_cast<__nv_bfloat16*>(ep.pre)[at + i] = __float2bfloat16(x);
    x = act_f32(ep.act, x);
    if (ep.out_f32) {
      if (ep.residual) x += static_cast<const float*>(ep.residual)[at + i];
      static_cast<float*>(ep.out)[at + i] = x;
    } else {
      if (ep.residual) x += __bfloat162float(static_cast<const __nv_bfloat16*>(ep.residual)[at + i]);
      static_cast<__nv_bfloat16*>(ep.out)[at + i] = __float2bfloat16(x);
    }
  }
}

}  // namespace moe
