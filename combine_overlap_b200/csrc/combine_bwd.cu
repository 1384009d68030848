// combine_bwd.cu -- the gradient of the weighted reduction (moe_combine_backward):
// with r = row_of[t*k + j],
//   dy[r] = bf16(g[t][j] * dout[t]),   dgate[t][j] = sum_c dout[t][c] y[r][c].
// One warp per token: dout[t] is read once for all k rows, each y row once, each dy
// row written once with 16-byte stores; the dots are fp32 sums per lane, joined by a
// shuffle tree, so the bits do not depend on the grid.
#include "kernels.h"
#include "combine.cuh"

namespace moe {

__global__ void __launch_bounds__(256)
combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                   const int32_t* __restrict__ row_of, const float* __restrict__ gate, int T, int dv,
                   int k, uint4* __restrict__ dy, float* __restrict__ dgate) {
  pdl_trigger();
  pdl_wait();
  const unsigned R = (unsigned)T * (unsigned)k;
  const int lane = threadIdx.x & 31;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < T; t += gridDim.x * 8) {
    const int my_row = lane < k ? row_of[(size_t)t * k + lane] : -1;
    const float my_gate = lane < k ? gate[(size_t)t * k + lane] : 0.0f;
    int rows[MAX_K];
    float g[MAX_K], dot[MAX_K];
#pragma unroll
    for (int j = 0; j < MAX_K; ++j) {
      rows[j] = __shfl_sync(0xffffffffu, my_row, j);
      g[j] = __shfl_sync(0xffffffffu, my_gate, j);
      dot[j] = 0.0f;
    }
    for (int v = lane; v < dv; v += 32) {
      float a[8];
      bf16x8_to_f32(dout[(size_t)t * dv + v], a);
#pragma unroll
      for (int j = 0; j < MAX_K; ++j) {
        if (j < k && (unsigned)rows[j] < R) {
          float b[8];
          bf16x8_to_f32(y[(size_t)rows[j] * dv + v], b);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(a[i], b[i], dot[j]);
          if (dy)
            dy[(size_t)rows[j] * dv + v] = make_uint4(
                pack_bf16x2(g[j] * a[0], g[j] * a[1]), pack_bf16x2(g[j] * a[2], g[j] * a[3]),
                pack_bf16x2(g[j] * a[4], g[j] * a[5]), pack_bf16x2(g[j] * a[6], g[j] * a[7]));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < MAX_K; ++j) {
      if (j < k) {
        float s = dot[j];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane == j) dgate[(size_t)t * k + j] = s;
      }
    }
  }
}

cudaError_t launch_combine_bwd(const __nv_bfloat16* dout, const __nv_bfloat16* y, const int32_t* row_of,
                               const float* gate, int T, int d, int k, __nv_bfloat16* dy, float* dgate,
                               int num_sms, cudaStream_t s) {
  const int grid = max(1, min(cdiv(T, 8), num_sms * 8));
  return launch_pdl(combine_bwd_kernel, dim3(grid), dim3(256), 0, s, reinterpret_cast<const uint4*>(dout),
                    reinterpret_cast<const uint4*>(y), row_of, gate, T, d / 8, k,
                    reinterpret_cast<uint4*>(dy), dgate);
}

}  // namespace moe
