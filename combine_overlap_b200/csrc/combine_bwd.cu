// combine_bwd.cu -- the gradient of the weighted reduction (moe_combine_backward):
// with r = row_of[t*k + j],
//   dy[r] = bf16(g[t][j] * dout[t]),   dgate[t][j] = sum_c dout[t][c] y[r][c].
// Memory-bound: dout[t] is read once for all k rows, each y row once, each dy row written
// once.  W warps share a token (W by d alone: 1 up to d = 512, 8 from 4096), each lane with
// U 16-byte vectors of dout and of the k rows in flight.  The dots are fp32 sums per lane,
// joined by a shuffle tree and then warp by warp, so the bits depend on d and k only.
#include "kernels.h"
#include "combine.cuh"

namespace moe {

namespace {

template <int KM, int U>
__global__ void __launch_bounds__(256)
combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                   const int32_t* __restrict__ row_of, const float* __restrict__ gate, int T, int dv,
                   int k, int W, uint4* __restrict__ dy, float* __restrict__ dgate) {
  pdl_trigger();
  pdl_wait();
  __shared__ float part[8][KM];
  const unsigned R = (unsigned)T * (unsigned)k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp & (W - 1);
  const int t = blockIdx.x * (8 / W) + warp / W;
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  if (t < T) {
    unsigned rows[KM];
    float g[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      rows[j] = j < k ? (unsigned)__ldg(row_of + (size_t)t * k + j) : R;
      g[j] = j < k ? __ldg(gate + (size_t)t * k + j) : 0.0f;
    }
    for (int v0 = w * 32 + lane; v0 < dv; v0 += 32 * W * U) {
      uint4 in[U], b[U][KM];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * 32 * W;
        if (v >= dv) break;
        in[u] = __ldg(dout + (size_t)t * dv + v);
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (rows[j] < R) b[u][j] = __ldg(y + (size_t)rows[j] * dv + v);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * 32 * W;
        if (v >= dv) break;
        float a[8];
        bf16x8_to_f32(in[u], a);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (rows[j] >= R) continue;
          float f[8];
          bf16x8_to_f32(b[u][j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(a[i], f[i], dot[j]);
          if (dy)
            dy[(size_t)rows[j] * dv + v] = make_uint4(
                pack_bf16x2(g[j] * a[0], g[j] * a[1]), pack_bf16x2(g[j] * a[2], g[j] * a[3]),
                pack_bf16x2(g[j] * a[4], g[j] * a[5]), pack_bf16x2(g[j] * a[6], g[j] * a[7]));
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], off);
    if (lane == 0) part[warp][j] = dot[j];
  }
  __syncthreads();
  if (w == 0 && lane < k && t < T) {
    float s = part[warp][lane];
    for (int i = 1; i < W; ++i) s += part[warp + i][lane];
    dgate[(size_t)t * k + lane] = s;
  }
}

}  // namespace

cudaError_t launch_combine_bwd(const __nv_bfloat16* dout, const __nv_bfloat16* y, const int32_t* row_of,
                               const float* gate, int T, int d, int k, __nv_bfloat16* dy, float* dgate,
                               cudaStream_t s) {
  const int dv = d / 8;
  int W = 1;
  while (W < 8 && dv > 64 * W) W *= 2;
  auto kernel = k <= 1 ? combine_bwd_kernel<1, 2> : k <= 2 ? combine_bwd_kernel<2, 2>
                : k <= 4 ? combine_bwd_kernel<4, 2> : combine_bwd_kernel<8, 1>;
  return launch_pdl(kernel, dim3(cdiv(T, 8 / W)), dim3(256), 0, s, reinterpret_cast<const uint4*>(dout),
                    reinterpret_cast<const uint4*>(y), row_of, gate, T, dv, k, W, reinterpret_cast<uint4*>(dy), dgate);
}

}  // namespace moe
