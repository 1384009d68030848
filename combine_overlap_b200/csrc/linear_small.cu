// linear_small.cu -- the linear layer for a few rows (decode): 8 to a block.  out = x W is
// bound by reading W once, so no tensor core is fed: each lane streams vectors of V columns of W,
// 8 of them in flight, against x in shared memory, and keeps M x V fp32 sums.  The k-range
// is shared by a block's warps (and a warp's lane groups, where N is small) and by a cluster
// of S blocks; sums join by shuffles, through shared memory and through distributed shared
// memory, always in the same order.  W is read as it lies: V is what N's divisors allow, so
// rows that are no multiple of 16 bytes need no padded copy.
#include "gemm.cuh"
#include "combine.cuh"

namespace moe {

namespace {

constexpr int SM_KC = 512;                        // x's k per pass through shared memory
constexpr int SM_U = 8;                           // vectors of W in flight per lane

struct SmallArgs {
  int M, K, N;
  const __nv_bfloat16* x;
  const __nv_bfloat16* W;
  int tx;                                         // lanes along the columns, a power of two
  int S;                                          // blocks of a cluster, sharing k
  LinearEpi ep;
};

template <int V> struct Vec;
template <> struct Vec<8> { typedef uint4 T; };
template <> struct Vec<4> { typedef uint2 T; };
template <> struct Vec<2> { typedef uint32_t T; };
template <> struct Vec<1> { typedef unsigned short T; };

template <int V>
__device__ __forceinline__ void widen(const typename Vec<V>::T& r, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = __uint_as_float((uint32_t)r << 16);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void finish1(const LinearEpi& e, int N, int m, int n, float v) {
  const size_t at = (size_t)m * N + n;
  if (e.bias) v += __ldg(e.bias + n);
  if (e.pre) static_cast<__nv_bfloat16*>(e.pre)[at] = __float2bfloat16(v);
  v = act_f32(e.act, v, e.out_f32);
  if (e.out_f32) {
    if (e.residual) v += static_cast<const float*>(e.residual)[at];
    static_cast<float*>(e.out)[at] = v;
  } else {
    if (e.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at]);
    static_cast<__nv_bfloat16*>(e.out)[at] = __float2bfloat16(v);
  }
}

template <int MB, int V>
__global__ void __launch_bounds__(256) linear_small_kernel(const SmallArgs a) {
  __shared__ float xs[MB][SM_KC];
  __shared__ float red[8][32 * V];
  __shared__ float sums[MB][32 * V];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tx = a.tx, G = 32 / tx, S = a.S, K = a.K, N = a.N;
  const int m0 = blockIdx.y * 8, M = min(8, a.M - m0);
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = blockIdx.x / S * (tx * V), n = n0 + (lane & (tx - 1)) * V;
  const int row = warp * G + lane / tx, rows = 8 * G;
  const int k0 = (int)((long long)K * rank / S), k1 = (int)((long long)K * (rank + 1) / S);
  float acc[MB][V];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[m][i] = 0.0f;

  for (int kc = k0; kc < k1; kc += SM_KC) {
    const int len = min(SM_KC, k1 - kc);
    for (int i = threadIdx.x; i < MB * SM_KC; i += 256) {
      const int m = i / SM_KC, k = i % SM_KC;
      xs[m][k] = m < M && k < len ? __bfloat162float(__ldg(a.x + (size_t)(m0 + m) * K + kc + k)) : 0.0f;
    }
    __syncthreads();
    if (n < N) {
      const __nv_bfloat16* w = a.W + (size_t)kc * N + n;
      for (int k = row; k < len; k += rows * SM_U) {
        typename Vec<V>::T r[SM_U];
#pragma unroll
        for (int u = 0; u < SM_U; ++u)
          if (k + u * rows < len) r[u] = __ldg(reinterpret_cast<const typename Vec<V>::T*>(w + (size_t)(k + u * rows) * N));
#pragma unroll
        for (int u = 0; u < SM_U; ++u) {
          if (k + u * rows >= len) break;
          float f[V];
          widen<V>(r[u], f);
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const float xv = xs[m][k + u * rows];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[m][i] = fmaf(xv, f[i], acc[m][i]);
          }
        }
      }
    }
    __syncthreads();
  }
  // over the lane groups, then the warps
  for (int off = tx; off < 32; off <<= 1) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], off);
  }
  const int cols = tx * V;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    if (lane < tx) {
#pragma unroll
      for (int i = 0; i < V; ++i) red[warp][lane * V + i] = acc[m][i];
    }
    __syncthreads();
    if ((int)threadIdx.x < cols) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
      sums[m][threadIdx.x] = s;
    }
    __syncthreads();
  }
  if (S > 1) cluster_sync();
  for (int i = rank * 256 + threadIdx.x; i < M * cols; i += S * 256) {
    const int m = i / cols, c = i - m * cols;
    if (n0 + c >= N) continue;
    float v = 0.0f;
    if (S > 1) {
      float part[8];
      const uint32_t at = smem_u32(&sums[m][c]);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < S) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part[s]) : "r"(mapa_shared(at, (uint32_t)s)) : "memory");
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < S) v += part[s];
    } else {
      v = sums[m][c];
    }
    finish1(a.ep, N, m0 + m, n0 + c, v);
  }
  if (S > 1) cluster_sync();                      // no block leaves while its sums are read
}

template <int MB, int V>
cudaError_t run(const SmallArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)cdiv(a.M, 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_small_kernel<MB, V>, a);
}

template <int V>
cudaError_t run_rows(const SmallArgs& a, int grid, cudaStream_t s) {
  if (a.M <= 1) return run<1, V>(a, grid, s);
  if (a.M <= 2) return run<2, V>(a, grid, s);
  if (a.M <= 4) return run<4, V>(a, grid, s);
  return run<8, V>(a, grid, s);
}

}  // namespace

cudaError_t launch_linear_small(const LinearArgs& l, int num_sms, cudaStream_t s) {
  SmallArgs a = {l.M, l.K, l.N, static_cast<const __nv_bfloat16*>(l.x), static_cast<const __nv_bfloat16*>(l.W), 1, 1, l.ep};
  const int V = a.N % 8 == 0 ? 8 : a.N % 4 == 0 ? 4 : a.N % 2 == 0 ? 2 : 1;
  while (a.tx < 32 && a.tx * V < a.N) a.tx *= 2;
  const int tiles = cdiv(a.N, a.tx * V) * cdiv(a.M, 8), rows = 8 * (32 / a.tx);
  // k shared by up to 8 blocks, while there are fewer than 4 blocks per SM and each lane
  // keeps its loads in flight
  while (a.S < 8 && tiles * a.S < 4 * num_sms && a.K >= a.S * 2 * rows * SM_U) a.S *= 2;
  const int grid = cdiv(a.N, a.tx * V) * a.S;
  return V == 8 ? run_rows<8>(a, grid, s) : V == 4 ? run_rows<4>(a, grid, s) : V == 2 ? run_rows<2>(a, grid, s)
                                                                                      : run_rows<1>(a, grid, s);
}

}  // namespace moe
