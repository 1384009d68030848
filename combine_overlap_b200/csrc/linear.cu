// linear.cu -- the linear layer (moe_linear) and its gradients (include/moe.h states the
// formulas): what stands before and beside the tensor-core products of gemm.cu.
//
//   pack      rows that are no multiple of 16 bytes (TMA's stride rule) -> padded copies
//   dact      du = dout act'(pre) as bf16 terms, and per block of rows du's column sums
//   dbias     the sums of those sums
#include "gemm.cuh"
#include "combine.cuh"

#include <math.h>

namespace moe {

namespace {

// EXACT: for a du that is kept in more than bf16.
template <bool EXACT>
__device__ __forceinline__ float dact_f32(int act, float u) {
  switch (act) {
    case 1: return u > 0.0f ? 1.0f : 0.0f;
    case 2: {
      if (EXACT) {
        const Sigmoid s = sigmoid_f32(u);
        return s.p * (1.0f + u * s.q);
      }
      const float p = __fdividef(1.0f, 1.0f + __expf(-u));
      return p * (1.0f + u * (1.0f - p));
    }
    case 3: {
      const Normal g = normal_f32<EXACT>(u);
      return g.P + u * g.e * 0.39894228f;
    }
  }
  return 1.0f;
}

inline int pad8(int n) { return cdiv(n, 8) * 8; }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// ------------------------------------------------------------------- pack ---
// Up to two matrices [rows][n] -> [rows][n8], the pad zero: one thread per 8 output columns.
struct PackJob {
  const unsigned short* in;
  uint4* out;
  long rows;
  int n;                                  // 0: no such job
};

__global__ void __launch_bounds__(256) pack_kernel(const PackJob a, const PackJob b) {
  pdl_trigger();
  pdl_wait();
  const long first = a.rows * cdiv(a.n, 8), total = first + b.rows * cdiv(b.n, 8);
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const bool second = i >= first;
    const long at = second ? i - first : i;
    const int n = second ? b.n : a.n, per = cdiv(n, 8);
    const long r = at / per;
    const int c = (int)(at - r * per) * 8;
    const unsigned short* src = (second ? b.in : a.in) + r * n + c;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < n ? src[2 * j] : 0u, hi = c + 2 * j + 1 < n ? src[2 * j + 1] : 0u;
      w[j] = lo | hi << 16;
    }
    (second ? b.out : a.out)[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// `in` [rows][n] as an operand: itself, or its padded copy at `at` (advanced past it), which
// *job makes.
GemmOperand operand(const void* in, long rows, int n, char** at, PackJob* job) {
  const int n8 = pad8(n);
  GemmOperand o = {in, (size_t)n8 * 2, 0, 1};
  if (n8 == n || !in) return o;
  o.p = *at;
  *job = {static_cast<const unsigned short*>(in), reinterpret_cast<uint4*>(*at), rows, n};
  *at += up256((size_t)rows * n8 * 2);
  return o;
}

cudaError_t pack(const PackJob& a, const PackJob& b, cudaStream_t s) {
  const long total = a.rows * cdiv(a.n, 8) + b.rows * cdiv(b.n, 8);
  if (total == 0) return cudaSuccess;
  const int grid = (int)(total + 255 < 148L * 16 * 256 ? (total + 255) / 256 : 148L * 16);
  return launch_pdl(pack_kernel, dim3(grid), dim3(256), 0, s, a, b);
}

size_t pack_bytes(long rows, int n) { return n % 8 ? up256((size_t)rows * pad8(n) * 2) : 0; }

// ------------------------------------------------------------------- dact ---
// A block takes 128 columns (16 threads of 8) and `rows` rows, 16 at a time.  du's terms
// stand side by side in a row of its own: term 0 = bf16(du), term p = bf16(du - the
// earlier terms), n8 columns each.  `part`
// [gridDim.y][N] (optional): the block's column sums, in a fixed order.
// Memory bounds it: the loads of DACT_R rows are issued before the first is used, in 4 blocks
// per SM (8192 x 1408 with SiLU: 15.0 us with the sums; 16.9 with 4 rows and 2 blocks).  MODE: dout
// in bf16 or fp32 with rows of 16-byte multiples, or any (element by element).
constexpr int DACT_R = 2;
enum { DACT_BF16, DACT_F32, DACT_ANY };

template <int ACT, int MODE, bool EXACT>
__global__ void __launch_bounds__(256, 4) dact_kernel(const void* __restrict__ dout, int f32,
                                                   const __nv_bfloat16* __restrict__ pre, int M,
                                                   int N, int rows, int planes, __nv_bfloat16* __restrict__ du,
                                                   int n8, float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int n = blockIdx.x * 128 + tx * 8;
  const int m1 = min(M, (int)(blockIdx.y + 1) * rows);
  float sum[8] = {};
  if (n < n8) {
    for (int m0 = blockIdx.y * rows + ty; m0 < m1; m0 += 16 * DACT_R) {
      float v[DACT_R][8], u[DACT_R][8];
      if constexpr (MODE == DACT_ANY) {
#pragma unroll
        for (int r = 0; r < DACT_R; ++r) {
          const size_t at = (size_t)min(m0 + 16 * r, m1 - 1) * N + n;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[r][i] = n + i >= N ? 0.0f : f32 ? static_cast<const float*>(dout)[at + i]
                                              : __bfloat162float(static_cast<const __nv_bfloat16*>(dout)[at + i]);
            if (ACT) u[r][i] = n + i >= N ? 0.0f : __bfloat162float(pre[at + i]);
          }
        }
      } else {
        uint4 d[DACT_R][MODE == DACT_F32 ? 2 : 1], x[DACT_R];
#pragma unroll
        for (int r = 0; r < DACT_R; ++r) {
          const size_t at = (size_t)min(m0 + 16 * r, m1 - 1) * N + n;
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(dout) + at * (MODE == DACT_F32 ? 4 : 2));
          d[r][0] = __ldg(q);
          if (MODE == DACT_F32) d[r][MODE == DACT_F32 ? 1 : 0] = __ldg(q + 1);
          if (ACT) x[r] = __ldg(reinterpret_cast<const uint4*>(pre + at));
        }
#pragma unroll
        for (int r = 0; r < DACT_R; ++r) {
          if constexpr (MODE == DACT_F32) {
            v[r][0] = __uint_as_float(d[r][0].x); v[r][1] = __uint_as_float(d[r][0].y);
            v[r][2] = __uint_as_float(d[r][0].z); v[r][3] = __uint_as_float(d[r][0].w);
            v[r][4] = __uint_as_float(d[r][1].x); v[r][5] = __uint_as_float(d[r][1].y);
            v[r][6] = __uint_as_float(d[r][1].z); v[r][7] = __uint_as_float(d[r][1].w);
          } else {
            bf16x8_to_f32(d[r][0], v[r]);
          }
          if (ACT) bf16x8_to_f32(x[r], u[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < DACT_R; ++r) {
        const int m = m0 + 16 * r;
        if (m >= m1) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (ACT) v[r][i] *= dact_f32<EXACT>(ACT, u[r][i]);
          sum[i] += v[r][i];
        }
        __nv_bfloat16* to = du + (size_t)m * planes * n8 + n;
        for (int p = 0; p < planes; ++p, to += n8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[r][2 * i], v[r][2 * i + 1]);
          *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
          if (p + 1 == planes) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
            v[r][2 * i] = isfinite(lo) ? v[r][2 * i] - lo : 0.0f;   // an infinity has no remainder
            v[r][2 * i + 1] = isfinite(hi) ? v[r][2 * i + 1] - hi : 0.0f;
          }
        }
      }
    }
  }
  if (part == nullptr) return;
  __shared__ float sh[16][129];
#pragma unroll
  for (int i = 0; i < 8; ++i) sh[ty][tx * 8 + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 128 && blockIdx.x * 128 + c < N) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += sh[r][c];
    part[(size_t)blockIdx.y * N + blockIdx.x * 128 + c] = s;
  }
}

template <int ACT, bool EXACT>
cudaError_t launch_dact(const LinearBwdArgs& a, int rows, int planes, __nv_bfloat16* du, int n8, float* part,
                        cudaStream_t s) {
  auto kernel = a.N % 8 ? dact_kernel<ACT, DACT_ANY, EXACT>
                : a.dout_f32 ? dact_kernel<ACT, DACT_F32, EXACT> : dact_kernel<ACT, DACT_BF16, EXACT>;
  return launch_pdl(kernel, dim3(cdiv(n8, 128), cdiv(a.M, rows)), dim3(256), 0, s, a.dout, a.dout_f32,
                    static_cast<const __nv_bfloat16*>(a.pre), a.M, a.N, rows, planes, du, n8, part);
}

__global__ void __launch_bounds__(1024) dbias_kernel(const ColumnSums sums) {
  __shared__ float sh[32][33];
  pdl_trigger();
  pdl_wait();
  column_sums<32>(sums, blockIdx.x, sh);
}

// Rows per dact block: 16 at the least, so that a block has work; 64 where that leaves
// blocks for every SM; and not so few that there are more than 256 blocks of rows.
int dact_rows(int M, int N) {
  const int most = max(16, cdiv(cdiv(M, 256), 16) * 16);
  return (long long)cdiv(M, 64) * cdiv(N, 128) >= 600 ? max(64, most) : most;
}

// The bf16 terms that du is kept as.  With dW in bf16 it is rounded once, as a stored bf16
// gradient would be: an error of the size of the gradients' own rounding.  An fp32 dW takes
// three terms, all 24 bits, and dx beside it the first two: 16 bits, far below the rounding of a
// bf16 dx.  Whether dW is wanted in this call changes no bit of the others.  dout in bf16
// without an activation is du itself.
int terms_of(const LinearBwdArgs& a) { return !(a.dout_f32 || a.act) || !a.dW_f32 ? 1 : a.dW ? 3 : 2; }

}  // namespace

// Without the tensor cores (linear_small.cu) where that measured faster, launch included.
// Rows as they are: 3.4 against 4.5 us at 1 x 2048 x 64, 7.2 against 7.5 at 4 x 2048 x 1024;
// the tensor cores' stream is ahead from 8 x 2048 x 64 (5.8 / 4.7) and 1 x 4096 x 4096
// (13.2 / 12.7).  Where they need padded copies first (a launch and a workspace): 9 against
// 15 us at 4 x 2048 x 1023, 16 against 15 at 16 x 2048 x 1023, 25 against 26 at
// 1 x 4096 x 4095, 37 against 26 at 8.
bool is_small(int M, int K, int N) {
  if (K % 8 == 0 && N % 8 == 0) return M <= 4 && (long long)K * N <= 1LL << 22;
  return M <= 16 && (long long)M * K * N <= 1LL << 25;
}

size_t linear_ws_bytes(int M, int K, int N) { return is_small(M, K, N) ? 0 : pack_bytes(M, K) + pack_bytes(K, N); }

size_t linear_bwd_ws_bytes(int M, int K, int N) {
  return up256((size_t)cdiv(M, dact_rows(M, N)) * N * 4) + 3 * up256((size_t)M * pad8(N) * 2) + pack_bytes(M, K) +
         pack_bytes(K, N) + gemm_ws_bytes(K, N);
}

cudaError_t launch_linear(const LinearArgs& a, void* ws, cudaStream_t s) {
  if (is_small(a.M, a.K, a.N)) {
    int nsm = 0;
    const cudaError_t e = device_of(nullptr, &nsm);
    return e == cudaSuccess ? launch_linear_small(a, nsm, s) : e;
  }
  char* at = static_cast<char*>(ws);
  GemmProblem p = {};
  PackJob jx = {}, jw = {};
  p.A = operand(a.x, a.M, a.K, &at, &jx);
  p.B = operand(a.W, a.K, a.N, &at, &jw);
  const cudaError_t e = pack(jx, jw, s);
  if (e != cudaSuccess) return e;
  p.b_mn = 1;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.ep = a.ep;
  return launch_gemm(p, s);
}

cudaError_t launch_linear_bwd(const LinearBwdArgs& a, void* ws, cudaStream_t s) {
  char* at = static_cast<char*>(ws);
  const int rows = dact_rows(a.M, a.N), nblk = cdiv(a.M, rows), n8 = pad8(a.N);
  float* part = reinterpret_cast<float*>(at);
  at += up256((size_t)nblk * a.N * 4);
  const int terms = terms_of(a);
  GemmOperand du = {at, (size_t)terms * n8 * 2, (size_t)n8 * 2, terms};
  at += 3 * up256((size_t)a.M * n8 * 2);
  PackJob jx = {}, jw = {};
  const GemmOperand x = operand(a.dW ? a.x : nullptr, a.M, a.K, &at, &jx);
  const GemmOperand W = operand(a.dx ? a.W : nullptr, a.K, a.N, &at, &jw);
  cudaError_t e = pack(jx, jw, s);
  if (e != cudaSuccess) return e;
  // dout is an operand as it stands if it is bf16, unpadded and without an activation
  const bool direct = !a.dout_f32 && !a.act && n8 == a.N;
  if (!direct || a.dbias) {
    float* sums = !a.dbias ? nullptr : nblk == 1 ? a.dbias : part;
    __nv_bfloat16* to = (__nv_bfloat16*)du.p;
    const int n = direct || !(a.dx || a.dW) ? 0 : terms;   // 0: for dbias alone
    switch (a.act * 2 + (terms > 1)) {
      case 0: case 1: e = launch_dact<0, false>(a, rows, n, to, n8, sums, s); break;
      case 2: case 3: e = launch_dact<1, false>(a, rows, n, to, n8, sums, s); break;
      case 4: e = launch_dact<2, false>(a, rows, n, to, n8, sums, s); break;
      case 5: e = launch_dact<2, true>(a, rows, n, to, n8, sums, s); break;
      case 6: e = launch_dact<3, false>(a, rows, n, to, n8, sums, s); break;
      default: e = launch_dact<3, true>(a, rows, n, to, n8, sums, s); break;
    }
    if (e != cudaSuccess) return e;
  }
  if (direct) du = {a.dout, (size_t)n8 * 2, 0, 1};
  ColumnSums sums = {part, nblk, a.N, nblk > 1 ? a.dbias : nullptr};
  if (a.dx) {
    GemmProblem p = {};
    p.A = du;
    p.A.planes = min(terms, 2);
    p.B = W;
    p.M = a.M; p.N = a.K; p.K = a.N;
    p.ep.out = a.dx;
    e = launch_gemm(p, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dW) {
    GemmProblem p = {};
    p.A = x;
    p.B = du;
    p.a_mn = p.b_mn = 1;
    p.M = a.K; p.N = a.N; p.K = a.M;
    p.ep.out = a.dW;
    p.ep.out_f32 = a.dW_f32;
    p.ws = at;
    p.sums = &sums;
    e = launch_gemm(p, s);
    if (e != cudaSuccess) return e;
  }
  return sums.out ? launch_pdl(dbias_kernel, dim3(cdiv(a.N, 32)), dim3(1024), 0, s, sums) : cudaSuccess;
}

}  // namespace moe
