// route_scored.cu -- the scored router (moe_route_scored) and the gradient of its
// gates: softmax or sigmoid scores, a selection bias, expert groups, top-k,
// renormalised and scaled gates (include/moe.h states the formulas).
#include "kernels.h"

#include <float.h>
#include <math.h>

namespace moe {

constexpr int RS_WARPS = 8;                       // warps per block; ROUTE_TOK / 8 tokens each
constexpr int RS_EPL = MAX_E / 32;                // experts per lane: lane l holds l, l + 32, ...

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One warp routes one token, every value in 64 bits.  z[i]: logit of expert
// lane + 32 i; bit i of live: that expert exists and is not masked; bit i of have:
// it exists.  Lane j < k returns slot j's expert and gate.
__device__ void route_token_f64(const float (&z)[RS_EPL], uint32_t live, uint32_t have, int E, int k,
                                const RouterArgs& r, int lane, int* my_e, double* my_p) {
  constexpr double MASKED = -DBL_MAX;             // below every key, above an excluded expert
  double p[RS_EPL], key[RS_EPL];
  if (r.score == 0) {
    double m = -DBL_MAX;
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i)
      if (live >> i & 1u) m = fmax(m, (double)z[i]);
    m = warp_max(m);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) {
      p[i] = (live >> i & 1u) ? exp((double)z[i] - m) : 0.0;
      s += p[i];
    }
    s = warp_sum(s);
    s = s > 0.0 ? s : 1.0;
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) p[i] /= s;
  } else {
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) p[i] = (live >> i & 1u) ? 1.0 / (1.0 + exp(-(double)z[i])) : 0.0;
  }
  double biased[RS_EPL];
#pragma unroll
  for (int i = 0; i < RS_EPL; ++i) {
    const int e = lane + 32 * i;
    biased[i] = p[i] + ((have >> i & 1u) && r.bias ? (double)__ldg(r.bias + e) : 0.0);
    key[i] = (live >> i & 1u) ? (r.bias ? biased[i] : (double)z[i]) : MASKED;
  }
  uint32_t open = have;                           // experts that may still be chosen
  if (r.topk_groups < r.n_groups) {
    const int S = E / r.n_groups;
    double mine = -INFINITY;                      // lane g: the value of group g
    for (int g = 0; g < r.n_groups; ++g) {
      double a = -INFINITY, b = -INFINITY;        // the two largest, a >= b
#pragma unroll
      for (int i = 0; i < RS_EPL; ++i) {
        if ((live >> i & 1u) && (lane + 32 * i) / S == g) {
          const double v = r.group_top2 ? biased[i] : key[i];
          if (v > a) { b = a; a = v; } else if (v > b) b = v;
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const double oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
        b = fmax(fmin(a, oa), a >= oa ? b : ob);
        a = fmax(a, oa);
      }
      const double v = r.group_top2 && b != -INFINITY ? a + b : a;
      if (lane == g) mine = v;
    }
    int rank = 0;
    for (int g = 0; g < r.n_groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const uint32_t chosen = __ballot_sync(0xffffffffu, lane < r.n_groups && rank < r.topk_groups);
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) {
      const int e = lane + 32 * i;
      if ((have >> i & 1u) && !(chosen >> (e / S) & 1u)) open &= ~(1u << i);
    }
  }
  for (int j = 0; j < k; ++j) {
    double bv = -INFINITY, bp = 0.0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) {
      if ((open >> i & 1u) && key[i] > bv) { bv = key[i]; be = lane + 32 * i; bp = p[i]; }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, bv, off);
      const double op = __shfl_xor_sync(0xffffffffu, bp, off);
      const int oe = __shfl_xor_sync(0xffffffffu, be, off);
      if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; bp = op; }
    }
    if ((be & 31) == lane) open &= ~(1u << (be >> 5));
    if (lane == j) { *my_e = be; *my_p = bp; }
  }
}

__global__ void __launch_bounds__(RS_WARPS * 32)
route_scored_kernel(const float* __restrict__ logits, int T, int E, int k, const RouterArgs r,
                    int32_t* __restrict__ topk_idx, float* __restrict__ topk_gate,
                    int32_t* __restrict__ blk_hist, uint32_t* __restrict__ arrive,
                    uint32_t* __restrict__ ready_q) {
  pdl_trigger();
  pdl_wait();
  __shared__ int hist[MAX_E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  for (int q = 0; q < ROUTE_TOK / RS_WARPS; ++q) {
    const int t = blockIdx.x * ROUTE_TOK + q * RS_WARPS + warp;
    if (t >= T) break;
    float z[RS_EPL];
    uint32_t live = 0, have = 0;
#pragma unroll
    for (int i = 0; i < RS_EPL; ++i) {
      const int e = lane + 32 * i;
      z[i] = e < E ? __ldg(logits + (size_t)t * E + e) : 0.0f;
      if (e < E) have |= 1u << i;
      if (e < E && z[i] >= -FLT_MAX) live |= 1u << i;   // not NaN, not -infinity
      z[i] = fminf(z[i], FLT_MAX);
    }
    int my_e = 0;
    double my_p = 0.0;
    route_token_f64(z, live, have, E, k, r, lane, &my_e, &my_p);
    double sum = 0.0;
    for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, my_p, j);
    if (lane < k) {
      double g = my_p;
      if (r.renorm) g = sum > 0.0 ? my_p / sum : 0.0;
      topk_idx[(size_t)t * k + lane] = my_e;
      topk_gate[(size_t)t * k + lane] = (float)((double)r.scale * g);
      if (blk_hist) atomicAdd(&hist[my_e], 1);
    }
    if (lane == 0) {
      if (arrive) arrive[t] = 0u;
      if (ready_q) ready_q[t] = 0u;
    }
  }
  if (blk_hist == nullptr) return;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) blk_hist[(size_t)blockIdx.x * E + e] = hist[e];
}

cudaError_t launch_route_scored(const float* logits, int T, int E, int k, const RouterArgs& r,
                                int32_t* topk_idx, float* topk_gate, int32_t* blk_hist,
                                uint32_t* arrive, uint32_t* ready_q, cudaStream_t s) {
  return launch_pdl(route_scored_kernel, dim3(route_blocks(T)), dim3(RS_WARPS * 32), 0, s, logits, T, E,
                    k, r, topk_idx, topk_gate, blk_hist, arrive, ready_q);
}

// The gradient: one warp per token; lane j < k holds slot j.  With w the chosen
// scores, S their sum and c_j = scale * dgate_j:
//   dp_j = c_j, or (c_j - sum_i c_i w_i / S) / S with renorm;
//   softmax: dz_e = p_e (dp_e - sum_j p_j dp_j);  sigmoid: dz_e = dp_e p_e (1 - p_e).
// With renorm the softmax's own normaliser cancels, and dz is 0 beside the chosen.
__global__ void __launch_bounds__(256)
route_scored_bwd_kernel(const float* __restrict__ dgate, const float* __restrict__ logits,
                        const int32_t* __restrict__ topk_idx, int T, int E, int k, const RouterArgs r,
                        float* __restrict__ dlogits) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < T; t += gridDim.x * 8) {
    const float* z = logits + (size_t)t * E;
    int e = lane < k ? topk_idx[(size_t)t * k + lane] : -1;
    if ((unsigned)e >= (unsigned)E) e = -1;
    const float ze = e >= 0 ? fminf(z[e], FLT_MAX) : 0.0f;
    const bool live = e >= 0 && z[e] >= -FLT_MAX;
    const double c = e >= 0 ? (double)r.scale * (double)dgate[(size_t)t * k + lane] : 0.0;
    double m = 0.0, total = 1.0, w;
    if (r.score == 0) {
      m = -DBL_MAX;
      for (int i = lane; i < E; i += 32)
        if (z[i] >= -FLT_MAX) m = fmax(m, (double)fminf(z[i], FLT_MAX));
      m = warp_max(m);
      total = 0.0;
      for (int i = lane; i < E; i += 32)
        if (z[i] >= -FLT_MAX) total += exp((double)fminf(z[i], FLT_MAX) - m);
      total = warp_sum(total);
      if (!(total > 0.0)) total = 1.0;
      w = live ? exp((double)ze - m) / total : 0.0;
    } else {
      w = live ? 1.0 / (1.0 + exp(-(double)ze)) : 0.0;
    }
    double dp = c;
    if (r.renorm) {
      const double S = warp_sum(w);
      const double cw = warp_sum(c * w);
      dp = S > 0.0 ? (c - cw / S) / S : 0.0;
    }
    const double dot = r.score == 0 ? warp_sum(w * dp) : 0.0;
    for (int i = lane; i < E; i += 32) {
      float dz = 0.0f;
      if (r.score == 0 && z[i] >= -FLT_MAX)
        dz = (float)(exp((double)fminf(z[i], FLT_MAX) - m) / total * -dot);
      dlogits[(size_t)t * E + i] = dz;
    }
    __syncwarp();
    if (live) {
      const double dz = r.score == 0 ? w * (dp - dot) : dp * w * (1.0 - w);
      dlogits[(size_t)t * E + e] = (float)dz;
    }
  }
}

cudaError_t launch_route_scored_bwd(const float* dgate, const float* logits, const int32_t* topk_idx,
                                    int T, int E, int k, const RouterArgs& r, float* dlogits,
                                    int num_sms, cudaStream_t s) {
  const int grid = max(1, min(cdiv(T, 8), num_sms * 8));
  return launch_pdl(route_scored_bwd_kernel, dim3(grid), dim3(256), 0, s, dgate, logits, topk_idx, T, E, k,
                    r, dlogits);
}

}  // namespace moe
