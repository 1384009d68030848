// route_scored.cu -- the scored router (moe_route_scored) and the gradient of its
// gates: softmax or sigmoid scores, a selection bias, expert groups, top-k,
// renormalised and scaled gates (include/moe.h states the formulas).
#include "kernels.h"

#include <float.h>
#include <math.h>

namespace moe {

namespace {

constexpr int RS_WARPS = 8;                       // warps per block; ROUTE_TOK / 8 tokens each
constexpr int RS_TOK = ROUTE_TOK / RS_WARPS;
static_assert(RS_TOK * MAX_K <= 32, "a lane for each slot of a warp's tokens");

// Keys as unsigned integers of the same order; 0: not to be chosen, 1: masked (after every
// live expert, before none), so a warp's largest is one redux instruction away.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);   // -0 and 0 are one key
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu)); }

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// An E-expert row over a warp: lane l holds experts l C .. l C + C - 1, C = ceil(E / 32).
template <int CM>
struct Row {
  float z[CM];
  uint32_t live, have;                            // bits over i: not masked, exists
};

template <int CM>
__device__ __forceinline__ void load_row(const float* __restrict__ p, int E, int C, int lane, Row<CM>& r) {
  const int e0 = lane * C;
  if (CM >= 4 && C == CM && (E & 3) == 0) {
#pragma unroll
    for (int i = 0; i < CM / 4; ++i) {
      const float4 v = e0 + 4 * i < E ? __ldg(reinterpret_cast<const float4*>(p + e0) + i) : make_float4(0, 0, 0, 0);
      r.z[4 * i] = v.x; r.z[4 * i + 1] = v.y; r.z[4 * i + 2] = v.z; r.z[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CM; ++i) r.z[i] = i < C && e0 + i < E ? __ldg(p + e0 + i) : 0.0f;
  }
}

// Sets the masks; a logit of +infinity counts as FLT_MAX, masked ones as 0.
template <int CM>
__device__ __forceinline__ void mask_row(int E, int C, int lane, Row<CM>& r) {
  r.live = r.have = 0;
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    const bool have = i < C && lane * C + i < E, live = have && r.z[i] >= -FLT_MAX;   // not NaN, not -infinity
    r.have |= have ? 1u << i : 0u;
    r.live |= live ? 1u << i : 0u;
    r.z[i] = live ? fminf(r.z[i], FLT_MAX) : 0.0f;
  }
}

// The row's largest live logit (-FLT_MAX if none), and the sum of exp(z - largest) in fp32.
template <int CM>
__device__ __forceinline__ float top_row(const Row<CM>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CM; ++i)
    if (r.live >> i & 1u) m = max(m, ordered(r.z[i]));
  m = warp_max(m);
  return m ? unordered(m) : -FLT_MAX;
}
template <int CM>
__device__ __forceinline__ void softmax_row(const Row<CM>& r, float (&ex)[CM], float* top, float* sum) {
  *top = top_row<CM>(r);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    ex[i] = (r.live >> i & 1u) ? expf(r.z[i] - *top) : 0.0f;
    s += ex[i];
  }
  *sum = warp_sum(s);
}

// One warp chooses one token's experts: lane `slot0 + j` gets slot j's id in *my_e.  Keys
// and group values are formed in F (float or double) and compared as they are.  In float
// every decision is checked: a key is within 2^-19 + 2^-22 |key| of its 64-bit value (the
// scores are at most 1; their sum has 13 roundings at the most, an exponential and a
// division two each), so two that differ by more than twice that are in the right order; without a bias the keys are the logits themselves, and exact.
// False: too close to call, the caller has the choice made in double.
template <typename F, typename U, int CM>
__device__ bool choose(const Row<CM>& r, int E, int C, int k, const RouterArgs& o, int lane, int slot0, int* my_e) {
  constexpr bool FAST = sizeof(F) == 4;
  const bool grouped = o.topk_groups < o.n_groups;
  const bool scores = o.bias != nullptr || (grouped && o.group_top2);   // p is needed
  F biased[CM];
  U key[CM];
  float reach = 0.0f;                             // the largest |p + bias|
  if (scores) {
    if (o.score == 0) {
      if constexpr (FAST) {
        float top, sum;
        softmax_row(r, biased, &top, &sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < CM; ++i) biased[i] *= inv;
      } else {
        const double top = top_row<CM>(r);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < CM; ++i) {
          biased[i] = (r.live >> i & 1u) ? exp((double)r.z[i] - top) : 0.0;
          s += biased[i];
        }
        s = warp_sum(s);
        s = s > 0.0 ? s : 1.0;
#pragma unroll
        for (int i = 0; i < CM; ++i) biased[i] /= s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        if constexpr (FAST) biased[i] = (r.live >> i & 1u) ? __fdividef(1.0f, 1.0f + expf(-r.z[i])) : 0.0f;
        else biased[i] = (r.live >> i & 1u) ? 1.0 / (1.0 + exp(-(double)r.z[i])) : 0.0;
      }
    }
    if (o.bias) {
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (r.have >> i & 1u) biased[i] += (F)__ldg(o.bias + lane * C + i);
    }
  }
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    const F v = o.bias ? biased[i] : (F)r.z[i];
    key[i] = (r.live >> i & 1u) ? ordered(v) : (r.have >> i & 1u) ? (U)1 : (U)0;
    if (FAST && scores && (r.live >> i & 1u)) reach = fmaxf(reach, fabsf((float)biased[i]));
  }
  bool sure = true;
  if (FAST && scores) reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(reach)));

  if (grouped) {
    const int S = E / o.n_groups, L = S / C;
    U mine = 0;                                   // the value of this lane's group, if it speaks for one
    int shift = 0;                                // group g's speaker is lane g << shift
    if (S % C == 0 && (L & (L - 1)) == 0) {
      // groups are aligned runs of L lanes
      F a = -INFINITY, b = -INFINITY;             // the two largest, a >= b
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        if (r.live >> i & 1u) {
          const F v = (o.group_top2 || o.bias) ? biased[i] : (F)r.z[i];
          if (v > a) { b = a; a = v; } else if (v > b) b = v;
        }
      }
      for (int off = 1; off < L; off <<= 1) {
        const F oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
        b = a >= oa ? (oa > b ? oa : b) : (a > ob ? a : ob);
        a = a >= oa ? a : oa;
      }
      shift = __ffs(L) - 1;
      const F v = o.group_top2 && b != -INFINITY ? a + b : a;
      if ((lane & (L - 1)) == 0 && (lane >> shift) < o.n_groups) mine = ordered(v);
    } else {
      for (int g = 0; g < o.n_groups; ++g) {
        F a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < CM; ++i) {
          const int e = lane * C + i;
          if ((r.live >> i & 1u) && e >= g * S && e < g * S + S) {
            const F v = (o.group_top2 || o.bias) ? biased[i] : (F)r.z[i];
            if (v > a) { b = a; a = v; } else if (v > b) b = v;
          }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const F oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
          b = a >= oa ? (oa > b ? oa : b) : (a > ob ? a : ob);
          a = a >= oa ? a : oa;
        }
        const F v = o.group_top2 && b != -INFINITY ? a + b : a;
        if (lane == g) mine = ordered(v);
      }
    }
    uint32_t chosen = 0;
    U last = 0;
    for (int j = 0; j < o.topk_groups; ++j) {
      last = warp_max(mine);
      const int who = __ffs(__ballot_sync(0xffffffffu, mine == last)) - 1;
      chosen |= 1u << (who >> shift);
      if (lane == who) mine = 0;
    }
    if constexpr (FAST) {
      const uint32_t next = warp_max(mine);
      if (scores && next > ordered(-INFINITY))
        sure = unordered(last) - unordered(next) > 7.63e-6f + 9.54e-7f * reach;   // 2^-17, 2^-20: two keys' errors each
    }
#pragma unroll
    for (int i = 0; i < CM; ++i)
      if (!(chosen >> ((lane * C + i) / S) & 1u)) key[i] = 0;
  }

  // the lane's best, then the warp's, k times
  U best = 0;
  int at = 0;
  auto rescan = [&] {
    best = 0;
#pragma unroll
    for (int i = 0; i < CM; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
  };
  rescan();
  const int rounds = k + (FAST && o.bias ? 1 : 0);
  U prev = 0;
  for (int j = 0; j < rounds; ++j) {
    const U top = warp_max(best);
    if constexpr (FAST) {
      if (o.bias && j > 0 && top > 1 && !(unordered(prev) - unordered(top) > 3.815e-6f + 4.77e-7f * reach)) sure = false;
    }
    prev = top;
    if (j == k) break;
    // lanes hold ascending runs of experts: the lowest lane has the lowest id
    const int who = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    const int e = __shfl_sync(0xffffffffu, lane * C + at, who);
    if (lane == slot0 + j) *my_e = e;
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (i == at) key[i] = 0;
      rescan();
    }
  }
  return sure;
}

// A warp routes RS_TOK tokens one after the other; then lane 8 q + j makes the gate of
// token q's slot j in 64 bits, one exponential for all of them.
template <int CM>
__global__ void __launch_bounds__(RS_WARPS * 32)
route_scored_kernel(const float* __restrict__ logits, int T, int E, int k, const RouterArgs o,
                    int32_t* __restrict__ topk_idx, float* __restrict__ topk_gate,
                    int32_t* __restrict__ blk_hist, uint32_t* __restrict__ arrive,
                    uint32_t* __restrict__ ready_q) {
  pdl_trigger();
  pdl_wait();
  __shared__ int hist[MAX_E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = cdiv(E, 32);
  if (blk_hist) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int t0 = blockIdx.x * ROUTE_TOK + warp;   // its tokens: t0, t0 + 8, ..
  int my_e = 0;
  float my_top = 0.0f, my_sum = 1.0f;
  Row<CM> next;
  if (t0 < T) load_row<CM>(logits + (size_t)t0 * E, E, C, lane, next);
#pragma unroll 1
  for (int q = 0; q < RS_TOK; ++q) {
    const int t = t0 + q * RS_WARPS;
    if (t >= T) break;
    Row<CM> r = next;
    if (q + 1 < RS_TOK && t + RS_WARPS < T) load_row<CM>(logits + (size_t)(t + RS_WARPS) * E, E, C, lane, next);
    mask_row<CM>(E, C, lane, r);
    if (!choose<float, uint32_t, CM>(r, E, C, k, o, lane, q * MAX_K, &my_e))
      choose<double, uint64_t, CM>(r, E, C, k, o, lane, q * MAX_K, &my_e);
    if (o.score == 0) {
      float ex[CM], top, sum = 1.0f;
      if (o.renorm) top = top_row<CM>(r);         // the sum cancels
      else softmax_row<CM>(r, ex, &top, &sum);
      if (lane >> 3 == q) { my_top = top; my_sum = sum; }
    }
    if (lane == 0) {
      if (arrive) arrive[t] = 0u;
      if (ready_q) ready_q[t] = 0u;
    }
  }
  const int j = lane & 7, t = t0 + (lane >> 3) * RS_WARPS;
  const bool slot = j < k && t < T;
  const float z = slot ? __ldg(logits + (size_t)t * E + my_e) : -INFINITY;
  const bool live = z >= -FLT_MAX;
  const double zd = (double)fminf(z, FLT_MAX);
  double w = 0.0;
  if (live) w = exp(o.score == 0 ? zd - (double)my_top : -zd);
  if (o.score != 0) w = live ? 1.0 / (1.0 + w) : 0.0;
  double total = w;                               // over the token's slots
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (!o.renorm) total = o.score == 0 ? (double)my_sum : 1.0;
  if (slot) {
    topk_idx[(size_t)t * k + j] = my_e;
    topk_gate[(size_t)t * k + j] = (float)(total > 0.0 ? (double)o.scale * w / total : 0.0);
    if (blk_hist) atomicAdd(&hist[my_e], 1);
  }
  if (blk_hist == nullptr) return;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) blk_hist[(size_t)blockIdx.x * E + e] = hist[e];
}

// The gradient.  With w the chosen scores, S their sum and c_j = scale * dgate_j:
//   dp_j = c_j, or (c_j - sum_i c_i w_i / S) / S with renorm;
//   softmax: dz_e = p_e (dp_e - sum_j p_j dp_j);  sigmoid: dz_e = dp_e p_e (1 - p_e).
// With renorm the softmax's own normaliser cancels, and dz is 0 beside the chosen.
// A warp takes 4 tokens: lane 8 q + j is token q's slot j, in 64 bits; then the warp
// writes the 4 rows.  `zero`: nothing but the chosen experts' own gradients.
template <int CM>
__global__ void __launch_bounds__(256)
route_scored_bwd_kernel(const float* __restrict__ dgate, const float* __restrict__ logits,
                        const int32_t* __restrict__ topk_idx, int T, int E, int k, const RouterArgs o,
                        float* __restrict__ dlogits) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = lane & 7, C = cdiv(E, 32);
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
  if (t0 >= T) return;
  const int t = t0 + (lane >> 3);
  const bool slot = j < k && t < T;
  int e = slot ? topk_idx[(size_t)t * k + j] : -1;
  if ((unsigned)e >= (unsigned)E) e = -1;
  const float z = e >= 0 ? __ldg(logits + (size_t)t * E + e) : -INFINITY;
  const double c = e >= 0 ? (double)o.scale * (double)dgate[(size_t)t * k + j] : 0.0;
  const bool live = z >= -FLT_MAX;
  const double zd = (double)fminf(z, FLT_MAX);
  const bool zero = o.score != 0 || o.renorm;
  float my_top = 0.0f, my_sum = 1.0f;
  if (o.score == 0) {
#pragma unroll 1
    for (int q = 0; q < 4 && t0 + q < T; ++q) {
      Row<CM> r;
      load_row<CM>(logits + (size_t)(t0 + q) * E, E, C, lane, r);
      mask_row<CM>(E, C, lane, r);
      float ex[CM], top, sum;
      softmax_row<CM>(r, ex, &top, &sum);
      if (lane >> 3 == q) { my_top = top; my_sum = sum > 0.0f ? sum : 1.0f; }
    }
  }
  auto sum8 = [](double v) {
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  double w = 0.0;
  if (live) w = exp(o.score == 0 ? zd - (double)my_top : -zd);
  if (o.score == 0) w /= (double)my_sum;
  else w = live ? 1.0 / (1.0 + w) : 0.0;
  double dp = c;
  if (o.renorm) {
    const double S = sum8(w), cw = sum8(c * w);
    dp = S > 0.0 ? (c - cw / S) / S : 0.0;
  }
  const double dot = zero ? 0.0 : sum8(w * dp);
  const float dz = live ? (float)(o.score == 0 ? w * (dp - dot) : dp * w * (1.0 - w)) : 0.0f;
#pragma unroll 1
  for (int q = 0; q < 4 && t0 + q < T; ++q) {
    float v[CM] = {};
    if (!zero) {
      const float top = __shfl_sync(0xffffffffu, my_top, q * 8);
      const float by = (float)-__shfl_sync(0xffffffffu, dot / (double)my_sum, q * 8);
      Row<CM> r;
      load_row<CM>(logits + (size_t)(t0 + q) * E, E, C, lane, r);
      mask_row<CM>(E, C, lane, r);
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (r.live >> i & 1u) v[i] = expf(r.z[i] - top) * by;
    }
    for (int s = 0; s < k; ++s) {
      const int es = __shfl_sync(0xffffffffu, e, q * 8 + s);
      const float ds = __shfl_sync(0xffffffffu, dz, q * 8 + s);
      const int at = es - lane * C;
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (i < C && es >= 0 && at == i) v[i] = ds;
    }
    float* out = dlogits + (size_t)(t0 + q) * E + lane * C;
    if (CM >= 4 && C == CM && (E & 3) == 0) {
#pragma unroll
      for (int i = 0; i < CM / 4; ++i)
        if (lane * C + 4 * i < E)
          reinterpret_cast<float4*>(out)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (i < C && lane * C + i < E) out[i] = v[i];
    }
  }
}

}  // namespace

cudaError_t launch_route_scored(const float* logits, int T, int E, int k, const RouterArgs& r,
                                int32_t* topk_idx, float* topk_gate, int32_t* blk_hist,
                                uint32_t* arrive, uint32_t* ready_q, cudaStream_t s) {
  auto kernel = E <= 32 ? route_scored_kernel<1> : E <= 64 ? route_scored_kernel<2>
                : E <= 128 ? route_scored_kernel<4> : route_scored_kernel<8>;
  return launch_pdl(kernel, dim3(route_blocks(T)), dim3(RS_WARPS * 32), 0, s, logits, T, E, k, r, topk_idx, topk_gate,
                    blk_hist, arrive, ready_q);
}

cudaError_t launch_route_scored_bwd(const float* dgate, const float* logits, const int32_t* topk_idx,
                                    int T, int E, int k, const RouterArgs& r, float* dlogits,
                                    cudaStream_t s) {
  auto kernel = E <= 32 ? route_scored_bwd_kernel<1> : E <= 64 ? route_scored_bwd_kernel<2>
                : E <= 128 ? route_scored_bwd_kernel<4> : route_scored_bwd_kernel<8>;
  return launch_pdl(kernel, dim3(cdiv(T, 32)), dim3(256), 0, s, dgate, logits, topk_idx, T, E, k, r, dlogits);
}

}  // namespace moe
