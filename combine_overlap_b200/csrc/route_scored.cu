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

// Keys as unsigned integers of the same order, so a warp's largest is one redux instruction
// away; 0: not to be chosen; a masked expert comes after every live one: 1, or in 32 bits
// MASKED, the key of -infinity.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);   // -0 and 0 are one key
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
constexpr uint32_t MASKED = 0x007fffffu;
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu)); }

// exp(x) and 1 / x, a few units in the last place off; what underflows is 0.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}
// Over the 8 lanes of a token's slots.
template <typename F>
__device__ __forceinline__ F sum8(F v) {
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// What a softmax's renormalised shares take their exponentials from: the largest chosen
// logit, since the softmax's own normaliser cancels.  From the row's largest they lose their
// bits as subnormals where a bias or a group limit leaves only experts 708 and more below
// it.  Scores are 64-bit values, which end 745.13 below: what is all beyond that is 0.
__device__ __forceinline__ float share_top(float z, bool live, float row_top) {
  const float top = max8(live ? fminf(z, FLT_MAX) : -FLT_MAX);
  return (double)top - (double)row_top < -745.13 ? INFINITY : top;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// What a warp has to know, in registers.
struct Plan {
  const float *bias, *row;                        // row: the token's logits
  int E, C, k;                                    // C = ceil(E / 32)
  int softmax, top2, n_groups, topk_groups;
  bool grouped, scores;                           // groups limit the choice; p is needed for it
  int S, L, shift;                                // experts per group; lanes per group, if aligned (or 0)
};
__device__ __forceinline__ Plan plan_of(int E, int k, const RouterArgs& o) {
  Plan p;
  p.bias = o.bias;
  p.row = nullptr;
  p.E = E; p.k = k; p.C = cdiv(E, 32);
  p.softmax = o.score == 0; p.top2 = o.group_top2;
  p.n_groups = o.n_groups; p.topk_groups = o.topk_groups;
  p.grouped = o.topk_groups < o.n_groups;
  p.scores = o.bias != nullptr || (p.grouped && o.group_top2);
  p.S = E / o.n_groups;
  p.L = p.S / p.C;
  if (p.S % p.C != 0 || (p.L & (p.L - 1)) != 0) p.L = 0;
  p.shift = p.L ? __ffs(p.L) - 1 : 0;
  return p;
}

// A warp's candidates, by id and by rank.
struct Pool {
  uint2 found[32], sorted[MAX_K + 1];
};

// An E-expert row over a warp: lane l holds experts l C .. l C + C - 1, C = ceil(E / 32).
// CM >= C is its compile-time bound; FULL: E = 32 CM.
template <int CM>
struct Row {
  float z[CM];
  uint32_t live, have;                            // bits over i: not masked, exists
};

template <int CM, bool FULL>
__device__ __forceinline__ void load_row(const float* __restrict__ p, int E, int C, int lane, Row<CM>& r) {
  const int e0 = lane * C;
  if constexpr (FULL && CM == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p + e0));
    r.z[0] = v.x; r.z[1] = v.y;
  } else if constexpr (FULL && CM >= 4) {
#pragma unroll
    for (int i = 0; i < CM / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + e0) + i);
      r.z[4 * i] = v.x; r.z[4 * i + 1] = v.y; r.z[4 * i + 2] = v.z; r.z[4 * i + 3] = v.w;
    }
  } else if (CM >= 4 && C == CM && (E & 3) == 0) {
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
template <int CM, bool FULL>
__device__ __forceinline__ void mask_row(int E, int C, int lane, Row<CM>& r) {
  r.live = 0;
  r.have = FULL ? (1u << CM) - 1u : (1u << max(0, min(C, E - lane * C))) - 1u;
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    const bool live = (FULL || (r.have >> i & 1u)) && r.z[i] >= -FLT_MAX;   // not NaN, not -infinity
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
// The same of z with -infinity for what is masked; never -infinity itself.
template <int CM>
__device__ __forceinline__ float top_of(const float (&z)[CM]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < CM; ++i) m = fmaxf(m, z[i]);
  return fmaxf(unordered(warp_max(ordered(m))), -FLT_MAX);
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

// The group limit: bit of each chosen group, from the lanes' values of their groups.
// `next`: the largest value left out.
template <typename U>
__device__ __forceinline__ uint32_t choose_groups(const Plan& o, int lane, U mine, U* last, U* next) {
  uint32_t chosen = 0;
  for (int j = 0; j < o.topk_groups; ++j) {
    *last = warp_max(mine);
    const int who = __ffs(__ballot_sync(0xffffffffu, mine == *last)) - 1;
    chosen |= 1u << (who >> o.shift);
    if (lane == who) mine = 0;
  }
  *next = warp_max(mine);
  return chosen;
}

// The two largest values seen, a >= b.
template <typename F>
struct Two {
  F a, b;
  __device__ __forceinline__ void add(F v) {
    const F low = a < v ? a : v;
    b = b > low ? b : low;
    a = a > v ? a : v;
  }
  __device__ __forceinline__ void join(F oa, F ob) {
    const F low = a < oa ? a : oa, side = b > ob ? b : ob;
    b = side > low ? side : low;
    a = a > oa ? a : oa;
  }
  // over aligned runs of L lanes
  __device__ __forceinline__ void join_lanes(int L) {
    for (int off = 1; off < L; off <<= 1) join(__shfl_xor_sync(0xffffffffu, a, off), __shfl_xor_sync(0xffffffffu, b, off));
  }
};

// The value of each group, as an ordered key in the lane that speaks for it (lane g << shift
// for group g), 0 elsewhere.  v: what the groups compare, of this lane's live experts.
template <typename U, typename F, int CM>
__device__ __forceinline__ U group_values(const Plan& o, int lane, const F (&v)[CM], uint32_t live, Two<F>* seen) {
  Two<F> t = {-INFINITY, -INFINITY};
  U mine = 0;
  if (o.L) {                                      // groups are aligned runs of L lanes
#pragma unroll
    for (int i = 0; i < CM; ++i) t.add((live >> i & 1u) ? v[i] : -INFINITY);
    t.join_lanes(o.L);
    *seen = t;
    if ((lane & (o.L - 1)) == 0 && (lane >> o.shift) < o.n_groups) mine = ordered(o.top2 && t.b != -INFINITY ? t.a + t.b : t.a);
    return mine;
  }
  for (int g = 0; g < o.n_groups; ++g) {
    t = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const int e = lane * o.C + i;
      if ((live >> i & 1u) && e >= g * o.S && e < g * o.S + o.S) t.add(v[i]);
    }
    t.join_lanes(32);
    if (lane == g) mine = ordered(o.top2 && t.b != -INFINITY ? t.a + t.b : t.a);
  }
  return mine;
}

template <typename U, int CM>
__device__ __forceinline__ void close_groups(const Plan& o, int lane, uint32_t chosen, U (&key)[CM]) {
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    const int g = o.L ? lane >> o.shift : min(31, (lane * o.C + i) / o.S);
    if (!(chosen >> g & 1u)) key[i] = 0;
  }
}

// One warp chooses one token's experts, every key and group value in 64 bits: lane
// `slot0 + j` gets slot j's id.  k rounds of a warp-wide largest.
template <int CM, bool FULL>
__device__ __noinline__ int choose_f64(const Plan o, int lane, int slot0, int my_e) {
  const int C = o.C;
  Row<CM> r;
  load_row<CM, FULL>(o.row, o.E, C, lane, r);
  mask_row<CM, FULL>(o.E, C, lane, r);
  double v[CM];
  if (!o.scores) {
#pragma unroll
    for (int i = 0; i < CM; ++i) v[i] = (double)r.z[i];
  } else if (o.softmax) {
    const double top = top_row<CM>(r);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      v[i] = (r.live >> i & 1u) ? exp((double)r.z[i] - top) : 0.0;
      sum += v[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < CM; ++i) v[i] /= sum > 0.0 ? sum : 1.0;
  } else {
#pragma unroll
    for (int i = 0; i < CM; ++i) v[i] = (r.live >> i & 1u) ? 1.0 / (1.0 + exp(-(double)r.z[i])) : 0.0;
  }
  uint64_t key[CM];
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    if (o.bias && (r.have >> i & 1u)) v[i] += (double)__ldg(o.bias + lane * C + i);
    const double w = o.bias ? v[i] : (double)r.z[i];
    key[i] = (r.live >> i & 1u) ? ordered(w) : (r.have >> i & 1u) ? 1ull : 0ull;
  }
  if (o.grouped) {
    uint64_t last, next;
    Two<double> seen;
    const uint32_t chosen = choose_groups(o, lane, group_values<uint64_t>(o, lane, v, r.live, &seen), &last, &next);
    close_groups(o, lane, chosen, key);
  }
  for (int j = 0; j < o.k; ++j) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < CM; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
    const uint64_t top = warp_max(best);
    // lanes hold ascending runs of experts: the lowest lane has the lowest id
    const int who = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    const int e = __shfl_sync(0xffffffffu, lane * C + at, who);
    if (lane == slot0 + j) my_e = e;
#pragma unroll
    for (int i = 0; i < CM; ++i)
      if (lane == who && i == at) key[i] = 0;
  }
  return my_e;
}

// One token's scores in 64 bits, for a few experts.
struct Exact {
  int softmax;
  double top, sum;
  __device__ __forceinline__ double score(float z) const {
    const double e = exp(softmax ? (double)z - top : -(double)z);
    return softmax ? e / sum : 1.0 / (1.0 + e);
  }
};
template <int CM, bool FULL>
__device__ __forceinline__ Exact exact_of(const float* __restrict__ row, int E, int softmax, int lane) {
  Exact x = {softmax, 0.0, 1.0};
  if (softmax) {
    const int C = cdiv(E, 32);
    Row<CM> r;
    load_row<CM, FULL>(row, E, C, lane, r);
    mask_row<CM, FULL>(E, C, lane, r);
    x.top = top_row<CM>(r);
    double sum = 0.0;
    for (int i = 0; i < CM; ++i)
      if (r.live >> i & 1u) sum += exp((double)r.z[i] - x.top);
    sum = warp_sum(sum);
    x.sum = sum > 0.0 ? sum : 1.0;
  }
  return x;
}

// The groups to choose from by their values in 64 bits.  todo: this lane's experts that may
// be among their group's largest.
template <int CM, bool FULL>
__device__ __noinline__ uint32_t groups_f64(const Plan o, const float* sbias, int lane, uint32_t todo) {
  const Exact x = exact_of<CM, FULL>(o.row, o.E, o.softmax, lane);
  Two<double> t = {-INFINITY, -INFINITY};
  while (__any_sync(0xffffffffu, todo != 0)) {
    const int e = lane * o.C + __ffs(todo) - 1;
    if (todo) t.add(x.score(fminf(__ldg(o.row + e), FLT_MAX)) + (o.bias ? (double)sbias[e] : 0.0));
    todo &= todo - 1;
    __syncwarp();
  }
  t.join_lanes(o.L);
  uint64_t last, next, mine = 0;
  if ((lane & (o.L - 1)) == 0 && (lane >> o.shift) < o.n_groups) mine = ordered(o.top2 && t.b != -INFINITY ? t.a + t.b : t.a);
  return choose_groups(o, lane, mine, &last, &next);
}

// A candidate's place among n by their keys in 64 bits; me: its 32-bit key and id.
template <int CM, bool FULL>
__device__ __noinline__ int rank_f64(const float* __restrict__ row, int E, int softmax, const float* sbias, int lane,
                                     int n, uint2 me) {
  const Exact x = exact_of<CM, FULL>(row, E, softmax, lane);
  uint64_t key = 0;
  if (lane < n) key = me.x <= MASKED ? 1ull : ordered(x.score(fminf(__ldg(row + me.y), FLT_MAX)) + (double)sbias[me.y]);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t other = __shfl_sync(0xffffffffu, key, j);
    rank += other > key || (other == key && j < lane);
  }
  return rank;
}

// The same in 32 bits, with every decision checked.  A key is within err = 2^-19 (softmax) or
// 2^-21 (sigmoid) + 2^-23 |key| of its 64-bit value: the scores are at most 1; a sigmoid has
// the errors of an exponential (2^-22 of it, where it moves the score by a quarter at the
// most), an addition (2^-24) and a reciprocal (2^-23), a softmax those and the 13 roundings
// of its sum; the bias adds half a step of the key.  Keys more than 2 err apart are in the
// right order; those that are not, and those only, are compared in 64 bits.  Without a bias
// the keys are the logits themselves, and exact.  False: too many ties for this way.
//
// The k largest are in the k lanes with the largest lane maxima, so they are not below the
// k-th largest maximum (if that many lanes have an open expert).  What reaches that (some
// 12 of 256 experts) goes to a lane each, in the order of ids, and finds its place by
// comparing itself with all the others.
template <int CM, bool FULL>
__device__ __forceinline__ bool choose_f32(const float (&z)[CM], const Plan& o, const float* sbias, float err, int lane,
                                           int slot0, Pool* pool, int* my_e) {
  const int C = FULL ? CM : o.C;
  float v[CM];                                    // p + bias, or the logits; -infinity: masked
  if (o.scores) {
    if (o.softmax) {
      const float top = top_of<CM>(z);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        v[i] = exp_fast(z[i] - top);
        sum += v[i];
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int i = 0; i < CM; ++i) v[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < CM; ++i) v[i] = rcp_fast(1.0f + exp_fast(-z[i]));
    }
    if (o.bias) {
      if constexpr (FULL && CM >= 4) {
#pragma unroll
        for (int i = 0; i < CM / 4; ++i) {
          const float4 b = reinterpret_cast<const float4*>(sbias + lane * CM)[i];
          v[4 * i] += b.x; v[4 * i + 1] += b.y; v[4 * i + 2] += b.z; v[4 * i + 3] += b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < CM; ++i)
          if (z[i] != -INFINITY) v[i] += sbias[lane * C + i];
      }
    }
#pragma unroll
    for (int i = 0; i < CM; ++i) v[i] = z[i] == -INFINITY ? -INFINITY : v[i];
  } else {
#pragma unroll
    for (int i = 0; i < CM; ++i) v[i] = z[i];
  }
  uint32_t key[CM];
#pragma unroll
  for (int i = 0; i < CM; ++i) {
    key[i] = ordered(o.bias ? v[i] : z[i]);
    if (!FULL && !(i < C && lane * C + i < o.E)) key[i] = 0;
  }
  if (o.grouped) {
    uint32_t last = 0, next = 0;
    Two<float> seen = {0.0f, 0.0f};
    uint32_t chosen = choose_groups(o, lane, group_values<uint32_t>(o, lane, v, ~0u, &seen), &last, &next);
    // a group's value has the errors of two keys and of their sum
    if (o.scores && next > MASKED && !(unordered(last) - unordered(next) > 6.0f * err)) {
      if (!o.L) return false;
      // in 64 bits: the experts that may be among their group's largest
      const float least = (o.top2 && seen.b != -INFINITY ? seen.b : seen.a) - 2.0f * err;
      uint32_t todo = 0;
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (v[i] != -INFINITY && !(v[i] < least)) todo |= 1u << i;
      chosen = groups_f64<CM, FULL>(o, sbias, lane, todo);
    }
    close_groups(o, lane, chosen, key);
  }
  const int want = o.k + (o.bias ? 1 : 0);        // with a bias the next one too, for its distance
  uint32_t best = 0, floor = 0;
#pragma unroll
  for (int i = 0; i < CM; ++i) best = max(best, key[i]);
  for (int j = 0; j < want; ++j) {
    floor = warp_max(best);
    if (best == floor) best = 0;                  // ties go at once: the floor is only lower for it
  }
  // no lanes left: every open expert may be needed; with a bias what is as good as the floor
  if (o.bias && floor > MASKED) floor = ordered(unordered(floor) - 2.0f * err);
  floor = max(floor, 1u);
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < CM; ++i) in |= key[i] >= floor ? 1u << i : 0u;
  // ids ascend from lane to lane: this lane's candidates stand behind the lower lanes'
  const int mine = __popc(in);
  const uint32_t below = (1u << lane) - 1u;
  int at = 0, n = 0;
#pragma unroll
  for (int b = 0; (1 << b) <= CM; ++b) {
    const uint32_t votes = __ballot_sync(0xffffffffu, mine >> b & 1);
    at += __popc(votes & below) << b;
    n += __popc(votes) << b;
  }
  if (n > 32) return false;
#pragma unroll
  for (int i = 0; i < CM; ++i)
    if (in >> i & 1u) pool->found[at++] = make_uint2(key[i], (uint32_t)(lane * C + i));
  __syncwarp();
  const uint2 me = lane < n ? pool->found[lane] : make_uint2(0u, 0u);
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint32_t other = pool->found[j].x;
    rank += other > me.x || (other == me.x && j < lane);
  }
  if (lane < n && rank < want) pool->sorted[rank] = me;
  __syncwarp();
  if (o.bias) {
    bool close = false;
    if (lane + 1 < min(want, n)) {
      const uint32_t a = pool->sorted[lane].x, b = pool->sorted[lane + 1].x;
      close = b > MASKED && !(unordered(a) - unordered(b) > 2.0f * err);
    }
    if (__any_sync(0xffffffffu, close)) {
      // in 64 bits: every candidate's key, and its place again
      rank = rank_f64<CM, FULL>(o.row, o.E, o.softmax, sbias, lane, n, me);
      if (lane < n && rank < want) pool->sorted[rank] = me;
      __syncwarp();
    }
  }
  if (lane >= slot0 && lane < slot0 + o.k) *my_e = (int)pool->sorted[lane - slot0].y;
  __syncwarp();
  return true;
}

// A warp routes RS_TOK tokens one after the other; then lane 8 q + j makes the gate of
// token q's slot j in 64 bits, one exponential for all of them.
template <int CM, bool FULL>
__global__ void __launch_bounds__(RS_WARPS * 32, 4)
route_scored_kernel(const float* __restrict__ logits, int T, int E, int k, const RouterArgs o,
                    int32_t* __restrict__ topk_idx, float* __restrict__ topk_gate,
                    int32_t* __restrict__ blk_hist, uint32_t* __restrict__ arrive,
                    uint32_t* __restrict__ ready_q) {
  pdl_trigger();
  pdl_wait();
  __shared__ int hist[MAX_E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = FULL ? CM : cdiv(E, 32);
  __shared__ __align__(16) float sbias[MAX_E];
  if (blk_hist || o.bias) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      hist[e] = 0;
      if (o.bias) sbias[e] = __ldg(o.bias + e);
    }
    __syncthreads();
  }
  __shared__ Pool pools[RS_WARPS];
  Pool* pool = &pools[warp];
  Plan plan = plan_of(E, k, o);
  float reach = 0.0f;                             // the largest |bias|: a key is no further out than that and 1
  if (o.bias) {
    for (int e = lane; e < E; e += 32) reach = fmaxf(reach, fabsf(sbias[e]));
    reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(reach)));
  }
  const float err = !plan.scores ? 0.0f : (plan.softmax ? 1.91e-6f : 4.77e-7f) + 1.2e-7f * (1.0f + reach);
  const int t0 = blockIdx.x * ROUTE_TOK + warp;   // its tokens: t0, t0 + 8, ..
  int my_e = 0;
  float my_top = 0.0f, my_sum = 1.0f;
#pragma unroll 1
  for (int q = 0; q < RS_TOK; ++q) {
    const int t = t0 + q * RS_WARPS;
    if (t >= T) break;
    Row<CM> r;
    load_row<CM, FULL>(logits + (size_t)t * E, E, C, lane, r);
    float z[CM];
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const bool have = FULL || (i < C && lane * C + i < E);
      z[i] = have && r.z[i] >= -FLT_MAX ? fminf(r.z[i], FLT_MAX) : -INFINITY;   // NaN and -infinity: masked
    }
    plan.row = logits + (size_t)t * E;
    if (!choose_f32<CM, FULL>(z, plan, sbias, err, lane, q * MAX_K, pool, &my_e))
      my_e = choose_f64<CM, FULL>(plan, lane, q * MAX_K, my_e);
    if (o.score == 0) {
      const float top = top_of<CM>(z);
      float sum = 1.0f;
      if (!o.renorm) {                            // else the sum cancels
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < CM; ++i) sum += expf(z[i] - top);
        sum = warp_sum(sum);
      }
      if (lane >> 3 == q) { my_top = top; my_sum = sum; }
    }
    if (lane == 0) {
      if (arrive) arrive[t] = 0u;
      if (ready_q) ready_q[t] = 0u;
    }
  }
  const int j = lane & 7, t = t0 + (lane >> 3) * RS_WARPS;
  const bool slot = j < k && t < T;
  if ((unsigned)my_e >= (unsigned)E) my_e = 0;    // a bias that is not finite can leave a slot open
  const float z = slot ? __ldg(logits + (size_t)t * E + my_e) : -INFINITY;
  const bool live = z >= -FLT_MAX;
  const double zd = (double)fminf(z, FLT_MAX);
  if (o.score == 0 && o.renorm) my_top = share_top(z, live, my_top);
  double w = 0.0;
  if (live) w = exp(o.score == 0 ? zd - (double)my_top : -zd);
  if (o.score != 0) w = live ? 1.0 / (1.0 + w) : 0.0;
  double total = sum8(w);                         // over the token's slots
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
//   softmax: dz_e = p_e (c_e - sum_j w_j c_j), c_e = 0 beside the chosen;
//   sigmoid: dz_e = c_e p_e (1 - p_e);
//   with renorm and the shares q_j = w_j / S: dz_e = q_e (c_e - sum_j q_j c_j), for the sigmoid
//   times 1 - p_e.  The softmax's own normaliser cancels, and dz is 0 beside the chosen.
// Shares, not scores over S^2: 1 / S overflows where the chosen scores are below 2^-1024.
// Where one expert has the whole sum the gradient is exactly 0.
// A warp takes 4 tokens: lane 8 q + j is token q's slot j, in 64 bits; then the warp
// writes the 4 rows, and the slots their experts' values over them.  `zero`: there is
// nothing beside the chosen.
template <int CM, bool FULL>
__global__ void __launch_bounds__(256)
route_scored_bwd_kernel(const float* __restrict__ dgate, const float* __restrict__ logits,
                        const int32_t* __restrict__ topk_idx, int T, int E, int k, const RouterArgs o,
                        float* __restrict__ dlogits) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = lane & 7, C = FULL ? CM : cdiv(E, 32);
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
  if (t0 >= T) return;
  const int t = t0 + (lane >> 3);
  const bool slot = j < k && t < T;
  int e = slot ? topk_idx[(size_t)t * k + j] : -1;
  if ((unsigned)e >= (unsigned)E) e = -1;
  const float dg = slot ? __ldg(dgate + (size_t)t * k + j) : 0.0f;   // on its way beside the chain of id and logit
  const float z = e >= 0 ? __ldg(logits + (size_t)t * E + e) : -INFINITY;
  const bool live = z >= -FLT_MAX;
  // a masked expert's gate is the constant 0: what its dgate holds, NaN or not, counts for nothing
  const double c = live ? (double)o.scale * (double)dg : 0.0;
  const double zd = (double)fminf(z, FLT_MAX);
  const bool zero = o.score != 0 || o.renorm;
  float my_top = 0.0f, my_sum = 1.0f;
  if (o.score == 0) {
#pragma unroll 1
    for (int q = 0; q < 4 && t0 + q < T; ++q) {
      Row<CM> r;
      load_row<CM, FULL>(logits + (size_t)(t0 + q) * E, E, C, lane, r);
      mask_row<CM, FULL>(E, C, lane, r);
      float ex[CM], top, sum;
      softmax_row<CM>(r, ex, &top, &sum);
      if (lane >> 3 == q) { my_top = top; my_sum = sum > 0.0f ? sum : 1.0f; }
    }
  }
  if (o.score == 0 && o.renorm) my_top = share_top(z, live, my_top);
  double w = 0.0;
  if (live) w = exp(o.score == 0 ? zd - (double)my_top : -zd);
  double rest = 1.0;                              // sigmoid: 1 - p, from the exponential where p is near 1
  if (o.score == 0) {
    w /= (double)my_sum;
  } else {
    const double x = w;
    w = live ? 1.0 / (1.0 + x) : 0.0;
    rest = w < 0.5 ? 1.0 - w : x * w;
  }
  double share = w, dot = 0.0;
  if (o.score == 0 || o.renorm) dot = sum8(c * w);
  if (o.renorm) {
    const double S = sum8(w);
    dot = S > 0.0 ? dot / S : 0.0;
    share = w < S ? w / S : 0.0;                  // w = S: the share is 1, the difference 0
  }
  const float dz = live ? (float)(share * (c - dot) * rest) : 0.0f;
  if (zero) {
    // 4 rows of zeros in one run
    const int rows = min(4, T - t0), n = rows * E;
    float* out = dlogits + (size_t)t0 * E;
    if ((E & 3) == 0) {
      for (int i = lane * 4; i < n; i += 128) *reinterpret_cast<float4*>(out + i) = make_float4(0, 0, 0, 0);
    } else {
      for (int i = lane; i < n; i += 32) out[i] = 0.0f;
    }
  } else {
#pragma unroll 1
    for (int q = 0; q < 4 && t0 + q < T; ++q) {
      float v[CM] = {};
      const float top = __shfl_sync(0xffffffffu, my_top, q * 8);
      const float by = (float)-__shfl_sync(0xffffffffu, dot / (double)my_sum, q * 8);
      Row<CM> r;
      load_row<CM, FULL>(logits + (size_t)(t0 + q) * E, E, C, lane, r);
      mask_row<CM, FULL>(E, C, lane, r);
#pragma unroll
      for (int i = 0; i < CM; ++i)
        if (r.live >> i & 1u) v[i] = expf(r.z[i] - top) * by;
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
  __syncwarp();                                   // the chosen experts' own values come after
  if (e >= 0) dlogits[(size_t)t * E + e] = dz;
}

}  // namespace

template <template <int, bool> class K, typename... Args>
cudaError_t launch_rows(int E, int grid, cudaStream_t s, Args... args) {
  const bool full = E == 32 || E == 64 || E == 128 || E == 256;
  auto kernel = E <= 32 ? (full ? K<1, true>::at : K<1, false>::at)
                : E <= 64 ? (full ? K<2, true>::at : K<2, false>::at)
                : E <= 128 ? (full ? K<4, true>::at : K<4, false>::at)
                           : (full ? K<8, true>::at : K<8, false>::at);
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(256), 0, s, args...);
}
template <int CM, bool FULL> struct Forward { static constexpr auto at = route_scored_kernel<CM, FULL>; };
template <int CM, bool FULL> struct Backward { static constexpr auto at = route_scored_bwd_kernel<CM, FULL>; };

cudaError_t launch_route_scored(const float* logits, int T, int E, int k, const RouterArgs& r,
                                int32_t* topk_idx, float* topk_gate, int32_t* blk_hist,
                                uint32_t* arrive, uint32_t* ready_q, cudaStream_t s) {
  return launch_rows<Forward>(E, route_blocks(T), s, logits, T, E, k, r, topk_idx, topk_gate, blk_hist, arrive, ready_q);
}

cudaError_t launch_route_scored_bwd(const float* dgate, const float* logits, const int32_t* topk_idx,
                                    int T, int E, int k, const RouterArgs& r, float* dlogits,
                                    cudaStream_t s) {
  return launch_rows<Backward>(E, cdiv(T, 32), s, dgate, logits, topk_idx, T, E, k, r, dlogits);
}

}  // namespace moe
