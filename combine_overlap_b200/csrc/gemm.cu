// gemm.cu -- the linear layer's products on the 5th-generation tensor cores: TMA tiles
// into a ring of shared-memory stages, tcgen05 MMAs (bf16, fp32 accumulators in TMEM)
// issued by one warp (a lane of it elected), and an epilogue (bias, activation, residual,
// one rounding) that runs beside the next tile's main loop: two accumulators of up to 256
// columns.
//
// Tiles and splits:
//   CG = 1  a CTA per 128 x BN tile;
//   CG = 2  a pair of CTAs per 256 x BN tile (cta_group::2): each loads its own 128 rows
//           of A and half of B's columns, so a stage's bytes per FLOP are a third less;
//   S > 1   the reduction is cut over a cluster of S tiles' CTAs: each leaves its fp32
//           tile in its shared memory, and CTA s finishes rows [s 128/S, (s+1) 128/S) by
//           adding the S tiles through distributed shared memory in order 0 .. S-1 -- no
//           workspace, no atomics, the same bits every time;
//   SW > 1  the reduction is cut over SW tiles' CTAs that need not run together: each
//           leaves its fp32 tile in the workspace, and join_kernel adds the slices in
//           order.  For the weight's gradient, whose tiles are few and reductions long.
//
// The tensor cores truncate as they add a product to an accumulator, so a sum's error
// grows with the number of MMAs in its chain: by at most a step, 2^-23, of sum|a b| per MMA.
// Sums therefore leave the accumulator every `chunk` k-blocks and are summed on in registers,
// rounded to nearest (PROMO): every CHAIN_F32 for outputs in fp32; the lower terms of B have
// accumulator columns of their own, so that they add nothing to the chain of the highest.
// bf16 outputs, whose last rounding is far larger, do it every CHAIN_BF16, and up to that
// length run in kernels without the sums.
#include "gemm.cuh"

#include <limits.h>
#include <string.h>

namespace moe {

namespace {

constexpr int G_THREADS = 320;            // warp 0 TMA, warp 1 MMA, warps 2-9 epilogue
constexpr int G_EPI = 8;
constexpr int G_MAX_NST = 12;
constexpr int A_BYTES = 16384;            // a CTA's A tile of a k-block: 128 rows x 64 bf16
constexpr int LOW_COLS = 128;             // where an accumulator keeps the lower terms' products
constexpr int G_RING = 196608;            // bytes of the operand ring
constexpr int G_STAGING = G_EPI * 4096;   // per epilogue warp: 32 rows x 32 fp32 columns
constexpr int CHAIN_F32 = 8;              // k-blocks of 4 MMAs: within 32 2^-23 = 2^-18 of sum|a b|
constexpr int CHAIN_BF16 = 256;           // within 1024 2^-23 = 2^-13: a 32nd of bf16's last rounding
constexpr double G_FILL = 50.0;           // see cost()
constexpr uint64_t G_TIMEOUT = 2000000000ull;   // ns; moe_linear_debug_set may set another

struct GemmCtl {
  uint64_t full[G_MAX_NST], empty[G_MAX_NST];   // full: counted on the pair's leader
  uint64_t tfull[2], tempty[2];                 // tempty: counted on the pair's leader
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t abort;                         // a bounded wait of this CTA ran out
  uint64_t limit;                         // ns that a wait may take
  alignas(16) float bias[G_EPI][32];                  // of each epilogue warp's chunk
};

constexpr size_t G_SMEM = 1024 + (size_t)G_RING + G_STAGING + sizeof(GemmCtl);
static_assert(G_SMEM <= 227 * 1024, "over the 227 KB per-CTA limit");

// How many CTAs of products have given up a bounded wait so far.
__device__ uint32_t g_linear_timeouts;

struct GemmArgs {
  int M, N, K;
  int tiles_m, tiles_n;
  int BN;                                 // columns per tile, a multiple of 16, <= 256
  int S, SW;                              // split of the reduction: in a cluster, in slices
  int PA, PB;                             // planes
  int nst, stage_bytes;                   // ring
  int kps;                                // k-blocks of 64 per stage; 1 with two planes of A
  int b_bytes;                            // a stage's bytes of one plane of one CTA's B tile
  int b_boxes;                            // B, n contiguous: 64-column atoms per CTA and plane
  int a_whole, b_whole;                   // one copy brings all of a stage's A (B)
  int chunk;                              // k-blocks per accumulator chain, a multiple of kps
  int group;                              // row tiles per raster group
  int tma_out, tma_pre;                   // rows of 16-byte multiples: chunks leave by TMA
  int withhold;                           // debug: block 0 brings no operands
  uint64_t limit;                         // ns that a wait may take
  LinearEpi ep;
};

// A value to be kept in a register.  Left alone, the compiler reads kernel arguments from
// constant memory where they are used, in every turn of a loop: some 50 cycles each for a
// warp with nothing else to issue, 500 in a k-block of the MMA issuer.
__device__ __forceinline__ int keep(int v) { asm volatile("" : "+r"(v)); return v; }
template <typename T>
__device__ __forceinline__ T* keep(T* p) { asm volatile("" : "+l"(p)); return p; }

// A load that stays where it stands: others sink to their first use, behind the main loop.
__device__ __forceinline__ float ld_here(const float* p) {
  float v;
  asm volatile("ld.volatile.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// A converged warp waits, and leaves with one answer.  The clock is read only once a wait
// has spun for a while: reading it costs as much as half a k-block's MMAs.
template <int CG>
__device__ __forceinline__ bool g_wait(uint64_t* bar, uint32_t parity, GemmCtl* ctl) {
  volatile uint32_t* ab = &ctl->abort;
  uint64_t deadline = 0;
  for (uint32_t n = 0;;) {
    const bool ready = CG == 2 ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ready)) return true;
    if ((++n & 1023u) != 0) continue;
    const uint64_t now = globaltimer();
    if (deadline == 0) deadline = now + *const_cast<volatile uint64_t*>(&ctl->limit);
    if (__any_sync(0xffffffffu, *ab != 0 || now > deadline)) {
      if (atomicExch(const_cast<uint32_t*>(ab), 1u) == 0) atomicAdd(&g_linear_timeouts, 1u);
      return false;
    }
  }
}

// True in one lane of a converged warp.  The producer and the MMA issuer run as whole
// warps with one lane elected for the copies and MMAs: descriptors and addresses then stay
// in uniform registers.  One thread alone took 690 cycles of issue per k-block of four MMAs
// (512 cycles of tensor work at BN = 256).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const void* tmap, uint32_t bar_cluster, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      :: "r"(smem_u32(dst)), "l"(tmap), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, uint32_t on) {
  if (CG == 2) tc_mma_f16_pair(d, x, y, idesc, on);
  else tc_mma_f16(d, x, y, idesc, on);
}

// Tile t of the raster: groups of `group` row tiles, within a group column by column,
// so a wave of CTAs shares few row tiles and few column tiles.
__device__ __forceinline__ void tile_at(const GemmArgs& a, int t, int* tm, int* tn) {
  const int per = a.group * a.tiles_n;
  const int g = t / per, r = t - g * per;
  const int rows = min(a.group, a.tiles_m - g * a.group);
  *tn = r / rows;
  *tm = g * a.group + (r - *tn * rows);
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
         "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
         "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
         "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------- epilogue chunk ---
// One warp's 32 rows x 32 columns: lane l holds row l.  Rows leave through the warp's 4 KB of
// shared memory, its 16-byte units XORed with the row as a TMA store of that box expects
// them (64-byte swizzle for bf16 rows, 128-byte for fp32), free of bank conflicts.
__device__ __forceinline__ int at16(int row, int u) { return row * 4 + (u ^ (row >> 1 & 3)); }
__device__ __forceinline__ int at32(int row, int u) { return row * 8 + (u ^ (row & 7)); }

__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
               :: "l"(tmap), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// What an epilogue warp knows of the output, in registers.
struct Epilogue {
  const float* bias;
  const void* residual;
  void *out, *pre;
  const CUtensorMap *tm_out, *tm_pre;     // null: rows that are no multiple of 16 bytes
  int act, f32;
  int M, N, lane;
  uint8_t* st;
  float* cols;                            // 32 floats of the warp: the chunk's bias
  int turn;                               // which half of st a bf16 chunk takes next
  int part;                               // slice of the reduction (SW > 1), or 0
};

// v as bf16 -> dst[row0 + lane][col ..], columns < cend
__device__ __forceinline__ void emit16(Epilogue& e, const float (&v)[32], const CUtensorMap* tm, void* dst, int row0,
                                       int col, int cend) {
  uint4* st = reinterpret_cast<uint4*>(e.st + e.turn * 2048);
  e.turn ^= 1;
  if (e.lane == 0) {
    if (e.f32) bulk_wait_read<0>();       // an fp32 chunk takes all of st
    else bulk_wait_read<1>();             // the other half's copy may still be under way
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    st[at16(e.lane, u)] = make_uint4(pack2(v[8 * u], v[8 * u + 1]), pack2(v[8 * u + 2], v[8 * u + 3]),
                                     pack2(v[8 * u + 4], v[8 * u + 5]), pack2(v[8 * u + 6], v[8 * u + 7]));
  if (tm) {
    fence_proxy_async_shared();
    __syncwarp();
    if (e.lane == 0) tma_store_3d(tm, st, col, row0, 0);
    return;
  }
  __syncwarp();
  const int c = e.lane & 15, n = cend - col - 2 * c;   // columns left from the lane's pair on
  const bool even = (e.N & 1) == 0;
#pragma unroll 8
  for (int i = 0; i < 16; ++i) {
    const int r = i * 2 + (e.lane >> 4);
    const uint32_t x = reinterpret_cast<const uint32_t*>(st + at16(r, c >> 2))[c & 3];
    unsigned short* o = static_cast<unsigned short*>(dst) + (size_t)(row0 + r) * e.N + col + 2 * c;
    if (row0 + r >= e.M || n <= 0) continue;
    if (even) {
      *reinterpret_cast<uint32_t*>(o) = x;
    } else {
      o[0] = (unsigned short)x;
      if (n > 1) o[1] = (unsigned short)(x >> 16);
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void emit32(Epilogue& e, const float (&v)[32], int row0, int col, int cend) {
  float4* st = reinterpret_cast<float4*>(e.st);
  if (e.lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 8; ++u) st[at32(e.lane, u)] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
  if (e.tm_out) {
    fence_proxy_async_shared();
    __syncwarp();
    if (e.lane == 0) tma_store_3d(e.tm_out, st, col, row0, e.part);
    return;
  }
  __syncwarp();
  const bool mine = col + e.lane < cend;
  float* o = static_cast<float*>(e.out) + (size_t)row0 * e.N + col + e.lane;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    const float x = reinterpret_cast<const float*>(st + at32(r, e.lane >> 2))[e.lane & 3];
    if (mine && row0 + r < e.M) o[(size_t)r * e.N] = x;
  }
  __syncwarp();
}

// A lane's 32 columns of the residual (its own row).
__device__ __forceinline__ void residual32(const Epilogue& e, int row, int col, int cend, float (&v)[32]) {
  if (row >= e.M) return;
  const size_t at = (size_t)row * e.N + col;
  if (e.f32) {
    const float* r = static_cast<const float*>(e.residual) + at;
    if (e.tm_out && col + 32 <= cend) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = reinterpret_cast<const float4*>(r)[i];
        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = col + i < cend ? r[i] : 0.0f;
    }
    return;
  }
  const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(e.residual) + at;
  if (e.tm_out && col + 32 <= cend) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(r)[i];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else if ((e.N & 1) == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t w = col + 2 * i < cend ? reinterpret_cast<const uint32_t*>(r)[i] : 0u;
      v[2 * i] = __uint_as_float(w << 16);
      v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = col + i < cend ? __bfloat162float(r[i]) : 0.0f;
  }
}

// tacc: the chunk's columns in TMEM; b: this lane's bias (column col + lane)
__device__ __forceinline__ void finish_chunk(Epilogue& e, uint32_t tacc, float b, int row0, int col, int cend) {
  float res[32];
  if (e.residual) residual32(e, row0 + e.lane, col, cend, res);
  uint32_t r[32];
  tmem_ld32(tacc, r);
  tmem_ld_wait();
  float v[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
  if (e.bias) {
    e.cols[e.lane] = b;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 c = reinterpret_cast<const float4*>(e.cols)[j];
      v[4 * j] += c.x; v[4 * j + 1] += c.y; v[4 * j + 2] += c.z; v[4 * j + 3] += c.w;
    }
    __syncwarp();
  }
  if (e.pre) emit16(e, v, e.tm_pre, e.pre, row0, col, cend);
  if (e.act == 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_f32(1, v[i], e.f32);
  } else if (e.act == 2) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_f32(2, v[i], e.f32);
  } else if (e.act == 3) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_f32(3, v[i], e.f32);
  }
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += res[i];
  }
  if (e.f32) emit32(e, v, row0, col, cend);
  else emit16(e, v, e.tm_out, e.out, row0, col, cend);
}

// Four outputs of row m from column n on, in a thread of their own.
__device__ __forceinline__ void finish4(const Epilogue& e, int m, int n, float4 v) {
  const size_t at = (size_t)m * e.N + n;
  float u[4] = {v.x, v.y, v.z, v.w};
  const bool vec = (e.N & 3) == 0;
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < e.N) u[i] += __ldg(e.bias + n + i);
  }
  if (e.pre) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(e.pre) + at;
    if (vec) *reinterpret_cast<uint2*>(p) = make_uint2(pack2(u[0], u[1]), pack2(u[2], u[3]));
    else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < e.N) p[i] = __float2bfloat16(u[i]);
    }
  }
  if (e.act) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = act_f32(e.act, u[i], e.f32);
  }
  if (e.f32) {
    float* o = static_cast<float*>(e.out) + at;
    const float* r = static_cast<const float*>(e.residual) + (e.residual ? at : 0);
    if (vec) {
      if (e.residual) {
        const float4 x = *reinterpret_cast<const float4*>(r);
        u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
      }
      *reinterpret_cast<float4*>(o) = make_float4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < e.N) o[i] = u[i] + (e.residual ? r[i] : 0.0f);
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + at;
    const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(e.residual) + (e.residual ? at : 0);
    if (vec) {
      if (e.residual) {
        const uint2 x = *reinterpret_cast<const uint2*>(r);
        u[0] += __uint_as_float(x.x << 16); u[1] += __uint_as_float(x.x & 0xffff0000u);
        u[2] += __uint_as_float(x.y << 16); u[3] += __uint_as_float(x.y & 0xffff0000u);
      }
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2(u[0], u[1]), pack2(u[2], u[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < e.N) o[i] = __float2bfloat16(u[i] + (e.residual ? __bfloat162float(r[i]) : 0.0f));
    }
  }
}

// The S partial tiles of one output tile, through distributed shared memory in order
// 0 .. S-1: U vectors at a time, all S U loads in flight.  base: the tile in this CTA;
// rows [row, row + 128 / S) of it, which start at m0 of the output.
template <int S, int U>
__device__ __forceinline__ void join_tiles(const Epilogue& e, uint32_t base, int BN, int m0, int n0, int row, int cg,
                                           int rank) {
  const int rows = min(128 / S, e.M - m0);
  const int per = BN / 4, pitch = (per + 1) * 16;
  uint32_t from[S];
#pragma unroll
  for (int s = 0; s < S; ++s) from[s] = mapa_shared(base + (uint32_t)(row * pitch), (uint32_t)(s * cg + rank));
  int r = threadIdx.x / per, c = threadIdx.x - r * per;
  const int dr = G_THREADS / per, dc = G_THREADS - dr * per;
  while (r < rows) {
    float4 w[U][S];
    int rr[U], cc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rr[u] = r; cc[u] = c;
      const uint32_t at = (uint32_t)(min(r, rows - 1) * pitch + c * 16);
#pragma unroll
      for (int s = 0; s < S; ++s) w[u][s] = ld_cluster_v4(from[s] + at);
      r += dr; c += dc;
      if (c >= per) { c -= per; ++r; }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = m0 + rr[u], n = n0 + cc[u] * 4;
      if (rr[u] >= rows || m >= e.M || n >= e.N) continue;
      float4 v = w[u][0];
#pragma unroll
      for (int s = 1; s < S; ++s) { v.x += w[u][s].x; v.y += w[u][s].y; v.z += w[u][s].z; v.w += w[u][s].w; }
      finish4(e, m, n, v);
    }
  }
}

template <bool F32>
__device__ __forceinline__ Epilogue load_epilogue(const GemmArgs& a, const CUtensorMap& tm_out, const CUtensorMap& tm_pre,
                                                  int lane, uint8_t* st, float* cols) {
  Epilogue e;
  e.bias = keep(a.ep.bias);
  e.residual = keep(a.ep.residual);
  e.out = keep(a.ep.out);
  e.pre = keep(a.ep.pre);
  e.tm_out = keep(a.tma_out ? &tm_out : nullptr);
  e.tm_pre = keep(a.tma_pre ? &tm_pre : nullptr);
  e.act = keep(a.ep.act);
  e.f32 = F32;
  e.M = keep(a.M);
  e.N = keep(a.N);
  e.lane = lane;
  e.st = st;
  e.cols = cols;
  e.turn = e.part = 0;
  return e;
}

// The i-th 32-column chunk of an epilogue warp: the two warps of a lane quadrant take
// alternate pairs of chunks, so one warp writes a whole 128-byte line of bf16.
__device__ __forceinline__ int chunk_of(int half, int i) { return ((i >> 1) * 2 + half) * 2 + (i & 1); }

// PROMO: chunks per epilogue warp whose sums are kept in registers (2 for BN <= 128: with 4
// the sums leave too few registers, and the epilogue's own spill), or 0.  F32: the tiles leave
// in fp32, as outputs or slices.
template <int CG, bool AMN, bool BMN, int PROMO, bool F32>
__global__ void __launch_bounds__(G_THREADS, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
            const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_pre,
            const GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* staging = smem + G_RING;
  GemmCtl* ctl = reinterpret_cast<GemmCtl*>(staging + G_STAGING);
  pdl_trigger();
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = a.S;
  const bool cluster = CG * S > 1;
  const int crank = cluster ? (int)cluster_ctarank() : 0;
  const int rank = CG == 2 ? crank & 1 : 0;          // in the pair
  const int lead = crank - rank;                     // the pair's leader
  const int split = crank / CG;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.nst; ++i) { mbar_init(&ctl->full[i], 1); mbar_init(&ctl->empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&ctl->tfull[i], 1); mbar_init(&ctl->tempty[i], G_EPI * CG); }
    mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    ctl->limit = a.limit;
    mbar_fence_init();
    fence_proxy_async_shared();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    if (a.tma_out) tma_prefetch_desc(&tm_out);
  }
  if (warp == 1) {
    if (CG == 2) tmem_alloc_pair(&ctl->tmem_base, TMEM_COLS);
    else tmem_alloc(&ctl->tmem_base, TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  if (CG == 2) cluster_sync();            // both CTAs' barriers stand before a remote arrival
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_wait();

  const int nkb = cdiv(a.K, 64);
  const int t0 = blockIdx.x / (S * CG), tstep = gridDim.x / (S * CG);
  const int ntiles = a.tiles_m * a.tiles_n, units = ntiles * a.SW;
  // unit t: tile t % ntiles, slice t / ntiles; its k-blocks: as even as can be
  const int parts = S * a.SW;
  auto slice = [&](int t, int* tm, int* tn, int* kb0, int* kb1) {
    const int z = a.SW > 1 ? t / ntiles : 0, part = S > 1 ? split : z;
    tile_at(a, t - z * ntiles, tm, tn);
    *kb0 = (int)((long long)nkb * part / parts);
    *kb1 = (int)((long long)nkb * (part + 1) / parts);
    return z;
  };

  if (warp == 0) {
    int stage = 0;
    uint32_t ph = 0;
    bool ok = !(a.withhold && blockIdx.x == 0);
    const int kps = keep(a.kps), nst = keep(a.nst), PB = keep(a.PB), boxes = keep(a.b_boxes);
    const int b_bytes = keep(a.b_bytes), stage_bytes = keep(a.stage_bytes);
    const int a_whole = keep(a.a_whole), b_whole = keep(a.b_whole), PA = keep(a.PA);
    uint8_t* const ring = keep(smem);
    const CUtensorMap *ma = keep(&tm_a), *mb = keep(&tm_b);
    for (int t = t0; t < units && ok; t += tstep) {
      int tm, tn, kb0, kb1;
      slice(t, &tm, &tn, &kb0, &kb1);
      const int m0 = tm * (128 * CG) + rank * 128, n0 = tn * a.BN + rank * (a.BN / CG);
      for (int kb = kb0; kb < kb1; kb += kps) {
        if (!g_wait<CG>(&ctl->empty[stage], ph ^ 1u, ctl)) { ok = false; break; }
        if (elect_one()) {
          uint64_t* fb = &ctl->full[stage];
          const uint32_t fbl = CG == 2 ? mapa_shared(smem_u32(fb), (uint32_t)lead) : 0u;
          if (rank == 0) mbar_arrive_expect_tx(fb, (uint32_t)(CG * stage_bytes));
          auto load = [&](void* d, const CUtensorMap* m, int x, int y, int z, int p) {
            if (CG == 2) tma_load_4d_pair(d, m, fbl, x, y, z, p);
            else tma_load_4d(d, m, fb, x, y, z, p);
          };
          uint8_t* d = ring + stage * stage_bytes;
          const int k = kb * 64;
          if constexpr (AMN) {
            if (a_whole) {
              load(d, ma, 0, k, m0 >> 6, 0);
            } else {
              load(d, ma, m0, k, 0, 0);
              load(d + kps * 8192, ma, m0 + 64, k, 0, 0);
            }
          } else {
            if (a_whole) load(d, ma, 0, m0, kb, 0);
            else if (PA > 1)
              for (int p = 0; p < PA; ++p) load(d + p * A_BYTES, ma, k, m0, 0, p);
            else
              for (int i = 0; i < kps; ++i) load(d + i * A_BYTES, ma, k + i * 64, m0, 0, 0);
          }
          d += kps * PA * A_BYTES;
          if constexpr (BMN) {
            if (b_whole) load(d, mb, 0, k, n0 >> 6, 0);
            else
              for (int p = 0; p < PB; ++p)
                for (int j = 0; j < boxes; ++j, d += kps * 8192) load(d, mb, n0 + j * 64, k, 0, p);
          } else {
            if (b_whole) load(d, mb, 0, n0, kb, 0);
            else
              for (int i = 0, step = b_bytes / kps; i < kps; ++i, d += step) load(d, mb, k + i * 64, n0, 0, 0);
          }
        }
        __syncwarp();
        if (++stage == nst) { stage = 0; ph ^= 1u; }
      }
    }
    if (!ok) {
      // copies may still be landing: a bounded wait until every stage's are in (a pair's
      // second CTA, whose copies are counted on the leader, waits a fixed time)
      const uint64_t until = globaltimer() + (rank == 0 ? a.limit : 1000000ull);
      for (int i = 0; i < a.nst; ++i)
        for (uint32_t par = 0; par < 2; ++par)
          while ((rank || !mbar_try_wait(&ctl->full[i], par)) && globaltimer() < until) {}
    }
  } else if (warp == 1 && rank == 0) {
    const uint32_t idesc = (uint32_t)keep((int)(idesc_bf16_f32(128 * CG, a.BN, BMN) | (AMN ? 1u << 15 : 0u)));
    const uint16_t mask = (uint16_t)(3u << lead);
    auto commit = [&](uint64_t* bar) {
      if (CG == 2) tc_commit_pair(bar, mask);
      else tc_commit(bar);
    };
    const int kps = keep(a.kps), nst = keep(a.nst), PB = keep(a.PB), chunk = keep(a.chunk);
    // two planes of A are multiplied as two k-blocks of one B, the last k-block whole (TMA's zeros)
    const int PA = keep(a.PA), K = keep(PA > 1 ? INT_MAX : a.K);
    // Descriptors of the first stage.  16 of k further on: 32 bytes in a K-major row, 16 rows
    // of 128 bytes otherwise; the next k-block: the next tile, or 64 rows (the address field
    // is in units of 16 bytes)
    constexpr uint64_t KA = AMN ? 128 : 2, KB = BMN ? 128 : 2;
    const uint64_t ad0 = smem_desc_sw128(smem_u32(smem), AMN ? kps * 8192 : 16, 1024);
    const uint64_t bd0 = smem_desc_sw128(smem_u32(smem) + kps * PA * A_BYTES, BMN ? kps * 8192 : 16, 1024);
    const int stage16 = keep(a.stage_bytes >> 4), b16 = keep(a.b_bytes >> 4);
    const int xkb = AMN ? 512 : A_BYTES >> 4, ykb = keep(BMN ? 512 : PA > 1 ? 0 : (a.b_bytes / a.kps) >> 4);
    int stage = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (int t = t0; t < units && ok; t += tstep) {
      int tm, tn, kb0, kb1;
      slice(t, &tm, &tn, &kb0, &kb1);
      for (int kb = kb0, in = 0; kb < kb1; kb += kps) {
        if (in == 0 && !g_wait<CG>(&ctl->tempty[acc], aph ^ 1u, ctl)) { ok = false; break; }
        if (!g_wait<CG>(&ctl->full[stage], ph, ctl)) { ok = false; break; }
        tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)(acc * ACC_COLS);
        const int n = PA > 1 ? PA : min(kps, kb1 - kb);
        const uint32_t more = in ? 1u : 0u;
        in += kps;
        const bool end = in == chunk || kb + kps >= kb1;
        if (elect_one()) {
          uint64_t x = ad0 + (uint64_t)(stage * stage16), y = bd0 + (uint64_t)(stage * stage16);
          if (K - kb * 64 <= n * 64 - 16) {
            // the last k-block, not all of it there
            for (int i = 0; i < n; ++i, x += xkb, y += ykb) {
              const int ks = min(4, cdiv(K - (kb + i) * 64, 16));
              for (int pb = 0; pb < PB; ++pb)
                for (int k = 0; k < ks; ++k)
                  mma<CG>(dt + (pb ? LOW_COLS : 0), x + k * KA, y + pb * b16 + k * KB, idesc, i || pb > 1 || k ? 1u : more);
            }
          } else if (PB == 1) {
            mma<CG>(dt, x, y, idesc, more);
#pragma unroll
            for (int k = 1; k < 4; ++k) mma<CG>(dt, x + k * KA, y + k * KB, idesc, 1u);
            for (int i = 1; i < n; ++i) {
              x += xkb;
              y += ykb;
#pragma unroll
              for (int k = 0; k < 4; ++k) mma<CG>(dt, x + k * KA, y + k * KB, idesc, 1u);
            }
          } else {
            for (int i = 0; i < n; ++i, x += xkb, y += ykb)
              for (int pb = 0; pb < PB; ++pb) {
                const uint64_t z = y + (uint64_t)(pb * b16);
                const uint32_t dp = dt + (pb ? LOW_COLS : 0);
                mma<CG>(dp, x, z, idesc, i || pb > 1 ? 1u : more);
#pragma unroll
                for (int k = 1; k < 4; ++k) mma<CG>(dp, x + k * KA, z + k * KB, idesc, 1u);
              }
          }
          commit(&ctl->empty[stage]);
          if (end) commit(&ctl->tfull[acc]);
        }
        __syncwarp();
        if (++stage == nst) { stage = 0; ph ^= 1u; }
        if (end) {
          in = 0;
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
    }
    // every MMA is done before TMEM is released
    if (elect_one()) {
      if (CG == 2) tc_commit_pair(&ctl->mma_done, (uint16_t)(1u << lead));
      else tc_commit(&ctl->mma_done);
    }
    __syncwarp();
    g_wait<CG>(&ctl->mma_done, 0u, ctl);
  } else if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q ..
    int acc = 0;
    uint32_t aph = 0;
    Epilogue ep = load_epilogue<F32>(a, tm_out, tm_pre, lane, staging + (warp - 2) * 4096, ctl->bias[warp - 2]);
    const int BN = keep(a.BN);
    const bool low = a.PB > 1;
    bool ok = true;
    auto release = [&](int i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || rank == 0) mbar_arrive(&ctl->tempty[i]);
        else mbar_arrive_remote(mapa_shared(smem_u32(&ctl->tempty[i]), (uint32_t)lead));
      }
    };
    for (int t = t0; t < units && ok; t += tstep) {
      int tm, tn, kb0, kb1;
      ep.part = slice(t, &tm, &tn, &kb0, &kb1);
      const int row0 = tm * (128 * CG) + rank * 128 + q * 32, n0 = tn * a.BN;
      const int cend = min(a.N, n0 + a.BN), nch = cdiv(kb1 - kb0, a.chunk);
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
      const bool mine = row0 < ep.M;
      float b[4] = {};                    // lane's bias of each chunk, read while the main loop runs
      if (ep.bias && S == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = chunk_of(half, i) * 32 + lane;
          if (c < BN && n0 + c < ep.N) b[i] = ld_here(ep.bias + n0 + c);
        }
      }
      float sum[PROMO ? PROMO : 1][32];
      // sum (+)= this warp's chunks of the accumulator at `tb`
      auto promote = [&](uint32_t tb, bool first) {
#pragma unroll
        for (int i = 0; i < PROMO; ++i) {
          const int ch = chunk_of(half, i);
          if (ch * 32 < BN) {
            uint32_t r[32];
            tmem_ld32(tb + ch * 32, r);
            tmem_ld_wait();
            if (first) {
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[i][j] = __uint_as_float(r[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(r[j]);
            }
          }
        }
        if (low) {                        // BN <= 128
#pragma unroll
          for (int i = 0; i < min(PROMO, 2); ++i) {
            const int ch = chunk_of(half, i);
            if (ch * 32 < BN) {
              uint32_t r[32];
              tmem_ld32(tb + LOW_COLS + ch * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(r[j]);
            }
          }
        }
      };
      if constexpr (PROMO != 0) {
        for (int c = 0; c + 1 < nch && ok; ++c) {
          if (!g_wait<CG>(&ctl->tfull[acc], aph, ctl)) { ok = false; break; }
          tc_fence_after();
          promote(lanes + (uint32_t)(acc * ACC_COLS), c == 0);
          release(acc);
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
      if (!ok || !g_wait<CG>(&ctl->tfull[acc], aph, ctl)) { ok = false; break; }
      tc_fence_after();
      const uint32_t tb = lanes + (uint32_t)(acc * ACC_COLS);
      if constexpr (PROMO != 0) {
        if (nch > 1 || low) {
          // the last chain joins the sums, and the sums go where the code below reads
          promote(tb, nch == 1);
#pragma unroll
          for (int i = 0; i < PROMO; ++i) {
            const int ch = chunk_of(half, i);
            if (ch * 32 < BN) {
              uint32_t r[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(sum[i][j]);
              tmem_st32(tb + ch * 32, r);
            }
          }
          tmem_st_wait();
        }
      }
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int ch = chunk_of(half, i);
        if (ch * 32 >= BN) break;
        if (S == 1) {
          if (mine && n0 + ch * 32 < ep.N)
            finish_chunk(ep, tb + ch * 32, i < 2 ? (i ? b[1] : b[0]) : (i == 2 ? b[2] : b[3]), row0, n0 + ch * 32, cend);
          continue;
        }
        // the whole tile to this CTA's shared memory (the ring is drained by now), rows
        // (BN + 4) floats apart
        uint32_t r[32];
        tmem_ld32(tb + ch * 32, r);
        tmem_ld_wait();
        float4* dst = reinterpret_cast<float4*>(smem) + (size_t)(q * 32 + lane) * (BN / 4 + 1) + ch * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (ch * 32 + j * 4 < BN)
            dst[j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                 __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
      }
      release(acc);
      acc ^= 1;
      if (acc == 0) aph ^= 1u;
    }
    if (lane == 0) bulk_wait_read<0>();   // before this shared memory goes
  }
  __syncwarp();
  if (S > 1) {
    cluster_sync();                       // all S tiles are in shared memory
    if (!*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {
      int tm, tn;
      tile_at(a, t0, &tm, &tn);
      const Epilogue ep = load_epilogue<F32>(a, tm_out, tm_pre, lane, staging, nullptr);
      const int row = split * (128 / S), m0 = tm * (128 * CG) + rank * 128 + row, n0 = tn * a.BN;
      if (S == 2) join_tiles<2, 4>(ep, smem_u32(smem), a.BN, m0, n0, row, CG, rank);
      else if (S == 4) join_tiles<4, 2>(ep, smem_u32(smem), a.BN, m0, n0, row, CG, rank);
      else join_tiles<8, 1>(ep, smem_u32(smem), a.BN, m0, n0, row, CG, rank);
    }
    __syncwarp();
  }
  __syncthreads();
  if (CG * S > 1) cluster_sync();         // no CTA leaves while its tile, ring or barriers are in use
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2) tmem_dealloc_pair(tmem, TMEM_COLS);
    else tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------- launch ---
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

// An operand of `inner` contiguous elements x `outer` rows: 128-byte rows of 64 elements,
// 128-byte swizzle; what lies outside reads as zero.  whole: {64, outer, inner / 64, planes}
// (inner a multiple of 64) in boxes of `rows` rows, `blocks` 64-element blocks and
// `planes` planes, or else {inner, outer, 1, planes} in boxes of one block of one plane.
// Copies cost about 0.1 us of the copy unit each, whatever their size, so a stage is
// brought by as few as can be: the up
// projection of 4096 x 4096 x 14336 takes 311 us with whole boxes, 344 us with one
// per 64 columns.
bool encode4(CUtensorMap* m, const GemmOperand& o, int inner, int outer, int rows, bool whole, int blocks, int planes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)(whole ? 64 : inner), (cuuint64_t)outer, (cuuint64_t)(whole ? inner / 64 : 1),
                              (cuuint64_t)o.planes};
  const cuuint64_t strides[3] = {(cuuint64_t)o.ld, 128, (cuuint64_t)(o.planes > 1 ? o.plane : 128)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)(whole ? blocks : 1), (cuuint32_t)(whole ? planes : 1)};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(o.p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Outputs {N, M, slices} of rows `ld` elements apart: boxes of 32 rows x 32 columns,
// swizzled as the epilogue stages them.
bool encode_out(CUtensorMap* m, void* p, int M, int N, int ld, int slices, int f32) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t pitch = (cuuint64_t)ld * (f32 ? 4 : 2);
  const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)slices}, strides[2] = {pitch, pitch * M};
  const cuuint32_t box[3] = {32, 32, 1}, es[3] = {1, 1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, bool AMN, bool BMN, int PROMO, bool F32>
cudaError_t run(const CUtensorMap (&m)[4], const GemmArgs& a, int grid, int dev, cudaStream_t s) {
  static bool configured[64] = {false};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(gemm_kernel<CG, AMN, BMN, PROMO, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)G_SMEM);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(G_THREADS);
  cfg.dynamicSmemBytes = G_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)(CG * a.S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG * a.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_kernel<CG, AMN, BMN, PROMO, F32>, m[0], m[1], m[2], m[3], a);
}

template <int CG, int PROMO, bool F32>
cudaError_t run_major(const GemmProblem& p, const CUtensorMap (&m)[4], const GemmArgs& a, int grid, int dev,
                      cudaStream_t s) {
  if (p.a_mn) return p.b_mn ? run<CG, true, true, PROMO, F32>(m, a, grid, dev, s) : cudaErrorInvalidValue;
  if (p.b_mn) return run<CG, false, true, PROMO, F32>(m, a, grid, dev, s);
  if constexpr (F32) return cudaErrorInvalidValue;          // no product of the layer has an fp32 output here
  else return run<CG, false, false, PROMO, false>(m, a, grid, dev, s);
}

template <int CG>
cudaError_t run_sums(const GemmProblem& p, const CUtensorMap (&m)[4], const GemmArgs& a, bool f32, bool promo, int grid,
                     int dev, cudaStream_t s) {
  if (f32) return a.BN <= 128 ? run_major<CG, 2, true>(p, m, a, grid, dev, s) : run_major<CG, 4, true>(p, m, a, grid, dev, s);
  return promo ? run_major<CG, 4, false>(p, m, a, grid, dev, s) : run_major<CG, 0, false>(p, m, a, grid, dev, s);
}

// A product's tiles and the splits of its reduction.
struct Shape { int CG, BN, S, SW; };

// Clusters of `size` CTAs that a device holds at once (one CTA per SM): fewer than SMs /
// size, as a cluster stays within a GPC.
int clusters_of(int dev, int nsm, int size) {
  static int most[64][9];
  if (size == 1) return nsm;
  if (most[dev][size] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(nsm / size * size));
    cfg.blockDim = dim3(G_THREADS);
    cfg.dynamicSmemBytes = G_SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    auto kernel = gemm_kernel<2, false, true, 0, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G_SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = max(1, nsm / size * 3 / 4);
    }
    most[dev][size] = n;
  }
  return most[dev][size];
}

// SM cycles of one tile configuration, from rates measured on one B200: an MMA of
// 128 (per CTA) x BN x 16 takes BN / 2 cycles, and a stage's bytes arrive at no more than
// FILL per cycle and SM; a tile's epilogue is hidden but for the last, and a pair's two
// CTAs cost a tile some cycles to keep in step.  (Four k-blocks per tile, dx of 16384 x 4096
// over 128 in two terms: 52 us in single blocks, 56 in pairs; eight of them: 82 and 76.)
double cost(const GemmProblem& p, int dev, int nsm, Shape c) {
  const int nkb = cdiv(p.K, 64), units = cdiv(p.M, 128 * c.CG) * cdiv(p.N, c.BN) * c.SW;
  const int cols = c.BN / c.CG, P = p.B.planes * p.A.planes;
  // per k-block: the MMAs; shared memory's 128 bytes per cycle for the tiles' way in and
  // the MMAs' operands; the way from L2
  const double in = 16384.0 * p.A.planes + p.B.planes * (p.b_mn ? cdiv(cols, 64) * 8192.0 : cols * 128.0);
  const double mma = max(2.0 * c.BN * P, (in + P * (16384.0 + cols * 128.0)) / 128.0);
  const double kb = max(max(mma, in / G_FILL), 150.0);
  const int waves = cdiv(units, clusters_of(dev, nsm, c.CG * c.S));
  double tail = 2500.0 + 8.0 * c.BN + (c.CG > 1 ? 800.0 : 0.0);
  if (c.S > 1) tail += 2500.0 + 16.0 * c.BN;
  if (c.SW > 1) tail += 3500.0 + c.SW * (double)p.M * p.N * 8.0 / (nsm * 40.0);
  return waves * (cdiv(nkb, c.S * c.SW) * kb + (c.CG > 1 ? 1800.0 : 300.0)) + tail;
}

// BN is a multiple of 32, so that a chunk of the epilogue lies in one tile, or 16 for N <= 16.
Shape pick(const GemmProblem& p, int dev, int nsm) {
  Shape best = {1, 16, 1, 1};
  double least = 1e300;
  auto consider = [&](Shape c) {
    const double t = cost(p, dev, nsm, c);
    if (t < least) { least = t; best = c; }
  };
  const int nkb = cdiv(p.K, 64), most = min(p.B.planes > 1 ? 128 : 256, cdiv(p.N, 32) * 32);
  const int slices = p.ws ? gemm_slices(p.M, p.N) : 1;
  for (int CG = 1; CG <= (p.M > 128 ? 2 : 1); ++CG) {
    const int rows = cdiv(p.M, 128 * CG), fit = clusters_of(dev, nsm, CG);
    for (int BN = CG == 1 && p.N <= 16 ? 16 : 32, before = 0; BN <= most; BN += 32) {
      const int cols = cdiv(p.N, BN);
      if (cols == before && BN % 128 != 0) continue;   // wider for no fewer tiles
      before = cols;
      const int tiles = rows * cols;
      consider({CG, BN, 1, 1});
      for (int S = 2; S * CG <= 8; S *= 2) {
        if (nkb < 4 * S || tiles > clusters_of(dev, nsm, S * CG)) break;
        consider({CG, BN, S, 1});
      }
      // slices that fill one wave of CTAs, or two
      for (int w = 1; w <= 2 && slices > 1; ++w) {
        const int SW = min(min(slices, fit * w / tiles), nkb / 4);
        if (SW > 1) consider({CG, BN, 1, SW});
      }
    }
  }
  return best;
}

// Whether a shape given by gemm_debug is one that pick() may come to for some size.
bool legal(const GemmProblem& p, int dev, int nsm, Shape c) {
  const int nkb = cdiv(p.K, 64), slices = p.ws ? gemm_slices(p.M, p.N) : 1;
  if (c.CG < 1 || c.CG > 2 || (c.CG == 2 && p.M <= 128)) return false;
  if (c.BN != 16 && (c.BN < 32 || c.BN % 32 != 0 || c.BN > min(p.B.planes > 1 ? 128 : 256, cdiv(p.N, 32) * 32))) return false;
  if (c.BN == 16 && (c.CG == 2 || p.N > 16)) return false;
  if (c.S < 1 || c.SW < 1 || (c.S & (c.S - 1)) != 0 || c.S * c.CG > 8 || (c.S > 1 && c.SW > 1)) return false;
  if (c.SW > 1 && (c.SW > slices || c.SW > nkb / 4)) return false;
  const int tiles = cdiv(p.M, 128 * c.CG) * cdiv(p.N, c.BN);
  return c.S == 1 || (nkb >= 4 * c.S && tiles <= clusters_of(dev, nsm, c.S * c.CG));
}

// out = the sum of the slices, in order: one thread per 4 columns.  The first blocks take
// the column sums.
template <int U>
__global__ void __launch_bounds__(256) join_kernel(const float4* __restrict__ ws, int SW, int M, int N, int ld4,
                                                   void* __restrict__ out, int f32, const ColumnSums sums) {
  __shared__ float sh[8][33];
  pdl_trigger();
  pdl_wait();
  const int first = sums.out ? cdiv(sums.N, 32) : 0;
  if ((int)blockIdx.x < first) {
    column_sums<8>(sums, blockIdx.x, sh);
    return;
  }
  const long total = (long)M * ld4;
  const bool vec = (N & 3) == 0;
  for (long i = (long)(blockIdx.x - first) * 256 + threadIdx.x; i < total; i += (long)(gridDim.x - first) * 256) {
    float4 v = __ldcg(ws + i);
    for (int s = 1; s < SW; s += U) {
      float4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = s + u < SW ? __ldcg(ws + (s + u) * total + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u < SW) { v.x += w[u].x; v.y += w[u].y; v.z += w[u].z; v.w += w[u].w; }
    }
    const long m = i / ld4;
    const int n = (int)(i - m * ld4) * 4;
    const size_t at = (size_t)m * N + n;
    if (vec) {
      if (f32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
      else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
      continue;
    }
    const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= N) break;
      if (f32) static_cast<float*>(out)[at + j] = u[j];
      else static_cast<__nv_bfloat16*>(out)[at + j] = __float2bfloat16(u[j]);
    }
  }
}

}  // namespace

// What moe_linear_debug_set has set for the calling thread's products.
struct GemmDebug {
  Shape shape;                            // CG = 0: chosen by cost
  uint64_t limit;
  int withhold;
};
thread_local GemmDebug gemm_debug = {{0, 0, 0, 0}, G_TIMEOUT, 0};

// Slices for which the workspace has room: up to 16, and no more than 40 MB of them (two
// waves of 256 x 256 tiles).
int gemm_slices(int M, int N) {
  const long long one = (long long)M * (cdiv(N, 4) * 4);
  const long long n = 10000000 / one;
  return n < 2 ? 1 : (int)(n < 16 ? n : 16);
}
size_t gemm_ws_bytes(int M, int N) {
  const int n = gemm_slices(M, N);
  return n > 1 ? (size_t)n * M * (cdiv(N, 4) * 4) * 4 : 0;
}

cudaError_t device_of(int* dev, int* sms) {
  static int count[64] = {0};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  if (count[d] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
    if (e != cudaSuccess) return e;
    count[d] = n;
  }
  if (dev) *dev = d;
  *sms = count[d];
  return cudaSuccess;
}

cudaError_t launch_gemm(const GemmProblem& p, cudaStream_t s) {
  int dev = 0, nsm = 0;
  cudaError_t e = device_of(&dev, &nsm);
  if (e != cudaSuccess) return e;
  // Encoding a tensor map takes a current context, which a thread that has launched nothing
  // yet does not have: setting its device makes that device's context current.
  static thread_local int bound = -1;
  if (bound != dev) {
    e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    bound = dev;
  }
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  a.M = p.M; a.N = p.N; a.K = p.K;
  a.PA = p.A.planes;
  a.PB = p.B.planes;
  if (a.PA > 1 && (a.PA > 2 || p.a_mn || p.b_mn || a.PB > 1)) return cudaErrorInvalidValue;
  a.ep = p.ep;
  a.limit = gemm_debug.limit;
  a.withhold = gemm_debug.withhold;
  Shape c = gemm_debug.shape;
  if (c.CG == 0) c = pick(p, dev, nsm);
  else if (!legal(p, dev, nsm, c)) return cudaErrorNotSupported;
  a.BN = c.BN;
  a.S = c.S;
  a.SW = c.SW;
  a.tiles_m = cdiv(p.M, 128 * c.CG);
  a.tiles_n = cdiv(p.N, a.BN);
  const int ntiles = a.tiles_m * a.tiles_n, cols = a.BN / c.CG;
  a.b_boxes = cdiv(cols, 64);
  const int b_kb = p.b_mn ? a.b_boxes * 8192 : cols * 128;   // one k-block of one plane
  // the ring's tiles start on 1024-byte boundaries (cols is a multiple of 16)
  a.kps = a.PA == 1 && A_BYTES + a.PB * b_kb <= 24576 ? 2 : 1;
  a.b_bytes = a.kps * b_kb;
  a.stage_bytes = a.kps * a.PA * A_BYTES + a.PB * a.b_bytes;
  a.a_whole = (p.a_mn ? p.M : p.K) % 64 == 0;
  a.b_whole = p.b_mn ? p.N % 64 == 0 && cols % 64 == 0 : p.K % 64 == 0;
  a.nst = min(G_MAX_NST, G_RING / a.stage_bytes);
  a.group = c.CG == 2 ? 8 : 16;
  const bool f32 = p.ep.out_f32 || a.SW > 1;
  a.chunk = (p.ep.out_f32 ? CHAIN_F32 : CHAIN_BF16) / a.PA;
  const bool promo = cdiv(cdiv(p.K, 64), a.S * a.SW) > a.chunk;
  CUtensorMap m[4];
  if (!(p.a_mn ? encode4(&m[0], p.A, p.M, p.K, 64 * a.kps, a.a_whole, 2, 1)
               : encode4(&m[0], p.A, p.K, p.M, 128, a.a_whole, a.kps, a.PA)) ||
      !(p.b_mn ? encode4(&m[1], p.B, p.N, p.K, 64 * a.kps, a.b_whole, a.b_boxes, a.PB)
               : encode4(&m[1], p.B, p.K, p.N, cols, a.b_whole, a.kps, 1)))
    return cudaErrorInvalidValue;
  a.tma_out = a.S == 1 && p.N % (p.ep.out_f32 ? 4 : 8) == 0;
  a.tma_pre = a.S == 1 && p.ep.pre && p.N % 8 == 0;
  m[2] = m[3] = m[0];                     // read with tma_out, tma_pre only
  const int ld4 = cdiv(p.N, 4);
  if (a.SW > 1) {
    a.tma_out = 1;
    if (!encode_out(&m[2], p.ws, p.M, p.N, ld4 * 4, a.SW, 1)) return cudaErrorInvalidValue;
  } else if (a.tma_out && !encode_out(&m[2], p.ep.out, p.M, p.N, p.N, 1, p.ep.out_f32)) {
    return cudaErrorInvalidValue;
  }
  if (a.tma_pre && !encode_out(&m[3], p.ep.pre, p.M, p.N, p.N, 1, 0)) return cudaErrorInvalidValue;
  const int grid = c.CG * (a.S > 1 ? ntiles * a.S : min(ntiles * a.SW, clusters_of(dev, nsm, c.CG)));
  e = c.CG == 2 ? run_sums<2>(p, m, a, f32, promo, grid, dev, s) : run_sums<1>(p, m, a, f32, promo, grid, dev, s);
  if (e != cudaSuccess || a.SW == 1) return e;
  const long vecs = (long)p.M * ld4;
  const int blocks = (int)(vecs < 16L * nsm * 256 ? (vecs + 255) / 256 : 16L * nsm);
  ColumnSums sums = {};
  if (p.sums && p.sums->out) {
    sums = *p.sums;
    p.sums->out = nullptr;
  }
  return launch_pdl(join_kernel<4>, dim3(blocks + (sums.out ? cdiv(sums.N, 32) : 0)), dim3(256), 0, s,
                    static_cast<const float4*>(p.ws), a.SW, p.M, p.N, ld4, p.ep.out, p.ep.out_f32, sums);
}

void linear_debug(int CG, int BN, int S, int SW, int timeout_us, int withhold) {
  gemm_debug = {{CG, BN, S, SW}, timeout_us > 0 ? timeout_us * 1000ull : G_TIMEOUT, withhold};
}

cudaError_t linear_timeouts(cudaStream_t s, uint32_t* count) {
  const cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_linear_timeouts, 4, 0, cudaMemcpyDeviceToHost, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace moe
