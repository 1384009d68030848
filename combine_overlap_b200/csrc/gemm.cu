// gemm.cu -- the linear layer's products on the 5th-generation tensor cores: TMA tiles
// into a ring of shared-memory stages, tcgen05 MMAs (bf16, fp32 accumulators in TMEM)
// issued by one thread, and an epilogue (bias, activation, residual, one rounding) that
// runs beside the next tile's main loop.
//
// Tiles and splits:
//   MT = 1  128 rows x BN columns; two accumulators, so the epilogue of tile i overlaps
//           the main loop of tile i + 1;
//   MT = 2  256 x BN as two 128-row MMAs per k-step against one B stage: a third less
//           operand traffic per FLOP, both accumulators belong to one tile;
//   S > 1   the reduction is cut over a cluster of S CTAs: each leaves its fp32 tile in
//           its shared memory, and CTA r finishes rows [r 128/S, (r+1) 128/S) by adding
//           the S tiles through distributed shared memory in order 0 .. S-1 -- no
//           workspace, no atomics, the same bits every time.
#include "gemm.cuh"

#include <string.h>

namespace moe {

namespace {

constexpr int G_THREADS = 320;            // warp 0 TMA, warp 1 MMA, warps 2-9 epilogue
constexpr int G_EPI = 8;
constexpr int G_MAX_NST = 12;
constexpr int G_RING = 196608;            // bytes of the operand ring
constexpr int G_STAGING = G_EPI * 4096;   // per epilogue warp: 32 rows x 32 fp32 columns
constexpr uint64_t G_TIMEOUT = 2000000000ull;

struct GemmCtl {
  uint64_t full[G_MAX_NST], empty[G_MAX_NST];
  uint64_t tfull[2], tempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t abort;                         // a bounded wait of this CTA ran out
};

constexpr size_t G_SMEM = 1024 + (size_t)G_RING + G_STAGING + sizeof(GemmCtl);
static_assert(G_SMEM <= 227 * 1024, "over the 227 KB per-CTA limit");

// Set when a bounded wait of a product ran out; read and cleared by
// moe_linear_get_status.
__device__ uint32_t g_linear_timeout;

struct GemmArgs {
  int M, N, K;
  int tiles_m, tiles_n;
  int BN;                                 // columns per tile, a multiple of 16, <= 256
  int S;                                  // CTAs per tile (split of the reduction)
  int PA, PB;                             // planes of A and of B
  int nst, stage_bytes, a_bytes, b_bytes; // ring; bytes of one A (128 rows) and one B plane tile
  int group;                              // row tiles per raster group
  LinearEpi ep;
};

__device__ __forceinline__ bool g_wait(uint64_t* bar, uint32_t parity, GemmCtl* ctl) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t deadline = globaltimer() + G_TIMEOUT;
  volatile uint32_t* ab = &ctl->abort;
  if (mbar_wait(bar, parity, deadline, ab)) return true;
  if (!*ab) {
    *ab = 1;
    atomicExch(&g_linear_timeout, 1u);
  }
  return false;
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

template <int MT, bool AMN, bool BMN>
__global__ void __launch_bounds__(G_THREADS, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
            const GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* staging = smem + G_RING;
  GemmCtl* ctl = reinterpret_cast<GemmCtl*>(staging + G_STAGING);
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.nst; ++i) { mbar_init(&ctl->full[i], 1); mbar_init(&ctl->empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&ctl->tfull[i], 1); mbar_init(&ctl->tempty[i], G_EPI); }
    mbar_init(&ctl->mma_done, 1);
    ctl->abort = 0;
    mbar_fence_init();
    fence_proxy_async_shared();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_wait();

  const int nkb = cdiv(a.K, 64);
  const int S = a.S;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int t0 = blockIdx.x / S, tstep = gridDim.x / S;
  const int ntiles = a.tiles_m * a.tiles_n;
  // this CTA's k-blocks: as even as can be
  const int kb0 = (int)((long long)nkb * rank / S), kb1 = (int)((long long)nkb * (rank + 1) / S);
  const bool vec = (a.N & 3) == 0;

  if (warp == 0 && lane == 0) {
    int stage = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = t0; t < ntiles && ok; t += tstep) {
      int tm, tn;
      tile_at(a, t, &tm, &tn);
      const int m0 = tm * (128 * MT), n0 = tn * a.BN;
      const int blocks = MT == 2 && a.M - m0 > 128 ? 2 : 1;
      const uint32_t bytes = (uint32_t)(blocks * a.PA * a.a_bytes + a.PB * a.b_bytes);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!g_wait(&ctl->empty[stage], ph ^ 1u, ctl)) { ok = false; break; }
        uint8_t* dst = smem + (size_t)stage * a.stage_bytes;
        mbar_arrive_expect_tx(&ctl->full[stage], bytes);
        for (int p = 0; p < a.PA; ++p) {
          for (int b = 0; b < blocks; ++b) {
            uint8_t* d = dst + (p * MT + b) * a.a_bytes;
            if constexpr (AMN) {
              tma_load_3d(d, &tm_a, &ctl->full[stage], m0 + b * 128, kb * 64, p);
              tma_load_3d(d + 8192, &tm_a, &ctl->full[stage], m0 + b * 128 + 64, kb * 64, p);
            } else {
              tma_load_3d(d, &tm_a, &ctl->full[stage], kb * 64, m0 + b * 128, p);
            }
          }
        }
        uint8_t* db = dst + a.PA * MT * a.a_bytes;
        for (int p = 0; p < a.PB; ++p) {
          if constexpr (BMN) {
            for (int j = 0; j * 64 < a.BN; ++j)
              tma_load_3d(db + p * a.b_bytes + j * 8192, &tm_b, &ctl->full[stage], n0 + j * 64, kb * 64, p);
          } else {
            tma_load_3d(db + p * a.b_bytes, &tm_b, &ctl->full[stage], kb * 64, n0, p);
          }
        }
        if (++stage == a.nst) { stage = 0; ph ^= 1u; }
      }
    }
    if (!ok) {
      // copies may still be landing: wait (bounded) until every stage's are in
      const uint64_t until = globaltimer() + G_TIMEOUT;
      for (int i = 0; i < a.nst; ++i)
        for (uint32_t par = 0; par < 2; ++par)
          while (!mbar_try_wait(&ctl->full[i], par) && globaltimer() < until) {}
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16_f32(128, a.BN, BMN) | (AMN ? 1u << 15 : 0u);
    int stage = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (int t = t0; t < ntiles && ok; t += tstep) {
      int tm, tn;
      tile_at(a, t, &tm, &tn);
      const int blocks = MT == 2 && a.M - tm * 256 > 128 ? 2 : 1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!g_wait(&ctl->full[stage], ph, ctl)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + (size_t)stage * a.stage_bytes);
        const uint32_t sb = sa + (uint32_t)(a.PA * MT * a.a_bytes);
        const int ks = min(4, cdiv(a.K - kb * 64, 16));
        for (int b = 0; b < (MT == 2 ? 2 : 1); ++b) {
          const int ai = MT == 2 ? b : acc;
          if (kb == kb0) {
            if (!g_wait(&ctl->tempty[ai], aph ^ 1u, ctl)) { ok = false; break; }
            tc_fence_after();
          }
          if (b >= blocks) continue;
          const uint32_t dt = tmem + (uint32_t)(ai * ACC_COLS);
          for (int pa = 0; pa < a.PA; ++pa) {
            for (int pb = 0; pb < a.PB; ++pb) {
              const uint32_t ta = sa + (uint32_t)((pa * MT + b) * a.a_bytes), tb = sb + (uint32_t)(pb * a.b_bytes);
              for (int k = 0; k < ks; ++k) {
                const uint64_t ad = AMN ? smem_desc_sw128(ta + k * 2048, 8192, 1024) : smem_desc_sw128(ta + k * 32, 16, 1024);
                const uint64_t bd = BMN ? smem_desc_sw128(tb + k * 2048, 8192, 1024) : smem_desc_sw128(tb + k * 32, 16, 1024);
                tc_mma_f16(dt, ad, bd, idesc, (kb > kb0 || pa || pb || k) ? 1u : 0u);
              }
            }
          }
        }
        if (!ok) break;
        tc_commit(&ctl->empty[stage]);
        if (++stage == a.nst) { stage = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (MT == 2) {
        tc_commit(&ctl->tfull[0]);
        tc_commit(&ctl->tfull[1]);
        aph ^= 1u;
      } else {
        tc_commit(&ctl->tfull[acc]);
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      }
    }
    tc_commit(&ctl->mma_done);
    g_wait(&ctl->mma_done, 0u, ctl);      // every MMA is done before TMEM is released
  } else if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q .., every other chunk of columns
    int acc = 0;
    uint32_t aph = 0;
    float4* st = reinterpret_cast<float4*>(staging + (warp - 2) * 4096);
    bool ok = true;
    for (int t = t0; t < ntiles && ok; t += tstep) {
      int tm, tn;
      tile_at(a, t, &tm, &tn);
      for (int b = 0; b < (MT == 2 ? 2 : 1); ++b) {
        const int ai = MT == 2 ? b : acc;
        if (!g_wait(&ctl->tfull[ai], aph, ctl)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem + (uint32_t)(ai * ACC_COLS) + ((uint32_t)(q * 32) << 16);
        const int row0 = tm * (128 * MT) + b * 128 + q * 32;
        for (int c = half; c * 32 < a.BN; c += 2) {
          const int col = tn * a.BN + c * 32;
          if (S == 1 && (row0 >= a.M || col >= a.N)) break;
          uint32_t r[32];
          tmem_ld32(tb + c * 32, r);
          tmem_ld_wait();
          if (S > 1) {
            // the whole tile to this CTA's shared memory (the ring is drained by now),
            // rows (BN + 4) floats apart
            float4* dst = reinterpret_cast<float4*>(smem) + (size_t)(q * 32 + lane) * (a.BN / 4 + 1) + c * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c * 32 + i * 4 < a.BN)
                dst[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                     __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
            continue;
          }
          // 32 x 32 through shared memory (16-byte units XORed with the row), so that
          // eight lanes hold one row's 32 columns
#pragma unroll
          for (int i = 0; i < 8; ++i)
            st[lane * 8 + (i ^ (lane & 7))] =
                make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                            __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
          __syncwarp();
          const int n = col + (lane & 7) * 4;
          if (n < a.N && c * 32 + (lane & 7) * 4 < a.BN) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3);
              if (row0 + rr < a.M) epilogue4(a.ep, a.N, row0 + rr, n, st[rr * 8 + ((lane & 7) ^ (rr & 7))], vec);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (lane == 0) mbar_arrive(&ctl->tempty[ai]);
        __syncwarp();
      }
      if (MT == 2) aph ^= 1u;
      else { acc ^= 1; if (acc == 0) aph ^= 1u; }
    }
  }
  __syncwarp();
  if (S > 1) {
    cluster_sync();                       // all S tiles are in shared memory
    if (!*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) {
      int tm, tn;
      tile_at(a, t0, &tm, &tn);
      const int rows = 128 / S, pitch = (a.BN / 4 + 1) * 16;
      const uint32_t base = smem_u32(smem);
      const int per = a.BN / 4;
      for (int i = threadIdx.x; i < rows * per; i += G_THREADS) {
        const int r = rank * rows + i / per, c4 = i % per;
        const int m = tm * 128 + r, n = tn * a.BN + c4 * 4;
        if (m >= a.M || n >= a.N) continue;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < S; ++s) {
          const float4 w = ld_cluster_v4(mapa_shared(base + (uint32_t)(r * pitch + c4 * 16), (uint32_t)s));
          v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
        }
        epilogue4(a.ep, a.N, m, n, v, vec);
      }
    }
    __syncwarp();
    cluster_sync();                       // no CTA leaves while its tile is read
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
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

// {inner, outer, planes}: boxes of 64 inner elements x box_rows, 128-byte swizzle; what
// lies outside reads as zero.
bool encode3(CUtensorMap* m, const GemmOperand& o, int inner, int outer, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)o.planes};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld, (cuuint64_t)(o.planes > 1 ? o.plane : o.ld * (size_t)outer)};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MT, bool AMN, bool BMN>
cudaError_t run(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& a, int grid, int dev, cudaStream_t s) {
  static bool configured[64] = {false};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(gemm_kernel<MT, AMN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  attr[1].val.clusterDim.x = (unsigned)a.S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, gemm_kernel<MT, AMN, BMN>, ma, mb, a);
}

}  // namespace

cudaError_t launch_gemm(const GemmProblem& p, cudaStream_t s) {
  int dev = 0, nsm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  GemmArgs a;
  memset(&a, 0, sizeof(a));
  a.M = p.M; a.N = p.N; a.K = p.K;
  a.PA = p.A.planes; a.PB = p.B.planes;
  a.ep = p.ep;
  const int nkb = cdiv(p.K, 64);
  int MT = 1;
  a.BN = min(256, cdiv(p.N, 16) * 16);
  if (a.PB > 1) a.BN = min(a.BN, 128);
  if (a.PA == 1 && a.PB == 1 && (long long)cdiv(p.M, 256) * cdiv(p.N, a.BN) >= 2 * nsm) MT = 2;
  a.tiles_m = cdiv(p.M, 128 * MT);
  a.tiles_n = cdiv(p.N, a.BN);
  const int ntiles = a.tiles_m * a.tiles_n;
  a.S = 1;
  while (MT == 1 && a.S < 8 && ntiles * a.S * 2 <= nsm && nkb >= a.S * 4) a.S *= 2;
  a.a_bytes = 16384;
  a.b_bytes = cdiv(a.BN, 64) * 8192;
  if (!p.b_mn) a.b_bytes = cdiv(a.BN * 128, 1024) * 1024;
  a.stage_bytes = a.PA * MT * a.a_bytes + a.PB * a.b_bytes;
  a.nst = min(G_MAX_NST, G_RING / a.stage_bytes);
  a.group = 16;
  CUtensorMap ma, mb;
  if (!(p.a_mn ? encode3(&ma, p.A, p.M, p.K, 64) : encode3(&ma, p.A, p.K, p.M, 128))) return cudaErrorInvalidValue;
  if (!(p.b_mn ? encode3(&mb, p.B, p.N, p.K, 64) : encode3(&mb, p.B, p.K, p.N, a.BN))) return cudaErrorInvalidValue;
  const int grid = a.S > 1 ? ntiles * a.S : min(ntiles, nsm);
  if (p.a_mn) {
    if (!p.b_mn) return cudaErrorInvalidValue;
    return MT == 2 ? run<2, true, true>(ma, mb, a, grid, dev, s) : run<1, true, true>(ma, mb, a, grid, dev, s);
  }
  if (p.b_mn) return MT == 2 ? run<2, false, true>(ma, mb, a, grid, dev, s) : run<1, false, true>(ma, mb, a, grid, dev, s);
  return MT == 2 ? run<2, false, false>(ma, mb, a, grid, dev, s) : run<1, false, false>(ma, mb, a, grid, dev, s);
}

cudaError_t linear_timeout(cudaStream_t s, uint32_t* word) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_linear_timeout, 4, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || *word == 0) return e;
  const uint32_t zero = 0;
  e = cudaMemcpyToSymbolAsync(g_linear_timeout, &zero, 4, 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace moe
