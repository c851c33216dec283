// gemm_fp8.cu -- product of e4m3 matrices with a scale for each 1 x 128 block of the activations
// and each 128 x 128 block of the weights, on the fifth-generation tensor cores:
//
//   out[i][j] = sum_b sa[b][i] sw[b][j / 128] (sum_{l in block b} a[i][l] w[j][l])
//
// The scales change with every block of 128 along k, so each block's product is a tensor-memory
// accumulator of its own (four kind::f8f6f4 instructions of K = 32) that the epilogue warps read,
// scale and add to float32 sums in registers while the tensor cores work on the next blocks.
//
// Tiles of 128 output features (the instruction's M, so that a tile has one weight scale per
// block) x 32, 64 or 128 tokens (its N):
//   warp 5      TMA producer: per block the weights' 128 x 128 and the tokens' codes, and the
//               tokens' scales;
//   warp 4      TMEM owner and MMA issuer (one thread);
//   warps 0..3  epilogue: thread = output feature, one float32 sum per token.
// With fewer tiles than SMs a cluster of up to 8 CTAs shares a tile, each taking a contiguous
// range of the blocks; their sums meet in distributed shared memory, each CTA adding a share of
// the tokens in rank order.
#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace hs2 {

namespace {

constexpr int kGtWarpMma = 4, kGtWarpTma = 5, kGtThreads = 6 * 32;
constexpr int kGtAcc = 4;                       // accumulators in TMEM
constexpr int kGtWBytes = 128 * 128;

template <int TN>
struct GtCfg {
  static constexpr int kABytes = TN * 128, kSBytes = TN * 4;
  static constexpr int kStageBytes = (kGtWBytes + kABytes + kSBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = TN == 128 ? 6 : 8;
  static constexpr uint32_t kTx = kGtWBytes + kABytes + kSBytes;
  static constexpr uint32_t kCols = TN * kGtAcc;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStageBytes + (2 * kStages + 2 * kGtAcc + 1) * 8 + 16;
  static_assert(TN * 128 * 4 <= kStages * kStageBytes, "the partial sums reuse the stages");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int TN>
struct GtSmem {
  using C = GtCfg<TN>;
  uint8_t *stages;
  uint64_t *full, *empty, *acc_full, *acc_empty, *done;
  uint32_t *tmem_base;
  volatile int *abort_flag;
  __device__ explicit GtSmem(uint8_t *raw) {
    stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    full = reinterpret_cast<uint64_t *>(stages + C::kStages * C::kStageBytes);
    empty = full + C::kStages;
    acc_full = empty + C::kStages;
    acc_empty = acc_full + kGtAcc;
    done = acc_empty + kGtAcc;
    tmem_base = reinterpret_cast<uint32_t *>(done + 1);
    abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
  }
};

// bounded wait by lane 0, the result broadcast to the warp (records a timeout)
__device__ __forceinline__ bool gt_wait(uint32_t *status, volatile int *abort_flag, uint64_t *bar,
                                        uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    ok = mbar_wait(smem_u32(bar), parity);
    if (!ok) {
      record_status(status, kStatusTimeout);
      *abort_flag = 1;
    }
    if (*abort_flag) ok = false;
  }
  return __shfl_sync(0xffffffffu, ok, 0);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

__device__ __forceinline__ void gemm_store(const GemmParams &P, int64_t row, int col, float v) {
  if (P.out_f32) static_cast<float *>(P.out)[row * P.ldo + col] = v;
  else static_cast<__nv_bfloat16 *>(P.out)[row * P.ldo + col] = __float2bfloat16_rn(v);
}

template <int TN>
__global__ void __launch_bounds__(kGtThreads, 1)
    gemm_fp8_tokens_kernel(const __grid_constant__ GemmMaps tm, const __grid_constant__ GemmParams P) {
  using C = GtCfg<TN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  GtSmem<TN> sm(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % P.split, tile = blockIdx.x / P.split;
  const int nt = tile % P.n_tiles, mt = tile / P.n_tiles;
  const int kb0 = (int)((int64_t)rank * P.kb / P.split), kb1 = (int)((int64_t)(rank + 1) * P.kb / P.split);
  const int nk = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 5);   // the products, and four warps' scale reads
    }
    for (int a = 0; a < kGtAcc; ++a) {
      mbar_init(smem_u32(&sm.acc_full[a]), 1);
      mbar_init(smem_u32(&sm.acc_empty[a]), 4);
    }
    mbar_init(smem_u32(&sm.done[0]), 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kGtWarpTma && lane == 0) {
    prefetch_tensormap(&tm.a);
    prefetch_tensormap(&tm.w);
    prefetch_tensormap(&tm.sa);
  }
  if (warp == kGtWarpMma) {
    tmem_alloc(smem_u32(sm.tmem_base), C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_base;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  float acc[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) acc[j] = 0.f;
  if (warp == kGtWarpTma) {
    // ------------------------------------------------------------ producer
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % C::kStages;
      if (it >= C::kStages && !gt_wait(P.status, sm.abort_flag, &sm.empty[s], ((it / C::kStages) & 1) ^ 1)) break;
      if (lane == 0) {
        const uint32_t st = smem_u32(sm.stages + s * C::kStageBytes), bar = smem_u32(&sm.full[s]);
        mbar_arrive_expect_tx(bar, C::kTx);
        tma_load_2d(st, &tm.w, bar, (kb0 + it) * 128, nt * 128);
        tma_load_2d(st + kGtWBytes, &tm.a, bar, (kb0 + it) * 128, mt * TN);
        tma_load_2d(st + kGtWBytes + C::kABytes, &tm.sa, bar, mt * TN, kb0 + it);
      }
      __syncwarp();
    }
    if (lane == 0 && it < nk)   // gave up: the copies in flight land before the CTA ends
      for (int j = max(0, it - C::kStages); j < it; ++j)
        mbar_wait(smem_u32(&sm.full[j % C::kStages]), (j / C::kStages) & 1);
    __syncwarp();
  } else if (warp == kGtWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = umma_idesc_e4m3(128, TN);
    for (int it = 0; it < nk; ++it) {
      const int s = it % C::kStages, a = it % kGtAcc;
      if (it >= kGtAcc && !gt_wait(P.status, sm.abort_flag, &sm.acc_empty[a], ((it / kGtAcc) & 1) ^ 1)) break;
      if (!gt_wait(P.status, sm.abort_flag, &sm.full[s], (it / C::kStages) & 1)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t st = smem_u32(sm.stages + s * C::kStageBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_e4m3(tmem + a * TN, umma_desc_sw128(st + k * 32, 1024),
                    umma_desc_sw128(st + kGtWBytes + k * 32, 1024), idesc, k != 0);
        umma_commit(smem_u32(&sm.empty[s]));
        umma_commit(smem_u32(&sm.acc_full[a]));
      }
      __syncwarp();
    }
    if (lane == 0) {   // every product has landed before TMEM is released
      umma_commit(smem_u32(&sm.done[0]));
      if (!mbar_wait(smem_u32(&sm.done[0]), 0)) {
        record_status(P.status, kStatusTimeout);
        *sm.abort_flag = 1;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    const float *sw = P.w_scale + nt;
    float w_next = nk > 0 ? sw[(int64_t)kb0 * P.w_scale_ld] : 0.f;
    for (int it = 0; it < nk; ++it) {
      const int s = it % C::kStages, a = it % kGtAcc;
      const float w = w_next;
      if (it + 1 < nk) w_next = sw[(int64_t)(kb0 + it + 1) * P.w_scale_ld];
      if (!gt_wait(P.status, sm.abort_flag, &sm.full[s], (it / C::kStages) & 1)) break;   // the scales
      if (!gt_wait(P.status, sm.abort_flag, &sm.acc_full[a], (it / kGtAcc) & 1)) break;
      tc_fence_after();
      const float4 *sa = reinterpret_cast<const float4 *>(sm.stages + s * C::kStageBytes + kGtWBytes + C::kABytes);
      const float2 w2 = make_float2(w, w);
#pragma unroll
      for (int c = 0; c < TN; c += 32) {
        float v[32];
        tmem_ld32(lane_addr + a * TN + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = sa[(c + j) >> 2];
          const float2 s0 = fmul2(make_float2(f.x, f.y), w2), s1 = fmul2(make_float2(f.z, f.w), w2);
          const float2 r0 = ffma2(make_float2(v[j], v[j + 1]), s0, make_float2(acc[c + j], acc[c + j + 1]));
          const float2 r1 = ffma2(make_float2(v[j + 2], v[j + 3]), s1, make_float2(acc[c + j + 2], acc[c + j + 3]));
          acc[c + j] = r0.x;
          acc[c + j + 1] = r0.y;
          acc[c + j + 2] = r1.x;
          acc[c + j + 3] = r1.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&sm.acc_empty[a]));
        mbar_arrive(smem_u32(&sm.empty[s]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kGtWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  const int n = nt * 128 + threadIdx.x, m0 = mt * TN;
  const int nm = min(TN, P.m - m0);
  if (P.split == 1) {
    if (threadIdx.x < 128 && n < P.n) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (j < nm) gemm_store(P, (int64_t)m0 + j, n, acc[j]);
    }
    return;
  }
  // ------------------------------------------------------------ the cluster's sums, in rank order
  float *part = reinterpret_cast<float *>(sm.stages);   // [token][128]
  const bool aborted = *sm.abort_flag != 0;
  if (threadIdx.x < 128 && !aborted) {
#pragma unroll
    for (int j = 0; j < TN; ++j) part[j * 128 + threadIdx.x] = acc[j];
  }
  cluster_sync();
  if (threadIdx.x < 128 && n < P.n) {
    const int j0 = rank * nm / P.split, j1 = (rank + 1) * nm / P.split;
    for (int j = j0; j < j1; ++j) {
      const uint32_t at = smem_u32(part + j * 128 + threadIdx.x);
      float v = 0.f;
      for (int r = 0; r < P.split; ++r) v += ld_cluster(at, r);
      gemm_store(P, (int64_t)m0 + j, n, v);
    }
  }
  cluster_sync();   // no CTA leaves while another reads its sums
}

template <int TN>
cudaError_t launch_gt(const GemmMaps &tm, const GemmParams &p, cudaStream_t s) {
  auto kern = gemm_fp8_tokens_kernel<TN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, GtCfg<TN>::kBytes, done);
  if (e != cudaSuccess) return e;
  const int grid = p.n_tiles * p.m_tiles * p.split;
  e = p.split > 1 ? launch_pdl_cluster(kern, grid, kGtThreads, GtCfg<TN>::kBytes, p.split, s, tm, p)
                  : launch_pdl(kern, grid, kGtThreads, GtCfg<TN>::kBytes, s, tm, p);
  return e;
}

}  // namespace

cudaError_t launch_gemm_fp8_tokens(int tokens, const GemmMaps &tm, const GemmParams &p, cudaStream_t s) {
  switch (tokens) {
    case 32: return launch_gt<32>(tm, p, s);
    case 64: return launch_gt<64>(tm, p, s);
    case 128: return launch_gt<128>(tm, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace hs2
