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
//   TMA warp    per block the weights' 128 x 128 and the tokens' codes, and the tokens' scales;
//   MMA warp    TMEM owner and issuer;
//   epilogue    four warps (eight for 128 tokens, two per 32 features): thread = output feature, one
//               float32 sum per token (of its half).
// The weights are read once for all tokens of a tile: with few tokens the time is theirs. With fewer
// tiles than CTAs fit, a cluster of up to 8 CTAs shares a tile, each taking a contiguous range of the
// blocks; their sums meet in distributed shared memory, each CTA adding a share of the tokens in
// rank order. Tiles of 32 tokens leave room for two CTAs per SM.
//
// What bounds it: with few tokens the stream of weights (8 x 16384 x 16384: 47 us, 5.7 TB/s, 0.87 of
// measured; 8 x 16384 x 4096, 67 MB: 14.4 us, of which about 4 are start and end), with one small matrix the
// start and end alone (1 x 256 x 4096: 4.4 us).
#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace hs2 {

namespace {

constexpr int kGtAcc = 4;                       // accumulators in TMEM
constexpr int kGtWBytes = 128 * 128;

template <int TN>
struct GtCfg {
  static constexpr int kParts = TN == 128 ? 2 : 1;   // epilogue warps per 32 features
  static constexpr int kCols = TN / kParts;          // tokens per epilogue thread
  static constexpr int kEpi = 4 * kParts, kWarpMma = kEpi, kWarpTma = kEpi + 1, kThreads = (kEpi + 2) * 32;
  static constexpr int kABytes = TN * 128, kSBytes = TN * 4;
  static constexpr int kStageBytes = (kGtWBytes + kABytes + kSBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = TN == 32 ? 5 : TN == 64 ? 8 : 6;
  static constexpr int kPerSm = TN == 32 ? 2 : 1;
  static constexpr uint32_t kTx = kGtWBytes + kABytes + kSBytes;
  static constexpr uint32_t kTmem = TN * kGtAcc;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStageBytes + (2 * kStages + 2 * kGtAcc + 1) * 8 + 16;
  static_assert(TN * 128 * 4 <= kStages * kStageBytes, "the partial sums reuse the stages");
  static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory");
  static_assert(kPerSm * kTmem <= 512, "tensor memory");
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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
  return v;
}

__device__ __forceinline__ void gemm_store(const GemmParams &P, int64_t row, int col, float v) {
  if (P.out_f32) static_cast<float *>(P.out)[row * P.ldo + col] = v;
  else static_cast<__nv_bfloat16 *>(P.out)[row * P.ldo + col] = __float2bfloat16_rn(v);
}

// four neighbouring columns, as far as they exist; wide: rows start on 16 bytes
__device__ __forceinline__ void gemm_store4(const GemmParams &P, int64_t row, int col, float4 v, bool wide) {
  if (wide && col + 4 <= P.n) {
    if (P.out_f32)
      *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + row * P.ldo + col) = v;
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(P.out) + row * P.ldo + col) =
          make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < P.n) gemm_store(P, row, col + i, f[i]);
}

template <int TN>
__global__ void __launch_bounds__(GtCfg<TN>::kThreads, GtCfg<TN>::kPerSm)
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
      mbar_init(smem_u32(&sm.empty[s]), 1 + C::kEpi);   // the products, and the epilogue warps' scale reads
    }
    for (int a = 0; a < kGtAcc; ++a) {
      mbar_init(smem_u32(&sm.acc_full[a]), 1);
      mbar_init(smem_u32(&sm.acc_empty[a]), C::kEpi);
    }
    mbar_init(smem_u32(&sm.done[0]), 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == C::kWarpTma && lane == 0) {
    prefetch_tensormap(&tm.a);
    prefetch_tensormap(&tm.w);
    prefetch_tensormap(&tm.sa);
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_u32(sm.tmem_base), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_base;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  float2 acc[C::kCols / 2];
#pragma unroll
  for (int j = 0; j < C::kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
  if (warp == C::kWarpTma) {
    // ------------------------------------------------------------ producer
    const bool issuer = elect_one();
    const uint32_t st0 = smem_u32(sm.stages);
    bool ok = true;
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % C::kStages;
      ok = it < C::kStages || warp_wait_all(P.status, sm.abort_flag, &sm.empty[s], ((it / C::kStages) & 1) ^ 1);
      if (!ok) break;
      if (issuer) {
        const uint32_t st = st0 + s * C::kStageBytes, bar = smem_u32(&sm.full[s]);
        mbar_arrive_expect_tx(bar, C::kTx);
        tma_load_2d(st, &tm.w, bar, (kb0 + it) * 128, nt * 128);
        tma_load_2d(st + kGtWBytes, &tm.a, bar, (kb0 + it) * 128, mt * TN);
        tma_load_2d(st + kGtWBytes + C::kABytes, &tm.sa, bar, mt * TN, kb0 + it);
      }
      __syncwarp();
    }
    if (!ok && lane == 0)   // gave up: the copies in flight land before the CTA ends
      for (int j = max(0, it - C::kStages); j < it; ++j)
        mbar_wait(smem_u32(&sm.full[j % C::kStages]), (j / C::kStages) & 1);
    __syncwarp();
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = umma_idesc_e4m3(128, TN);
    const uint64_t desc0 = umma_desc_sw128(smem_u32(sm.stages), 1024);
    const bool issuer = elect_one();
    bool ok = true;
    for (int it = 0; it < nk && ok; ++it) {
      const int s = it % C::kStages, a = it % kGtAcc;
      ok = lanes_wait(P.status, sm.abort_flag, &sm.full[s], (it / C::kStages) & 1) &&
           (it < kGtAcc || lanes_wait(P.status, sm.abort_flag, &sm.acc_empty[a], ((it / kGtAcc) & 1) ^ 1));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (issuer) {
        const uint64_t dw = desc0 + (uint32_t)(s * (C::kStageBytes >> 4));   // the address field counts 16 bytes
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_e4m3(tmem + a * TN, dw + 2 * k, dw + (kGtWBytes >> 4) + 2 * k, idesc, k != 0);
        umma_commit(smem_u32(&sm.acc_full[a]));
        umma_commit(smem_u32(&sm.empty[s]));
      }
      __syncwarp();
    }
    if (issuer) {   // every product has landed before TMEM is released
      umma_commit(smem_u32(&sm.done[0]));
      if (!mbar_wait(smem_u32(&sm.done[0]), 0)) {
        record_status(P.status, kStatusTimeout);
        *sm.abort_flag = 1;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int c0 = (warp >> 2) * C::kCols;               // this warp's first token
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
    const float *sw = P.w_scale + (int64_t)kb0 * P.w_scale_ld + nt;
    // the weights' scales of 32 blocks, a block per lane; the next 32 are on their way
    float ws = lane < nk ? sw[lane * P.w_scale_ld] : 0.f, ws_next = 0.f;
    bool ok = true;
    for (int it = 0; it < nk && ok; ++it) {
      const int s = it % C::kStages, a = it % kGtAcc;
      if ((it & 31) == 0) {
        if (it > 0) ws = ws_next;
        ws_next = it + 32 + lane < nk ? sw[(it + 32 + lane) * P.w_scale_ld] : 0.f;
      }
      const float w = __shfl_sync(0xffffffffu, ws, it & 31);
      const float2 w2 = make_float2(w, w);
      ok = lanes_wait(P.status, sm.abort_flag, &sm.acc_full[a], (it / kGtAcc) & 1) &&
           lanes_wait(P.status, sm.abort_flag, &sm.full[s], (it / C::kStages) & 1);   // the scales (there by now)
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float4 *sa = reinterpret_cast<const float4 *>(sm.stages + s * C::kStageBytes + kGtWBytes + C::kABytes) + c0 / 4;
      float v[C::kCols / 32][32];
#pragma unroll
      for (int c = 0; c < C::kCols / 32; ++c) tmem_ld32_issue(lane_addr + a * TN + c * 32, v[c]);
#pragma unroll
      for (int c = 0; c < C::kCols / 32; ++c) {
        tmem_wait_ld32(v[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 f = sa[c * 8 + j];
          float2 *o = acc + c * 16 + 2 * j;
          o[0] = ffma2(make_float2(v[c][4 * j], v[c][4 * j + 1]), fmul2(make_float2(f.x, f.y), w2), o[0]);
          o[1] = ffma2(make_float2(v[c][4 * j + 2], v[c][4 * j + 3]), fmul2(make_float2(f.z, f.w), w2), o[1]);
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
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  const bool wide = (P.ldo * (P.out_f32 ? 4 : 2)) % 16 == 0 && (reinterpret_cast<uintptr_t>(P.out) & 15) == 0;
  const int m0 = mt * TN, nm = min(TN, P.m - m0);
  // the sums, [token][128] in shared memory: this CTA's alone, or a share of the cluster's in rank order
  float *part = reinterpret_cast<float *>(sm.stages);
  if (warp < C::kEpi && *sm.abort_flag == 0) {
    const int c0 = (warp >> 2) * C::kCols, f = threadIdx.x & 127;
#pragma unroll
    for (int j = 0; j < C::kCols / 2; ++j) {
      part[(c0 + 2 * j) * 128 + f] = acc[j].x;
      part[(c0 + 2 * j + 1) * 128 + f] = acc[j].y;
    }
  }
  if (P.split > 1) cluster_sync();
  else __syncthreads();
  const int j0 = rank * nm / P.split, j1 = (rank + 1) * nm / P.split;
  const int n = nt * 128 + lane * 4;
  constexpr int kWarps = C::kThreads / 32;
#pragma unroll 2
  for (int j = j0 + warp; j < j1; j += kWarps) {
    const uint32_t at = smem_u32(part + j * 128 + lane * 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (P.split == 1) {
      v = *reinterpret_cast<const float4 *>(part + j * 128 + lane * 4);
    } else {
      float4 x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < P.split) x[r] = ld_cluster4(at, r);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < P.split) {
          v.x += x[r].x;
          v.y += x[r].y;
          v.z += x[r].z;
          v.w += x[r].w;
        }
    }
    if (n < P.n) gemm_store4(P, (int64_t)m0 + j, n, v, wide);
  }
  if (P.split > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

template <int TN>
cudaError_t launch_gt(const GemmMaps &tm, const GemmParams &p, cudaStream_t s) {
  auto kern = gemm_fp8_tokens_kernel<TN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, GtCfg<TN>::kBytes, done);
  if (e != cudaSuccess) return e;
  const int grid = p.n_tiles * p.m_tiles * p.split;
  e = p.split > 1 ? launch_pdl_cluster(kern, grid, GtCfg<TN>::kThreads, GtCfg<TN>::kBytes, p.split, s, tm, p)
                  : launch_pdl(kern, grid, GtCfg<TN>::kThreads, GtCfg<TN>::kBytes, s, tm, p);
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
