// gemm_fp8_pair.cu -- the e4m3 product with block scales for many tokens: 256 x 256 tiles of the
// result, each by a pair of CTAs (a cluster of two on neighbouring SMs, tcgen05 cta_group::2).
//
// A CTA of the pair holds 128 tokens' codes and 128 output features' codes of each 128-wide
// block along k (32 KB per stage): the pair's product of 256 x 256 reads each byte from L2 once
// per 256 rows of the other operand, which the e4m3 rate needs (a 128 x 128 tile would ask L2
// for twice the bytes). Its accumulator is 256 TMEM columns in each CTA, tokens on the lanes; two of
// them alternate. The scales change with every block, so the epilogue warps read each block's
// accumulator, scale it (one factor per thread: a token's scale times its 128 features') and add it
// to float32 sums in registers, while the tensor cores work on the next block.
//   warp 9      TMA producer of its CTA's stages; bytes of both CTAs complete on the leader's barrier
//   warp 8      TMEM owner; in the leader (rank 0) also the MMA issuer for both
//   warps 10, 11  nothing (the register split goes by groups of four warps)
//   warps 0..7  epilogue: warp w has lanes 32 (w % 4) .. + 31 and features 128 (w / 4) .. + 127
// What bounds it: 32768 x 4096 x 4096 takes 505 to 525 us in ten calls or so (2.1 to 2.2 PFLOP/s, 0.63 to 0.65 of
// twice the measured bf16 rate), 548 in 200 calls, about 600 (1.8 PFLOP/s) under the power cap of a long run. The products and loads alone (accumulators
// handed back unread) take 411 us, reading and adding them (with a quarter of the products) 441 us: two
// accumulators, all of TMEM, do not hide one behind the other altogether. The epilogue warps are busy
// throughout: of about 830 clocks a block 190 go to the barrier, 70 to the first columns, 390 to the rest. No
// faster were halves of 128 features handed over by themselves (515 against 505 us), 32 columns a load
// (518 against 523) and the next accumulator's barrier tested, or its first columns fetched, ahead (spills).
// Persistent over the tiles, features fastest: the CTAs at work share a few token tiles and the
// weights, which stay in L2. Results pass through shared memory, a 4 KB square per warp, so that
// rows are stored in 128-byte pieces.
#include "common.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace hs2 {

namespace {

constexpr int kGpWarpMma = 8, kGpWarpTma = 9, kGpThreads = 12 * 32;
// Registers: 384 threads x 168 at launch = 64,512 = 256 epilogue threads x 216 + 128 others x 72.
constexpr int kGpRegsEpilogue = 216, kGpRegsOther = 72;
static_assert(256 * kGpRegsEpilogue + 128 * kGpRegsOther <= kGpThreads * 168, "register split");
constexpr int kGpTile = 256;
constexpr int kGpHalf = 128 * 128;               // a CTA's codes of one operand and block
constexpr int kGpStageBytes = 2 * kGpHalf;
constexpr int kGpStages = 6;
constexpr int kGpOutBytes = 4096;                // per epilogue warp: 32 rows x 128 bytes
constexpr size_t kGpBytes = 1024 + (size_t)kGpStages * kGpStageBytes + 8 * kGpOutBytes + (2 * kGpStages + 5) * 8 + 16;
static_assert(kGpBytes <= 227 * 1024, "shared memory");

struct GpSmem {
  uint8_t *stages, *out;
  uint64_t *full, *empty, *acc_full, *acc_empty, *done;
  uint32_t *tmem_base;
  volatile int *abort_flag;
  __device__ explicit GpSmem(uint8_t *raw) {
    stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    out = stages + kGpStages * kGpStageBytes;
    full = reinterpret_cast<uint64_t *>(out + 8 * kGpOutBytes);
    empty = full + kGpStages;
    acc_full = empty + kGpStages;
    acc_empty = acc_full + 2;
    done = acc_empty + 2;
    tmem_base = reinterpret_cast<uint32_t *>(done + 1);
    abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
  }
};

__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

// 2-D tile load of a CTA pair: into this CTA's memory, completing on a barrier of either CTA
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t cluster_bar,
                                                 int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate));
}

// Arrives once on the barrier at this offset in both CTAs when the pair's products so far are done.
__device__ __forceinline__ void umma_commit_pair(uint32_t mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar),
      "h"((uint16_t)3)
      : "memory");
}

// Relaxed: what the arrival hands over is tensor memory, ordered by the tcgen05 fence before it; a
// release at cluster scope waits for the thread's global loads (32768 x 4096 x 4096: 1,247 us with it, 815
// without).
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Eight elements of a row that starts anywhere, by pairs, behind the first element where that is an odd one.
// (13,674 x 973 x 128 in bf16: 18.5 us, with a row's elements by neighbouring lanes, one at a time, 30.)
__device__ __forceinline__ void store_piece(__nv_bfloat16 *o, uint4 u) {
  const bool odd = reinterpret_cast<uintptr_t>(o) & 2;
  uint32_t *p = reinterpret_cast<uint32_t *>(o + odd);
  p[0] = odd ? __byte_perm(u.x, u.y, 0x5432) : u.x;
  p[1] = odd ? __byte_perm(u.y, u.z, 0x5432) : u.y;
  p[2] = odd ? __byte_perm(u.z, u.w, 0x5432) : u.z;
  if (odd) {
    uint16_t *h = reinterpret_cast<uint16_t *>(o);
    h[0] = (uint16_t)u.x;
    h[7] = (uint16_t)(u.w >> 16);
  } else {
    p[3] = u.w;
  }
}

// One warp's 32 rows x 128 bytes through its square of shared memory: lane = row writes its 8
// pieces of 16 bytes (swizzled), then each row leaves by 8 neighbouring lanes. `cols`: elements of
// the row that exist.
template <class T>
__device__ __forceinline__ void store_square(uint8_t *sq, const uint4 (&v)[8], T *out, int64_t ldo, int rows, int cols,
                                             bool wide) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(sq + sw128(lane, c * 16)) = v[c];
  __syncwarp();
  constexpr int per = 16 / sizeof(T);
  if (wide) {
    const int c = lane & 7;
#pragma unroll
    for (int r = lane >> 3; r < 32; r += 4)
      if (r < rows) {
        const uint4 u = *reinterpret_cast<const uint4 *>(sq + sw128(r, c * 16));
        T *o = out + r * ldo + c * per;
        if ((c + 1) * per <= cols) {
          *reinterpret_cast<uint4 *>(o) = u;
        } else {
          const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
          for (int i = 0; i < per; ++i)
            if (c * per + i < cols) o[i] = e[i];
        }
      }
  } else if constexpr (sizeof(T) == 4) {   // a row per instruction
    for (int r = 0; r < min(rows, 32); ++r)
      if (lane < cols) out[r * ldo + lane] = *reinterpret_cast<const T *>(sq + sw128(r, lane * 4));
  } else {
    const int c = lane & 7, left = cols - c * per;
    T *o = out + (lane >> 3) * ldo + c * per;
#pragma unroll 1
    for (int r = lane >> 3; r < min(rows, 32); r += 4, o += 4 * ldo) {
      const uint4 u = *reinterpret_cast<const uint4 *>(sq + sw128(r, c * 16));
      if (left >= per) {
        store_piece(o, u);
      } else {
        const T *e = reinterpret_cast<const T *>(sq + sw128(r, c * 16));
#pragma unroll 1
        for (int i = 0; i < left; ++i) o[i] = e[i];
      }
    }
  }
}

__global__ void __launch_bounds__(kGpThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ GemmMaps tm, const __grid_constant__ GemmParams P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  GpSmem sm(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;                 // in the pair
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int n_tiles = P.n_tiles * P.m_tiles, kb = P.kb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGpStages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&sm.acc_full[a]), 1);
      mbar_init(smem_u32(&sm.acc_empty[a]), 16);   // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&sm.done[0]), 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kGpWarpTma && lane == 0) {
    prefetch_tensormap(&tm.a);
    prefetch_tensormap(&tm.w);
  }
  if (warp == kGpWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(sm.tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_base;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGpRegsOther));
  if (warp == kGpWarpTma) {
    // ------------------------------------------------------------ producer
    const bool issuer = elect_one();
    const uint32_t bar0 = map_rank(smem_u32(&sm.full[0]), 0), st0 = smem_u32(sm.stages);
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < n_tiles && ok; tile += stride) {
      const int nt = tile % P.n_tiles, mt = tile / P.n_tiles;
      for (int b = 0; b < kb; ++b, ++it) {
        const int s = it % kGpStages;
        ok = it < kGpStages || warp_wait_all(P.status, sm.abort_flag, &sm.empty[s], ((it / kGpStages) & 1) ^ 1);
        if (!ok) break;
        if (issuer) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[s]), 2 * kGpStageBytes);
          tma_load_2d_pair(st0 + s * kGpStageBytes, &tm.a, bar0 + 8 * s, b * 128, mt * kGpTile + rank * 128);
          tma_load_2d_pair(st0 + s * kGpStageBytes + kGpHalf, &tm.w, bar0 + 8 * s, b * 128, nt * kGpTile + rank * 128);
        }
        __syncwarp();
      }
    }
    // The leader's products hand the last stages back in both CTAs: each sees these arrivals before it ends.
    for (int j = max(0, it - kGpStages); j < it && ok; ++j)
      ok = warp_wait_all(P.status, sm.abort_flag, &sm.empty[j % kGpStages], (j / kGpStages) & 1);
    if (!ok) {   // gave up: copies in flight land before the CTA ends (they take microseconds)
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 1000000ull) {}
    }
    __syncwarp();
  } else if (warp == kGpWarpMma && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    // The warp runs the loop as one and an elected lane issues: the operands stay warp-uniform.
    const uint32_t idesc = umma_idesc_e4m3(kGpTile, kGpTile);
    const uint64_t desc0 = umma_desc_sw128(smem_u32(sm.stages), 1024);
    const bool issuer = elect_one();
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < n_tiles && ok; tile += stride) {
      for (int b = 0; b < kb; ++b, ++it) {
        const int s = it % kGpStages, a = it & 1;
        ok = lanes_wait(P.status, sm.abort_flag, &sm.full[s], (it / kGpStages) & 1) &&
             (it < 2 || lanes_wait(P.status, sm.abort_flag, &sm.acc_empty[a], ((it >> 1) & 1) ^ 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t da = desc0 + (uint32_t)(s * (kGpStageBytes >> 4));   // the address field counts 16 bytes
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_e4m3_pair(tmem + a * 256, da + 2 * k, da + (kGpHalf >> 4) + 2 * k, idesc, k != 0);
          umma_commit_pair(smem_u32(&sm.acc_full[a]));
          umma_commit_pair(smem_u32(&sm.empty[s]));
        }
        __syncwarp();
      }
    }
    if (issuer) {   // every product has landed before TMEM is released
      umma_commit_pair(smem_u32(&sm.done[0]));
      if (!mbar_wait(smem_u32(&sm.done[0]), 0)) {
        record_status(P.status, kStatusTimeout);
        *sm.abort_flag = 1;
      }
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGpRegsEpilogue));
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
    const uint32_t freed[2] = {map_rank(smem_u32(&sm.acc_empty[0]), 0), map_rank(smem_u32(&sm.acc_empty[1]), 0)};
    uint8_t *sq = sm.out + warp * kGpOutBytes;
    const bool wide = (P.ldo * (P.out_f32 ? 4 : 2)) % 16 == 0 && (reinterpret_cast<uintptr_t>(P.out) & 15) == 0;
    int it = 0;
    bool ok = true;
    for (int tile = first; tile < n_tiles && ok; tile += stride) {
      const int nt = tile % P.n_tiles, mt = tile / P.n_tiles;
      const int m0 = mt * kGpTile + rank * 128 + quad * 32, n0 = nt * kGpTile + half * 128;
      // scales: this token's, and the features' (clamped where neither exists)
      const float *sa = P.a_scale + min(m0 + lane, P.m - 1);
      const float *sw = P.w_scale + min(n0, P.n - 1) / 128;
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      // four blocks' scales are loaded while the four before are used: a load's register that is
      // moved, or multiplied, too early waits for L2 (688 us with the next block's alone, 584 so)
      float fa[4], fw[4], na[4], nw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = min(i, kb - 1);
        fa[i] = sa[b * P.a_scale_ld];
        fw[i] = sw[b * P.w_scale_ld];
      }
      for (int b0 = 0; b0 < kb && ok; b0 += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = min(b0 + 4 + i, kb - 1);
          na[i] = sa[b * P.a_scale_ld];
          nw[i] = sw[b * P.w_scale_ld];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (b0 + i < kb && ok) {
            const int a = it & 1;
            ok = warp_wait_all(P.status, sm.abort_flag, &sm.acc_full[a], (it >> 1) & 1);
            tc_fence_after();
            const float s0 = fa[i] * fw[i];
            const float2 sc = make_float2(s0, s0);
            uint32_t v[2][16];   // 16 columns are scaled and added while the next 16 are on their way
            tmem_ld16_issue(lane_addr + a * 256, v[0]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              tmem_wait_ld16(v[q & 1]);
              if (q < 7) {
                tmem_ld16_issue(lane_addr + a * 256 + (q + 1) * 16, v[(q + 1) & 1]);
              } else {   // all columns are in registers: the accumulator is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(freed[a]);
              }
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[q * 8 + j] = ffma2(make_float2(__uint_as_float(v[q & 1][2 * j]), __uint_as_float(v[q & 1][2 * j + 1])),
                                       sc, acc[q * 8 + j]);
            }
            ++it;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fa[i] = na[i];
          fw[i] = nw[i];
        }
      }
      if (!ok) break;
      const int rows = P.m - m0, cols = P.n - n0;
      if (rows <= 0 || cols <= 0) continue;
      if (P.out_f32) {
        float *o = static_cast<float *>(P.out) + (int64_t)m0 * P.ldo + n0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 x = acc[q * 16 + 2 * c], y = acc[q * 16 + 2 * c + 1];
            v[c] = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
          }
          if (cols > q * 32) store_square<float>(sq, v, o + q * 32, P.ldo, rows, cols - q * 32, wide);
        }
      } else {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(P.out) + (int64_t)m0 * P.ldo + n0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 *x = acc + q * 32 + 4 * c;
            v[c] = make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                              pack_bf16(x[3].x, x[3].y));
          }
          if (cols > q * 64) store_square<__nv_bfloat16>(sq, v, o + q * 64, P.ldo, rows, cols - q * 64, wide);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // The leader's last commit arrives here too, and a cluster barrier does not order it: the memory of a CTA that
  // has ended may be the next kernel's already.
  if (rank == 1 && threadIdx.x == 0 && !mbar_wait(smem_u32(&sm.done[0]), 0)) record_status(P.status, kStatusTimeout);
  __syncthreads();
  cluster_sync_all();   // the pair's products and copies are over in both CTAs
  if (warp == kGpWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

cudaError_t launch_gemm_fp8_pair(const GemmMaps &tm, const GemmParams &p, int pairs, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(gemm_fp8_pair_kernel, kGpBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(gemm_fp8_pair_kernel, 2 * pairs, kGpThreads, kGpBytes, 2, s, tm, p);
}

}  // namespace hs2
