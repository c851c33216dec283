// rms_norm.cu -- root-mean-square norm with the residual's addition and an e4m3 output with one
// scale for each 128 columns: the step in front of the block's projections (and of KV Bridging,
// whose hidden states it writes).
//
//   h = x + residual;  residual_out = h;  y = h w / sqrt(mean(h^2) + eps)
//
// A CTA has 256 threads or more for a row (or several rows of fewer threads) and, in a long batch, goes
// from row to row, the next one's x and residual on their way while this one is worked on (32768 x 4096
// with e4m3 output, 0.96 GB: 145 us, 6.6 TB/s, the measured copy rate, in calls on the same tensors, and 168 in turn
// over three sets of them; 248 us with a CTA per row and no row ahead). A thread holds kChunks chunks of 8
// columns of h in registers, so x and the residual are read once. The sum of squares goes through warp shuffles
// and one word of shared memory per warp. 16 neighbouring threads hold 128 columns: the maximum that gives their
// scale takes four shuffles.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace hs2 {

namespace {

constexpr int kNormMaxThreads = 1024;  // threads per row, at most

// 8 columns as they lie in memory: bf16 in u[0], float32 in both
template <bool kF32>
struct Raw8 {
  uint4 u[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (kF32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) u[k] = q[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) u[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    if constexpr (kF32) {
      v[0] = make_float2(__uint_as_float(u[0].x), __uint_as_float(u[0].y));
      v[1] = make_float2(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
      v[2] = make_float2(__uint_as_float(u[1].x), __uint_as_float(u[1].y));
      v[3] = make_float2(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
    } else {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
  }
};

__device__ __forceinline__ void store8(void *p, int64_t i, bool f32, const float2 (&v)[4]) {
  if (f32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) =
        make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
  }
}

// the largest |v| of this thread's 8 columns
__device__ __forceinline__ float amax8(const float2 (&v)[4]) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) a = fmax3(a, fabsf(v[j].x), fabsf(v[j].y));
  return a;
}

// ... and of its 15 neighbours'
__device__ __forceinline__ float amax16(const float2 (&v)[4]) {
  float a = amax8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

// blockDim = (threads per row, 16 or a multiple of 32; rows per CTA). kAhead: the next row is fetched
// while this one is worked on.
template <int kChunks, int kRes, bool kWF32, int kMaxThreads, bool kAhead>
__global__ void __launch_bounds__(kMaxThreads)
    rms_norm_kernel(const __grid_constant__ NormParams P) {
  __shared__ float s_sum[2][kMaxThreads / 32];
  const int T = blockDim.x, tid = threadIdx.x, lane = (threadIdx.y * T + tid) & 31;
  const int warps = T >> 5;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  int64_t left = P.rows - row;                        // rows from this one on (the thread's own)
  int64_t base_left = P.rows - (int64_t)blockIdx.x * blockDim.y;   // the CTA's
  bool in_row[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) in_row[c] = (c * T + tid) * 8 < P.d;
  // this thread's first column of the row at hand, in each array
  constexpr int kRB = kRes == kResF32 ? 4 : 2;
  const uint8_t *xp = static_cast<const uint8_t *>(P.x) + (row * P.x_stride + tid * 8) * 2;
  const uint8_t *rp = static_cast<const uint8_t *>(P.res) + (row * P.res_stride + tid * 8) * kRB;
  uint8_t *rop = static_cast<uint8_t *>(P.res_out) + (row * P.res_stride + tid * 8) * kRB;
  const int ob = P.out_f32 ? 4 : 2;
  uint8_t *op = static_cast<uint8_t *>(P.out) + (row * P.out_stride + tid * 8) * ob;
  uint8_t *cp = P.codes + row * P.codes_stride + tid * 8;
  float *sp = P.scales + (int64_t)(tid >> 4) * P.scale_ld + row;
  Raw8<false> xr[kChunks];
  Raw8<kRes == kResF32> rr[kRes == kResNone ? 1 : kChunks];
  const auto fetch = [&](bool live) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const bool in = live && in_row[c];
      if (in) xr[c].load(xp, (int64_t)c * T * 8);
      else xr[c].zero();
      if (kRes != kResNone) {
        if (in) rr[c].load(rp, (int64_t)c * T * 8);
        else rr[c].zero();
      }
    }
    xp += step * P.x_stride * 2;
    rp += step * P.res_stride * kRB;
  };
  griddep_launch_dependents();
  griddep_wait();
  Raw8<kWF32> w[kAhead ? kChunks : 1];
  if (kAhead) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      w[c].zero();
      if (in_row[c]) w[c].load(P.w, (c * T + tid) * 8);
    }
    fetch(left > 0);
  }
  for (int turn = 0; base_left > 0; base_left -= step, turn ^= 1) {
    const bool live = left > 0;
    if (!kAhead) fetch(live);
    float2 h[kChunks][4];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      xr[c].get(h[c]);
      if (kRes != kResNone) {
        float2 r[4];
        rr[c].get(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[c][j] = fadd2(h[c][j], r[j]);
      }
    }
    left -= step;
    // (residual_out may be residual or x: the rows ahead are others)
    if (kAhead && base_left > step) fetch(left > 0);
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (kRes != kResNone && live && in_row[c]) store8(rop, (int64_t)c * T * 8, kRes == kResF32, h[c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = ffma2(h[c][j], h[c][j], s2);
    }
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (T > 16) ss += __shfl_xor_sync(0xffffffffu, ss, 16);
    if (warps > 1) {
      // one barrier a row: a warp that is ahead writes the other half
      float *s = s_sum[turn] + threadIdx.y * warps;
      if (lane == 0) s[tid >> 5] = ss;
      __syncthreads();
      ss = lane < warps ? s[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float inv = __frsqrt_rn(fmaf(ss, P.inv_d, P.eps));
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const bool in = live && in_row[c];
      if (!kAhead && in) w[0].load(P.w, (c * T + tid) * 8);
      float2 y[4];
      w[kAhead ? c : 0].get(y);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = in ? fmul2(fmul2(h[c][j], inv2), y[j]) : make_float2(0.f, 0.f);
      if (P.out && in) store8(op, (int64_t)c * T * 8, P.out_f32, y);
      if (P.codes) {
        const float sc = fp8_block_scale(amax16(y));
        if (in) {
          *reinterpret_cast<uint2 *>(cp + c * T * 8) = fp8_codes8(y, sc, fp8_row_recip(sc));
          if ((lane & 15) == 0) sp[(int64_t)(c * (T >> 4)) * P.scale_ld] = sc;
        }
      }
    }
    rop += step * P.res_stride * kRB;
    op += step * P.out_stride * ob;
    cp += step * P.codes_stride;
    sp += step;
  }
}

// ------------------------------------------------------------------ quantiser

constexpr int kQuThreads = 256;
constexpr int kQuGroups = 4;          // 1 x 128 blocks per 16 threads, all loads first

// 1 x 128 blocks: 16 threads per block, kQuGroups blocks each, in rows one below the other. A CTA has 2^tile_shift
// column blocks of kQuThreads / 16 * kQuGroups >> tile_shift rows. The four maxima meet by a reduction that leaves
// each with a quarter of the threads, which form its scale and reciprocal and hand them round (32768 x 4096 75
// us; with every thread reducing and forming all four, and blocks numbered by a division, 97).
__global__ void __launch_bounds__(kQuThreads)
    fp8_quantize_rows_kernel(const __grid_constant__ QuantParams P) {
  static_assert(kQuGroups == 4, "the reduction below");
  const unsigned ct = (((P.cols + 127) >> 7) + (1 << P.tile_shift) - 1) >> P.tile_shift;
  const unsigned rt = blockIdx.x / ct;
  const int grp = threadIdx.x >> 4, sub = threadIdx.x & 15, lane = threadIdx.x & 31;
  const int j = (int)((blockIdx.x - rt * ct) << P.tile_shift) + (grp & ((1 << P.tile_shift) - 1));
  const int col = j * 128 + sub * 8;
  const int step = kQuThreads / 16 >> P.tile_shift;                       // rows between a thread's blocks
  const int64_t row = (int64_t)rt * step * kQuGroups + (grp >> P.tile_shift);
  const int left = col < P.cols ? (int)min(P.rows - row, (int64_t)INT32_MAX) : 0;   // rows from its first on
  griddep_launch_dependents();
  griddep_wait();
  Raw8<false> raw[kQuGroups];
#pragma unroll
  for (int u = 0; u < kQuGroups; ++u) {
    if (u * step < left) raw[u].load(P.x, (row + u * step) * P.x_stride + col);
    else raw[u].zero();
  }
  float a[kQuGroups];
#pragma unroll
  for (int u = 0; u < kQuGroups; ++u) {
    float2 v[4];
    raw[u].get(v);
    a[u] = amax8(v);
  }
  const bool b0 = sub & 1, b1 = sub & 2;
  float k0 = b0 ? a[2] : a[0], k1 = b0 ? a[3] : a[1];                     // blocks 2 b0, 2 b0 + 1
  k0 = fmaxf(k0, __shfl_xor_sync(0xffffffffu, b0 ? a[0] : a[2], 1));
  k1 = fmaxf(k1, __shfl_xor_sync(0xffffffffu, b0 ? a[1] : a[3], 1));
  float k = fmaxf(b1 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2));   // block 2 b0 + b1
  k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, 4));
  k = fmaxf(k, __shfl_xor_sync(0xffffffffu, k, 8));
  const float sc = fp8_block_scale(k), rc = fp8_row_recip(sc);
  if (sub < 4) {
    const int u = 2 * b0 + b1;
    const bool any = j * 128 < P.cols && row + u * step < P.rows;
    if (any) P.scales[(int64_t)j * P.scale_ld + row + u * step] = sc;
  }
#pragma unroll
  for (int u = 0; u < kQuGroups; ++u) {
    const int src = (lane & 16) + (u >> 1) + 2 * (u & 1);
    const float s = __shfl_sync(0xffffffffu, sc, src), r = __shfl_sync(0xffffffffu, rc, src);
    float2 v[4];
    raw[u].get(v);
    if (u * step < left)
      *reinterpret_cast<uint2 *>(P.codes + (row + u * step) * P.codes_stride + col) = fp8_codes8(v, s, r);
  }
}

// 128 x 128 blocks: one CTA per block, 8 chunks of 8 columns per thread, so that x is read once (weights of
// 16384 x 4096: 45.4 us, 4.4 TB/s, bounded by the CTAs' starts: each loads, meets once and stores; 4096 x 4096: 14.2).
// Weights are quantised once, when they are loaded.
__global__ void __launch_bounds__(kQuThreads)
    fp8_quantize_blocks_kernel(const __grid_constant__ QuantParams P) {
  __shared__ float s_max[kQuThreads / 32];
  const int kb = (P.cols + 127) >> 7;
  const int64_t ib = blockIdx.x / kb;
  const int jb = (int)(blockIdx.x - ib * kb);
  const int col = jb * 128 + (threadIdx.x & 15) * 8;
  griddep_launch_dependents();
  griddep_wait();
  Raw8<false> raw[8];
  float a = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = ib * 128 + u * 16 + (threadIdx.x >> 4);
    if (row < P.rows && col < P.cols) raw[u].load(P.x, row * P.x_stride + col);
    else raw[u].zero();
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float2 v[4];
    raw[u].get(v);
    a = fmaxf(a, amax8(v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuThreads / 32; ++i) a = fmaxf(a, s_max[i]);
  const float sc = fp8_row_scale(a), rc = fp8_row_recip(sc);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = ib * 128 + u * 16 + (threadIdx.x >> 4);
    float2 v[4];
    raw[u].get(v);
    if (row < P.rows && col < P.cols)
      *reinterpret_cast<uint2 *>(P.codes + row * P.codes_stride + col) = fp8_codes8(v, sc, rc);
  }
  if (threadIdx.x == 0) P.scales[(int64_t)jb * P.scale_ld + ib] = sc;
}

template <class Kernel, class Params>
cudaError_t launch2d(Kernel kernel, int64_t grid, dim3 block, cudaStream_t s, const Params &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

namespace {
template <int kChunks, int kMaxThreads, bool kAhead = true>
cudaError_t launch_norm(const NormParams &p, int64_t grid, dim3 block, cudaStream_t s) {
  const int res = !p.res ? kResNone : p.res_f32 ? kResF32 : kResBf16;
  const auto with = [&](auto res_c, auto w_c) {
    return launch2d(rms_norm_kernel<kChunks, decltype(res_c)::value, decltype(w_c)::value, kMaxThreads, kAhead>, grid,
                    block, s, p);
  };
  const auto weights = [&](auto res_c) { return p.w_f32 ? with(res_c, std::true_type{}) : with(res_c, std::false_type{}); };
  if (res == kResNone) return weights(std::integral_constant<int, kResNone>{});
  if (res == kResBf16) return weights(std::integral_constant<int, kResBf16>{});
  return weights(std::integral_constant<int, kResF32>{});
}
}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, int sms, cudaStream_t s) {
  const int chunks = (p.d + 7) / 8;
  // Few rows: a chunk per thread, as many threads as that takes. Many rows: CTAs that go from row to row, two or
  // four chunks per thread, whose loads are in flight together. Four from 448 chunks on (32768 x 4096 with a
  // bf16 residual 147 us, 159 with two; x 2560 101 with two, 110 with four), but for a float32 residual, which
  // takes the registers (8192 x 8192 142 us with two, 167 with four), and from 8 rows an SM (300 x 4096 3.6 us with
  // two, 4.3 with four). At most 512 threads, since a row ahead takes more than 64 registers (32768 x 5120: 190 us;
  // 294 with two chunks and 64 registers).
  int per = p.rows <= 2 * sms || chunks <= 64 ? 1 : chunks >= 448 && p.rows > 8 * sms && !(p.res && p.res_f32) ? 4 : 2;
  while ((chunks + per - 1) / per > (per == 1 ? kNormMaxThreads : 512) && per < 4) per *= 2;
  const int t = chunks <= 16 ? 16 : ((chunks + per - 1) / per + 31) / 32 * 32;
  int rows_per = chunks <= 16 ? 2 : 1;
  while (per < 4 && t * rows_per * 2 <= 256 && (int64_t)rows_per * 2 <= p.rows / sms) rows_per *= 2;
  const dim3 block(t, rows_per);
  const int64_t ctas = (p.rows + rows_per - 1) / rows_per;
  // threads per SM that the registers let stay: a CTA beyond them starts when others have ended (500,000 x 128 with
  // bf16 residual and codes 72 us, 94 at 1280)
  const int threads = per == 4 ? 512 : per == 1 ? 1024 : t * rows_per > 256 ? 704 : p.res && p.res_f32 ? 512 : 768;
  const int64_t grid = std::min<int64_t>(ctas, (int64_t)sms * std::max(1, threads / (t * rows_per)));
  if (t * rows_per <= 256) {
    switch (per) {
      case 1: return launch_norm<1, 256>(p, grid, block, s);
      case 2: return launch_norm<2, 256>(p, grid, block, s);
      case 4: return launch_norm<4, 256>(p, grid, block, s);
    }
  } else if (t <= 512 && per > 1) {
    if (per == 2) return launch_norm<2, 512>(p, grid, block, s);
    return launch_norm<4, 512>(p, grid, block, s);
  } else if (t <= kNormMaxThreads) {
    if (per == 1) return launch_norm<1, kNormMaxThreads>(p, grid, block, s);
    if (per == 4) return launch_norm<4, kNormMaxThreads, false>(p, grid, block, s);   // 64 registers a thread
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_quantize(const QuantParams &p, cudaStream_t s) {
  const int64_t kb = (p.cols + 127) / 128;
  const dim3 block(kQuThreads);
  if (p.block_rows == 1) {
    // the most column blocks per CTA, up to 16, that leave at most an eighth of the threads without one
    QuantParams q = p;
    q.tile_shift = 4;
    while (q.tile_shift && ((kb + (1 << q.tile_shift) - 1) >> q.tile_shift << q.tile_shift) * 8 > kb * 9) --q.tile_shift;
    const int64_t rows = kQuThreads / 16 * kQuGroups >> q.tile_shift;
    const int64_t grid = ((kb + (1 << q.tile_shift) - 1) >> q.tile_shift) * ((p.rows + rows - 1) / rows);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch2d(fp8_quantize_rows_kernel, grid, block, s, q);
  }
  const int64_t grid = (p.rows + 127) / 128 * kb;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch2d(fp8_quantize_blocks_kernel, grid, block, s, p);
}

}  // namespace hs2
