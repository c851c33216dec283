// rms_norm.cu -- root-mean-square norm with the residual's addition and an e4m3 output with one
// scale for each 128 columns: the step in front of the block's projections (and of KV Bridging,
// whose hidden states it writes).
//
//   h = x + residual;  residual_out = h;  y = h w / sqrt(mean(h^2) + eps)
//
// One CTA per row (several rows per CTA when a row needs fewer than 256 threads): a thread holds
// kChunks chunks of 8 columns of h in registers, so x and the residual are read once. The sum of
// squares goes through warp shuffles and one word of shared memory per warp. 16 neighbouring
// threads hold 128 columns: the maximum that gives their scale takes four shuffles.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace hs2 {

namespace {

constexpr int kNormMaxThreads = 512;   // threads per row, at most

__device__ __forceinline__ void load8(const void *p, int64_t i, bool f32, float (&v)[8]) {
  if (f32) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void *p, int64_t i, bool f32, const float (&v)[8]) {
  if (f32) {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
}

// the largest |v| of this thread's 8 columns and its 15 neighbours'
__device__ __forceinline__ float amax16(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) a = fmax3(a, fabsf(v[j]), fabsf(v[j + 1]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// blockDim = (threads per row, a multiple of 32; rows per CTA)
template <int kChunks>
__global__ void __launch_bounds__(kNormMaxThreads)
    rms_norm_kernel(const __grid_constant__ NormParams P) {
  __shared__ float s_sum[kNormMaxThreads / 32];
  const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < P.rows;
  griddep_launch_dependents();
  griddep_wait();
  float h[kChunks][8];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * T + tid) * 8;
    if (live && col < P.d) {
      load8(P.x, row * P.x_stride + col, false, h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = 0.f;
    }
  }
  if (P.res) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * T + tid) * 8;
      if (live && col < P.d) {
        float r[8];
        load8(P.res, row * P.res_stride + col, P.res_f32, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
      }
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {   // after every load: residual_out may be residual or x
      const int col = (c * T + tid) * 8;
      if (live && col < P.d) store8(P.res_out, row * P.res_stride + col, P.res_f32, h[c]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[c][j], h[c][j], ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const int warps = T >> 5;
  if (warps > 1) {
    float *s = s_sum + threadIdx.y * warps;
    if (lane == 0) s[tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < warps; ++i) ss += s[i];
  }
  const float inv = __frsqrt_rn(__fdiv_rn(ss, (float)P.d) + P.eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * T + tid) * 8;
    const bool in = live && col < P.d;
    float y[8] = {};
    if (in) {
      float w[8];
      load8(P.w, col, P.w_f32, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[c][j] * inv * w[j];
      if (P.out) store8(P.out, row * P.out_stride + col, P.out_f32, y);
    }
    if (P.codes) {
      const float sc = fp8_row_scale(amax16(y));
      if (in) {
        *reinterpret_cast<uint2 *>(P.codes + row * P.codes_stride + col) = fp8_codes8(y, sc, fp8_row_recip(sc));
        if ((lane & 15) == 0) P.scales[(int64_t)(col >> 7) * P.scale_ld + row] = sc;
      }
    }
  }
}

// ------------------------------------------------------------------ quantiser

constexpr int kQuThreads = 256;
constexpr int kQuGroups = 4;          // 1 x 128 blocks per 16 threads, all loads first

// 1 x 128 blocks: 16 threads per block, kQuGroups blocks each
__global__ void __launch_bounds__(kQuThreads)
    fp8_quantize_rows_kernel(const __grid_constant__ QuantParams P) {
  const int kb = (P.cols + 127) >> 7;
  const int64_t n = P.rows * kb;
  const int64_t g0 = (int64_t)blockIdx.x * (kQuThreads / 16 * kQuGroups) + (threadIdx.x >> 4);
  const int sub = threadIdx.x & 15;
  griddep_launch_dependents();
  griddep_wait();
  float v[kQuGroups][8];
#pragma unroll
  for (int u = 0; u < kQuGroups; ++u) {
    const int64_t g = g0 + u * (kQuThreads / 16);
    const int64_t row = g / kb;
    const int col = (int)(g - row * kb) * 128 + sub * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
    if (g < n && col < P.cols) load8(P.x, row * P.x_stride + col, false, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kQuGroups; ++u) {
    const int64_t g = g0 + u * (kQuThreads / 16);
    const int64_t row = g / kb;
    const int j = (int)(g - row * kb), col = j * 128 + sub * 8;
    const float sc = fp8_row_scale(amax16(v[u]));
    if (g < n && col < P.cols) {
      *reinterpret_cast<uint2 *>(P.codes + row * P.codes_stride + col) = fp8_codes8(v[u], sc, fp8_row_recip(sc));
      if (sub == 0) P.scales[(int64_t)j * P.scale_ld + row] = sc;
    }
  }
}

// 128 x 128 blocks: one CTA per block, 8 chunks of 8 columns per thread
__global__ void __launch_bounds__(kQuThreads)
    fp8_quantize_blocks_kernel(const __grid_constant__ QuantParams P) {
  __shared__ float s_max[kQuThreads / 32];
  const int kb = (P.cols + 127) >> 7;
  const int64_t ib = blockIdx.x / kb;
  const int jb = (int)(blockIdx.x - ib * kb);
  const int col = jb * 128 + (threadIdx.x & 15) * 8;
  griddep_launch_dependents();
  griddep_wait();
  float v[8][8];
  float a = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = ib * 128 + u * 16 + (threadIdx.x >> 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
    if (row < P.rows && col < P.cols) load8(P.x, row * P.x_stride + col, false, v[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(v[u][j]));
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
    if (row < P.rows && col < P.cols)
      *reinterpret_cast<uint2 *>(P.codes + row * P.codes_stride + col) = fp8_codes8(v[u], sc, rc);
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

cudaError_t launch_rms_norm(const NormParams &p, cudaStream_t s) {
  const int chunks = (p.d + 7) / 8;
  int per = 1;
  while ((chunks + per - 1) / per > kNormMaxThreads) per *= 2;
  const int t = ((chunks + per - 1) / per + 31) / 32 * 32;
  int rows_per = 1;
  while (t * rows_per * 2 <= 256 && (int64_t)rows_per * 2 <= p.rows / 148) rows_per *= 2;
  const dim3 block(t, rows_per);
  const int64_t grid = (p.rows + rows_per - 1) / rows_per;
  switch (per) {
    case 1: return launch2d(rms_norm_kernel<1>, grid, block, s, p);
    case 2: return launch2d(rms_norm_kernel<2>, grid, block, s, p);
    case 4: return launch2d(rms_norm_kernel<4>, grid, block, s, p);
    case 8: return launch2d(rms_norm_kernel<8>, grid, block, s, p);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_quantize(const QuantParams &p, cudaStream_t s) {
  const int64_t kb = (p.cols + 127) / 128;
  const dim3 block(kQuThreads);
  if (p.block_rows == 1) {
    const int64_t per = kQuThreads / 16 * kQuGroups;
    const int64_t grid = (p.rows * kb + per - 1) / per;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch2d(fp8_quantize_rows_kernel, grid, block, s, p);
  }
  const int64_t grid = (p.rows + 127) / 128 * kb;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch2d(fp8_quantize_blocks_kernel, grid, block, s, p);
}

}  // namespace hs2
