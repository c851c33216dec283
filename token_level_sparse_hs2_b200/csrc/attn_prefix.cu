// attn_prefix.cu -- full attention of a batch whose sequences share a prefix.
//
// With one K/V head, every (sequence, query token, head) row of the batch meets the same prefix
// rows, so the batch is one product with R = B n_q H rows and the prefix is read once for all
// of them. Each CTA takes two blocks of 128 consecutive rows (so that a K/V tile is read from L2
// once for 256 rows) and a contiguous range of their 128-row K/V tiles: the prefix's, then the
// own tiles of each sequence that has rows in the pair, up to the last position its rows see. Per
// tile i and block g:
//   S_g = Q_g . K_i^T            tcgen05.mma, both operands in shared memory, D in TMEM
//   P_g = exp2(c log2e S_g - m)  four softmax warps per block, one row per thread: the row's
//                                running maximum m, the exponentials, the row sum; P is written
//                                over S as bf16 pairs
//   O_g += P_g . V_i             tcgen05.mma, A = P (TMEM), B = V tile (MN-major)
// in two halves of 64 columns with an S buffer each: S of the next tile's half follows the product
// that frees its buffer, so the softmax warps find it ready. An own tile concerns the lanes of its
// sequence alone: blocks without such rows skip it, and the product leaves the other lanes of O
// untouched (its output-lane mask), so a row never meets another sequence's values. The reference
// maximum only moves when a tile's row maximum exceeds it by more than 8 (P <= 2^8); then the row of
// O is rescaled in TMEM. P is rounded to bf16, whatever the output's type (the tensor cores take no wider
// operand next to bf16 V; half a step, 2^-8 of each weight, averaged over the keys: a relative error of 1.6e-3 of
// the output, next to the 1.7e-3 of rounding that to bf16); m, the sums and O are float32. For an e4m3 cache f16
// could hold V's codes exactly too and the weights with three bits more; bf16 is taken for its range, since what
// is rounded there is the weight times the V scale, and a scale may be as small or large as float32 allows: f16
// would need a reference scale that moves as the maximum does.
//
// What bounds it: 4 x 128 queries x 32 heads behind 30,001 rows take 213 us in ten calls or so (1,185 TFLOP/s, 0.71
// of the measured bf16 rate), 225 in 200 calls and 246 (1,025 TFLOP/s) under the power cap of a long run; the tensor pipe is active 64 % of the time, its operand reads take 61 % of
// shared memory's cycles (S with 64 columns reads Q for every 64 keys), the special-function unit is
// busy 64 %: each waits for the others at times, and none alone is the limit. Slower were S in one piece of 128
// columns without a second buffer (267 us), 16 softmax warps with half the columns each (275 us), one
// MMA warp for both blocks, and part of the exponentials on the FMA pipe. Few rows behind a long prefix
// (32 x 1 behind 131,072: 66 us, 0.63 of the rate; with up to 2,048 own rows a sequence 80, three sets of
// inputs in turn) add 7 us of set-up and results and the merge's 5.
//
// An e4m3 cache (value = scale[t] code): S comes from the cached codes as they are (kind::f8f6f4), the
// query split into two e4m3 terms after a power of two per row that puts its largest element in
// [128, 256): hi is q rounded to e4m3, lo the remainder, exact for every element of at least 2^-9 of
// the row's largest and within 2^-17 of the largest for smaller ones. Four more warps widen the V codes to bf16 (exact). The K scale and the row's power
// of two multiply S, the V scale the weight before its rounding: they and the widening cost 403 us
// where bf16 takes 213. 32 x 1 queries behind 131,072 rows: 116 us, 106 without the K
// scales, 109 without the V scales, 101 without the widening, 82 without all three; bf16 66. No pipe is
// busy for half the time (tensor 39 %, shared memory's loads and stores 41 %, special functions 28 %): a
// warp's chain through a half tile is longer, 2,300 to 3,500 clocks. A quarter of the columns of four rows per
// thread, which reads a quarter of the scales, was slower (132 us), as were no turns (130); S in one piece (116),
// the next barriers tested ahead (118) and other orders of the widened codes (116) changed nothing.
//
// Rows of a tile behind the prefix's or the sequence's last never count, whatever the cache
// holds there: their columns are masked, and their V rows are zero (the prefix's tensor maps end at its
// last row; of an own tile they are cleared in shared memory), so that 0 x NaN does not arise.
//
// With more than one range per pair each CTA writes its rows' O and log-sum-exp, which
// prefix_merge_kernel joins.
#include "attn_pipeline.cuh"
#include "internal.h"
#include "tc05.cuh"

namespace hs2 {

namespace {

constexpr int kPxTile = 128;                       // prefix rows per tile
constexpr int kPxRows = 128;                       // (query, head) rows per block
constexpr int kPxTileBytes = kPxTile * 256;        // two [128][128 B] swizzled dim blocks
constexpr int kPxRawBytes = kPxTile * 128;         // a tile of codes
constexpr int kPxScaleSlots = 4;                   // e4m3: tiles whose scales are in flight
constexpr int kPxOutRow = 528, kPxOutWarp = 32 * kPxOutRow;   // a warp's rows of O on their way out: 512 bytes + 16
constexpr float kPxLazy = 8.f;
constexpr int kPxWarpMma = 8, kPxWarpTma = 10, kPxWarpScale = 11, kPxWarpWiden = 12;   // MMA: a warp per block
constexpr uint32_t kPxCols = 512;                  // S/P at 0 and 128, O at 256 and 384

template <int KV>
struct PxCfg {
  static constexpr bool kFp8 = KV == kKvFp8;
  static constexpr int kThreads = (kFp8 ? 16 : 12) * 32;
  // e4m3: 512 threads x 128 registers at launch = 256 softmax threads x 160 + 256 others x 96
  static constexpr int kRegsSoftmax = 160, kRegsOther = 96;
  static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= 512 * 128, "register split");
  // bf16: one ring of five tiles, K_0, V_0, K_1, V_1, ...; e4m3: three tiles of K codes, two of V codes and
  // two of widened V, and four tiles' scales
  static constexpr int kKSlots = kFp8 ? 3 : 5, kVSlots = kFp8 ? 2 : 5;
  static constexpr int kKBytes = kFp8 ? kPxRawBytes : kPxTileBytes;
  static constexpr int kRaw = kFp8 ? 2 : 0, kScaleSlots = kFp8 ? kPxScaleSlots : 1;
  static constexpr size_t kKOff = 2 * (size_t)kPxRows * 256;   // behind Q
  static constexpr size_t kVOff = kFp8 ? kKOff + (size_t)kKSlots * kPxRawBytes : kKOff;
  static constexpr size_t kRawOff = kVOff + (size_t)kVSlots * kPxTileBytes;
  static constexpr size_t kScaleOff = kRawOff + (size_t)kRaw * kPxRawBytes;
  static constexpr size_t kQScaleOff = kScaleOff + (kFp8 ? (size_t)kScaleSlots * 2 * kPxTile * 4 : 0);
  static constexpr size_t kBarOff = kQScaleOff + (kFp8 ? 2 * kPxRows * 4 : 0);
  static constexpr int kBars = 2 * 5 + 2 * 2 + 2 * 2 + 2 * 4 + 4 + 4 + 2 + 2 + 1;
  static_assert(8 * kPxOutWarp <= kScaleOff, "the results leave through the tiles' memory");
  static constexpr size_t kBytes = 1024 + kBarOff + kBars * 8 + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  // slot and parity of tile it's K and V
  __device__ static __forceinline__ int ks(int it) { return kFp8 ? it % kKSlots : (2 * it) % kKSlots; }
  __device__ static __forceinline__ uint32_t kp(int it) { return (kFp8 ? it / kKSlots : (2 * it) / kKSlots) & 1; }
  __device__ static __forceinline__ int vs(int it) { return kFp8 ? it % kVSlots : (2 * it + 1) % kVSlots; }
  __device__ static __forceinline__ uint32_t vp(int it) { return (kFp8 ? it / kVSlots : (2 * it + 1) / kVSlots) & 1; }
};

template <int KV>
struct PxSmem {
  using C = PxCfg<KV>;
  uint8_t *q, *k, *v, *raw;
  float *scale, *qscale;      // [slot][K, V][128]; [row]: c log2 e and the row's power of two
  uint64_t *k_full, *k_empty, *v_full, *v_empty;   // bf16: the same ring
  uint64_t *raw_full, *raw_empty, *sc_full, *sc_empty, *s_full, *p_full, *o_done, *done, *q_full;
  uint32_t *tmem_base;
  volatile int *abort_flag;
  __device__ explicit PxSmem(uint8_t *p) {
    q = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
    k = q + C::kKOff;
    v = q + C::kVOff;
    raw = q + C::kRawOff;
    scale = reinterpret_cast<float *>(q + C::kScaleOff);
    qscale = reinterpret_cast<float *>(q + C::kQScaleOff);
    k_full = reinterpret_cast<uint64_t *>(q + C::kBarOff);
    k_empty = k_full + 5;
    v_full = C::kFp8 ? k_empty + 5 : k_full;
    v_empty = C::kFp8 ? v_full + 2 : k_empty;
    raw_full = k_empty + 5 + 4;
    raw_empty = raw_full + 2;
    sc_full = raw_empty + 2;
    sc_empty = sc_full + 4;
    s_full = sc_empty + 4;
    p_full = s_full + 4;
    o_done = p_full + 4;
    done = o_done + 2;
    q_full = done + 2;
    tmem_base = reinterpret_cast<uint32_t *>(q_full + 1);
    abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
  }
};

// The pair's rows, and a walk over the own tiles of its sequences.
struct PxWalk {
  int64_t row0;               // first row of the pair
  int b_last, i_last;         // sequence and query token of its last row
  int b, j, count;            // sequence, tile j of its count

  __device__ __forceinline__ int own_tiles(const PrefixParams &P, int seq) const {
    const int i = seq == b_last ? i_last : P.n_q - 1;
    return (P.seq.len[seq] - P.n_q + i) / kPxTile + 1;
  }
  __device__ __forceinline__ PxWalk(const PrefixParams &P, int pair) {
    row0 = (int64_t)pair * 2 * kPxRows;
    const int64_t last = min(P.rows, row0 + 2 * kPxRows) - 1;
    const int q = (int)(last / P.n_heads);
    b_last = q / P.n_q;
    i_last = q - b_last * P.n_q;
    b = (int)(row0 / P.n_heads) / P.n_q;
    j = 0;
    count = own_tiles(P, b);
  }
  __device__ __forceinline__ int total(const PrefixParams &P) const {   // own tiles of the pair
    int n = 0;
    for (int s = b; s <= b_last; ++s) n += own_tiles(P, s);
    return n;
  }
  __device__ __forceinline__ void seek(const PrefixParams &P, int tile) {
    j = tile;
    while (j >= count && b < b_last) {
      j -= count;
      count = own_tiles(P, ++b);
    }
  }
  __device__ __forceinline__ void next(const PrefixParams &P) {
    if (++j >= count && b < b_last) {
      j = 0;
      count = own_tiles(P, ++b);
    }
  }
  __device__ __forceinline__ int64_t y(const PrefixParams &P) const { return P.seq.start[b] + j * kPxTile; }
  // rows of the tile that exist for this pair (may exceed the tile)
  __device__ __forceinline__ int valid(const PrefixParams &P) const {
    return P.seq.len[b] - P.n_q + (b == b_last ? i_last : P.n_q - 1) + 1 - j * kPxTile;
  }
  // lanes [lo, hi) of block g that see some row of the tile; `rows`: the block's rows
  __device__ __forceinline__ void lanes(const PrefixParams &P, int g, int rows, int &lo, int &hi) const {
    const int64_t r0 = row0 + g * kPxRows;
    const int i = max(0, j * kPxTile - (P.seq.len[b] - P.n_q));   // first query token that reaches it
    lo = (int)max((int64_t)0, ((int64_t)b * P.n_q + i) * P.n_heads - r0);
    hi = (int)min((int64_t)rows, ((int64_t)b + 1) * P.n_q * P.n_heads - r0);
  }
};

// P of 32 columns from their scores: exp2(x sc - m) as bf16 pairs, times the V scales (e4m3); the sum
// (before the V scales) is added to ls. All exponentials on the special-function unit: moving 4, 6 or 8 of 16
// to the FMA pipe by a quartic took 32 x 1 x 32 heads behind 131,072 from 93 to 96, 101 and 108 us.
template <bool kFp8>
__device__ __forceinline__ void px_weights(const float (&x)[32], float2 sc2, float2 neg, const float *vsc, float2 &ls,
                                           uint32_t (&pk)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 z = ffma2(make_float2(x[2 * k], x[2 * k + 1]), sc2, neg);
    float2 e = make_float2(fast_exp2(z.x), fast_exp2(z.y));
    ls = fadd2(ls, e);
    if (kFp8) e = fmul2(e, *reinterpret_cast<const float2 *>(vsc + 2 * k));
    pk[k] = pack_bf16(e.x, e.y);
  }
}

// Eight elements of a query row as e4m3 terms hi and lo (two [128 rows][128 B] operands), by 16 threads
// per row; the row's factor c log2 e 2^ex goes to *factor.
__device__ __forceinline__ void px_split_q(uint4 v, uint8_t *qb, int r, int ch, float scale_log2, float *factor) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    amax = fmax3(amax, fabsf(f[2 * i]), fabsf(f[2 * i + 1]));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // exponents kept in the range whose powers of two are normal both ways
  const int ex = amax > 0.f ? min(max((int)(__float_as_uint(amax) >> 23) - 134, -120), 120) : 0;
  const float down = __int_as_float((127 - ex) << 23);
  const float2 down2 = make_float2(down, down);
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 x = fmul2(make_float2(f[4 * i + 2 * j], f[4 * i + 2 * j + 1]), down2);
      const __nv_fp8x2_storage_t hc = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(hc, __NV_E4M3);
      const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
      h[j] = hc;
      l[j] = __nv_cvt_float2_to_fp8x2(make_float2(x.x - hf.x, x.y - hf.y), __NV_SATFINITE, __NV_E4M3);
    }
    hi[i] = h[0] | (h[1] << 16);
    lo[i] = l[0] | (l[1] << 16);
  }
  *reinterpret_cast<uint2 *>(qb + sw128(r, ch * 8)) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2 *>(qb + kPxRows * 128 + sw128(r, ch * 8)) = make_uint2(lo[0], lo[1]);
  // an infinite element has no such terms: every score of its row is infinite or NaN, and so its softmax NaN
  // (the factor stays above zero, which would make NaN of the -inf of masked columns)
  if (ch == 0)
    *factor = amax == INFINITY ? __int_as_float(0x7fc00000) : fmaxf(scale_log2 * __int_as_float((127 + ex) << 23), 0x1p-149f);
}

// 32 scores of this thread's row times their K scales (e4m3).
__device__ __forceinline__ void px_scale(float (&x)[32], const float *ksc) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 f = *reinterpret_cast<const float4 *>(ksc + i);
    const float2 a = fmul2(make_float2(x[i], x[i + 1]), make_float2(f.x, f.y));
    const float2 b = fmul2(make_float2(x[i + 2], x[i + 3]), make_float2(f.z, f.w));
    x[i] = a.x;
    x[i + 1] = a.y;
    x[i + 2] = b.x;
    x[i + 3] = b.y;
  }
}

// A warp's rows (a multiple of 16, as the heads are) from shared memory, four columns per lane, eight rows read
// before the first is stored (one at a time 2 x 1 queries behind 1,000 rows took 8.6 us, so 8.1).
template <class Store>
__device__ __forceinline__ void store_rows(const uint8_t *mem, int rows, Store store) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    float4 f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = *reinterpret_cast<const float4 *>(mem + (r0 + i) * kPxOutRow + lane * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) store(r0 + i, f[i]);
  }
}

// Turns of two warps: wait for the partner's pass; pass on (but after the last turn of all).
__device__ __forceinline__ void px_turn(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void px_pass(int id, int g, bool last) {
  if (!(g == 1 && last)) asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

template <int KV>
__global__ void __launch_bounds__(PxCfg<KV>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixMaps tm, const __grid_constant__ PrefixParams P) {
  using C = PxCfg<KV>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PxSmem<KV> sm(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // neighbouring CTAs take the same tiles for different rows, so that these are read from HBM once
  const int pair = blockIdx.x % P.n_pairs, split = blockIdx.x / P.n_pairs;
  PxWalk W(P, pair);
  const int total = P.n_tiles + W.total(P);
  const int tile0 = (int)((int64_t)split * total / P.n_splits);
  const int n = (int)((int64_t)(split + 1) * total / P.n_splits) - tile0;
  const int64_t row0 = W.row0;
  const int nb = P.rows - row0 > kPxRows ? 2 : 1;     // blocks with rows
  const int np = max(0, min(n, P.n_tiles - tile0));   // the first np tiles are the prefix's, the others own ones
  W.seek(P, max(0, tile0 - P.n_tiles));
  const int rows_g[2] = {(int)min((int64_t)kPxRows, P.rows - row0), (int)min((int64_t)kPxRows, P.rows - row0 - kPxRows)};

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKSlots; ++s) {
      mbar_init(smem_u32(&sm.k_full[s]), 1);
      mbar_init(smem_u32(&sm.k_empty[s]), nb);
    }
    if constexpr (C::kFp8) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(smem_u32(&sm.v_full[s]), 4);
        mbar_init(smem_u32(&sm.v_empty[s]), nb);
        mbar_init(smem_u32(&sm.raw_full[s]), 1);
        mbar_init(smem_u32(&sm.raw_empty[s]), 4);
      }
      for (int s = 0; s < C::kScaleSlots; ++s) {
        mbar_init(smem_u32(&sm.sc_full[s]), 32);
        mbar_init(smem_u32(&sm.sc_empty[s]), 4 * nb);
      }
    }
    for (int i = 0; i < 4; ++i) {   // block i / 2, half i % 2
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
    }
    mbar_init(smem_u32(&sm.o_done[0]), 1);
    mbar_init(smem_u32(&sm.o_done[1]), 1);
    mbar_init(smem_u32(&sm.done[0]), 1);
    mbar_init(smem_u32(&sm.done[1]), 1);
    mbar_init(smem_u32(&sm.q_full[0]), 1);
    *sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kPxWarpTma && lane == 0) {
    if constexpr (!C::kFp8) prefetch_tensormap(&tm.q);   // (the maps that the host has made)
    if (P.n_tiles > 0) {
      prefetch_tensormap(&tm.pk);
      prefetch_tensormap(&tm.pv);
    }
    prefetch_tensormap(&tm.k);
    prefetch_tensormap(&tm.v);
  }
  if (warp == kPxWarpMma) {
    tmem_alloc(smem_u32(sm.tmem_base), kPxCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_base;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  const int g = warp >> 2;                             // softmax warps: the block
  const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const int64_t row = row0 + g * kPxRows + (warp & 3) * 32 + lane;   // softmax warps: the thread's row
  float m_run = -INFINITY, l_run = 0.f;
  if (warp < 8) {
    if constexpr (C::kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    if constexpr (C::kFp8) {   // Q blocks -> shared memory: 16 threads per row, all loads first
      const __nv_bfloat16 *qg = static_cast<const __nv_bfloat16 *>(P.q) + row0 * kHeadDim;
      const int64_t left = P.rows - row0;
      const int ch = threadIdx.x & 15, r0 = threadIdx.x >> 4;
      uint4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        const int r = r0 + 16 * i;
        if (r < left) v[i] = *reinterpret_cast<const uint4 *>(qg + (size_t)r * kHeadDim + ch * 8);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = r0 + 16 * i;
        if (i < 8 || nb == 2) px_split_q(v[i], sm.q + (r >> 7) * (kPxRows * 256), r & 127, ch, P.scale_log2, sm.qscale + r);
      }
      fence_proxy_async_smem();
    }
    if (g < nb) {   // O = 0: every product accumulates, on the lanes that it concerns
      const uint32_t zero[32] = {};
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_st32(lane_addr + 256 + g * 128 + c, zero);
      tmem_wait_st();
    }
    tc_fence_before();
    asm volatile("bar.arrive 1, 320;" ::: "memory");   // the MMA warps wait for these alone
    if constexpr (C::kFp8) asm volatile("bar.sync 10, 256;" ::: "memory");   // the row factors
    if (g < nb) {
      // ------------------------------------------------------------ softmax
      const uint32_t s_addr = lane_addr + g * 128, o_addr = lane_addr + 256 + g * 128;
      const float sc = C::kFp8 ? sm.qscale[g * kPxRows + (warp & 3) * 32 + lane] : P.scale_log2;
      const float2 sc2 = make_float2(sc, sc);
      const int rl = (warp & 3) * 32 + lane;
      const int my_q = (int)(row / P.n_heads);           // flat query token
      int c_s = 0;                                       // tiles that concerned this block
      bool ok = true;
      // The two warps of a scheduler (w and w + 4) take turns at their exponentials while both have prefix
      // tiles: one's loads, maximum and waits run beside the other's exponentials. (In step, both waited
      // for the special-function unit and then left it idle.) A warp that gave up keeps taking its turns.
      const bool both = nb == 2;
      const int my_turn = 2 + (warp & 3) * 2 + g, your_turn = my_turn ^ 1;
      if (both && np > 0 && g == 1) px_pass(your_turn, 0, false);
      for (int it = 0; it < n; ++it) {
        int lo = 0, hi = rows_g[g], tile_valid = P.prefix_len - (tile0 + it) * kPxTile, valid = tile_valid;
        const bool own = it >= np;
        if (own) {
          W.lanes(P, g, rows_g[g], lo, hi);
          tile_valid = W.valid(P);
          valid = (rl >= lo && rl < hi) ? P.seq.len[W.b] - P.n_q + (my_q - W.b * P.n_q) + 1 - W.j * kPxTile : 0;
          W.next(P);
        }
        const float *ksc = sm.scale, *vsc = sm.scale;
        if constexpr (C::kFp8) {
          const int c = it % C::kScaleSlots;
          ok = ok && warp_wait_all(P.status, sm.abort_flag, &sm.sc_full[c], (it / C::kScaleSlots) & 1);
          ksc += c * 2 * kPxTile;
          vsc += (c * 2 + 1) * kPxTile;
        }
        if (hi > lo) {
          const bool mine = lo < (warp & 3) * 32 + 32 && hi > (warp & 3) * 32;   // some lane of this warp
          const bool turns = both && !own;
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // columns 64 h .. + 63
            ok = ok && warp_wait_all(P.status, sm.abort_flag, &sm.s_full[2 * g + h], c_s & 1);
            tc_fence_after();
            if (h == 0 && own && !C::kFp8 && tile_valid < kPxTile && ok) {   // V rows behind the sequence's last: zero
              ok = warp_wait_all(P.status, sm.abort_flag, &sm.v_full[C::vs(it)], C::vp(it));
              uint8_t *vt = sm.v + C::vs(it) * kPxTileBytes;
              for (int e = tile_valid * 16 + (threadIdx.x & 127); e < kPxTile * 16; e += 128)
                *reinterpret_cast<uint4 *>(vt + (e & 1) * (kPxTile * 128) + (e >> 1) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
            if (mine && ok) {
              float x[2][32];
              tmem_ld32_issue(s_addr + h * 64, x[0]);
              tmem_ld32_issue(s_addr + h * 64 + 32, x[1]);
              tmem_wait_ld32(x[0]);
              tmem_wait_ld32(x[1]);
              if constexpr (C::kFp8) {
                px_scale(x[0], ksc + h * 64);
                px_scale(x[1], ksc + h * 64 + 32);
              }
              if (__any_sync(0xffffffffu, valid < h * 64 + 64)) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                  if (h * 64 + i >= valid) x[i >> 5][i & 31] = -INFINITY;
              }
              float mq[4];   // the row maximum
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float *xc = x[c >> 1] + (c & 1) * 16;
                mq[c] = fmaxf(xc[0], xc[1]);
#pragma unroll
                for (int i = 2; i < 16; i += 2) mq[c] = fmax3(mq[c], xc[i], xc[i + 1]);
              }
              const float mt = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]) * sc;
              const bool move = mt > m_run + kPxLazy;
              if (__any_sync(0xffffffffu, move)) {
                const float m_new = move ? mt : m_run;
                const float alpha = move ? (m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new)) : 1.f;
                l_run *= alpha;
                m_run = m_new;
                if (c_s > 0 || h > 0) {   // rescale this row of O once the last product, number 2 c_s + h - 1, is
                                          // done (those before it are: this S was issued behind them)
                  ok = warp_wait_all(P.status, sm.abort_flag, &sm.o_done[g], (h ^ 1) & 1);
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < 128; c += 16) {
                    uint32_t v[16];
                    tmem_ld16_issue(o_addr + c, v);
                    tmem_wait_ld16(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                    tmem_st16(o_addr + c, v);
                  }
                  tmem_wait_st();
                }
              }
              const float mref = (m_run == -INFINITY) ? 0.f : m_run;
              float2 neg = make_float2(-mref, -mref);
              float2 ls = make_float2(0.f, 0.f);
              if (turns) {
                px_turn(my_turn);
                asm volatile("" : "+f"(neg.x), "+f"(neg.y));   // the exponentials stay behind it
              }
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
                px_weights<C::kFp8>(x[c], sc2, neg, vsc + h * 64 + c * 32, ls, pk);
                tmem_st16(s_addr + h * 64 + c * 16, pk);   // over scores that are in registers
              }
              if (turns) px_pass(your_turn, g, it == np - 1 && h == 1);
              l_run += ls.x + ls.y;
              tmem_wait_st();
            } else if (turns) {
              px_turn(my_turn);
              px_pass(your_turn, g, it == np - 1 && h == 1);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(smem_u32(&sm.p_full[2 * g + h]));
          }
          if (!ok && !turns) break;
          ++c_s;
        }
        if (!ok && own) break;
        if constexpr (C::kFp8) {
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(smem_u32(&sm.sc_empty[it % C::kScaleSlots]));
        }
      }
    }
  } else {
    if constexpr (C::kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kPxWarpTma) {
      // ------------------------------------------------------------ producer
      const bool issuer = elect_one();
      bool ok = true;
      if (!C::kFp8 && issuer) {   // Q (K-major, 128-byte swizzle; rows behind the last read as zero)
        mbar_arrive_expect_tx(smem_u32(&sm.q_full[0]), nb * kPxRows * 256);
        for (int i = 0; i < 2 * nb; ++i)
          tma_load_2d(smem_u32(sm.q) + i * (kPxRows * 128), &tm.q, smem_u32(&sm.q_full[0]), (i & 1) * 64,
                      (int)row0 + (i >> 1) * kPxRows);
      }
      __syncwarp();
      for (int it = 0; it < n; ++it) {
        const bool own = it >= np;
        const CUtensorMap *mk = own ? &tm.k : &tm.pk, *mv = own ? &tm.v : &tm.pv;
        const int y = own ? (int)W.y(P) : (tile0 + it) * kPxTile;
        if (own) W.next(P);
        const int sk = C::ks(it), sv = C::kFp8 ? it % 2 : C::vs(it);
        if (it >= 3)
          ok = warp_wait_all(P.status, sm.abort_flag, &sm.k_empty[sk], C::kp(it) ^ 1);
        if (!ok) break;
        if (issuer) {
          const uint32_t st = smem_u32(sm.k + sk * C::kKBytes), bar = smem_u32(&sm.k_full[sk]);
          mbar_arrive_expect_tx(bar, C::kKBytes);
          tma_load_2d(st, mk, bar, 0, y);
          if (!C::kFp8) tma_load_2d(st + kPxTile * 128, mk, bar, 64, y);
        }
        __syncwarp();
        if constexpr (C::kFp8) {
          if (it >= 2) ok = warp_wait_all(P.status, sm.abort_flag, &sm.raw_empty[sv], ((it / 2) & 1) ^ 1);
        } else {
          if (it >= 2) ok = warp_wait_all(P.status, sm.abort_flag, &sm.v_empty[sv], C::vp(it) ^ 1);
        }
        if (!ok) break;
        if (issuer) {
          const uint32_t st = smem_u32(C::kFp8 ? sm.raw + sv * kPxRawBytes : sm.v + sv * kPxTileBytes);
          const uint32_t bar = smem_u32(C::kFp8 ? &sm.raw_full[sv] : &sm.v_full[sv]);
          mbar_arrive_expect_tx(bar, C::kKBytes);
          tma_load_2d(st, mv, bar, 0, y);
          if (!C::kFp8) tma_load_2d(st + kPxTile * 128, mv, bar, 64, y);
        }
        __syncwarp();
      }
      if (!ok) {   // gave up: copies in flight land before the CTA ends (they take microseconds)
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {}
      }
      __syncwarp();
    } else if (C::kFp8 && warp == kPxWarpScale) {
      // ------------------------------------------------------------ the tiles' scales
      for (int it = 0; it < n; ++it) {
        const bool own = it >= np;
        const int64_t y = own ? W.y(P) : P.prefix_start + (int64_t)(tile0 + it) * kPxTile;
        const int valid = own ? W.valid(P) : P.prefix_len - (tile0 + it) * kPxTile;
        if (own) W.next(P);
        const int c = it % kPxScaleSlots;
        if (it >= kPxScaleSlots && !warp_wait_all(P.status, sm.abort_flag, &sm.sc_empty[c], ((it / kPxScaleSlots) & 1) ^ 1)) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = u * 32 + lane;
          const bool in = r < valid;
          cp_async_4(smem_u32(sm.scale + c * 2 * kPxTile + r), P.k_scale + y + (in ? r : 0), in ? 4u : 0u);
          cp_async_4(smem_u32(sm.scale + (c * 2 + 1) * kPxTile + r), P.v_scale + y + (in ? r : 0), in ? 4u : 0u);
        }
        cp_async_mbar_arrive(smem_u32(&sm.sc_full[c]));
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    } else if (C::kFp8 && warp >= kPxWarpWiden) {
      // ------------------------------------------------------------ V codes -> bf16 tiles
      // 16 codes per thread and step: eight neighbouring threads take four chunks of two rows, which
      // the swizzle spreads over all banks. (Shifting the exponent and fraction into bf16's place by integer
      // instructions instead of converting took 4 x 128 queries behind 30,001 rows from 423 to 476 us.)
      const int t = threadIdx.x - kPxWarpWiden * 32;
      for (int it = 0; it < n; ++it) {
        const int s = it % 2;
        const bool own = it >= np;
        const int valid = own ? W.valid(P) : kPxTile;   // (the prefix's maps end with it)
        if (own) W.next(P);
        if (!warp_wait_all(P.status, sm.abort_flag, &sm.raw_full[s], (it / 2) & 1)) break;
        if (it >= 2 && !warp_wait_all(P.status, sm.abort_flag, &sm.v_empty[s], ((it / 2) & 1) ^ 1)) break;
        const uint8_t *src = sm.raw + s * kPxRawBytes;
        uint8_t *dst = sm.v + s * kPxTileBytes;
#pragma unroll 4
        for (int u = 0; u < 8; ++u) {
          const int e = u * 128 + t;                     // (row pair, half, row of the pair, chunk)
          const int row = (e >> 4) * 2 + ((e >> 2) & 1), ch = ((e >> 3) & 1) * 4 + (e & 3);
          uint4 c = *reinterpret_cast<const uint4 *>(src + row * 128 + ch * 16);
          if (row >= valid) c = make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {c.x, c.y, c.z, c.w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[2 * j] = e4m3x2_to_bf16x2((uint16_t)(w[j] & 0xffffu));
            o[2 * j + 1] = e4m3x2_to_bf16x2((uint16_t)(w[j] >> 16));
          }
          uint8_t *box = dst + (ch >> 2) * (kPxTile * 128);
          *reinterpret_cast<uint4 *>(box + sw128(row, (ch & 3) * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(box + sw128(row, (ch & 3) * 32 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.v_full[s]));
          mbar_arrive(smem_u32(&sm.raw_empty[s]));
        }
      }
    } else if (warp == kPxWarpMma || warp == kPxWarpMma + 1) {
      // ------------------------------------------------------------ MMA issuers, one warp per block
      // S runs a tile ahead of P . V: while the softmax warps work on one 64-column buffer the other is
      // filled, and each P . V is followed by the S that takes its buffer.
      const int g2 = warp - kPxWarpMma;
      asm volatile("bar.sync 1, 320;" ::: "memory");   // Q and O are ready
      tc_fence_after();
      const uint32_t id_s = C::kFp8 ? umma_idesc_e4m3(kPxRows, 64) : umma_idesc_bf16(kPxRows, 64);
      const uint32_t id_o = umma_idesc_bf16_bmn(kPxRows, kHeadDim);
      // operand descriptors: the address field counts 16 bytes
      const uint64_t q_desc = umma_desc_sw128(smem_u32(sm.q) + g2 * (kPxRows * 256), 1024);
      const uint64_t k_desc = umma_desc_sw128(smem_u32(sm.k), 1024);
      const uint64_t v_desc = umma_desc_sw128_mn(smem_u32(sm.v), kPxTile * 128, 1024);
      const uint32_t s_tmem = tmem + g2 * 128, o_tmem = tmem + 256 + g2 * 128;
      const bool issuer = elect_one();                 // the operands stay warp-uniform
      const int rows = g2 == 0 ? rows_g[0] : rows_g[1];
      bool ok = g2 < nb;
      if (!C::kFp8) ok = ok && warp_wait_all(P.status, sm.abort_flag, &sm.q_full[0], 0);
      int cur = -1, lo = 0, hi = 0;                    // tile of P . V and its lanes; none yet
      int next = 0, nlo = 0, nhi = 0;                  // tile of S, if it concerns this block, and its lanes
      int used = 0;                                    // tiles that concerned this block
      const auto look = [&] {
        if (next < np) {
          nlo = 0;
          nhi = rows;
        } else if (next < n) {
          W.lanes(P, g2, rows, nlo, nhi);
          W.next(P);
        }
      };
      look();
      while (ok) {
        // Tiles that do not concern this block go back as they are -- behind the P . V before them, whose
        // slot the ring needs to bring them.
        while (cur < 0 && next < n && nhi <= nlo && ok) {
          ok = warp_wait_all(P.status, sm.abort_flag, &sm.k_full[C::ks(next)], C::kp(next));
          if (ok && lane == 0) mbar_arrive(smem_u32(&sm.k_empty[C::ks(next)]));
          ok = ok && warp_wait_all(P.status, sm.abort_flag, &sm.v_full[C::vs(next)], C::vp(next));
          if (ok && lane == 0) mbar_arrive(smem_u32(&sm.v_empty[C::vs(next)]));
          ++next;
          look();
        }
        const bool more = next < n && nhi > nlo;
        if (!ok || (!more && cur < 0)) break;
        const int sk = C::ks(next), sv = C::vs(max(cur, 0));
        const uint64_t kd = k_desc + (uint32_t)(sk * (C::kKBytes >> 4));
        const uint64_t vd = v_desc + (uint32_t)(sv * (kPxTileBytes >> 4));
        if (more) ok = warp_wait_all(P.status, sm.abort_flag, &sm.k_full[sk], C::kp(next));
        if (ok && cur >= 0) ok = warp_wait_all(P.status, sm.abort_flag, &sm.v_full[sv], C::vp(cur));
        if (!ok) break;
        const bool every = lo == 0 && hi == kPxRows;
        uint32_t off[4];       // lanes left as they are
#pragma unroll
        for (int w = 0; w < 4; ++w) off[w] = ~lane_bits(lo - 32 * w, hi - 32 * w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (cur >= 0) {      // O += P . V on the tile's lanes
            ok = warp_wait_all(P.status, sm.abort_flag, &sm.p_full[2 * g2 + h], (used - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (issuer) {
              if (every) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_bf16_ts(o_tmem, s_tmem + h * 64 + 8 * k, vd + (4 * h + k) * (2048 >> 4), id_o, true);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  umma_bf16_ts_lanes(o_tmem, s_tmem + h * 64 + 8 * k, vd + (4 * h + k) * (2048 >> 4), id_o, off);
              }
              umma_commit(smem_u32(&sm.o_done[g2]));
            }
            __syncwarp();
          }
          if (issuer) {        // S = Q . K^T for 64 rows of K, over the P that the product before has read
            if (more) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                // bf16: 16 dims a step, two boxes of 64; e4m3: 32 dims a step, the hi and then the lo terms
                const uint32_t o = ((k >> 2) * (kPxTile * 128) + (k & 3) * 32) >> 4;
                const uint32_t kof = h * (64 * 128 >> 4) + (C::kFp8 ? (k & 3) * 2 : o);
                if (C::kFp8) umma_e4m3(s_tmem + h * 64, q_desc + o, kd + kof, id_s, k > 0);
                else umma_bf16(s_tmem + h * 64, q_desc + o, kd + kof, id_s, k > 0);
              }
              umma_commit(smem_u32(&sm.s_full[2 * g2 + h]));
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (issuer) {          // the slots are free once these products are done
          if (cur >= 0) umma_commit(smem_u32(&sm.v_empty[sv]));
          if (more) umma_commit(smem_u32(&sm.k_empty[sk]));
        }
        __syncwarp();
        cur = -1;
        if (more) {
          cur = next++;
          lo = nlo;
          hi = nhi;
          ++used;
          look();
        }
      }
      if (issuer && g2 < nb) {   // every issued product has landed before TMEM is read or released
        umma_commit(smem_u32(&sm.done[g2]));
        if (!mbar_wait(smem_u32(&sm.done[g2]), 0)) {
          record_status(P.status, kStatusTimeout);
          *sm.abort_flag = 1;
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();   // the MMA warps have seen every product land
  tc_fence_after();
  const bool aborted = *sm.abort_flag != 0;
  if (warp < 8 && g < nb && !aborted) {
    // ------------------------------------------------------------ O and log-sum-exp
    const bool whole = P.n_splits == 1;
    // A row may see nothing in this range. (With one range it sees its own position at least: a sum of zero is that
    // of scores of -inf, and the result the NaN of the formula, as the merge's.)
    const bool some = whole || m_run != -INFINITY || l_run != 0.f;
    const float inv = some ? 1.f / l_run : 0.f;
    // through shared memory (the tiles are done with), a warp's 32 rows at a time, so that rows leave
    // in one piece: a thread storing its own row took 6 us
    uint8_t *mem = sm.q + warp * kPxOutWarp;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      float v[32];
      tmem_ld32_issue(lane_addr + 256 + g * 128 + c, v);
      tmem_wait_ld32(v);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4 *>(mem + lane * kPxOutRow + (c + i) * 4) =
            some ? make_float4(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncwarp();
    const int64_t first = row - lane;                  // the warp's first row
    const int rows_w = (int)min((int64_t)32, P.rows - first);
    if (!whole || P.out_f32) {
      float *o = (whole ? static_cast<float *>(P.out) : P.part_o + (int64_t)split * P.rows * kHeadDim) + first * kHeadDim;
      store_rows(mem, rows_w, [&](int r, const float4 &f) { *reinterpret_cast<float4 *>(o + r * kHeadDim + lane * 4) = f; });
    } else {
      __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(P.out) + first * kHeadDim;
      store_rows(mem, rows_w, [&](int r, const float4 &f) {
        *reinterpret_cast<uint2 *>(o + r * kHeadDim + lane * 4) = make_uint2(pack_bf16(f.x, f.y), pack_bf16(f.z, f.w));
      });
    }
    const float lse = some ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
    if (row < P.rows) {
      if (!whole) P.part_lse[(int64_t)split * P.rows + row] = lse;
      else if (P.lse) P.lse[row] = lse;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPxWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kPxCols);
  }
}

// out = sum_j w_j O_j / sum_j w_j, w_j = exp(lse_j - max lse), over the ranges of a row's tiles. kW warps
// share a row: each sums every kW-th part, four columns per lane, and the warps' sums meet in shared
// memory, in warp order. Few rows take eight warps each, many one for each four parts or so: with eight, 16,384
// rows of two parts took 29 us of instructions (4 x 128 queries behind 30,001 rows 234 us in all, 217 so).
constexpr int kPmWarps = 8;           // per CTA

template <int kW>
__global__ void __launch_bounds__(kPmWarps * 32) prefix_merge_kernel(const __grid_constant__ PrefixParams P) {
  constexpr int kRows = kPmWarps / kW;
  __shared__ float4 s_o[kW > 1 ? kPmWarps : 1][32];
  __shared__ float s_l[kPmWarps];
  __shared__ float s_m[kPmWarps];
  __shared__ float s_w[kRows][kW * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = warp / kW, w0 = warp % kW, t = threadIdx.x % (kW * 32);   // the CTA's row, the warp and thread in it
  const int64_t row = min((int64_t)blockIdx.x * kRows + slot, P.rows - 1);   // (the last row may be done twice)
  griddep_launch_dependents();
  griddep_wait();
  // the parts' log-sum-exps and their maximum; the first parts of O are on their way meanwhile
  constexpr int kAhead = 4;
  const float *part = P.part_o + row * kHeadDim + lane * 4;
  const int64_t stride = P.rows * kHeadDim;
  float4 v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int j = w0 + i * kW;
    v[i] = j < P.n_splits ? *reinterpret_cast<const float4 *>(part + j * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
  if (t < P.n_splits) s_w[slot][t] = M = P.part_lse[t * P.rows + row];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (kW > 1) {
    if (lane == 0) s_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kW; ++i) M = fmaxf(M, s_m[slot * kW + i]);
  } else {
    __syncwarp();
  }
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](int j, const float4 &x) {
    const float w = expf(s_w[slot][j] - ref);
    L += w;
    o.x = fmaf(w, x.x, o.x);
    o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z);
    o.w = fmaf(w, x.w, o.w);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (w0 + i * kW < P.n_splits) add(w0 + i * kW, v[i]);
#pragma unroll 4
  for (int j = w0 + kAhead * kW; j < P.n_splits; j += kW)
    add(j, *reinterpret_cast<const float4 *>(part + j * stride));
  if (kW > 1) {
    s_o[warp][lane] = o;
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (w0 != 0) return;
#pragma unroll
    for (int i = 1; i < kW; ++i) {
      const float4 x = s_o[warp + i][lane];
      o.x += x.x;
      o.y += x.y;
      o.z += x.z;
      o.w += x.w;
      L += s_l[warp + i];
    }
  }
  const float inv = 1.f / L;
  const int64_t at = row * kHeadDim + lane * 4;
  if (P.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(P.out) + at) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (P.lse && lane == 0) P.lse[row] = M + logf(L);
}

template <int KV>
cudaError_t launch_px(const PrefixMaps &tm, const PrefixParams &p, cudaStream_t s) {
  using C = PxCfg<KV>;
  auto kern = prefix_attn_kernel<KV>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, C::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, p.n_pairs * p.n_splits, C::kThreads, C::kBytes, s, tm, p);
}

}  // namespace

cudaError_t launch_prefix_attn(int kv_dtype, const PrefixMaps &tm, const PrefixParams &p, cudaStream_t s) {
  return kv_dtype == HS2_KV_BF16 ? launch_px<kKvBf16>(tm, p, s) : launch_px<kKvFp8>(tm, p, s);
}

cudaError_t launch_prefix_merge(const PrefixParams &p, cudaStream_t s) {
  const auto launch = [&](auto kern, int per_row) {
    const int rows = kPmWarps / per_row;
    return launch_pdl(kern, (int)((p.rows + rows - 1) / rows), kPmWarps * 32, 0, s, p);
  };
  if (p.rows <= 8 * 148) return launch(prefix_merge_kernel<kPmWarps>, kPmWarps);   // at most 8 CTAs an SM
  if (p.n_splits < 8) return launch(prefix_merge_kernel<1>, 1);
  if (p.n_splits < 16) return launch(prefix_merge_kernel<2>, 2);
  if (p.n_splits < 32) return launch(prefix_merge_kernel<4>, 4);
  return launch(prefix_merge_kernel<kPmWarps>, kPmWarps);
}

}  // namespace hs2
