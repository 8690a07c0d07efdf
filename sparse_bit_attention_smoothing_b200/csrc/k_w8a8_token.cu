// k_w8a8_token.cu -- the linear layer in 8-bit integers with one scale per
// token (row of x) and per output channel (row of W).
//
//   s = fl32(amax/127), code = RNE(fl32(x * fl32(127/amax))) per row;
//   y[m][n] = (integer dot of the codes) * s_x[m] * s_w[n] + bias[n].
//
// Times in this file are of kernels one after another on the same buffers, so
// small operands come from L2.  A call on inputs from HBM, 5120 -> 5120: 1 token
// 10.2 us, 1024 tokens 33.5, 75600 tokens 1540.
//
// The scales leave the sum over K, so the product runs through the whole of K
// in INT32 (exact for K <= 131056: 2^14 K < 2^31) and the scales, the bias
// and the one rounding are the epilogue of the output tile.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

namespace sagesla {

namespace {

// A row whose largest magnitude is below this counts as zeros (scale 1, codes
// 0): under 2^-121 the multiplier 127/amax leaves fp32, and such rows (1e-31)
// hold nothing that a bf16 product keeps beside any other row.
constexpr float kTiny = 0x1p-100f;

__device__ __forceinline__ void widen8(const uint4& v, int dtype, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == 0) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

}  // namespace

// Largest magnitude of two lanes of 16-bit values, by their bits: for both
// types the order of the bits without the sign is the order of magnitudes,
// with infinity and then NaN above every number.
__device__ __forceinline__ uint32_t max_bits(const uint4& v, uint32_t m) {
  const uint32_t k = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(m, __vmaxu2(v.x & k, v.y & k)), __vmaxu2(v.z & k, v.w & k));
}
// Eight codes.  |x * mult| <= 127 (1 + 2^-23), so adding 1.5 * 2^23 rounds the
// fp32 product to the nearest whole number (even on a tie) and leaves the
// code in the low byte; no clamp is left to do.
template <int kType>
__device__ __forceinline__ uint2 codes8(const uint4& v, float mult) {
  float f[8];
  widen8(v, kType, f);
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)  // scalar: a packed product and sum were joined into one rounding, another code at ties
    r[j] = __float_as_uint(__fadd_rn(__fmul_rn(f[j], mult), 12582912.f));
  return make_uint2(__byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(r[4], r[5], 0x0040), __byte_perm(r[6], r[7], 0x0040), 0x5410));
}

// A row is held by the registers of W warps, up to kHeld pieces of 8 values a
// lane, so x is read once (rows longer than that are read twice); a CTA has
// 4/W rows for W <= 4, or one.  75600 x 5120, us with 2, 4, 8 pieces a lane:
// 233, 180, 166 (7.0 TB/s).  NaN or an infinity in a row: scale NaN, codes
// 0, so every output of that token is NaN.
constexpr int kHeld = 8;
template <int kType>
__global__ void __launch_bounds__(1024) w8a8_token_quant_kernel(const uint16_t* __restrict__ a, long lda, int rows,
                                                                int cols, int W, int8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  __shared__ uint32_t red[32];
  launch_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / W, R = (blockDim.x >> 5) / W;
  const long row = (long)blockIdx.x * R + sub;
  const bool live = row < rows;
  const uint4* src = reinterpret_cast<const uint4*>(a + (live ? row : 0) * lda);
  const int n8 = live ? cols / 8 : 0, t = (warp - sub * W) * 32 + lane, T = 32 * W;
  uint4 v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) v[i] = t + i * T < n8 ? __ldg(src + t + i * T) : make_uint4(0, 0, 0, 0);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) m = max_bits(v[i], m);
  for (int i = t + kHeld * T; i < n8; i += T) m = max_bits(__ldg(src + i), m);
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if (W > 1) {
    if (lane == 0) red[warp] = m;
    __syncthreads();
    for (int w = 0; w < W; ++w) m = max(m, red[sub * W + w]);
  }
  const uint16_t mh = (uint16_t)m;
  const float amax = kType == 0 ? __uint_as_float(m << 16) : __half2float(*reinterpret_cast<const __half*>(&mh));
  const bool bad = m >= (kType == 0 ? 0x7f80u : 0x7c00u), some = amax >= kTiny && !bad;
  const float mult = some ? __fdiv_rn(127.f, amax) : 0.f;
  if (t == 0 && live) scales[row] = bad ? __int_as_float(0x7fffffff) : some ? __fdiv_rn(amax, 127.f) : 1.f;
  uint2* dst = reinterpret_cast<uint2*>(codes + row * cols);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (t + i * T < n8) dst[t + i * T] = some ? codes8<kType>(v[i], mult) : make_uint2(0, 0);
  for (int i = t + kHeld * T; i < n8; i += T) dst[i] = some ? codes8<kType>(__ldg(src + i), mult) : make_uint2(0, 0);
}

// ----------------------------------------------------------------- product --
// More than 64 tokens.  Persistent, one CTA pair per two SMs, tiles of 256
// tokens x BN channels: each CTA has 128 rows of x and BN/2 of W in shared
// memory and 128 rows of the INT32 accumulator in its TMEM, so a byte from L2
// feeds twice the products that it would in a single CTA (at 75600 x 5120 ->
// 5120: 1169 us against 1302 with single CTAs of 128 x 256).
//   warp 0     TMA loads of x and W, 128 bytes of K a step, into a ring;
//   warp 1     the leader's MMAs, K = 32 each;
//   warps 2-5  the epilogue of the previous tile while the next one runs (two
//              accumulators of 256 TMEM columns): scales, bias, rounding, and
//              out through swizzled shared memory by TMA, or element by
//              element where the rows of y are not 16-byte aligned.
// Every wait is bounded (watchdog).
namespace {

constexpr int kStageA = 128 * 128, kMaxBN = 256;
constexpr int kEpiWarps = 4;
constexpr int kGemmThreads = 32 * (2 + kEpiWarps);
constexpr int kOutStage = 32 * 64;  // 32 rows of 32 outputs
constexpr int kFew = 64;  // tokens
constexpr int kFewStages = 5, kMaxSplits = 7;

constexpr int kStages = 6, kStageBytes = kStageA + kMaxBN / 2 * 128;
// ring; two output stages, scales and biases a warp; barriers; alignment
constexpr int kGemmSmem = kStages * kStageBytes + kEpiWarps * (2 * kOutStage + 2 * kMaxBN * 4) + 512 + 1024;

template <int kType>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (kType == 0) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int kType>
__device__ __forceinline__ float widen1(uint16_t v) {
  return kType == 0 ? __uint_as_float((uint32_t)v << 16) : __half2float(*reinterpret_cast<const __half*>(&v));
}

// 32 x 32 outputs from their swizzled stage to rows of y that are not 16-byte
// aligned: two columns a lane where N is even, else one; sixteen rows' loads in
// flight.  The product 21704 x 960 -> 5510 takes 217 us (one row and column at
// a time 373), -> 5509 317, -> 5504, whose rows are aligned, 139.
template <typename T>
__device__ __forceinline__ void rows_out(const uint8_t* o, uint16_t* y, int row0, int n0, int M, int N, int lane) {
  constexpr int kE = sizeof(T) / 2, kLanes = 32 / kE;  // columns a lane, lanes a row
  const int c = kE * (lane % kLanes), n = n0 + c;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 16) {
    T h[16 / kE];
#pragma unroll
    for (int i = 0; i < 16 / kE; ++i) {
      const int r = r0 + kE * i + lane / kLanes;
      h[i] = *reinterpret_cast<const T*>(o + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + (c & 7) * 2);
    }
#pragma unroll
    for (int i = 0; i < 16 / kE; ++i) {
      const int r = row0 + r0 + kE * i + lane / kLanes;
      if (r < M && n < N) *reinterpret_cast<T*>(y + (size_t)r * N + n) = h[i];
    }
  }
}

}  // namespace

template <int kType>
__global__ void __launch_bounds__(kGemmThreads, 1)
    w8a8_token_gemm_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                           const __grid_constant__ CUtensorMap my, const float* sx,
                           const float* __restrict__ sw, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y,
                           int M, int N, int K, int BN, int tma_out, int* wd) {
  constexpr int S = kStages, SB = kStageBytes, kBM = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* outs = smem + S * SB;
  float* scal = reinterpret_cast<float*>(outs + kEpiWarps * 2 * kOutStage);  // [warp][scale, bias][kMaxBN]
  struct Bars {
    uint64_t full[S], empty[S], acc_full[2], acc_empty[2], fin;
    uint32_t tmem;
    int abort;
  };
  Bars* bars = reinterpret_cast<Bars*>(scal + kEpiWarps * 2 * kMaxBN);
  static_assert(sizeof(Bars) <= 512, "barriers");
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int nM = (M + kBM - 1) / kBM, nN = (N + BN - 1) / BN, nK = (K + 127) / 128;
  const long ntiles = (long)nM * nN;
  const long first = blockIdx.x / 2, step = gridDim.x / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->acc_full[b], 1);
      mbar_init(&bars->acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&bars->fin, 1);
    bars->abort = 0;
    mbar_fence_init();
    prefetch_map(&mx);
    prefetch_map(&mw);
    prefetch_map(&my);
  }
  if (warp == 1) tmem_alloc_pair(&bars->tmem, 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------ producer ------------------------------
    // W does not come from the kernel before this one: the first tile's rows
    // of it are brought to L2 while the quantiser ends.
    if (first < ntiles && elect_one()) {
      const int n0 = (int)(first % nN) * BN + (BN / 2) * rank;
      for (int kb = 0; kb < min(nK, 64); ++kb) tma_prefetch_2d(&mw, kb * 128, n0);
    }
    __syncwarp();
    wait_previous();
    const uint32_t bytes = 2 * (kStageA + (BN / 2) * 128);
    int st = 0;
    uint32_t ph = 0;
    long it = 0;
    for (long t = first; ok && t < ntiles; t += step) {
      const int m0 = (int)(t / nN) * kBM + 128 * rank, n0 = (int)(t % nN) * BN + (BN / 2) * rank;
      for (int kb = 0; kb < nK; ++kb, ++it) {
        ok = mbar_wait(&bars->empty[st], ph ^ 1, abort, wd);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (elect_one()) {
          uint8_t* dst = smem + st * SB;
          const uint32_t bar = map_rank(smem_u32(&bars->full[st]), 0);
          if (rank == 0) mbar_expect_tx(&bars->full[st], bytes);
          tma_load_2d<1>(dst, &mx, kb * 128, m0, bar);
          tma_load_2d<1>(dst + kStageA, &mw, kb * 128, n0, bar);
        }
        __syncwarp();
        if (++st == S) st = 0, ph ^= 1;
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    // Drain what is in flight (both CTAs' loads count on the leader's barriers).
    if (rank == 0)
      for (long g = it > S ? it - S : 0; g < it; ++g)
        if (!mbar_wait_drain(&bars->full[g % S], (g / S) & 1, wd)) break;
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ----------------------------
    if (rank == 0) {
      const uint64_t d0 = smem_desc_sw128(smem);
      const uint32_t id = idesc_i8(kBM, BN);
      int st = 0;
      uint32_t ph = 0;
      long tl = 0;
      for (long t = first; ok && t < ntiles; t += step, ++tl) {
        const int buf = (int)(tl & 1);
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_empty[buf], ((tl >> 1) & 1) ^ 1, abort, wd));
        tc_fence_after();
        for (int kb = 0; ok && kb < nK; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[st], ph, abort, wd));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t da = desc_at(d0, st * SB), db = desc_at(d0, st * SB + kStageA);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_i8_pair(tmem + buf * 256, desc_at(da, kk * 32), desc_at(db, kk * 32), id, kb > 0 || kk > 0);
            mma_commit_pair(&bars->empty[st]);
            if (kb == nK - 1) mma_commit_pair(&bars->acc_full[buf]);
          }
          __syncwarp();
          if (++st == S) st = 0, ph ^= 1;
        }
      }
      if (elect_one()) mma_commit_pair(&bars->fin);
      __syncwarp();
    }
  } else {
    // ------------------------------- epilogue -----------------------------
    wait_previous();
    const int q = warp & 3;  // TMEM lane quadrant: rows 32q .. 32q+31
    uint8_t* stage = outs + (warp - 2) * 2 * kOutStage;
    const uint32_t tl0 = tmem + ((uint32_t)(32 * q) << 16);
    float* ws = scal + (warp - 2) * 2 * kMaxBN;
    long tl = 0;
    uint32_t chunk = 0;
    for (long t = first; t < ntiles; t += step, ++tl) {
      const int buf = (int)(tl & 1);
      const int row0 = (int)(t / nN) * kBM + 128 * rank + 32 * q, n0 = (int)(t % nN) * BN;
      for (int c = lane; c < BN; c += 32) {  // a copy of its own for each warp: no barrier that an abort could leave
        const bool in = n0 + c < N;
        ws[c] = in ? __ldg(sw + n0 + c) : 0.f;
        ws[kMaxBN + c] = in && bias ? widen1<kType>(__ldg(bias + n0 + c)) : 0.f;
      }
      const float rs = row0 + lane < M ? ld_previous(sx + row0 + lane) : 0.f;
      __syncwarp();
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->acc_full[buf], (tl >> 1) & 1, abort, wd));
      tc_fence_after();
      for (int c0 = 0; ok && c0 < BN; c0 += 32, ++chunk) {
        uint32_t v[32];
        SAGESLA_TMEM_LD32(tl0 + buf * 256 + c0, v);
        tmem_ld_wait();
        uint8_t* o = stage + (chunk & 1) * kOutStage;
        if (tma_out && lane == 0) bulk_wait_read<1>();  // the store that last used this half
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(ws + c0 + j + e);
            const float4 b4 = *reinterpret_cast<const float4*>(ws + kMaxBN + c0 + j + e);
            const float f0 = __fmaf_rn(__fmul_rn((float)(int)v[j + e], rs), s4.x, b4.x);
            const float f1 = __fmaf_rn(__fmul_rn((float)(int)v[j + e + 1], rs), s4.y, b4.y);
            const float f2 = __fmaf_rn(__fmul_rn((float)(int)v[j + e + 2], rs), s4.z, b4.z);
            const float f3 = __fmaf_rn(__fmul_rn((float)(int)v[j + e + 3], rs), s4.w, b4.w);
            pk[e / 2] = pack2<kType>(f0, f1);
            pk[e / 2 + 1] = pack2<kType>(f2, f3);
          }
          // 64-byte swizzle: 16-byte piece p of row r lies at p ^ (r/2 % 4)
          *reinterpret_cast<uint4*>(o + lane * 64 + (((j >> 3) ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < M && n0 + c0 < N) tma_store_2d(&my, o, n0 + c0, row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          if (N % 2 == 0)
            rows_out<uint32_t>(o, y, row0, n0 + c0, M, N, lane);
          else
            rows_out<uint16_t>(o, y, row0, n0 + c0, M, N, lane);
          __syncwarp();
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(map_rank(smem_u32(&bars->acc_empty[buf]), 0));
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  if (!ok && lane == 0) st_cluster(map_rank(smem_u32(&bars->abort), rank ^ 1), 1);
  __syncthreads();
  // The last MMAs and the arrivals of their commits, which reach both CTAs.
  if (threadIdx.x == 0) mbar_wait_drain(&bars->fin, 0, wd);
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------ few tokens --
// Up to 64 tokens: the bytes of W bound the product, so the roles turn round.
// A tile is 128 rows of W (the MMA's M side) and all BN tokens (its N side),
// every byte of W enters one SM once, and a cluster of CTAs splits K, so that
// the SMs are full where N alone gives few tiles.  Each CTA leaves its INT32
// sums in shared memory; after a cluster barrier the CTAs add each other's
// (exact in any order), a warp a token, and finish the outputs.
// One token, N = K = 5120: 9.2 us (26 MB of W, 2.8 TB/s, of which 5 us are
// the launch and the two cluster barriers: a product of 1536 takes 5.0).
// W does not come from the kernel before this one (the quantiser of x), so
// the ring starts to fill with W before that one is done.
template <int kType>
__global__ void __launch_bounds__(kGemmThreads)
    w8a8_token_few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                          const float* sx, const float* __restrict__ sw,
                          const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int M, int N, int K, int BN,
                          int S, int splits, int* wd) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  struct Bars {
    uint64_t full[kFewStages], empty[kFewStages], fin;
    uint32_t tmem;
    int abort;
  };
  const int SB = kStageA + BN * 128;
  Bars* bars = reinterpret_cast<Bars*>(smem + S * SB);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int n0 = (int)(blockIdx.x / splits) * 128;
  const int nK = (K + 127) / 128, k0 = nK * rank / splits, k1 = nK * (rank + 1) / splits;
  const uint32_t ncols = BN <= 32 ? 32 : 64;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->fin, 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem, ncols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------ producer ------------------------------
    const int pre = min(S, k1 - k0);
    if (elect_one())
      for (int i = 0; i < pre; ++i) {
        mbar_expect_tx(&bars->full[i], SB);
        tma_load_2d<0>(smem + i * SB, &mw, (k0 + i) * 128, n0, smem_u32(&bars->full[i]));
      }
    __syncwarp();
    wait_previous();
    if (elect_one())
      for (int i = 0; i < pre; ++i)
        tma_load_2d<0>(smem + i * SB + kStageA, &mx, (k0 + i) * 128, 0, smem_u32(&bars->full[i]));
    __syncwarp();
    int st = 0;
    uint32_t ph = 0;
    int it = pre;
    for (; it < k1 - k0; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[st], ph, abort, wd));
      if (!ok) break;
      if (elect_one()) {
        mbar_expect_tx(&bars->full[st], SB);
        tma_load_2d<0>(smem + st * SB, &mw, (k0 + it) * 128, n0, smem_u32(&bars->full[st]));
        tma_load_2d<0>(smem + st * SB + kStageA, &mx, (k0 + it) * 128, 0, smem_u32(&bars->full[st]));
      }
      __syncwarp();
      if (++st == S) st = 0, ph ^= 1;
    }
    for (int g = max(0, it - S); g < it; ++g)  // drain what is in flight
      if (!mbar_wait_drain(&bars->full[g % S], (g / S) & 1, wd)) break;
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ----------------------------
    const uint64_t d0 = smem_desc_sw128(smem);
    const uint32_t id = idesc_i8(128, BN);
    int st = 0;
    uint32_t ph = 0;
    for (int kb = k0; kb < k1; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[st], ph, abort, wd));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t da = desc_at(d0, st * SB), db = desc_at(d0, st * SB + kStageA);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_i8(tmem, desc_at(da, kk * 32), desc_at(db, kk * 32), id, kb > k0 || kk > 0);
        mma_commit(&bars->empty[st]);
      }
      __syncwarp();
      if (++st == S) st = 0, ph ^= 1;
    }
    if (elect_one()) mma_commit(&bars->fin);
    __syncwarp();
  }
  // All operands of the ring are read once `fin` has arrived (a producer that
  // gave up has drained its copies by the barrier below); the sums go over it.
  __syncthreads();
  mbar_wait_drain(&bars->fin, 0, wd);
  __syncwarp();
  tc_fence_after();
  int* part = reinterpret_cast<int*>(smem);  // [BN tokens][128 rows of W]
  if (warp >= 2) {
    const int q = warp & 3;
    for (int c0 = 0; c0 < BN; c0 += 16) {
      uint32_t v[16];
      SAGESLA_TMEM_LD16(tmem + ((uint32_t)(32 * q) << 16) + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + 32 * q + lane] = (int)v[j];
    }
  }
  tc_fence_before();
  if (splits > 1)
    cluster_sync();
  else
    __syncthreads();
  wait_previous();  // the scales of x
  const int n = n0 + 4 * lane;
  float s4[4], b4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s4[i] = n + i < N ? __ldg(sw + n + i) : 0.f;
    b4[i] = n + i < N && bias ? widen1<kType>(__ldg(bias + n + i)) : 0.f;
  }
  const bool wide = N % 4 == 0;
  for (int c = warp * splits + rank; c < M; c += (kGemmThreads / 32) * splits) {
    int4 s = *reinterpret_cast<const int4*>(part + c * 128 + 4 * lane);
    int4 o[kMaxSplits - 1];  // all peers' loads in flight together
#pragma unroll
    for (int r = 1; r < kMaxSplits; ++r) {
      const int peer = rank + r >= splits ? rank + r - splits : rank + r;
      o[r - 1] = r < splits ? ld_cluster_int4(map_rank(smem_u32(part + c * 128 + 4 * lane), peer)) : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < kMaxSplits - 1; ++r) s.x += o[r].x, s.y += o[r].y, s.z += o[r].z, s.w += o[r].w;
    const float rs = ld_previous(sx + c);
    const float f0 = __fmaf_rn(__fmul_rn((float)s.x, rs), s4[0], b4[0]), f1 = __fmaf_rn(__fmul_rn((float)s.y, rs), s4[1], b4[1]);
    const float f2 = __fmaf_rn(__fmul_rn((float)s.z, rs), s4[2], b4[2]), f3 = __fmaf_rn(__fmul_rn((float)s.w, rs), s4[3], b4[3]);
    const uint32_t lo = pack2<kType>(f0, f1), hi = pack2<kType>(f2, f3);
    uint16_t* dst = y + (size_t)c * N + n;
    if (wide) {
      if (n < N) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
      if (n < N) dst[0] = (uint16_t)lo;
      if (n + 1 < N) dst[1] = (uint16_t)(lo >> 16);
      if (n + 2 < N) dst[2] = (uint16_t)hi;
      if (n + 3 < N) dst[3] = (uint16_t)(hi >> 16);
    }
  }
  __syncwarp();
  if (splits > 1)
    cluster_sync();  // no CTA leaves while its sums may be read
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, ncols);
  }
}

namespace {

// A row-major [rows][cols] matrix, boxes of bc columns x br rows.
bool matrix_map(CUtensorMap* m, const void* p, bool half, long rows, long cols, int bc, int br, CUtensorMapSwizzle sw) {
  const unsigned long dims[2] = {(unsigned long)cols, (unsigned long)rows}, stride = (unsigned long)cols * (half ? 2 : 1);
  const unsigned box[2] = {(unsigned)bc, (unsigned)br};
  return tensor_map(m, p, half ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dims, &stride, box, sw);
}

// Cluster of `ctas` CTAs, and the programmatic launch behind the quantiser.
void launch_cluster(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&at)[2], int ctas, bool chained) {
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = chained ? 2 : 1;
}

template <int kType>
cudaError_t gemm_launch(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, const void* bias, void* y,
                        int M, int N, int K, int BN, int sms, int* wd, cudaStream_t st, bool chained) {
  CUtensorMap mx, mw, my;
  const int tma_out = N % 8 == 0;
  if (!matrix_map(&mx, xq, false, M, K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !matrix_map(&mw, wq, false, N, K, 128, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (tma_out) {
    if (!matrix_map(&my, y, true, M, N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) return cudaErrorInvalidValue;
  } else {
    my = mx;
  }
  const long tiles = (long)((M + 255) / 256) * ((N + BN - 1) / BN);
  const long pairs = tiles < sms / 2 ? tiles : sms / 2;
  auto* fn = w8a8_token_gemm_kernel<kType>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), kGemmSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  launch_cluster(cfg, at, 2, chained);
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, my, sx, sw, static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y),
                            M, N, K, BN, tma_out, wd);
}

template <int kType>
cudaError_t few_launch(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, const void* bias, void* y,
                       int M, int N, int K, int sms, int* wd, cudaStream_t st, bool chained) {
  const int BN = (M + 15) / 16 * 16, SB = kStageA + BN * 128, nK = (K + 127) / 128, tiles = (N + 127) / 128;
  // A ring of 96 KB, so that two CTAs fit an SM.  K is split so that about
  // three CTAs stand for two SMs, each with two steps at least: more did not
  // fit at once (clusters have to be placed whole).  One token, K = 5120, us:
  // N = 5120 with 1, 2, 3, 4, 5, 7 parts 13.2, 10.5, 9.8, 9.3, 9.2, 13.4;
  // N = 13824 with 1, 2, 3, 5: 16.1, 15.6, 19.8, 18.9; N = K = 1536 with 1, 3,
  // 5, 7: 6.1, 5.2, 5.0, 4.9.  A ring of 190 KB (one CTA an SM) lost with it.
  const int S = 96 * 1024 / SB;
  int splits = 3 * sms / 2 / tiles;
  splits = splits > nK / 2 ? nK / 2 : splits;
  splits = splits > kMaxSplits ? kMaxSplits : splits < 1 ? 1 : splits;
  CUtensorMap mx, mw;
  if (!matrix_map(&mx, xq, false, M, K, 128, BN, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !matrix_map(&mw, wq, false, N, K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto* fn = w8a8_token_few_kernel<kType>;
  const int smem = S * SB + 256 + 1024;  // the sums (BN * 512 bytes) fit the ring
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), 112 * 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  launch_cluster(cfg, at, splits, chained);
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, sx, sw, static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), M, N,
                            K, BN, S, splits, wd);
}

}  // namespace

cudaError_t launch_w8a8_token_quant(const void* a, int dtype, int rows, int cols, long lda, int8_t* codes,
                                    float* scales, cudaStream_t st) {
  int W = (cols / 8 + 32 * kHeld - 1) / (32 * kHeld);
  W = W > 32 ? 32 : W;
  const int R = W > 4 ? 1 : 4 / W;
  const unsigned grid = (unsigned)(((long)rows + R - 1) / R);
  if (dtype == 0)
    w8a8_token_quant_kernel<0><<<grid, 32 * W * R, 0, st>>>(static_cast<const uint16_t*>(a), lda, rows, cols, W, codes,
                                                            scales);
  else
    w8a8_token_quant_kernel<1><<<grid, 32 * W * R, 0, st>>>(static_cast<const uint16_t*>(a), lda, rows, cols, W, codes,
                                                            scales);
  return cudaGetLastError();
}

cudaError_t launch_w8a8_token_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                   const void* bias, void* y, int dtype, int M, int N, int K, int sms, int* wd,
                                   cudaStream_t st, bool chained) {
  // Few tokens, us with this kernel and with the pairs' (N = K = 5120): 1 token
  // 9.2 and 20, 64 tokens 11.7 and 13.9, 128 tokens 14.2 and 14.0 (N = 13824:
  // 21.9 and 19.1).
  if (M <= kFew)
    return dtype == 0 ? few_launch<0>(xq, sx, wq, sw, bias, y, M, N, K, sms, wd, st, chained)
                      : few_launch<1>(xq, sx, wq, sw, bias, y, M, N, K, sms, wd, st, chained);
  // The width of the tiles: the one whose rounds over the SM pairs take the
  // least.  A step of 128 of K takes about as long as BN + 220 columns would
  // at the MMA's rate (the loads of x from L2 beside those of W): 1024 x 5120
  // -> 5120 takes 30.7, 23.6, 21.3, 28.2 us with 256, 192, 160, 128.
  long best = -1;
  int BN = 256;
  for (int bn = 256; bn >= 32; bn -= 32) {
    const long tiles = (long)((M + 255) / 256) * ((N + bn - 1) / bn);
    const long cost = ((tiles + sms / 2 - 1) / (sms / 2)) * (bn + 220);
    if (best < 0 || cost < best) best = cost, BN = bn;
  }
  return dtype == 0 ? gemm_launch<0>(xq, sx, wq, sw, bias, y, M, N, K, BN, sms, wd, st, chained)
                    : gemm_launch<1>(xq, sx, wq, sw, bias, y, M, N, K, BN, sms, wd, st, chained);
}

}  // namespace sagesla
