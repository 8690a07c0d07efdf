// k_w8a8_token.cu -- the linear layer in 8-bit integers with one scale per
// token (row of x) and per output channel (row of W).
//
//   s = fl32(amax/127), code = RNE(fl32(x * fl32(127/amax))) per row;
//   y[m][n] = (integer dot of the codes) * s_x[m] * s_w[n] + bias[n].
//
// The scales leave the sum over K, so the product runs through the whole of K
// in INT32 (exact for K <= 131056: 2^14 K < 2^31) and the scales, the bias
// and the one rounding are the epilogue of the output tile.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

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

// One CTA a row.  NaN or an infinity in a row: scale NaN, codes 0, so every
// output of that token is NaN.
template <int kType>
__global__ void __launch_bounds__(256) w8a8_token_quant_kernel(const uint16_t* __restrict__ a, long lda, int cols,
                                                               int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t red[8];
  const long row = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(a + row * lda);
  const int n8 = cols / 8, t = threadIdx.x;
  uint32_t m = 0;  // largest magnitude by its fp32 bits: NaN and infinity compare above every number
  for (int i = t; i < n8; i += 256) {
    float f[8];
    widen8(__ldg(src + i), kType, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((t & 31) == 0) red[t >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, red[w]);
  const float amax = __uint_as_float(m);
  const bool bad = m >= 0x7f800000u, some = amax >= kTiny && !bad;
  const float mult = some ? __fdiv_rn(127.f, amax) : 0.f;
  if (t == 0) scales[row] = bad ? __int_as_float(0x7fffffff) : some ? __fdiv_rn(amax, 127.f) : 1.f;
  uint2* dst = reinterpret_cast<uint2*>(codes + row * cols);
  for (int i = t; i < n8; i += 256) {
    float f[8];
    widen8(__ldg(src + i), kType, f);
    uint32_t pk[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = max(-127, min(127, __float2int_rn(__fmul_rn(f[j], mult))));
      pk[j >> 2] |= ((uint32_t)c & 0xffu) << (8 * (j & 3));
    }
    dst[i] = some ? make_uint2(pk[0], pk[1]) : make_uint2(0, 0);
  }
}

// Simple product: 64 x 64 outputs a CTA of 256 threads (4 x 4 each), K in
// steps of 64 bytes through shared memory, four products a dp4a.
__global__ void __launch_bounds__(256) w8a8_token_simple_kernel(const int8_t* __restrict__ xq,
                                                                const float* __restrict__ sx,
                                                                const int8_t* __restrict__ wq,
                                                                const float* __restrict__ sw,
                                                                const void* __restrict__ bias, void* __restrict__ y,
                                                                int M, int N, int K, int dtype) {
  __shared__ int A[64][17], B[64][17];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, t = threadIdx.x, tm = t / 16, tn = t % 16;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    for (int i = t; i < 64 * 16; i += 256) {
      const int r = i / 16, c = i % 16, k = k0 + 4 * c;
      A[r][c] = (m0 + r < M && k < K) ? *reinterpret_cast<const int*>(xq + (size_t)(m0 + r) * K + k) : 0;
      B[r][c] = (n0 + r < N && k < K) ? *reinterpret_cast<const int*>(wq + (size_t)(n0 + r) * K + k) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(A[tm + 16 * i][c], B[tn + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
      if (m >= M || n >= N) continue;
      float f = (float)acc[i][j] * sx[m] * sw[n];
      if (bias)
        f += dtype == 0 ? __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[n])
                        : __half2float(static_cast<const __half*>(bias)[n]);
      if (dtype == 0)
        static_cast<__nv_bfloat16*>(y)[(size_t)m * N + n] = __float2bfloat16_rn(f);
      else
        static_cast<__half*>(y)[(size_t)m * N + n] = __float2half_rn(f);
    }
}

cudaError_t launch_w8a8_token_quant(const void* a, int dtype, int rows, int cols, long lda, int8_t* codes,
                                    float* scales, cudaStream_t st) {
  if (dtype == 0)
    w8a8_token_quant_kernel<0><<<rows, 256, 0, st>>>(static_cast<const uint16_t*>(a), lda, cols, codes, scales);
  else
    w8a8_token_quant_kernel<1><<<rows, 256, 0, st>>>(static_cast<const uint16_t*>(a), lda, cols, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_w8a8_token_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                   const void* bias, void* y, int dtype, int M, int N, int K, int* wd,
                                   cudaStream_t st) {
  (void)wd;
  w8a8_token_simple_kernel<<<dim3((N + 63) / 64, (M + 63) / 64), 256, 0, st>>>(xq, sx, wq, sw, bias, y, M, N, K,
                                                                               dtype);
  return cudaGetLastError();
}

}  // namespace sagesla
