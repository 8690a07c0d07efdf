// k_linear_decay.cu -- causal linear attention with a decay for each head:
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,
// the state S [d][d] in fp32 throughout.
#include "common.cuh"
#include "kernels.h"

namespace sagesla {

namespace {

__device__ __forceinline__ float bf(const uint16_t* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

}  // namespace

// Simple form: a CTA of 8 warps walks one head's tokens for 32 channels of v
// (one a lane); warp w holds rows w, w + 8, ... of the state's slice.
template <int D>
__global__ void __launch_bounds__(256) linear_decay_simple_kernel(const DecayArgs a) {
  __shared__ float red[8][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z, c = blockIdx.x * 32 + lane;
  const int hk = h / (a.H / a.Hk);
  const int len = a.lens ? max(0, min(a.N, a.lens[b])) : a.N;
  const float lam = expf(a.log_decay[h]);
  const size_t s0 = ((size_t)b * a.H + h) * D * D;
  float S[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) S[i] = a.state_in ? a.state_in[s0 + (size_t)(warp + 8 * i) * D + c] : 0.f;
  const uint16_t* q = a.q + b * a.qs[0] + h * a.qs[2];
  const uint16_t* k = a.k + b * a.ks[0] + hk * a.ks[2];
  const uint16_t* v = a.v + b * a.vs[0] + hk * a.vs[2];
  uint16_t* o = a.o + b * a.os[0] + h * a.os[2];
  for (int n = 0; n < len; ++n) {
    const float vv = bf(v + n * a.vs[1] + c);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      S[i] = lam * S[i] + bf(k + n * a.ks[1] + warp + 8 * i) * vv;
      s += bf(q + n * a.qs[1] + warp + 8 * i) * S[i];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0) {
      float t = 0.f;
      for (int w = 0; w < 8; ++w) t += red[w][lane];
      const __nv_bfloat16 r = __float2bfloat16_rn(t * a.scale);
      o[n * a.os[1] + c] = *reinterpret_cast<const uint16_t*>(&r);
    }
    __syncthreads();
  }
  for (int n = len + warp; n < a.N; n += 8) o[n * a.os[1] + c] = 0;  // rows of padding
  if (a.state_out)
#pragma unroll
    for (int i = 0; i < D / 8; ++i) a.state_out[s0 + (size_t)(warp + 8 * i) * D + c] = S[i];
}

cudaError_t launch_linear_decay(const DecayArgs& a, int* wd, cudaStream_t st) {
  (void)wd;
  const dim3 grid(a.d / 32, a.H, a.B);
  if (a.d == 64)
    linear_decay_simple_kernel<64><<<grid, 256, 0, st>>>(a);
  else
    linear_decay_simple_kernel<128><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sagesla
