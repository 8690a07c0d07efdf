// k_qk_norm_rope.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, and its backward pass.
//
// Per row (token, head) of d channels, everything in fp32:
//   r = 1 / sqrt(mean x^2 + eps),  n = x r gamma,
//   y = R(p) n: the first `rot` channels in pairs turned by the angles of the
//   token's position p, (a, b) -> (a cos - b sin, a sin + b cos); the rest of
//   the channels pass; one rounding to the tensor's type.
// Backward, with g = R(p)^T dy, xh = x r, u = g gamma:
//   dx = r (u - xh mean(u xh)),   dgamma = sum over rows of g xh.
//
// Bound by HBM in both directions: a row is read once and written once (the
// backward pass recomputes r from the x it has to read anyway, so the forward
// pass saves nothing).  A lane owns 8 consecutive channels (16 bytes of a
// 16-bit type), L = d/8 lanes (rounded up to a power of two) a row, so a row
// sum is log2(L) shuffles and no shared memory.  A warp serves several heads
// of ONE token: the token's cos/sin row and gamma are loaded once for them,
// and the loads of all its rows are in flight together.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace sagesla {

namespace {

constexpr int kWarps = 8;

// Eight consecutive channels as stored: one 16-byte piece (16-bit types) or two (fp32).
template <typename T>
struct Piece {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Piece<T> load8(const T* p) {
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ Piece<T> zero8() {
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}
__device__ __forceinline__ void widen(const Piece<__nv_bfloat16>& p, float (&f)[8]) {
  const uint32_t w[4] = {p.v[0].x, p.v[0].y, p.v[0].z, p.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void widen(const Piece<__half>& p, float (&f)[8]) {
  const uint32_t w[4] = {p.v[0].x, p.v[0].y, p.v[0].z, p.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void widen(const Piece<float>& p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(p.v[i].x);
    f[4 * i + 1] = __uint_as_float(p.v[i].y);
    f[4 * i + 2] = __uint_as_float(p.v[i].z);
    f[4 * i + 3] = __uint_as_float(p.v[i].w);
  }
}
__device__ __forceinline__ void narrow(const float (&f)[8], Piece<__nv_bfloat16>& p) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  p.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(const float (&f)[8], Piece<__half>& p) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  p.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(const float (&f)[8], Piece<float>& p) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    p.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                        __float_as_uint(f[4 * i + 3]));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  Piece<T> r;
  narrow(f, r);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

// The lane's part of the token's cos/sin row.  Interleaved pairs: channels
// 8c .. 8c+7 are pairs 4c .. 4c+3 (four values of each).  Halves: channel j
// of the first half pairs with j + rot/2, both with value j (eight of each).
template <bool kIl>
struct Turn {
  float c[kIl ? 4 : 8], s[kIl ? 4 : 8];
  bool on;      // the lane's channels turn
  bool second;  // (halves) the lane's channels are the second of their pairs
  int peer;     // (halves) the lane of the row's group that holds the other ones
};
template <bool kIl>
__device__ __forceinline__ Turn<kIl> load_turn(const float* __restrict__ ct, const float* __restrict__ stb, long p,
                                               int rot, int sub) {
  Turn<kIl> t;
  const int half = rot / 2;
  t.on = 8 * sub < rot;
  t.second = false;
  t.peer = sub;
  constexpr int kNv = kIl ? 1 : 2;
  int at = 4 * sub;
  if (!kIl) {
    t.second = 8 * sub >= half;
    at = t.second ? 8 * sub - half : 8 * sub;
    if (t.on) t.peer = t.second ? sub - half / 8 : sub + half / 8;
  }
#pragma unroll
  for (int i = 0; i < kNv; ++i) {
    float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t.on) {
      a = __ldg(reinterpret_cast<const float4*>(ct + p * half + at) + i);
      b = __ldg(reinterpret_cast<const float4*>(stb + p * half + at) + i);
    }
    t.c[4 * i] = a.x, t.c[4 * i + 1] = a.y, t.c[4 * i + 2] = a.z, t.c[4 * i + 3] = a.w;
    t.s[4 * i] = b.x, t.s[4 * i + 1] = b.y, t.s[4 * i + 2] = b.z, t.s[4 * i + 3] = b.w;
  }
  return t;
}
// f <- R f (dir = 1) or R^T f (dir = -1), the lanes of a row together.
template <bool kIl>
__device__ __forceinline__ void turn(float (&f)[8], const Turn<kIl>& t, float dir, int L) {
  if (kIl) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1], s = dir * t.s[i];
      if (t.on) {
        f[2 * i] = a * t.c[i] - b * s;
        f[2 * i + 1] = a * s + b * t.c[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, f[i], t.peer, L);
      const float s = t.second ? dir * t.s[i] : -dir * t.s[i];
      if (t.on) f[i] = f[i] * t.c[i] + o * s;
    }
  }
}
__device__ __forceinline__ float row_sum(float v, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace

// ----------------------------------------------------------------- forward --
// Warp w of the grid: token w / G, head group w % G (the Gq groups of q, then
// k's); a group is U passes of R = 32/L heads.
template <typename T, bool kIl, int U>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const RopeArgs a) {
  const long w = (long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, L = a.L, R = 32 / L;
  const long token = w / a.G;
  if (token >= a.tokens) return;
  int grp = (int)(w - token * a.G);
  const int tsr = grp >= a.Gq;
  if (tsr) grp -= a.Gq;
  const long b = token / a.N, n = token - b * a.N;
  const RopeTensor& t = a.t[tsr];
  const int sub = lane & (L - 1), h0 = grp * R * U + lane / L;
  const bool mine = 8 * sub < a.d;
  const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[1] + 8 * sub;
  T* y = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[1] + 8 * sub;
  const long p = a.pos ? (long)__ldg(a.pos + token) : n;
  if (p < 0) {  // padding: zeros
    const float z[8] = {};
    for (int u = 0; u < U; ++u)
      if (mine && h0 + u * R < t.H) store8(y + (h0 + u * R) * t.ys[2], z);
    return;
  }
  Piece<T> in[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    in[u] = (mine && h0 + u * R < t.H) ? load8(x + (h0 + u * R) * t.xs[2]) : zero8<T>();
  const bool far = p >= a.T;  // no such row of the tables: NaN
  float gm[8] = {};
  if (mine) widen(load8(static_cast<const T*>(t.gamma) + 8 * sub), gm);
  const Turn<kIl> tn = load_turn<kIl>(a.cos, a.sin, far ? 0 : p, a.rot, sub);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[8];
    widen(in[u], f);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
    ss = row_sum(ss, L);
    const float r = far ? __int_as_float(0x7fffffff) : __frcp_rn(__fsqrt_rn(ss * a.inv_d + a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * r * gm[i];
    turn<kIl>(f, tn, 1.f, L);
    if (mine && h0 + u * R < t.H) store8(y + (h0 + u * R) * t.ys[2], f);
  }
}

// ---------------------------------------------------------------- backward --
// Persistent: warp w keeps its head group w % G and walks the tokens
// w / G, w / G + stride, ..., so its lanes hold the running dgamma of their
// eight channels in fp32 registers.  The sums of a CTA's warps are joined in
// shared memory in a fixed order and written as one partial row of q and one
// of k; dgamma_kernel adds the CTAs' rows in fp64, again in a fixed order:
// no atomics, the same bits every time.
template <typename T, bool kIl, int U>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_bwd_kernel(const RopeArgs a) {
  __shared__ float part[kWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, L = a.L, R = 32 / L;
  const long w = (long)blockIdx.x * kWarps + warp;
  int grp = (int)(w % a.G);
  const int tsr = grp >= a.Gq;
  if (tsr) grp -= a.Gq;
  const RopeTensor& t = a.t[tsr];
  const int sub = lane & (L - 1), h0 = grp * R * U + lane / L;
  const bool mine = 8 * sub < a.d;
  float gm[8] = {}, acc[8] = {};
  if (mine) widen(load8(static_cast<const T*>(t.gamma) + 8 * sub), gm);
  for (long token = w / a.G; token < a.tokens && w / a.G < a.stride; token += a.stride) {
    const long b = token / a.N, n = token - b * a.N;
    const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[1] + 8 * sub;
    const T* dy = static_cast<const T*>(t.dy) + b * t.dys[0] + n * t.dys[1] + 8 * sub;
    T* dx = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[1] + 8 * sub;
    const long p = a.pos ? (long)__ldg(a.pos + token) : n;
    if (p < 0) {  // padding: no gradient
      const float z[8] = {};
      for (int u = 0; u < U; ++u)
        if (mine && h0 + u * R < t.H) store8(dx + (h0 + u * R) * t.ys[2], z);
      continue;
    }
    Piece<T> in[U], gr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = mine && h0 + u * R < t.H;
      in[u] = ok ? load8(x + (h0 + u * R) * t.xs[2]) : zero8<T>();
      gr[u] = ok ? load8(dy + (h0 + u * R) * t.dys[2]) : zero8<T>();
    }
    const bool far = p >= a.T;
    const Turn<kIl> tn = load_turn<kIl>(a.cos, a.sin, far ? 0 : p, a.rot, sub);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8], g[8];
      widen(in[u], f);
      widen(gr[u], g);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
      ss = row_sum(ss, L);
      const float r = far ? __int_as_float(0x7fffffff) : __frcp_rn(__fsqrt_rn(ss * a.inv_d + a.eps));
      turn<kIl>(g, tn, -1.f, L);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] *= r;  // xh
        const float gx = g[i] * f[i];
        if (h0 + u * R < t.H) acc[i] += gx;
        dot += gx * gm[i];
      }
      dot = row_sum(dot, L) * a.inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = r * (g[i] * gm[i] - f[i] * dot);
      if (mine && h0 + u * R < t.H) store8(dx + (h0 + u * R) * t.ys[2], f);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  if (lane < L && mine)
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][8 * sub + i] = acc[i];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < a.d) {
    float s[2] = {0.f, 0.f};
    for (int v = 0; v < kWarps; ++v) s[(int)(((long)blockIdx.x * kWarps + v) % a.G) >= a.Gq] += part[v][c];
    a.part[((size_t)blockIdx.x * 2) * a.d + c] = s[0];
    a.part[((size_t)blockIdx.x * 2 + 1) * a.d + c] = s[1];
  }
}

// dgamma of q (block.y 0) and k (1): eight channels a CTA, its 32 threads of a
// channel add the CTAs' partial rows in fp64.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* __restrict__ part, int rows, int d,
                                                     float* __restrict__ gq, float* __restrict__ gk) {
  __shared__ double s[32][8];
  float* out = blockIdx.y ? gk : gq;
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), r0 = threadIdx.x >> 3;
  double v = 0.0;
  for (int r = r0; r < rows; r += 32) v += (double)part[((size_t)r * 2 + blockIdx.y) * d + c];
  s[r0][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8 && out) {
    v = 0.0;
    for (int r = 0; r < 32; ++r) v += s[r][threadIdx.x];
    out[c] = (float)v;
  }
}

namespace {

constexpr int kBwdCtasPerSm = 4;

template <typename T, bool kIl>
cudaError_t rope_launch(const RopeArgs& a0, bool back, int sms, cudaStream_t st) {
  constexpr int U = 4, UB = 2;
  RopeArgs a = a0;
  const int per = (32 / a.L) * (back ? UB : U);
  a.Gq = (a.t[0].H + per - 1) / per;
  a.G = a.Gq + (a.t[1].H + per - 1) / per;
  if (!back) {
    const long ctas = (a.tokens * a.G + kWarps - 1) / kWarps;
    qk_norm_rope_kernel<T, kIl, U><<<(unsigned)ctas, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int ctas = rope_bwd_ctas(a.tokens, a.G, sms);
  a.stride = (long)ctas * kWarps / a.G;
  qk_norm_rope_bwd_kernel<T, kIl, UB><<<ctas, 32 * kWarps, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  dgamma_kernel<<<dim3(a.d / 8, 2), 256, 0, st>>>(a.part, ctas, a.d, a.dgq, a.dgk);
  return cudaGetLastError();
}

}  // namespace

// CTAs of the backward pass: enough for every (token, group) pair or four an SM, and at least one warp a group.
int rope_bwd_ctas(long tokens, int G, int sms) {
  const long need = (tokens * G + kWarps - 1) / kWarps;
  long ctas = need < (long)kBwdCtasPerSm * sms ? need : (long)kBwdCtasPerSm * sms;
  const long least = ((long)G + kWarps - 1) / kWarps;
  return (int)(ctas > least ? ctas : least);
}

size_t rope_bwd_workspace(int B, int N, int Hq, int Hk, int d, int sms) {
  // G is at most one group a head
  return (size_t)rope_bwd_ctas((long)B * N, Hq + Hk, sms) * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a0, int dtype, bool interleaved, bool back, int sms,
                                cudaStream_t st) {
  RopeArgs a = a0;
  a.L = 2;
  while (8 * a.L < a.d) a.L <<= 1;
  a.inv_d = 1.f / (float)a.d;
  if (dtype == 0)
    return interleaved ? rope_launch<__nv_bfloat16, true>(a, back, sms, st)
                       : rope_launch<__nv_bfloat16, false>(a, back, sms, st);
  if (dtype == 1)
    return interleaved ? rope_launch<__half, true>(a, back, sms, st) : rope_launch<__half, false>(a, back, sms, st);
  return interleaved ? rope_launch<float, true>(a, back, sms, st) : rope_launch<float, false>(a, back, sms, st);
}

}  // namespace sagesla
