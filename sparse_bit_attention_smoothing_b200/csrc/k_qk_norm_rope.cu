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
// Times in this file are of calls one after another on the same buffers, bf16
// where no type is named.  On other inputs with every call: 75600 tokens x 40/40
// heads of 128 forward 582 us; 32760 x 12/12 backward 137.  fp32 at 32760 x 12/12
// from HBM: forward 143 us (5.6 TB/s), backward 205 (5.9 TB/s).
//
// Bound by HBM in both directions: a row is read once and written once (the
// backward pass recomputes r from the x it has to read anyway, so the forward
// pass saves nothing); what the kernels cost beside the bytes is issue slots.
// A lane owns pieces of 8 consecutive channels (16 bytes of a 16-bit type): one
// with interleaved pairs, the two that are each other's with pairs of halves,
// so a rotation is arithmetic of one lane in both pairings.  (With one piece
// the halves trade theirs by shuffles: 190 us against 168 for q of 40 heads, k
// of 8, 32760 tokens; with two the interleaved pairs' coefficients cost a third
// of the warps: 720p 584 us against 517.)  L = d/8 or d/16 lanes (rounded up
// to a power of two) hold a row, so a row sum is log2(L) shuffles and no
// shared memory.  A warp serves several heads of ONE token: the token's cos/sin
// row and gamma are loaded once for them, and the loads of all its rows are in
// flight together.
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
__device__ __forceinline__ Piece<T> fill8(uint32_t w) {
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(w, w, w, w);
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

// Eight channels as four packed pairs of fp32 (one instruction for two).
// Interleaved pairs: e[0], e[1] hold the first and second channels of pairs 0
// and 1, e[2], e[3] those of pairs 2 and 3.  Halves: channels in order.
struct Row {
  uint64_t e[4];
};
template <bool kIl>
__device__ __forceinline__ Row row_of(const float (&f)[8]) {
  Row r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.e[i] = kIl ? f32x2_pack(f[4 * (i / 2) + (i & 1)], f[4 * (i / 2) + (i & 1) + 2]) : f32x2_pack(f[2 * i], f[2 * i + 1]);
  return r;
}
template <bool kIl>
__device__ __forceinline__ void row_to(const Row& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (kIl)
      f32x2_unpack(r.e[i], f[4 * (i / 2) + (i & 1)], f[4 * (i / 2) + (i & 1) + 2]);
    else
      f32x2_unpack(r.e[i], f[2 * i], f[2 * i + 1]);
}
template <bool kIl, typename T>
__device__ __forceinline__ Row widen_row(const Piece<T>& p) {
  float f[8];
  widen(p, f);
  return row_of<kIl>(f);
}
__device__ __forceinline__ uint64_t neg2(uint64_t v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint64_t both(float v) { return f32x2_pack(v, v); }
__device__ __forceinline__ float add_halves(uint64_t v) {
  float a, b;
  f32x2_unpack(v, a, b);
  return a + b;
}
__device__ __forceinline__ float dot_row(const Row& a, const Row& b) {
  return add_halves(f32x2_fma(a.e[0], b.e[0], f32x2_fma(a.e[1], b.e[1], f32x2_fma(a.e[2], b.e[2], f32x2_mul(a.e[3], b.e[3])))));
}

// The lane's pieces of a row: P = 1 with interleaved pairs, 2 with halves.
template <int P>
struct Part {
  Row r[P];
};
template <int P>
__device__ __forceinline__ float dot_part(const Part<P>& x, const Part<P>& y) {
  float v = dot_row(x.r[0], y.r[0]);
  if (P == 2) v += dot_row(x.r[P - 1], y.r[P - 1]);
  return v;
}
template <int P>
__device__ __forceinline__ Part<P> mul_part(const Part<P>& x, const Part<P>& y) {
  Part<P> z;
#pragma unroll
  for (int i = 0; i < 4 * P; ++i) z.r[i / 4].e[i % 4] = f32x2_mul(x.r[i / 4].e[i % 4], y.r[i / 4].e[i % 4]);
  return z;
}
template <int P>
__device__ __forceinline__ Part<P> mul_part(const Part<P>& x, uint64_t y) {
  Part<P> z;
#pragma unroll
  for (int i = 0; i < 4 * P; ++i) z.r[i / 4].e[i % 4] = f32x2_mul(x.r[i / 4].e[i % 4], y);
  return z;
}

// Where the lane's pieces lie (in pieces of 8 channels).  Halves, r pieces
// turned: lane s < r/2 has pieces s and s + r/2 (channels c and c + rot/2), and
// the lanes behind share out the rest the same way.
template <int P>
struct Place {
  int at[P];
  bool mine, on;  // the lane has channels; they turn
  __device__ __forceinline__ Place(int d, int rot, int s) {
    const int n = d / 8, r = rot / 8;
    on = P * s < r;
    mine = P * s < n;
    if (P == 1) {
      at[0] = s;
    } else {
      at[0] = on ? s : r / 2 + s;
      at[P - 1] = on ? s + r / 2 : at[0] + (n - r) / 2;
    }
  }
};

// The lane's part of the token's rotation: y = own * c + other * s, where
// `other` is the pair's other channel: with halves the other piece's, with
// interleaved pairs its own neighbour (s of the first channels negative).
template <int P>
struct Turn {
  Part<P> c, s;
};
template <int P>
__device__ __forceinline__ Turn<P> load_turn(const float* __restrict__ ct, const float* __restrict__ stb, long p, int rot,
                                             const Place<P>& pl) {
  Turn<P> t;
  const float4* c = reinterpret_cast<const float4*>(ct + p * (rot / 2)) + P * pl.at[0];
  const float4* s = reinterpret_cast<const float4*>(stb + p * (rot / 2)) + P * pl.at[0];
  // Interleaved: piece x has values 4x .. 4x + 3.  Halves: both pieces have 8x .. 8x + 7.
  float4 c4[P], s4[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    c4[i] = pl.on ? __ldg(c + i) : make_float4(1.f, 1.f, 1.f, 1.f);
    s4[i] = pl.on ? __ldg(s + i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if constexpr (P == 1) {
    Row &cr = t.c.r[0], &sr = t.s.r[0];
    cr.e[0] = cr.e[1] = f32x2_pack(c4[0].x, c4[0].y), cr.e[2] = cr.e[3] = f32x2_pack(c4[0].z, c4[0].w);
    sr.e[1] = f32x2_pack(s4[0].x, s4[0].y), sr.e[3] = f32x2_pack(s4[0].z, s4[0].w);
    sr.e[0] = neg2(sr.e[1]), sr.e[2] = neg2(sr.e[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t.c.r[0].e[2 * i] = f32x2_pack(c4[i].x, c4[i].y), t.c.r[0].e[2 * i + 1] = f32x2_pack(c4[i].z, c4[i].w);
      t.s.r[1].e[2 * i] = f32x2_pack(s4[i].x, s4[i].y), t.s.r[1].e[2 * i + 1] = f32x2_pack(s4[i].z, s4[i].w);
    }
    t.c.r[1] = t.c.r[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) t.s.r[0].e[i] = neg2(t.s.r[1].e[i]);
  }
  return t;
}
// The other channels of the lane's pairs.
template <int P>
__device__ __forceinline__ Part<P> others(const Part<P>& x) {
  Part<P> y;
  if constexpr (P == 2) {
    y.r[0] = x.r[1], y.r[1] = x.r[0];
  } else {
    y.r[0].e[0] = x.r[0].e[1], y.r[0].e[1] = x.r[0].e[0], y.r[0].e[2] = x.r[0].e[3], y.r[0].e[3] = x.r[0].e[2];
  }
  return y;
}
template <int P>
__device__ __forceinline__ Part<P> turn(const Part<P>& x, const Turn<P>& t, bool on) {
  const Part<P> o = others(x);
  Part<P> y = mul_part(x, t.c);
#pragma unroll
  for (int i = 0; i < 4 * P; ++i)
    if (on) y.r[i / 4].e[i % 4] = f32x2_fma(o.r[i / 4].e[i % 4], t.s.r[i / 4].e[i % 4], y.r[i / 4].e[i % 4]);
  return y;
}
__device__ __forceinline__ float row_sum(float v, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The row sums of U passes at once (U a power of two): in each of the first
// log2(U) steps a lane gives away half of the values it still holds, so U sums
// take U - 1 + log2(L) - log2(U) shuffles instead of U log2(L).  The sum of
// pass u ends in the lanes whose leading bits of `sub` are u's: take() brings
// it to the others.  Rows of fewer than U lanes take the plain way.
template <int U>
struct Sums {
  float v[U];
  bool split;
  __device__ __forceinline__ void reduce(int L, int sub) {
    split = L >= U;
    if (!split) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = row_sum(v[u], L);
      return;
    }
    int o = L >> 1;
#pragma unroll
    for (int half = U / 2; half > 0; half >>= 1, o >>= 1) {
      const bool up = sub & o;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  }
  template <class F>
  __device__ __forceinline__ void apply(F f) {  // one evaluation a lane where a lane holds one sum
    v[0] = f(v[0]);
    if (!split)
#pragma unroll
      for (int u = 1; u < U; ++u) v[u] = f(v[u]);
  }
  __device__ __forceinline__ float take(int u, int L) const {
    return split ? __shfl_sync(0xffffffffu, v[0], u * (L / U), L) : v[u];
  }
};
// 1 / sqrt(mean + eps); NaN for a position outside the tables.
__device__ __forceinline__ float inv_rms(float ss, const RopeArgs& a, bool far) {
  return far ? __int_as_float(0x7fffffff) : rsqrtf(ss * a.inv_d + a.eps);
}

// A head group of a tensor: `pass` passes of R = 32/L heads; the lane's first
// head is h0, and it has `heads` of the passes' heads.
struct Group {
  int tsr, h0, sub, heads;
  __device__ __forceinline__ Group(const RopeArgs& a, unsigned g) {
    const int lane = threadIdx.x & 31, R = 32 / a.L;
    tsr = g >= (unsigned)a.Gq;
    const int grp = (int)g - (tsr ? a.Gq : 0), pass = a.pass[tsr], H = a.t[tsr].H;
    sub = lane & (a.L - 1);
    h0 = grp * R * pass + lane / a.L;
    heads = h0 < H ? min(pass, (H - 1 - h0) / R + 1) : 0;
  }
};
// Rows of up to U heads: their loads are all on their way before the first is used.
template <typename T, int P, int U>
struct Rows {
  Piece<T> v[U][P];
  __device__ __forceinline__ void load(const T* p, const Place<P>& pl, long step, int heads, uint32_t none = 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < P; ++i) v[u][i] = u < heads ? load8(p + 8 * pl.at[i]) : fill8<T>(none);
      p += step;
    }
  }
  __device__ __forceinline__ Part<P> get(int u) const {
    Part<P> x;
#pragma unroll
    for (int i = 0; i < P; ++i) x.r[i] = widen_row<P == 1>(v[u][i]);
    return x;
  }
};
template <typename T, int P>
__device__ __forceinline__ void store_part(T* p, const Place<P>& pl, const Part<P>& y) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float v[8];
    row_to<P == 1>(y.r[i], v);
    store8(p + 8 * pl.at[i], v);
  }
}
template <typename T, int P>
__device__ __forceinline__ Part<P> load_part(const T* p, const Place<P>& pl) {
  Part<P> x = {};
  if (pl.mine)
#pragma unroll
    for (int i = 0; i < P; ++i) x.r[i] = widen_row<P == 1>(load8(p + 8 * pl.at[i]));
  return x;
}
template <typename T, int P>
__device__ __forceinline__ void store_zeros(T* p, const Place<P>& pl, long step, int heads) {
  const float z[8] = {};
  for (int u = 0; u < heads; ++u, p += step)
#pragma unroll
    for (int i = 0; i < P; ++i) store8(p + 8 * pl.at[i], z);
}

}  // namespace

// ----------------------------------------------------------------- forward --
// A warp takes one head group of one token (warp w of the grid: token w / G,
// group w % G; the Gq groups of q come before k's); its rows share the token's
// rotation, the index arithmetic and one transposing reduction.
template <typename T, int P, int U>
__global__ void __launch_bounds__(32 * kWarps, P == 1 ? 3 : 2) qk_norm_rope_kernel(const RopeArgs a) {
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5), token = w / (unsigned)a.G;
  if (token >= (unsigned)a.tokens) return;
  const Group gr(a, w - token * (unsigned)a.G);
  const Place<P> pl(a.d, a.rot, gr.sub);
  const RopeTensor& t = a.t[gr.tsr];
  const int L = a.L, pass = a.pass[gr.tsr];
  const unsigned b = a.tokens == a.N ? 0 : token / (unsigned)a.N, n = token - b * (unsigned)a.N;
  const int heads = pl.mine ? gr.heads : 0;
  const long xstep = (32 / L) * t.xs[2], ystep = (32 / L) * t.ys[2];
  Rows<T, P, U> in;
  in.load(static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[1] + gr.h0 * t.xs[2], pl, xstep, heads);
  T* y0 = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[1] + gr.h0 * t.ys[2];
  const long p = a.pos ? (long)__ldg(a.pos + token) : n;
  if (p < 0) {  // padding
    store_zeros(y0, pl, ystep, heads);
    return;
  }
  const bool far = p >= a.T;  // no such row of the tables: NaN
  Turn<P> tn = load_turn(a.cos, a.sin, far ? 0 : p, a.rot, pl);
  // gamma goes into the rotation once for all of the warp's rows
  const Part<P> gm = load_part(static_cast<const T*>(t.gamma), pl);
  tn.c = mul_part(tn.c, gm);
  tn.s = mul_part(tn.s, others(gm));
  Sums<U> r;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r.v[u] = 0.f;
    if (u < pass) {
      const Part<P> f = in.get(u);
      r.v[u] = dot_part(f, f);
    }
  }
  r.reduce(L, gr.sub);
  r.apply([&](float ss) { return inv_rms(ss, a, far); });
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= pass) break;
    const uint64_t rr = both(r.take(u, L));
    const Part<P> y = mul_part(turn(in.get(u), tn, pl.on), rr);
    if (u < heads) store_part(y0, pl, y);
    y0 += ystep;
  }
}

// ---------------------------------------------------------------- backward --
// Warp w keeps its head group w % G and walks the tokens w / G, w / G + stride,
// ..., so its lanes hold the running dgamma of their channels in fp32
// registers: over kMostTokens tokens of at most 4 rows each, so that the error
// does not grow with the tokens (more of them are more rounds of CTAs: 720p x
// 40 heads 839 -> 843 us; sums taken to fp64 in shared memory every 32 tokens
// cost 1 % with one piece a lane and 7 % with two).  The sums of a CTA's warps
// are joined in shared memory in a fixed order and written as one partial row
// of q and one of k; dgamma_kernel adds the CTAs' rows in fp64, again in a
// fixed order: no atomics, the same bits every time.
template <typename T, int P, int U>
__global__ void __launch_bounds__(32 * kWarps, 2) qk_norm_rope_bwd_kernel(const RopeArgs a) {
  __shared__ float part[kWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, L = a.L;
  const unsigned w = blockIdx.x * kWarps + warp;
  const Group grp(a, w % (unsigned)a.G);
  const Place<P> pl(a.d, a.rot, grp.sub);
  const RopeTensor& t = a.t[grp.tsr];
  const int pass = a.pass[grp.tsr], heads = pl.mine ? grp.heads : 0;
  const long R = 32 / L, xstep = R * t.xs[2], gstep = R * t.dys[2], ystep = R * t.ys[2];
  launch_next();
  // A place without a head must not have a row of zeros: without eps its norm is
  // infinite, and 0 * inf would be in dgamma.  With one piece a lane its x is
  // about one (in all three types; g is 0), with two its factor is dropped: 0.5
  // and 0.7 % of the time, each the other way round 1.5 %.
  const uint32_t none = P == 1 && pl.mine ? 0x3f803f80u : 0;
  const Part<P> gm = load_part(static_cast<const T*>(t.gamma), pl);
  Part<P> sums = {};
  const unsigned first = w / (unsigned)a.G;
  const bool one = a.tokens == a.N;
  for (unsigned token = first; token < (unsigned)a.tokens && first < (unsigned)a.stride; token += (unsigned)a.stride) {
    const unsigned b = one ? 0 : token / (unsigned)a.N, n = token - b * (unsigned)a.N;
    Rows<T, P, U> in, gr;
    in.load(static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[1] + grp.h0 * t.xs[2], pl, xstep, heads, none);
    gr.load(static_cast<const T*>(t.dy) + b * t.dys[0] + n * t.dys[1] + grp.h0 * t.dys[2], pl, gstep, heads);
    T* dx = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[1] + grp.h0 * t.ys[2];
    const long p = a.pos ? (long)__ldg(a.pos + token) : n;
    if (p < 0) {  // padding: no gradient
      store_zeros(dx, pl, ystep, heads);
      continue;
    }
    const bool far = p >= a.T;
    Turn<P> tn = load_turn(a.cos, a.sin, far ? 0 : p, a.rot, pl);
#pragma unroll
    for (int i = 0; i < 4 * P; ++i) tn.s.r[i / 4].e[i % 4] = neg2(tn.s.r[i / 4].e[i % 4]);  // turned back
    // Both row sums come from x as it is: mean(u xh) = r mean(u x), and
    //   dx = r u - x r^3 mean(u x).
    Sums<U> r, m;
    Part<P> g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r.v[u] = m.v[u] = 0.f;
      g[u] = {};
      if (u < pass) {
        const Part<P> f = in.get(u);
        g[u] = turn(gr.get(u), tn, pl.on);
        r.v[u] = dot_part(f, f);
        m.v[u] = dot_part(g[u], mul_part(f, gm));
      }
    }
    r.reduce(L, grp.sub);
    m.reduce(L, grp.sub);
    r.apply([&](float ss) { return inv_rms(ss, a, far); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= pass) break;
      const float rt = r.take(u, L), rv = P == 1 || u < heads ? rt : 0.f;
      const uint64_t rr = both(rv), k = both(-(rv * (m.take(u, L) * a.inv_d)) * rv * rv);  // in this order: no overflow
      const Part<P> f = in.get(u), gs = mul_part(g[u], rr);
      Part<P> y = mul_part(gs, gm);
#pragma unroll
      for (int i = 0; i < 4 * P; ++i) {  // (where there is no head g is 0)
        sums.r[i / 4].e[i % 4] = f32x2_fma(gs.r[i / 4].e[i % 4], f.r[i / 4].e[i % 4], sums.r[i / 4].e[i % 4]);
        y.r[i / 4].e[i % 4] = f32x2_fma(f.r[i / 4].e[i % 4], k, y.r[i / 4].e[i % 4]);
      }
      if (u < heads) store_part(dx, pl, y);
      dx += ystep;
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j) {
    float acc[8];
    row_to<P == 1>(sums.r[j], acc);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < L && pl.mine)
#pragma unroll
      for (int i = 0; i < 8; ++i) part[warp][8 * pl.at[j] + i] = acc[i];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < a.d) {
    float s[2] = {0.f, 0.f};
    for (int v = 0; v < kWarps; ++v) s[(int)((blockIdx.x * kWarps + v) % (unsigned)a.G) >= a.Gq] += part[v][c];
    a.part[((size_t)blockIdx.x * 2) * a.d + c] = s[0];
    a.part[((size_t)blockIdx.x * 2 + 1) * a.d + c] = s[1];
  }
}

// dgamma of q (block.y 0) and k (1): eight channels a CTA, its 32 threads of a
// channel add the CTAs' partial rows in fp64.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* part, int rows, int d,
                                                     float* __restrict__ gq, float* __restrict__ gk) {
  __shared__ double s[32][8];
  float* out = blockIdx.y ? gk : gq;
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), r0 = threadIdx.x >> 3;
  double v = 0.0;
  wait_previous();
  for (int r = r0; r < rows; r += 32 * 10) {  // ten rows' loads in flight
    float x[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) x[i] = r + 32 * i < rows ? part[((size_t)(r + 32 * i) * 2 + blockIdx.y) * d + c] : 0.f;
#pragma unroll
    for (int i = 0; i < 10; ++i) v += (double)x[i];
  }
  s[r0][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8 && out) {
    v = 0.0;
    for (int r = 0; r < 32; ++r) v += s[r][threadIdx.x];
    out[c] = (float)v;
  }
}

namespace {

constexpr int kCtasPerSm = 2, kMostTokens = 128;

template <typename T, int P>
cudaError_t rope_launch(const RopeArgs& a0, bool back, int sms, cudaStream_t st) {
  constexpr int U = (sizeof(T) == 4 ? 4 : 8) / P, UB = (sizeof(T) == 4 ? 2 : 4) / P;
  RopeArgs a = a0;
  const int R = 32 / a.L, most = back ? UB : U;
  // Even groups of at most `most` passes; single ones where the tokens are too
  // few to give every SM four warps otherwise.
  const auto groups = [&](int tsr, int cap) {
    const int passes = (a.t[tsr].H + R - 1) / R, g = (passes + cap - 1) / cap;
    a.pass[tsr] = g ? (passes + g - 1) / g : 0;
    return g ? (passes + a.pass[tsr] - 1) / a.pass[tsr] : 0;
  };
  for (int cap = most;; cap = 1) {
    a.Gq = groups(0, cap);
    a.G = a.Gq + groups(1, cap);
    if (cap == 1 || a.tokens * a.G >= 4L * sms) break;
  }
  if (!back) {
    const long ctas = (a.tokens * a.G + kWarps - 1) / kWarps;
    qk_norm_rope_kernel<T, P, U><<<(unsigned)ctas, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int ctas = (int)rope_bwd_ctas(a.tokens, a.G, sms);  // under 2^23: tokens * G < 2^32
  a.stride = (long)ctas * kWarps / a.G;
  qk_norm_rope_bwd_kernel<T, P, UB><<<ctas, 32 * kWarps, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};  // may start under the end of the kernel before
  cfg.gridDim = dim3(a.d / 8, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dgamma_kernel, static_cast<const float*>(a.part), ctas, a.d, a.dgq, a.dgk);
}

}  // namespace

// CTAs of the backward pass: enough for every (token, group) pair or two an
// SM, and at least one warp a group.  Where a warp would walk more than
// kMostTokens, as many rounds of two an SM as leave it no more.
long rope_bwd_ctas(long tokens, int G, int sms) {
  const long full = (long)kCtasPerSm * sms, need = (tokens * G + kWarps - 1) / kWarps;
  const long rounds = (need + full * kMostTokens - 1) / (full * kMostTokens);
  const long ctas = need < full ? need : full * rounds;
  const long least = ((long)G + kWarps - 1) / kWarps;
  return ctas > least ? ctas : least;
}

size_t rope_bwd_workspace(int B, int N, int Hq, int Hk, int d, int sms) {
  // G is at most one group a head
  return (size_t)rope_bwd_ctas((long)B * N, Hq + Hk, sms) * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a0, int dtype, bool interleaved, bool back, int sms,
                                cudaStream_t st) {
  RopeArgs a = a0;
  a.L = 1;
  while ((interleaved ? 8 : 16) * a.L < a.d) a.L <<= 1;
  a.inv_d = 1.f / (float)a.d;
  if (dtype == 0)
    return interleaved ? rope_launch<__nv_bfloat16, 1>(a, back, sms, st) : rope_launch<__nv_bfloat16, 2>(a, back, sms, st);
  if (dtype == 1) return interleaved ? rope_launch<__half, 1>(a, back, sms, st) : rope_launch<__half, 2>(a, back, sms, st);
  return interleaved ? rope_launch<float, 1>(a, back, sms, st) : rope_launch<float, 2>(a, back, sms, st);
}

}  // namespace sagesla
