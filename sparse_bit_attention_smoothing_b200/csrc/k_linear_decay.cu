// k_linear_decay.cu -- causal linear attention with a decay for each head:
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   l = e^{g_h},
// the state S [d][d] in fp32 throughout.
//
// Prompts, in chunks of 64 tokens (i, j within the chunk, n of them valid):
//   P = Q K^T,   P'_ij = l^{i-j} P_ij for j <= i, else 0,
//   o_i = scale (sum_j P'_ij v_j + l^{i+1} q_i^T S),
//   S  <- l^n S + sum_j k_j (l^{n-1-j} v_j)^T.
// Only powers of l from 0 to 64 occur, so nothing overflows.
//
// Every product runs on the tensor cores with fp32 sums, transposed so that
// the channels of v are the MMA's rows: a thread then owns one row of the
// state (its channel of v, all channels of k) in fp32 registers, and S and P'
// never need a transposition.  What is not bf16 by itself is held in bf16
// parts whose sum is it: P' and S, which end in a bf16 output, in two parts
// (2^-16), l^{n-1-j} v_j, which ends in the fp32 state, in three (2^-24:
// with two the state is off by 3e-6, with three by 2e-7).
//
// Bound by HBM (4 rows of d a token and head, 64 KB a chunk at d = 128, 2850
// cycles of an SM's share).  Few heads do not fill the SMs, so a long sequence
// is cut into segments: a first launch sums each segment's own state, a second
// one carries the states across the segments, the third walks each segment
// from its state.  That reads k and v twice.
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

namespace sagesla {

namespace {

constexpr int kC = 64;            // tokens of a chunk
constexpr int kBlk = kC * 128;    // 64 tokens x 64 channels of bf16: rows of 128 bytes, 128-byte swizzle
constexpr int kPowers = kC + 1;

// TMEM columns.
constexpr uint32_t kTP = 0;      // P, two buffers of 64 (64 rows: lanes 0-15 of each quadrant)
constexpr uint32_t kTOI = 128;   // sum_j v_j P'_ij  [channels of v][i]
constexpr uint32_t kTOS = 192;   // S^T q_i          [channels of v][i]
constexpr uint32_t kTU = 256;    // the chunk's own state [channels of v][channels of k] (states only: two buffers, at 0 and 256)
constexpr uint32_t kTSH = 384, kTSL = 448;  // S^T in two bf16 parts, two channels of k a column

template <int D, bool kOut>
struct Lay {
  static constexpr int tile = D / 64 * kBlk;                 // one tensor's chunk
  static constexpr int tensors = kOut ? 3 : 2;               // (q), k, v
  static constexpr int stages = kOut ? 3 : 3;
  static constexpr int vbufs = kOut ? 1 : 2;                 // buffers of the three parts of l^{n-1-j} v_j
  static constexpr int stage = tensors * tile;
  static constexpr int vpart = stages * stage;
  static constexpr int pbuf = vpart + vbufs * 3 * tile;      // P' in two parts
  static constexpr int misc = pbuf + (kOut ? 2 * kBlk : 0);
  static constexpr int bytes = misc + 2048 + 1024;
  static constexpr int threads = kOut ? 384 : 256;
};

__device__ __forceinline__ uint64_t desc_mn(const void* p, uint32_t block_stride) {  // MN-major, 128-byte swizzle
  uint64_t d = (uint64_t)((smem_u32(p) >> 4) & 0x3FFF);
  d |= (uint64_t)((block_stride >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__host__ __device__ constexpr uint32_t idesc_ab(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16(M, N, b_mn) | ((uint32_t)a_mn << 15);
}
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int x, int n, int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(n), "r"(h), "r"(b), "r"(smem_u32(bar))
      : "memory");
}

// Two values in bf16 parts, packed (a low, b high); `a`, `b` become what is left.
__device__ __forceinline__ uint32_t take_part(float& a, float& b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
  a -= bf16_lo(w);
  b -= bf16_hi(w);
  return w;
}

}  // namespace

// kOut: the walk over a segment, with outputs.  Otherwise the segment's own
// state.  One CTA a (segment, head, sequence).  Warps: 0 the copies, 1 the
// MMAs, 4-7 the state (and the parts of v), 8-11 P' and the outputs.
template <int D, bool kOut>
__global__ void __launch_bounds__(kOut ? 384 : 256, 1)
    linear_decay_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, const DecayArgs a, int* wd) {
  using L = Lay<D, kOut>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  struct Misc {
    uint64_t full[L::stages], empty[L::stages], p_full[2], p_empty[2], vp_full[2], u_full[2], pp_full, o_full, o_empty, fin;
    float power[kPowers + 3];
    int bad[128];  // per channel of v: the segment's first token that is not finite
    uint32_t tmem;
    int abort;
  };
  static_assert(sizeof(Misc) <= 2048, "shared memory");
  Misc* ms = reinterpret_cast<Misc*>(smem + L::misc);
  volatile int* abort = &ms->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x, h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hk);
  const int len = a.lens ? max(0, min(a.N, __ldg(a.lens + b))) : a.N;
  const int t0 = seg * a.seg_tokens, t1 = min(a.N, t0 + a.seg_tokens);
  const int valid = max(0, min(len, t1) - t0), nc = (valid + kC - 1) / kC;
  const size_t bh = (size_t)b * a.H + h;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::stages; ++s) {
      mbar_init(&ms->full[s], 1);
      mbar_init(&ms->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->p_full[i], 1);
      mbar_init(&ms->p_empty[i], 4);
      mbar_init(&ms->vp_full[i], 4);
      mbar_init(&ms->u_full[i], 1);
    }
    mbar_init(&ms->pp_full, 4);
    mbar_init(&ms->o_full, 1);
    mbar_init(&ms->o_empty, 4);
    mbar_init(&ms->fin, 1);
    ms->abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x < 128) ms->bad[threadIdx.x] = INT32_MAX;
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kPowers) {
    const int m = threadIdx.x - 128;
    ms->power[m] = m ? (float)exp((double)__ldg(a.log_decay + h) * m) : 1.f;
  }
  if (warp == 1) tmem_alloc(&ms->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;  // the warp's TMEM lanes
  constexpr int oK = (kOut ? 1 : 0) * L::tile, oV = oK + L::tile;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------- copies -------------------------------
    int c = 0;
    for (; c < nc; ++c) {
      const int st = c % L::stages;
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->empty[st], ((c / L::stages) & 1) ^ 1, abort, wd));
      if (!ok) break;
      if (elect_one()) {
        uint8_t* dst = smem + st * L::stage;
        mbar_expect_tx(&ms->full[st], L::stage);
        const int n = t0 + c * kC;
#pragma unroll
        for (int x = 0; x < D; x += 64) {
          tma_load_4d(dst + oK + x / 64 * kBlk, &mk, x, n, hk * a.step[1][0], b * a.step[1][1], &ms->full[st]);
          if (kOut) tma_load_4d(dst + x / 64 * kBlk, &mq, x, n, h * a.step[0][0], b * a.step[0][1], &ms->full[st]);
          tma_load_4d(dst + oV + x / 64 * kBlk, &mv, x, n, hk * a.step[2][0], b * a.step[2][1], &ms->full[st]);
        }
      }
      __syncwarp();
    }
    // The copies are over before the CTA ends, also where a role gave up.
    for (int g = max(0, c - L::stages); g < c; ++g)
      if (!mbar_wait_drain(&ms->full[g % L::stages], (g / L::stages) & 1, wd)) break;
  } else if (warp == 1) {
    // -------------------------------- MMAs --------------------------------
    const uint64_t kd = smem_desc_sw128(smem), mnd = desc_mn(smem, D == 128 ? kBlk : 0);
    constexpr uint32_t idP = idesc_ab(64, 64, 0, 0), idOI = idesc_ab(128, 64, 1, 0), idOS = idesc_ab(128, 64, 0, 0),
                       idU = idesc_ab(128, D, 1, 1);
    auto scores = [&](int c) {  // P of chunk c
      const int st = c % L::stages;
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->full[st], (c / L::stages) & 1, abort, wd) &&
                                       mbar_wait(&ms->p_empty[c & 1], ((c >> 1) & 1) ^ 1, abort, wd));
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = st * L::stage + (kk / 4) * kBlk + (kk % 4) * 32;
          mma_bf16(tmem + kTP + 64 * (c & 1), desc_at(kd, off), desc_at(kd, off + oK), idP, kk > 0);
        }
        mma_commit(&ms->p_full[c & 1]);
      }
      __syncwarp();
    };
    if (kOut && nc) scores(0);
    for (int c = 0; ok && c < nc; ++c) {
      const int st = c % L::stages;
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->full[st], (c / L::stages) & 1, abort, wd) &&
                                       mbar_wait(&ms->vp_full[c & 1], (c >> 1) & 1, abort, wd));
      if (kOut && ok) ok = __all_sync(0xffffffffu, mbar_wait(&ms->o_empty, (c & 1) ^ 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t tu = kOut ? kTU : (c & 1) * 256;
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            mma_bf16(tmem + tu, desc_at(mnd, L::vpart + ((kOut ? 0 : (c & 1) * 3) + p) * L::tile + kk * 2048),
                     desc_at(mnd, st * L::stage + oK + kk * 2048), idU, p > 0 || kk > 0);
        if (kOut) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ta(tmem + kTOS, tmem + (p ? kTSL : kTSH) + kk * 8,
                          desc_at(kd, st * L::stage + (kk / 4) * kBlk + (kk % 4) * 32), idOS, p > 0 || kk > 0);
        } else {
          mma_commit(&ms->empty[st]);
        }
        mma_commit(&ms->u_full[c & 1]);
      }
      __syncwarp();
      if (!kOut) continue;
      if (c + 1 < nc) scores(c + 1);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&ms->pp_full, c & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            mma_bf16(tmem + kTOI, desc_at(mnd, st * L::stage + oV + kk * 2048),
                     desc_at(kd, L::pbuf + p * kBlk + kk * 32), idOI, p > 0 || kk > 0);
        mma_commit(&ms->o_full);
        mma_commit(&ms->empty[st]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&ms->fin);
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------- the state, parts of v ----------------------
    const int ch = 32 * (warp & 3) + lane;  // the thread's channel of v
    const bool mine = ch < D;
    float S[D];
    if (kOut) {
      const float* s0 = a.nseg > 1 ? a.ws + (bh * a.nseg + seg) * D * D : a.state_in ? a.state_in + bh * D * D : nullptr;
#pragma unroll
      for (int k = 0; k < D; ++k) S[k] = s0 && mine ? s0[(size_t)k * D + ch] : 0.f;
    } else {
#pragma unroll
      for (int k = 0; k < D; ++k) S[k] = 0.f;
    }
    auto put_state = [&]() {  // S^T in two bf16 parts, the A operand of S^T q
#pragma unroll
      for (int k0 = 0; k0 < D; k0 += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float x = S[k0 + k], y = S[k0 + k + 1];
          hi[k / 2] = take_part(x, y);
          lo[k / 2] = take_part(x, y);
        }
        SAGESLA_TMEM_ST16(tmem + quad + kTSH + k0 / 2, hi);
        SAGESLA_TMEM_ST16(tmem + quad + kTSL + k0 / 2, lo);
      }
      tmem_st_wait();
      tc_fence_before();
    };
    // The three parts of l^{n-1-j} v_j of chunk c (the fp32 product exactly).
    auto parts = [&](int c) {
      const int st = c % L::stages, n = min(kC, valid - c * kC);
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->full[st], (c / L::stages) & 1, abort, wd));
      if (!ok) return;
      uint8_t* kt = smem + st * L::stage + oK;
      uint8_t* vt = smem + st * L::stage + oV;
      uint8_t* vp = smem + L::vpart + (kOut ? 0 : (c & 1) * 3) * L::tile;
      const int u = lane & 7;
#pragma unroll 2
      for (int r = (warp & 3) * 4 + (lane >> 3); r < kC * (D / 64); r += 16) {
        const int j = r % kC;
        const uint32_t off = r * 128 + ((u ^ (j & 7)) << 4);  // row j of channel block r / 64
        uint4 v = *reinterpret_cast<const uint4*>(vt + off);
        if (j >= n) {  // rows behind the sequence's end hold anything: zeros in every product
          v = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(vt + off) = v;
          *reinterpret_cast<uint4*>(kt + off) = v;
        }
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t k7 = 0x7fff7fffu;
        const uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & k7, w[1] & k7), __vmaxu2(w[2] & k7, w[3] & k7));
        if (max(m2 & 0xffffu, m2 >> 16) >= 0x7f80u) {
          // Not finite: 0 * NaN would reach earlier tokens of the chunk.  The
          // value leaves the products, and its channel is NaN from here on.
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (((w[i / 2] >> (16 * (i & 1))) & 0x7f80u) == 0x7f80u) {
              w[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
              atomicMin(&ms->bad[r / kC * 64 + 8 * u + i], c * kC + j);
            }
          *reinterpret_cast<uint4*>(vt + off) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const float f = j < n ? ms->power[n - 1 - j] : 0.f;
        uint32_t o[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = __fmul_rn(bf16_lo(w[i]), f), y = __fmul_rn(bf16_hi(w[i]), f);
          o[0][i] = take_part(x, y);
          o[1][i] = take_part(x, y);
          o[2][i] = take_part(x, y);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *reinterpret_cast<uint4*>(vp + p * L::tile + off) = make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->vp_full[c & 1]);
    };
    if (kOut && nc) put_state();
    if (nc) parts(0);
    for (int c = 0; ok && c < nc; ++c) {
      if (!kOut && c + 1 < nc) parts(c + 1);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&ms->u_full[c & 1], (c >> 1) & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const float f = ms->power[min(kC, valid - c * kC)];
      const uint32_t tu = tmem + quad + (kOut ? kTU : (c & 1) * 256);
#pragma unroll
      for (int k0 = 0; k0 < D; k0 += 32) {
        uint32_t u[32];
        SAGESLA_TMEM_LD32(tu + k0, u);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k) S[k0 + k] = __fmaf_rn(S[k0 + k], f, __uint_as_float(u[k]));
      }
      tc_fence_before();
      if (kOut && c + 1 < nc) {
        put_state();  // u_full stands for the product that read the old one too
        parts(c + 1);
      }
    }
    float* to = kOut ? (a.nseg > 1 || !a.state_out ? nullptr : a.state_out + bh * D * D)
                     : a.ws + (bh * a.nseg + seg) * D * D;
    if (to && mine) {
      const bool nan = *reinterpret_cast<volatile int*>(&ms->bad[ch]) != INT32_MAX;
#pragma unroll
      for (int k = 0; k < D; ++k) to[(size_t)k * D + ch] = nan ? __int_as_float(0x7fffffff) : S[k];
    }
  } else if (kOut && warp >= 8) {
    // ----------------------------- P', outputs ----------------------------
    const int q = warp & 3, i = 16 * q + (lane & 15), jb = 32 * (lane >> 4);  // the thread's row and columns of P
    const int ch = 32 * q + lane;
    uint16_t* out = a.o + b * a.os[0] + h * a.os[2] + (long)t0 * a.os[1];
    for (int c = 0; c < nc; ++c) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->p_full[c & 1], (c >> 1) & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      uint32_t p[32];
      SAGESLA_TMEM_LD2H_X32(tmem + quad + kTP + 64 * (c & 1), 32, p);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->p_empty[c & 1]);
      uint8_t* pb = smem + L::pbuf;
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint32_t o[2][4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int g0 = i - (jb + j + e), g1 = g0 - 1;
          float x = g0 >= 0 ? __uint_as_float(p[j + e]) * ms->power[max(g0, 0)] : 0.f;
          float y = g1 >= 0 ? __uint_as_float(p[j + e + 1]) * ms->power[max(g1, 0)] : 0.f;
          o[0][e / 2] = take_part(x, y);
          o[1][e / 2] = take_part(x, y);
        }
        const uint32_t off = i * 128 + ((((jb + j) >> 3) ^ (i & 7)) << 4);
        *reinterpret_cast<uint4*>(pb + off) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
        *reinterpret_cast<uint4*>(pb + kBlk + off) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->pp_full);
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->o_full, c & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const int n = min(kC, valid - c * kC);
      if (32 * q < D) {
        const int bad = *reinterpret_cast<volatile int*>(&ms->bad[ch]) - c * kC;
        uint16_t* row = out + (long)c * kC * a.os[1] + ch;
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += 32) {
          uint32_t oi[32], os[32];
          SAGESLA_TMEM_LD32(tmem + quad + kTOI + i0, oi);
          SAGESLA_TMEM_LD32(tmem + quad + kTOS + i0, os);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float f = a.scale * __fmaf_rn(__uint_as_float(os[x]), ms->power[i0 + x + 1], __uint_as_float(oi[x]));
            if (i0 + x >= bad) f = __int_as_float(0x7fffffff);
            const __nv_bfloat16 r = __float2bfloat16_rn(f);
            if (i0 + x < n) row[(long)(i0 + x) * a.os[1]] = *reinterpret_cast<const uint16_t*>(&r);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->o_empty);
    }
    for (int n = valid + q; n < t1 - t0; n += 4)  // rows of padding
      if (lane < D / 8) *reinterpret_cast<uint4*>(out + (long)n * a.os[1] + 8 * lane) = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_drain(&ms->fin, 0, wd);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Across the segments of a (sequence, head): the state before each one in the
// place of its own state, and the last one out.  A thread takes 4 elements.
__global__ void __launch_bounds__(256) linear_decay_carry_kernel(const DecayArgs a) {
  const int dd = a.d * a.d, at = (blockIdx.x * 256 + threadIdx.x) * 4, h = blockIdx.y, b = blockIdx.z;
  if (at >= dd) return;
  const size_t bh = (size_t)b * a.H + h;
  const int len = a.lens ? max(0, min(a.N, __ldg(a.lens + b))) : a.N;
  const float g = __ldg(a.log_decay + h);
  float* ws = a.ws + bh * a.nseg * dd + at;
  float4 s = a.state_in ? *reinterpret_cast<const float4*>(a.state_in + bh * dd + at) : make_float4(0, 0, 0, 0);
  float4 next = *reinterpret_cast<const float4*>(ws);
  for (int i = 0; i < a.nseg; ++i) {
    const float4 u = next;
    if (i + 1 < a.nseg) next = *reinterpret_cast<const float4*>(ws + (size_t)(i + 1) * dd);
    *reinterpret_cast<float4*>(ws + (size_t)i * dd) = s;
    const int n = max(0, min(len, (i + 1) * a.seg_tokens) - i * a.seg_tokens);
    const float f = n ? (float)exp((double)g * n) : 1.f;
    s.x = __fmaf_rn(s.x, f, u.x);
    s.y = __fmaf_rn(s.y, f, u.y);
    s.z = __fmaf_rn(s.z, f, u.z);
    s.w = __fmaf_rn(s.w, f, u.w);
  }
  if (a.state_out) *reinterpret_cast<float4*>(a.state_out + bh * dd + at) = s;
}

// ----------------------------------------------------------- single tokens --
// Bound by the state's bytes (read and written once).  A CTA holds CW columns
// of one head's state, four a thread; all of a thread's loads are in flight
// before the first product.
template <int D, int CW>
__global__ void __launch_bounds__(256) linear_decay_step_kernel(const DecayArgs a) {
  constexpr int kLanes = CW / 4, kRows = 256 / kLanes, kEach = D / kRows;
  __shared__ float red[kRows][CW + 4];
  const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hk), t = threadIdx.x;
  const int cl = t % kLanes, rg = t / kLanes, c = blockIdx.x * CW + 4 * cl;
  const size_t at = ((size_t)b * a.H + h) * D * D + c;
  float4 s[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4*>(a.state_in + at + (size_t)(rg + i * kRows) * D));
  const uint16_t* q = a.q + b * a.qs[0] + h * a.qs[2];
  const uint16_t* k = a.k + b * a.ks[0] + hk * a.ks[2];
  const uint2 vw = __ldg(reinterpret_cast<const uint2*>(a.v + b * a.vs[0] + hk * a.vs[2] + c));
  const float v[4] = {bf16_lo(vw.x), bf16_hi(vw.x), bf16_lo(vw.y), bf16_hi(vw.y)};
  const float f = expf(__ldg(a.log_decay + h));
  float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = rg + i * kRows;
    const float kr = __uint_as_float((uint32_t)__ldg(k + r) << 16), qr = __uint_as_float((uint32_t)__ldg(q + r) << 16);
    s[i].x = __fmaf_rn(s[i].x, f, kr * v[0]);
    s[i].y = __fmaf_rn(s[i].y, f, kr * v[1]);
    s[i].z = __fmaf_rn(s[i].z, f, kr * v[2]);
    s[i].w = __fmaf_rn(s[i].w, f, kr * v[3]);
    __stcs(reinterpret_cast<float4*>(a.state_out + at + (size_t)r * D), s[i]);
    o.x = __fmaf_rn(qr, s[i].x, o.x);
    o.y = __fmaf_rn(qr, s[i].y, o.y);
    o.z = __fmaf_rn(qr, s[i].z, o.z);
    o.w = __fmaf_rn(qr, s[i].w, o.w);
  }
  *reinterpret_cast<float4*>(&red[rg][4 * cl]) = o;
  __syncthreads();
  if (t < CW) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) x += red[r][t];
    const __nv_bfloat16 r = __float2bfloat16_rn(x * a.scale);
    a.o[b * a.os[0] + h * a.os[2] + blockIdx.x * CW + t] = *reinterpret_cast<const uint16_t*>(&r);
  }
}

namespace {

// [B][N][H][d] rows of any strides as a 4-D map (channel, token, head, batch);
// an extent that is one, or read again and again (stride 0), becomes one with
// coordinate 0 (step 0).
bool rows_map(CUtensorMap* m, const void* p, const long s[3], int B, int N, int H, int d, int step[2]) {
  step[0] = H > 1 && s[2] > 0;
  step[1] = B > 1 && s[0] > 0;
  const bool many = N > 1 && s[1] > 0;
  if (N > 1 && !many) return false;
  const unsigned long dims[4] = {(unsigned long)d, (unsigned long)N, (unsigned long)(step[0] ? H : 1),
                                 (unsigned long)(step[1] ? B : 1)};
  const unsigned long str[3] = {(unsigned long)(many ? s[1] : d) * 2, (unsigned long)(step[0] ? s[2] : d) * 2,
                                (unsigned long)(step[1] ? s[0] : d) * 2};
  const unsigned box[4] = {64, kC, 1, 1};
  return tensor_map(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
cudaError_t decay_launch(DecayArgs a, int* wd, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, a.q, a.qs, a.B, a.N, a.H, D, a.step[0]) || !rows_map(&mk, a.k, a.ks, a.B, a.N, a.Hk, D, a.step[1]) ||
      !rows_map(&mv, a.v, a.vs, a.B, a.N, a.Hk, D, a.step[2]))
    return cudaErrorInvalidValue;
  const dim3 grid(a.nseg, a.H, a.B);
  cudaError_t e;
  if (a.nseg > 1) {
    auto* fn = linear_decay_kernel<D, false>;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, false>::bytes);
    if (e != cudaSuccess) return e;
    fn<<<grid, Lay<D, false>::threads, Lay<D, false>::bytes, st>>>(mq, mk, mv, a, wd);
    linear_decay_carry_kernel<<<dim3(D * D / 1024, a.H, a.B), 256, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto* fn = linear_decay_kernel<D, true>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, true>::bytes);
  if (e != cudaSuccess) return e;
  fn<<<grid, Lay<D, true>::threads, Lay<D, true>::bytes, st>>>(mq, mk, mv, a, wd);
  return cudaGetLastError();
}

}  // namespace

// Segments of a sequence: as many as keep the SMs busy, where the walk that
// they shorten is worth the second pass over k and v and two more launches
// (in chunks: a walk takes 1 a chunk, the first pass 0.6, the launches 8).
int linear_decay_segments(int B, int N, int H, int sms) {
  const long heads = (long)B * H, nc = (N + kC - 1) / kC;
  long best = 1;
  double cost = (double)nc * ((heads + sms - 1) / sms);
  for (long s = 2; s <= nc && heads * s <= 2L * sms; ++s) {
    const double c = 1.6 * (double)((nc + s - 1) / s) * ((heads * s + sms - 1) / sms) + 8;
    if (c < cost) cost = c, best = s;
  }
  const long per = (nc + best - 1) / best;  // chunks of a segment
  return (int)((nc + per - 1) / per);
}

cudaError_t launch_linear_decay(const DecayArgs& a0, int* wd, cudaStream_t st) {
  DecayArgs a = a0;
  const int nc = (a.N + kC - 1) / kC;
  a.seg_tokens = (nc + a.nseg - 1) / a.nseg * kC;
  return a.d == 64 ? decay_launch<64>(a, wd, st) : decay_launch<128>(a, wd, st);
}

cudaError_t launch_linear_decay_step(const DecayArgs& a, int sms, cudaStream_t st) {
  // Whole rows of the state a CTA where that fills the SMs, else quarters of them.
  const bool wide = (long)a.B * a.H >= 2L * sms;
  const dim3 grid(wide ? 1 : 4, a.H, a.B);
  if (a.d == 64) {
    if (wide)
      linear_decay_step_kernel<64, 64><<<grid, 256, 0, st>>>(a);
    else
      linear_decay_step_kernel<64, 16><<<grid, 256, 0, st>>>(a);
  } else {
    if (wide)
      linear_decay_step_kernel<128, 128><<<grid, 256, 0, st>>>(a);
    else
      linear_decay_step_kernel<128, 32><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace sagesla
