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
constexpr uint32_t kTU = 256;    // the chunk's own state [channels of v][channels of k]
constexpr uint32_t kTSH = 384, kTSL = 448;  // S^T in two bf16 parts, two channels of k a column

template <int D, bool kOut>
struct Lay {
  static constexpr int tile = D / 64 * kBlk;                 // one tensor's chunk
  static constexpr int tensors = kOut ? 3 : 2;               // (q), k, v
  static constexpr int stages = D == 128 && kOut ? 2 : 3;
  static constexpr int stage = tensors * tile;
  static constexpr int vpart = stages * stage;               // two buffers of the parts of l^{n-1-j} v_j
  static constexpr int pbuf = vpart + 2 * 3 * tile;          // two of P' in two parts
  static constexpr int misc = pbuf + (kOut ? 4 * kBlk : 0);
  static constexpr int bytes = misc + 1536 + 1024;
  static constexpr int threads = kOut ? 640 : 384;
};
// Registers of the walk's five warpgroups (copies and MMAs, state, state, P',
// outputs): they share what the CTA was launched with, 96 a thread.
constexpr int kRegs = 96, kRegsIssue = 40, kRegsState = 120, kRegsP = 88, kRegsO = 104;
static_assert(kRegsIssue + 2 * kRegsState + kRegsP + kRegsO <= 5 * kRegs, "registers");
constexpr int kAhead = 4;  // chunks that are brought to L2 before their copy to shared memory is issued

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

template <int kN>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}
__device__ __forceinline__ void tma_prefetch_4d(const void* map, int x, int n, int h, int b) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map), "r"(x), "r"(n),
               "r"(h), "r"(b)
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
// MMAs, 4-11 the state (a channel of v and half of the channels of k a
// thread) and the parts of v, 12-15 P', 16-19 the outputs.
// kParts of v: three where the state leaves the kernel, two where it only
// feeds outputs (a walk whose states come from the carried segments).
template <int D, bool kOut, int kParts>
__global__ void __launch_bounds__(kOut ? 640 : 384, 1)
    linear_decay_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, const DecayArgs a, int* wd) {
  using L = Lay<D, kOut>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  struct Misc {
    uint64_t full[L::stages], empty[L::stages], p_full[2], p_empty[2], vp_full[2], u_full, s_full, s_read, pp_full[2], pp_empty[2], o_full, o_empty, fin;
    float power[kPowers + 3];   // l^m
    float out_power[kC];        // scale l^{i+1}
    int bad[128];  // per channel of v: the segment's first token that is not finite
    uint32_t tmem;
    int abort;
  };
  static_assert(sizeof(Misc) <= 1536 && L::bytes <= 227 * 1024, "shared memory");
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
      mbar_init(&ms->vp_full[i], 8);
      mbar_init(&ms->pp_full[i], 4);
      mbar_init(&ms->pp_empty[i], 4);
    }
    mbar_init(&ms->u_full, 1);
    mbar_init(&ms->s_full, 8);
    mbar_init(&ms->s_read, 1);
    mbar_init(&ms->o_full, 1);
    mbar_init(&ms->o_empty, 4);
    mbar_init(&ms->fin, 1);
    ms->abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x < 128) ms->bad[threadIdx.x] = INT32_MAX;
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kPowers) {
    const int m = threadIdx.x - 128;
    const float f = m ? (float)exp((double)__ldg(a.log_decay + h) * m) : 1.f;
    ms->power[m] = f;
    if (m) ms->out_power[m - 1] = a.scale * f;
  }
  if (warp == 1) tmem_alloc(&ms->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;  // the warp's TMEM lanes
  constexpr int oK = (kOut ? 1 : 0) * L::tile, oV = oK + L::tile;
  bool ok = true;

  if (kOut && warp < 4) regs_fewer<kRegsIssue>();
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
        const int n = t0 + c * kC, ahead = n + kAhead * kC;
#pragma unroll
        for (int x = 0; x < D; x += 64) {
          if (c + kAhead < nc) {
            tma_prefetch_4d(&mk, x, ahead, hk * a.step[1][0], b * a.step[1][1]);
            if (kOut) tma_prefetch_4d(&mq, x, ahead, h * a.step[0][0], b * a.step[0][1]);
            tma_prefetch_4d(&mv, x, ahead, hk * a.step[2][0], b * a.step[2][1]);
          }
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
    // What is ready goes first: the next scores, the next chunk's own state,
    // S^T q and V^T P' of the next chunk, each when its operands are there and
    // its accumulator has been read (a fixed order waits for one of them with
    // the others ready: 5350 cycles a chunk).
    auto done = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)); };
    int ns = 0, nu = 0, nq = 0, no = 0;  // next chunk of each
    long idle = 0;
    while ((kOut ? no : nu) < nc) {
      bool some = false;
      if (kOut && ns < nc && done(&ms->full[ns % L::stages], ns / L::stages) && done(&ms->p_empty[ns & 1], (ns >> 1) + 1)) {
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (ns % L::stages) * L::stage + (kk / 4) * kBlk + (kk % 4) * 32;
            mma_bf16(tmem + kTP + 64 * (ns & 1), desc_at(kd, off), desc_at(kd, off + oK), idP, kk > 0);
          }
          mma_commit(&ms->p_full[ns & 1]);
        }
        __syncwarp();
        ++ns;
        some = true;
      }
      if (nu < nc && done(&ms->full[nu % L::stages], nu / L::stages) && done(&ms->vp_full[nu & 1], nu >> 1) &&
          done(&ms->s_full, kOut ? nu : nu + 1)) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t k0 = (nu % L::stages) * L::stage + oK, v0 = L::vpart + (nu & 1) * 3 * L::tile;
#pragma unroll
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int kk = 0; kk < kC / 16; ++kk)
              mma_bf16(tmem + kTU, desc_at(mnd, v0 + p * L::tile + kk * 2048), desc_at(mnd, k0 + kk * 2048), idU,
                       p > 0 || kk > 0);
          if (!kOut) mma_commit(&ms->empty[nu % L::stages]);
          mma_commit(&ms->u_full);
        }
        __syncwarp();
        ++nu;
        some = true;
      }
      if (kOut && nq < nu && done(&ms->o_empty, nq + 1)) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t q0 = (nq % L::stages) * L::stage;
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ta(tmem + kTOS, tmem + (p ? kTSL : kTSH) + kk * 8, desc_at(kd, q0 + (kk / 4) * kBlk + (kk % 4) * 32),
                          idOS, p > 0 || kk > 0);
          mma_commit(&ms->s_read);
        }
        __syncwarp();
        ++nq;
        some = true;
      }
      if (kOut && no < nq && done(&ms->pp_full[no & 1], no >> 1)) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t v0 = (no % L::stages) * L::stage + oV, p0 = L::pbuf + (no & 1) * 2 * kBlk;
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < kC / 16; ++kk)
              mma_bf16(tmem + kTOI, desc_at(mnd, v0 + kk * 2048), desc_at(kd, p0 + p * kBlk + kk * 32), idOI,
                       p > 0 || kk > 0);
          mma_commit(&ms->o_full);
          mma_commit(&ms->empty[no % L::stages]);
        }
        __syncwarp();
        ++no;
        some = true;
      }
      idle = some ? 0 : idle + 1;
      ok = !__any_sync(0xffffffffu, *abort || idle > kSpinLimit);
      if (!ok) {
        if (lane == 0 && !*abort) {
          *abort = 1;
          atomicExch(wd, 1);
        }
        break;
      }
    }
    if (elect_one()) mma_commit(&ms->fin);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ------------------------- the state, parts of v ----------------------
    if (kOut) regs_more<kRegsState>();
    constexpr int KD = D / 2;               // channels of k of the thread's
    const int ch = 32 * (warp & 3) + lane;  // channel of v
    const int kb = (warp >> 3) * KD;        // first channel of k
    const bool mine = ch < D;
    float S[KD];
    if (kOut) {
      const float* s0 = a.nseg > 1 ? a.ws + (bh * a.nseg + seg) * D * D : a.state_in ? a.state_in + bh * D * D : nullptr;
#pragma unroll
      for (int k = 0; k < KD; ++k) S[k] = s0 && mine ? s0[(size_t)(kb + k) * D + ch] : 0.f;
    } else {
#pragma unroll
      for (int k = 0; k < KD; ++k) S[k] = 0.f;
    }
    auto put_state = [&]() {  // S^T in two bf16 parts, the A operand of S^T q
#pragma unroll
      for (int k0 = 0; k0 < KD; k0 += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float x = S[k0 + k], y = S[k0 + k + 1];
          hi[k / 2] = take_part(x, y);
          lo[k / 2] = take_part(x, y);
        }
        SAGESLA_TMEM_ST16(tmem + quad + kTSH + (kb + k0) / 2, hi);
        SAGESLA_TMEM_ST16(tmem + quad + kTSL + (kb + k0) / 2, lo);
      }
      tmem_st_wait();
      tc_fence_before();
    };
    // The parts of l^{n-1-j} v_j of chunk c.
    auto parts = [&](int c) {
      const int st = c % L::stages, n = min(kC, valid - c * kC);
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->full[st], (c / L::stages) & 1, abort, wd));
      if (!ok) return;
      uint8_t* kt = smem + st * L::stage + oK;
      uint8_t* vt = smem + st * L::stage + oV;
      uint8_t* vp = smem + L::vpart + (c & 1) * 3 * L::tile;
      constexpr int kRows = kC * (D / 64) / 32;  // rows (of 64 channels) a thread
      const int u = lane & 7, r0 = (warp - 4) * 4 + (lane >> 3);
      uint4 v[kRows];
      uint32_t m2 = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {  // row j of channel block r / 64
        const int r = r0 + 32 * i, j = r % kC;
        v[i] = *reinterpret_cast<const uint4*>(vt + r * 128 + ((u ^ (j & 7)) << 4));
      }
      if (n < kC) {  // rows behind the sequence's end hold anything: zeros in every product
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + 32 * i, j = r % kC;
          if (j >= n) {
            v[i] = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(vt + r * 128 + ((u ^ (j & 7)) << 4)) = v[i];
            *reinterpret_cast<uint4*>(kt + r * 128 + ((u ^ (j & 7)) << 4)) = v[i];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint32_t k7 = 0x7fff7fffu;
        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[i].x & k7, v[i].y & k7), __vmaxu2(v[i].z & k7, v[i].w & k7)));
      }
      if (max(m2 & 0xffffu, m2 >> 16) >= 0x7f80u) {
        // Not finite: 0 * NaN would reach earlier tokens of the chunk.  The
        // value leaves the products, and its channel is NaN from here on.
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + 32 * i, j = r % kC;
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (((w[e / 2] >> (16 * (e & 1))) & 0x7f80u) == 0x7f80u) {
              w[e / 2] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
              atomicMin(&ms->bad[r / kC * 64 + 8 * u + e], c * kC + j);
            }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(vt + r * 128 + ((u ^ (j & 7)) << 4)) = v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = r0 + 32 * i, j = r % kC;
        const float f = ms->power[max(n - 1 - j, 0)];
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[kParts][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = __fmul_rn(bf16_lo(w[e]), f), y = __fmul_rn(bf16_hi(w[e]), f);
#pragma unroll
          for (int p = 0; p < kParts; ++p) o[p][e] = take_part(x, y);
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          *reinterpret_cast<uint4*>(vp + p * L::tile + r * 128 + ((u ^ (j & 7)) << 4)) =
              make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->vp_full[c & 1]);
    };
    if (kOut && nc) {
      put_state();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->s_full);
    }
    if (nc) parts(0);
    for (int c = 0; ok && c < nc; ++c) {
      // The next chunk's parts come first where its copies are there already.
      const int nx = (c + 1) % L::stages;
      const bool early = c + 1 < nc && __all_sync(0xffffffffu, mbar_test(&ms->full[nx], ((c + 1) / L::stages) & 1));
      if (early) parts(c + 1);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&ms->u_full, c & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const float f = ms->power[min(kC, valid - c * kC)];
#pragma unroll
      for (int k0 = 0; k0 < KD; k0 += 32) {
        uint32_t u[32];
        SAGESLA_TMEM_LD32(tmem + quad + kTU + kb + k0, u);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k) S[k0 + k] = __fmaf_rn(S[k0 + k], f, __uint_as_float(u[k]));
      }
      tc_fence_before();
      if (c + 1 < nc) {
        if (kOut) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ms->s_read, c & 1, abort, wd));  // S^T q has read the old state
          if (!ok) break;
          tc_fence_after();
          put_state();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->s_full);
        if (!early) parts(c + 1);
      }
    }
    float* to = kOut ? (a.nseg > 1 || !a.state_out ? nullptr : a.state_out + bh * D * D)
                     : a.ws + (bh * a.nseg + seg) * D * D;
    if (to && mine) {
      const bool nan = *reinterpret_cast<volatile int*>(&ms->bad[ch]) != INT32_MAX;
#pragma unroll
      for (int k = 0; k < KD; ++k) to[(size_t)(kb + k) * D + ch] = nan ? __int_as_float(0x7fffffff) : S[k];
    }
  } else if (kOut && warp >= 12 && warp < 16) {
    // --------------------------------- P' ---------------------------------
    regs_fewer<kRegsP>();
    const int q = warp & 3, i = 16 * q + (lane & 15), jb = 32 * (lane >> 4);  // the thread's row and columns of P
    float fac[32];  // scale l^{i-j}: the same in every chunk
#pragma unroll
    for (int j = 0; j < 32; ++j) fac[j] = a.scale * ms->power[max(i - jb - j, 0)];
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
      // the outputs of two chunks ago have left this buffer
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->pp_empty[c & 1], ((c >> 1) & 1) ^ 1, abort, wd));
      if (!ok) break;
      uint8_t* pb = smem + L::pbuf + (c & 1) * 2 * kBlk + i * 128;
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint32_t o[2][4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // a later token's score is dropped, not multiplied: it may be anything
          float x = i - jb >= j + e ? __uint_as_float(p[j + e]) * fac[j + e] : 0.f;
          float y = i - jb >= j + e + 1 ? __uint_as_float(p[j + e + 1]) * fac[j + e + 1] : 0.f;
          o[0][e / 2] = take_part(x, y);
          o[1][e / 2] = take_part(x, y);
        }
        const uint32_t off = (((jb + j) >> 3) ^ (i & 7)) << 4;
        *reinterpret_cast<uint4*>(pb + off) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
        *reinterpret_cast<uint4*>(pb + kBlk + off) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->pp_full[c & 1]);
    }
  } else if (kOut && warp >= 16) {
    // ------------------------------- outputs ------------------------------
    regs_more<kRegsO>();
    const int q = warp & 3, ch = 32 * q + lane;
    uint16_t* out = a.o + b * a.os[0] + h * a.os[2] + (long)t0 * a.os[1];
    for (int c = 0; c < nc; ++c) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ms->o_full, c & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const int n = min(kC, valid - c * kC);
      if (32 * q < D) {
        // [channel of v][token] from TMEM to rows of 32 channels: 64-byte rows
        // in shared memory, then 16 bytes a lane.  They lie where this chunk's
        // P' was, which no MMA reads any more.
        uint8_t* ob = smem + L::pbuf + (c & 1) * 2 * kBlk + q * 4096;
        const int bad = *reinterpret_cast<volatile int*>(&ms->bad[ch]) - c * kC;
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += 32) {
          uint32_t oi[32], os[32];
          SAGESLA_TMEM_LD32(tmem + quad + kTOI + i0, oi);
          SAGESLA_TMEM_LD32(tmem + quad + kTOS + i0, os);
          tmem_ld_wait();
          if (i0 + 32 == kC) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->o_empty);
          }
          uint16_t* to = reinterpret_cast<uint16_t*>(ob + i0 * 64) + lane;
          if (bad < kC) {
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (i0 + x >= bad) oi[x] = 0x7fffffffu;
          }
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(
                __fmaf_rn(__uint_as_float(os[x]), ms->out_power[i0 + x], __uint_as_float(oi[x])),
                __fmaf_rn(__uint_as_float(os[x + 1]), ms->out_power[i0 + x + 1], __uint_as_float(oi[x + 1])));
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&r);
            to[x * 32] = (uint16_t)w;
            to[(x + 1) * 32] = (uint16_t)(w >> 16);
          }
        }
        __syncwarp();
        uint16_t* row = out + (long)(c * kC + (lane >> 2)) * a.os[1] + 32 * q + 8 * (lane & 3);
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += 8) {
          const uint4 w = *reinterpret_cast<const uint4*>(ob + (i0 + (lane >> 2)) * 64 + 16 * (lane & 3));
          if (i0 + (lane >> 2) < n) *reinterpret_cast<uint4*>(row) = w;
          row += 8 * a.os[1];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->pp_empty[c & 1]);
      } else if (lane == 0) {
        mbar_arrive(&ms->o_empty);
        mbar_arrive(&ms->pp_empty[c & 1]);
      }
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
// place of its own state, and the last one out.  An element a thread.
__global__ void __launch_bounds__(256) linear_decay_carry_kernel(const DecayArgs a) {
  const int dd = a.d * a.d, at = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y, b = blockIdx.z;
  const size_t bh = (size_t)b * a.H + h;
  const int len = a.lens ? max(0, min(a.N, __ldg(a.lens + b))) : a.N;
  const float g = __ldg(a.log_decay + h);
  float* ws = a.ws + bh * a.nseg * dd + at;
  float s = a.state_in ? a.state_in[bh * dd + at] : 0.f;
  for (int i0 = 0; i0 < a.nseg; i0 += 16) {  // sixteen segments' loads in flight
    float u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = i0 + i < a.nseg ? ws[(size_t)(i0 + i) * dd] : 0.f;
    const float whole = (float)exp((double)g * a.seg_tokens);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i0 + i >= a.nseg) break;
      ws[(size_t)(i0 + i) * dd] = s;
      const int n = max(0, min(len, (i0 + i + 1) * a.seg_tokens) - (i0 + i) * a.seg_tokens);
      s = __fmaf_rn(s, n == a.seg_tokens ? whole : n ? (float)exp((double)g * n) : 1.f, u[i]);
    }
  }
  if (a.state_out) a.state_out[bh * dd + at] = s;
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
  const auto run = [&](auto* fn, int threads, int bytes) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (threads == 640) {  // the walk's warpgroups share out exactly these registers: with fewer they would wait for ever
      cudaFuncAttributes at;
      if ((e = cudaFuncGetAttributes(&at, fn)) != cudaSuccess) return e;
      if (at.numRegs < kRegs) return cudaErrorInvalidKernelImage;
    }
    fn<<<grid, threads, bytes, st>>>(mq, mk, mv, a, wd);
    return cudaGetLastError();
  };
  using States = Lay<D, false>;
  using Walk = Lay<D, true>;
  if (a.nseg == 1) return run(linear_decay_kernel<D, true, 3>, Walk::threads, Walk::bytes);
  cudaError_t e = run(linear_decay_kernel<D, false, 3>, States::threads, States::bytes);
  if (e != cudaSuccess) return e;
  linear_decay_carry_kernel<<<dim3(D * D / 256, a.H, a.B), 256, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return run(linear_decay_kernel<D, true, 2>, Walk::threads, Walk::bytes);
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
