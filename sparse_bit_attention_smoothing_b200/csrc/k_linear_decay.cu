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
// the channels of v are the MMA's rows: a thread then owns half a row of the
// state (its channel of v, half of those of k) in fp32 registers, and S and P'
// never need a transposition.  What is not bf16 by itself is held in bf16
// parts whose sum is it: P' and S, which end in a bf16 output, in two parts
// (2^-16 of the value is left), l^{n-1-j} v_j, which ends in the fp32 state, in
// three (2^-24).
//
// HBM would allow 62 us at 12 heads of 32760 tokens of 128 (4 rows of d a token
// and head).  A call on inputs from HBM takes 188 us, one after another on the
// same buffers 157; all times in this file but the single tokens' are of the
// second kind.  Bound by latency: a chunk is 540 ns of an SM's
// share of HBM and 1700 cycles of the tensor pipe, but 4300 cycles (2.35 us)
// from one to the next, in which every step waits for another one: parts of v
// (2900 cycles of a warpgroup), products, the state (1650), S^T q, outputs (1300
// until their accumulator is free).  So each is a warpgroup of its own, with
// two buffers between them where TMEM has the columns.  Measured on the way
// (the same case, us): one order of the products for all chunks 224; what is
// ready first 171; the next chunk's own state beside the state that is still
// read (two areas), one test for all barriers, a second warp for the products
// of the outputs 165; the copies without a prefetch to L2 four chunks ahead 158.
// Slower: unrolled loops (184: the roles' code has to stay in the instruction
// cache), half chunks of v (178), two warpgroups for the outputs (159).
//
// Few heads do not fill the SMs, so a long sequence is cut into segments: a
// first launch sums each segment's own state, a second one carries the states
// across the segments, the third walks each segment from its state.  That reads
// k and v twice.  Up to kFold segments the walk carries the states itself, one
// launch less: 48 heads of 1000 tokens (d = 64, 3 segments) 31 -> 27 us; with
// 4 segments (d = 64) it is even, with 6 (d = 128) 24 heads of 4096 take 70 us
// and not 57 (a CTA reads up to 5 states one after another).
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "tensormap.h"

namespace sagesla {

namespace {

constexpr int kC = 64;            // tokens of a chunk
constexpr int kBlk = kC * 128;    // 64 tokens x 64 channels of bf16: rows of 128 bytes, 128-byte swizzle
constexpr int kPowers = kC + 1;

// TMEM columns.  v parts: l^{n-1-j} v_j [channels of v][two tokens a column],
// 32 columns a part.  The walk:
//   two buffers of P (64 rows: lanes 0-15 of each quadrant), each in turn
//   sum_j v_j P'_ij [channels of v][i] when P has been read;
//   S^T q_i [channels of v][i];
//   two areas of the state.  Chunk c's own state [channels of v][of k] comes
//   into area c + 1, and the threads that read it put the state before chunk
//   c + 1 in its place (S^T in two bf16 parts, two channels of k a column, each
//   warpgroup's high parts and then its low ones) while the state before chunk
//   c is still read in area c.
constexpr uint32_t kTOS = 192;
__device__ __forceinline__ uint32_t oi_col(int c) { return (c & 1) * 64; }
__device__ __forceinline__ uint32_t s_col(int c) { return 256 + (c & 1) * 128; }
template <bool kOut>
__device__ __forceinline__ uint32_t vp_col(int c) { return kOut ? 128 : (c & 1) * 96; }
template <bool kOut>
__device__ __forceinline__ uint32_t u_col(int c) { return s_col(kOut ? c + 1 : c); }

template <int D, bool kOut>
struct Lay {
  static constexpr int tile = D / 64 * kBlk;                 // one tensor's chunk
  static constexpr int tensors = kOut ? 3 : 2;               // (q), k, v
  static constexpr int stages = D == 64 ? (kOut ? 6 : 8) : kOut ? 3 : 5;
  static constexpr int stage = tensors * tile;
  static constexpr int third = stages * stage;               // walk: the third part of v [tokens][channels]
  static constexpr int pbuf = third + (kOut ? tile : 0);     // two of P' in two parts
  static constexpr int misc = pbuf + (kOut ? 4 * kBlk : 0);
  static constexpr int bytes = misc + 2816 + 1024;
};
constexpr int kThreads = 768;
// Registers of the six warpgroups (copies and MMAs, state, state, parts of v,
// P', outputs): they share what the CTA was launched with, 80 a thread.
constexpr int kRegs = 80, kRegsIssue = 40, kRegsState = 112, kRegsParts = 72, kRegsP = 72, kRegsOut = 72;
static_assert(kRegsIssue + 2 * kRegsState + kRegsParts + kRegsP + kRegsOut <= 6 * kRegs, "registers");
constexpr int kMaxSegments = 256;  // a thread of the carry's CTA for each
constexpr int kFold = 3;           // see above

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
// 16 lanes in fragments of 8 x 8 16-bit matrices.  Store: register 2k holds,
// of lane t/4, column 4k + t%4, register 2k + 1 the same of lane t/4 + 8.
__device__ __forceinline__ void tmem_st_16x128b(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
// Load: registers 4k, 4k + 1 hold, of lane t/4, columns 8k + 2 (t%4) and the
// next, registers 4k + 2, 4k + 3 the same of lane t/4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// Four 8 x 8 matrices of 16-bit values, transposed on the way.
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
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
// MMAs (of a walk: those that do not need the state, 2 the others), 4-11 the
// state (a channel of v and half of the channels of k a thread), 12-15 the
// parts of v, 16-19 P' (a segment's own state: the parts of v of every second
// chunk), 20-23 the outputs.
// kParts of v: three where the state leaves the kernel, two where it only
// feeds outputs (a walk whose states come from the carried segments).
//
// The parts of v are in TMEM: from shared memory the walk's MMAs would read
// 170 KB of it a chunk, not 100 KB, and two chunks' copies would fit, not three.
template <int D, bool kOut, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    linear_decay_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, const DecayArgs a, int* wd) {
  using L = Lay<D, kOut>;
  constexpr int NB = kOut ? 1 : 2;  // buffers of the parts of v and of the chunk's own state
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  struct Misc {
    uint64_t full[L::stages], empty[L::stages], vp_full[2], u_full[2], u_read[2];
    uint64_t p_full[2], s_full[2], s_read[2], pp_full[2], pp_empty[2], o_full, o_empty[2], fin;
    // l^m and scale l^m (twice, 16 banks apart) at kC + m, m <= kC; zeros before them
    float power[2 * kC + 16], out_power[2][2 * kC + 16];
    float whole[kFold];  // l^tokens of the segments, where the walk carries
    int bad[128];  // per channel of v: the segment's first token that is not finite
    uint32_t tmem;
    int abort;
  };
  static_assert(sizeof(Misc) <= 2816 && L::bytes <= 227 * 1024, "shared memory");
  Misc* ms = reinterpret_cast<Misc*>(smem + L::misc);
  volatile int* abort = &ms->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x, h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hk);
  const int len = a.lens ? max(0, min(a.N, __ldg(a.lens + b))) : a.N;
  const int t0 = seg * a.seg_tokens, t1 = min(a.N, t0 + a.seg_tokens);
  const int valid = max(0, min(len, t1) - t0), nc = (valid + kC - 1) / kC;
  const size_t bh = (size_t)b * a.H + h;
  if (!kOut) launch_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::stages; ++s) {
      mbar_init(&ms->full[s], 1);
      mbar_init(&ms->empty[s], kOut ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->vp_full[i], 4);
      mbar_init(&ms->u_full[i], 1);
      mbar_init(&ms->u_read[i], 8);
      mbar_init(&ms->pp_full[i], 4);
      mbar_init(&ms->pp_empty[i], 4);
      mbar_init(&ms->p_full[i], 1);
      mbar_init(&ms->s_full[i], 8);
      mbar_init(&ms->s_read[i], 1);
      mbar_init(&ms->o_empty[i], 4);
    }
    mbar_init(&ms->o_full, 1);
    mbar_init(&ms->fin, kOut ? 2 : 1);
    ms->abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x < 128) ms->bad[threadIdx.x] = INT32_MAX;
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kPowers) {
    const int m = threadIdx.x - 128;
    const float f = m ? (float)exp((double)__ldg(a.log_decay + h) * m) : 1.f;
    ms->power[kC + m] = f;
    ms->out_power[0][kC + m] = ms->out_power[1][kC + m] = a.scale * f;
    if (m < kC) ms->power[m] = ms->out_power[0][m] = ms->out_power[1][m] = 0.f;
  }
  constexpr bool kAlone = kOut && kParts == 3;  // one segment
  const bool fold = !kAlone && a.slots > a.nseg;
  if (kOut && fold && threadIdx.x >= 256 && threadIdx.x < 256 + a.nseg) {
    const int i = threadIdx.x - 256, n = max(0, min(len - i * a.seg_tokens, a.seg_tokens));
    ms->whole[i] = n ? (float)exp((double)__ldg(a.log_decay + h) * n) : 1.f;
  }
  if (warp == 1) tmem_alloc(&ms->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;  // the warp's TMEM lanes
  constexpr int oK = (kOut ? 1 : 0) * L::tile, oV = oK + L::tile;
  bool ok = true;
  auto all = [](bool x) { return __all_sync(0xffffffffu, x); };

  // The parts of l^{n-1-j} v_j of chunk c, a channel of v a thread, into TMEM
  // (two tokens a column), the walk's third part into shared memory.
  auto parts = [&](int c) {
    const int st = c % L::stages, n = min(kC, valid - c * kC);
    ok = all(mbar_wait(&ms->full[st], (c / L::stages) & 1, abort, wd));
    if (!ok) return;
    // The product that reads the buffer's last contents is over.  (Every warp
    // waits, with channels or without: none may arrive for a later chunk.)
    auto free_now = [&] {
      const int u = c + 2 - NB;  // that of the chunk NB before
      ok = all(mbar_wait(&ms->u_full[u & 1], ((u / 2) & 1) ^ 1, abort, wd));
      tc_fence_after();
    };
    const int q = warp & 3;
    bool touched = kOut && kParts == 3;
    if (32 * q < D) {
      // Row j of a tile: 128 bytes, 16-byte piece x at x ^ (j % 8).  The warp's
      // 32 channels are four pieces of block q / 2.
      uint8_t* vt = smem + st * L::stage + oV + (q / 2) * kBlk;
      const int p0 = 4 * (q & 1);
      if (n < kC) {  // rows behind the sequence's end hold anything: zeros in every product
        touched = true;
        for (int j = n + (lane >> 2); j < kC; j += 8) {
          const int off = j * 128 + (((p0 + (lane & 3)) ^ (j & 7)) << 4);
          *reinterpret_cast<uint4*>(vt + off) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(vt + (oK - oV) + off) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // Fragments: the lane holds channels lane / 4 and + 8 of 16, tokens
      // 2 (lane % 4) and the next of every 8.
      const float* pw = ms->power + kC + n - 1 - 2 * (lane & 3);
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t v[16], part[kParts][16];
        const int piece = p0 + 2 * hf + ((lane >> 3) & 1);
        const uint32_t row = (lane & 7) * 128 + ((piece ^ (lane & 7)) << 4) + (lane >> 4) * 1024;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ldsm_t(smem_u32(vt) + row + 2048 * k, v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        uint32_t tops[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 16; ++k) tops[k & 3] = __vmaxu2(tops[k & 3], v[k] & 0x7fff7fffu);
        const uint32_t top = __vmaxu2(__vmaxu2(tops[0], tops[1]), __vmaxu2(tops[2], tops[3]));
        if (max(top & 0xffffu, top >> 16) >= 0x7f80u) {
          // Not finite: 0 * NaN would reach earlier tokens of the chunk.  The
          // value leaves the products, and its channel is NaN from here on.
          touched = true;
#pragma unroll
          for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (((v[k] >> (16 * e)) & 0x7f80u) == 0x7f80u) {
                const int j = 8 * (k >> 1) + 2 * (lane & 3) + e, x = 16 * hf + 8 * (k & 1) + (lane >> 2);
                v[k] &= e ? 0x0000ffffu : 0xffff0000u;
                *reinterpret_cast<uint16_t*>(vt + j * 128 + (((p0 + x / 8) ^ (j & 7)) << 4) + 2 * (x & 7)) = 0;
                atomicMin(&ms->bad[32 * q + x], c * kC + j);
              }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {  // behind the end the power is 0
          float f = __fmul_rn(bf16_lo(v[k]), pw[-8 * (k >> 1)]), g = __fmul_rn(bf16_hi(v[k]), pw[-8 * (k >> 1) - 1]);
#pragma unroll
          for (int p = 0; p < kParts; ++p) part[p][k] = take_part(f, g);
        }
        if (hf == 0) free_now();  // the first half is computed under it
        const uint32_t to = tmem + quad + ((uint32_t)(16 * hf) << 16) + vp_col<kOut>(c);
        tmem_st_16x128b(to, part[0]);
        tmem_st_16x128b(to + 32, part[1]);
        if constexpr (kParts == 3) {
          if constexpr (kOut) {
            const uint32_t third = smem_u32(smem + L::third + (q / 2) * kBlk) + row;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              stsm_t(third + 2048 * k, part[2][4 * k], part[2][4 * k + 1], part[2][4 * k + 2], part[2][4 * k + 3]);
          } else {
            tmem_st_16x128b(to + 64, part[2]);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
    } else {
      free_now();
    }
    if (touched) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&ms->vp_full[c % NB]);
  };

  if (warp < 4) regs_fewer<kRegsIssue>();
  if (warp == 0) {
    // ------------------------------- copies -------------------------------
    int c = 0;
    for (; c < nc; ++c) {
      const int st = c % L::stages;
      ok = all(mbar_wait(&ms->empty[st], ((c / L::stages) & 1) ^ 1, abort, wd));
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
  } else if (warp == 1 || (kOut && warp == 2)) {
    // -------------------------------- MMAs --------------------------------
    const uint64_t kd = smem_desc_sw128(smem), mnd = desc_mn(smem, D == 128 ? kBlk : 0);
    constexpr uint32_t idP = idesc_ab(64, 64, 0, 0), idOI = idesc_ab(128, 64, 1, 0), idOS = idesc_ab(128, 64, 0, 0),
                       idU = idesc_ab(128, D, 0, 1), idU3 = idesc_ab(128, D, 1, 1);
    // What is ready goes first, each product when its operands are there and
    // its accumulator has been read (a fixed order waits for one of them with
    // the others ready).  A lane watches a barrier, so that one test asks for
    // all of them.
    constexpr uint32_t kOS = 0x103, kU = 0x1c, kP = 0x60, kOI = 0x280;  // the lanes of each
    uint64_t* bar = ms->s_full;  // its buffers, how many, the next one and its phase
    int bufs = 2, buf = 0, phase = 0;
    if (lane == 1) bar = ms->o_empty, buf = 1, phase = 1;  // of the chunk before
    if (lane == 2) bar = ms->vp_full, bufs = NB;
    if (lane == 3 || lane == 5 || lane == 8) bar = ms->full, bufs = L::stages;
    // its area: the state before the last chunk was in it (a segment's own: the last but one)
    if (lane == 4) bar = kOut ? ms->s_read : ms->u_read, buf = kOut, phase = 1;
    if (lane == 6) bar = ms->o_empty, phase = 1;  // of the chunk two before
    if (lane == 7) bar = ms->pp_full;
    if (lane == 9) bar = ms->u_full;  // v has no NaN left
    auto next = [&](uint32_t lanes) {
      if ((lanes >> lane & 1) && ++buf == bufs) buf = 0, phase ^= 1;
    };
    int ns = 0, nu = 0, nq = 0, no = 0, ne = 0;  // next chunk of each; next one whose copy is read
    long idle = 0;
    const bool outs = warp == 2;  // S^T q and V^T P', else the chunk's own state and P
    while ((kOut ? ne : nu) < nc) {
      const uint32_t ready = __ballot_sync(0xffffffffu, mbar_test(bar + buf, phase));
      bool some = false;
      __syncwarp();
      if (kOut && outs && nq < nc && (ready & kOS) == kOS) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t q0 = (nq % L::stages) * L::stage, ts = tmem + s_col(nq);
#pragma unroll 1
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ta(tmem + kTOS, ts + (kk / (D / 32)) * (D / 2) + p * (D / 4) + kk % (D / 32) * 8,
                          desc_at(kd, q0 + (kk / 4) * kBlk + (kk % 4) * 32), idOS, p > 0 || kk > 0);
          mma_commit(&ms->s_read[nq & 1]);
          if (no > nq) mma_commit(&ms->o_full);
        }
        __syncwarp();
        ++nq;
        next(kOS);
        some = true;
      }
      if (!outs && nu < nc && (ready & kU) == kU) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t k0 = (nu % L::stages) * L::stage + oK, tu = tmem + u_col<kOut>(nu), tv = tmem + vp_col<kOut>(nu);
#pragma unroll 1
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int kk = 0; kk < kC / 16; ++kk) {
              if (kOut && p == 2)
                mma_bf16(tu, desc_at(mnd, L::third + kk * 2048), desc_at(mnd, k0 + kk * 2048), idU3, 1);
              else
                mma_bf16_ta(tu, tv + 32 * p + 8 * kk, desc_at(mnd, k0 + kk * 2048), idU, p > 0 || kk > 0);
            }
          if (!kOut) mma_commit(&ms->empty[nu % L::stages]);
          mma_commit(&ms->u_full[nu & 1]);
        }
        __syncwarp();
        ++nu;
        next(kU);
        some = true;
      }
      if (kOut && !outs && ns < nc && (ready & kP) == kP) {
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (ns % L::stages) * L::stage + (kk / 4) * kBlk + (kk % 4) * 32;
            mma_bf16(tmem + oi_col(ns), desc_at(kd, off), desc_at(kd, off + oK), idP, kk > 0);
          }
          mma_commit(&ms->p_full[ns & 1]);
        }
        __syncwarp();
        ++ns;
        next(kP);
        some = true;
      }
      if (kOut && outs && no < nc && (ready & kOI) == kOI) {
        tc_fence_after();
        if (elect_one()) {
          const uint32_t v0 = (no % L::stages) * L::stage + oV, p0 = L::pbuf + (no & 1) * 2 * kBlk;
#pragma unroll 1
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < kC / 16; ++kk)
              mma_bf16(tmem + oi_col(no), desc_at(mnd, v0 + kk * 2048), desc_at(kd, p0 + p * kBlk + kk * 32), idOI,
                       p > 0 || kk > 0);
          if (nq > no) mma_commit(&ms->o_full);
        }
        __syncwarp();
        ++no;
        next(kOI);
        some = true;
      }
      // both of the warp's products have read it
      if (kOut && (outs ? ne < nq && ne < no : ne < nu && ne < ns)) {
        if (elect_one()) mma_commit(&ms->empty[ne % L::stages]);
        __syncwarp();
        ++ne;
      }
      if (some) {
        idle = 0;
      } else if (__any_sync(0xffffffffu, *abort || ++idle > kSpinLimit)) {
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
    // ------------------------------ the state -----------------------------
    regs_more<kRegsState>();
    constexpr int KD = D / 2;               // channels of k of the thread's
    const int ch = 32 * (warp & 3) + lane;  // channel of v
    const int kb = (warp >> 3) * KD;        // first channel of k
    const bool mine = ch < D;
    float S[KD];
    // Where the walk carries (fold): slot 0 of the workspace is a copy of the
    // state before the first token (state_out may be state_in), slot i + 1
    // segment i's own state, of the first one what leaves it.
    float* ws = a.ws + bh * a.slots * D * D + (size_t)kb * D + ch;
    const float* s0 = a.state_in && mine ? a.state_in + bh * D * D + (size_t)kb * D + ch : nullptr;
    if (kAlone) {
    } else if (kOut) {
      wait_previous();  // the segments' states (all else is the caller's)
      s0 = !mine || (fold && !seg && !a.state_in) ? nullptr : ws + (size_t)(fold ? min(seg, 1) : seg) * D * D;
    } else if (!fold || seg) {
      s0 = nullptr;
    }
#pragma unroll
    for (int k = 0; k < KD; ++k) S[k] = s0 ? s0[(size_t)k * D] : 0.f;
    if (!kOut && s0) {
#pragma unroll
      for (int k = 0; k < KD; ++k) ws[(size_t)k * D] = S[k];
    }
    if (kOut && fold && mine)
      for (int i = 1; i < seg; ++i) {
        const float* u = ws + (size_t)(i + 1) * D * D;
#pragma unroll
        for (int k = 0; k < KD; ++k) S[k] = __fmaf_rn(S[k], ms->whole[i], u[(size_t)k * D]);
      }
    auto put_state = [&](int c) {  // S^T in two bf16 parts, the A operand of chunk c's S^T q
      const uint32_t to = tmem + quad + s_col(c) + kb;
#pragma unroll
      for (int k0 = 0; k0 < KD; k0 += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float x = S[k0 + k], y = S[k0 + k + 1];
          hi[k / 2] = take_part(x, y);
          lo[k / 2] = take_part(x, y);
        }
        SAGESLA_TMEM_ST16(to + k0 / 2, hi);
        SAGESLA_TMEM_ST16(to + KD / 2 + k0 / 2, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->s_full[c & 1]);
    };
    if (kOut && nc) put_state(0);
    if (kOut && fold && mine && seg == a.nseg - 1 && a.state_out) {  // the last segment's state in fp32, as the others'
      float* to = a.state_out + bh * D * D + (size_t)kb * D + ch;
      const float* u = ws + (size_t)a.nseg * D * D;
#pragma unroll
      for (int k = 0; k < KD; ++k) to[(size_t)k * D] = __fmaf_rn(S[k], ms->whole[seg], u[(size_t)k * D]);
    }
    for (int c = 0; c < nc; ++c) {
      ok = all(mbar_wait(&ms->u_full[c & 1], (c / 2) & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const float f = ms->power[kC + min(kC, valid - c * kC)];
#pragma unroll
      for (int k0 = 0; k0 < KD; k0 += 32) {
        uint32_t u[32];
        SAGESLA_TMEM_LD32(tmem + quad + u_col<kOut>(c) + kb + k0, u);
        tmem_ld_wait();
        if (!kOut && k0 + 32 == KD) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->u_read[c & 1]);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) S[k0 + k] = __fmaf_rn(S[k0 + k], f, __uint_as_float(u[k]));
      }
      if (kOut && c + 1 < nc) put_state(c + 1);
    }
    float* to = !kOut ? ws + (size_t)(seg + fold) * D * D
                : kAlone && a.state_out ? a.state_out + bh * D * D + (size_t)kb * D + ch : nullptr;
    if (to && mine) {
      const bool nan = *reinterpret_cast<volatile int*>(&ms->bad[ch]) != INT32_MAX;
#pragma unroll
      for (int k = 0; k < KD; ++k) to[(size_t)k * D] = nan ? __int_as_float(0x7fffffff) : S[k];
    }
  } else if (warp >= 12 && warp < (kOut ? 16 : 20)) {
    // ------------------------------ parts of v ----------------------------
    regs_fewer<kRegsParts>();
    for (int c = kOut ? 0 : (warp - 12) / 4; ok && c < nc; c += kOut ? 1 : 2) parts(c);
  } else if (kOut && warp >= 16 && warp < 20) {
    // --------------------------------- P' ---------------------------------
    regs_fewer<kRegsP>();
    const int q = warp & 3, i = 16 * q + (lane & 15), jb = 32 * (lane >> 4);  // the thread's row and columns of P
    const float* pw = ms->out_power[lane >> 4] + kC + i - jb;  // scale l^{i-j} at -j (zeros behind the diagonal)
    for (int c = 0; c < nc; ++c) {
      ok = all(mbar_wait(&ms->p_full[c & 1], (c >> 1) & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      // the outputs of two chunks ago have left this buffer
      ok = all(mbar_wait(&ms->pp_empty[c & 1], ((c >> 1) & 1) ^ 1, abort, wd));
      if (!ok) break;
      uint8_t* pb = smem + L::pbuf + (c & 1) * 2 * kBlk + i * 128;
#pragma unroll 1
      for (int j0 = 0; j0 < 32; j0 += 16) {
        uint32_t p[16];
        SAGESLA_TMEM_LD2H_X16(tmem + quad + oi_col(c) + j0, 32, p);
        tmem_ld_wait();
        const float* pj = pw - j0;
        const int d = i - jb - j0;
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          uint32_t o[2][4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {  // a later token's score is dropped, not multiplied: it may be anything
            float x = d >= j + e ? __uint_as_float(p[j + e]) * pj[-(j + e)] : 0.f;
            float y = d >= j + e + 1 ? __uint_as_float(p[j + e + 1]) * pj[-(j + e + 1)] : 0.f;
            o[0][e / 2] = take_part(x, y);
            o[1][e / 2] = take_part(x, y);
          }
          const uint32_t off = (((jb + j0 + j) >> 3) ^ (i & 7)) << 4;
          *reinterpret_cast<uint4*>(pb + off) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<uint4*>(pb + kBlk + off) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->pp_full[c & 1]);
    }
  } else if (!kOut && warp >= 20) {
    regs_fewer<kRegsOut>();
  } else if (warp >= 20) {
    // ------------------------------- outputs ------------------------------
    regs_fewer<kRegsOut>();
    const int q = warp & 3;
    uint16_t* out = a.o + b * a.os[0] + h * a.os[2] + (long)t0 * a.os[1];
    for (int c = 0; c < nc; ++c) {
      ok = all(mbar_wait(&ms->o_full, c & 1, abort, wd));
      if (!ok) break;
      tc_fence_after();
      const int n = min(kC, valid - c * kC);
      if (32 * q < D) {
        // [channel of v][token] from TMEM to rows of 32 channels: transposed by
        // matrix stores into 64-byte rows of shared memory (piece x of row i at
        // x ^ (i / 2 % 4)), then 16 bytes a lane.  They lie where this chunk's
        // P' was, which no MMA reads any more.
        uint8_t* ob = smem + L::pbuf + (c & 1) * 2 * kBlk + q * 4096;
        const float* pw = ms->out_power[0] + kC + 1 + 2 * (lane & 3);  // scale l^{i+1}
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          const int b0 = ms->bad[32 * q + 16 * hf + (lane >> 2)] - c * kC, b1 = ms->bad[32 * q + 16 * hf + 8 + (lane >> 2)] - c * kC;
#pragma unroll 1
          for (int i0 = 0; i0 < kC; i0 += 32) {
            const uint32_t from = tmem + quad + ((uint32_t)(16 * hf) << 16) + i0;
            uint32_t oi[16], os[16], w[8];
            tmem_ld_16x256b(from + oi_col(c), oi);
            tmem_ld_16x256b(from + kTOS, os);
            tmem_ld_wait();
            if (hf == 1 && i0 + 32 == kC) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ms->o_empty[c & 1]);
            }
            if (min(b0, b1) < kC) {  // a v that was not finite: its channel is NaN from its token on
#pragma unroll
              for (int x = 0; x < 16; ++x)
                if (i0 + 8 * (x >> 2) + 2 * (lane & 3) + (x & 1) >= (x & 2 ? b1 : b0)) oi[x] = 0x7fffffffu;
            }
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const float2 f = *reinterpret_cast<const float2*>(pw - 1 + i0 + 8 * (x >> 2));
              const float g = pw[i0 + 8 * (x >> 2) + 1];
              const __nv_bfloat162 r = __floats2bfloat162_rn(__fmaf_rn(__uint_as_float(os[x]), f.y, __uint_as_float(oi[x])),
                                                             __fmaf_rn(__uint_as_float(os[x + 1]), g, __uint_as_float(oi[x + 1])));
              w[x / 2] = *reinterpret_cast<const uint32_t*>(&r);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int i = i0 + 16 * k + 8 * (lane >> 4) + (lane & 7);
              stsm_t(smem_u32(ob) + i * 64 + (((2 * hf + ((lane >> 3) & 1)) ^ ((i >> 1) & 3)) << 4), w[4 * k], w[4 * k + 1],
                     w[4 * k + 2], w[4 * k + 3]);
            }
          }
        }
        __syncwarp();
        uint16_t* row = out + (long)(c * kC + (lane >> 2)) * a.os[1] + 32 * q + 8 * (lane & 3);
#pragma unroll
        for (int i0 = 0; i0 < kC; i0 += 8) {
          const int i = i0 + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(ob + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
          if (i0 + (lane >> 2) < n) *reinterpret_cast<uint4*>(row) = w;
          row += 8 * a.os[1];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->pp_empty[c & 1]);
      } else if (lane == 0) {
        mbar_arrive(&ms->o_empty[c & 1]);
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

// More than kFold segments: across those of a (sequence, head), the state
// before each one in the place of its own state, and the last one out.  An
// element a thread.
__global__ void __launch_bounds__(256) linear_decay_carry_kernel(const DecayArgs a) {
  const int dd = a.d * a.d, at = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y, b = blockIdx.z;
  const size_t bh = (size_t)b * a.H + h;
  // Each segment's decay, once a CTA (64-bit exponentials in every thread took
  // as long as the sums).
  __shared__ float decay[kMaxSegments];
  const int len = a.lens ? max(0, min(a.N, __ldg(a.lens + b))) : a.N;
  launch_next();
  if (threadIdx.x < a.nseg) {
    const int n = max(0, min(len, ((int)threadIdx.x + 1) * a.seg_tokens) - (int)threadIdx.x * a.seg_tokens);
    decay[threadIdx.x] = n ? (float)exp((double)__ldg(a.log_decay + h) * n) : 1.f;
  }
  __syncthreads();
  float s = a.state_in ? a.state_in[bh * dd + at] : 0.f;
  wait_previous();
  float* ws = a.ws + bh * a.slots * dd + at;
  for (int i0 = 0; i0 < a.nseg; i0 += 16) {  // sixteen segments' loads in flight
    float u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = i0 + i < a.nseg ? ws[(size_t)(i0 + i) * dd] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i0 + i >= a.nseg) break;
      ws[(size_t)(i0 + i) * dd] = s;
      s = __fmaf_rn(s, decay[i0 + i], u[i]);
    }
  }
  if (a.state_out) a.state_out[bh * dd + at] = s;
}

// ----------------------------------------------------------- single tokens --
// Bound by the state's bytes (read and written once): 64 sequences of 40 heads
// take 54 us, 6.3 TB/s; one of 40 heads is all latency (4.9 us).  A CTA holds CW columns
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

// Shared memory, and that the warpgroups find the registers that they share
// out: with fewer they would wait for ever.
cudaError_t allow_walk(const void* fn, int bytes, std::atomic<unsigned long long>& done) {
  if (!done.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, fn);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kRegs) return cudaErrorInvalidKernelImage;
  }
  return allow_smem(fn, bytes, done);
}

template <int D>
cudaError_t decay_launch(DecayArgs a, int* wd, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, a.q, a.qs, a.B, a.N, a.H, D, a.step[0]) || !rows_map(&mk, a.k, a.ks, a.B, a.N, a.Hk, D, a.step[1]) ||
      !rows_map(&mv, a.v, a.vs, a.B, a.N, a.Hk, D, a.step[2]))
    return cudaErrorInvalidValue;
  const dim3 grid(a.nseg, a.H, a.B);
  // The second and third launch may start under the end of the one before.
  const auto run = [&](auto* fn, dim3 grid, int threads, int bytes, bool chained, auto... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, args...);
  };
  static std::atomic<unsigned long long> done[3] = {};
  const auto walk = [&](int i, auto* fn, int bytes, bool chained) {
    const cudaError_t e = allow_walk(reinterpret_cast<const void*>(fn), bytes, done[i]);
    if (e != cudaSuccess) return e;
    return run(fn, grid, kThreads, bytes, chained, mq, mk, mv, a, wd);
  };
  if (a.nseg == 1) return walk(0, linear_decay_kernel<D, true, 3>, Lay<D, true>::bytes, false);
  cudaError_t e = walk(1, linear_decay_kernel<D, false, 3>, Lay<D, false>::bytes, false);
  if (e != cudaSuccess) return e;
  if (a.slots == a.nseg && (e = run(linear_decay_carry_kernel, dim3(D * D / 256, a.H, a.B), 256, 0, true, a)) != cudaSuccess) return e;
  return walk(2, linear_decay_kernel<D, true, 2>, Lay<D, true>::bytes, true);
}

}  // namespace

// Segments of a sequence: as many as there are SMs for, where the walk that
// they shorten is worth the second pass over k and v and two more launches.  In
// chunks of a walk (2.35 us each): both passes take 1.34 a chunk, the launches
// and the ends of the kernels 5, or 3.5 without the carry's.  Measured, us with 1 and with s segments: 12
// heads of 32760 tokens 1204, 157 (12); 8 of 4096 156, 28 (16); 48 of 1000 (d =
// 64) 36, 27 (3); 2 of 500 20, 10 (8); 48 of 300 18, 33 (3); 80 of 4096 161, 188
// (3: two rounds of CTAs, never taken).
int linear_decay_segments(int B, int N, int H, int sms) {
  const long heads = (long)B * H, nc = (N + kC - 1) / kC;
  long best = 1;
  double cost = (double)nc;
  for (long s = 2; s <= nc && heads * s <= sms && s <= kMaxSegments; ++s) {
    const double c = 1.34 * (double)((nc + s - 1) / s) + (s <= kFold ? 3.5 : 5);
    if (c < cost) cost = c, best = s;
  }
  const long per = (nc + best - 1) / best;  // chunks of a segment
  return (int)((nc + per - 1) / per);
}

int linear_decay_slots(int nseg) { return nseg == 1 ? 0 : nseg <= kFold ? nseg + 1 : nseg; }

cudaError_t launch_linear_decay(const DecayArgs& a0, int* wd, cudaStream_t st) {
  DecayArgs a = a0;
  const int nc = (a.N + kC - 1) / kC;
  a.seg_tokens = (nc + a.nseg - 1) / a.nseg * kC;
  a.slots = linear_decay_slots(a.nseg);
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
