// kernels.h -- host-side launchers of the SageSLA kernels (internal; the
// public C ABI is include/sagesla.h).  All launchers are asynchronous on
// `st` and return the cudaGetLastError() of their launch.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace sagesla {

// Raises a kernel's dynamic shared memory limit once per device (`done`: a bit
// a device; the call costs as much as a small launch's checks).
inline cudaError_t allow_smem(const void* fn, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Geometry shared by the launchers.
struct Geom {
  int BH;      // B*H
  int N;       // tokens
  int block;   // 64 or 128 (mask block)
  int nb;      // ceil(N/block)
  int nq;      // 64-token quantisation tiles per head, padded: 2*ceil(N/128)
  int kc;      // key blocks kept per query block
  int split;   // row splits of the statistics pass
  int H = 1;   // heads (B = BH / H)
  int tok = 0; // q, k, v, out layout: 0 = [B][H][N][d], 1 = [B][N][H][d] (token-major, as a DiT emits it)
};

// QK RMSNorm applied where a kernel loads q or k (inv == nullptr: off):
// x * inv[b][n] * gamma[h*d + c], rounded to bf16.
struct QKNorm {
  const float* inv = nullptr;  // [B][N] per-token 1 / rms over the H*d channels
  const uint4* gamma = nullptr;  // bf16 [H*d] as 16-byte units (8 channels each)
  int H = 1, N = 1;
};
// Per-token 1 / rms of q and k (QK RMSNorm), [B][N] each.
cudaError_t launch_rms_inv(const void* q, const void* k, int B, int H, int N, double eps, float* inv_q, float* inv_k,
                           cudaStream_t st, int tok = 0);
// K1: per-split fp64 sums of K and fp32 max|V| per channel.
cudaError_t launch_stats_partial(const void* k, const void* v, const Geom& g, double* psum, float* pmax,
                                 cudaStream_t st, QKNorm nk = QKNorm());
// K1b: mu = fl32(sum/N); V scale amax/448 and multiplier 448/amax per channel.
cudaError_t launch_stats_final(const double* psum, const float* pmax, const Geom& g, float* mu, float* sv,
                               float* mv, cudaStream_t st);
// K2: smoothing + INT8 Q/K tiles + FP8 V^T tiles + per-64-row pooled sums.
cudaError_t launch_quant(const void* q, const void* k, const void* v, const float* mu, const float* mv,
                         const Geom& g, uint8_t* q8t, uint8_t* k8t, uint8_t* v8t, float* sq, float* sk,
                         float* qsum, float* ksum, int* wd, cudaStream_t st, int qmax = 127, int q_tok = 0,
                         QKNorm nq = QKNorm(), QKNorm nk = QKNorm());
// Untile the quantised tiles back to row-major codes (parity entry only).
cudaError_t launch_untile(const uint8_t* q8t, const uint8_t* k8t, const uint8_t* v8t, const Geom& g, int8_t* q8,
                          int8_t* k8, uint8_t* v8, cudaStream_t st);
// K3: pooled block means (written to qbar/kbar, [BH][nb][128], required),
// then block scores and the per-query-block top-k list (ascending).
// With zin != NULL also writes the selection bitmask (2*ceil(nb/64) words
// per query block) and Z_i = sum of z_j over the unselected key blocks.
cudaError_t launch_pool_topk(const float* qsum, const float* ksum, const Geom& g, int32_t* idx, float* qbar,
                             float* kbar, const float* zin, float* ztot, uint32_t* selbits, float* zout,
                             cudaStream_t st);
// K4a: per key block h_j = phi(K_j)^T V_j (bf16 mask-GEMM tiles) and z_j.
cudaError_t launch_linear_kv(const void* k, const void* v, const Geom& g, uint8_t* hs, float* z, int* wd,
                             cudaStream_t st, QKNorm nk = QKNorm());
// K4b: H_i = sum over unselected j of h_j, as bf16 operand images [nb][128*128].
cudaError_t launch_linear_sum(const uint8_t* hs, const uint32_t* selbits, const Geom& g, uint16_t* hout, int* wd,
                              cudaStream_t st);
// K4c: y = (phi(Q_i) H_i / phi(Q_i) Z_i) W^T per row, written (bf16) to out.
cudaError_t launch_linear_apply(const void* q, const uint16_t* himg, const float* zl, const uint16_t* wimg,
                                const Geom& g, void* out, int* wd, cudaStream_t st, QKNorm nq = QKNorm());
// proj_w [d][d] -> the bf16 B-operand image read by the flash epilogue.
cudaError_t launch_w_tile(const void* w, uint16_t* wt, cudaStream_t st);
// K5: block-sparse INT8/FP8 flash attention over the index lists.
struct FlashArgs {
  const uint8_t* q8t;
  const uint8_t* k8t;
  const uint8_t* v8t;
  const float* sq;
  const float* sk;
  const float* sv;
  const int32_t* idx;  // [BH][nb][kc]; NULL = dense (every block, ascending)
  void* out;           // bf16 rows of 128 in the Geom's layout
  int add_out;          // 1: out already holds the linear branch y (bf16); add O_s to it
  int q_tok;            // 1: sq holds one Q scale per token ([BH][nq*64]) instead of per 64-token tile
  // Watchdog test of the block-64 kernel (all 0 in a normal call): a grid of
  // dbg_grid CTAs instead of the persistent grid, dbg_spin probes per
  // bounded wait instead of the default, and, for dbg_stall > 0, slot 0's K
  // producer of CTA 0 omits the copies of its step dbg_stall - 1.
  int dbg_grid;
  int dbg_stall;
  long dbg_spin;
};
cudaError_t launch_flash(const FlashArgs& a, const Geom& g, cudaStream_t st, int* wd);
// W8A8 linear layer (k_w8a8.cu).
size_t w8a8_codes_bytes(int rows, int cols);
size_t w8a8_scales_count(int rows, int cols);
cudaError_t launch_w8a8_quant(const void* a, int rows, int cols, uint8_t* codes, float* scales, cudaStream_t st);
cudaError_t launch_w8a8_gemm(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, void* y, int M,
                             int N, int K, int* wd, cudaStream_t st);
// QK norm and rotation (k_qk_norm_rope.cu): one tensor of the pair.  Strides
// in elements: batch, token, head.
struct RopeTensor {
  const void* x = nullptr;
  const void* dy = nullptr;  // backward: the gradient of the output
  void* y = nullptr;         // the output, or dx
  const void* gamma = nullptr;
  long xs[3] = {}, dys[3] = {}, ys[3] = {};
  int H = 0;
};
struct RopeArgs {
  RopeTensor t[2];  // q, k (H = 0: none)
  const float *cos = nullptr, *sin = nullptr;  // [T][rot/2]
  const int32_t* pos = nullptr;                // [B][N], or nullptr: the token index
  float* part = nullptr;                       // backward: a row of q and of k per CTA, [ctas][2][d]
  float *dgq = nullptr, *dgk = nullptr;
  long tokens = 0, N = 0, T = 0, stride = 0;
  int d = 0, rot = 0, L = 0, Gq = 0, G = 0, pass[2] = {};
  float eps = 0.f, inv_d = 0.f;
};
long rope_bwd_ctas(long tokens, int G, int sms);
size_t rope_bwd_workspace(int B, int N, int Hq, int Hk, int d, int sms);
cudaError_t launch_qk_norm_rope(const RopeArgs& a, int dtype, bool interleaved, bool back, int sms,
                                cudaStream_t st);
// W8A8 linear layer with a scale per token and per output channel (k_w8a8_token.cu).
cudaError_t launch_w8a8_token_quant(const void* a, int dtype, int rows, int cols, long lda, int8_t* codes,
                                    float* scales, cudaStream_t st);
cudaError_t launch_w8a8_token_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                   const void* bias, void* y, int dtype, int M, int N, int K, int sms, int* wd,
                                   cudaStream_t st, bool chained);  // chained: xq, sx are the previous launch's
// Causal linear attention with a decay for each head (k_linear_decay.cu).
struct DecayArgs {
  const uint16_t *q = nullptr, *k = nullptr, *v = nullptr;  // bf16 rows of d
  uint16_t* o = nullptr;
  const float* log_decay = nullptr;  // [H]
  const float* state_in = nullptr;   // [B][H][d][d], or nullptr: zeros
  float* state_out = nullptr;        // may be state_in; nullptr: not kept
  const int32_t* lens = nullptr;     // [B], or nullptr: N
  long qs[3] = {}, ks[3] = {}, vs[3] = {}, os[3] = {};  // strides in elements: batch, token, head
  float* ws = nullptr;               // [B][H][slots][d][d]: the segments' states
  float scale = 1.f;
  int B = 0, N = 0, H = 0, Hk = 0, d = 0;
  int nseg = 1, seg_tokens = 0, slots = 0;  // segments of a sequence, tokens of each, states in ws
  int step[3][2] = {};               // q, k, v: whether the maps' head and batch coordinates move
};
int linear_decay_segments(int B, int N, int H, int sms);
int linear_decay_slots(int nseg);  // states of the workspace a (sequence, head)
cudaError_t launch_linear_decay(const DecayArgs& a, int* wd, cudaStream_t st);
cudaError_t launch_linear_decay_step(const DecayArgs& a, int sms, cudaStream_t st);
// Waits `probes` times on an mbarrier that never completes, then sets *wd.
cudaError_t launch_watchdog_selftest(int probes, int* wd, cudaStream_t st);

}  // namespace sagesla
