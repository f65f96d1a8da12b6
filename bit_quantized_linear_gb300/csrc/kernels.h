// Internal launcher declarations shared by the C-ABI shim and the kernel files.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "qlin.h"

namespace qlin {

struct DeviceInfo {
  int device = -1;
  int sms = 0;
  int cc_major = 0, cc_minor = 0;
  unsigned *status = nullptr;  // device status word (QLIN_ERR_TIMEOUT on a run-out wait)
};

// Host-side count of kernels enqueued by the library (qlin_launch_count).
void note_launches(int n);

// Argument checks of the W8A8 static linear apart from its workspace, and the
// current-device check (qlin_api.cu); QLIN_OK or the status to return.
qlin_status w8a8_check_args(int qtype, int64_t M, int64_t K, int64_t N, const void *x, const float *input_scale,
                            const void *qw, const float *w_scale, const void *bias, const void *y);
qlin_status device_ready();

// The current device's cached facts; QLIN_OK or the status to return.
qlin_status current_device(DeviceInfo **out);
// Its SM count for choices made before or without a launch (152, a GB300's, without a device).
int sm_count();

// Small checks shared by the entry points.
inline bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool valid_qtype(int t) { return t == QLIN_INT8 || t == QLIN_E4M3; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline qlin_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QLIN_OK : QLIN_ERR_CUDA; }
qlin_status check_linear_shape(int64_t M, int64_t K, int64_t N);
qlin_status check_kv(int64_t T, int64_t H, int64_t D, const int64_t *slots, int64_t num_slots, const void *k_cache,
                     const void *k_scale, const void *v_cache, const void *v_scale);

// Launches `kernel` on `st` with programmatic stream serialization (the kernel
// calls pdl_wait() before reading global inputs) and an optional cluster
// shape along z.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          unsigned cluster_z, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  int na = 0;
  attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  if (cluster_z > 1) {
    attrs[na].id = cudaLaunchAttributeClusterDimension;
    attrs[na].val.clusterDim.x = 1;
    attrs[na].val.clusterDim.y = 1;
    attrs[na].val.clusterDim.z = cluster_z;
    ++na;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = na;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// A cooperative launch (every CTA resident at once, which the fused-quantization
// GEMM's cross-CTA flags rely on), with an optional cluster shape along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_coop(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                               unsigned cluster_x, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  int na = 0;
  attrs[na].id = cudaLaunchAttributeCooperative;
  attrs[na].val.cooperative = 1;
  ++na;
  if (cluster_x > 1) {
    attrs[na].id = cudaLaunchAttributeClusterDimension;
    attrs[na].val.clusterDim.x = cluster_x;
    attrs[na].val.clusterDim.y = 1;
    attrs[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = na;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (e == cudaSuccess) note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// As launch_kernel, with a cluster shape along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_x(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            unsigned cluster_x, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster_x;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// How many clusters of `cz` CTAs along z (block, dynamic shared memory as
// given) can be resident on the current device at once; 0 if the query fails.
// Remembered per device and cluster size in `cache` (kMaxDevices x 9 entries,
// one table per kernel), since the answer depends only on the kernel's
// resources and the device.
constexpr int kMaxDevices = 64;  // devices a process may use (per-device tables)
template <typename... KArgs>
int max_active_clusters_z(void (*kernel)(KArgs...), dim3 block, size_t smem, unsigned cz, int device,
                          std::atomic<int> *cache) {
  if (cz < 2 || cz > 8 || device < 0 || device >= kMaxDevices) return 0;
  std::atomic<int> &slot = cache[device * 9 + cz];
  int n = slot.load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, cz);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 1;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = cz;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, (const void *)kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  slot.store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_quantize_weight(int qtype, int64_t N, int64_t K, const float *w, void *qw,
                                   float *s, cudaStream_t st);
cudaError_t launch_act_scale(int qtype, int64_t rows, int64_t K, const void *x, float *scale,
                             void *ws, int sms, cudaStream_t st);
cudaError_t launch_quantize_act(int qtype, int64_t M, int64_t K, const void *x, const float *s,
                                void *qx, int sms, cudaStream_t st);

// GEMM epilogue / operand modes.
enum GemmMode {
  kW8A16 = 0,   // A = BF16 x, B = 8-bit weight codes, acc fp32, y = acc*s_w[n] + b
  kW8A8 = 1,    // A = 8-bit activation codes, B = 8-bit weight codes, y = acc*(s_x*s_w[n]) + b
  kI8Raw = 2    // INT8 codes, raw int32 accumulator out
};

struct GemmArgs {
  int mode;
  int qtype;
  int64_t M, K, N;
  const void *a;          // x (BF16) or qx (codes)
  const void *qw;         // [N,K] codes
  const float *w_scale;   // [N]
  const float *x_scale;   // device scalar (kW8A8), per-token [M] (x_scale_per_token), or null
  const uint16_t *bias;   // [N] or null
  void *y;                // [M,N] BF16, or int32 for kI8Raw
  int x_scale_per_token = 0;  // x_scale holds one scale per token row (dynamic W8A8)
  int glu = 0;  // merged gate_up: qw/w_scale/bias have 2N rows (gate rows first), y = silu(gate) * up [M, N]
  // FP8 W8A8 with the static quantization inside the GEMM: `a` is the codes
  // workspace, xq the BF16 activations, xq_flags the zeroed task flags
  const void *xq = nullptr;
  unsigned *xq_flags = nullptr;
};

// E4M3 W8A16 on the FP8 tensor cores (w8a16_f8.cu): up to kW8A16F8MaxM tokens,
// plain or merged gate_up; the activations are split into four E4M3 terms in
// the workspace (w8a16_f8_workspace bytes).
constexpr int kW8A16F8MaxM = 32;
int w8a16_f8_tt(int64_t M);
int w8a16_f8_splits(int units, int kblocks, int sms);
size_t w8a16_f8_workspace(int64_t M, int64_t K);
cudaError_t launch_w8a16_f8(const GemmArgs &g, void *ws, const DeviceInfo &dev, cudaStream_t st);

// Fused-quantization FP8 GEMM: task-flag area (u32) for these sizes, and
// whether the fused kernel is used.
size_t fp8_xq_flag_bytes(int64_t M, int64_t K);
bool fp8_xq_used(int64_t M, int64_t K, int64_t N, int sms);

// Mixed KV cache (kv_kernels.cu): INT8 keys with float16 group-32 scales,
// E4M3 values with float16 per-(token, head) scales.
struct KvArgs {
  int64_t T, H, D;        // tokens, kv heads, head_dim (32, 64, 128 or 256)
  const void *k, *v;      // BF16 rows of the new tokens (store), row strides ldk / ldv elements
  int64_t ldk, ldv;
  const int64_t *slots;   // [T] cache slot of each token; negative = padding
  int64_t num_slots;
  void *k_cache, *k_scale, *v_cache, *v_scale;  // [S,H,D] int8, [S,H,D/32] f16, [S,H,D] e4m3, [S,H] f16
  void *k_out, *v_out;    // BF16 [T,H,D] (load)
};
cudaError_t launch_kv_store(const KvArgs &a, unsigned *status, int sms, cudaStream_t st);
cudaError_t launch_kv_load(const KvArgs &a, unsigned *status, cudaStream_t st);

// RMSNorm with the residual's addition (norm_kernels.cu).  Strides in elements;
// residual and h_out may be null, x_scale is null for a static scale.
constexpr int64_t kNormMaxK = 32768;  // a row stays in the registers of at most 16 warps
enum NormOut { kNormBf16 = 0, kNormInt8 = 1, kNormE4m3 = 2 };
struct NormArgs {
  int64_t M, K;
  int out;                   // NormOut
  const void *x, *residual;  // BF16 [M, K]
  int64_t ldx, ldr;
  const void *weight;        // BF16 [K]
  float eps;
  const float *input_scale;  // static scale (device scalar) or null: per-token scales
  void *h_out;               // BF16 [M, K], the sum
  void *y;                   // BF16 [M, K] or codes
  float *x_scale;            // [M]
};
cudaError_t launch_rmsnorm(const NormArgs &a, int sms, cudaStream_t st);

// Rotary positions (rope_kernels.cu), alone or with the store into the mixed
// KV cache (kv.k, kv.v, kv.slots and the caches; kv.T and kv.D as here).
struct RopeArgs {
  int layout;  // qlin_rope_layout
  int64_t T, Hq, Hk, D, rot;
  const float *table;  // [max_pos, rot]: rot/2 cosines, then rot/2 sines
  int64_t max_pos;
  const int64_t *positions;  // [T]; negative = padding
  const void *q, *k;         // BF16 rows of Hq*D / Hk*D elements
  int64_t ldq, ldk;
  void *q_out, *k_out;
  int64_t ldqo, ldko;
};
cudaError_t launch_rope_table(int64_t max_pos, int64_t rot, double theta, int scaling, double factor,
                              double original_context, double beta_fast, double beta_slow, double amplitude,
                              float *table, cudaStream_t st);
cudaError_t launch_rope(const RopeArgs &r, unsigned *status, int sms, cudaStream_t st);
cudaError_t launch_rope_kv_store(const RopeArgs &r, const KvArgs &kv, unsigned *status, int sms, cudaStream_t st);

// Attention over the mixed KV cache.  attn_split.cu: sequences of few rows, the
// positions split over CTAs.  attn_prefill.cu: sequences of many rows, on tcgen05.
struct AttnArgs {
  int64_t B, T, Hq, H, D;
  const void *q;
  int64_t ldq;
  const int32_t *q_start;
  int64_t max_q;
  const int32_t *kv_len;
  int64_t max_kv;
  const int32_t *block_table;
  int64_t max_blocks, block_size, num_slots;
  const void *k_cache, *k_scale, *v_cache, *v_scale;
  float scale;
  int causal;
  int64_t window;
  void *out;
  int64_t ldo;
};
struct AttnSplitPlan {
  int row_tiles;   // row tiles of a (sequence, kv head)
  int rows;        // rows of a tile: 8 or 16
  int splits;      // parts of the positions, each a CTA
  int64_t chunk;   // positions of a part (a multiple of 16)
  size_t ws_bytes;
};
// `rows`: the most rows (new tokens times heads of a group) a sequence has for this kernel; sequences of more
// than few_rows are left to the other one.
AttnSplitPlan attn_split_plan(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t rows, int64_t max_kv,
                              int64_t window, int sms);
cudaError_t launch_attn_split(const AttnArgs &a, const AttnSplitPlan &plan, int few_rows, void *ws, unsigned *status,
                              cudaStream_t st);
bool attn_prefill_has(int64_t D);
struct AttnPrefillPlan {
  int64_t heads;      // kv heads whose keys and values are in the workspace at once
  int64_t row_tiles;  // of 256 rows, for a sequence
  int64_t splits;     // parts of the positions, each a CTA
  int64_t chunk;      // position tiles of a part
  size_t image_bytes, ws_bytes;
};
AttnPrefillPlan attn_prefill_plan(int64_t B, int64_t H, int64_t G, int64_t D, int64_t max_q, int64_t max_kv,
                                  int64_t window, int sms);
cudaError_t launch_attn_prefill(const AttnArgs &a, const AttnPrefillPlan &plan, int few_rows, void *ws,
                                unsigned *status, cudaStream_t st);

// tcgen05 kernels (gemm_tc.cu)
cudaError_t launch_fp8_gemm(const GemmArgs &g, const DeviceInfo &dev, cudaStream_t st);
cudaError_t launch_w8a16_swap(const GemmArgs &g, const DeviceInfo &dev, cudaStream_t st);
cudaError_t launch_i8_swap(const GemmArgs &g, const void *xb, bool raw, const DeviceInfo &dev, cudaStream_t st,
                           bool fused = false);
int w8_swap_bnt(int64_t M, int64_t N, int64_t K, int sms);
int i8_swap_bnt(int64_t M);
int w8_swap_splits(int64_t tiles, int64_t K, int sms, int bnt);

// INT8 operand preparation for the tensor-core INT8 path (quant_kernels.cu)
cudaError_t launch_quantize_act_i8bf16(int64_t M, int64_t K, const void *x, const float *s, void *out, int sms,
                                       cudaStream_t st);
cudaError_t launch_i8_to_bf16(int64_t M, int64_t K, const void *q, void *out, int sms, cudaStream_t st);
// Dynamic per-token quantization: scales s[M]; codes (1 byte) or INT8 codes as BF16.
cudaError_t launch_quantize_act_dyn(int qtype, bool out_bf16, int64_t M, int64_t K, const void *x, float *s, void *q,
                                    cudaStream_t st);

}  // namespace qlin
