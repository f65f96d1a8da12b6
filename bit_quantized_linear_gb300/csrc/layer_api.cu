// C-ABI shims of the decoder-layer operators around the linears: RMSNorm,
// the W8A8 linear on given codes, rotary positions and attention over the mixed
// KV cache.  Argument checks on the host, then launches on the caller's stream.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

using namespace qlin;

namespace {

bool al4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool bad_stride(int64_t ld, int64_t least) { return ld < least || (ld % 8); }

qlin_status check_norm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                       const void *weight, float eps, const void *h_out, const void *y) {
  if (M < 0 || M > ((int64_t)1 << 31) - 1 || K < 16 || (K % 16) || K > kNormMaxK) return QLIN_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return QLIN_ERR_INVALID_ARG;
  if (!weight || !al16(weight)) return QLIN_ERR_INVALID_ARG;
  if ((residual != nullptr) != (h_out != nullptr)) return QLIN_ERR_INVALID_ARG;
  if (bad_stride(ldx, K) || (residual && bad_stride(ldr, K))) return QLIN_ERR_INVALID_ARG;
  if (!al16(residual) || !al16(h_out)) return QLIN_ERR_INVALID_ARG;
  if (M > 0 && (!x || !y || !al16(x) || !al16(y))) return QLIN_ERR_INVALID_ARG;
  return QLIN_OK;
}

bool valid_layout(int l) { return l == QLIN_ROPE_HALF || l == QLIN_ROPE_PAIRS; }
bool valid_kv_dim(int64_t D) { return D == 32 || D == 64 || D == 128 || D == 256; }

qlin_status check_rope(int layout, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rot, const float *table,
                       int64_t max_pos, const int64_t *positions, const void *q, int64_t ldq, const void *q_out,
                       int64_t ldqo) {
  if (!valid_layout(layout)) return QLIN_ERR_INVALID_ARG;
  if (T < 0 || T > (int64_t)1 << 40 || Hq < 1 || Hk < 0 || Hq > 4096 || Hk > 4096) return QLIN_ERR_INVALID_ARG;
  if (D < 16 || D > 512 || (D % 16) || rot < 16 || rot > D || (rot % 16)) return QLIN_ERR_INVALID_ARG;
  if (max_pos < 1 || !table || !al16(table)) return QLIN_ERR_INVALID_ARG;
  if (bad_stride(ldq, Hq * D) || bad_stride(ldqo, Hq * D)) return QLIN_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !q || !q_out || !al16(positions) || !al16(q) || !al16(q_out)))
    return QLIN_ERR_INVALID_ARG;
  if (q == q_out && ldq != ldqo) return QLIN_ERR_INVALID_ARG;
  return QLIN_OK;
}

// Size checks shared by the attention entry points.
qlin_status check_attn_sizes(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t max_q, int64_t max_kv,
                             int64_t window) {
  if (B < 0 || B > 1 << 20 || H < 1 || H > 4096 || Hq < 1 || Hq % H || Hq / H > 128 || !valid_kv_dim(D))
    return QLIN_ERR_INVALID_ARG;
  if (max_q < 0 || max_kv < 0 || max_q > 1 << 30 || max_kv > 1 << 30 || window < 0) return QLIN_ERR_INVALID_ARG;
  // rows of a sequence and grid sizes stay below 2^31
  if (max_q * (Hq / H) > 1 << 30) return QLIN_ERR_INVALID_ARG;
  if (B * H > ((int64_t)1 << 31) / (max_q * (Hq / H) / 8 + 1)) return QLIN_ERR_INVALID_ARG;
  return QLIN_OK;
}

// Which kernel takes which sequences.  With u = sequences x kv heads x positions a row
// sees at most, the split kernel reads all of u once for every 16 rows: 8 us and, of a
// ragged batch, 4.3e-5 us (head size 64: 2.9e-5) for each (16 rows, unit of u).  The tcgen05
// kernels unpack u once: 22 us and 3e-4 us a unit, whatever the rows.  The limit is where
// the two meet; a lone sequence has no second kernel to launch, and no raggedness: its limit
// falls with 1 / u from 512 rows, and at u = 32768 the tcgen05 kernels lead from 84 rows on.
// Beyond it they take those sequences of the batch that have more than kFewRows rows,
// and the split kernel the others; each leaves the other's sequences.  Measured (split and
// tcgen05, us), one sequence of 28 heads over 4 of 128: 84 rows over 8192 positions 28.7
// and 26.3, 168 over 8192 42.5 and 30.6, 420 over 2048 31.8 and 23.6.  Batches: 4 x 84 rows
// over 8192 33.3 and 60.2, 2 x 280 over 4096 45.9 and 33.4, 8 x 196 over 2492 48.6 and 48.6;
// 8 heads of 128, 4 x 200 over 2048 40.4 and 33.9; of 64, 5 x 333 over 1024 33.1 and 38.4.
constexpr int64_t kFewRows = 64;
int64_t attn_most_split_rows(int64_t B, int64_t H, int64_t D, int64_t max_kv, int64_t window) {
  const int64_t range = window > 0 ? std::min(window, max_kv) : max_kv;
  const int64_t u = std::max<int64_t>(1, B * H * range);
  const int64_t rows = B == 1 ? 2000000 / u : D == 64 ? 165 + 7700000 / u : 112 + 5200000 / u;
  return std::min<int64_t>(std::max<int64_t>(rows, kFewRows), 512);
}
struct AttnRoute {
  bool few, many;  // the split kernel, the tcgen05 kernel
  int few_rows;
  AttnSplitPlan split;
  AttnPrefillPlan prefill;
  size_t ws_bytes() const { return split.ws_bytes + prefill.ws_bytes; }
};
AttnRoute attn_route(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t max_q, int64_t max_kv, int64_t window) {
  AttnRoute r{};
  const int64_t rows = max_q * (Hq / H);
  r.many = attn_prefill_has(D) && rows > attn_most_split_rows(B, H, D, max_kv, window);
  r.few = !r.many || B > 1;
  r.few_rows = r.many ? (r.few ? (int)kFewRows : 0) : (int)rows;
  const int sms = sm_count();
  if (r.many) r.prefill = attn_prefill_plan(B, H, Hq / H, D, max_q, max_kv, window, sms);
  if (r.few) r.split = attn_split_plan(B, Hq, H, D, r.few_rows, max_kv, window, sms);
  return r;
}

}  // namespace

extern "C" {

qlin_status qlin_rmsnorm(int64_t M, int64_t K, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                         const void *weight, float eps, void *h_out, void *y_out, qlin_stream_t stream) {
  if (qlin_status s = check_norm(M, K, x, ldx, residual, ldr, weight, eps, h_out, y_out)) return s;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (M == 0) return QLIN_OK;
  NormArgs a{M, K, kNormBf16, x, residual, ldx, ldr, weight, eps, nullptr, h_out, y_out, nullptr};
  return from_cuda(launch_rmsnorm(a, dev->sms, (cudaStream_t)stream));
}

qlin_status qlin_rmsnorm_quant(qlin_qtype qtype, int64_t M, int64_t K, const void *x, int64_t ldx,
                               const void *residual, int64_t ldr, const void *weight, float eps,
                               const float *input_scale, void *h_out, void *qx, float *x_scale,
                               qlin_stream_t stream) {
  if (!valid_qtype(qtype)) return QLIN_ERR_INVALID_ARG;
  if (qlin_status s = check_norm(M, K, x, ldx, residual, ldr, weight, eps, h_out, qx)) return s;
  if (input_scale ? (x_scale != nullptr || !al4(input_scale)) : (M > 0 && (!x_scale || !al16(x_scale))))
    return QLIN_ERR_INVALID_ARG;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (M == 0) return QLIN_OK;
  NormArgs a{M,   K,           qtype == QLIN_INT8 ? kNormInt8 : kNormE4m3, x, residual, ldx, ldr, weight,
             eps, input_scale, h_out,                                      qx, x_scale};
  return from_cuda(launch_rmsnorm(a, dev->sms, (cudaStream_t)stream));
}

qlin_status qlin_w8a8_linear_codes(qlin_qtype qtype, int64_t M, int64_t K, int64_t N, const void *qx,
                                   const float *x_scale, int per_token, const void *qw, const float *w_scale,
                                   const void *bias, void *y, void *ws, size_t ws_bytes, qlin_stream_t stream) {
  if (qlin_status s = w8a8_check_args(qtype, M, K, N, qx, x_scale, qw, w_scale, bias, y)) return s;
  const size_t need = qlin_workspace_bytes(QLIN_OP_W8A8_LINEAR_CODES, qtype, M, K, N);
  if (need && (!ws || !al16(ws) || ws_bytes < need)) return QLIN_ERR_WORKSPACE;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (M == 0) return QLIN_OK;
  cudaStream_t st = (cudaStream_t)stream;
  GemmArgs g{kW8A8, qtype, M, K, N, qtype == QLIN_E4M3 ? qx : ws, qw, w_scale, x_scale, (const uint16_t *)bias, y};
  g.x_scale_per_token = per_token != 0;
  if (qtype == QLIN_E4M3) return from_cuda(launch_fp8_gemm(g, *dev, st));
  if (launch_i8_to_bf16(M, K, qx, ws, dev->sms, st) != cudaSuccess) return QLIN_ERR_CUDA;
  return from_cuda(launch_i8_swap(g, ws, false, *dev, st));
}

qlin_status qlin_rope_table(int64_t max_pos, int64_t rot, double theta, qlin_rope_scaling scaling, double factor,
                            double original_context, double beta_fast, double beta_slow, double amplitude,
                            float *table, qlin_stream_t stream) {
  if (max_pos < 1 || max_pos > (int64_t)1 << 31 || rot < 16 || rot > 512 || (rot % 16)) return QLIN_ERR_INVALID_ARG;
  if (!(theta > 0.0) || !std::isfinite(theta) || !std::isfinite(amplitude)) return QLIN_ERR_INVALID_ARG;
  if (scaling < QLIN_ROPE_PLAIN || scaling > QLIN_ROPE_BY_PARTS) return QLIN_ERR_INVALID_ARG;
  if (scaling != QLIN_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor))) return QLIN_ERR_INVALID_ARG;
  if (scaling == QLIN_ROPE_BY_PARTS && !(original_context > 0.0 && std::isfinite(original_context) &&
                                         beta_fast > beta_slow && std::isfinite(beta_fast) && beta_slow >= 0.0))
    return QLIN_ERR_INVALID_ARG;
  if (!table || !al16(table)) return QLIN_ERR_INVALID_ARG;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  return from_cuda(launch_rope_table(max_pos, rot, theta, scaling, factor, original_context, beta_fast, beta_slow,
                                     amplitude, table, (cudaStream_t)stream));
}

qlin_status qlin_rope(qlin_rope_layout layout, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rot,
                      const float *table, int64_t max_pos, const int64_t *positions, const void *q, int64_t ldq,
                      const void *k, int64_t ldk, void *q_out, int64_t ldqo, void *k_out, int64_t ldko,
                      qlin_stream_t stream) {
  if (qlin_status s = check_rope(layout, T, Hq, Hk, D, rot, table, max_pos, positions, q, ldq, q_out, ldqo)) return s;
  if (Hk > 0) {
    if (bad_stride(ldk, Hk * D) || bad_stride(ldko, Hk * D)) return QLIN_ERR_INVALID_ARG;
    if (T > 0 && (!k || !k_out || !al16(k) || !al16(k_out))) return QLIN_ERR_INVALID_ARG;
    if (k == k_out && ldk != ldko) return QLIN_ERR_INVALID_ARG;
  }
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (T == 0) return QLIN_OK;
  RopeArgs r{layout, T, Hq, Hk, D, rot, table, max_pos, positions, q, k, ldq, ldk, q_out, k_out, ldqo, ldko};
  return from_cuda(launch_rope(r, dev->status, dev->sms, (cudaStream_t)stream));
}

qlin_status qlin_rope_kv_store_mixed(qlin_rope_layout layout, int64_t T, int64_t Hq, int64_t H, int64_t D,
                                     int64_t rot, const float *table, int64_t max_pos, const int64_t *positions,
                                     const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                     int64_t ldv, void *q_out, int64_t ldqo, const int64_t *slots,
                                     int64_t num_slots, void *k_cache, void *k_scale, void *v_cache, void *v_scale,
                                     qlin_stream_t stream) {
  if (qlin_status s = check_kv(T, H, D, slots, num_slots, k_cache, k_scale, v_cache, v_scale)) return s;
  if (qlin_status s = check_rope(layout, T, Hq, H, D, rot, table, max_pos, positions, q, ldq, q_out, ldqo)) return s;
  if (bad_stride(ldk, H * D) || bad_stride(ldv, H * D)) return QLIN_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || !al16(k) || !al16(v))) return QLIN_ERR_INVALID_ARG;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (T == 0) return QLIN_OK;
  RopeArgs r{layout, T, Hq, H, D, rot, table, max_pos, positions, q, k, ldq, ldk, q_out, nullptr, ldqo, 0};
  KvArgs kv{T, H, D, k, v, ldk, ldv, slots, num_slots, k_cache, k_scale, v_cache, v_scale, nullptr, nullptr};
  return from_cuda(launch_rope_kv_store(r, kv, dev->status, dev->sms, (cudaStream_t)stream));
}

size_t qlin_attn_mixed_workspace_bytes(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t max_q, int64_t max_kv,
                                       int64_t window) {
  if (check_attn_sizes(B, Hq, H, D, max_q, max_kv, window)) return (size_t)-1;
  if (B == 0 || max_q == 0) return 0;
  return attn_route(B, Hq, H, D, max_q, max_kv, window).ws_bytes();
}

const char *qlin_attn_mixed_kernel_name(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t max_q, int64_t max_kv,
                                        int64_t window) {
  if (check_attn_sizes(B, Hq, H, D, max_q, max_kv, window)) return "invalid";
  if (B == 0 || max_q == 0) return "none";
  const AttnRoute r = attn_route(B, Hq, H, D, max_q, max_kv, window);
  static const char *many[2][3] = {
      {"k_attn_unpack+k_attn_prefill", "k_attn_unpack+k_attn_prefill+k_attn_split",
       "k_attn_unpack+k_attn_prefill+k_attn_split+k_attn_join"},
      {"k_attn_unpack+k_attn_prefill+k_attn_join", "k_attn_unpack+k_attn_prefill+k_attn_join+k_attn_split",
       "k_attn_unpack+k_attn_prefill+k_attn_join+k_attn_split+k_attn_join"}};
  if (r.many) return many[r.prefill.splits > 1][!r.few ? 0 : r.split.splits > 1 ? 2 : 1];
  return r.split.splits > 1 ? "k_attn_split+k_attn_join" : "k_attn_split";
}

qlin_status qlin_attn_mixed(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D, const void *q, int64_t ldq,
                            const int32_t *q_start, int64_t max_q, const int32_t *kv_len, int64_t max_kv,
                            const int32_t *block_table, int64_t max_blocks, int64_t block_size, int64_t num_slots,
                            const void *k_cache, const void *k_scale, const void *v_cache, const void *v_scale,
                            float scale, int causal, int64_t window, void *out, int64_t ldo, void *ws,
                            size_t ws_bytes, qlin_stream_t stream) {
  if (qlin_status s = check_attn_sizes(B, Hq, H, D, max_q, max_kv, window)) return s;
  if (T < 0 || T > ((int64_t)1 << 31) - 1 || max_blocks < 0 || block_size < 1 || block_size > 1 << 30 ||
      num_slots < 0 || num_slots > ((int64_t)1 << 40) / H || num_slots % block_size ||
      num_slots / block_size > ((int64_t)1 << 31) - 1 || max_blocks > ((int64_t)1 << 40) / (B + 1))
    return QLIN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || bad_stride(ldq, Hq * D) || bad_stride(ldo, Hq * D)) return QLIN_ERR_INVALID_ARG;
  const bool work = B > 0 && T > 0 && max_q > 0;
  if (work) {
    if (!q || !out || !q_start || !kv_len || !al16(q) || !al16(out) || !al4(q_start) || !al4(kv_len))
      return QLIN_ERR_INVALID_ARG;
    if (max_kv > 0 && (!block_table || !al4(block_table) || !k_cache || !k_scale || !v_cache || !v_scale ||
                       !al16(k_cache) || !al16(k_scale) || !al16(v_cache) || !al16(v_scale)))
      return QLIN_ERR_INVALID_ARG;
  }
  // one plan, for the check of the workspace and for the launches
  const AttnRoute r = work ? attn_route(B, Hq, H, D, max_q, max_kv, window) : AttnRoute{};
  const size_t need = r.ws_bytes();
  if (need && (!ws || !al16(ws) || ws_bytes < need)) return QLIN_ERR_WORKSPACE;
  DeviceInfo *dev;
  if (qlin_status s = current_device(&dev)) return s;
  if (!work) return QLIN_OK;
  AttnArgs a{B,         T,          Hq,        H,       D,       q,       ldq,     q_start, max_q, kv_len, max_kv, block_table,
             max_blocks, block_size, num_slots, k_cache, k_scale, v_cache, v_scale, scale,   causal, window, out,   ldo};
  if (r.many && launch_attn_prefill(a, r.prefill, r.few_rows, ws, dev->status, (cudaStream_t)stream) != cudaSuccess)
    return QLIN_ERR_CUDA;
  if (!r.few) return QLIN_OK;
  void *parts = r.split.ws_bytes ? (char *)ws + r.prefill.ws_bytes : nullptr;
  return from_cuda(launch_attn_split(a, r.split, r.few_rows, parts, dev->status, (cudaStream_t)stream));
}

}  // extern "C"
