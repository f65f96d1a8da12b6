// What the attention kernels share: the call as the device sees it, a sequence's
// counts with their checks, the positions a token sees, and code conversions.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace qlin {

constexpr float kLog2e = 1.44269504088896341f;

struct AttnDev {
  const uint16_t *q;
  const int32_t *q_start, *kv_len, *block_table;
  const uint8_t *kc, *vc;
  const uint16_t *ks, *vs;
  uint16_t *out;
  int64_t ldq, ldo, max_blocks;
  int B, T, H, G, max_q, max_kv, block_size, block_shift, num_blocks, causal, window;
  int few_rows;  // sequences of at most this many rows a kv head are the split kernel's
  float scale_log2;
  unsigned *status;
};
AttnDev attn_dev(const AttnArgs &a, int few_rows, unsigned *status);

// What a CTA knows of its sequence.  Counts that break the contract are cut to
// what is in bounds; `broken` says so.
struct Sequence {
  int first, n, kept, kv;  // first row, new tokens, those within max_q, positions
  bool broken;
};
__device__ __forceinline__ Sequence sequence(const AttnDev &p, int b) {
  Sequence s;
  const int end = p.q_start[b + 1];
  s.first = p.q_start[b];
  s.n = end - s.first;
  s.kv = p.kv_len[b];
  const int64_t room = p.max_blocks * p.block_size;
  const bool rows_ok = s.first >= 0 && end >= s.first && end <= p.T;
  s.broken = !rows_ok || s.n > p.max_q || s.kv < 0 || s.kv > p.max_kv || s.kv > room;
  if (!rows_ok) s.n = 0;
  s.kept = min(s.n, p.max_q);
  s.kv = max(0, min(s.kv, p.max_kv));
  if (s.kv > room) s.kv = (int)room;
  return s;
}
// Positions [lo, hi) that the new token `tok` of a sequence sees (both grow with tok).
__device__ __forceinline__ void sees(const AttnDev &p, const Sequence &s, int tok, int &lo, int &hi) {
  const int pos = s.kv - s.n + tok;
  lo = 0;
  hi = s.kv;
  if (p.causal) hi = min(hi, pos + 1);
  if (p.window > 0) {
    lo = max(lo, pos - p.window + 1);
    if (!p.causal) hi = (int)min((int64_t)hi, (int64_t)pos + p.window);
  }
}
__device__ __forceinline__ int block_of(const AttnDev &p, int position) {
  return p.block_shift >= 0 ? position >> p.block_shift : position / p.block_size;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The power of two that brings a q row, whose largest magnitude is `top`, to
// 2^14..2^15: 2^(14 - e); its inverse is 2^(e - 14).
__device__ __forceinline__ int q_exponent(float top) {
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  return top > 0.0f && e < 128 ? max(e, -100) : 14;
}

// Four INT8 codes c -> two words of float16 holding 1152 + c: with the sign bit
// flipped a code is u = c + 128, and the bytes (u, 0x64) are the float16 1024 + u.
__device__ __forceinline__ void int8x4_to_offset_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x4140);
  hi = __byte_perm(u, 0x64646464u, 0x4342);
}
// The codes themselves.
__device__ __forceinline__ void int8x4_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const __half2 offset = __half2half2(__ushort_as_half(0x6480));
  int8x4_to_offset_half(w, lo, hi);
  lo = half2_bits(__hsub2(bits_half2(lo), offset));
  hi = half2_bits(__hsub2(bits_half2(hi), offset));
}
// Two E4M3 codes -> float16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// Partial results of rows whose positions several CTAs share: [unit][part][row of
// the unit's tile] O (D fp32, divided by its sum), and the sum with the base-2
// reference it was taken under ({-inf, 0}: nothing seen; kept apart, as a logarithm
// of the sum would round away beside a large reference),
// unit = (b * H + h) * row_tiles + tile.
struct AttnParts {
  float *o;
  float2 *sum;  // {reference, sum}
  int row_tiles, rows, splits;
};
// Joins them into `out`.  many: of the sequences with more than p.few_rows rows, else of the others.
cudaError_t launch_attn_join(const AttnDev &p, const AttnParts &parts, int64_t D, bool many, cudaStream_t st);

}  // namespace qlin
