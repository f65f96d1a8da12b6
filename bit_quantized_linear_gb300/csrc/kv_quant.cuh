// Device helpers shared by the kernels that write the mixed KV cache: vector
// loads and stores of 32-bit words, the float16 scale of a group, and the INT8
// and E4M3 codes of quotients.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace qlin {

// N 32-bit words at an address aligned to 4*min(N,4) bytes.
template <int N>
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = ld_input(reinterpret_cast<const uint32_t *>(p));
  } else if constexpr (N == 2) {
    const uint2 v = ld_input(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = ld_input(reinterpret_cast<const uint4 *>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

template <int N>
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    *reinterpret_cast<uint32_t *>(p) = w[0];
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// Max over aligned groups of W lanes (W a power of two <= 32).
template <int W>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// float16 scale of a group: RN_fp16(fl32(amax / qmax)), saturating at 65504;
// 1.0 when the cast gives zero.
__device__ __forceinline__ uint16_t scale16(float amax, float qmax) {
  // qmax is 127 or 448: its reciprocal is a compile-time constant and the
  // quotient amax / qmax the correctly rounded one (qlin::quotient)
  const Scale q{qmax, 1.0f / qmax, true};
  const float s32 = fminf(quotient<true>(amax, q), 65504.0f);
  uint16_t h = __half_as_ushort(__float2half_rn(s32));
  return (h & 0x7FFFu) ? h : (uint16_t)0x3C00u;
}

__device__ __forceinline__ float half_bits_to_f32(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// INT8 code of a quotient v: clamp to [-127,127], then add 1.5 * 2^23.  The
// sum lies in [2^23, 2^24), where the float spacing is 1, so the addition
// rounds v half to even and the low byte of the sum's bit pattern is the code
// in two's complement.
__device__ __forceinline__ uint32_t int8_code_word(float v) {
  return __float_as_uint(__fadd_rn(fminf(fmaxf(v, -127.0f), 127.0f), 0x1.8p23f));
}

// Four low bytes -> one word (byte i from the i-th argument).
__device__ __forceinline__ uint32_t pack4_low(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four saturating E4M3 codes, two per conversion instruction (byte i from the
// i-th argument).
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return __byte_perm(lo, hi, 0x5410);
}

}  // namespace qlin
