// RMSNorm with the residual's addition and an output in BF16 or 8-bit codes.
//
//   h = bf16(x + residual)                                  (h = x without one)
//   r = fl32(1 / sqrt(sum_k h^2 / K + eps))
//   y = fl32(fl32(h * r) * w)
//   BF16: bf16(y);  codes: Q(fl32(y / s)), s static or max_k |y| / QMAX per row.
//
// The codes are defined by single binary32 operations on h, r, w and s, so they
// are reproducible bit for bit once r is.  r is therefore made independent of
// the order of the sum: squares of BF16 values are exact in binary32, and they
// are summed with their rounding errors kept (two-sum: D. E. Knuth, The Art of
// Computer Programming 2, 4.2.2, theorem B), which leaves about 2^-46 relative
// error before the one rounding to binary32.  FP64, at 1/64 of the FP32 rate
// here, is kept for rows whose sum leaves the range in which the squares are
// exact.
//
// One pass: a row's vectors stay in registers between the sum and the output
// (and, for per-token scales, between the output's maximum and its codes).  A
// row is shared by `wpr` warps.  Bound by HBM: x, residual and h_out are 2
// bytes an element, the output 1 or 2.
#include "common.cuh"
#include "kernels.h"
#include "kv_quant.cuh"

#include <algorithm>

namespace qlin {

namespace {

constexpr int kMaxWarpsPerRow = 16;
constexpr int kMaxVecs = 8;       // 16-byte vectors of a row a thread holds
constexpr int kWarpsPerCta = 8;

// hi + lo, an unevaluated sum.
struct TwoFloat {
  float hi, lo;
};
__device__ __forceinline__ void add_value(TwoFloat &a, float b) {
  const float s = __fadd_rn(a.hi, b);
  const float bb = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  a.hi = s;
  a.lo = __fadd_rn(a.lo, e);
}
__device__ __forceinline__ void add_pair(TwoFloat &a, TwoFloat b) {
  const float lo = __fadd_rn(a.lo, b.lo);
  a.lo = 0.0f;
  add_value(a, b.hi);
  a.lo = __fadd_rn(a.lo, lo);
}

// fl32(1 / sqrt(S * invK + eps)) from two-float operands: one Newton step from
// the approximation r0, its residual 1 - v r0^2 formed from exact products.
__device__ __forceinline__ float rms_reciprocal(TwoFloat S, TwoFloat inv_k, float eps) {
  TwoFloat v;
  v.hi = __fmul_rn(S.hi, inv_k.hi);
  v.lo = __fmaf_rn(S.hi, inv_k.hi, -v.hi);
  v.lo = __fmaf_rn(S.hi, inv_k.lo, __fmaf_rn(S.lo, inv_k.hi, v.lo));
  add_value(v, eps);
  const float r0 = rsqrtf(v.hi);
  const float p = __fmul_rn(r0, r0), pl = __fmaf_rn(r0, r0, -p);
  float e = __fmaf_rn(-v.hi, p, 1.0f);
  e = __fmaf_rn(-v.hi, pl, e);
  e = __fmaf_rn(-v.lo, p, e);
  return __fmaf_rn(0.5f * r0, e, r0);
}

struct RmsParams {
  const uint16_t *x, *res, *w;
  int64_t ldx, ldr, M;
  int K8, wpr;  // vectors of a row, warps per row
  double eps64, inv_k64;
  float eps;
  TwoFloat inv_k;
  const float *in_scale;
  uint16_t *h_out;
  void *y;
  float *x_scale;
};

template <int OUT, bool BOUNDED>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], const Scale &c) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = quotient<BOUNDED>(y[j], c);
  if constexpr (OUT == kNormInt8) {
    return make_uint2(
        pack4_low(int8_code_word(q[0]), int8_code_word(q[1]), int8_code_word(q[2]), int8_code_word(q[3])),
        pack4_low(int8_code_word(q[4]), int8_code_word(q[5]), int8_code_word(q[6]), int8_code_word(q[7])));
  } else {
    return make_uint2(e4m3_pack4(q[0], q[1], q[2], q[3]), e4m3_pack4(q[4], q[5], q[6], q[7]));
  }
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const float lo = __fadd_rn(__uint_as_float(a << 16), __uint_as_float(b << 16));
  const float hi = __fadd_rn(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u));
  return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

// y of one vector: fl32(fl32(h * r) * w).
__device__ __forceinline__ void normed8(const uint4 &h, const uint4 &w, float r, float (&y)[8]) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[2 * j] = __fmul_rn(__fmul_rn(__uint_as_float(hw[j] << 16), r), __uint_as_float(ww[j] << 16));
    y[2 * j + 1] =
        __fmul_rn(__fmul_rn(__uint_as_float(hw[j] & 0xFFFF0000u), r), __uint_as_float(ww[j] & 0xFFFF0000u));
  }
}

template <int NV, int OUT, bool DYN>
__global__ void __launch_bounds__(32 * kMaxWarpsPerRow) k_rmsnorm(const RmsParams p) {
  __shared__ TwoFloat s_sum[kMaxWarpsPerRow];
  __shared__ double s_sum64[kMaxWarpsPerRow];
  __shared__ float s_max[kMaxWarpsPerRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / p.wpr, sub = warp % p.wpr, first = group * p.wpr;
  const int64_t m = (int64_t)blockIdx.x * ((blockDim.x >> 5) / p.wpr) + group;
  // the warps of one row meet at a barrier of their own
  const auto row_barrier = [&] {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(p.wpr * 32) : "memory");
  };
  if (m >= p.M) return;

  uint4 w[NV], h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = (i * p.wpr + sub) * 32 + lane;
    w[i] = v < p.K8 ? __ldg(reinterpret_cast<const uint4 *>(p.w) + v) : make_uint4(0, 0, 0, 0);
  }
  pdl_wait();
  pdl_trigger();
  const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + m * p.ldx);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = (i * p.wpr + sub) * 32 + lane;
    h[i] = v < p.K8 ? xr[v] : make_uint4(0, 0, 0, 0);
  }
  if (p.res) {
    const uint4 *rr = reinterpret_cast<const uint4 *>(p.res + m * p.ldr);
    uint4 *ho = reinterpret_cast<uint4 *>(p.h_out) + m * p.K8;
    uint4 r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = (i * p.wpr + sub) * 32 + lane;
      r[i] = v < p.K8 ? rr[v] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = (i * p.wpr + sub) * 32 + lane;
      h[i] = make_uint4(add_bf16x2(h[i].x, r[i].x), add_bf16x2(h[i].y, r[i].y), add_bf16x2(h[i].z, r[i].z),
                        add_bf16x2(h[i].w, r[i].w));
      if (v < p.K8) ho[v] = h[i];
    }
  }

  // sum of squares
  TwoFloat S{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t hw[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = __uint_as_float(hw[j] << 16), b = __uint_as_float(hw[j] & 0xFFFF0000u);
      add_value(S, __fmul_rn(a, a));
      add_value(S, __fmul_rn(b, b));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add_pair(S, TwoFloat{__shfl_xor_sync(~0u, S.hi, o), __shfl_xor_sync(~0u, S.lo, o)});
  if (p.wpr > 1) {
    if (lane == 0) s_sum[warp] = S;
    row_barrier();
    S = lane < p.wpr ? s_sum[first + lane] : TwoFloat{0.0f, 0.0f};
#pragma unroll
    for (int o = kMaxWarpsPerRow / 2; o > 0; o >>= 1)
      add_pair(S, TwoFloat{__shfl_xor_sync(~0u, S.hi, o), __shfl_xor_sync(~0u, S.lo, o)});
    S.hi = __shfl_sync(~0u, S.hi, 0);  // lanes 16..31 hold no partial sums
    S.lo = __shfl_sync(~0u, S.lo, 0);
  }
  float r;
  if (S.hi >= 0x1p-80f && S.hi < 0x1p126f) {
    r = rms_reciprocal(S, p.inv_k, p.eps);
  } else {
    // squares beyond binary32 (or an all-zero row): the same sum in FP64
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t hw[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const uint32_t u = hw[j >> 1];
        const double a = (double)__uint_as_float(j & 1 ? u & 0xFFFF0000u : u << 16);
        d += a * a;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
    if (p.wpr > 1) {
      if (lane == 0) s_sum64[warp] = d;
      row_barrier();
      d = 0.0;
      for (int i = 0; i < p.wpr; ++i) d += s_sum64[first + i];
    }
    r = (float)(1.0 / sqrt(d * p.inv_k64 + p.eps64));
  }

  if constexpr (OUT == kNormBf16) {
    uint4 *yo = reinterpret_cast<uint4 *>(p.y) + m * p.K8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = (i * p.wpr + sub) * 32 + lane;
      float y[8];
      normed8(h[i], w[i], r, y);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = (uint32_t)f32_to_bf16_bits(y[2 * j]) | ((uint32_t)f32_to_bf16_bits(y[2 * j + 1]) << 16);
      if (v < p.K8) yo[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    float s;
    if constexpr (DYN) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8];
        normed8(h[i], w[i], r, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
      }
      amax = warp_max(amax);
      if (p.wpr > 1) {
        if (lane == 0) s_max[warp] = amax;
        row_barrier();
        amax = warp_max(lane < p.wpr ? s_max[first + lane] : 0.0f);
      }
      s = __fdiv_rn(amax, OUT == kNormInt8 ? kQmaxInt8 : kQmaxE4m3);
      s = s > 0.0f ? s : 1.0f;
      if (sub == 0 && lane == 0) p.x_scale[m] = s;
    } else {
      s = *p.in_scale;
    }
    const Scale c = make_scale(s);
    uint2 *yo = reinterpret_cast<uint2 *>(p.y) + m * p.K8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = (i * p.wpr + sub) * 32 + lane;
      float y[8];
      normed8(h[i], w[i], r, y);
      const uint2 o = codes8<OUT, DYN>(y, c);
      if (v < p.K8) yo[v] = o;
    }
  }
}

template <int OUT, bool DYN>
cudaError_t launch_nv(int nv, const RmsParams &p, dim3 grid, dim3 block, cudaStream_t st) {
  switch (nv) {
    case 1: return launch_kernel(k_rmsnorm<1, OUT, DYN>, grid, block, 0, st, 1, p);
    case 2: return launch_kernel(k_rmsnorm<2, OUT, DYN>, grid, block, 0, st, 1, p);
    case 4: return launch_kernel(k_rmsnorm<4, OUT, DYN>, grid, block, 0, st, 1, p);
    case 8: return launch_kernel(k_rmsnorm<8, OUT, DYN>, grid, block, 0, st, 1, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, int sms, cudaStream_t st) {
  const int K8 = (int)(a.K / 8);
  int wpr = 1;
  while (wpr < kMaxWarpsPerRow && wpr * 32 * kMaxVecs < K8) wpr *= 2;
  if (wpr * 32 * kMaxVecs < K8) return cudaErrorInvalidValue;
  const auto vecs = [&] {
    int nv = 1;
    while (nv * wpr * 32 < K8) nv *= 2;
    return nv;
  };
  // few rows: more warps on each
  while (wpr < kMaxWarpsPerRow && vecs() > 1 && a.M * wpr < (int64_t)sms * 16) wpr *= 2;
  RmsParams p{};
  p.x = (const uint16_t *)a.x, p.res = (const uint16_t *)a.residual, p.w = (const uint16_t *)a.weight;
  p.ldx = a.ldx, p.ldr = a.ldr, p.M = a.M, p.K8 = K8, p.wpr = wpr;
  p.eps = a.eps, p.eps64 = (double)a.eps, p.inv_k64 = 1.0 / (double)a.K;
  p.inv_k.hi = (float)p.inv_k64;
  p.inv_k.lo = (float)(p.inv_k64 - (double)p.inv_k.hi);
  p.in_scale = a.input_scale, p.h_out = (uint16_t *)a.h_out, p.y = a.y, p.x_scale = a.x_scale;
  const int rows = std::max(1, kWarpsPerCta / wpr);
  const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(32 * wpr * rows);
  const int nv = vecs();
  switch (a.out) {
    case kNormBf16: return launch_nv<kNormBf16, false>(nv, p, grid, block, st);
    case kNormInt8:
      return a.input_scale ? launch_nv<kNormInt8, false>(nv, p, grid, block, st)
                           : launch_nv<kNormInt8, true>(nv, p, grid, block, st);
    case kNormE4m3:
      return a.input_scale ? launch_nv<kNormE4m3, false>(nv, p, grid, block, st)
                           : launch_nv<kNormE4m3, true>(nv, p, grid, block, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
