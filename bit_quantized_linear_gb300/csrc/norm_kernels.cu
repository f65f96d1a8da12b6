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
// row is the work of `wpr` warps.  Bound by HBM: x, residual and h_out are 2
// bytes an element, the output 1 or 2.  With codes the arithmetic is close
// behind, so it runs on pairs of elements as packed binary32 operations (the
// same roundings, lane by lane), and a CTA walks over rows: the weights are
// unpacked once, and the next row is on its way while this one is worked on
// (8192 x 2048 static E4M3 with residual: 25.6 us without; 21.2 us, 5.5 TB/s,
// with it and the residual added as BF16).  BF16 output has arithmetic to spare
// and gains more from whole rows in flight (32640 x 3584: 146 us walking, 134 not).
#include "common.cuh"
#include "kernels.h"
#include "kv_quant.cuh"

#include <algorithm>

namespace qlin {

namespace {

constexpr int kMaxWarpsPerRow = 16;
constexpr int kMaxVecs = 8;       // 16-byte vectors of a row a thread holds
constexpr int kWarpsPerCta = 8;
constexpr int kCtaWarps = 16;     // warps of an SM the registers are budgeted for

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

// ---- two binary32 values in a 64-bit register
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float f32x2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f32x2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
constexpr uint64_t kMinusOne2 = 0xBF800000BF800000ull;
__device__ __forceinline__ uint64_t f32x2_sub(uint64_t a, uint64_t b) { return f32x2_fma(b, kMinusOne2, a); }  // exact product
__device__ __forceinline__ uint64_t f32x2_of(uint32_t bf16x2) {
  return (uint64_t)(bf16x2 << 16) | ((uint64_t)(bf16x2 & 0xFFFF0000u) << 32);
}
__device__ __forceinline__ uint32_t bf16x2_of(uint64_t v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(f32x2_lo(v), f32x2_hi(v));
  return *reinterpret_cast<const uint32_t *>(&b);
}
// Two running sums with their errors (add_value, lane by lane).
struct TwoFloat2 {
  uint64_t hi, lo;
};
__device__ __forceinline__ void add_values(TwoFloat2 &a, uint64_t b) {
  const uint64_t s = f32x2_add(a.hi, b);
  const uint64_t bb = f32x2_sub(s, a.hi);
  const uint64_t e = f32x2_add(f32x2_sub(a.hi, f32x2_sub(s, bb)), f32x2_sub(b, bb));
  a.hi = s;
  a.lo = f32x2_add(a.lo, e);
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
  int K8;                     // vectors of a row
  int wpr, wpr_log2;          // its warps
  double eps64, inv_k64;
  float eps;
  TwoFloat inv_k;
  const float *in_scale;
  uint16_t *h_out;
  void *y;
  float *x_scale;
};

// The quantizer of a row: codes of fl32(y / s), by quotient() of common.cuh two
// elements at a time.  Under a static scale y is first cut to +-`bound`, beyond
// which every code is the largest (127.25 s rounds to 127, 512 s saturates); that
// also keeps the quotient's intermediates finite.  A NaN stays one for E4M3; for INT8
// it becomes -bound, which gives quantize_one's code of a NaN (-127).
template <int OUT, bool BOUNDED>
struct RowQuantizer {
  Scale c;
  float bound;
  uint64_t r2, ns2;
  __device__ __forceinline__ explicit RowQuantizer(float s) : c(make_scale(s)) {
    bound = (OUT == kNormInt8 ? 127.25f : 512.0f) * s;
    r2 = f32x2_pack(c.r, c.r);
    ns2 = f32x2_pack(-s, -s);
  }
  __device__ __forceinline__ float cut(float y) const {
    if constexpr (OUT == kNormInt8) {
      y = fmaxf(y, -bound);  // of a NaN and a number, the number
      return BOUNDED ? y : fminf(y, bound);
    } else if constexpr (BOUNDED) {
      return y;
    } else {
      float d;  // the sign of y, the smaller magnitude
      asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(y), "f"(bound));
      return d;
    }
  }
  __device__ __forceinline__ uint64_t quotients(uint64_t y) const {
    y = f32x2_pack(cut(f32x2_lo(y)), cut(f32x2_hi(y)));
    const uint64_t q = f32x2_mul(y, r2);
    return f32x2_fma(f32x2_fma(q, ns2, y), r2, q);
  }
  // Four codes of two pairs, element i in byte i.
  __device__ __forceinline__ uint32_t codes4(uint64_t y0, uint64_t y1) const {
    if (__builtin_expect(!c.fast, 0)) {
      constexpr int QT = OUT == kNormInt8 ? QLIN_INT8 : QLIN_E4M3;
      return (uint32_t)quantize_one<QT, BOUNDED>(f32x2_lo(y0), c) |
             ((uint32_t)quantize_one<QT, BOUNDED>(f32x2_hi(y0), c) << 8) |
             ((uint32_t)quantize_one<QT, BOUNDED>(f32x2_lo(y1), c) << 16) |
             ((uint32_t)quantize_one<QT, BOUNDED>(f32x2_hi(y1), c) << 24);
    }
    uint64_t q0 = quotients(y0), q1 = quotients(y1);
    if constexpr (OUT == kNormInt8) {
      // 1.5 * 2^23 rounds to an integer, whose low byte is the code (int8_code_word);
      // a quotient by the row's own maximum stays below 127.5
      constexpr uint64_t kRound2 = 0x4B4000004B400000ull;
      q0 = f32x2_add(q0, kRound2);
      q1 = f32x2_add(q1, kRound2);
      return pack4_low((uint32_t)q0, (uint32_t)(q0 >> 32), (uint32_t)q1, (uint32_t)(q1 >> 32));
    } else {
      // the correction step loses the sign of a quotient that is zero: it comes from y
      const uint32_t code = e4m3_pack4(f32x2_lo(q0), f32x2_hi(q0), f32x2_lo(q1), f32x2_hi(q1));
      const uint32_t sign = __byte_perm(__byte_perm((uint32_t)y0, (uint32_t)(y0 >> 32), 0x0073),
                                        __byte_perm((uint32_t)y1, (uint32_t)(y1 >> 32), 0x0073), 0x5410);
      return code | (sign & 0x80808080u);
    }
  }
};

// bf16(x + r) of two pairs: one rounding of the exact sum.  (Rounding to binary32
// first, as the definition has it, gives the same: binary32 only rounds a sum whose
// smaller term is below 2^-16 of the larger, which is then the nearest BF16 itself.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s =
      __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&s);
}

// Eight BF16 values of a row as a thread keeps them: as binary32 pairs where the
// registers allow (up to four vectors a thread), else packed.
template <bool WIDE>
struct Values;
template <>
struct Values<true> {
  uint64_t v[4];
  __device__ __forceinline__ void set(const uint4 &p) {
    v[0] = f32x2_of(p.x), v[1] = f32x2_of(p.y), v[2] = f32x2_of(p.z), v[3] = f32x2_of(p.w);
  }
  __device__ __forceinline__ uint64_t pair(int j) const { return v[j]; }
};
template <>
struct Values<false> {
  uint4 p;
  __device__ __forceinline__ void set(const uint4 &q) { p = q; }
  __device__ __forceinline__ uint64_t pair(int j) const {
    return f32x2_of(j == 0 ? p.x : j == 1 ? p.y : j == 2 ? p.z : p.w);
  }
};

template <int NV, int OUT, bool DYN>
__global__ void __launch_bounds__(32 * kMaxWarpsPerRow) k_rmsnorm(const RmsParams p) {
  constexpr bool kWalk = NV <= 4 && OUT != kNormBf16;
  using V = Values<kWalk>;
  __shared__ TwoFloat s_sum[2][kMaxWarpsPerRow];  // by turns: one barrier a row may be all that parts two rows
  __shared__ double s_sum64[kMaxWarpsPerRow];
  __shared__ float s_max[kMaxWarpsPerRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp >> p.wpr_log2, sub = warp & (p.wpr - 1), first = group << p.wpr_log2;
  // the warps of one row meet at a barrier of their own
  const auto row_barrier = [&] {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(p.wpr * 32) : "memory");
  };
  const int at_once = (int)blockDim.x >> (p.wpr_log2 + 5);  // rows of a CTA
  const int64_t step = (int64_t)gridDim.x * at_once;
  int64_t m = (int64_t)blockIdx.x * at_once + group;
  const int index0 = sub * 32 + lane, index_step = p.wpr * 32;
  const auto index = [&](int i) { return index0 + i * index_step; };

  V w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    w[i].set(index(i) < p.K8 ? __ldg(reinterpret_cast<const uint4 *>(p.w) + index(i)) : make_uint4(0, 0, 0, 0));
  pdl_wait();
  pdl_trigger();
  uint4 x[NV], r4[NV];
  const auto load = [&](int64_t row) {
    const uint4 *xr = reinterpret_cast<const uint4 *>(p.x + row * p.ldx);
    const uint4 *rr = reinterpret_cast<const uint4 *>(p.res + row * p.ldr);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool ok = row < p.M && index(i) < p.K8;
      x[i] = ok ? xr[index(i)] : make_uint4(0, 0, 0, 0);
      if (p.res) r4[i] = ok ? rr[index(i)] : make_uint4(0, 0, 0, 0);
    }
  };
  load(m);
  for (int turn = 0; m < p.M; m += step, turn ^= 1) {
    V h[NV];
    if (p.res) {
      uint4 *ho = reinterpret_cast<uint4 *>(p.h_out) + m * p.K8;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint4 s = make_uint4(add_bf16x2(x[i].x, r4[i].x), add_bf16x2(x[i].y, r4[i].y),
                                   add_bf16x2(x[i].z, r4[i].z), add_bf16x2(x[i].w, r4[i].w));
        if (index(i) < p.K8) ho[index(i)] = s;
        h[i].set(s);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) h[i].set(x[i]);
    }
    if (kWalk) load(m + step);

    // sum of squares
    TwoFloat2 S2{0, 0};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) add_values(S2, f32x2_mul(h[i].pair(j), h[i].pair(j)));
    }
    TwoFloat S{f32x2_lo(S2.hi), f32x2_lo(S2.lo)};
    add_pair(S, TwoFloat{f32x2_hi(S2.hi), f32x2_hi(S2.lo)});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add_pair(S, TwoFloat{__shfl_xor_sync(~0u, S.hi, o), __shfl_xor_sync(~0u, S.lo, o)});
    if (p.wpr > 1) {
      if (lane == 0) s_sum[turn][warp] = S;
      row_barrier();
      if (p.wpr <= 4) {
        S = s_sum[turn][first];
#pragma unroll 1
        for (int i = 1; i < p.wpr; ++i) add_pair(S, s_sum[turn][first + i]);
      } else {
        S = lane < p.wpr ? s_sum[turn][first + lane] : TwoFloat{0.0f, 0.0f};
#pragma unroll
        for (int o = kMaxWarpsPerRow / 2; o > 0; o >>= 1)
          add_pair(S, TwoFloat{__shfl_xor_sync(~0u, S.hi, o), __shfl_xor_sync(~0u, S.lo, o)});
        S.hi = __shfl_sync(~0u, S.hi, 0);  // lanes 16..31 hold no partial sums
        S.lo = __shfl_sync(~0u, S.lo, 0);
      }
    }
    float r = rms_reciprocal(S, p.inv_k, p.eps);
    if (__builtin_expect(!(S.hi >= 0x1p-80f && S.hi < 0x1p126f), 0)) {
      // squares beyond binary32 (or an all-zero row): the same sum in FP64.  (All of a
      // row's lanes come here or none: their sum is the same.)
      double d = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t a = h[i].pair(j);
          d += (double)f32x2_lo(a) * (double)f32x2_lo(a) + (double)f32x2_hi(a) * (double)f32x2_hi(a);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        d += __shfl_xor_sync(~0u, d, o);
      if (p.wpr > 1) {
        if (lane == 0) s_sum64[warp] = d;
        row_barrier();
        d = 0.0;
        for (int i = 0; i < p.wpr; ++i) d += s_sum64[first + i];
        row_barrier();
      }
      r = (float)(1.0 / sqrt(d * p.inv_k64 + p.eps64));
    }

    const uint64_t r2 = f32x2_pack(r, r);
    const auto normed = [&](int i, int j) { return f32x2_mul(f32x2_mul(h[i].pair(j), r2), w[i].pair(j)); };
    if constexpr (OUT == kNormBf16) {
      uint4 *yo = reinterpret_cast<uint4 *>(p.y) + m * p.K8;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (index(i) < p.K8)
          yo[index(i)] = make_uint4(bf16x2_of(normed(i, 0)), bf16x2_of(normed(i, 1)), bf16x2_of(normed(i, 2)),
                                    bf16x2_of(normed(i, 3)));
    } else {
      float s;
      if constexpr (DYN) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t y = normed(i, j);
            amax = fmaxf(amax, fmaxf(fabsf(f32x2_lo(y)), fabsf(f32x2_hi(y))));
          }
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
      const RowQuantizer<OUT, DYN> quantize(s);
      uint2 *yo = reinterpret_cast<uint2 *>(p.y) + m * p.K8;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (index(i) < p.K8)
          yo[index(i)] = make_uint2(quantize.codes4(normed(i, 0), normed(i, 1)),
                                    quantize.codes4(normed(i, 2), normed(i, 3)));
    }
    if (!kWalk) break;  // the grid covers all rows
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
  // warps of a row for at most four vectors a thread (BF16, or beyond 16 warps:
  // eight); few rows: more warps, down to one vector
  const int most = a.out == kNormBf16 ? kMaxVecs : 4;
  int wpr = 1;
  const auto vecs = [&] {
    int nv = 1;
    while (nv * wpr * 32 < K8) nv *= 2;
    return nv;
  };
  while (wpr < kMaxWarpsPerRow && vecs() > most) wpr *= 2;
  while (wpr < kMaxWarpsPerRow && vecs() > 1 && a.M * wpr < (int64_t)sms * kCtaWarps) wpr *= 2;
  if (vecs() > kMaxVecs) return cudaErrorInvalidValue;
  RmsParams p{};
  p.x = (const uint16_t *)a.x, p.res = (const uint16_t *)a.residual, p.w = (const uint16_t *)a.weight;
  p.ldx = a.ldx, p.ldr = a.ldr, p.M = a.M, p.K8 = K8;
  p.wpr = wpr;
  while (1 << p.wpr_log2 < wpr) ++p.wpr_log2;
  p.eps = a.eps, p.eps64 = (double)a.eps, p.inv_k64 = 1.0 / (double)a.K;
  p.inv_k.hi = (float)p.inv_k64;
  p.inv_k.lo = (float)(p.inv_k64 - (double)p.inv_k.hi);
  p.in_scale = a.input_scale, p.h_out = (uint16_t *)a.h_out, p.y = a.y, p.x_scale = a.x_scale;
  const int warps = std::max(wpr, kWarpsPerCta), rows = warps / wpr;
  const dim3 block(32 * warps);
  const int nv = vecs();
  const bool walk = nv <= 4 && a.out != kNormBf16;  // as in the kernel
  const int64_t all = (a.M + rows - 1) / rows;
  const dim3 grid((unsigned)(walk ? std::min<int64_t>(all, (int64_t)sms * (kCtaWarps / warps)) : all));
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
