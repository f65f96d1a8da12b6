// Rotary positions: the pair (a, b) of a head's dimensions turns by the angle
// of its token's position,
//   a' = a cos - b sin,  b' = b cos + a sin,
// each product and sum one binary32 operation, the result rounded to BF16.
// Pairs are (i, i + rot/2) in the half layout and (2i, 2i + 1) in the pairs
// layout; dimensions from rot on pass unchanged.  Cosines and sines come from a
// table of one row per position, written once by k_rope_table in FP64, so any
// scaling of the frequencies for long contexts costs nothing per token and the
// angles of far positions lose nothing.
//
// With the store, a token's rotated key goes to the mixed cache through the
// quantizer of qlin_kv_store_mixed without passing through memory as BF16.
// Bound by HBM: q in and out, k and v in, codes out.
#include "common.cuh"
#include "kernels.h"
#include "kv_quant.cuh"

#include <algorithm>

namespace qlin {

namespace {

constexpr int kWarps = 8;         // warps of a CTA; each takes work units of its own
constexpr int kHeadsPerItem = 4;  // kv heads of one token a warp quantizes at once

// ---------------------------------------------------------------- frequencies
// Radians per position of pair i, scaled for long contexts:
//   linear:   f_i / factor
//   NTK:      theta' = theta * factor^(rot / (rot - 2))
//   by parts: pairs that turn often within the original context keep f_i, pairs
//             that turn rarely get f_i / factor, with a linear ramp in the
//             number of turns between beta_slow and beta_fast (B. Peng et al.,
//             "YaRN: Efficient Context Window Extension of Large Language
//             Models", 2023, section 3.2).
__global__ void k_rope_table(int64_t max_pos, int half, double theta, int scaling, double factor,
                             double original_context, double beta_fast, double beta_slow, double amplitude,
                             float *__restrict__ table) {
  pdl_wait();
  const int64_t n = max_pos * half;
  for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < n; j += (int64_t)gridDim.x * blockDim.x) {
    const int64_t pos = j / half;
    const int i = (int)(j % half);
    const double rot = 2.0 * half;
    double base = theta;
    if (scaling == QLIN_ROPE_NTK) base = theta * pow(factor, rot / (rot - 2.0));
    double f = pow(base, -2.0 * i / rot);
    if (scaling == QLIN_ROPE_LINEAR) f /= factor;
    if (scaling == QLIN_ROPE_BY_PARTS) {
      const double turns = original_context * f / 6.283185307179586;
      const double keep = fmin(fmax((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
      f = (1.0 - keep) * f / factor + keep * f;
    }
    double s, c;
    sincos((double)pos * f, &s, &c);
    table[pos * 2 * half + i] = (float)(c * amplitude);
    table[pos * 2 * half + half + i] = (float)(s * amplitude);
  }
}

// ------------------------------------------------------------------- rotation
struct RopeParams {
  const float *table;
  const int64_t *positions;
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  int64_t T, ldq, ldk, ldqo, ldko, max_pos;
  int Hq, Hk, D, rot, half_layout;
  int units_q, units;  // work units of a token: q (and k) slices, all
  int slice;           // heads of a q slice
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Heads [h0, h1) of one token.  A lane keeps 16 dimensions of a head (8 pairs,
// whose cosines and sines it loads once, or 16 dimensions past rot) and walks
// over the heads; D/16 lanes make a head.
__device__ __forceinline__ void rotate_heads(const RopeParams &p, int64_t t, const float *row, int h0, int h1,
                                             int lane) {
  const int per = p.D / 16;              // lanes of a head
  const int at_once = 32 / per;          // heads a warp handles at once
  const int item = lane % per, first = lane / per;
  if (first >= at_once) return;
  const bool turns = item * 16 < p.rot;
  const int half = p.rot / 2;
  // the two 8-dimension pieces of the lane
  const int d0 = turns && p.half_layout ? item * 8 : item * 16;
  const int d1 = turns && p.half_layout ? half + item * 8 : item * 16 + 8;
  float c[8], s[8];
  if (turns) {
    *reinterpret_cast<float4 *>(c) = __ldg(reinterpret_cast<const float4 *>(row + item * 8));
    *reinterpret_cast<float4 *>(c + 4) = __ldg(reinterpret_cast<const float4 *>(row + item * 8) + 1);
    *reinterpret_cast<float4 *>(s) = __ldg(reinterpret_cast<const float4 *>(row + half + item * 8));
    *reinterpret_cast<float4 *>(s + 4) = __ldg(reinterpret_cast<const float4 *>(row + half + item * 8) + 1);
  }
#pragma unroll 4
  for (int h = h0 + first; h < h1; h += at_once) {
    const bool isq = h < p.Hq;
    const int64_t head = (int64_t)(isq ? h : h - p.Hq) * p.D;
    const uint16_t *in = (isq ? p.q + t * p.ldq : p.k + t * p.ldk) + head;
    uint16_t *out = (isq ? p.q_out + t * p.ldqo : p.k_out + t * p.ldko) + head;
    uint4 a = *reinterpret_cast<const uint4 *>(in + d0), b = *reinterpret_cast<const uint4 *>(in + d1);
    if (turns) {
      uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (p.half_layout) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float al = lo_f(x[j]), ah = hi_f(x[j]), bl = lo_f(x[4 + j]), bh = hi_f(x[4 + j]);
          x[j] = pack_bf16(turn_a(al, bl, c[2 * j], s[2 * j]), turn_a(ah, bh, c[2 * j + 1], s[2 * j + 1]));
          x[4 + j] = pack_bf16(turn_b(al, bl, c[2 * j], s[2 * j]), turn_b(ah, bh, c[2 * j + 1], s[2 * j + 1]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float al = lo_f(x[j]), bl = hi_f(x[j]);
          x[j] = pack_bf16(turn_a(al, bl, c[j], s[j]), turn_b(al, bl, c[j], s[j]));
        }
      }
      a = make_uint4(x[0], x[1], x[2], x[3]);
      b = make_uint4(x[4], x[5], x[6], x[7]);
    }
    *reinterpret_cast<uint4 *>(out + d0) = a;
    *reinterpret_cast<uint4 *>(out + d1) = b;
  }
}

// N (4 or 8) consecutive dimensions from d0 on of a rotated head, as BF16 words
// (the partner dimensions of the half layout are read from memory again).
template <int N>
__device__ __forceinline__ void rotated_piece(const uint16_t *head, int d0, const float *row, int rot,
                                              bool half_layout, uint32_t (&o)[N / 2]) {
  load_words<N / 2>(head + d0, o);
  if (d0 >= rot) return;
  const int half = rot / 2;
  if (half_layout) {
    const bool is_a = d0 < half;
    uint32_t other[N / 2];
    load_words<N / 2>(head + (is_a ? d0 + half : d0 - half), other);
    const float *c = row + (is_a ? d0 : d0 - half), *s = c + half;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float2 cc = __ldg(reinterpret_cast<const float2 *>(c) + j);
      float2 ss = __ldg(reinterpret_cast<const float2 *>(s) + j);
      if (is_a) ss = make_float2(-ss.x, -ss.y);
      o[j] = pack_bf16(turn_b(lo_f(other[j]), lo_f(o[j]), cc.x, ss.x), turn_b(hi_f(other[j]), hi_f(o[j]), cc.y, ss.y));
    }
  } else {
    const float *c = row + d0 / 2, *s = c + half;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float a = lo_f(o[j]), b = hi_f(o[j]), cc = __ldg(c + j), ss = __ldg(s + j);
      o[j] = pack_bf16(turn_a(a, b, cc, ss), turn_b(a, b, cc, ss));
    }
  }
}

// The table row of token t's position, or null: a negative position is padding,
// one beyond the table is reported.
__device__ __forceinline__ const float *table_row(const RopeParams &p, int64_t t, unsigned *status) {
  const int64_t pos = p.positions[t];
  if (pos >= p.max_pos) set_status(status, QLIN_ERR_INVALID_ARG);
  return pos >= 0 && pos < p.max_pos ? p.table + pos * p.rot : nullptr;
}

__global__ void __launch_bounds__(32 * kWarps) k_rope(const RopeParams p, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < p.T * p.units; u += nwarps) {
    const int64_t t = u / p.units;
    const int part = (int)(u % p.units);
    const float *row = table_row(p, t, status);
    if (row) rotate_heads(p, t, row, part * p.slice, min((part + 1) * p.slice, p.Hq + p.Hk), lane);
  }
}

// ------------------------------------------------------- rotation and store
struct StoreParams {
  const uint16_t *v;
  int64_t ldv, num_slots;
  const int64_t *slots;
  int H;
  uint8_t *kc, *vc;
  uint16_t *ks, *vs;
};

// Quantizes kv heads [h0, h0 + 4) of token t into its slot: lanes 8j..8j+7 hold
// head h0 + j, each E = D/8 consecutive dimensions, as the plain store does.
template <int E>
__device__ __forceinline__ void store_item(const RopeParams &p, const StoreParams &s, int64_t t, int64_t slot,
                                           const float *row, int h0, int lane) {
  constexpr int D = 8 * E;
  constexpr int GL = E >= 32 ? 1 : 32 / E;  // lanes of a 32-dimension key group
  constexpr int N = E < 8 ? E : 8;
  const int j = lane / 8, sub = lane % 8, h = h0 + j;
  uint32_t kw[E / 2], vw[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) kw[i] = vw[i] = 0u;
  if (h < s.H) {
    const uint16_t *kh = p.k + t * p.ldk + (int64_t)h * D;
    load_words<E / 2>(s.v + t * s.ldv + (int64_t)h * D + sub * E, vw);
#pragma unroll
    for (int i = 0; i < E / N; ++i) {
      uint32_t o[N / 2];
      rotated_piece<N>(kh, sub * E + i * N, row, p.rot, p.half_layout, o);
#pragma unroll
      for (int n = 0; n < N / 2; ++n) kw[i * (N / 2) + n] = o[n];
    }
  }
  float ka = 0.0f, va = 0.0f;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    ka = fmaxf(ka, fmaxf(fabsf(lo_f(kw[i])), fabsf(hi_f(kw[i]))));
    va = fmaxf(va, fmaxf(fabsf(lo_f(vw[i])), fabsf(hi_f(vw[i]))));
  }
  ka = group_max<GL>(ka);
  va = group_max<8>(va);
  const uint16_t ks16 = scale16(ka, kQmaxInt8), vs16 = scale16(va, kQmaxE4m3);
  const Scale ksc = make_scale(half_bits_to_f32(ks16)), vsc = make_scale(half_bits_to_f32(vs16));
  uint32_t kq[E / 4], vq[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    kq[i] = pack4_low(int8_code_word(quotient<true>(lo_f(kw[2 * i]), ksc)),
                      int8_code_word(quotient<true>(hi_f(kw[2 * i]), ksc)),
                      int8_code_word(quotient<true>(lo_f(kw[2 * i + 1]), ksc)),
                      int8_code_word(quotient<true>(hi_f(kw[2 * i + 1]), ksc)));
    vq[i] = e4m3_pack4(quotient<true>(lo_f(vw[2 * i]), vsc), quotient<true>(hi_f(vw[2 * i]), vsc),
                       quotient<true>(lo_f(vw[2 * i + 1]), vsc), quotient<true>(hi_f(vw[2 * i + 1]), vsc));
  }
  if (h < s.H) {
    const int64_t base = slot * s.H + h;
    store_words<E / 4>(s.kc + base * D + sub * E, kq);
    store_words<E / 4>(s.vc + base * D + sub * E, vq);
    if (sub % GL == 0) s.ks[base * (D / 32) + sub / GL] = ks16;
    if (sub == 0) s.vs[base] = vs16;
  }
}

template <int E>
__global__ void __launch_bounds__(32 * kWarps) k_rope_kv_store(const RopeParams p, const StoreParams s,
                                                              unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * kWarps;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < p.T * p.units; u += nwarps) {
    const int64_t t = u / p.units;
    const int part = (int)(u % p.units);
    const float *row = table_row(p, t, status);
    if (part < p.units_q) {
      if (row) rotate_heads(p, t, row, part * p.slice, min((part + 1) * p.slice, p.Hq), lane);
      continue;
    }
    const int64_t slot = s.slots[t];
    if (slot >= s.num_slots) {
      if (lane == 0) set_status(status, QLIN_ERR_INVALID_ARG);
    } else if (slot >= 0 && row) {
      store_item<E>(p, s, t, slot, row, (part - p.units_q) * kHeadsPerItem, lane);
    }
  }
}

// Heads of a q slice: as few as a warp handles at once while the tokens do not
// fill the GPU (latency), a token's whole row of heads when they do (the lane
// then loads its cosines and sines once).
int slice_heads(int64_t T, int heads, int D, int sms) {
  const int at_once = std::max(1, 32 / (D / 16));
  int slices = (heads + at_once - 1) / at_once;
  while (slices > 1 && T * slices > (int64_t)sms * 32) slices = (slices + 1) / 2;
  return ((heads + slices - 1) / slices + at_once - 1) / at_once * at_once;
}

RopeParams rope_params(const RopeArgs &r, int heads, int sms) {
  RopeParams p{};
  p.table = r.table, p.positions = r.positions, p.max_pos = r.max_pos;
  p.q = (const uint16_t *)r.q, p.k = (const uint16_t *)r.k;
  p.q_out = (uint16_t *)r.q_out, p.k_out = (uint16_t *)r.k_out;
  p.T = r.T, p.ldq = r.ldq, p.ldk = r.ldk, p.ldqo = r.ldqo, p.ldko = r.ldko;
  p.Hq = (int)r.Hq, p.Hk = (int)r.Hk, p.D = (int)r.D, p.rot = (int)r.rot;
  p.half_layout = r.layout == QLIN_ROPE_HALF;
  p.slice = slice_heads(r.T, heads, p.D, sms);
  p.units_q = p.units = (heads + p.slice - 1) / p.slice;
  return p;
}

dim3 unit_grid(int64_t units, int sms) {
  const int64_t need = (units + kWarps - 1) / kWarps;
  return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(need, (int64_t)sms * 64)));
}

template <int E>
cudaError_t launch_store_e(const RopeParams &p, const StoreParams &s, unsigned *status, int sms, cudaStream_t st) {
  return launch_kernel(k_rope_kv_store<E>, unit_grid(p.T * p.units, sms), dim3(32 * kWarps), 0, st, 1, p, s, status);
}

}  // namespace

cudaError_t launch_rope_table(int64_t max_pos, int64_t rot, double theta, int scaling, double factor,
                              double original_context, double beta_fast, double beta_slow, double amplitude,
                              float *table, cudaStream_t st) {
  const int64_t n = max_pos * (rot / 2);
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, 4096));
  return launch_kernel(k_rope_table, grid, dim3(256), 0, st, 1, max_pos, (int)(rot / 2), theta, scaling, factor,
                       original_context, beta_fast, beta_slow, amplitude, table);
}

cudaError_t launch_rope(const RopeArgs &r, unsigned *status, int sms, cudaStream_t st) {
  const RopeParams p = rope_params(r, (int)(r.Hq + r.Hk), sms);
  return launch_kernel(k_rope, unit_grid(p.T * p.units, sms), dim3(32 * kWarps), 0, st, 1, p, status);
}

cudaError_t launch_rope_kv_store(const RopeArgs &r, const KvArgs &kv, unsigned *status, int sms, cudaStream_t st) {
  RopeParams p = rope_params(r, (int)r.Hq, sms);
  p.units = p.units_q + (int)((r.Hk + kHeadsPerItem - 1) / kHeadsPerItem);
  StoreParams s{};
  s.v = (const uint16_t *)kv.v, s.ldv = kv.ldv, s.num_slots = kv.num_slots, s.slots = kv.slots, s.H = (int)r.Hk;
  s.kc = (uint8_t *)kv.k_cache, s.ks = (uint16_t *)kv.k_scale;
  s.vc = (uint8_t *)kv.v_cache, s.vs = (uint16_t *)kv.v_scale;
  switch (r.D) {
    case 32: return launch_store_e<4>(p, s, status, sms, st);
    case 64: return launch_store_e<8>(p, s, status, sms, st);
    case 128: return launch_store_e<16>(p, s, status, sms, st);
    case 256: return launch_store_e<32>(p, s, status, sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
