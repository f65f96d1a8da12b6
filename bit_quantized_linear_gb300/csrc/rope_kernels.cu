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
// Bound by HBM: q in and out, k and v in, codes out.  A warp asks for all of its
// heads before it waits for its position and the table's row, so a token costs one
// trip to memory and not three (8192 tokens of 28 + 2 x 4 heads of 128: 40.6 us
// with three, 27.4 us, 5.4 TB/s, with one and the heads' batches below).
#include "common.cuh"
#include "kernels.h"
#include "kv_quant.cuh"

#include <algorithm>

namespace qlin {

namespace {

constexpr int kWarps = 8;         // warps of a CTA; each takes a work unit of its own
constexpr int kHeadsPerItem = 4;  // (token, kv head) pairs a warp quantizes at once

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
  // A unit of rotation is `tokens` tokens' heads, or (few tokens) one token's slice of
  // `slice` heads, `slices` of them to a token.
  int tokens, slice, slices;
  int64_t units;
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

// The table row of a position, or null: a negative position is padding, one
// beyond the table is reported.
__device__ __forceinline__ const float *table_row(const RopeParams &p, int64_t pos, unsigned *status) {
  if (pos >= p.max_pos) set_status(status, QLIN_ERR_INVALID_ARG);
  return pos >= 0 && pos < p.max_pos ? p.table + pos * p.rot : nullptr;
}

// Unit u: heads of p.tokens tokens, or a slice of one's.  A lane keeps 16
// dimensions of a head of one token (8 pairs, whose cosines and sines it loads
// once, or 16 dimensions past rot) and walks over the heads; D/16 lanes make a
// head.
constexpr int kHeadBatch = 2;  // heads of a lane that are in flight at once (more cost more warps than they hide)
__device__ __forceinline__ void rotate_heads(const RopeParams &p, int64_t u, int lane, unsigned *status) {
  const int per = p.D / 16;              // lanes of a head
  const int item = lane % per, group = lane / per;
  int at_once = 32 / per;                // heads a warp handles at once
  if (group >= at_once) return;
  int64_t t;
  int first = group, h0 = 0, h1 = p.Hq + p.Hk;
  if (p.slices == 1) {
    at_once /= p.tokens;                 // of each token (tokens is 1 or divides it)
    t = u * p.tokens + group / at_once;
    first = group % at_once;
  } else {
    t = u / p.slices;
    h0 = (int)(u - t * p.slices) * p.slice;
    h1 = min(h0 + p.slice, h1);
  }
  if (t >= p.T) return;
  const int64_t pos = ld_input(p.positions + t);
  const bool turns = item * 16 < p.rot;
  const int half = p.rot / 2;
  // the two 8-dimension pieces of the lane
  const int d0 = turns && p.half_layout ? item * 8 : item * 16;
  const int d1 = turns && p.half_layout ? half + item * 8 : item * 16 + 8;
  const auto place = [&](const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, int h) {
    return h < p.Hq ? q + t * ldq + (int64_t)h * p.D : k + t * ldk + (int64_t)(h - p.Hq) * p.D;
  };
  float c[8], s[8];
  bool ready = false;
  for (int hb = h0 + first; hb < h1; hb += kHeadBatch * at_once) {
    uint4 a[kHeadBatch], b[kHeadBatch];
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = hb + i * at_once;
      if (h < h1) {
        const uint16_t *in = place(p.q, p.ldq, p.k, p.ldk, h);
        a[i] = *reinterpret_cast<const uint4 *>(in + d0);
        b[i] = *reinterpret_cast<const uint4 *>(in + d1);
      }
    }
    if (!ready) {
      const float *row = table_row(p, pos, status);
      if (!row) return;
      if (turns) {
        *reinterpret_cast<float4 *>(c) = ld_input(reinterpret_cast<const float4 *>(row + item * 8));
        *reinterpret_cast<float4 *>(c + 4) = ld_input(reinterpret_cast<const float4 *>(row + item * 8) + 1);
        *reinterpret_cast<float4 *>(s) = ld_input(reinterpret_cast<const float4 *>(row + half + item * 8));
        *reinterpret_cast<float4 *>(s + 4) = ld_input(reinterpret_cast<const float4 *>(row + half + item * 8) + 1);
      }
      ready = true;
    }
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = hb + i * at_once;
      if (h >= h1) break;
      if (turns) {
        uint32_t x[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
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
        a[i] = make_uint4(x[0], x[1], x[2], x[3]);
        b[i] = make_uint4(x[4], x[5], x[6], x[7]);
      }
      uint16_t *out = const_cast<uint16_t *>(place(p.q_out, p.ldqo, p.k_out, p.ldko, h));
      *reinterpret_cast<uint4 *>(out + d0) = a[i];
      *reinterpret_cast<uint4 *>(out + d1) = b[i];
    }
  }
}

// N (4 or 8) consecutive dimensions from d0 on of a head and, in the half layout,
// their partner dimensions: as loaded, then rotated.
template <int N>
struct Piece {
  uint32_t own[N / 2], other[N / 2];
  __device__ __forceinline__ void load(const uint16_t *head, int d0, int rot, bool half_layout) {
    load_words<N / 2>(head + d0, own);
    if (d0 < rot && half_layout) load_words<N / 2>(head + (d0 < rot / 2 ? d0 + rot / 2 : d0 - rot / 2), other);
  }
  // Its cosines and sines (both layouts: N, or N/2, consecutive ones).
  float c[N], s[N];
  __device__ __forceinline__ void load_angles(int d0, const float *row, int rot, bool half_layout) {
    if (d0 >= rot) return;
    const int half = rot / 2;
    const float *from = row + (half_layout ? (d0 < half ? d0 : d0 - half) : d0 / 2);
    if (half_layout) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        *reinterpret_cast<float4 *>(c + j) = ld_input(reinterpret_cast<const float4 *>(from + j));
        *reinterpret_cast<float4 *>(s + j) = ld_input(reinterpret_cast<const float4 *>(from + half + j));
      }
    } else {
#pragma unroll
      for (int j = 0; j < N / 2; j += 2) {
        *reinterpret_cast<float2 *>(c + j) = ld_input(reinterpret_cast<const float2 *>(from + j));
        *reinterpret_cast<float2 *>(s + j) = ld_input(reinterpret_cast<const float2 *>(from + half + j));
      }
    }
  }
  __device__ __forceinline__ void rotate(int d0, int rot, bool half_layout) {
    if (d0 >= rot) return;
    if (half_layout) {
      const float sign = d0 < rot / 2 ? -1.0f : 1.0f;  // a' = a c - b s, b' = b c + a s
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        own[j] = pack_bf16(turn_b(lo_f(other[j]), lo_f(own[j]), c[2 * j], sign * s[2 * j]),
                           turn_b(hi_f(other[j]), hi_f(own[j]), c[2 * j + 1], sign * s[2 * j + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float a = lo_f(own[j]), b = hi_f(own[j]);
        own[j] = pack_bf16(turn_a(a, b, c[j], s[j]), turn_b(a, b, c[j], s[j]));
      }
    }
  }
};

__global__ void __launch_bounds__(32 * kWarps, 4) k_rope(const RopeParams p, unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u < p.units) rotate_heads(p, u, threadIdx.x & 31, status);
}

// ------------------------------------------------------- rotation and store
struct StoreParams {
  const uint16_t *v;
  int64_t ldv, num_slots;
  unsigned ctas;  // of the store
  const int64_t *slots;
  int H;
  uint8_t *kc, *vc;
  uint16_t *ks, *vs;
};

// A (token, kv head) pair as eight lanes hold it: E = D/8 consecutive dimensions
// each, as the plain store does.
template <int E>
struct StorePair {
  static constexpr int D = 8 * E, N = E < 8 ? E : 8;
  int64_t pos, slot;
  int h;
  Piece<N> k[E / N];
  uint32_t v[E / 2];

  __device__ __forceinline__ void load(const RopeParams &p, const StoreParams &s, int64_t pair, int sub) {
    const int64_t t = pair >> 32 ? pair / s.H : (int64_t)((uint32_t)pair / (uint32_t)s.H);
    h = (int)(pair - t * s.H);
    pos = slot = -1;
    if (t >= p.T) return;
    pos = ld_input(p.positions + t);
    slot = ld_input(s.slots + t);
    const uint16_t *kh = p.k + t * p.ldk + (int64_t)h * D;
#pragma unroll
    for (int i = 0; i < E / N; ++i) k[i].load(kh, sub * E + i * N, p.rot, p.half_layout);
    load_words<E / 2>(s.v + t * s.ldv + (int64_t)h * D + sub * E, v);
  }

  // (the lanes of a pair that is not stored take part in the shuffles)
  __device__ __forceinline__ void store(const RopeParams &p, const StoreParams &s, int sub, unsigned *status) {
    constexpr int GL = E >= 32 ? 1 : 32 / E;  // lanes of a 32-dimension key group
    if (slot >= s.num_slots) set_status(status, QLIN_ERR_INVALID_ARG);
    const float *row = table_row(p, pos, status);
    const bool stored = row && slot >= 0 && slot < s.num_slots;
    uint32_t kw[E / 2];
    if (stored) {
#pragma unroll
      for (int i = 0; i < E / N; ++i) k[i].load_angles(sub * E + i * N, row, p.rot, p.half_layout);
    }
#pragma unroll
    for (int i = 0; i < E / N; ++i) {
      if (stored) k[i].rotate(sub * E + i * N, p.rot, p.half_layout);
#pragma unroll
      for (int n = 0; n < N / 2; ++n) kw[i * (N / 2) + n] = k[i].own[n];
    }
    float ka = 0.0f, va = 0.0f;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      ka = fmaxf(ka, fmaxf(fabsf(lo_f(kw[i])), fabsf(hi_f(kw[i]))));
      va = fmaxf(va, fmaxf(fabsf(lo_f(v[i])), fabsf(hi_f(v[i]))));
    }
    ka = group_max<GL>(ka);
    va = group_max<8>(va);
    if (!stored) return;
    const uint16_t ks16 = scale16(ka, kQmaxInt8), vs16 = scale16(va, kQmaxE4m3);
    const Scale ksc = make_scale(half_bits_to_f32(ks16)), vsc = make_scale(half_bits_to_f32(vs16));
    uint32_t kq[E / 4], vq[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      kq[i] = pack4_low(int8_code_word(quotient<true>(lo_f(kw[2 * i]), ksc)),
                        int8_code_word(quotient<true>(hi_f(kw[2 * i]), ksc)),
                        int8_code_word(quotient<true>(lo_f(kw[2 * i + 1]), ksc)),
                        int8_code_word(quotient<true>(hi_f(kw[2 * i + 1]), ksc)));
      vq[i] = e4m3_pack4(quotient<true>(lo_f(v[2 * i]), vsc), quotient<true>(hi_f(v[2 * i]), vsc),
                         quotient<true>(lo_f(v[2 * i + 1]), vsc), quotient<true>(hi_f(v[2 * i + 1]), vsc));
    }
    const int64_t base = slot * s.H + h;
    store_words<E / 4>(s.kc + base * D + sub * E, kq);
    store_words<E / 4>(s.vc + base * D + sub * E, vq);
    if (sub % GL == 0) s.ks[base * (D / 32) + sub / GL] = ks16;
    if (sub == 0) s.vs[base] = vs16;
  }
};

// CTAs of rotation (q) and of the store take turns, in proportion, so that both
// kinds are in flight all the time.
template <int E>
__global__ void __launch_bounds__(32 * kWarps, E >= 32 ? 2 : 4) k_rope_kv_store(const RopeParams p, const StoreParams s,
                                                                 unsigned *status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned before = (unsigned)((uint64_t)blockIdx.x * s.ctas / gridDim.x);
  const unsigned after = (unsigned)(((uint64_t)blockIdx.x + 1) * s.ctas / gridDim.x);
  if (after == before) {
    const int64_t u = (int64_t)(blockIdx.x - before) * kWarps + warp;
    if (u < p.units) rotate_heads(p, u, lane, status);
    return;
  }
  StorePair<E> pair;
  pair.load(p, s, ((int64_t)before * kWarps + warp) * kHeadsPerItem + lane / 8, lane % 8);
  pair.store(p, s, lane % 8, status);
}

// Tokens that fill the GPU: as many to a unit as give a lane up to kHeadBatch
// heads.  Fewer: slices of a token, down to the heads a warp handles at once.
RopeParams rope_params(const RopeArgs &r, int heads, int sms) {
  RopeParams p{};
  p.table = r.table, p.positions = r.positions, p.max_pos = r.max_pos;
  p.q = (const uint16_t *)r.q, p.k = (const uint16_t *)r.k;
  p.q_out = (uint16_t *)r.q_out, p.k_out = (uint16_t *)r.k_out;
  p.T = r.T, p.ldq = r.ldq, p.ldk = r.ldk, p.ldqo = r.ldqo, p.ldko = r.ldko;
  p.Hq = (int)r.Hq, p.Hk = heads - (int)r.Hq, p.D = (int)r.D, p.rot = (int)r.rot;
  p.half_layout = r.layout == QLIN_ROPE_HALF;
  const int at_once = std::max(1, 32 / (p.D / 16));
  const int64_t full = (int64_t)sms * 32;  // units that fill the GPU
  p.tokens = 1;
  while (at_once % (2 * p.tokens) == 0 && heads * 2 * p.tokens <= kHeadBatch * at_once && r.T >= full * 2 * p.tokens)
    p.tokens *= 2;
  p.slices = p.tokens > 1 ? 1 : (heads + at_once - 1) / at_once;
  while (p.slices > 1 && r.T * p.slices > full) p.slices = (p.slices + 1) / 2;
  p.slice = ((heads + p.slices - 1) / p.slices + at_once - 1) / at_once * at_once;
  p.slices = (heads + p.slice - 1) / p.slice;
  p.units = p.slices > 1 ? r.T * p.slices : (r.T + p.tokens - 1) / p.tokens;
  return p;
}

unsigned unit_ctas(int64_t units) { return (unsigned)((units + kWarps - 1) / kWarps); }

template <int E>
cudaError_t launch_store_e(const RopeParams &p, StoreParams s, unsigned *status, cudaStream_t st) {
  s.ctas = unit_ctas((p.T * s.H + kHeadsPerItem - 1) / kHeadsPerItem);
  return launch_kernel(k_rope_kv_store<E>, dim3(unit_ctas(p.units) + s.ctas), dim3(32 * kWarps), 0, st, 1, p, s,
                       status);
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
  return launch_kernel(k_rope, dim3(unit_ctas(p.units)), dim3(32 * kWarps), 0, st, 1, p, status);
}

cudaError_t launch_rope_kv_store(const RopeArgs &r, const KvArgs &kv, unsigned *status, int sms, cudaStream_t st) {
  const RopeParams p = rope_params(r, (int)r.Hq, sms);
  StoreParams s{};
  s.v = (const uint16_t *)kv.v, s.ldv = kv.ldv, s.num_slots = kv.num_slots, s.slots = kv.slots, s.H = (int)r.Hk;
  s.kc = (uint8_t *)kv.k_cache, s.ks = (uint16_t *)kv.k_scale;
  s.vc = (uint8_t *)kv.v_cache, s.vs = (uint16_t *)kv.v_scale;
  switch (r.D) {
    case 32: return launch_store_e<4>(p, s, status, st);
    case 64: return launch_store_e<8>(p, s, status, st);
    case 128: return launch_store_e<16>(p, s, status, st);
    case 256: return launch_store_e<32>(p, s, status, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
