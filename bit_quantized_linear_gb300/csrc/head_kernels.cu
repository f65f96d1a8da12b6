// Norms of the query and key heads with the rotary positions in the same pass, and
// the same with keys and values stored into the 4-bit cache.
//
//   r  = fl32(1 / sqrt(sum_d x^2 / D + eps)),  y = fl32(fl32(x r) w)     (y = x without weights)
//   a' = y_a cos - y_b sin,  b' = y_b cos + y_a sin,  rounded to BF16
//
// For the keys, each is a single binary32 operation, and r does not depend on the order of its sum
// (the errors of the additions are kept, as in norm_kernels.cu), so their codes
// are reproducible bit for bit.  Queries with a weight, which nothing quantizes, take the sum, the weights and the
// turn as fused operations (within 2^-19 of a pair's magnitude before the rounding to BF16), for a quarter of the
// instructions; heads that these do not hold take the single operations.  Positions may have up to four axes (time, height,
// width): a pair's angle then comes from the table's row of its own axis.
//
// Bound by HBM: heads in and out, codes out (29.8 us for 8192 tokens of 28 + 4 heads of 128 into the cache, 4.8 TB/s; 25.8
// us for the norms alone, 5.4 TB/s).  A head is D/16 lanes of 16 dimensions, whose rows come by
// asynchronous copies some heads ahead.  Queries and keys run different code beside each other, and its size shows: one
// kernel for both layouts took 32.3 and 27.6 us where two took 31.3 and 27.0, loops unrolled by two 36.5 and 32.0.
#include "common.cuh"
#include "int4_cache.cuh"
#include "kernels.h"
#include "kv_quant.cuh"
#include "rms.cuh"
#include "rope.cuh"

#include <algorithm>

namespace qlin {

namespace {

constexpr int kWarps = 4;         // warps of a CTA; each takes a work unit of its own
constexpr int kCtas = 4;          // resident CTAs

struct HeadParams {
  const float *table;
  const int64_t *positions;  // [axes, T]
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *q_out, *k_out;
  int64_t T, ldq, ldk, ldqo, ldko, max_pos;
  int Hq, Hk, D, rot, half_layout, axes;
  uint32_t axis[16];         // two bits for each pair
  float eps, one;            // 1, where the compiler does not see it (sum_of)
  float least;               // sums of squares below lose bits beside eps (head_rms_fast)
  TwoFloat inv_d;
  double eps64, inv_d64;
  int per, width;            // a head is `per` of `width` (a power of two) lanes
  // Heads of one kind in batches of those that a warp has at once: `batches` of a token, or one of `tokens` tokens' few.
  struct Units {
    int heads, tokens, batches;
    int64_t count;  // of all tokens
  } uq, uk;
  int64_t key_warps;  // of the grid's warps, those that work on the keys (or the store)
};

// The rows of a token's positions (rows of the table, 0 for axes that are not there);
// false: the token is left out.
struct Rows {
  int at[4];
  __device__ __forceinline__ int of(int axis) const {
    return axis & 2 ? (axis & 1 ? at[3] : at[2]) : (axis & 1 ? at[1] : at[0]);
  }
};
__device__ __forceinline__ bool rows_of(const HeadParams &p, const int64_t (&pos)[4], Rows &rows, unsigned *status) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    if (a < p.axes && pos[a] >= p.max_pos) set_status(status, QLIN_ERR_INVALID_ARG);
    ok = ok && (a >= p.axes || (pos[a] >= 0 && pos[a] < p.max_pos));
    rows.at[a] = (int)pos[a];
  }
  return ok;
}
__device__ __forceinline__ bool token_rows(const HeadParams &p, int64_t t, Rows &rows, unsigned *status) {
  int64_t pos[4] = {0, 0, 0, 0};
#pragma unroll
  for (int a = 0; a < 4; ++a)
    if (a < p.axes) pos[a] = ld_input(p.positions + a * p.T + t);
  return rows_of(p, pos, rows, status);
}

// x + y and x - y, lane by lane, of products already rounded.  (A packed addition of a packed product is
// compiled to one fused operation, although both are asked to round: so it is a fused one with 1.)
__device__ __forceinline__ uint64_t sum_of(const HeadParams &p, uint64_t x, uint64_t y) {
  return f32x2_fma(y, f32x2_pack(p.one, p.one), x);
}
__device__ __forceinline__ uint64_t difference_of(const HeadParams &p, uint64_t x, uint64_t y) {
  return f32x2_fma(y, f32x2_pack(-p.one, -p.one), x);
}

// A lane's 16 dimensions of a head: two pieces of 8, d0 and d0 + piece on.  HALF: the first and second elements of eight
// pairs, or pieces past rot half of what is there apart; otherwise four pairs each, `per` pieces apart, so that lanes side by side have a row's
// pieces side by side (16 dimensions one after the other, half of each sector at a time, took 36.5 us against 27.9 for 8192
// tokens of 28 + 4 heads of 128, with the store 40.8 against 29.1).  Pairs pair[i] ... pair[i] + 3 turn where turns[i].
struct Pieces {
  int d0, piece, pair[2];
  bool turns[2];
};
template <bool HALF>
__device__ __forceinline__ Pieces pieces_of(const HeadParams &p, int item, int per) {
  if constexpr (HALF) {
    const bool turns = item * 16 < p.rot;
    return {turns ? item * 8 : p.rot / 2 + item * 8, turns ? p.rot / 2 : (p.D - p.rot) / 2, {item * 8, item * 8 + 4}, {turns, turns}};
  }
  return {item * 8, per * 8, {item * 4, (item + per) * 4}, {item * 8 < p.rot, (item + per) * 8 < p.rot}};
}
// The axes of N pairs (`pair` a multiple of N), two bits each.
template <int N>
__device__ __forceinline__ uint32_t axes_of(const HeadParams &p, int pair) {
  return (p.axis[pair >> 4] >> (2 * (pair & 15))) & ((1u << (2 * N)) - 1);
}
template <int N>
__device__ __forceinline__ bool same_axis(uint32_t axes) { return axes == (axes & 3u) * (((1u << (2 * N)) - 1) / 3); }
// Cosines and sines of N pairs.
template <int N>
__device__ __forceinline__ void load_angles(const HeadParams &p, const Rows &rows, int pair, float *c, float *s) {
  const int half = p.rot / 2;
  const uint32_t axes = axes_of<N>(p, pair);
  if (same_axis<N>(axes)) {
    const float *row = p.table + (int64_t)rows.of(axes & 3) * p.rot + pair;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      *reinterpret_cast<float4 *>(c + j) = ld_input(reinterpret_cast<const float4 *>(row + j));
      *reinterpret_cast<float4 *>(s + j) = ld_input(reinterpret_cast<const float4 *>(row + half + j));
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float *row = p.table + (int64_t)rows.of((axes >> (2 * j)) & 3) * p.rot + pair + j;
      c[j] = ld_input(row);
      s[j] = ld_input(row + half);
    }
  }
}
template <bool HALF>
__device__ __forceinline__ void load_angles(const HeadParams &p, const Rows &rows, const Pieces &l, float (&c)[8],
                                            float (&s)[8]) {
  if constexpr (HALF) {
    if (l.turns[0]) load_angles<8>(p, rows, l.pair[0], c, s);
  } else {
    if (l.turns[0]) load_angles<4>(p, rows, l.pair[0], c, s);
    if (l.turns[1]) load_angles<4>(p, rows, l.pair[1], c + 4, s + 4);
  }
}
// The same on their way to shared memory: two chunks of cosines, two of sines, 512 bytes apart.
template <int BYTES>
__device__ __forceinline__ void copy_bytes(const void *to, const void *from);
template <int N>
__device__ __forceinline__ void copy_angles(const HeadParams &p, const Rows &rows, int pair, uint8_t *to) {
  const int half = p.rot / 2;
  const uint32_t axes = axes_of<N>(p, pair);
  if (same_axis<N>(axes)) {
    const float *row = p.table + (int64_t)rows.of(axes & 3) * p.rot + pair;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      copy_bytes<16>(to + j / 4 * 512, row + j);
      copy_bytes<16>(to + 1024 + j / 4 * 512, row + half + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float *row = p.table + (int64_t)rows.of((axes >> (2 * j)) & 3) * p.rot + pair + j;
      copy_bytes<4>(to + j / 4 * 512 + j % 4 * 4, row);
      copy_bytes<4>(to + 1024 + j / 4 * 512 + j % 4 * 4, row + half);
    }
  }
}
template <bool HALF>
__device__ __forceinline__ void copy_angles(const HeadParams &p, const Rows &rows, const Pieces &l, uint8_t *to) {
  if constexpr (HALF) {
    if (l.turns[0]) copy_angles<8>(p, rows, l.pair[0], to);
  } else {
    if (l.turns[0]) copy_angles<4>(p, rows, l.pair[0], to);
    if (l.turns[1]) copy_angles<4>(p, rows, l.pair[1], to + 512);
  }
}

// Reciprocal root mean square of the head whose N words (BF16 pairs) each of its `width`
// lanes holds; all 32 lanes take part.
template <int N, int width>
__device__ __forceinline__ float head_rms(const HeadParams &p, const uint32_t *x, int lane) {
  // four chains, the first square of each as it is
  static_assert(N % 2 == 0, "two packed sums");
  TwoFloat2 S2[2] = {{f32x2_mul(f32x2_of(x[0]), f32x2_of(x[0])), 0}, {f32x2_mul(f32x2_of(x[1]), f32x2_of(x[1])), 0}};
#pragma unroll
  for (int j = 2; j < N; ++j) add_values(S2[j % 2], f32x2_mul(f32x2_of(x[j]), f32x2_of(x[j])));
  TwoFloat S{f32x2_lo(S2[0].hi), f32x2_lo(S2[0].lo)}, Z{f32x2_lo(S2[1].hi), f32x2_lo(S2[1].lo)};
  add_pair(S, TwoFloat{f32x2_hi(S2[0].hi), f32x2_hi(S2[0].lo)});
  add_pair(Z, TwoFloat{f32x2_hi(S2[1].hi), f32x2_hi(S2[1].lo)});
  add_pair(S, Z);
#pragma unroll
  for (int o = width / 2; o > 0; o >>= 1)
    add_pair(S, TwoFloat{__shfl_xor_sync(~0u, S.hi, o), __shfl_xor_sync(~0u, S.lo, o)});
  if (__builtin_expect(!(S.hi >= 0x1p-80f && S.hi < 0x1p126f) && !(S.hi == 0.0f && p.eps >= 0x1p-80f), 0)) {
    // squares beyond binary32: the same sum in FP64, by the lanes of this head.  (Zeros come from lanes
    // without a head, too; there r is that of eps alone.)
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j)
      d += (double)lo_f(x[j]) * (double)lo_f(x[j]) + (double)hi_f(x[j]) * (double)hi_f(x[j]);
    const unsigned mask = width == 32 ? ~0u : ((1u << (width % 32)) - 1) << (lane & ~(width - 1));
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) d += __shfl_xor_sync(mask, d, o);
    return (float)(1.0 / sqrt(d * p.inv_d64 + p.eps64));
  }
  return rms_reciprocal(S, p.inv_d, p.eps);
}

// Reciprocal root mean square of a query head, within 2^-20.4 (the sum's and the quotient's roundings, fourteen of 2^-24 at
// most, halved by the root, and two ulp of rsqrtf): one packed operation for each pair, against eight above.  `wild`: the
// sum of squares is beyond what binary32 holds so well, or below where eps does not hide it.
template <int width>
__device__ __forceinline__ float head_rms_fast(const HeadParams &p, const uint32_t (&x)[8], bool &wild) {
  uint64_t S2[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) S2[j % 2] = f32x2_fma(f32x2_of(x[j]), f32x2_of(x[j]), S2[j % 2]);
  float S = (f32x2_lo(S2[0]) + f32x2_hi(S2[0])) + (f32x2_lo(S2[1]) + f32x2_hi(S2[1]));
#pragma unroll
  for (int o = width / 2; o > 0; o >>= 1) S += __shfl_xor_sync(~0u, S, o);
  wild = !(S >= p.least && S < 0x1p126f);
  return rsqrtf(fmaf(S, p.inv_d.hi, p.eps));
}

// A warp's ring of rows on their way, by asynchronous copies.  A stage is chunks of 16 bytes a lane, each lane's its own,
// so that nothing but its own wait comes between a copy and its use.
template <int BYTES>
__device__ __forceinline__ void copy_bytes(const void *to, const void *from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void end_stage() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_stages() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two of a lane's chunks.
__device__ __forceinline__ void get_chunks(const uint8_t *from, uint32_t (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(from), b = *reinterpret_cast<const uint4 *>(from + 512);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The heads of a warp, token t's for this lane, by the binary32 steps as they are written, from a stage of the ring into dst
// where `store` is set.  For queries that the fused operations do not hold: rare, so apart, with loads of its own.
template <int width, bool HALF>
__device__ __noinline__ void exact_heads(const HeadParams &p, const uint8_t *stage, const uint16_t *w, int64_t t, uint16_t *dst,
                                         bool store, unsigned *status) {
  const int lane = threadIdx.x & 31;
  const Pieces own = pieces_of<HALF>(p, lane % width, p.per);
  uint32_t x[8], o[8];
  get_chunks(stage, x);
  const float r = head_rms<8, width>(p, x, lane);
  if (!store) return;
  Rows rows;
  token_rows(p, t, rows, status);
  float c[8], s[8], y[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
  load_angles<HALF>(p, rows, own, c, s);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float v = j & 1 ? hi_f(x[j / 2]) : lo_f(x[j / 2]);
    y[j] = __fmul_rn(__fmul_rn(v, r), __uint_as_float((uint32_t)ld_input(w + own.d0 + (j < 8 ? j : own.piece + j - 8)) << 16));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = HALF ? j : 2 * j, k = HALF ? 8 + j : 2 * j + 1;
    if (!own.turns[HALF ? 0 : j / 4]) continue;
    const float a = y[i], b = y[k];
    y[i] = turn_a(a, b, c[j], s[j]), y[k] = turn_b(a, b, c[j], s[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = pack_bf16(y[2 * j], y[2 * j + 1]);
  *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4 *>(dst + own.piece) = make_uint4(o[4], o[5], o[6], o[7]);
}

constexpr int kDepth = 4, kRingBytes = kDepth * 1024;  // the stages of norm_rotate, a head of each lane in one
// Batches [u, end) of the heads of one kind: in -> out with weight w (or null).  A head is `width` lanes, of 16
// dimensions each (Pieces).  FAST (with a weight): the weights' products with cosines and sines are
// made once for a token, and the rest is fused; otherwise every step is rounded by itself.
template <bool FAST, int width, bool HALF>
__device__ __forceinline__ void norm_rotate(const HeadParams &p, const HeadParams::Units &units, int64_t u, int64_t end,
                                            const uint16_t *in, int64_t ld, uint16_t *out, int64_t ldo,
                                            const uint16_t *w, uint8_t *ring, int lane, unsigned *status) {
  if (u >= end) return;
  const int item = lane % width, group = lane / width;
  const int at_once = 32 / width / units.tokens;  // heads of each token: first, first + at_once, ...
  const int first = group % at_once;
  const bool has = item < p.per;
  const Pieces own = pieces_of<HALF>(p, item, p.per);
  const int d0 = own.d0, piece = own.piece;
  const int step = at_once * p.D, count = (int)(end - u);
  int64_t t = u / units.batches;
  int batch = (int)(u - t * units.batches);
  t = t * units.tokens + group / at_once;
  const int64_t at = (int64_t)(batch * at_once + first) * p.D + d0;
  uint16_t *dst = out + t * ldo + at;
  // what is copied next
  const uint16_t *src = in + t * ld + at;
  const int64_t src_token = units.tokens * ld - (int64_t)(units.batches - 1) * step;
  const int64_t dst_token = units.tokens * ldo - (int64_t)(units.batches - 1) * step;
  int64_t src_t = t;
  int src_batch = batch;
  const auto copy = [&](int k) {
    if (k < count) {
      if (has && src_t < p.T && src_batch * at_once + first < units.heads) {
        copy_bytes<16>(ring + k % kDepth * 1024, src);
        copy_bytes<16>(ring + k % kDepth * 1024 + 512, src + piece);
      }
      if (++src_batch == units.batches) {
        src_batch = 0;
        src_t += units.tokens;
        src += src_token;
      } else {
        src += step;
      }
    }
    end_stage();
  };
  if (!has) {  // lanes without dimensions add nothing to a head's sum
    for (int k = 0; k < kDepth; ++k) {
      uint4 *x = reinterpret_cast<uint4 *>(ring + k * 1024);
      x[0] = x[32] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll 1
  for (int k = 0; k < kDepth - 1; ++k) copy(k);
  // What the pieces a and b are multiplied by.  FAST: for the pair's first and second element, with the weights
  uint64_t ca[4], sb[4], cb[4], sa[4];
  float c[8], s[8];  // otherwise the angles
  uint32_t wb[8];    // and the weights
  bool stored;       // the token takes part
  const auto token = [&] {
    Rows rows;
    stored = has && t < p.T && token_rows(p, t, rows, status);
#pragma unroll
    for (int j = 0; j < 8; ++j) wb[j] = 0u;
    if (has && w) {
      const uint4 a = ld_input(reinterpret_cast<const uint4 *>(w + d0));
      const uint4 b = ld_input(reinterpret_cast<const uint4 *>(w + d0 + piece));
      wb[0] = a.x, wb[1] = a.y, wb[2] = a.z, wb[3] = a.w, wb[4] = b.x, wb[5] = b.y, wb[6] = b.z, wb[7] = b.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    if (stored) load_angles<HALF>(p, rows, own, c, s);
    if constexpr (FAST) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (HALF) {
          const uint64_t wa = f32x2_of(wb[j]), wz = f32x2_of(wb[4 + j]);
          const uint64_t c2 = f32x2_pack(c[2 * j], c[2 * j + 1]), s2 = f32x2_pack(s[2 * j], s[2 * j + 1]);
          ca[j] = f32x2_mul(wa, c2), sa[j] = f32x2_mul(wa, s2);
          cb[j] = f32x2_mul(wz, c2), sb[j] = f32x2_mul(wz, f32x2_pack(-s[2 * j], -s[2 * j + 1]));
        } else {  // pairs 2j and 2j + 1: (w_a cos, w_b cos), (-w_b sin, w_a sin)
          const uint64_t w0 = f32x2_of(wb[2 * j]), w1 = f32x2_of(wb[2 * j + 1]);
          const float c0 = c[2 * j], s0 = s[2 * j], c1 = c[2 * j + 1], s1 = s[2 * j + 1];
          ca[j] = f32x2_mul(w0, f32x2_pack(c0, c0)), cb[j] = f32x2_mul(w1, f32x2_pack(c1, c1));
          sa[j] = f32x2_pack(-s0 * f32x2_hi(w0), s0 * f32x2_lo(w0));
          sb[j] = f32x2_pack(-s1 * f32x2_hi(w1), s1 * f32x2_lo(w1));
        }
      }
    }
  };
  token();
  for (int k = 0; k < count; ++k) {
    wait_stages<kDepth - 2>();
    uint32_t x[8];
    get_chunks(ring + k % kDepth * 1024, x);
    copy(k + kDepth - 1);
    float r = 0.0f;
    bool wild = false;
    if (FAST) r = head_rms_fast<width>(p, x, wild);
    else if (w) r = head_rms<8, width>(p, x, lane);
    const uint64_t r2 = f32x2_pack(r, r);
    uint64_t y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = f32x2_of(x[j]);
      if (FAST || w) y[j] = f32x2_mul(y[j], r2);
      if (!FAST && w) y[j] = f32x2_mul(y[j], f32x2_of(wb[j]));
    }
    if (FAST || own.turns[0]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (HALF) {
          const uint64_t a = y[j], b = y[4 + j];
          if constexpr (FAST) {
            y[j] = f32x2_fma(a, ca[j], f32x2_mul(b, sb[j]));
            y[4 + j] = f32x2_fma(b, cb[j], f32x2_mul(a, sa[j]));
          } else {
            const uint64_t c2 = f32x2_pack(c[2 * j], c[2 * j + 1]), s2 = f32x2_pack(s[2 * j], s[2 * j + 1]);
            y[j] = difference_of(p, f32x2_mul(a, c2), f32x2_mul(b, s2));
            y[4 + j] = sum_of(p, f32x2_mul(b, c2), f32x2_mul(a, s2));
          }
        } else {
#pragma unroll
          for (int n = 2 * j; n < 2 * j + 2; ++n) {
            const float a = f32x2_lo(y[n]), b = f32x2_hi(y[n]);
            if constexpr (FAST)  // (by 1 and 0 where nothing turns)
              y[n] = f32x2_fma(y[n], n & 1 ? cb[j] : ca[j], f32x2_mul(f32x2_pack(b, a), n & 1 ? sb[j] : sa[j]));
            else if (own.turns[j / 2])
              y[n] = f32x2_pack(turn_a(a, b, c[n], s[n]), turn_b(a, b, c[n], s[n]));
          }
        }
      }
    }
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = bf16x2_of(y[j]);
    const bool here = stored && batch * at_once + first < units.heads;
    if (here) {
      *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4 *>(dst + piece) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (FAST && __builtin_expect(__any_sync(~0u, wild && here), 0))
      exact_heads<width, HALF>(p, ring + k % kDepth * 1024, w, t, dst, wild && here, status);
    if (++batch == units.batches) {
      batch = 0;
      t += units.tokens;
      dst += dst_token;
      if (k + 1 < count) token();
    } else {
      dst += step;
    }
  }
  wait_stages<0>();
}

// Part `i` of `n` of the units 0 ... count - 1: equal runs of consecutive ones.
struct Run {
  int64_t begin, end;
};
__device__ __forceinline__ Run run_of(int64_t count, int64_t i, int64_t n) {
  const int64_t each = count / n, longer = count - each * n;
  return {i * each + min(i, longer), (i + 1) * each + min(i + 1, longer)};
}

// Which of the grid's warps work on queries and which on the keys (or the store), in turn all over the GPU: the
// latter compute more, and the former wait for memory meanwhile.  Each has its part of its kind's units.
struct Share {
  bool keys;
  Run run;
};
__device__ __forceinline__ Share share_of(const HeadParams &p, int warp) {
  const int64_t n = (int64_t)gridDim.x * kWarps, i = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t before = i * p.key_warps / n, after = (i + 1) * p.key_warps / n;
  if (after != before) return {true, run_of(p.uk.count, before, p.key_warps)};
  return {false, run_of(p.uq.count, i - before, n - p.key_warps)};
}

template <int width, bool HALF>
__device__ __forceinline__ void norm_rotate_queries(const HeadParams &p, Run run, uint8_t *ring, int lane,
                                                    unsigned *status) {
  if (p.qw) norm_rotate<true, width, HALF>(p, p.uq, run.begin, run.end, p.q, p.ldq, p.q_out, p.ldqo, p.qw, ring, lane, status);
  else norm_rotate<false, width, HALF>(p, p.uq, run.begin, run.end, p.q, p.ldq, p.q_out, p.ldqo, nullptr, ring, lane, status);
}
// What the store has beside the heads.
struct StoreParams {
  const uint16_t *v;
  int64_t ldv;
  const int64_t *slots;
  Int4Cache cache;
};

// Items [run.begin, run.end): each as many (token, kv head) pairs as a warp has lanes for, `width` = D/16 to a pair.  A
// lane has 16 dimensions of the key, in the two pieces that a turn takes, and 16 consecutive ones of the value: two
// octets each, so two words of codes.  The maxima of a key's octets meet in shared memory, where those of a
// 32-dimension group are read together whichever lanes have them.  An item is one long chain of dependent operations,
// so all that the next one loads, its angles and slot too, is copied meanwhile (its positions are known by then).
constexpr int kStoreStages = 2, kStoreBytes = kStoreStages * (4096 + 384);
template <int width, bool HALF>
__device__ __forceinline__ void store_items(const HeadParams &p, const StoreParams &s, Run run, uint8_t *warp_ring,
                                            uint16_t *s_max, int lane, unsigned *status) {
  if (run.begin >= run.end) return;
  constexpr int D = 16 * width, kGroups = D / 32, kAtOnce = 32 / width, kStages = kStoreStages;
  const int H = s.cache.H, item = lane % width, group = lane / width;
  const Pieces own = pieces_of<HALF>(p, item, width);
  const int d0 = own.d0, piece = own.piece;
  const int oa = d0 / 8, ob = (d0 + piece) / 8;  // the key's octets
  uint16_t *const maxima = s_max + group * (D / 8);
  const int count = (int)(run.end - run.begin);
  // stages: key, value, cosines, sines (two chunks each); then the pair's slot (-1: none) and its head
  uint8_t *const ring = warp_ring + lane * 16;
  int64_t *const slots = reinterpret_cast<int64_t *>(warp_ring + kStages * 4096) + lane;
  int *const heads = reinterpret_cast<int *>(warp_ring + kStages * (4096 + 256)) + lane;
  // the pair that is copied next, and the step to the lane's pair of the next item
  const int64_t pair = run.begin * kAtOnce + group;
  const int64_t t0 = pair >> 32 ? pair / H : (int64_t)((uint32_t)pair / (uint32_t)H);
  int64_t t = t0;
  int h = (int)(pair - t0 * H);
  const int dt = kAtOnce / H, dh = kAtOnce - dt * H;
  int64_t pos[4] = {0, 0, 0, 0};  // its positions
  const auto positions = [&] {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (a < p.axes && t < p.T) pos[a] = ld_input(p.positions + a * p.T + t);
  };
  const auto copy = [&](int k) {
    const int stage = k % kStages;
    uint8_t *to = ring + stage * 4096;
    bool ok = false;
    if (k < count) {
      if (t < p.T) {
        Rows rows;
        ok = rows_of(p, pos, rows, status);
        const uint16_t *x = p.k + t * p.ldk + h * D + d0, *v = s.v + t * s.ldv + h * D + item * 16;
        copy_bytes<16>(to, x);
        copy_bytes<16>(to + 512, x + piece);
        copy_bytes<16>(to + 1024, v);
        copy_bytes<16>(to + 1536, v + 8);
        if (ok) {
          copy_angles<HALF>(p, rows, own, to + 2048);
          copy_bytes<8>(slots + stage * 32, s.slots + t);
        }
        heads[stage * 32] = h;
      }
      t += dt;
      h += dh;
      if (h >= H) h -= H, ++t;
      if (k + 1 < count) positions();
    }
    if (!ok) slots[stage * 32] = -1;
    end_stage();
  };
  uint32_t wb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wb[j] = 0u;
  if (p.kw) {
    const uint4 a = ld_input(reinterpret_cast<const uint4 *>(p.kw + d0));
    const uint4 b = ld_input(reinterpret_cast<const uint4 *>(p.kw + d0 + piece));
    wb[0] = a.x, wb[1] = a.y, wb[2] = a.z, wb[3] = a.w, wb[4] = b.x, wb[5] = b.y, wb[6] = b.z, wb[7] = b.w;
  }
  // Largest magnitude of a piece, by its bits; NaN the largest, or (`numbers`) not counted.
  const auto most = [](const uint32_t *x, bool numbers) {
    if (!numbers) return largest_bits<4>(x);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(lo_f(x[j])), fabsf(hi_f(x[j]))));
    return __float_as_uint(m) >> 16;
  };
  const auto plain = [](uint32_t bits) { return bits >= kPlainFrom && bits <= kPlainTo; };
  positions();
  copy(0);
  for (int k = 0; k < count; ++k) {
    const uint8_t *at = ring + k % kStages * 4096;
    wait_stages<0>();
    copy(k + 1);
    uint32_t x[8], v[8], cs[16];
    get_chunks(at, x);
    get_chunks(at + 2 * 512, v);
    get_chunks(at + 4 * 512, *reinterpret_cast<uint32_t(*)[8]>(cs));
    get_chunks(at + 6 * 512, *reinterpret_cast<uint32_t(*)[8]>(cs + 8));
    const int64_t slot = slots[k % kStages * 32];
    if (slot >= s.cache.num_slots) set_status(status, QLIN_ERR_INVALID_ARG);
    const bool stored = slot >= 0 && slot < s.cache.num_slots;
    const auto cosine = [&](int j) { return __uint_as_float(cs[j]); };
    const auto sine = [&](int j) { return __uint_as_float(cs[8 + j]); };

    // The value's scale and codes, as if its group were within the plain quantizer's range; beside the key's chain.
    uint32_t vm = max(largest_bits<4>(v), largest_bits<4>(v + 4));
    vm = max(vm, __shfl_xor_sync(~0u, vm, 1));
    uint16_t sv = scale4(__uint_as_float(vm << 16));
    uint32_t qv[2];
    int4_codes<8, true>(v, make_scale(half_bits_to_f32(sv)), qv);

    // the key, as the BF16 output of the norm and the rotation
    float r = 0.0f;
    if (p.kw) r = head_rms<8, width>(p, x, lane);
    uint64_t y[8];
    const uint64_t r2 = f32x2_pack(r, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = f32x2_of(x[j]);
      if (p.kw) y[j] = f32x2_mul(f32x2_mul(y[j], r2), f32x2_of(wb[j]));
    }
    if (own.turns[0]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (HALF) {
          const uint64_t c2 = f32x2_pack(cosine(2 * j), cosine(2 * j + 1)), s2 = f32x2_pack(sine(2 * j), sine(2 * j + 1));
          const uint64_t a = y[j], b = y[4 + j];
          y[j] = difference_of(p, f32x2_mul(a, c2), f32x2_mul(b, s2));
          y[4 + j] = sum_of(p, f32x2_mul(b, c2), f32x2_mul(a, s2));
        } else {
#pragma unroll
          for (int n = 2 * j; n < 2 * j + 2; ++n) {
            const float a = f32x2_lo(y[n]), b = f32x2_hi(y[n]);
            if (own.turns[j / 2]) y[n] = f32x2_pack(turn_a(a, b, cosine(n), sine(n)), turn_b(a, b, cosine(n), sine(n)));
          }
        }
      }
    }
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = bf16x2_of(y[j]);
    uint32_t ka, kb;  // largest bits of the groups of the key's two octets
    const auto groups = [&](bool numbers) {
      __syncwarp();
      maxima[oa] = (uint16_t)most(o, numbers);
      maxima[ob] = (uint16_t)most(o + 4, numbers);
      __syncwarp();
      const auto of_four = [&](int octet) {
        const uint2 w = *reinterpret_cast<const uint2 *>(maxima + (octet & ~3));
        const uint32_t m = __vmaxu2(w.x, w.y);
        return max(m & 0xFFFFu, m >> 16);
      };
      ka = of_four(oa), kb = of_four(ob);
    };
    groups(false);
    uint16_t sa = scale4(__uint_as_float(ka << 16)), sb = scale4(__uint_as_float(kb << 16));
    uint32_t qa[1], qb[1];
    int4_codes<4, true>(o, make_scale(half_bits_to_f32(sa)), qa);
    int4_codes<4, true>(o + 4, make_scale(half_bits_to_f32(sb)), qb);
    if (!__all_sync(~0u, !stored || (plain(ka) && plain(kb) && plain(vm)))) {
      // small, huge or not finite somewhere; a NaN counts for nothing in the maximum
      groups(true);
      vm = max(most(v, true), most(v + 4, true));
      vm = max(vm, __shfl_xor_sync(~0u, vm, 1));
      sa = scale4(__uint_as_float(ka << 16)), sb = scale4(__uint_as_float(kb << 16));
      sv = scale4(__uint_as_float(vm << 16));
      int4_codes<4, false>(o, make_scale(half_bits_to_f32(sa)), qa);
      int4_codes<4, false>(o + 4, make_scale(half_bits_to_f32(sb)), qb);
      int4_codes<8, false>(v, make_scale(half_bits_to_f32(sv)), qv);
    }
    if (stored) {
      const int64_t row = s.cache.row(slot, heads[k % kStages * 32]);
      uint32_t *kc = reinterpret_cast<uint32_t *>(s.cache.kc + row * (D / 2));
      kc[oa % 4 * kGroups + oa / 4] = qa[0];
      kc[ob % 4 * kGroups + ob / 4] = qb[0];
      store_words<2>(s.cache.vc + row * (D / 2) + item * 8, qv);
      if (oa % 4 == 0) s.cache.ks[row * kGroups + oa / 4] = sa;
      if (ob % 4 == 0) s.cache.ks[row * kGroups + ob / 4] = sb;
      if (item % 2 == 0) s.cache.vs[row * kGroups + item / 2] = sv;
    }
  }
  wait_stages<0>();
}

template <int width, bool HALF>
__global__ void __launch_bounds__(32 * kWarps, kCtas) k_qk_norm_rope(const __grid_constant__ HeadParams p, unsigned *status) {
  __shared__ __align__(16) uint8_t s_ring[kWarps][kRingBytes];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t *const ring = s_ring[warp] + lane * 16;
  const Share share = share_of(p, warp);
  if (share.keys)
    norm_rotate<false, width, HALF>(p, p.uk, share.run.begin, share.run.end, p.k, p.ldk, p.k_out, p.ldko, p.kw, ring, lane, status);
  else
    norm_rotate_queries<width, HALF>(p, share.run, ring, lane, status);
}

template <int width, bool HALF>
__global__ void __launch_bounds__(32 * kWarps, kCtas)
    k_qk_norm_rope_kv4(const __grid_constant__ HeadParams p, const __grid_constant__ StoreParams s, unsigned *status) {
  __shared__ __align__(16) uint8_t s_ring[kWarps][kStoreBytes > kRingBytes ? kStoreBytes : kRingBytes];
  __shared__ __align__(8) uint16_t s_max[kWarps][64];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Share share = share_of(p, warp);
  if (share.keys) store_items<width, HALF>(p, s, share.run, s_ring[warp], s_max[warp], lane, status);
  else norm_rotate_queries<width, HALF>(p, share.run, s_ring[warp] + lane * 16, lane, status);
}

// Batches of as many heads as a warp has at once; of few heads, those of several tokens, where there are tokens enough.
HeadParams::Units head_units(int64_t T, int heads, int at_once, int sms) {
  HeadParams::Units u{heads, 1, 1, 0};
  if (heads == 0) return u;
  while (at_once % (2 * u.tokens) == 0 && heads * 2 * u.tokens <= at_once && T >= (int64_t)sms * 32 * 2 * u.tokens)
    u.tokens *= 2;
  u.batches = (heads * u.tokens + at_once - 1) / at_once;
  u.count = (T + u.tokens - 1) / u.tokens * u.batches;
  return u;
}
HeadParams head_params(const HeadArgs &a, int key_heads, int sms) {
  HeadParams p{};
  p.table = a.table, p.positions = a.positions, p.max_pos = a.max_pos;
  p.q = (const uint16_t *)a.q, p.k = (const uint16_t *)a.k;
  p.qw = (const uint16_t *)a.q_weight, p.kw = (const uint16_t *)a.k_weight;
  p.q_out = (uint16_t *)a.q_out, p.k_out = (uint16_t *)a.k_out;
  p.T = a.T, p.ldq = a.ldq, p.ldk = a.ldk, p.ldqo = a.ldqo, p.ldko = a.ldko;
  p.Hq = (int)a.Hq, p.Hk = key_heads, p.D = (int)a.D, p.rot = (int)a.rot;
  p.half_layout = a.layout == QLIN_ROPE_HALF;
  p.axes = a.rot > 0 ? (int)a.axes : 0;
  for (int i = 0; a.pair_axis && i < p.rot / 2; ++i) p.axis[i / 16] |= (uint32_t)a.pair_axis[i] << (2 * (i % 16));
  p.one = 1.0f;
  p.eps = a.eps, p.eps64 = (double)a.eps, p.inv_d64 = 1.0 / (double)a.D;
  p.least = a.eps >= 0x1p-80f ? 0.0f : 0x1p-80f;
  p.inv_d.hi = (float)p.inv_d64;
  p.inv_d.lo = (float)(p.inv_d64 - (double)p.inv_d.hi);
  p.per = p.D / 16;
  p.width = 1;
  while (p.width < p.per) p.width *= 2;
  p.uq = head_units(p.T, p.Hq, 32 / p.width, sms);
  p.uk = head_units(p.T, p.Hk, 32 / p.width, sms);
  return p;
}

// Times of a warp, in those of a batch of query heads: of a batch of keys, of a token's angles (which each token's batches
// share, and wait for), of an item of the store.  Best for 8192 tokens of 28 + 4 heads of 128: keys' units at 2.4 times the
// queries' 25.7 us (2: 26.9, 2.8: 26.0), the store's at 3.4 29.6 us (3: 31.1, 4: 31.0); but for 16000 of 6 + 6, where
// both kinds have two batches to a token, at 1 32 us (2.4: 43; these times 36).
constexpr double kKeyTime = 1.2, kTokenTime = 1.8, kStoreTime = 4.3;
// A warp for each unit of the queries and of the keys (or the store), or as many as are resident, with a share for the
// keys, a unit of which takes `key_time`.
unsigned share_warps(HeadParams &p, double key_time, int sms) {
  const int64_t queries = p.uq.count, keys = p.uk.count;
  const int64_t need = (queries + keys + kWarps - 1) / kWarps, ctas = std::min<int64_t>(need, (int64_t)sms * kCtas);
  const int64_t n = ctas * kWarps;
  p.key_warps = keys;
  if (need > ctas) {
    const double work = key_time * (double)keys, others = (1.0 + kTokenTime / p.uq.batches) * (double)queries;
    const double share = work / (work + others);
    p.key_warps = std::min<int64_t>(n, (int64_t)(share * (double)n + 0.5));
    if (keys > 0) p.key_warps = std::max<int64_t>(p.key_warps, 1);
    if (queries > 0) p.key_warps = std::min<int64_t>(p.key_warps, n - 1);
  }
  return (unsigned)ctas;
}

template <int width>
cudaError_t launch_norm_rope(const HeadParams &p, unsigned ctas, unsigned *status, cudaStream_t st) {
  return launch_kernel(p.half_layout ? k_qk_norm_rope<width, true> : k_qk_norm_rope<width, false>, dim3(ctas),
                       dim3(32 * kWarps), 0, st, 1, p, status);
}
template <int width>
cudaError_t launch_store(HeadParams p, const StoreParams &s, unsigned *status, int sms, cudaStream_t st) {
  constexpr int kAtOnce = 32 / width;
  p.uk.count = (p.T * s.cache.H + kAtOnce - 1) / kAtOnce;
  const unsigned ctas = share_warps(p, kStoreTime, sms);
  return launch_kernel(p.half_layout ? k_qk_norm_rope_kv4<width, true> : k_qk_norm_rope_kv4<width, false>, dim3(ctas),
                       dim3(32 * kWarps), 0, st, 1, p, s, status);
}

}  // namespace

int block_shift_of(int64_t block_size) {
  for (int s = 0; s < 31; ++s)
    if (block_size == (int64_t)1 << s) return s;
  return -1;
}

cudaError_t launch_qk_norm_rope(const HeadArgs &a, unsigned *status, int sms, cudaStream_t st) {
  HeadParams p = head_params(a, (int)a.Hk, sms);
  const unsigned ctas = share_warps(p, kKeyTime + kTokenTime / p.uk.batches, sms);
  switch (p.width) {
    case 1: return launch_norm_rope<1>(p, ctas, status, st);
    case 2: return launch_norm_rope<2>(p, ctas, status, st);
    case 4: return launch_norm_rope<4>(p, ctas, status, st);
    case 8: return launch_norm_rope<8>(p, ctas, status, st);
    case 16: return launch_norm_rope<16>(p, ctas, status, st);
    case 32: return launch_norm_rope<32>(p, ctas, status, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_qk_norm_rope_kv4(const HeadArgs &a, const KvArgs &kv, int64_t block_size, unsigned *status, int sms,
                                    cudaStream_t st) {
  const HeadParams p = head_params(a, (int)kv.H, sms);
  StoreParams s{};
  s.v = (const uint16_t *)kv.v, s.ldv = kv.ldv, s.slots = kv.slots;
  s.cache.kc = (uint8_t *)kv.k_cache, s.cache.ks = (uint16_t *)kv.k_scale;
  s.cache.vc = (uint8_t *)kv.v_cache, s.cache.vs = (uint16_t *)kv.v_scale;
  s.cache.num_slots = kv.num_slots, s.cache.H = (int)kv.H, s.cache.block_size = (int)block_size;
  s.cache.block_shift = block_shift_of(block_size);
  switch (a.D) {
    case 32: return launch_store<2>(p, s, status, sms, st);
    case 64: return launch_store<4>(p, s, status, sms, st);
    case 128: return launch_store<8>(p, s, status, sms, st);
    case 256: return launch_store<16>(p, s, status, sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
