// Attention over the mixed 8-bit KV cache for few rows: decode, and short runs
// of new tokens.  Bound by HBM: a (token, kv head) is 2D codes, D/16 bytes of key
// scales and 2 of value scale, read once for all of the head's rows.
//
// Rows and positions.  The rows of a sequence that read one kv head (its new
// tokens times the Hq/H query heads of the group) are tiled by 8*NT.  Each CTA
// takes one row tile and one part of the positions; its four warps take 32 (D
// 256: 16) positions at a time, each with a ring of its own in shared memory that
// it fills with 16-byte cp.async, so nothing but the end of the part makes warps
// wait for one another.
//
// Arithmetic.  Scores and outputs are transposed, S^T = K q^T and O^T = V^T P^T,
// so that positions (then head dimensions) fill the 16 rows of
// mma.m16n8k16 and the 8 query heads its columns: with the usual orientation
// the heads of one group would leave half of the 16 rows empty.  tcgen05 would
// want 128 rows of one operand staged in shared memory as 16-bit values; here
// codes go from the ring to registers once and the tensor pipe is far from its
// limit.  Codes become float16 exactly: INT8 as 1152 + code by a byte permute (the
// sums start at -1152 times the sum of q, in fp32, which takes the offset out
// again), E4M3 by conversion; q is scaled by a power of two per row to
// use float16's whole range; the products of one 32-dimension key group are
// summed in fp32 and then scaled by the group's scale in fp32.  P is multiplied
// by the value scales in fp32 and rounded once to float16.  The scales of a tile share
// a power of two, taken from that tile, under which P of a score at the maximum lies
// between 1 and 2^15.  Where they lie too far apart for that (a position that few rows
// see, or that has no weight, can have any scale) or one is zero, the part is done
// again in a general form: each position's exponent joins its score, and O has a
// reference of its own for each row.  P^T as the second operand needs P's fragments
// transposed: two movmatrix per 16 positions.
//
// What bounds it beside HBM is the instructions of the conversions, so positions
// of whole pages take their addresses from one table entry and one multiplication
// per 32, and the maxima of 32 positions are reduced at once.
#include <algorithm>

#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv_quant.cuh"
#include "tc_ptx.cuh"

namespace qlin {

namespace {

constexpr int kAttnWarps = 4;
constexpr int kSpan = 14;    // exponents of the value scales of a tile: this far apart they share a window
constexpr unsigned kWindow = (kSpan + 1u) << 23, kNoWindow = 0xFF000000u;
constexpr float kWideBias = 14.0f;  // in the general form P of the maximum lies between 2^14 and 2^15
constexpr int kAlign = 32;   // parts begin at multiples of this: the most positions a warp handles at once

struct SplitParams : AttnDev {
  unsigned group_inverse;  // 2^16 / G rounded up: (x * it) >> 16 is x / G for x < 256 (G <= 128)
  AttnParts parts;
  int64_t chunk;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 0 : 16) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with sums that start at (c0, c1) in both rows.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                             float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// Exponent e of a value scale, 2^e <= |s| < 2^(e+1), from its bits (0, and what is not finite: the ends of float16).
__device__ __forceinline__ int scale_exponent(unsigned abs_bits) {
  return min(max((int)(abs_bits >> 23) - 127, -24), 15);
}
// base + i * step (one instruction).
__device__ __forceinline__ const uint8_t *step_from(const uint8_t *base, uint32_t step, uint32_t i) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(step), "r"(i), "l"(reinterpret_cast<uint64_t>(base)));
  return reinterpret_cast<const uint8_t *>(r);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// N consecutive floats of shared memory (aligned to 4 min(N, 4) bytes).
template <int N>
__device__ __forceinline__ void load_shared(float (&v)[N], const float *p) {
  if constexpr (N == 1) {
    v[0] = *p;
  } else if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(p + i);
      v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
  }
}

template <int D, int NT>
struct Geometry {
  static constexpr int kTile = D >= 256 ? 16 : 32;  // positions a warp handles at once
  static constexpr int kRows = 8 * NT;
  static constexpr int kGroups = D / 32;
  static constexpr int kChunks = D / 16;               // 16-byte pieces of a row of codes
  static constexpr int kPieces = kTile * kChunks / 32;  // pieces a lane copies
  static constexpr int kRowStep = 32 / kChunks;         // rows the warp copies at once
  static constexpr int kCodes = kTile * D;
  static constexpr int kStages = D >= 128 ? 2 : 3;  // tiles in a warp's ring
  // one stage: key codes, value codes, key scales, value scales, {valid, window that its value scales fit}
  static constexpr int kScaleAt = 2 * kCodes;
  static constexpr int kVScaleAt = kScaleAt + kTile * kGroups * 4;
  static constexpr int kInfoAt = kVScaleAt + kTile * 4;
  static constexpr int kStageBytes = kInfoAt + 16;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kJoinFloats = kRows * D + 4 * kRows + 4;  // a warp's result: O, m, l, window or references of O
  static constexpr int kWarpBytes = kRingBytes > kJoinFloats * 4 ? kRingBytes : kJoinFloats * 4;
  static constexpr int kSmem = kAttnWarps * kWarpBytes;
  static constexpr int kCtas = D >= 256 || NT > 1 ? 2 : 3;  // resident CTAs the registers are budgeted for
};

// Key rows are read 32 bytes (a group) at a time by four lanes, four rows of a
// half-warp at once: groups are rotated by the row so that those four rows sit in
// different banks.  Value rows are read D/8 bytes a lane, rows 2t by the lanes t:
// their 16-byte pieces are exchanged by bits of the row.
template <int D>
__device__ __forceinline__ int key_chunk(int row, int c) {
  if constexpr (D == 32) return c;
  const int r = D == 64 ? row >> 1 : row;
  return ((((c >> 1) + r) & (D / 32 - 1)) << 1) | (c & 1);
}
template <int D>
__device__ __forceinline__ int value_chunk(int row, int c) {
  if constexpr (D == 32) return c;
  return D == 64 ? c ^ (row & 2) : c ^ (row & 6);
}

// The work of a CTA.  Without WIDE false, and nothing written, where the value scales of a
// tile lie too far apart for one exponent, or one of them is zero.
template <int D, int NT, bool WIDE>
__device__ __forceinline__ bool split_part(const SplitParams &p) {
  using Geo = Geometry<D, NT>;
  constexpr int kGroups = Geo::kGroups, kRows = Geo::kRows, kStages = Geo::kStages;
  constexpr int kTile = Geo::kTile, kHalves = kTile / 16;  // 16 positions are the rows of an MMA
  constexpr int kDims = D / 8;  // dimensions of a value row a lane holds
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t *ring = smem + warp * Geo::kWarpBytes;
  const uint32_t ring_at = tc::smem_u32(ring);

  const int64_t cta = blockIdx.x;
  const int split = (int)(cta % p.parts.splits);
  const int64_t unit = cta / p.parts.splits;
  const int tile = (int)(unit % p.parts.row_tiles);
  const int h = (int)(unit / p.parts.row_tiles % p.H), b = (int)(unit / p.parts.row_tiles / p.H);
  const int32_t *table = p.block_table + (int64_t)b * p.max_blocks;
  const int own = lane & (kTile - 1);  // the position of a tile whose scales (and page) a lane sees to
  const bool even = p.block_size % kTile == 0;  // a tile lies in one page
  pdl_wait();
  pdl_trigger();
  // without a window a part's first position does not wait for the sequence's counts: nor does its page
  const int64_t guess = (int64_t)split * p.chunk + warp * kTile + (even ? 0 : own);
  int guessed = -1;
  if (p.window == 0 && guess < p.max_kv && block_of(p, (int)guess) < p.max_blocks)
    guessed = ld_input(table + block_of(p, (int)guess));
  const Sequence sq = sequence(p, b);
  if (sq.broken && h == 0 && tile == 0 && split == 0 && threadIdx.x == 0) set_status(p.status, QLIN_ERR_INVALID_ARG);
  const int R = sq.kept * p.G, r0 = tile * kRows;
  if (r0 >= R || R > p.few_rows) return true;

  // token and head of row r0 + i: one division for the tile
  const int tok0 = r0 / p.G, head0 = r0 - tok0 * p.G;
  const auto token_of = [&](int i) { return tok0 + (int)(((unsigned)(head0 + i) * p.group_inverse) >> 16); };
  // q is asked for before the codes, which would keep it waiting
  uint4 qw[NT][kGroups];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int i = nt * 8 + g, tok = token_of(i);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      qw[nt][k] = make_uint4(0, 0, 0, 0);
      if (r0 + i < R) {
        const uint16_t *row = p.q + (int64_t)(sq.first + tok) * p.ldq +
                              (int64_t)(h * p.G + r0 + i - tok * p.G) * D + k * 32 + t * 8;
        qw[nt][k] = ld_input(reinterpret_cast<const uint4 *>(row));
      }
    }
  }

  // positions of this CTA: what any of its rows sees, cut into parts
  const int last = min(kRows, R - r0) - 1;
  int lo, hi, beg, end;
  {
    int unused;
    sees(p, sq, tok0, lo, unused);
    sees(p, sq, token_of(last), unused, hi);
    const int64_t from = (int64_t)(lo & ~(kAlign - 1)) + (int64_t)split * p.chunk;
    beg = (int)min(from, (int64_t)max(hi, 0));
    end = split == p.parts.splits - 1 ? max(hi, beg) : (int)min(from + p.chunk, (int64_t)max(hi, beg));
  }

  // ---- the ring: tile n covers positions beg + (n * warps + warp) * 16 ...
  const int tiles = (end - beg + kTile - 1) / kTile;  // beg is a multiple of it
  const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
  const auto first_of = [&](int n) { return beg + (n * kAttnWarps + warp) * kTile; };
  const auto whole = [&](int n) { return even && n < mine && first_of(n) >= lo && first_of(n) + kTile <= end; };
  const auto page = [&](int n) {  // page of the lane's position of tile n (-1: none)
    const int j = first_of(n) + (even ? 0 : own);
    return n < mine && (whole(n) || (j + (even ? own : 0) >= lo && j + (even ? own : 0) < end))
               ? ld_input(table + block_of(p, j)) : -1;
  };
  const int piece_row = lane / Geo::kChunks, piece = lane % Geo::kChunks;
  const int64_t row_bytes = (int64_t)p.H * D;
  const uint32_t step_bytes = (uint32_t)(Geo::kRowStep * row_bytes);  // at most 16 * 4096 * 256
  const int64_t lane_off = piece_row * row_bytes + (int64_t)h * D + piece * 16;
  uint32_t sc[(kGroups + 1) / 2];  // the lane's scales of the tile issued last
  uint32_t sv = 0;
  unsigned there = 0;  // which positions of that tile are there
  int next_page = p.window == 0 && mine > 0 ? guessed : page(0);
  const auto load_scales = [&](int64_t row) {  // row: (slot, head) of the lane's position
    sv = ld_input(p.vs + row);
    if constexpr (kGroups == 1) {
      sc[0] = ld_input(p.ks + row);
    } else {
      load_words<kGroups / 2>(p.ks + row * kGroups, sc);
    }
  };
  const auto issue = [&](int n) {
    const int blk = next_page, j0 = first_of(n);
    next_page = page(n + 1);
    const uint32_t at = ring_at + (n % kStages) * Geo::kStageBytes;
    if (whole(n) && (unsigned)blk < (unsigned)p.num_blocks) {
      // one page: rows at one distance
      const int64_t slot = (int64_t)blk * p.block_size + (j0 - block_of(p, j0) * p.block_size);
      const int64_t off = slot * row_bytes + lane_off;
      const uint8_t *k = p.kc + off, *v = p.vc + off;
#pragma unroll
      for (int i = 0; i < Geo::kPieces; ++i) {
        const int r = i * Geo::kRowStep + piece_row;
        cp_async16(at + r * D + key_chunk<D>(r, piece) * 16, step_from(k, step_bytes, i));
        cp_async16(at + Geo::kCodes + r * D + value_chunk<D>(r, piece) * 16, step_from(v, step_bytes, i));
      }
      if (kTile == 32 || lane < kTile) load_scales((slot + own) * p.H + h);
      there = ~0u >> (32 - kTile);
    } else if (n < mine) {
      // positions that are not there (before lo, from end on, without a page): zeros
      const int j = j0 + own;
      const bool wanted = j >= lo && j < end, ok = wanted && (unsigned)blk < (unsigned)p.num_blocks;
      if (wanted && !ok && lane < kTile) set_status(p.status, QLIN_ERR_INVALID_ARG);
      const int64_t row = ok ? ((int64_t)blk * p.block_size + (j - block_of(p, j) * p.block_size)) * p.H + h : 0;
      there = __ballot_sync(~0u, ok) & (~0u >> (32 - kTile));
#pragma unroll 4
      for (int i = 0; i < Geo::kPieces; ++i) {
        const int r = i * Geo::kRowStep + piece_row;
        const int64_t off = __shfl_sync(~0u, row, r) * D + piece * 16;
        const bool fill = !((there >> r) & 1);
        cp_async16_or_zero(at + r * D + key_chunk<D>(r, piece) * 16, p.kc + off, fill);
        cp_async16_or_zero(at + Geo::kCodes + r * D + value_chunk<D>(r, piece) * 16, p.vc + off, fill);
      }
      sv = 0;
#pragma unroll
      for (int k = 0; k < (kGroups + 1) / 2; ++k) sc[k] = 0;
      if (ok && lane < kTile) load_scales(row);
    }
    cp_async_commit();
  };
  // Value scales are taken relative to 2^vexp.  `window` is its bit pattern: scales from it to
  // 2^(vexp + 15) keep P of a score at the maximum between 1 and 2^15.
  unsigned window = kNoWindow;
  // the scales of the tile issued last, as fp32, into its stage
  const auto put_scales = [&](int n) {
    if (n >= mine) return;
    uint8_t *at = ring + (n % kStages) * Geo::kStageBytes;
    const float v = half_bits_to_f32((uint16_t)sv);
    const bool fits = !((there >> lane) & 1) || __float_as_uint(v) - window < kWindow;
    const unsigned fit = __all_sync(~0u, fits) ? window : ~0u;
    if (kTile == 32 || lane < kTile) {
      float *k = reinterpret_cast<float *>(at + Geo::kScaleAt) + lane * kGroups;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) k[i] = half_bits_to_f32((uint16_t)(sc[i / 2] >> (16 * (i & 1))));
      reinterpret_cast<float *>(at + Geo::kVScaleAt)[lane] = v;
    }
    if (lane == 0) *reinterpret_cast<uint2 *>(at + Geo::kInfoAt) = make_uint2(there, fit);
  };

  // warps without a tile (few positions) go to the join, which leaves them out: 149 x 8 kv
  // heads over 2 positions 15.2 us, 17.1 with all warps prepared, written and joined
  bool apart = false;
  if (mine > 0) {
    // the first tiles are on their way while q arrives
    for (int n = 0; n < kStages - 1; ++n) {
      issue(n);
      if (n < kStages - 2) put_scales(n);
    }

    // q: row 8*nt + g, as the second operand; its largest magnitude becomes 2^14..2^15
    uint32_t qf[NT][kGroups][4];
    float qoff[NT][kGroups][2];    // -1152 times the sums of columns 2t and 2t + 1 over a key group
    float cf[NT][2];               // score factors of columns 2t and 2t + 1
    int vlo[NT][2], vhi[NT][2];    // positions those columns see
    int all_lo = lo, all_hi = hi;  // positions every row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint32_t u[4] = {qw[nt][k].x, qw[nt][k].y, qw[nt][k].z, qw[nt][k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const int e = q_exponent(top);
      const float up = pow2i(14 - e), factor = p.scale_log2 * pow2i(max(e - 14, -126));
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint32_t u[4] = {qw[nt][k].x, qw[nt][k].y, qw[nt][k].z, qw[nt][k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[nt][k][j] = half2_of(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xFFFF0000u) * up);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = __half22float2(bits_half2(qf[nt][k][j]));
          sum += x.x + x.y;
        }
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
#pragma unroll
        for (int c = 0; c < 2; ++c) qoff[nt][k][c] = -1152.0f * __shfl_sync(~0u, sum, (2 * t + c) * 4);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cf[nt][c] = __shfl_sync(~0u, factor, (2 * t + c) * 4);
        const int i = nt * 8 + 2 * t + c;
        vlo[nt][c] = lo, vhi[nt][c] = hi;  // columns without a row see everything (their q is 0)
        if (r0 + i < R) sees(p, sq, token_of(i), vlo[nt][c], vhi[nt][c]);
        all_lo = max(all_lo, vlo[nt][c]);
        all_hi = min(all_hi, vhi[nt][c]);
      }
    }
    all_lo = __reduce_max_sync(~0u, all_lo);
    all_hi = __reduce_min_sync(~0u, all_hi);

    float m[NT][2], l[NT][2], O[NT][kDims / 2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kDims / 2; ++i) O[nt][i][0] = O[nt][i][1] = O[nt][i][2] = O[nt][i][3] = 0.0f;
    }
    // O is sum p v 2^-vexp with p = 2^(s - m); WIDE: sum 2^s v 2^(bias - ref_s - ref_v) with references for
    // each column, a score and the exponent of its value.  They are kept apart: differences of scores
    // are exact near the maximum, and the exponents join them, however large the scores are.
    float ref_s[NT][2], ref_v[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ref_s[nt][0] = ref_s[nt][1] = -INFINITY, ref_v[nt][0] = ref_v[nt][1] = 0.0f;

    for (int n = 0; n < mine; ++n) {
      cp_async_wait<kStages - 2>();
      put_scales(n + kStages - 2);
      __syncwarp();
      issue(n + kStages - 1);
      const uint32_t at = ring_at + (n % kStages) * Geo::kStageBytes;
      uint8_t *stage = ring + (n % kStages) * Geo::kStageBytes;
      const uint2 info = *reinterpret_cast<const uint2 *>(stage + Geo::kInfoAt);
      if (!WIDE && info.y != window) {
        // the tile needs another window, or has scales that no window holds
        const unsigned a =
            (info.x >> lane) & 1 ? __float_as_uint(fabsf(reinterpret_cast<float *>(stage + Geo::kVScaleAt)[own])) : ~0u;
        const unsigned low = __reduce_min_sync(~0u, a), top = __reduce_max_sync(~0u, a == ~0u ? 0u : a);
        const int e_top = scale_exponent(top), e_low = min(scale_exponent(low), e_top);
        apart |= low == 0 || e_top - e_low > kSpan;  // (a way out of the loop costs the others 0.5 %)
        const unsigned now = (unsigned)(max(e_top - kSpan, e_low - 4) + 127) << 23;
        const float by = window == kNoWindow ? 0.0f : __uint_as_float(0x3F800000u + window - now);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < kDims / 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) O[nt][i][c] *= by;
        window = now;
      }
      const int j0 = first_of(n);
      const bool full = info.x == (~0u >> (32 - kTile)) && j0 >= all_lo && j0 + kTile <= all_hi;
      float vs[kHalves][2];  // of positions g and g + 8 of each half

      // scores of those positions and columns 2t, 2t + 1
      float S[kHalves][NT][4];
#pragma unroll
      for (int f = 0; f < kHalves; ++f) {
        const int r0 = 16 * f + g, r1 = r0 + 8;
        vs[f][0] = reinterpret_cast<const float *>(stage + Geo::kVScaleAt)[r0];
        vs[f][1] = reinterpret_cast<const float *>(stage + Geo::kVScaleAt)[r1];
        float ks[2][kGroups];
        load_shared<kGroups>(ks[0], reinterpret_cast<const float *>(stage + Geo::kScaleAt) + r0 * kGroups);
        load_shared<kGroups>(ks[1], reinterpret_cast<const float *>(stage + Geo::kScaleAt) + r1 * kGroups);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          uint32_t w0[2], w1[2];
          const uint32_t a0 = at + r0 * D + key_chunk<D>(r0, 2 * k) * 16 + t * 8;
          const uint32_t a1 = at + r1 * D + key_chunk<D>(r1, 2 * k) * 16 + t * 8;
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0[0]), "=r"(w0[1]) : "r"(a0));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w1[0]), "=r"(w1[1]) : "r"(a1));
          float acc[NT][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t a[4];
            int8x4_to_offset_half(w0[j], a[0], a[2]);
            int8x4_to_offset_half(w1[j], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (j == 0) mma_f16_from(acc[nt], a, qf[nt][k][0], qf[nt][k][1], qoff[nt][k][0], qoff[nt][k][1]);
              else mma_f16(acc[nt], a, qf[nt][k][2], qf[nt][k][3]);
            }
          }
          const float k0 = ks[0][k], k1 = ks[1][k];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            S[f][nt][0] = k ? fmaf(acc[nt][0], k0, S[f][nt][0]) : acc[nt][0] * k0;
            S[f][nt][1] = k ? fmaf(acc[nt][1], k0, S[f][nt][1]) : acc[nt][1] * k0;
            S[f][nt][2] = k ? fmaf(acc[nt][2], k1, S[f][nt][2]) : acc[nt][2] * k1;
            S[f][nt][3] = k ? fmaf(acc[nt][3], k1, S[f][nt][3]) : acc[nt][3] * k1;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // rounded here: the differences from the maximum are those of the rounded scores
          S[f][nt][0] = __fmul_rn(S[f][nt][0], cf[nt][0]), S[f][nt][2] = __fmul_rn(S[f][nt][2], cf[nt][0]);
          S[f][nt][1] = __fmul_rn(S[f][nt][1], cf[nt][1]), S[f][nt][3] = __fmul_rn(S[f][nt][3], cf[nt][1]);
        }
      }
      if (!full) {
        // A NaN value code times P = 0 would reach rows that do not see it: such
        // codes become 0 and their position's scale NaN.  (Two lanes to a row.)
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          const int r0 = 16 * f + g, r1 = r0 + 8;
          const bool ok0 = (info.x >> r0) & 1, ok1 = (info.x >> r1) & 1;
          const int p0 = j0 + r0, p1 = p0 + 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (!ok0 || p0 < vlo[nt][c] || p0 >= vhi[nt][c]) S[f][nt][c] = -INFINITY;
              if (!ok1 || p1 < vlo[nt][c] || p1 >= vhi[nt][c]) S[f][nt][2 + c] = -INFINITY;
            }
          unsigned bad = 0;
          uint32_t *w = reinterpret_cast<uint32_t *>(stage + Geo::kCodes + (16 * f + (lane >> 1)) * D + (lane & 1) * (D / 2));
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t nan = __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (nan) w[i] &= ~nan;
            bad |= nan;
          }
          const unsigned rows = __ballot_sync(~0u, bad != 0);
          if ((rows >> (2 * g)) & 3) vs[f][0] = NAN;
          if ((rows >> (2 * g + 16)) & 3) vs[f][1] = NAN;
        }
        __syncwarp();
      }

      float ev[kHalves][2];  // WIDE: exponents of the scales, which are left between 1 and 2
#pragma unroll
      for (int f = 0; f < kHalves; ++f)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (WIDE) {
            const unsigned a = __float_as_uint(fabsf(vs[f][i]));
            ev[f][i] = a ? (float)scale_exponent(a) : -INFINITY;
            vs[f][i] *= pow2i(-scale_exponent(a));
          } else {
            vs[f][i] *= __uint_as_float(0x7F000000u - window);  // 2^-vexp
          }
        }

      // online softmax per column
      uint32_t pf[kHalves][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {fmaxf(S[0][nt][0], S[0][nt][2]), fmaxf(S[0][nt][1], S[0][nt][3])};
        if constexpr (kHalves == 2) {
          mx[0] = fmaxf(mx[0], fmaxf(S[kHalves - 1][nt][0], S[kHalves - 1][nt][2]));
          mx[1] = fmaxf(mx[1], fmaxf(S[kHalves - 1][nt][1], S[kHalves - 1][nt][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(~0u, mx[0], o));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(~0u, mx[1], o));
        }
        bool grew = mx[0] > m[nt][0] || mx[1] > m[nt][1];
        // WIDE: the largest score with its value's exponent
        float top_s[2] = {ref_s[nt][0], ref_s[nt][1]}, top_v[2] = {ref_v[nt][0], ref_v[nt][1]};
        if constexpr (WIDE) {
          const auto take = [&](int c, float x, float e) {
            if ((x - top_s[c]) + (e - top_v[c]) > 0.0f) top_s[c] = x, top_v[c] = e;
          };
#pragma unroll
          for (int f = 0; f < kHalves; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) take(i & 1, S[f][nt][i], ev[f][i >> 1]);
#pragma unroll
          for (int o = 4; o < 32; o *= 2)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = __shfl_xor_sync(~0u, top_s[c], o), e = __shfl_xor_sync(~0u, top_v[c], o);
              take(c, x, e);
            }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            grew = grew || (top_s[c] - ref_s[nt][c]) + (top_v[c] - ref_v[nt][c]) > 0.0f;
        }
        if (__any_sync(~0u, grew)) {
          float a[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float now = fmaxf(m[nt][c], mx[c]);
            a[c] = exp2_approx(m[nt][c] - (now == -INFINITY ? 0.0f : now));
            m[nt][c] = now;
            l[nt][c] *= a[c];
            if constexpr (WIDE) {
              const float by = (ref_s[nt][c] - top_s[c]) + (ref_v[nt][c] - top_v[c]);
              a[c] = top_s[c] == -INFINITY ? 1.0f : exp2_approx(by);
              ref_s[nt][c] = top_s[c], ref_v[nt][c] = top_v[c];
            }
          }
#pragma unroll
          for (int i = 0; i < kDims / 2; ++i) {
            O[nt][i][0] *= a[0], O[nt][i][2] *= a[0];
            O[nt][i][1] *= a[1], O[nt][i][3] *= a[1];
          }
        }
        const float z0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0], z1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          const float(&s)[4] = S[f][nt];
          const float p00 = exp2_approx(s[0] - z0), p01 = exp2_approx(s[1] - z1);
          const float p10 = exp2_approx(s[2] - z0), p11 = exp2_approx(s[3] - z1);
          l[nt][0] += p00 + p10;
          l[nt][1] += p01 + p11;
          float w00 = p00 * vs[f][0], w01 = p01 * vs[f][0], w10 = p10 * vs[f][1], w11 = p11 * vs[f][1];
          if constexpr (WIDE) {
            const float y0 = ref_s[nt][0] == -INFINITY ? 0.0f : ref_s[nt][0], e0 = kWideBias - ref_v[nt][0];
            const float y1 = ref_s[nt][1] == -INFINITY ? 0.0f : ref_s[nt][1], e1 = kWideBias - ref_v[nt][1];
            w00 = exp2_approx((s[0] - y0) + (ev[f][0] + e0)) * vs[f][0];
            w01 = exp2_approx((s[1] - y1) + (ev[f][0] + e1)) * vs[f][0];
            w10 = exp2_approx((s[2] - y0) + (ev[f][1] + e0)) * vs[f][1];
            w11 = exp2_approx((s[3] - y1) + (ev[f][1] + e1)) * vs[f][1];
          }
          if (WIDE || !full) {  // an unseen position adds nothing, whatever its scale
            if (s[0] == -INFINITY) w00 = 0.0f;
            if (s[1] == -INFINITY) w01 = 0.0f;
            if (s[2] == -INFINITY) w10 = 0.0f;
            if (s[3] == -INFINITY) w11 = 0.0f;
          }
          pf[f][nt][0] = transpose8x8(half2_of(w00, w01));
          pf[f][nt][1] = transpose8x8(half2_of(w10, w11));
        }
      }

      // O^T += V^T P^T: positions 2t, 2t+1 (and +8) of each half, dimensions g*D/8 ...
      constexpr int kW = kDims / 4;  // words of a lane's piece of a value row
#pragma unroll
      for (int f = 0; f < kHalves; ++f) {
        uint32_t v[4][kW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * f + 2 * t + (i & 1) + 8 * (i >> 1);
          const uint8_t *row = stage + Geo::kCodes + r * D;
          if constexpr (kDims >= 16) {
#pragma unroll
            for (int c = 0; c < kDims / 16; ++c) {
              const uint4 x =
                  *reinterpret_cast<const uint4 *>(row + value_chunk<D>(r, g * (kDims / 16) + c) * 16);
              v[i][4 * c] = x.x, v[i][4 * c + 1] = x.y, v[i][4 * c + 2] = x.z, v[i][4 * c + 3] = x.w;
            }
          } else if constexpr (kDims == 8) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row + value_chunk<D>(r, g >> 1) * 16 + (g & 1) * 8);
            v[i][0] = x.x, v[i][1] = x.y;
          } else {
            v[i][0] = *reinterpret_cast<const uint32_t *>(row + g * 4);
          }
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          // (position 2t, 2t+1) byte pairs of dimensions 4i, 4i+1 | 4i+2, 4i+3
          const uint32_t x0 = __byte_perm(v[0][i], v[1][i], 0x5140), x1 = __byte_perm(v[0][i], v[1][i], 0x7362);
          const uint32_t y0 = __byte_perm(v[2][i], v[3][i], 0x5140), y1 = __byte_perm(v[2][i], v[3][i], 0x7362);
          const uint32_t a0[4] = {e4m3x2_to_half((uint16_t)x0), e4m3x2_to_half((uint16_t)(x0 >> 16)),
                                  e4m3x2_to_half((uint16_t)y0), e4m3x2_to_half((uint16_t)(y0 >> 16))};
          const uint32_t a1[4] = {e4m3x2_to_half((uint16_t)x1), e4m3x2_to_half((uint16_t)(x1 >> 16)),
                                  e4m3x2_to_half((uint16_t)y1), e4m3x2_to_half((uint16_t)(y1 >> 16))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(O[nt][2 * i], a0, pf[f][nt][0], pf[f][nt][1]);
            mma_f16(O[nt][2 * i + 1], a1, pf[f][nt][0], pf[f][nt][1]);
          }
        }
      }
    }
    cp_async_wait<0>();

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int o = 4; o < 32; o *= 2) {
        l[nt][0] += __shfl_xor_sync(~0u, l[nt][0], o);
        l[nt][1] += __shfl_xor_sync(~0u, l[nt][1], o);
      }
    __syncwarp();
    float *res = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
#pragma unroll
        for (int i = 0; i < kDims / 2; ++i)
          *reinterpret_cast<float2 *>(res + r * D + g * kDims + 2 * i) = make_float2(O[nt][i][c], O[nt][i][2 + c]);
        if (g == 0) {
          res[kRows * D + r] = m[nt][c];
          res[kRows * D + kRows + r] = l[nt][c];
          if constexpr (WIDE) {
            res[kRows * D + 2 * kRows + r] = ref_s[nt][c];
            res[kRows * D + 3 * kRows + r] = ref_v[nt][c];
          }
        }
      }
    if (!WIDE && lane == 0) res[kRows * D + 2 * kRows] = __uint_as_float(window);  // 2^vexp
  }
  if constexpr (WIDE) {
    __syncthreads();
  } else if (__syncthreads_or(apart)) {
    return false;
  }
  const int active = min(tiles, kAttnWarps);
  for (int i = threadIdx.x; i < kRows * D / 4; i += 32 * kAttnWarps) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r0 + r >= R) break;
    const float *w = reinterpret_cast<const float *>(smem);
    constexpr int kStep = Geo::kWarpBytes / 4;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kAttnWarps; ++k)
      if (k < active) top = fmaxf(top, w[k * kStep + kRows * D + r]);
    const float z = top == -INFINITY ? 0.0f : top;
    float top_s = -INFINITY, top_v = 0.0f;  // WIDE: the reference of O
    if constexpr (WIDE) {
#pragma unroll
      for (int k = 0; k < kAttnWarps; ++k)
        if (k < active) {
          const float *x = w + k * kStep + kRows * D + 2 * kRows + r;
          if ((x[0] - top_s) + (x[kRows] - top_v) > 0.0f) top_s = x[0], top_v = x[kRows];
        }
      top_s = top_s == -INFINITY ? 0.0f : top_s;
    }
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kAttnWarps; ++k) {
      if (k >= active) break;
      const float *x = w + k * kStep;
      const float f = exp2_approx(x[kRows * D + r] - z);
      L = fmaf(f, x[kRows * D + kRows + r], L);
      const float *ref = x + kRows * D + 2 * kRows;
      const float fo = WIDE ? exp2_approx((ref[r] - top_s) + (ref[kRows + r] - top_v)) : f * ref[0];
      const float4 y = *reinterpret_cast<const float4 *>(x + r * D + d);
      o.x = fmaf(fo, y.x, o.x), o.y = fmaf(fo, y.y, o.y), o.z = fmaf(fo, y.z, o.z), o.w = fmaf(fo, y.w, o.w);
    }
    float inv = L == 0.0f ? 0.0f : 1.0f / L;
    if constexpr (WIDE) {
      // 2^(top_s + top_v - z) in two halves: it can lie below binary32's range where its product with O does not
      const float half = exp2_approx(0.5f * ((top_s - z) + (top_v - kWideBias)));
      o.x *= half, o.y *= half, o.z *= half, o.w *= half;
      inv *= half;
    }
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    if (p.parts.splits == 1) {
      const int rr = r0 + r;
      uint16_t *dst = p.out + (int64_t)(sq.first + rr / p.G) * p.ldo + (int64_t)(h * p.G + rr % p.G) * D + d;
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2((uint32_t)f32_to_bf16_bits(o.x) | ((uint32_t)f32_to_bf16_bits(o.y) << 16),
                     (uint32_t)f32_to_bf16_bits(o.z) | ((uint32_t)f32_to_bf16_bits(o.w) << 16));
    } else {
      const int64_t at = cta * kRows + r;
      *reinterpret_cast<float4 *>(p.parts.o + at * D + d) = o;
      if (d == 0) p.parts.sum[at] = make_float2(top, L);
    }
  }
  return true;
}

// The general form begins again: carried on from where the other leaves, its code costs that
// one 4 % (D 128, batch of 256 ragged contexts up to 4096: 77.7 us; as here 74.2).  From D 128 on it is
// a function of its own for the same reason (inline 79.0 us); below, the call costs more than the
// code (D 64, 64 contexts, 8 kv heads: 57.5 us with it, 54.6 inline).
template <int D, int NT>
__device__ __noinline__ void split_part_wide(const SplitParams &p) {
  split_part<D, NT, true>(p);
}
template <int D, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, Geometry<D, NT>::kCtas)
    k_attn_split(const __grid_constant__ SplitParams p) {
  if (split_part<D, NT, false>(p)) return;
  if constexpr (D >= 128) split_part_wide<D, NT>(p);
  else split_part<D, NT, true>(p);
}

// Joins the parts of one row: out = sum_s w_s o_s / sum_s w_s with
// w_s = l_s 2^(m_s - max m), the exponent of l_s joined to the other, which alone can be
// below binary32's range where w_s is not.  Many parts: a CTA per row, its warps over the parts;
// few: a warp per row.
constexpr int kFewParts = 16;
constexpr int kManyWarps = 16, kFewWarps = 8;  // warps of a CTA
template <int D, bool MANY, int CTAS>
__global__ void __launch_bounds__(32 * (MANY ? kManyWarps : kFewWarps), CTAS)
    k_attn_join(const AttnDev p, const AttnParts parts, bool many) {
  const int rows = parts.rows;
  constexpr int V = D / 32;                  // floats of a lane
  constexpr int kOver = MANY ? kManyWarps : 1;  // warps that share a row
  constexpr int kBatch = MANY ? 8 : 4;       // parts whose loads are in flight at once
  __shared__ float s_o[kOver][D];
  __shared__ float s_w[kOver];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = MANY ? warp : 0;
  const int64_t row = MANY ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kFewWarps + warp;
  const int64_t unit = row / rows;
  const int r = (int)(row % rows);
  const int tile = (int)(unit % parts.row_tiles);
  const int h = (int)(unit / parts.row_tiles % p.H), b = (int)(unit / parts.row_tiles / p.H);
  pdl_wait();
  pdl_trigger();
  if (b >= p.B) return;
  const Sequence sq = sequence(p, b);
  const int rr = tile * rows + r;
  if (rr >= sq.kept * p.G || (sq.kept * p.G > p.few_rows) != many) return;
  const float2 *sum = parts.sum + unit * parts.splits * rows + r;
  const float *src = parts.o + (unit * parts.splits * rows + r) * D + lane * V;
  uint32_t x[kBatch][V];
  float2 e[kBatch];
  const auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t s = s0 + i * kOver;
      e[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) x[i][v] = 0u;
      if (s < parts.splits) {
        e[i] = ld_input(sum + s * rows);
        load_words<V>(src + s * rows * D, x[i]);
      }
    }
  };
  load(part);
  float top = -INFINITY;
  for (int s = lane; s < parts.splits; s += 32) top = fmaxf(top, ld_input(&sum[(int64_t)s * rows].x));
  top = warp_max(top);
  const float z = top == -INFINITY ? 0.0f : top;
  float o[V], W = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  for (int s0 = part; s0 < parts.splits;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = (int)(__float_as_uint(e[i].y) >> 23);  // 0 beyond the last part, and w with it
      const float mantissa = e[i].y * __uint_as_float((unsigned)(254 - k) << 23);
      const float w = mantissa * exp2_approx((e[i].x - z) + (float)(k - 127));
      W += w;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = fmaf(w, __uint_as_float(x[i][v]), o[v]);
    }
    s0 += kBatch * kOver;
    if (s0 < parts.splits) load(s0);
  }
  uint16_t *dst = p.out + (int64_t)(sq.first + rr / p.G) * p.ldo + (int64_t)(h * p.G + rr % p.G) * D;
  if constexpr (MANY) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = o[i];
    if (lane == 0) s_w[warp] = W;
    __syncthreads();
    if (threadIdx.x < D / 2) {
      const int d = 2 * threadIdx.x;
      float a = 0.0f, c = 0.0f, w = 0.0f;
#pragma unroll
      for (int k = 0; k < kOver; ++k) {
        a += s_o[k][d];
        c += s_o[k][d + 1];
        w += s_w[k];
      }
      const float inv = w == 0.0f ? 0.0f : 1.0f / w;
      *reinterpret_cast<uint32_t *>(dst + d) =
          (uint32_t)f32_to_bf16_bits(a * inv) | ((uint32_t)f32_to_bf16_bits(c * inv) << 16);
    }
  } else {
    const float inv = W == 0.0f ? 0.0f : 1.0f / W;
    if constexpr (V == 1) {
      dst[lane] = f32_to_bf16_bits(o[0] * inv);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        w[i] = (uint32_t)f32_to_bf16_bits(o[2 * i] * inv) | ((uint32_t)f32_to_bf16_bits(o[2 * i + 1] * inv) << 16);
      store_words<V / 2>(dst + lane * V, w);
    }
  }
}

template <int D, int NT>
cudaError_t launch_nt(const SplitParams &p, int64_t units, cudaStream_t st) {
  using Geo = Geometry<D, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(k_attn_split<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  e = launch_kernel(k_attn_split<D, NT>, dim3((unsigned)(units * p.parts.splits)), dim3(32 * kAttnWarps), Geo::kSmem,
                    st, 1, p);
  if (e != cudaSuccess || p.parts.splits == 1) return e;
  return launch_attn_join(p, p.parts, D, false, st);
}
template <int D>
cudaError_t launch_join_d(const AttnDev &p, const AttnParts &parts, bool many, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.H * parts.row_tiles * parts.rows;
  if (parts.splits <= kFewParts)
    return launch_kernel(k_attn_join<D, false, 1>, dim3((unsigned)((rows + kFewWarps - 1) / kFewWarps)),
                         dim3(32 * kFewWarps), 0, st, 1, p, parts, many);
  // Rows for one CTA a multiprocessor at most: registers for all loads of a batch at once (one context of
  // 32768: 14.4 us, 15.2 with two CTAs' registers).  More: two CTAs (168 rows over 8192: 30.6 us; 34.1 against
  // 32.7 before the unpacking ahead of it had all its registers).
  constexpr int kTwo = D <= 128 ? 2 : 1;
  return launch_kernel(rows > sm_count() ? k_attn_join<D, true, kTwo> : k_attn_join<D, true, 1>, dim3((unsigned)rows),
                       dim3(32 * kManyWarps), 0, st, 1, p, parts, many);
}
template <int D>
cudaError_t launch_d(const SplitParams &p, int rows, int64_t units, cudaStream_t st) {
  return rows == 8 ? launch_nt<D, 1>(p, units, st) : launch_nt<D, 2>(p, units, st);
}

}  // namespace

cudaError_t launch_attn_join(const AttnDev &p, const AttnParts &parts, int64_t D, bool many, cudaStream_t st) {
  switch (D) {
    case 32: return launch_join_d<32>(p, parts, many, st);
    case 64: return launch_join_d<64>(p, parts, many, st);
    case 128: return launch_join_d<128>(p, parts, many, st);
    case 256: return launch_join_d<256>(p, parts, many, st);
  }
  return cudaErrorInvalidValue;
}

AttnDev attn_dev(const AttnArgs &a, int few_rows, unsigned *status) {
  AttnDev p{};
  p.q = (const uint16_t *)a.q, p.q_start = a.q_start, p.kv_len = a.kv_len, p.block_table = a.block_table;
  p.kc = (const uint8_t *)a.k_cache, p.vc = (const uint8_t *)a.v_cache;
  p.ks = (const uint16_t *)a.k_scale, p.vs = (const uint16_t *)a.v_scale;
  p.out = (uint16_t *)a.out, p.ldq = a.ldq, p.ldo = a.ldo, p.max_blocks = a.max_blocks;
  p.B = (int)a.B, p.T = (int)a.T, p.H = (int)a.H, p.G = (int)(a.Hq / a.H);
  p.max_q = (int)a.max_q, p.max_kv = (int)a.max_kv;
  p.block_size = (int)a.block_size;
  p.block_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a.block_size == (int64_t)1 << s) p.block_shift = s;
  p.num_blocks = (int)(a.num_slots / a.block_size);
  p.causal = a.causal != 0, p.window = (int)std::min<int64_t>(a.window, 1 << 30);
  p.few_rows = few_rows;
  p.scale_log2 = a.scale * kLog2e;
  p.status = status;
  return p;
}

// Rows are tiled by 8 where one tile holds them, else by 16 (each code is then
// converted for twice the rows).  Positions are split until one wave of CTAs
// fills the GPU, but not below 128 positions a part; where there are more units
// than that, into parts of at least 1024 so that ragged sequences even out.
AttnSplitPlan attn_split_plan(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t rows, int64_t max_kv,
                              int64_t window, int sms) {
  AttnSplitPlan plan{};
  const int64_t G = Hq / H;
  plan.rows = rows <= 8 ? 8 : 16;
  plan.row_tiles = (int)((rows + plan.rows - 1) / plan.rows);
  int64_t range = max_kv;
  if (window > 0 && window < max_kv) range = std::min(range, window + plan.rows / G + 1);
  const int64_t units = B * H * plan.row_tiles, slots = (int64_t)sms * (plan.rows == 8 ? 3 : 2);
  const int64_t fill = std::min((slots + units - 1) / units, (range + 127) / 128);
  const int64_t even = std::min((4 * slots + units - 1) / units, range / 1024);
  const int64_t want = std::max<int64_t>(1, std::max(fill, even));
  range += kAlign - 1;  // the first part begins at a multiple of 32; the last one takes what is left
  constexpr int64_t step = kAlign * kAttnWarps;
  plan.chunk = std::max(step, (range + want * step - 1) / (want * step) * step);
  plan.splits = (int)std::max<int64_t>(1, (range + plan.chunk - 1) / plan.chunk);
  plan.ws_bytes = plan.splits > 1 ? (size_t)(units * plan.splits * plan.rows * (D + 2) * 4) : 0;
  plan.ws_bytes = round_up(plan.ws_bytes, 256);
  return plan;
}

cudaError_t launch_attn_split(const AttnArgs &a, const AttnSplitPlan &plan, int few_rows, void *ws, unsigned *status,
                              cudaStream_t st) {
  SplitParams p{};
  static_cast<AttnDev &>(p) = attn_dev(a, few_rows, status);
  p.group_inverse = (65536u + p.G - 1) / p.G;
  p.parts.row_tiles = plan.row_tiles, p.parts.rows = plan.rows, p.parts.splits = plan.splits, p.chunk = plan.chunk;
  const int64_t units = a.B * a.H * plan.row_tiles;
  p.parts.o = (float *)ws;
  p.parts.sum = p.parts.o ? (float2 *)(p.parts.o + units * plan.splits * plan.rows * a.D) : nullptr;
  switch (a.D) {
    case 32: return launch_d<32>(p, plan.rows, units, st);
    case 64: return launch_d<64>(p, plan.rows, units, st);
    case 128: return launch_d<128>(p, plan.rows, units, st);
    case 256: return launch_d<256>(p, plan.rows, units, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
