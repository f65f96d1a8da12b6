// Attention over the 4-bit KV cache for few rows: decode, and short runs of new
// tokens.  A (position, kv head) is D bytes of codes and D/8 of scales, read once for
// up to 8 * NT rows (new tokens times the heads of the group).
//
// Work.  A unit is a row tile of a (sequence, kv head); its positions are tiles of 32 (D 256: 16).
// The steps (a tile for each of a CTA's four warps) of all units, one after the other, are cut into
// equal ranges, one for each resident CTA, whatever the lengths of the sequences are; every CTA finds its range by
// a sum over the sequences.  A unit that ends up in several ranges is joined by a second kernel.  (Ranges for
// each warp, without a join within the CTA: 71.7 us against 68.5 for a batch of 256 ragged contexts up to 4096.)
// Where ranges are of several steps, a unit's beginning counts as two more: 60 us without, 54.9 with.
//
// Arithmetic.  Scores and outputs are transposed, S^T = K q^T and O^T = V^T P^T, so that
// positions (then head dimensions) fill the 16 rows of mma.m16n8k16 and the query heads its
// 8 columns.  A warp's tiles come through a ring of its own in shared memory, by 16-byte asynchronous
// copies (a page's rows of a head are contiguous), and from there to registers in the layout of the operands.
//   * Keys: with its sign bit turned a code c is c + 8, and those four bits alone are a subnormal
//     float16, (c + 8) 2^-24 (or 2^-20, where they lie four bits higher: there q is 16 times less).
//     The sums start at -8 times the sum of q, in fp32.  The products of one 32-dimension group are
//     summed in fp32 and then scaled by the group's scale in fp32.
//   * Values: the same bits beside 0x6400 are 1024 + 8 + c, and minus 1032 the code; times the scale it is
//     rounded to float16 once.
//   * P is the weight under a row's reference, 2^8 for the largest score where it is taken, in float16; it is taken anew
//     only where a score is above it by more than 15.
// A position with a scale that the store does not write gives NaN to the rows that see it
// and nothing to the others: its scores are NaN where seen and its values 0.
#include <algorithm>
#include <cfloat>

#include "attn.cuh"
#include "common.cuh"
#include "int4_cache.cuh"
#include "kernels.h"

namespace qlin {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// A row's reference lies kBias below its largest score when it is taken, and no score passes it by more than kTop: P
// stays below 2^15.5.  Beyond kExact, where binary32 has no room for the bias (from 2^27 on it rounds by up to itself, and P
// left float16), the reference is the largest score.
constexpr float kBias = 8.0f, kTop = kBias + 7.0f, kExact = 0x1p22f;
constexpr int kAlign = 32;  // a unit's first position is rounded down to a multiple of this

// A unit whose steps are split, as the range where it begins notes it: in the list of ranges, or (few units) in
// that of all units.
struct __align__(16) JoinEntry {
  int ranges;       // how many hold a part; 0: nothing to join
  int first;        // the first one
  int first_slot;   // which of its two partial results; the others' is their first
  int h, r0, R;     // head, first row, rows of the sequence
  int first_token;
  int pad;
};

struct Int4Params : AttnDev {
  unsigned group_inverse;  // 2^16 / G rounded up: (x * it) >> 16 is x / G for x < 256 (G <= 128)
  int step_shift;          // a step is 2^it positions
  int start;               // a unit's beginning (its queries, its first tiles on their way) is counted as so many steps
  float *o;                // [range, 2, row] partial results: O (D), divided by its sum
  float2 *sum;             // {reference, sum}
  JoinEntry *list;         // [range], or [unit]
  bool by_unit;
  int row_tiles;           // of a sequence, at most
  // What the masked codes are combined with.  Here, where the compiler does not see them: a mask and a second
  // constant would be two instructions for each pair of codes.
  uint32_t turn0, turn4, magic0, magic4;
};

// Resident CTAs that the registers are budgeted for.  (Head size 64 in tiles of 16 rows: 30.5 us at 2, 28.8 at 3; one of
// 256 in tiles of 8: 25.5 us at 2, 28.7 with spills at 3.)
constexpr int attn_int4_ctas(int64_t D, int rows) { return D < 256 && rows <= 8 ? 4 : D <= 64 ? 3 : 2; }

template <int D, int NT>
struct Geometry4 {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = attn_int4_ctas(D, kRows);
  static constexpr int kGroups = D / 32;
  static constexpr int kTile = D >= 256 ? 16 : 32;  // positions of a warp
  static constexpr int kHalves = kTile / 16;        // 16 positions are the rows of an MMA
  static constexpr int kStep = kTile * kWarps;
  static constexpr int kDims = D / 8;               // dimensions of a value row a lane holds
  static constexpr int kMmas = D / 16;              // of 16 dimensions
  // a stage of a warp's ring: key codes, value codes, key scales, value scales of a tile
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;
  static constexpr int kStages = kCtas == 4 ? 2 : 3;  // as many as fit (3 at 2 or 3 CTAs: 2% over 2, 4: none)
  static constexpr int kResult = (kRows * D + 2 * kRows) * 4;  // a warp's result, over its ring
  static constexpr int kWarpBytes = kStages * kStage > kResult ? kStages * kStage : kResult;
  static constexpr int kWarpFloats = kWarpBytes / 4;
  static constexpr int kSmem = kWarps * kWarpBytes;
};

__device__ __forceinline__ void mma4(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma4_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                          float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// N words of shared memory (aligned to 4 min(N, 4) bytes).
template <int N>
__device__ __forceinline__ void shared_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}
// The position, of the eight that fill rows 0 to 7 (8 to 15) of an operand, that row r has.  Rows 2t and 2t + 1 have
// positions 2t and 2t + 1, exchanged for odd t: so the lanes of a key load, and those of a value load, read rows of both
// parities, which at 64 bytes a row lie in different banks.
__device__ __forceinline__ int row_position(int r) { return (r & 6) | ((r ^ (r >> 1)) & 1); }
// Half of a 16-bit pattern pair.
__device__ __forceinline__ float half_lo(uint32_t w) { return __low2float(bits_half2(w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __high2float(bits_half2(w)); }

// Steps of every row tile of a sequence (as many as the widest needs, and p.start before them), and its row tiles.
__device__ __forceinline__ int sequence_steps(const Int4Params &p, const Sequence &s, int rows) {
  int64_t range = s.kv;
  if (p.window > 0) {
    const int64_t w = (int64_t)p.window * (p.causal ? 1 : 2) + rows / p.G + 1;
    range = min(range, w) + kAlign - 1;
  }
  return p.start + max(1, (int)((range + (1 << p.step_shift) - 1) >> p.step_shift));
}
__device__ __forceinline__ int sequence_tiles(const AttnDev &p, const Sequence &s, int rows) {
  const int R = s.kept * p.G;
  return R > p.few_rows ? 0 : (R + rows - 1) / rows;
}

// Where the CTA stands in the list of all steps.
struct Place {
  int b, h, tile;
  int tiles;      // of sequence b
  int steps, at;  // of the unit; the step that comes next
};

// EVEN: pages are powers of two from 16 positions on, so those of half a tile lie in one page.
template <int D, int NT, bool EVEN>
__global__ void __launch_bounds__(kThreads, Geometry4<D, NT>::kCtas) k_attn_int4(const __grid_constant__ Int4Params p) {
  using Geo = Geometry4<D, NT>;
  constexpr int kRows = Geo::kRows, kGroups = Geo::kGroups, kTile = Geo::kTile, kHalves = Geo::kHalves;
  constexpr int kStep = Geo::kStep, kDims = Geo::kDims, kMmas = Geo::kMmas;
  constexpr int kScaleWords = (kGroups + 1) / 2;        // of a position's key scales
  constexpr int kValueWords = kDims >= 8 ? kDims / 8 : 1;  // of a lane's part of a value row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[kWarps];
  __shared__ Place s_place;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();

  // ---- the range of steps: thread i sums up sequences [i * per, (i + 1) * per)
  const int per = (p.B + kThreads - 1) / kThreads;
  const auto work_of = [&](int b, int &tiles, int &steps) {
    const Sequence s = sequence(p, b);
    if (s.broken && blockIdx.x == 0) set_status(p.status, QLIN_ERR_INVALID_ARG);
    tiles = sequence_tiles(p, s, kRows);
    steps = sequence_steps(p, s, kRows);
    return tiles * p.H * steps;
  };
  int mine = 0;
  Place at{};
  for (int b = threadIdx.x * per; b < min(p.B, ((int)threadIdx.x + 1) * per); ++b) mine += work_of(b, at.tiles, at.steps);
  int before = mine;  // inclusive sum over the warp, then over the CTA
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(~0u, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) s_sum[warp] = before;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += s_sum[i];
    total += s_sum[i];
  }
  // equal ranges: the first `longer` of them have one step more
  const int ranges = max(1, min((int)gridDim.x, total));
  const int shortest = total / ranges, longer = total - shortest * ranges;
  const auto range_begin = [&](int r) { return r * shortest + min(r, longer); };
  const int range = blockIdx.x;
  if (p.list && !p.by_unit && threadIdx.x == 0) p.list[range].ranges = 0;
  if (p.list && p.by_unit && blockIdx.x == 0) {  // units that no range has
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int tiles = sequence_tiles(p, sequence(p, b), kRows);
      for (int i = 0; i < p.H; ++i)
        for (int k = tiles; k < p.row_tiles; ++k) p.list[(b * p.H + i) * p.row_tiles + k].ranges = 0;
    }
  }
  if (range >= ranges || total == 0) return;
  int s = range_begin(range);
  const int s_end = range_begin(range + 1);
  if (s < before && s >= before - mine) {  // the thread among whose sequences the range begins
    int from = before - mine, work = mine;
    at.b = threadIdx.x * per;
    if (per > 1) {
      while ((work = work_of(at.b, at.tiles, at.steps)) <= s - from) {
        from += work;
        ++at.b;
      }
    }
    const int unit = (s - from) / at.steps;
    at.at = s - from - unit * at.steps;
    at.h = unit / at.tiles;
    at.tile = unit - at.h * at.tiles;
    s_place = at;
  }
  __syncthreads();
  at = s_place;

  uint8_t *const ring = smem + warp * Geo::kWarpBytes;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t page_bytes = (uint32_t)p.H * p.block_size * (D / 2);  // of codes
  // the lane's rows of keys (positions kr and kr + 8 of a half) and of values (va, vb, va + 8, vb + 8)
  const int kr = row_position(g), va = row_position(2 * t), vb = row_position(2 * t + 1);
  const unsigned last_page = (unsigned)p.num_blocks - 1;
  const uint32_t turn0 = p.turn0, turn4 = p.turn4, magic0 = p.magic0, magic4 = p.magic4;

  for (bool first = true; s < s_end; first = false) {
    const Sequence sq = sequence(p, at.b);
    const int R = sq.kept * p.G, r0 = at.tile * kRows, h = at.h;
    const int32_t *table = p.block_table + (int64_t)at.b * p.max_blocks;
    const int steps_here = min(at.steps - at.at, s_end - s);
    if (at.at + steps_here <= p.start) break;  // the range ends before the unit's first step: the next one has it
    const bool begins = at.at <= p.start;      // the unit's first step is here

    // token and head of row r0 + i: one division for the tile
    const int tok0 = r0 / p.G, head0 = r0 - tok0 * p.G;
    const auto token_of = [&](int i) { return tok0 + (int)(((unsigned)(head0 + i) * p.group_inverse) >> 16); };
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

    // positions [lo, end) that some row of the tile sees, from beg on this range's
    int lo, hi, beg, end;
    {
      int unused;
      const int last = min(kRows, R - r0) - 1;
      sees(p, sq, tok0, lo, unused);
      sees(p, sq, token_of(last), unused, hi);
      hi = max(hi, 0);
      const int64_t from = (int64_t)(lo & ~(kAlign - 1)) + ((int64_t)max(at.at - p.start, 0) << p.step_shift);
      beg = (int)min(from, (int64_t)hi);
      end = (int)min(from + ((int64_t)(steps_here - max(p.start - at.at, 0)) << p.step_shift), (int64_t)hi);
      if (beg < from) beg = end = 0;  // nothing left for this range
    }
    int tiles = (end - beg + kTile - 1) / kTile;
    int count = (tiles - warp + kWarps - 1) / kWarps;  // of this warp
    if (p.num_blocks == 0 && tiles > 0) {  // a cache without pages
      if (lane == 0) set_status(p.status, QLIN_ERR_INVALID_ARG);
      tiles = count = 0;
    }
    const auto first_of = [&](int n) { return beg + (n * kWarps + warp) * kTile; };

    // ---- copies.  All rows of a tile are copied, from a page of the cache wherever the table points; those that are
    // not the sequence's are masked where they are used.
    constexpr int kV = Geo::kCodes, kKS = 2 * Geo::kCodes, kVS = kKS + Geo::kScales;  // in a stage
    constexpr int kBatch = 32 / kHalves;  // EVEN: tiles whose pages are looked up at once, lane l those of half l
    bool suspect = false;                 // some page is not in the cache
    int pg[EVEN ? 1 : kHalves];           // pages of the batch (EVEN: of the tile) after the one at hand
    uint64_t row_now = 0;                 // EVEN: where the codes of the batch's halves begin
    const auto look_up = [&](int n) {
#pragma unroll
      for (int f = 0; f < (EVEN ? 1 : kHalves); ++f) {
        const int i = EVEN ? n + lane / kHalves : n;
        const int j = first_of(i) + (EVEN ? lane % kHalves * 16 : 16 * f + (lane & 15));
        pg[f] = i < count && j < end ? ld_input(table + (EVEN ? j >> p.block_shift : block_of(p, j))) : -1;
      }
    };
    const auto row_of = [&](int page, int j, bool wanted) {  // where position j's codes begin
      suspect |= wanted && (unsigned)page > last_page;
      const uint32_t off = EVEN ? j & (p.block_size - 1) : j - block_of(p, j) * p.block_size;
      return (uint64_t)min((unsigned)page, last_page) * page_bytes + ((uint32_t)h * p.block_size + off) * (uint32_t)(D / 2);
    };
    const auto copy = [&](int n) {  // starts the copy of tile n
      if (n >= count) return;
      const uint32_t to = ring_at + n % Geo::kStages * Geo::kStage;
      if constexpr (EVEN) {
        if (n % kBatch == 0) {
          const int i = n + lane / kHalves, j = first_of(i) + lane % kHalves * 16;
          row_now = row_of(pg[0], j, i < count && j < end && j + 15 >= lo);
          suspect = __any_sync(~0u, suspect);
          look_up(n + kBatch);
        }
        // lanes of a half: its codes 16 bytes a lane at a time, its scales at once
        constexpr int kLanes = 32 / kHalves, kScale = D / kLanes >= 4 ? D / kLanes : 4;
        const int half = lane / kLanes, i = lane % kLanes;
        const uint64_t row = __shfl_sync(~0u, row_now, n % kBatch * kHalves + half);
        const uint8_t *k = p.kc + row + i * 16, *v = p.vc + row + i * 16;
        const uint32_t d = to + half * (8 * D) + i * 16;
#pragma unroll
        for (int x = 0; x < 8 * D; x += kLanes * 16) {
          copy16(d + x, k + x);
          copy16(d + kV + x, v + x);
        }
        if (i < D / kScale) {
          const uint32_t e = to + kKS + half * D + i * kScale;
          copy_small<kScale>(e, reinterpret_cast<const uint8_t *>(p.ks) + row / 8 + i * kScale);
          copy_small<kScale>(e + Geo::kScales, reinterpret_cast<const uint8_t *>(p.vs) + row / 8 + i * kScale);
        }
      } else {
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          const int j = first_of(n) + 16 * f + (lane & 15);
          const uint64_t own = row_of(pg[f], j, j >= lo && j < end);
          // 16-byte pieces of a row, and rows that the warp copies at once
          constexpr int kPieces = D / 32, kAtOnce = 32 / kPieces;
#pragma unroll
          for (int i = 0; i < (16 + kAtOnce - 1) / kAtOnce; ++i) {
            const int r = i * kAtOnce + lane / kPieces, piece = lane % kPieces * 16;
            const uint64_t row = __shfl_sync(~0u, own, r & 15);
            const uint32_t d = (f * 16 + r) * (D / 2) + piece;
            if (r < 16) {
              copy16(to + d, p.kc + row + piece);
              copy16(to + kV + d, p.vc + row + piece);
            }
          }
          if (lane < 16) {
            const uint32_t e = (f * 16 + lane) * (D / 16);
            const uint8_t *ks = reinterpret_cast<const uint8_t *>(p.ks) + own / 8;
            const uint8_t *vs = reinterpret_cast<const uint8_t *>(p.vs) + own / 8;
            if constexpr (D == 32) {
              uint8_t *stage = ring + n % Geo::kStages * Geo::kStage;
              *reinterpret_cast<uint16_t *>(stage + kKS + e) = ld_input(reinterpret_cast<const uint16_t *>(ks));
              *reinterpret_cast<uint16_t *>(stage + kVS + e) = ld_input(reinterpret_cast<const uint16_t *>(vs));
            } else {
              copy_small<D / 16>(to + kKS + e, ks);
              copy_small<D / 16>(to + kVS + e, vs);
            }
          }
        }
        suspect = __any_sync(~0u, suspect);
        look_up(n + 1);
      }
    };

    const bool whole = begins && at.at + steps_here == at.steps;  // the unit's output, or a part of it
    const int64_t slot = (int64_t)(range * 2 + (first ? 0 : 1)) * kRows;
    const auto out_row = [&](int r) {
      const int rr = r0 + r;
      return p.out + (int64_t)(sq.first + rr / p.G) * p.ldo + (int64_t)(h * p.G + rr % p.G) * D;
    };
    if (count > 0) {
      look_up(0);
      for (int n = 0; n < Geo::kStages - 1; ++n) {
        copy(n);
        asm volatile("cp.async.commit_group;" ::: "memory");
      }

      // ---- q: row 8*nt + g, as the second operand; its largest magnitude becomes 2^14..2^15
      uint32_t qf[NT][kGroups][4];
      float qoff[NT][kGroups][2];    // -8 2^-24 times the sums of columns 2t and 2t + 1 over a key group
      float cf[NT][2];               // score factors of columns 2t and 2t + 1
      int all_lo = lo, all_hi = end;  // positions every row sees
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t most = 0;  // BF16 magnitudes are in the order of their bits
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const uint32_t u[4] = {qw[nt][k].x, qw[nt][k].y, qw[nt][k].z, qw[nt][k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) most = __vmaxu2(most, u[j] & 0x7FFF7FFFu);
        }
        most = __vmaxu2(most, __shfl_xor_sync(~0u, most, 1));
        most = __vmaxu2(most, __shfl_xor_sync(~0u, most, 2));
        const float top = __uint_as_float(max(most & 0xFFFFu, most >> 16) << 16);
        const int e = q_exponent(top);
        // A factor beyond binary32 (|q| from about 2^121 on) becomes its largest number: scores that are not equal lie far
        // apart under either, and those of 0 stay 0.
        const float up = pow2i(14 - e);
        const float factor = fminf(fmaxf((p.scale_log2 * pow2i(max(e - 14, -126))) * 0x1p24f, -FLT_MAX), FLT_MAX);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const uint32_t u[4] = {qw[nt][k].x, qw[nt][k].y, qw[nt][k].z, qw[nt][k].w};
          float x[8], sum = 0.0f;  // (what a small element loses in float16 is nothing beside 8 times the sum)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(u[j] << 16) * up;
            x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u) * (up * 0.0625f);
            sum = fmaf(x[2 * j + 1], 16.0f, sum + x[2 * j]);
          }
          // the order in which a word's codes meet the operand: (0, 4), 16-fold (1, 5), (2, 6), 16-fold (3, 7)
#pragma unroll
          for (int j = 0; j < 4; ++j) qf[nt][k][j] = half2_of(x[j], x[j + 4]);
          sum += __shfl_xor_sync(~0u, sum, 1);
          sum += __shfl_xor_sync(~0u, sum, 2);
#pragma unroll
          for (int c = 0; c < 2; ++c) qoff[nt][k][c] = -0x1p-21f * __shfl_sync(~0u, sum, (2 * t + c) * 4);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          cf[nt][c] = __shfl_sync(~0u, factor, (2 * t + c) * 4);
          const int i = nt * 8 + 2 * t + c;
          if (r0 + i < R) {
            int from, to;
            sees(p, sq, token_of(i), from, to);
            all_lo = max(all_lo, from);
            all_hi = min(all_hi, to);
          }
        }
      }
      all_lo = __reduce_max_sync(~0u, all_lo);
      all_hi = __reduce_min_sync(~0u, all_hi);

      // what P's exponents are counted from, the sum of P
      float ref[NT][2], l[NT][2], O[NT][kMmas][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        ref[nt][0] = ref[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < kMmas; ++i) O[nt][i][0] = O[nt][i][1] = O[nt][i][2] = O[nt][i][3] = 0.0f;
      }

      for (int n = 0; n < count; ++n) {
        const int j0 = first_of(n);
        asm volatile("cp.async.wait_group %0;" ::"n"(Geo::kStages - 2) : "memory");
        __syncwarp();  // the tile is there, and the one before it done with
        copy(n + Geo::kStages - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const uint8_t *stage = ring + n % Geo::kStages * Geo::kStage;
        uint32_t ks[kHalves][2][kScaleWords], vs[kHalves][2];
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          const uint8_t *k = stage + 2 * Geo::kCodes + (16 * f + kr) * (D / 16);
          const uint8_t *v = stage + 2 * Geo::kCodes + Geo::kScales + 16 * f * (D / 16) + g * kDims / 32 * 2;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (kGroups == 1) ks[f][i][0] = *reinterpret_cast<const uint16_t *>(k + 8 * i * (D / 16));
            else shared_words<kScaleWords>(k + 8 * i * (D / 16), ks[f][i]);
            vs[f][i] = __byte_perm(*reinterpret_cast<const uint16_t *>(v + (8 * i + va) * (D / 16)),
                                   *reinterpret_cast<const uint16_t *>(v + (8 * i + vb) * (D / 16)), 0x5410);
          }
        }

        // masks are for tiles that some row sees in part, or with a page that is not there, or with scales that
        // the store does not write
        constexpr uint32_t kTop2 = kTopScale4Bits * 0x10001u;
        uint32_t most = kTop2, some[2 * Geo::kScales / 128];  // the lane's share of all scales
        shared_words<2 * Geo::kScales / 128>(stage + 2 * Geo::kCodes + lane * (2 * Geo::kScales / 32), some);
#pragma unroll
        for (int i = 0; i < 2 * Geo::kScales / 128; ++i) most = __vmaxu2(most, some[i]);
        const bool masks = __any_sync(~0u, most != kTop2) || suspect || j0 < all_lo || j0 + kTile > all_hi;
        unsigned here = 0, poison = 0;  // positions that are there, and those with such scales
        if (masks) {
#pragma unroll
          for (int f = 0; f < kHalves; ++f) {
            const int from = lo - (j0 + 16 * f), to = end - (j0 + 16 * f);
            unsigned wanted = from <= 0 ? 0xFFFFu : from >= 16 ? 0u : (0xFFFFu << from) & 0xFFFFu;
            wanted &= to <= 0 ? 0u : to >= 16 ? 0xFFFFu : 0xFFFFu >> (16 - to);
            if (suspect) {
              const bool own = (wanted >> (lane & 15)) & 1;
              const bool ok = own && (unsigned)ld_input(table + block_of(p, j0 + 16 * f + (lane & 15))) <= last_page;
              if (own && !ok) set_status(p.status, QLIN_ERR_INVALID_ARG);
              wanted = __ballot_sync(~0u, ok) & 0xFFFFu;
            }
            here |= wanted << (16 * f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int k = 0; k < kScaleWords; ++k)
                if ((ks[f][i][k] & 0xFFFFu) > kTopScale4Bits || (ks[f][i][k] >> 16) > kTopScale4Bits)
                  poison |= 1u << (16 * f + 8 * i + kr);
              if ((vs[f][i] & 0xFFFFu) > kTopScale4Bits) poison |= 1u << (16 * f + 8 * i + va);
              if ((vs[f][i] >> 16) > kTopScale4Bits) poison |= 1u << (16 * f + 8 * i + vb);
            }
          }
          poison = __reduce_or_sync(~0u, poison) & here;
          const unsigned zero = ~here | poison;  // values
#pragma unroll
          for (int f = 0; f < kHalves; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if ((zero >> (16 * f + 8 * i + va)) & 1) vs[f][i] &= 0xFFFF0000u;
              if ((zero >> (16 * f + 8 * i + vb)) & 1) vs[f][i] &= 0x0000FFFFu;
            }
        }

        // scores of positions g and g + 8 of each half, columns 2t and 2t + 1
        uint64_t S2[kHalves][NT][2];
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          uint32_t kc[2][kGroups];
          shared_words<kGroups>(stage + (16 * f + kr) * (D / 2) + t * (kGroups * 4), kc[0]);
          shared_words<kGroups>(stage + (16 * f + 8 + kr) * (D / 2) + t * (kGroups * 4), kc[1]);
#pragma unroll
          for (int k = 0; k < kGroups; ++k) {
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w0 = j ? kc[0][k] >> 8 : kc[0][k], w1 = j ? kc[1][k] >> 8 : kc[1][k];
              const uint32_t a[4] = {(w0 & 0x000F000Fu) ^ turn0, (w1 & 0x000F000Fu) ^ turn0,
                                     (w0 & 0x00F000F0u) ^ turn4, (w1 & 0x00F000F0u) ^ turn4};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (j == 0) mma4_from(acc[nt], a, qf[nt][k][0], qf[nt][k][1], qoff[nt][k][0], qoff[nt][k][1]);
                else mma4(acc[nt], a, qf[nt][k][2], qf[nt][k][3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float ki = k & 1 ? half_hi(ks[f][i][k / 2]) : half_lo(ks[f][i][k / 2]);
              const uint64_t k2 = f32x2_pack(ki, ki);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint64_t x = f32x2_pack(acc[nt][2 * i], acc[nt][2 * i + 1]);
                S2[f][nt][i] = k ? f32x2_fma(x, k2, S2[f][nt][i]) : f32x2_mul(x, k2);
              }
            }
          }
        }
        float S[kHalves][NT][4];
#pragma unroll
        for (int f = 0; f < kHalves; ++f)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // rounded here: the differences from the maximum are those of the rounded scores
              const uint64_t x = f32x2_mul(S2[f][nt][i], f32x2_pack(cf[nt][0], cf[nt][1]));
              S[f][nt][2 * i] = __uint_as_float((uint32_t)x);
              S[f][nt][2 * i + 1] = __uint_as_float((uint32_t)(x >> 32));
            }
        if (masks) {
          int vlo[NT][2], vhi[NT][2];  // positions that columns 2t and 2t + 1 see
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int i = nt * 8 + 2 * t + c;
              vlo[nt][c] = lo, vhi[nt][c] = end;  // columns without a row see everything (their q is 0)
              if (r0 + i < R) sees(p, sq, token_of(i), vlo[nt][c], vhi[nt][c]);
            }
#pragma unroll
          for (int f = 0; f < kHalves; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 16 * f + 8 * i + kr, j = j0 + r;
              const bool ok = (here >> r) & 1, bad = (poison >> r) & 1;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float &x = S[f][nt][2 * i + c];
                  if (bad) x = NAN;
                  if (!ok || j < vlo[nt][c] || j >= vhi[nt][c]) x = -INFINITY;
                }
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
          if (__any_sync(~0u, mx[0] - ref[nt][0] > kTop || mx[1] - ref[nt][1] > kTop)) {
            // new references, by the largest scores
            float a[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int o = 4; o < 32; o *= 2) mx[c] = fmaxf(mx[c], __shfl_xor_sync(~0u, mx[c], o));
              const float now = fmaxf(ref[nt][c], fabsf(mx[c]) < kExact ? mx[c] - kBias : mx[c]);
              a[c] = exp2_approx(ref[nt][c] - (now == -INFINITY ? 0.0f : now));
              ref[nt][c] = now;
              l[nt][c] *= a[c];
            }
#pragma unroll
            for (int i = 0; i < kMmas; ++i) {
              O[nt][i][0] *= a[0], O[nt][i][2] *= a[0];
              O[nt][i][1] *= a[1], O[nt][i][3] *= a[1];
            }
          }
          const float z0 = ref[nt][0] == -INFINITY ? 0.0f : ref[nt][0];
          const float z1 = ref[nt][1] == -INFINITY ? 0.0f : ref[nt][1];
#pragma unroll
          for (int f = 0; f < kHalves; ++f) {
            const float(&x)[4] = S[f][nt];
            const float p00 = exp2_approx(x[0] - z0), p01 = exp2_approx(x[1] - z1);
            const float p10 = exp2_approx(x[2] - z0), p11 = exp2_approx(x[3] - z1);
            l[nt][0] += p00 + p10;
            l[nt][1] += p01 + p11;
            pf[f][nt][0] = transpose8x8(half2_of(p00, p01));
            pf[f][nt][1] = transpose8x8(half2_of(p10, p11));
          }
        }

        // O^T += V^T P^T: positions 2t, 2t+1 (and +8) of each half, dimensions g*D/8 ...
        const __half2 k1032 = __half2half2(__ushort_as_half(0x6408));
        const __half2 minus72 = __half2half2(__ushort_as_half(0xD480));
        const __half2 k16th = __half2half2(__ushort_as_half(0x2C00));
#pragma unroll
        for (int f = 0; f < kHalves; ++f) {
          const __half2 s0 = bits_half2(vs[f][0]), s1 = bits_half2(vs[f][1]);
          uint32_t vc[4][kValueWords];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t *v = stage + Geo::kCodes + (16 * f + (i & 1 ? vb : va) + 8 * (i >> 1)) * (D / 2) + g * (kDims / 2);
            if constexpr (kDims == 4) vc[i][0] = *reinterpret_cast<const uint16_t *>(v);
            else shared_words<kValueWords>(v, vc[i]);
          }
#pragma unroll
          for (int i = 0; i < (kDims + 3) / 4; ++i) {  // four dimensions: 16 bits of each row
            const uint32_t *v0 = vc[0], *v1 = vc[1], *v2 = vc[2], *v3 = vc[3];
            const uint32_t x = __byte_perm(v0[i / 2], v1[i / 2], i & 1 ? 0x7632 : 0x5410);
            const uint32_t y = __byte_perm(v2[i / 2], v3[i / 2], i & 1 ? 0x7632 : 0x5410);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t xj = j ? x >> 8 : x, yj = j ? y >> 8 : y;
              const auto low = [&](uint32_t w, __half2 sc) {
                return half2_bits(__hmul2(__hsub2(bits_half2((w & 0x000F000Fu) ^ magic0), k1032), sc));
              };
              const auto high = [&](uint32_t w, __half2 sc) {
                return half2_bits(__hmul2(__hfma2(bits_half2((w & 0x00F000F0u) ^ magic4), k16th, minus72), sc));
              };
              const uint32_t a[4] = {low(xj, s0), high(xj, s0), low(yj, s1), high(yj, s1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma4(O[nt][2 * i + j], a, pf[f][nt][0], pf[f][nt][1]);
            }
          }
        }
      }

      // ---- the warp's result
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          l[nt][0] += __shfl_xor_sync(~0u, l[nt][0], o);
          l[nt][1] += __shfl_xor_sync(~0u, l[nt][1], o);
        }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      float *res = reinterpret_cast<float *>(ring);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t + c;
#pragma unroll
          for (int i = 0; i < kMmas; ++i)
            *reinterpret_cast<float2 *>(res + r * D + g * kDims + 2 * i) = make_float2(O[nt][i][c], O[nt][i][2 + c]);
          if (g == 0) {
            res[kRows * D + r] = ref[nt][c];
            res[kRows * D + kRows + r] = l[nt][c];
          }
        }
    }
    __syncthreads();

    // ---- the CTA's
    const float *results = reinterpret_cast<const float *>(smem);
    const int active = min(tiles, kWarps);
    for (int i = threadIdx.x; i < kRows * D / 4; i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      if (r0 + r >= R) break;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < active) top = fmaxf(top, results[k * Geo::kWarpFloats + kRows * D + r]);
      const float z = top == -INFINITY ? 0.0f : top;
      float L = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        if (k >= active) break;
        const float *x = results + k * Geo::kWarpFloats;
        const float f = exp2_approx(x[kRows * D + r] - z);
        L = fmaf(f, x[kRows * D + kRows + r], L);
        const float4 y = *reinterpret_cast<const float4 *>(x + r * D + d);
        o.x = fmaf(f, y.x, o.x), o.y = fmaf(f, y.y, o.y), o.z = fmaf(f, y.z, o.z), o.w = fmaf(f, y.w, o.w);
      }
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
      if (whole) {
        *reinterpret_cast<uint2 *>(out_row(r) + d) =
            make_uint2((uint32_t)f32_to_bf16_bits(o.x) | ((uint32_t)f32_to_bf16_bits(o.y) << 16),
                       (uint32_t)f32_to_bf16_bits(o.z) | ((uint32_t)f32_to_bf16_bits(o.w) << 16));
      } else {
        *reinterpret_cast<float4 *>(p.o + (slot + r) * D + d) = o;
        if (d == 0) p.sum[slot + r] = make_float2(top, L);
      }
    }
    __syncthreads();
    if (p.list && begins && threadIdx.x == 0 && (!whole || p.by_unit)) {  // the unit begins here
      const int last = s + at.steps - at.at - 1, in_longer = longer * (shortest + 1);
      const int end_range = last < in_longer ? last / (shortest + 1) : longer + (last - in_longer) / shortest;
      p.list[p.by_unit ? (at.b * p.H + h) * p.row_tiles + at.tile : range] =
          JoinEntry{whole ? 0 : end_range - range + 1, range, first ? 0 : 1, h, r0, R, sq.first, 0};
    }
    s += steps_here;
    at.at = 0;
    if (s < s_end) {
      if (++at.tile == at.tiles) {
        at.tile = 0;
        if (++at.h == p.H) {
          at.h = 0;
          do ++at.b;
          while (work_of(at.b, at.tiles, at.steps) == 0);
        }
      }
    }
  }
}

// Joins the parts of a unit: out = sum_s w_s o_s / sum_s w_s with w_s = l_s 2^(m_s - max m), the
// exponent of l_s joined to the other, which alone can be below binary32's range where w_s is not.
struct JoinRow {
  JoinEntry e;
  int rows, r;
  const float2 *sum;
  const float *o;
  __device__ __forceinline__ int64_t slot(int k) const {
    return (int64_t)((e.first + k) * 2 + (k == 0 ? e.first_slot : 0)) * rows + r;
  }
  __device__ __forceinline__ uint16_t *out(const AttnDev &p, int D) const {
    const int rr = e.r0 + r, tok = rr / p.G;
    return p.out + (int64_t)(e.first_token + tok) * p.ldo + (int64_t)(e.h * p.G + rr - tok * p.G) * D;
  }
  __device__ __forceinline__ static float weight(float2 e, float top) {
    const int ex = (int)(__float_as_uint(e.y) >> 23);
    const float mantissa = e.y * __uint_as_float((unsigned)(254 - ex) << 23);
    return mantissa * exp2_approx((e.x - (top == -INFINITY ? 0.0f : top)) + (float)(ex - 127));
  }
};
__device__ __forceinline__ JoinEntry join_entry(const JoinEntry *from) {
  JoinEntry e;
  const uint4 a = ld_input(reinterpret_cast<const uint4 *>(from)), b = ld_input(reinterpret_cast<const uint4 *>(from) + 1);
  e.ranges = a.x, e.first = a.y, e.first_slot = a.z, e.h = a.w, e.r0 = b.x, e.R = b.y, e.first_token = b.z;
  return e;
}

// The sum over parts part, part + step, ... of a row: o += w o_s, W += w.  kBatch parts' loads are in flight at once,
// the first ones' before the largest reference is known; each weight is computed by one lane.
template <int V>
__device__ __forceinline__ void join_parts(const JoinRow &row, int part, int step, int lane, float (&o)[V], float &W) {
  constexpr int kBatch = V >= 8 ? 4 : 8;
  uint32_t x[kBatch][V];
  float2 sum;  // of part `lane` of the batch
  const auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * step;
#pragma unroll
      for (int v = 0; v < V; ++v) x[i][v] = 0u;
      if (k < row.e.ranges) load_words<V>(row.o + row.slot(k) * (32 * V) + lane * V, x[i]);
    }
    const int own = k0 + (lane & (kBatch - 1)) * step;
    sum = own < row.e.ranges ? ld_input(row.sum + row.slot(own)) : make_float2(-INFINITY, 0.0f);
  };
  load(part);
  float top = -INFINITY;
  for (int k = lane; k < row.e.ranges; k += 32) top = fmaxf(top, ld_input(&row.sum[row.slot(k)].x));
  top = warp_max(top);
  for (int k0 = part; k0 < row.e.ranges;) {
    const float w = JoinRow::weight(sum, top);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float wi = k0 + i * step < row.e.ranges ? __shfl_sync(~0u, w, i) : 0.0f;
      W += wi;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = fmaf(wi, __uint_as_float(x[i][v]), o[v]);
    }
    if ((k0 += kBatch * step) < row.e.ranges) load(k0);
  }
}

// Units that few ranges share: a warp for each row of the unit that begins in a range and ends in another.
constexpr int kJoinWarps = 8;
template <int D>
__device__ __forceinline__ void join_of_range(const Int4Params &p, int rows) {
  constexpr int V = D / 32;  // floats of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  JoinRow row{join_entry(p.list + blockIdx.x), rows, 0, p.sum, p.o};
  if (row.e.ranges == 0) return;
  for (row.r = warp; row.r < rows && row.e.r0 + row.r < row.e.R; row.r += kJoinWarps) {
    float o[V], W = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.0f;
    join_parts<V>(row, 0, 1, lane, o, W);
    const float inv = W == 0.0f ? 0.0f : 1.0f / W;
    uint16_t *dst = row.out(p, D) + lane * V;
    if constexpr (V == 1) {
      *dst = f32_to_bf16_bits(o[0] * inv);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int v = 0; v < V / 2; ++v)
        w[v] = (uint32_t)f32_to_bf16_bits(o[2 * v] * inv) | ((uint32_t)f32_to_bf16_bits(o[2 * v + 1] * inv) << 16);
      store_words<V / 2>(dst, w);
    }
  }
}

// Few units, in many parts each: a CTA for each row, its warps over the parts.
constexpr int kManyWarps = 16;
template <int D>
__device__ __forceinline__ void join_of_unit(const Int4Params &p, int rows) {
  constexpr int V = D / 32;
  __shared__ float s_o[kManyWarps][D];
  __shared__ float s_w[kManyWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinRow row{join_entry(p.list + blockIdx.x / rows), rows, (int)blockIdx.x % rows, p.sum, p.o};
  if (row.e.ranges == 0 || row.e.r0 + row.r >= row.e.R) return;
  float o[V], W = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = 0.0f;
  join_parts<V>(row, warp, kManyWarps, lane, o, W);
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = o[v];
  if (lane == 0) s_w[warp] = W;
  __syncthreads();
  if (threadIdx.x < D / 2) {
    const int d = 2 * threadIdx.x;
    float a = 0.0f, c = 0.0f, w = 0.0f;
#pragma unroll
    for (int k = 0; k < kManyWarps; ++k) {
      a += s_o[k][d];
      c += s_o[k][d + 1];
      w += s_w[k];
    }
    const float inv = w == 0.0f ? 0.0f : 1.0f / w;
    *reinterpret_cast<uint32_t *>(row.out(p, D) + d) =
        (uint32_t)f32_to_bf16_bits(a * inv) | ((uint32_t)f32_to_bf16_bits(c * inv) << 16);
  }
}

template <int D, bool BY_UNIT>
__global__ void __launch_bounds__(32 * (BY_UNIT ? kManyWarps : kJoinWarps))
    k_attn_int4_join(const __grid_constant__ Int4Params p, int rows) {
  pdl_wait();
  pdl_trigger();
  if constexpr (BY_UNIT) join_of_unit<D>(p, rows);
  else join_of_range<D>(p, rows);
}

template <int D, int NT, bool EVEN>
cudaError_t launch_nt(const Int4Params &p, const AttnInt4Plan &plan, cudaStream_t st) {
  using Geo = Geometry4<D, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(k_attn_int4<D, NT, EVEN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  e = launch_kernel(k_attn_int4<D, NT, EVEN>, dim3((unsigned)plan.ctas), dim3(kThreads), Geo::kSmem, st, 1, p);
  if (e != cudaSuccess || !plan.joins) return e;
  if (plan.by_unit)
    return launch_kernel(k_attn_int4_join<D, true>, dim3((unsigned)(plan.units * plan.rows)), dim3(32 * kManyWarps), 0, st,
                         1, p, plan.rows);
  return launch_kernel(k_attn_int4_join<D, false>, dim3((unsigned)plan.ctas), dim3(32 * kJoinWarps), 0, st, 1, p, plan.rows);
}
template <int D>
cudaError_t launch_d(const Int4Params &p, const AttnInt4Plan &plan, cudaStream_t st) {
  const bool even = p.block_shift >= 4;
  if constexpr (D < 256)
    if (plan.rows == 16) return even ? launch_nt<D, 2, true>(p, plan, st) : launch_nt<D, 2, false>(p, plan, st);
  return even ? launch_nt<D, 1, true>(p, plan, st) : launch_nt<D, 1, false>(p, plan, st);
}

}  // namespace

// Rows are tiled by 8 where one tile holds them, else by 16: each code is then converted
// for twice the rows, 38 us against 47 for 64 x 2 heads of 128 with 16 queries each.  (Of 256, whose sums of 16 rows
// spill, by 8 always: 87 us against 101.)  As many CTAs as are resident at once, or as there are steps.  Beginnings count where ranges are
// of two steps at least: where they are shorter, those that held nothing else would leave the others longer.
AttnInt4Plan attn_int4_plan(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t rows, int64_t max_kv, int64_t window,
                            int sms) {
  AttnInt4Plan plan{};
  plan.rows = rows <= 8 || D >= 256 ? 8 : 16;
  const int64_t tile = D >= 256 ? 16 : 32, tiles = (rows + plan.rows - 1) / plan.rows, units = B * H * tiles;
  int64_t range = max_kv;  // (a window may be as wide as its type: beyond max_kv it is none, doubled or not)
  if (window > 0) range = std::min(range, 2 * std::min(window, max_kv) + plan.rows / (Hq / H) + 1) + kAlign - 1;
  const int64_t resident = (int64_t)sms * attn_int4_ctas(D, plan.rows);
  plan.step_shift = tile == 16 ? 6 : 7;
  const auto steps_of = [&](int shift) { return std::max<int64_t>(1, (range + ((int64_t)1 << shift) - 1) >> shift); };
  while (units * steps_of(plan.step_shift) > 1 << 29) ++plan.step_shift;  // all steps are counted in 32 bits
  const int64_t steps = steps_of(plan.step_shift);
  plan.start = units * steps >= 2 * resident ? 2 : 0;
  plan.units = (int)units, plan.row_tiles = (int)tiles;
  plan.ctas = (int)std::max<int64_t>(1, std::min(resident, units * steps));
  plan.joins = steps > 1;
  plan.by_unit = units * 8 < plan.ctas;
  if (plan.joins) {
    plan.part_bytes = round_up((size_t)plan.ctas * 2 * plan.rows * (D + 2) * 4, 256);
    plan.ws_bytes = plan.part_bytes + round_up((size_t)(plan.by_unit ? plan.units : plan.ctas) * sizeof(JoinEntry), 256);
  }
  return plan;
}

cudaError_t launch_attn_int4(const AttnArgs &a, const AttnInt4Plan &plan, int few_rows, void *ws, unsigned *status,
                             cudaStream_t st) {
  Int4Params p{};
  static_cast<AttnDev &>(p) = attn_dev(a, few_rows, status);
  p.group_inverse = (65536u + p.G - 1) / p.G;
  p.step_shift = plan.step_shift, p.start = plan.start;
  p.by_unit = plan.by_unit, p.row_tiles = plan.row_tiles;
  p.turn0 = 0x00080008u, p.turn4 = 0x00800080u, p.magic0 = 0x64086408u, p.magic4 = 0x64806480u;
  if (plan.joins) {
    p.o = (float *)ws;
    p.sum = (float2 *)(p.o + (int64_t)plan.ctas * 2 * plan.rows * a.D);
    p.list = (JoinEntry *)((char *)ws + plan.part_bytes);
  }
  switch (a.D) {
    case 32: return launch_d<32>(p, plan, st);
    case 64: return launch_d<64>(p, plan, st);
    case 128: return launch_d<128>(p, plan, st);
    case 256: return launch_d<256>(p, plan, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qlin
