// Attention over the mixed 8-bit KV cache for many rows (prefill, chunks): bound
// by the tensor cores, 4 D flops for each (row, position).
//
// k_attn_unpack converts the positions that some row sees to float16 once, into
// the workspace, as the very images of shared memory that the products read: per
// 128 positions a K-major key tile and a V^T tile (positions along the row), both
// in the 128-byte swizzle, and what the softmax needs beside them.  (Converting
// in the product kernel, by warps of its own, took 1.75 ms against 1.36 ms at
// 8192 new tokens over 16384 positions, 28 heads over 4 of 128: every row tile
// converts the same codes again.)
//
// k_attn_prefill: a CTA takes 256 rows of one (sequence, kv head), packed
// token-major over the heads of the group, as two row tiles A and B of 128, and
// walks over the position tiles, each one contiguous bulk copy.  Where that would
// leave multiprocessors idle, several CTAs share the positions and a join follows.
// Roles:
//   * warps 0-3 and 4-7: softmax of tile A and of tile B, a thread per row.  S
//     comes from tensor memory, P goes back there (over S) as float16.
//   * warp 8: copies; warp 9: issues S = Q K^T (both from shared memory) and
//     O += P V (P from tensor memory).  While one tile's softmax runs, the other's
//     products do.
//
// Scaling.  q rows are scaled by powers of two to use float16's range.  The keys
// of 32 (D 128) or 64 (D 64) positions, a unit, are scaled by code scale * 2^-ek
// and the values by 2^-ev, with one exponent each for the unit (where its key or
// value scales lie too far apart for float16, one for each position: a position that
// a row does not see leaves that row's others in place), so float16 holds
// them whatever the cache's scales; 2^ek joins the score's factor and ev the
// exponent, so that neither costs the softmax an instruction per score.  O is
// rescaled only where a row's maximum grew by more than 2^6 since its reference;
// P stays below 2^14.  Positions whose value scale is 0 do not raise that
// reference (they would push P of the others out of float16): they count in the
// sum of the row alone, which for that has a reference of its own.  Scores too large
// for a reference in binary32 to be exact enough go the same rare way as wide units.
#include <algorithm>

#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace qlin {

namespace {

using namespace tc;

constexpr int kPos = 128;       // positions of a tile
constexpr int kRowTile = 128;   // rows of an MMA
constexpr int kSoftmaxWarps = 8;
constexpr int kCopier = 8, kIssuer = 9;
constexpr int kThreads = 320;
constexpr int kMetaSlots = 4;
constexpr float kPBias = 8.0f;  // P is 2^8 p: float16's subnormals lie below 2^-22 p
constexpr float kGrowth = 6.0f;
constexpr float kLead = 32.0f;  // a score may pass the sum's reference by 2^this where O has another
constexpr float kHuge = 0x1p24f;  // scores up to here have a reference good to 1/2: P stays below 2^14.5
constexpr int kValueUp = 6;     // a value's scale becomes 2^6..2^7 (times at most 448: below float16's 65504)
constexpr int kValueSpan = 11;  // scales of a unit within 2^11 share an exponent: E4M3's 2^-9 stays normal
constexpr int kKeySpan = 14;    // key scales within 2^14: a code of 1 stays normal
constexpr int kWide = 1024;     // added to TileMeta::code

// What the softmax needs of a position tile beside S, per 32 positions: the
// exponents of keys and values, positions present, positions whose value is not
// finite (zero in the tile, so that P = 0 leaves it alone), and (bits of `wide`) whether the
// scales of keys or values lie too far apart for one exponent.  `code` is the largest ek, and
// kWide more where something is wide.
struct __align__(16) TileMeta {
  int ek[4], ev[4];
  unsigned valid[4], poison[4];
  int code;
  unsigned wide;
};
// Of a position of a wide word: 2^ek of its key, and ev of its value (-inf: scale 0).
struct __align__(8) PositionMeta {
  float up_k, ev;
};

template <int D>
struct Config {
  static constexpr int kChunks = D / 16;             // 16-byte pieces of a row of codes
  static constexpr int kUnit = 256 / kChunks;        // positions of a unit (4 KB of codes)
  static constexpr int kUnits = kPos / kUnit;        // units of a key (or value) tile
  static constexpr int kQBytes = kRowTile * D * 2;   // a row tile of q
  static constexpr int kTileBytes = kPos * D * 2;    // a key or value tile
  static constexpr int kSub = kRowTile * 128;        // a 128-byte-wide column of a q or key tile
  static constexpr int kVSub = D * 128;              // 64 positions of V^T
  static constexpr int kKAt = 2 * kQBytes, kVAt = kKAt + 2 * kTileBytes, kBarAt = kVAt + 2 * kTileBytes;
  static constexpr int kSmem = kBarAt + 4096 + 1024;  // barriers and metadata; alignment
  static constexpr int kImage = 2 * kTileBytes;       // a position tile in the workspace
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  // tensor memory columns: S (P over it) of A and B, then O
  static constexpr int kS = 0, kO = 2 * kPos, kColumns = 512;
  static constexpr uint32_t kIdescS = umma_idesc(0, 0, kRowTile, kPos), kIdescO = umma_idesc(0, 0, kRowTile, D);
};

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], meta_full[kMetaSlots];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];  // of row tiles A and B
  uint32_t tmem;
  int abort;
  const PositionMeta *positions;  // of the CTA's first tile (here, since the common loop has no register for it)
  TileMeta meta[kMetaSlots];
};

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  mma_bf16(d, a, b, idesc, acc);  // kind::f16; the operand type is in the descriptor
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  mma_bf16_ts(d, a, b, idesc, acc);
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Values of a tcgen05.ld: not used before this point (which follows its wait).
__device__ __forceinline__ void tie(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ float f32x2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f32x2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Byte offset of 16-byte unit `u` of row `r` in a tile of 128-byte rows under the
// 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

struct PrefillParams : AttnDev {
  int row_tiles, tiles;      // row tiles (of A and B together) and position tiles of a sequence
  int head0, heads;          // kv heads of this pass
  AttnParts parts;           // splits > 1: parts of chunk position tiles, a CTA each (all heads in one pass)
  int chunk;
  uint8_t *images;           // [B, heads, tiles] key and value tile
  TileMeta *meta;            // [B, heads, tiles]
  PositionMeta *positions;   // [B, heads, tiles, kPos]
};

__device__ __forceinline__ float half_at(uint32_t w, int i) {
  return __half2float(__ushort_as_half((uint16_t)(w >> (16 * i))));
}

// One position tile of one (sequence, kv head): a warp for each unit of keys and
// of values.  A lane holds the codes of 16 dimensions (chunk lane % C) of positions
// 8 * (lane / C) + i.
template <int D>
__global__ void __launch_bounds__(64 * Config<D>::kUnits) k_attn_unpack(const PrefillParams p) {
  using C = Config<D>;
  constexpr int kWords = C::kUnit / 32;  // 32-position words of a unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = (int)(blockIdx.x % p.tiles);
  const int hh = (int)(blockIdx.x / p.tiles % p.heads), b = (int)(blockIdx.x / p.tiles / p.heads);
  const int h = p.head0 + hh;
  pdl_wait();
  pdl_trigger();
  const Sequence sq = sequence(p, b);
  if (sq.kept * p.G <= p.few_rows || sq.kept == 0) return;
  int lo, hi, unused;  // positions that some row sees
  sees(p, sq, 0, lo, unused);
  sees(p, sq, sq.kept - 1, unused, hi);
  if ((tile + 1) * kPos <= lo || tile * kPos >= hi) return;

  const bool value = warp >= C::kUnits;
  const int block = value ? warp - C::kUnits : warp;
  const int chunk = lane % C::kChunks, octet = lane / C::kChunks;
  const int64_t at_tile = ((int64_t)b * p.heads + hh) * p.tiles + tile;
  uint8_t *image = p.images + at_tile * C::kImage + (value ? C::kTileBytes : 0);
  TileMeta &tm = p.meta[at_tile];
  PositionMeta *pm = p.positions + at_tile * kPos;

  // rows (slot, head) of the lane's positions, and which are there
  const int32_t *table = p.block_table + (int64_t)b * p.max_blocks;
  int64_t row[kWords];
  unsigned valid[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int j = tile * kPos + block * C::kUnit + i * 32 + lane, blk = block_of(p, j);
    const bool wanted = j >= lo && j < hi;
    const int page = wanted ? ld_input(table + blk) : -1;
    const bool ok = page >= 0 && page < p.num_blocks;
    if (wanted && !ok) set_status(p.status, QLIN_ERR_INVALID_ARG);
    valid[i] = __ballot_sync(~0u, ok);
    row[i] = ok ? ((int64_t)page * p.block_size + (j - blk * p.block_size)) * p.H + h : 0;
  }
  const uint8_t *codes = (value ? p.vc : p.kc) + chunk * 16;
  uint4 code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = octet * 8 + i;
    int64_t at = __shfl_sync(~0u, row[0], t & 31);
    unsigned there = valid[0];
    if constexpr (kWords == 2) {
      const int64_t other = __shfl_sync(~0u, row[1], t & 31);
      if (t >= 32) at = other, there = valid[1];
    }
    code[i] = (there >> (t & 31)) & 1 ? ld_input(reinterpret_cast<const uint4 *>(codes + at * D))
                                      : make_uint4(0, 0, 0, 0);
  }
  uint32_t scale[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if (!((valid[i] >> lane) & 1)) continue;
    if (value) {
      scale[i] = ld_input(p.vs + row[i]);
    } else if constexpr (kWords == 1) {
      const uint2 w = ld_input(reinterpret_cast<const uint2 *>(p.ks + row[0] * (D / 32)));
      scale[0] = w.x, scale[1] = w.y;
    } else {
      scale[i] = ld_input(reinterpret_cast<const uint32_t *>(p.ks + row[i] * (D / 32)));
    }
  }
  // exponent e of a scale, 2^e <= |s| < 2^(e+1); those that are not finite count as the largest
  const auto exponent = [](uint32_t abs_bits) { return min((int)(abs_bits >> 23) - 127, 15); };
  // of the unit's largest and smallest scale (zeros apart)
  unsigned top = 0x33800000u, low = 0x7F800000u;  // 2^-24, float16's smallest
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned a = __float_as_uint(fabsf(half_at(scale[i / 2], i % 2)));
    top = max(top, a);
    low = a ? min(low, a) : low;
  }
  const int e = exponent(__reduce_max_sync(~0u, top));
  const int span = e - min(exponent(__reduce_min_sync(~0u, low)), e);
  bool nothing = false;  // a position there with a value scale of 0
#pragma unroll
  for (int i = 0; i < kWords; ++i) nothing |= value && ((valid[i] >> lane) & 1) && (scale[i] & 0x7FFFu) == 0;
  const bool wide = __any_sync(~0u, nothing) || span > (value ? kValueSpan : kKeySpan);
  __shared__ int s_code[2 * C::kUnits];
  if (lane == 0) s_code[warp] = (wide ? kWide : 0) + (value ? -kWide / 4 : e);
  __syncthreads();
  // the positions' own figures are written where either their keys or their values are wide
  const bool write_own = max(s_code[block], s_code[block + C::kUnits]) >= kWide / 2;
  if (threadIdx.x == 0) {
    int most = -kWide;
    unsigned words = 0;
#pragma unroll
    for (int i = 0; i < C::kUnits; ++i) {
      const bool own = max(s_code[i], s_code[i + C::kUnits]) >= kWide / 2;
      most = max(most, s_code[i] - (s_code[i] >= kWide / 2 ? kWide : 0));
      if (own) words |= (kWords == 1 ? 1u : 3u) << (i * kWords);
    }
    tm.code = most + (words ? kWide : 0);
    tm.wide = words;
  }

  if (!value) {
    if (lane < kWords) {
      tm.ek[block * kWords + lane] = e;
      tm.valid[block * kWords + lane] = lane == 0 ? valid[0] : valid[kWords - 1];
    }
    uint32_t sw[2];
    int ep = e;  // of the position whose scales word i holds
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < kWords) {
        uint32_t most = __vmaxu2(scale[i] & 0x7FFF7FFFu, kWords == 1 ? scale[1] & 0x7FFF7FFFu : 0u);
        most = max(most & 0xFFFFu, most >> 16);
        ep = wide && most ? exponent(__float_as_uint(half_at(most, 0))) : e;
        if (write_own) pm[block * C::kUnit + i * 32 + lane].up_k = pow2i(ep);
      }
      const float down = pow2i(-ep);
      sw[i] = half2_of(half_at(scale[i], 0) * down, half_at(scale[i], 1) * down);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = octet * 8 + i, r = block * C::kUnit + t;
      const uint32_t w0 = __shfl_sync(~0u, sw[0], t & 31), w1 = __shfl_sync(~0u, sw[1], t & 31);
      const uint32_t w = (kWords == 1 ? chunk >= 4 : t >= 32) ? w1 : w0;
      const __half2 sc = bits_half2(__byte_perm(w, w, chunk & 2 ? 0x3232 : 0x1010));
      const uint32_t c[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int8x4_to_half(c[k], o[2 * k], o[2 * k + 1]);
        o[2 * k] = half2_bits(__hmul2(bits_half2(o[2 * k]), sc));
        o[2 * k + 1] = half2_bits(__hmul2(bits_half2(o[2 * k + 1]), sc));
      }
      uint8_t *dst = image + (chunk / 4) * C::kSub;
      *reinterpret_cast<uint4 *>(dst + swizzled(r, (chunk % 4) * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4 *>(dst + swizzled(r, (chunk % 4) * 2 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    return;
  }

  // Values that are not finite: zeros in the tile, and a mark.
  unsigned poison[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) poison[i] = __ballot_sync(~0u, (scale[i] & 0x7FFFu) >= 0x7C00u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bad = __vcmpeq4(code[i].x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                         __vcmpeq4(code[i].y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                         __vcmpeq4(code[i].z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                         __vcmpeq4(code[i].w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const unsigned who = __ballot_sync(~0u, bad != 0);
    if (who == 0) continue;
    if ((who >> (octet * C::kChunks)) & ((1u << C::kChunks) - 1)) code[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int o = 0; o < 32 / C::kChunks; ++o)
      if ((who >> (o * C::kChunks)) & ((1u << C::kChunks) - 1)) poison[o / 4] |= 1u << ((o % 4) * 8 + i);
  }
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    if ((poison[i] >> lane) & 1) scale[i] = 0;
  // (e stands for the scales as loaded: one that is not finite only makes it the largest)
  if (lane < kWords) {
    tm.ev[block * kWords + lane] = e - kValueUp;
    tm.poison[block * kWords + lane] = lane == 0 ? poison[0] : poison[kWords - 1];
  }
  // scales as float16, the octet's then two positions at a time
  uint32_t sw[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const float s = half_at(scale[i], 0);
    const unsigned a = __float_as_uint(fabsf(s));
    const int es = wide && a ? exponent(a) : e;
    if (write_own) pm[block * C::kUnit + i * 32 + lane].ev = a ? (float)(es - kValueUp) : -INFINITY;
    const uint32_t w = __half_as_ushort(__float2half_rn(s * pow2i(kValueUp - es)));
    sw[i] = w | (__shfl_down_sync(~0u, w, 1) << 16);
  }
  __half2 sc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = octet * 8 + 2 * i;
    uint32_t w = __shfl_sync(~0u, sw[0], t & 31);
    if constexpr (kWords == 2) {
      const uint32_t other = __shfl_sync(~0u, sw[1], t & 31);
      if (t >= 32) w = other;
    }
    sc[i] = bits_half2(w);
  }
  const int first = block * C::kUnit + octet * 8;  // position within the tile
  uint8_t *dst = image + (first / 64) * C::kVSub;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 &c0 = code[2 * i], &c1 = code[2 * i + 1];
        const uint32_t s0 = w == 0 ? c0.x : w == 1 ? c0.y : w == 2 ? c0.z : c0.w;
        const uint32_t s1 = w == 0 ? c1.x : w == 1 ? c1.y : w == 2 ? c1.z : c1.w;
        const uint32_t two = __byte_perm(s0, s1, k | ((4 + k) << 4));
        o[i] = half2_bits(__hmul2(bits_half2(e4m3x2_to_half((uint16_t)two)), sc[i]));
      }
      *reinterpret_cast<uint4 *>(dst + swizzled(chunk * 16 + w * 4 + k, first % 64 / 8)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_prefill(const PrefillParams p) {
  using C = Config<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Shared &sh = *reinterpret_cast<Shared *>(smem + C::kBarAt);
  static_assert(sizeof(Shared) <= 4096, "barrier area");
  volatile int *abort_flag = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the last row tiles see the most positions: they go first
  const int heads = p.B * p.heads, split = (int)(blockIdx.x % p.parts.splits);
  const unsigned unit = blockIdx.x / p.parts.splits;
  const int tile = p.row_tiles - 1 - (int)(unit / heads);
  const int b = (int)(unit % heads) / p.heads, h = p.head0 + (int)(unit % heads) % p.heads;
  pdl_wait();
  const Sequence sq = sequence(p, b);
  if (sq.broken && h == 0 && tile == 0 && split == 0 && threadIdx.x == 0) set_status(p.status, QLIN_ERR_INVALID_ARG);
  const int R = sq.kept * p.G, r0 = tile * 2 * kRowTile;
  if (r0 >= R || R <= p.few_rows) return;

  // positions any row sees [beg, end), every row sees [all_lo, all_hi)
  int beg, end, all_lo, all_hi;
  const int last = min(r0 + 2 * kRowTile, R) - 1;
  sees(p, sq, r0 / p.G, beg, all_hi);
  sees(p, sq, last / p.G, all_lo, end);
  const int lo = beg;
  int tile0 = beg / kPos, n = end > lo ? (end + kPos - 1) / kPos - tile0 : 0;
  if (p.parts.splits > 1) {  // this CTA's part; the last one takes what is left
    const int skip = min(split * p.chunk, n);
    tile0 += skip;
    n -= skip;
    if (split < p.parts.splits - 1) n = min(n, p.chunk);
  }
  beg = tile0 * kPos;
  // of row r: where the parts' results go
  const auto part_row = [&](int r) {
    const int64_t unit_at = ((int64_t)b * p.H + h) * p.row_tiles + tile;
    return (unit_at * p.parts.splits + split) * p.parts.rows + (r - r0);
  };

  if (n == 0) {  // rows that see nothing
    for (int i = threadIdx.x; i < (last - r0 + 1) * (D / 8); i += kThreads) {
      const int r = r0 + i / (D / 8);
      if (p.parts.splits > 1) {
        float4 *o = reinterpret_cast<float4 *>(p.parts.o + part_row(r) * D) + i % (D / 8) * 2;
        o[0] = o[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i % (D / 8) == 0) p.parts.sum[part_row(r)] = make_float2(-INFINITY, 0.0f);
        continue;
      }
      uint16_t *dst = p.out + (int64_t)(sq.first + r / p.G) * p.ldo + (int64_t)(h * p.G + r % p.G) * D;
      reinterpret_cast<uint4 *>(dst)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], kSoftmaxWarps / 2);
      mbar_init(&sh.p_full[i], kSoftmaxWarps / 2);
      mbar_init(&sh.o_full[i], 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(&sh.meta_full[i], 1);
    sh.abort = 0;
    sh.positions = p.positions + (((int64_t)b * p.heads + (h - p.head0)) * p.tiles + tile0) * kPos;
    fence_barrier_init();
  }
  if (warp == kIssuer) tmem_alloc(&sh.tmem, C::kColumns);

  // q rows -> float16 in shared memory, by the softmax threads
  float row_factor = 0.0f;
  bool some = false;  // something but zeros
  const int r = r0 + threadIdx.x;  // a softmax thread's row
  if (warp < kSoftmaxWarps) {
    uint4 w[D / 8];
    float top = 0.0f;
    const uint16_t *src = p.q + (int64_t)(sq.first + r / p.G) * p.ldq + (int64_t)(h * p.G + r % p.G) * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      w[i] = r < R ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
    }
    const int e = q_exponent(top);
    // a negative softmax scale turns q around, so that the score's factor is positive
    const float up = p.scale_log2 < 0.0f ? -pow2i(14 - e) : pow2i(14 - e);
    row_factor = fabsf(p.scale_log2) * pow2i(max(e - 14, -126));
    some = top > 0.0f && row_factor > 0.0f;
    const uint32_t at = smem_u32(smem) + (warp >> 2) * C::kQBytes;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = half2_of(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xFFFF0000u) * up);
      sts128(at + (i / 8) * C::kSub + swizzled(threadIdx.x % kRowTile, i % 8), make_uint4(o[0], o[1], o[2], o[3]));
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // Dependents start only now: a linear's CTA, once resident, takes tensor memory and keeps it
  // until this kernel has ended, which a CTA still waiting for its columns would never do.
  pdl_trigger();

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------- softmax
    const int half = warp >> 2;  // tile A or B
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // lanes 32 * (warp % 4)
    const uint32_t s_at = at + C::kS + half * kPos, o_at = at + C::kO + half * D;
    int row_lo = lo, row_hi = end;
    if (r < R) sees(p, sq, r / p.G, row_lo, row_hi);
    // O is sum p v under the reference m + m_v (m_v: a value's exponent), l is sum p under m_l
    float m = -INFINITY, m_v = 0.0f, m_l = -INFINITY, l = 0.0f;
    bool ok = true;
    int j = 0;
    // Keys whose exponent passes this may give scores beyond kHuge, whose reference is rounded by
    // more than P in float16 can bear: |S| is below 2^15 * 254 * D.  (Rows of zeros have factor 1.)
    const int ek_most = __reduce_min_sync(
        ~0u, some ? (int)fminf(floorf(log2f(kHuge / (0x1p15f * 254.0f * D)) - log2f(row_factor)), 100.0f) : 100);
    const auto arrives = [&] {  // S of tile j, with its metadata
      ok = mbar_wait(&sh.meta_full[j % kMetaSlots], (j / kMetaSlots) & 1, abort_flag) &&
           mbar_wait(&sh.s_full[half], j & 1, abort_flag);
      tc_fence_after();
      return __all_sync(~0u, ok) != 0;
    };
    // Scores this row does not see become -inf, those of a NaN value NaN (32 columns
    // from c * 32 on).
    const auto mask = [&](const TileMeta &tm, int c, uint32_t (&s)[32]) {
      const int at_c = beg + j * kPos + c * 32, from = row_lo - at_c, to = row_hi - at_c;
      unsigned seen = tm.valid[c];
      seen &= from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
      seen &= to <= 0 ? 0u : to >= 32 ? ~0u : ~(~0u << to);
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = (seen >> i) & 1 ? s[i] : 0xFF800000u;
      const unsigned bad = tm.poison[c] & seen;
      if (bad) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = (bad >> i) & 1 ? 0x7FFFFFFFu : s[i];
      }
    };
    // a score's factor (never 0, so that -inf stays -inf)
    const auto factor = [&](int ek) { return fmaxf(row_factor * pow2i(ek), 0x1p-100f); };
    const auto rescale = [&](float a) {  // O under a new reference
      if (j == 0) return;
#pragma unroll 1
      for (int k = 0; k < D / 16; ++k) {
        uint32_t o[16];
        tmem_ld16(o_at + k * 16, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
        tmem_st16(o_at + k * 16, o);
      }
    };
    const auto hand_over = [&](uint64_t *bar) {  // P up to here
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    // Tiles with one exponent for each 32 positions, and scores within kHuge: m_v is 0 and m_l is m.
    const auto common = [&] {
      for (; j < n; ++j) {
        if (!arrives()) break;
        const TileMeta &tm = sh.meta[j % kMetaSlots];
        if (tm.code > ek_most) break;
        const int j0 = beg + j * kPos;
        const bool full = j0 >= all_lo && j0 + kPos <= all_hi && j0 >= lo &&
                          (tm.valid[0] & tm.valid[1] & tm.valid[2] & tm.valid[3]) == ~0u &&
                          (tm.poison[0] | tm.poison[1] | tm.poison[2] | tm.poison[3]) == 0;
        // The row's largest exponent.  P of the first half of the scores goes over them, so
        // they stay in registers; those of the second half (columns that P leaves alone)
        // are read again: 128 registers of scores spill (1173 us against 1162).
        uint32_t s[4][32];
        float f[4];
        int ev[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f[c] = factor(tm.ek[c]);
          ev[c] = tm.ev[c];
        }
        float now = m;
        const auto maximum = [&](int c, const uint32_t (&s)[32]) {
          float t[4];  // four chains
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = __uint_as_float(s[i]);
#pragma unroll
          for (int i = 4; i < 32; ++i) t[i % 4] = fmaxf(t[i % 4], __uint_as_float(s[i]));
          now = fmaxf(now, fmaf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), f[c], (float)ev[c]));
        };
        const auto arrived = [&](int c) {
          tmem_ld_wait();
          tie(s[c]);
          if (__builtin_expect(!full, 0)) mask(tm, c, s[c]);
        };
        tmem_ld32(s_at + 2 * 32, s[2]);
        arrived(2);
        tmem_ld32(s_at + 3 * 32, s[3]);
        maximum(2, s[2]);
        arrived(3);
        tmem_ld32(s_at, s[0]);
        maximum(3, s[3]);
        arrived(0);
        tmem_ld32(s_at + 32, s[1]);
        maximum(0, s[0]);
        arrived(1);
        maximum(1, s[1]);
        if (__any_sync(~0u, now > m + kGrowth)) {
          // a new reference: what was summed under the old one is scaled down
          const bool grew = now > m + kGrowth;
          const float a = grew ? exp2_approx(m - now) : 1.0f;
          if (grew) m = now;
          l *= a;
          rescale(a);
        }
        // P = 2^(s + ev - m + bias), over S
        const float z = kPBias - (m == -INFINITY ? 0.0f : m);
        const auto probabilities = [&](int k, const uint32_t (&s)[32]) {
          const float g = (float)ev[k] + z;
          const uint64_t f2 = f32x2_pack(f[k], f[k]), g2 = f32x2_pack(g, g);
          uint64_t sum2[2] = {0, 0};
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t x = f32x2_fma((uint64_t)s[2 * i] | ((uint64_t)s[2 * i + 1] << 32), f2, g2);
            const float a = exp2_approx(f32x2_lo(x)), e = exp2_approx(f32x2_hi(x));
            sum2[i & 1] = f32x2_add(sum2[i & 1], f32x2_pack(a, e));
            o[i] = half2_of(a, e);
          }
          sum2[0] = f32x2_add(sum2[0], sum2[1]);
          l += (f32x2_lo(sum2[0]) + f32x2_hi(sum2[0])) * pow2i(-ev[k]);
          tmem_st16(s_at + k * 16, o);
        };
        tmem_ld32(s_at + 2 * 32, s[2]);
        probabilities(0, s[0]);
        probabilities(1, s[1]);
        arrived(2);
        tmem_ld32(s_at + 3 * 32, s[3]);
        hand_over(&sh.p_half[half]);  // the first half of P: its products start
        probabilities(2, s[2]);
        arrived(3);
        probabilities(3, s[3]);
        hand_over(&sh.p_full[half]);
      }
      m_l = m;
    };
    // Other tiles are rare: a loop of their own with 32 scores at a time, in few registers (as a case of
    // the one above it cost that one 1342 us against 1169 at 8192 x 16384, 28 heads over 4 of 128).
    uint32_t s[32];
    const auto scores = [&](const TileMeta &tm, int c) {
      tmem_ld32(s_at + c * 32, s);
      tmem_ld_wait();
      tie(s);
      mask(tm, c, s);
    };
    // The figures of position c * 32 + lane; others read them by shuffles (as loads, 32 at once spill).
    const auto own_of = [&](const TileMeta &tm, int c) {
      if ((tm.wide >> c) & 1) return sh.positions[j * kPos + c * 32 + lane];
      return PositionMeta{pow2i(tm.ek[c]), (float)tm.ev[c]};
    };
    // A word of 32 positions that is wide, or whose scores may be huge, is taken position by position:
    // differences of scores, which are exact near the maximum, before the exponents of the values are
    // added.  l has a reference of its own, since scores without a value do not raise m.  True: the next
    // tile is common(), O is under m alone and l under m again.  (2048 of 8192 positions, 28 heads over 4
    // of 128: 236 us; with one such word 228 to 244, with all of them 407.)
    const auto general = [&] {
      for (; j < n; ++j) {
        if (!arrives()) break;
        const TileMeta &tm = sh.meta[j % kMetaSlots];
        if (tm.code <= ek_most && __all_sync(~0u, (m_l == m || m_l - m < 60.0f) && (m_v == 0.0f || fabsf(m) < 0x1p20f))) {
          m += m_v, m_v = 0.0f;
          if (m_l > -INFINITY) l *= exp2_approx(m_l - m);
          return true;
        }
        const unsigned single = tm.code - (tm.code >= kWide / 2 ? kWide : 0) > ek_most ? ~0u : tm.wide;
        float now[2] = {m, m}, now_v[2] = {m_v, m_v}, top = m_l;  // two chains
        const auto larger = [&](int k, float x, float e) {
          if ((x - now[k]) + (e - now_v[k]) > 0.0f) now[k] = x, now_v[k] = e;
        };
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          scores(tm, c);
          const PositionMeta own = own_of(tm, c);
          if ((single >> c) & 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float f = fmaxf(row_factor * __shfl_sync(~0u, own.up_k, i), 0x1p-100f);
              const float x = __fmul_rn(__uint_as_float(s[i]), f);  // rounded, wherever it is used
              larger(i % 2, x, __shfl_sync(~0u, own.ev, i));
              top = fmaxf(top, x);
            }
          } else {
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; ++i) t[i % 4] = fmaxf(t[i % 4], __uint_as_float(s[i]));
            const float x = __fmul_rn(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), factor(tm.ek[c]));
            larger(0, x, (float)tm.ev[c]);
            top = fmaxf(top, x);
          }
        }
        larger(0, now[1], now_v[1]);
        const float by = (now[0] - m) + (now_v[0] - m_v);
        if (top - m_l > kLead) {
          l *= exp2_approx(m_l - top);
          m_l = top;
        }
        if (__any_sync(~0u, by > kGrowth)) {
          const float a = by > kGrowth ? exp2_approx(-by) : 1.0f;
          if (by > kGrowth) m = now[0], m_v = now_v[0];
          rescale(a);
        }
        const float m_0 = m == -INFINITY ? 0.0f : m, l_0 = m_l == -INFINITY ? 0.0f : m_l;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          scores(tm, c);
          const PositionMeta own = own_of(tm, c);
          uint32_t o[16];
          float sum = 0.0f;
          if ((single >> c) & 1) {
            const auto one = [&](int i) {
              const float f = fmaxf(row_factor * __shfl_sync(~0u, own.up_k, i), 0x1p-100f);
              const float x = __fmul_rn(__uint_as_float(s[i]), f), e = __shfl_sync(~0u, own.ev, i);
              sum += exp2_approx((x - l_0) + kPBias);
              return exp2_approx((x - m_0) + (e - m_v + kPBias));
            };
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float a = one(2 * i), e = one(2 * i + 1);
              o[i] = half2_of(a, e);
            }
          } else {
            const float f = factor(tm.ek[c]), g = (float)tm.ev[c] - m_v + kPBias - m_0;
            const uint64_t f2 = f32x2_pack(f, f), g2 = f32x2_pack(g, g);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x = f32x2_fma((uint64_t)s[2 * i] | ((uint64_t)s[2 * i + 1] << 32), f2, g2);
              const float a = exp2_approx(f32x2_lo(x)), e = exp2_approx(f32x2_hi(x));
              sum += a + e;
              o[i] = half2_of(a, e);
            }
            sum *= pow2i(-tm.ev[c]) * exp2_approx((m_0 - l_0) + m_v);
          }
          l += sum;
          tmem_st16(s_at + c * 16, o);
          if (c & 1) hand_over(c == 1 ? &sh.p_half[half] : &sh.p_full[half]);
        }
      }
      return false;
    };
    do common();
    while (j < n && __all_sync(~0u, ok) && general());
    if (__all_sync(~0u, ok)) ok = mbar_wait(&sh.o_full[half], 0, abort_flag);
    if (__all_sync(~0u, ok)) {
      tc_fence_after();
      // 2^(m + m_v - m_l) goes on in two halves: it can be below binary32's range where its product with O is not
      const float half_to = m == -INFINITY ? 0.0f : exp2_approx(0.5f * ((m - m_l) + m_v));
      const float inv = l == 0.0f ? 0.0f : half_to / l;
      const auto out = [&](uint32_t x) { return (__uint_as_float(x) * half_to) * inv; };
      uint16_t *dst = p.out + (int64_t)(sq.first + r / p.G) * p.ldo + (int64_t)(h * p.G + r % p.G) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_at + c * 32, o);
        tmem_ld_wait();
        if (p.parts.splits > 1) {
          if (r < R) {
            float4 *to = reinterpret_cast<float4 *>(p.parts.o + part_row(r) * D + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              to[i] = make_float4(out(o[4 * i]), out(o[4 * i + 1]), out(o[4 * i + 2]), out(o[4 * i + 3]));
            if (c == 0) p.parts.sum[part_row(r)] = make_float2(m_l, l);
          }
          continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = (uint32_t)f32_to_bf16_bits(out(o[2 * i])) | ((uint32_t)f32_to_bf16_bits(out(o[2 * i + 1])) << 16);
        if (r < R) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4 *>(dst + c * 32)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
    } else {
      *abort_flag = 1;
    }
    tc_fence_before();
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t base = smem_u32(smem);
      const auto scores = [&](int half, int j) {
        const uint64_t a = umma_desc_sw128(base + half * C::kQBytes);
        const uint64_t bd = umma_desc_sw128(base + C::kKAt + (j & 1) * C::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (uint64_t)((k / 4) * (C::kSub >> 4) + (k % 4) * 2);
          mma_f16_ss(tmem + C::kS + half * kPos, a + step, bd + step, C::kIdescS, k > 0);
        }
        mma_commit(&sh.s_full[half]);
      };
      // O += P V over 64 of the positions
      const auto outputs = [&](int half, int j, int part) {
        const uint64_t bd = umma_desc_sw128(base + C::kVAt + (j & 1) * C::kTileBytes + part * C::kVSub);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(tmem + C::kO + half * D, tmem + C::kS + half * kPos + (part * 4 + k) * 8, bd + (uint64_t)(k * 2),
                     C::kIdescO, j > 0 || part > 0 || k > 0);
      };
      bool ok = mbar_wait(&sh.k_full[0], 0, abort_flag);
      if (ok) {
        tc_fence_after();
        scores(0, 0);
        scores(1, 0);
        mma_commit(&sh.k_empty[0]);
      }
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        ok = mbar_wait(&sh.v_full[j & 1], (j >> 1) & 1, abort_flag);
        for (int half = 0; half < 2 && ok; ++half) {
          ok = mbar_wait(&sh.p_half[half], j & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          outputs(half, j, 0);
          ok = mbar_wait(&sh.p_full[half], j & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          outputs(half, j, 1);
          if (half) mma_commit(&sh.v_empty[j & 1]);
          if (more) {
            ok = half || mbar_wait(&sh.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            scores(half, j + 1);  // over P: products run in the order of issue
            if (half) mma_commit(&sh.k_empty[(j + 1) & 1]);
          } else {
            mma_commit(&sh.o_full[half]);
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // every commit's arrival lands before the CTA leaves: the last one covers all
      if (ok) {
        mbar_wait_drain(&sh.o_full[1], 0);
      } else {
        mma_commit(&sh.o_full[1]);
        mbar_wait_drain(&sh.o_full[1], 0);
      }
    }
    __syncwarp();
  } else if (warp == kCopier) {
    // --------------------------------------------------------------- copies
    if (lane == 0) {
      const int64_t first = ((int64_t)b * p.heads + (h - p.head0)) * p.tiles + tile0;
      const uint8_t *src = p.images + first * C::kImage;
      bool ok = true;
      int j = 0;
      for (; j < n && ok; ++j) {
        const int s = j & 1;
        const uint32_t parity = ((j >> 1) & 1) ^ 1;
        ok = mbar_wait(&sh.k_empty[s], parity, abort_flag);
        if (!ok) break;
        uint64_t *mb = &sh.meta_full[j % kMetaSlots];
        mbar_arrive_expect_tx(mb, sizeof(TileMeta));
        bulk_load(&sh.meta[j % kMetaSlots], p.meta + first + j, sizeof(TileMeta), mb);
        mbar_arrive_expect_tx(&sh.k_full[s], C::kTileBytes);
        bulk_load(smem + C::kKAt + s * C::kTileBytes, src + (int64_t)j * C::kImage, C::kTileBytes, &sh.k_full[s]);
        ok = mbar_wait(&sh.v_empty[s], parity, abort_flag);
        if (!ok) break;
        mbar_arrive_expect_tx(&sh.v_full[s], C::kTileBytes);
        bulk_load(smem + C::kVAt + s * C::kTileBytes, src + (int64_t)j * C::kImage + C::kTileBytes, C::kTileBytes,
                  &sh.v_full[s]);
      }
      if (!ok) {  // what was started lands before the CTA leaves (tile j: keys and metadata at most)
        *abort_flag = 1;
        drain_ring(sh.meta_full, kMetaSlots, j + 1, kMetaSlots);
        drain_ring(sh.k_full, 2, j + 1, 2);
        drain_ring(sh.v_full, 2, j, 2);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, C::kColumns);
  if (threadIdx.x == 0 && *abort_flag) set_status(p.status, QLIN_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch_d(PrefillParams p, int64_t group, cudaStream_t st) {
  using C = Config<D>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(k_attn_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  for (p.head0 = 0; p.head0 < p.H; p.head0 += p.heads) {
    p.heads = (int)std::min<int64_t>(group, p.H - p.head0);  // the increment sees it, too
    const int64_t pairs = (int64_t)p.B * p.heads;
    p.meta = reinterpret_cast<TileMeta *>(p.images + pairs * p.tiles * C::kImage);
    p.positions = reinterpret_cast<PositionMeta *>(p.meta + pairs * p.tiles);
    e = launch_kernel(k_attn_unpack<D>, dim3((unsigned)(pairs * p.tiles)), dim3(64 * C::kUnits), 0, st, 1, p);
    if (e != cudaSuccess) return e;
    e = launch_kernel(k_attn_prefill<D>, dim3((unsigned)(pairs * p.row_tiles * p.parts.splits)), dim3(kThreads),
                      C::kSmem, st, 1, p);
    if (e != cudaSuccess) return e;
  }
  return p.parts.splits > 1 ? launch_attn_join(p, p.parts, D, true, st) : cudaSuccess;
}

}  // namespace

bool attn_prefill_has(int64_t D) { return D == 64 || D == 128; }

// kv heads are unpacked together until their images reach 2 GB (a quarter of
// the positions of a full GPU of 8-bit cache), then in groups one after the other.
// Where the row tiles leave multiprocessors idle, positions are split so that the
// waves of CTAs, times the position tiles of a part (and about two tiles' time to
// begin and end one), are fewest; the join counts three.
AttnPrefillPlan attn_prefill_plan(int64_t B, int64_t H, int64_t G, int64_t D, int64_t max_q, int64_t max_kv,
                                  int64_t window, int sms) {
  AttnPrefillPlan plan{};
  const int64_t tiles = std::max<int64_t>(1, (max_kv + kPos - 1) / kPos);
  const int64_t head = B * tiles * (4 * kPos * D + (int64_t)(sizeof(TileMeta) + kPos * sizeof(PositionMeta)));
  plan.heads = std::max<int64_t>(1, std::min(H, ((int64_t)2 << 30) / head));
  plan.image_bytes = round_up((size_t)(head * plan.heads), 256);
  constexpr int64_t rows = 2 * kRowTile;
  plan.row_tiles = (max_q * G + rows - 1) / rows;
  int64_t range = max_kv;
  if (window > 0 && window < max_kv) range = std::min(range, window + rows / G + 1 + kPos);
  const int64_t range_tiles = std::max<int64_t>(1, (range + kPos - 1) / kPos);
  const int64_t ctas = B * H * plan.row_tiles;
  plan.splits = 1;
  int64_t least = (ctas + sms - 1) / sms * (range_tiles + 2);
  for (int64_t s = 2; plan.heads == H && ctas < sms && s <= std::min<int64_t>(range_tiles / 2, 64); ++s) {
    const int64_t cost = (ctas * s + sms - 1) / sms * ((range_tiles + s - 1) / s + 2) + 3;
    if (cost < least) least = cost, plan.splits = s;
  }
  plan.chunk = (range_tiles + plan.splits - 1) / plan.splits;
  plan.splits = (range_tiles + plan.chunk - 1) / plan.chunk;
  plan.ws_bytes = plan.image_bytes;
  if (plan.splits > 1) plan.ws_bytes += round_up((size_t)(ctas * plan.splits * rows * (D + 2) * 4), 256);
  return plan;
}

cudaError_t launch_attn_prefill(const AttnArgs &a, const AttnPrefillPlan &plan, int few_rows, void *ws,
                                unsigned *status, cudaStream_t st) {
  PrefillParams p{};
  static_cast<AttnDev &>(p) = attn_dev(a, few_rows, status);
  p.row_tiles = (int)plan.row_tiles;
  p.tiles = (int)std::max<int64_t>(1, (a.max_kv + kPos - 1) / kPos);
  p.images = (uint8_t *)ws;
  p.heads = (int)plan.heads;
  p.chunk = (int)plan.chunk;
  p.parts.row_tiles = p.row_tiles, p.parts.rows = 2 * kRowTile, p.parts.splits = (int)plan.splits;
  p.parts.o = reinterpret_cast<float *>((char *)ws + plan.image_bytes);
  p.parts.sum = (float2 *)(p.parts.o + a.B * a.H * plan.row_tiles * plan.splits * p.parts.rows * a.D);
  if (a.D == 64) return launch_d<64>(p, plan.heads, st);
  if (a.D == 128) return launch_d<128>(p, plan.heads, st);
  return cudaErrorInvalidValue;
}

}  // namespace qlin
