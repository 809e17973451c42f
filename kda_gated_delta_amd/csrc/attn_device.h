// Device helpers shared by the full-attention kernels (gfx950 / CDNA4,
// wave64): matrix-instruction types, cross-half exchange, packed-sequence
// lookup and the swizzled tile loads.
#pragma once

#include "kda_device.h"

namespace kda {
namespace attn {

constexpr int D = kHead;                 // head width of q, k and v
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_ptr;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Matrix product D = A B + C with A 32 x 16, B 16 x 32.  Lane l holds row
// (A) or column (B) l % 32 at contraction indices 8 (l / 32) .. + 7, and of C
// and D column l % 32 at rows 8 (r / 4) + 4 (l / 32) + r % 4 for r = 0 .. 15.
__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// The same with 16 x 32 by 32 x 16: row or column l % 16 at indices
// 8 (l / 16) .. + 7; of C and D column l % 16 at rows 4 (l / 16) + r.
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// Sum and maximum of a lane's value and that of the lane 32 away.
__device__ __forceinline__ u32x2 halves(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return (u32x2){r[0], r[1]};
}
__device__ __forceinline__ float half_max(float x) {
  const u32x2 r = halves(x);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const u32x2 r = halves(x);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Eight float32 values to a matrix operand, each rounded to bfloat16 once.
__device__ __forceinline__ bf16x8 pack8(const float* x) {
  const u32x4 v = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  return as_bf16x8(v);
}
// What rounding to x's bfloat16 values left of them, rounded in turn: the two
// together hold 16 bits of each.
__device__ __forceinline__ bf16x8 pack8_rest(const float (&x)[8], const bf16x8& b) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = x[i] - float(b[i]);
  return pack8(rest);
}

// ---------------------------------------------------------------- running softmax

// How far (in powers of two) a row's maximum may grow before its sum and
// output are brought to the new one: weights stay below 2^8, far inside
// float32 and bfloat16, and most tiles skip the 64 multiplications.
constexpr float kSlack = 8.0f;

// What weights are taken relative to: a row whose scores so far are all -inf
// (keys that hold it, or sums that overflow) has no maximum, and weights of zero.
__device__ __forceinline__ float base(float m) { return m == -INFINITY ? 0.0f : m; }

// ---------------------------------------------------------------- packed sequences

// A launch covers the rows of every sequence in tiles of BM tokens.  With
// equal sequences tile and sequence follow from the index.  With packed ones
// they are looked up in the offsets, which may come in any order: sequences that
// do not overlap have at most floor(T / BM) + N tiles.  No lookup reads past the
// N + 1 offsets, whatever they hold.
struct Rows {
  int64_t first;   // the sequence's first token, counted over the whole batch
  int b, start;    // the same as batch row and place in it
  int len;         // its tokens
  int row0;        // the tile's first row within it; >= len: no such tile
  int n;           // the sequence
};

// Offset n, whatever cu holds: differences of two then fit 32 bits.
__device__ __forceinline__ int offset_of(const int32_t* cu, int n, int T) { return min(max(cu[n], 0), T); }

// The sequence that holds row `row` and begins before it, -1 if there is none:
// the wave looks at 256 sequences at a time.
__device__ __forceinline__ int find_holder(const int32_t* cu, int N, int row) {
  const int lane = threadIdx.x & 63;
  for (int n0 = 0; n0 < N; n0 += 256) {
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(n0 + 64 * i + lane, N);
      in[i] = cu[n] < row && row < cu[min(n + 1, N)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t m = __ballot(in[i]);
      if (m) return n0 + 64 * i + __builtin_ctzll(m);
    }
  }
  return -1;
}

// Tile `rank` of all packed sequences' tiles, those with the largest index first
// (N <= 64).  A lane holds one sequence's number of tiles; #tiles with an index
// >= t is looked up for 64 values of t at once.  Returns the sequence, -1 if
// there are not so many tiles, and the index.
__device__ __forceinline__ int find_ranked(int own_tiles, int N, int most, int rank, int& index) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = most + 1, above = 0;       // the index is in [lo, hi); #tiles with an index >= hi
  bool first = true;
  while (hi - lo > 1 || first) {
    const int step = (hi - lo + 63) / 64, t = lo + lane * step;
    int count = 0;
    for (int n = 0; n < N; ++n) count += max(__builtin_amdgcn_readlane(own_tiles, n) - t, 0);
    if (first && rank >= __builtin_amdgcn_readfirstlane(count)) return -1;
    first = false;
    const uint64_t more = __ballot(t < hi && count > rank);   // a stretch of lanes from 0
    const int k = 63 - __builtin_clzll(more);
    if (k < 63 && lo + (k + 1) * step < hi) {
      above = __builtin_amdgcn_readlane(count, k + 1);
      hi = lo + (k + 1) * step;
    }
    lo += k * step;
  }
  index = lo;
  uint64_t have = __ballot(lane < N && own_tiles > lo);
  for (int j = rank - above; j > 0; --j) have &= have - 1;
  return __builtin_ctzll(have);
}

// Whether row t, the same for the whole wave, lies in a sequence: the wave looks
// at 64 of them at a time.
__device__ __forceinline__ bool in_sequence(const int32_t* cu, int N, int t) {
  bool in = false;
  for (int n = threadIdx.x & 63; n < N; n += 64) in |= t >= cu[n] && t < cu[n + 1];
  return __any(in);
}

// Workgroups are dealt to the eight XCDs in turn, and each XCD has its own
// cache.  The query heads of one tile that share a key/value head read the same
// keys at about the same time: they follow one another on one XCD.  Of a
// launch of head_blocks(slots, HQ, HKV) workgroups, false for the few past the
// end.
constexpr int kXcds = 8;
__host__ __device__ inline int64_t head_blocks(int64_t slots, int HQ, int HKV) {
  return (slots * HKV + kXcds - 1) / kXcds * kXcds * (HQ / HKV);
}
__device__ __forceinline__ bool find_head(unsigned id, int slots, int HQ, int HKV, int& slot, int& hkv, int& hq) {
  const unsigned G = unsigned(HQ) / unsigned(HKV), j = id / kXcds;
  const unsigned pair = id % kXcds + kXcds * (j / G);
  slot = int(pair / unsigned(HKV));
  hkv = int(pair % unsigned(HKV));
  hq = hkv * int(G) + int(j % G);
  return slot < slots;
}

// The rows of workgroup `slot` (of slots) of a launch.  kEarly: the tiles that
// have most work are a sequence's first (backward's keys), else its last; they
// come first in the launch, so that the short ones fill the end.  With up to 64
// packed sequences that holds over all of them; with more, they come as the
// sequences do.
template <bool kEarly>
__device__ __forceinline__ Rows find_rows(const int32_t* cu, int N, int T, int slot, int slots, int BM) {
  Rows r;
  if (!cu) {
    const int tiles = slots / unsigned(N), t = int(slot / unsigned(N));
    r.b = r.n = slot % unsigned(N);
    r.start = 0;
    r.first = int64_t(r.b) * T;
    r.len = T;
    r.row0 = (kEarly ? t : tiles - 1 - t) * BM;
    return r;
  }
  int n, t = -1;
  if (N <= 64) {
    const int lane = threadIdx.x & 63;
    int own = 0;
    if (lane < N) own = max(offset_of(cu, lane + 1, T) - offset_of(cu, lane, T) + BM - 1, 0) / BM;
    n = find_ranked(own, N, T / BM + 1, slot, t);
    if (n >= 0 && kEarly) t = __builtin_amdgcn_readlane(own, n) - 1 - t;
    n = max(n, 0);
  } else {
    // N slots for the sequences' first tiles, and floor(T / BM) for the others: of
    // the rows behind a tile's first up to the next tile's, one is a multiple of
    // BM.  It leads from slot to tile, however the offsets are ordered, and only
    // these slots look at all sequences.  Where first tiles have most work the two
    // kinds are mixed evenly, so that most tiles of a sequence stay near one
    // another, else the others come first (backward in us, so and with the kinds
    // apart: 150 sequences of up to 700 tokens, 16 heads on 4, 721 and 752; forward,
    // so and mixed: 65 of up to 100, 8 on 2, 10.7 and 12.2).
    bool first;
    int other;                                           // of the slots for others
    if constexpr (kEarly) {
      const uint64_t at = uint64_t(unsigned(slot)) * unsigned(N);
      n = int(at / unsigned(slots));                     // first tiles before this slot
      first = at - uint64_t(n) * unsigned(slots) + unsigned(N) >= unsigned(slots);
      other = slot - n;
    } else {
      n = slot - (slots - N);
      first = n >= 0;
      other = -1 - n;
    }
    if (first) {
      t = 0;
    } else {
      const int row = (other + 1) * BM;
      n = find_holder(cu, N, row);
      if (n >= 0) t = (row - offset_of(cu, n, T) + BM - 1) / BM;
      n = max(n, 0);
    }
  }
  const int c0 = offset_of(cu, n, T), c1 = offset_of(cu, n + 1, T);
  r.b = 0;
  r.n = n;
  r.first = r.start = c0;
  r.len = max(c1 - c0, 0);
  r.row0 = t < 0 || t > r.len / BM ? r.len : t * BM;
  return r;
}

// ---------------------------------------------------------------- tiles in LDS

// A tile of 64 rows of 128 bf16 lies in LDS as 64 lines of 256 bytes, loaded
// straight from memory in 16-byte pieces (1 KB, four lines, by one instruction
// of a wave).  Piece c of line r is stored at place c ^ swizzle(r), which
// serves both ways of reading: 16 successive lines hold one piece in 16
// different places (read_rows), and 4 successive lines hold one 64-byte block
// in the four quarters of their 256 bytes (read_columns), so neither meets a
// bank twice.  The load writes lane after lane; the swizzle is made by what
// each lane reads.  Lines at or past `rows` read as zero (the buffer's size
// ends there), so nothing behind a sequence enters a product.
constexpr int kTile = 64;                 // rows of a tile
constexpr int kTileBytes = kTile * 256;

__device__ __forceinline__ int swizzle(int line) { return 4 * (line & 3) + ((line >> 2) & 3); }

template <int WAVES>
struct TileLoad {
  uint32_t lane_off;                      // byte offset of this lane's piece in the wave's first 1 KB block
  uint32_t step;                          // bytes between the wave's blocks: 4 * WAVES lines
  static_assert(16 % WAVES == 0 && WAVES % 4 == 0, "the swizzle must be the same in all blocks of a wave");

  __device__ __forceinline__ void init(int wave, int lane, int64_t stride) {
    const int line = 4 * wave + (lane >> 4);
    lane_off = uint32_t(line * stride * 2) + ((lane & 15) ^ swizzle(line)) * 16;
    step = uint32_t(4 * WAVES * stride * 2);
  }
  // base: the tile's first row; rows: how many of its rows exist (1 or more).
  __device__ __forceinline__ void issue(const uint16_t* base, int64_t stride, int rows, unsigned char* lds,
                                        int wave) const {
    const uint32_t bytes = uint32_t(min(rows, kTile)) * uint32_t(stride * 2);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, bytes, 0x00020000);
#pragma unroll
    for (int j = 0; j < 16 / WAVES; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr*)(lds + (wave + j * WAVES) * 1024), 16, lane_off,
                                               j * step, 0, 0);
  }
};

// 64 float32 of `src`, of which `rows` exist (the others read as zero), by one
// wave.
__device__ __forceinline__ void load_floats(const float* src, int rows, unsigned char* lds, int lane) {
  const auto rsrc =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(src), 0, uint32_t(min(rows, kTile)) * 4, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr*)lds, 4, lane * 4, 0, 0, 0);
}

// Rows r .. r + 31 of a tile as an A or B operand: contraction indices
// 16 s + 8 h .. + 7 of row r + l32.
__device__ __forceinline__ bf16x8 read_rows(const unsigned char* tile, int r, int l32, int h, int s) {
  const int line = r + l32;
  return *reinterpret_cast<const bf16x8*>(tile + line * 256 + (((2 * s + h) ^ swizzle(line)) * 16));
}

// The transpose of a tile's rows r + 16 m .. + 15 at columns c .. c + 31, as an
// A or B operand: lane l32 takes column c + l32 at rows
// r + 16 m + 4 h + j % 4 + 8 (j / 4) for j = 0 .. 7, the order in which the
// accumulator of a 32 x 32 product holds its rows.  (A transposing read
// gathers, in every 16 lanes, element i & 3 of the 8-byte pieces addressed by
// lanes (i >> 2) + 4 e into element e of lane i.)
__device__ __forceinline__ bf16x8 read_columns(const unsigned char* tile, int r, int m, int c, int lane) {
  const int j = lane & 15, h = lane >> 5;
  const int line = r + 16 * m + 4 * h + (j >> 2);
  const int col = c + (lane & 16) + 4 * (j & 3);
  const int piece = col >> 3, half = (col & 4) * 2;
  const unsigned char* p = tile + line * 256 + half;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + (piece ^ swizzle(line)) * 16));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * 256 + (piece ^ swizzle(line + 8)) * 16));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// Whether any row of a tile's first half, or two, holds an infinity or NaN.
__device__ __forceinline__ bool any_not_finite(const unsigned char* tile, int halves, int lane) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
#pragma unroll 8
  for (int i = 0; i < 8 * halves; ++i) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(tile + i * 1024 + lane * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[j] & 0x7fff7fffu));
  }
  return __any(top[0] >= 0x7f80 || top[1] >= 0x7f80);
}

// Row stores of a transposed accumulator (columns = rows of the output): the
// lane pair (l, l + 32) holds columns d of one row in groups of four; exchanged,
// each lane stores 16 bytes.
__device__ __forceinline__ void store_row32(uint16_t* row, const f32x16& acc, float f, int h) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    auto pair = [&](int j) { return pack_bf16(acc[4 * i + j] * f, acc[4 * i + j + 1] * f); };
    const uint32_t a0 = pair(0), a1 = pair(2), b0 = pair(4), b1 = pair(6);
    const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
    *reinterpret_cast<u32x4*>(row + 8 * (i + h)) = (u32x4){x[0], y[0], x[1], y[1]};
  }
}

// The same in float32.
__device__ __forceinline__ void store_row32(float* row, const f32x16& acc, float f, int h) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<f32x4*>(row + 8 * i + 4 * h) =
        (f32x4){acc[4 * i] * f, acc[4 * i + 1] * f, acc[4 * i + 2] * f, acc[4 * i + 3] * f};
}

// Four float32 values, as they are or each rounded to bfloat16 once.
__device__ __forceinline__ void store4(float* dst, f32x4 x) { *reinterpret_cast<f32x4*>(dst) = x; }
__device__ __forceinline__ void store4(uint16_t* dst, f32x4 x) {
  *reinterpret_cast<u32x2*>(dst) = (u32x2){pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}

// vmcnt(0), nothing else
constexpr int kWaitLoads = 0x0F70;

}  // namespace attn
}  // namespace kda
