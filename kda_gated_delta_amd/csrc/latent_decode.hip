// Attention of a few new tokens per sequence over the paged 8-bit cache of
// latents, in the absorbed form (export kda_latent_decode).
//
// A token's key is its latent and its shared part, 576 wide, and its value the
// latent, 512 wide, the same for all heads.  For query token i of Q (its position is
// len - Q + i) and head h, over the tokens j <= len - Q + i of the sequence:
//     z_j = scale q . [c_j s_j],   o = sum_j softmax(z)_j c_j.
// The Q queries of all heads are rows of one matrix, in tiles of at most 96.
//
// All (sequence, row tile) segments in order, in units of 32 tokens, form one line
// that is cut into equal pieces, one per workgroup (attn_line.h); a segment that
// lies in several leaves float32 parts, which latent_decode_join_kernel adds up.
//
// A unit lies in LDS as it came, in codes, and is used twice: S^T = [C s] Q^T, with Q
// in registers, and O^T += C^T P^T, where each wave has 128 of the 512 columns for all
// rows, so that a column is read (transposed) by one wave only.  Codes become
// bfloat16 (exactly) on their way from LDS into the operands.  A token's 128 values
// under one scale are one wave's columns: a key's scales enter as it is widened, a
// value's enter the weights, which go from the waves that made them to all through
// LDS, as operands.  The one rounding on the way is the weights', to bfloat16; scores,
// maximum, sum and output are float32.  The next units are on their way to LDS
// meanwhile.
//
// What bounds it: up to 32 rows a step of the output's waves (2500 cycles, of them a
// quarter waits to send the loads of a next unit), near to what memory allows (64
// sequences of up to 16384 tokens, 32 heads, 327 MB: 89 us; the walk reads 335 MB and
// writes 20 of parts, the join takes 6 us of it).  With more rows a unit's conversions,
// products and weights (48 sequences of up to 8192 tokens, 96 heads, 41 GFLOP: 76 us;
// 4100 cycles for a unit's 96 rows, of which products 1900, and 60 MB of parts written
// and read).  One short history is two launches.
//
// Tried and left: units widened once, as bfloat16 in LDS, which then cannot feed the
// products (115 us for the first of these, 101 for the second); scores by the e4m3
// instructions, which sum with fewer bits (a score off by 2^-14 of its products'
// magnitudes); for 32 rows the keys split over four pairs of waves that have all
// columns (111) and eight waves at one unit of 64 tokens, all of them through scores,
// weights and output (104); for 96 rows waves that hold 16 rows and all columns (118), or
// that go through all together (115); a next segment's loads before the results of the
// one before are stored (no gain); neighbouring pieces on one XCD (none).
#include "attn_line.h"
#include "kda_host.h"
#include "latent_device.h"

namespace {

using namespace kda::latent;
using kda::line::Piece;
using kda::line::length;
using kda::line::units_of;

constexpr int kWaves = 4;                    // that bring a unit, and have its columns
// A part: output, as the waves hold it ([row tile of 16][32 tiles of 16 columns][64
// lanes][4], lane l16 + 16 g4 with columns 4 g4 + e of row l16), then each row's
// maximum and sum.  Every store and load of a wave is then 1 KB in one piece.
constexpr int kPart = R + 2;                 // floats for a row
__device__ __forceinline__ int64_t in_part(int row_tile, int column_tile, int lane) {
  return ((int64_t(row_tile) * (R / 16) + column_tile) * 64 + lane) * 4;
}

struct Params {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *codes, *exponents;
  const uint16_t* shared;
  uint32_t c_stride, scale_stride, s_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int N, Q, H, width, shift, num_pages;
  float scale;
  uint16_t* o;
  float* lse;
  int rows, tile_rows, row_tiles;         // Q x H; rows of one tile (a multiple of 16); tiles
  int waves;                                 // pieces
  float* parts;                              // [2 x pieces][tile_rows x kPart]: of a piece's first segment, its last
  int *owner, *last_owner;                   // [segments]: first part (-1: not cut) and, of those cut, last piece
  int* cut;                                  // [pieces]: the segment that begins in the piece and is cut behind, or -1
  bool by_piece;                             // pieces, of which few are followed by a cut, are fewer than segments
};

// A word of four codes, times a power of two, as bfloat16 pairs.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 widen(uint32_t w, float f) {
  const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, false);
  const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, true);
  return (u32x2){__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// Eight codes as an operand.
__device__ __forceinline__ bf16x8 widen(uint32_t x, uint32_t y, float f) {
  const u32x2 a = widen(x, f), b = widen(y, f);
  return as_bf16x8((u32x4){a[0], a[1], b[0], b[1]});
}

constexpr int kUnit = 32;                    // tokens of a unit
constexpr int kOwn = kUnit / kWaves;         // tokens that a wave brings, all in one page
constexpr int kLoads = kOwn / 2 + 2;         // of a wave for a unit
// A unit in LDS: codes [kUnit][512], shared parts [kUnit][128 bytes], exponents (of
// kOwn tokens in 256 bytes).
constexpr int kShared = kUnit * R, kScale = kShared + kUnit * 2 * S, kBytes = kScale + kWaves * 256;

// Places of 16-byte pieces in a unit's lines: piece c of line r is at c ^ swirl(r), of
// the shared parts at c ^ swirl2(r).  Of 16 successive lines one piece is then in 16
// different places of the banks' 256 bytes, and of the 8 x 4 lines whose columns are
// read together (r, r + 16) two times 16.
__device__ __forceinline__ int swirl(int r) { return (r & 15) ^ ((r >> 1) & 8); }
__device__ __forceinline__ int swirl2(int r) { return (r >> 1) & 7; }

// Nothing moves across: operands are fetched in groups, one group ahead of the
// products that use the other.  (Left alone, the compiler reads each operand right
// before its product, and the wave waits for every one of them.)
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Sum and maximum over the four lanes that hold a row.
__device__ __forceinline__ u32x2 quarters(float x) {       // rows 0 and 1, or 2 and 3, of 16 lanes
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return (u32x2){r[0], r[1]};
}
__device__ __forceinline__ float quarter_max(float x) {
  const u32x2 r = quarters(x);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarter_sum(float x) {
  const u32x2 r = quarters(x);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Each lane's WIDE bytes at offset + more of `bytes` bytes, to WIDE * lane behind `to`.
template <int WIDE>                          // 16 or 4
__device__ __forceinline__ void load_lds(const void* from, int bytes, unsigned char* to, int offset, int more) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(from), 0, bytes, 0x00020000);
  if (WIDE == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr*)to, 16, offset, more, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr*)to, 4, offset, more, 0, 0);
}

// At most n loads are left, nothing else.
template <int n>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(kWaitLoads | (n & 15) | (n >> 4) << 14);
}

// A scale: byte `block` of a token's four exponents, as a factor.
__device__ __forceinline__ float scale_of(uint32_t exponents, int block) {
  return __uint_as_float((exponents >> (8 * block) & 255u) << 23);
}
// A key's four exponents in a unit, and those of four successive keys.
__device__ __forceinline__ const unsigned char* exponents_of(const unsigned char* tile, int key) {
  return tile + kScale + key / kOwn * 256 + key % kOwn * kBlocks;
}

// How a wave brings its kOwn tokens of a segment's units.
struct Tokens {
  const int32_t* table;
  int end, wave;           // tokens from `end` on are not brought
  int from, slots;         // the slots of the first tokens in 64 units, one to a lane; -1: no page

  struct Source {
    const uint8_t* codes;
    const uint16_t* shared;
    const uint8_t* exponents;
    int some;              // tokens
    unsigned char* tile;
  };

  __device__ __forceinline__ void look(const Params& p, int unit) {
    from = unit;
    slots = -1;
    const int64_t token = int64_t(unit + lane_now()) * kUnit + wave * kOwn;
    if (token < end) {
      const int id = table[token >> p.shift];
      if (id >= 0 && id < p.num_pages) slots = (id << p.shift) + (int(token) & ((1 << p.shift) - 1));
    }
  }
  // There: whether the wave's tokens have a page.
  __device__ __forceinline__ Source source(const Params& p, int unit, unsigned char* tile, int* there) {
    if (unit - from >= 64) look(p, unit);
    const int slot = __builtin_amdgcn_readlane(slots, unit - from);
    const int some = slot < 0 ? 0 : min(end - (unit * kUnit + wave * kOwn), kOwn);
    const uint64_t page = uint32_t(max(slot, 0)) >> p.shift;
    const int at = max(slot, 0) & ((1 << p.shift) - 1);
    if (lane_now() == 0) there[wave] = some;
    return Source{p.codes + page * p.c_stride + at * R, p.shared + page * p.s_stride + at * S,
                  p.exponents + page * p.scale_stride + at * kBlocks, some, tile};
  }
  // Load i of kLoads.  They come as buffers that end behind the sequence, or are empty:
  // what is not there is zero in LDS.
  __device__ __forceinline__ void load(const Source& x, int i) const {
    const int lane = lane_now(), r0 = wave * kOwn;
    if (i < kOwn / 2)                                      // two lines
      load_lds<16>(x.codes, x.some * R, x.tile + r0 * R + i * 1024,
                   (lane >> 5) * R + (((lane & 31) ^ swirl(r0) ^ (lane >> 5)) ^ 2 * i) * 16, i * 1024);
    else if (i == kOwn / 2)                                // eight lines
      load_lds<16>(x.shared, x.some * 2 * S, x.tile + kShared + r0 * 2 * S,
                   (lane >> 3) * 2 * S + ((lane & 7) ^ swirl2(r0 + (lane >> 3))) * 16, 0);
    else
      load_lds<4>(x.exponents, x.some * kBlocks, x.tile + kScale + wave * 256, lane * 4, 0);
  }
  // A token that only some of the queries see may hold codes of NaN, which a weight of
  // zero would not keep out of the others' products: its latent becomes zero and its
  // shared part NaN, which gives the same to those that see it (their scores are NaN)
  // and nothing to the others.
  __device__ __forceinline__ void without_nan(unsigned char* tile) const {
    const int lane = lane_now();
#pragma unroll 1
    for (int i = wave * kOwn; i < wave * kOwn + kOwn; ++i) {
      u32x2* code = reinterpret_cast<u32x2*>(tile + i * R) + lane;
      const u32x2 x = *code;
      const uint32_t nan = ((x[0] & 0x7f7f7f7fu) + 0x01010101u) | ((x[1] & 0x7f7f7f7fu) + 0x01010101u);
      if (!__any(nan & 0x80808080u)) continue;
      *code = (u32x2){0, 0};
      if (lane < 32) reinterpret_cast<uint32_t*>(tile + kShared + i * 2 * S)[lane] = 0x7fc07fc0u;
    }
  }
};

// ---------------------------------------------------------------- the walk

// Eight waves, four that make weights and four that use them a unit or two later, one
// of each kind on every SIMD.  Of the output a wave has 128 columns of all row tiles,
// which are one block of every token's scales.  Of the scores it has all 32 keys of one
// or two row tiles, so that maxima and sums are its own, or, with up to 32 rows, 16 keys
// of one.  The output's waves also bring the tokens.
constexpr int kThreads = 512;
// Units that a segment costs besides its own, for its beginning and end.  With 0, 4, 6 and
// 8, us: 48 sequences of up to 8192 tokens, 96 heads 81.7, 75.6, 75.4, 74.4; 600 of up to 1000 185,
// 148, 138, 139; 32 of up to 8000, 64 heads 59.2, 46.3, 46.5, 46.3.
constexpr int kExtra = 8;

// NT: row tiles of 16.
template <int NT>
__global__ __launch_bounds__(kThreads, 2) void latent_decode_kernel(Params p) {
  constexpr int kOwnRows = NT <= 4 ? 1 : 2;                // row tiles of a wave's scores
  constexpr int kSplit = NT <= 2 ? 2 : 1;                  // waves that share a unit's keys
  constexpr int kLag = kSplit;                             // from a unit's scores to its output
  constexpr int kRing = kSplit == 2 ? 6 : 4;               // units in LDS
  constexpr int kAheadUnits = kRing - 1 - kLag;            // on their way
  __shared__ __align__(1024) struct {
    unsigned char ring[kRing][kBytes];
    unsigned char weights[2][NT][1024];
    float factor[2][16 * NT];                              // of the output so far
    int grown[2][kWaves];                                  // whether a wave has factors that are not 1
    float most[2][2][16 * NT];                             // of a unit, with kSplit = 2
    float sum[kSplit][16 * NT], top[16 * NT];
    int there[kRing][kWaves];                          // whether a wave's tokens have a page
  } lds;
  auto &ring = lds.ring;
  auto &weights = lds.weights;
  auto &there = lds.there;
  const int role = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);

  const Piece piece = kda::line::find_piece<kUnit, 1, kExtra>(p, 0, p.row_tiles);
  if (threadIdx.x == 0) p.cut[blockIdx.x] = -1;
  int64_t left = piece.to - piece.from;
  int n = piece.n, len = piece.len, units = units_of<kUnit>(len);
  const int64_t inside = piece.from - piece.before;
  int seg = p.row_tiles == 1 ? 0 : __builtin_amdgcn_readfirstlane(int(inside / (units + kExtra)));
  int first = __builtin_amdgcn_readfirstlane(int(inside - int64_t(seg) * (units + kExtra)) - kExtra);
  left += min(first, 0);                                   // (the extra units are before the first)
  first = max(first, 0);
  bool begun = false;                                      // the piece's first segment is done
  const float c = p.scale * kLog2e;

  while (left > 0) {
    // -------- one segment: sequence n, rows row0 .. row0 + tile_rows - 1
    const int row0 = seg * p.tile_rows;
    const int last = int(min(int64_t(units), first + left));
    const int rows = min(p.rows - row0, p.tile_rows);
    const bool whole = first == 0 && last == units;
    const int64_t segment = int64_t(n) * p.row_tiles + seg;
    const int slot = 2 * piece.w + int(begun);

    if (role == 0) {
      // ======== weights of row tiles mine ..
      const int mine = wave / kSplit * kOwnRows, half = wave % kSplit;
      const bool busy = 16 * mine < rows;
      // Rows of Q as operands.  Along a key the order is what lanes of 16 codes make it:
      // steps 2 i and 2 i + 1 are the first and second 8 of lane group g4's 16.
      const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
      bf16x8 q[kOwnRows][18];
      int limit[kOwnRows];                                 // tokens that the lane's row sees
#pragma unroll
      for (int t = 0; t < kOwnRows; ++t) {
        const int r = row0 + min(16 * (mine + t) + l16, rows - 1), i = r / p.H;
        const uint16_t* src = p.q + (int64_t(n) * p.Q + i) * p.q_stride + (r - i * p.H) * (R + S);
#pragma unroll
        for (int s = 0; s < 16; ++s)
          q[t][s] = *reinterpret_cast<const bf16x8*>(src + 64 * (s >> 1) + 16 * g4 + 8 * (s & 1));
#pragma unroll
        for (int s = 0; s < 2; ++s) q[t][16 + s] = *reinterpret_cast<const bf16x8*>(src + R + 32 * s + 8 * g4);
        limit[t] = len - p.Q + i + 1;
      }
      wait_loads<0>();
      float m[kOwnRows], l[kOwnRows];                      // l: of this lane's keys only, until the end
#pragma unroll
      for (int t = 0; t < kOwnRows; ++t) m[t] = -INFINITY, l[t] = 0.0f;

      // Of half a unit's keys first the scores are made, and their maxima known to both
      // waves; a step later, beside the next unit's scores, the weights.
      f32x4 scores = (f32x4)(0.0f);
      for (int unit = first; kSplit == 2 && unit <= last; ++unit) {
        kda::lds_barrier();                                // the unit is there, and the maxima of the one before
        const int odd = (unit - 1) & 1;                    // (of the unit before)
        if (!busy) {
          if (lane == 0) lds.grown[odd][wave] = 0;
          continue;
        }
        unsigned char* tile = ring[unit % kRing];
        const int key0 = unit * kUnit;
        const bool edge = key0 + kUnit > len - p.Q + 1;    // some row does not see some key
        const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4, row = 16 * mine + l16;
        const f32x4 before = scores;
        const float mx0 = lds.most[odd][0][row], mx1 = lds.most[odd][1][row];
        if (unit < last) {
          f32x4 s = (f32x4)(0.0f);
          constexpr int kAhead = 3;                        // as below
          u32x4 a[kAhead];
          const int key = 16 * half + l16;
          const int key_at = key * R + ((g4 ^ swirl(key)) * 16);
          const int shared_at = kShared + key * 2 * S + ((g4 ^ swirl2(key)) * 16);
          auto fetch = [&](int i) {
            const int at = i < 8 ? key_at ^ i * 64 : shared_at ^ (i - 8) * 64;
            a[i % kAhead] = *reinterpret_cast<const u32x4*>(tile + at);
          };
          const uint32_t scales = *reinterpret_cast<const uint32_t*>(exponents_of(tile, key));
#pragma unroll
          for (int i = 0; i < kAhead - 1; ++i) fetch(i);
#pragma unroll
          for (int i = 0; i < 10; ++i) {
            fence();
            if (i + kAhead - 1 < 10) fetch(i + kAhead - 1);
            fence();
            const u32x4 x = a[i % kAhead];
            if (i < 8) {
              const float f = scale_of(scales, i >> 1);
              s = mfma16(widen(x[0], x[1], f), q[0][2 * i], s);
              s = mfma16(widen(x[2], x[3], f), q[0][2 * i + 1], s);
            } else {
              s = mfma16(as_bf16x8(x), q[0][i + 8], s);
            }
          }
          fence();
          const bool gone = there[unit % kRing][2 * half + (g4 >> 1)] == 0;
          if (edge || __any(gone)) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gone || key0 + 16 * half + 4 * g4 + e >= limit[0]) s[e] = -INFINITY;
          }
          const float mx = quarter_max(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
          if (g4 == 0) lds.most[unit & 1][half][row] = mx;
          scores = s;
        }
        if (unit > first) {
          const float mx = fmaxf(mx0, mx1);
          // (row by row: what a row sees does not change how another one is rounded)
          const float now = (mx - m[0]) * c > kSlack ? mx : m[0];
          const float f = __builtin_amdgcn_exp2f((m[0] - base(now)) * c);
          const bool grown = __any(now != m[0]);
          m[0] = now;
          l[0] *= f;
          if (g4 == 0 && half == 0) lds.factor[odd][row] = f;
          if (lane == 0) lds.grown[odd][wave] = grown;
          const float b = base(now) * c;
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(before[e], c, -b));
            l[0] += x[e];
          }
          *reinterpret_cast<u32x2*>(weights[odd][mine] + lane * 16 + half * 8) =
              (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
        }
      }
      for (int unit = first; kSplit == 1 && unit < last; ++unit) {
        kda::lds_barrier();                                // the unit is there
        if (!busy) {
          if (lane == 0) lds.grown[unit & 1][wave] = 0;
          continue;
        }
        unsigned char* tile = ring[unit % kRing];
        const int key0 = unit * kUnit;
        const bool edge = key0 + kUnit > len - p.Q + 1;    // some row does not see some key
        const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
        f32x4 s[2][kOwnRows];
        {
          // Of a key's 20 pieces of 16 bytes (eight of codes, two steps each, and two of the
          // shared part) kAhead are on their way.
          constexpr int kAhead = 4;
          u32x4 a[kAhead];
          uint32_t scales[2];
          const int key_at = l16 * R + ((g4 ^ swirl(l16)) * 16);
          const int shared_at = kShared + l16 * 2 * S + ((g4 ^ swirl2(l16)) * 16);
          auto fetch = [&](int i) {
            const int k = i & 1, at = i >> 1;
            int x = at < 8 ? key_at : shared_at;
            asm("" : "+v"(x));                             // (its variants are not worth a register each)
            a[i % kAhead] = *reinterpret_cast<const u32x4*>(  // (swirl(16 + l16) = swirl(l16) ^ 8)
                at < 8 ? tile + k * 16 * R + (x ^ at * 64 ^ k * 128) : tile + k * 32 * S + (x ^ (at - 8) * 64));
          };
#pragma unroll
          for (int k = 0; k < 2; ++k)
            scales[k] = *reinterpret_cast<const uint32_t*>(exponents_of(tile, 16 * k + l16));
#pragma unroll
          for (int i = 0; i < kAhead - 1; ++i) fetch(i);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int t = 0; t < kOwnRows; ++t) s[k][t] = (f32x4)(0.0f);
#pragma unroll
          for (int i = 0; i < 20; ++i) {
            const int k = i & 1, at = i >> 1;
            fence();
            if (i + kAhead - 1 < 20) fetch(i + kAhead - 1);
            fence();
            const u32x4 x = a[i % kAhead];
            if (at < 8) {
              const float f = scale_of(scales[k], at >> 1);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const bf16x8 y = widen(x[2 * half], x[2 * half + 1], f);
#pragma unroll
                for (int t = 0; t < kOwnRows; ++t) s[k][t] = mfma16(y, q[t][2 * at + half], s[k][t]);
              }
            } else {
#pragma unroll
              for (int t = 0; t < kOwnRows; ++t) s[k][t] = mfma16(as_bf16x8(x), q[t][at + 8], s[k][t]);
            }
          }
          fence();
        }
        bool gone[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) gone[k] = there[unit % kRing][2 * k + (g4 >> 1)] == 0;
        if (edge || __any(gone[0] || gone[1])) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int t = 0; t < kOwnRows; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (gone[k] || key0 + 16 * k + 4 * g4 + e >= limit[t]) s[k][t][e] = -INFINITY;
        }
        bool grown = false;
#pragma unroll
        for (int t = 0; t < kOwnRows; ++t) {
          float mx = s[0][t][0];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[k][t][e]);
          mx = quarter_max(mx);
          // (row by row: what a row sees does not change how another one is rounded)
          const float now = (mx - m[t]) * c > kSlack ? mx : m[t];
          const float f = __builtin_amdgcn_exp2f((m[t] - base(now)) * c);
          grown |= now != m[t];
          m[t] = now;
          l[t] *= f;
          if (g4 == 0) lds.factor[unit & 1][16 * (mine + t) + l16] = f;
          const float b = base(now) * c;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[k][t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][t][e], c, -b));
              l[t] += s[k][t][e];
            }
        }
        grown = __any(grown);
        if (lane == 0) lds.grown[unit & 1][wave] = grown;
#pragma unroll
        for (int t = 0; t < kOwnRows; ++t) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * k + e] = s[k][t][e];
          *reinterpret_cast<bf16x8*>(weights[unit & 1][mine + t] + lane * 16) = pack8(x);
        }
      }
      kda::lds_barrier();                                  // the last weights are there
      if (busy) {
#pragma unroll
        for (int t = 0; t < kOwnRows; ++t) {
          l[t] = quarter_sum(l[t]);
          if (g4 == 0) {
            lds.sum[half][16 * (mine + t) + l16] = l[t];
            lds.top[16 * (mine + t) + l16] = m[t];
          }
        }
      }
      kda::lds_barrier();                                  // and sums and maxima
      if (threadIdx.x == 0) {
        if (first == 0) p.owner[segment] = whole ? -1 : slot;
        if (first != 0 && last == units) p.last_owner[segment] = piece.w;
        if (first == 0 && !whole) p.cut[piece.w] = int(segment);
      }
    } else {
      // ======== columns 128 wave ..
      Tokens tokens{p.table + n * p.table_stride, min(len, last * kUnit), wave, 0, -1};
      auto source = [&](int unit) {                        // (behind the last unit nothing comes)
        return tokens.source(p, unit, ring[unit % kRing], there[unit % kRing]);
      };
      if (begun) wait_loads<0>();                          // (stores, that would count among the loads)
      tokens.look(p, first);
#pragma unroll
      for (int u = 0; u < kAheadUnits; ++u) {
        const auto next = source(first + u);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) tokens.load(next, i);
      }
      f32x4 o[NT][8];                                      // column 128 wave + 16 d + 4 g4 + e of row 16 t + l16
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);

      auto arrive = [&](int unit) {                        // this wave's tokens of the unit are there
        wait_loads<(kAheadUnits - 1) * kLoads>();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (p.Q > 1 && unit < last && unit * kUnit + kUnit > len - p.Q + 1) tokens.without_nan(ring[unit % kRing]);
        kda::lds_barrier();                                // and the weights of the one kLag before
      };
#pragma unroll
      for (int u = 0; u < kLag; ++u) {
        arrive(first + u);
        const auto next = source(first + u + kAheadUnits);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) tokens.load(next, i);
      }
      for (int unit = first + kLag; unit < last + kLag; ++unit) {
        arrive(unit);

        // -------- the unit kLag before: lane l16 takes column l16 of 16 at keys 16 (j / 4) + 4 g4 +
        // j % 4 for j = 0 .. 7, the order in which the scores hold them.  (A transposing
        // read gathers, in every 16 lanes, byte i & 7 of the 8-byte pieces addressed by
        // lanes (i >> 3) + 2 e into byte e of lane i.)
        const int before = unit - kLag;
        unsigned char* tile = ring[before % kRing];
        const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
        const int line = ((l16 >> 1) & 3) + 4 * g4 + (l16 & 8) * 2;
        const int place = line * R + ((8 * wave) ^ swirl(line)) * 16 + (l16 & 1) * 8;
        constexpr int kAhead = 2;                          // row tiles
        u32x4 w[kAhead];
        bf16x8 x[8];
        u32x2 a[8];
        auto fetch_weights = [&](int i) {
          w[i % kAhead] = *reinterpret_cast<const u32x4*>(weights[before & 1][i] + lane * 16);
        };
        u32x4 exponents[2];                                // of the lane's eight keys
#pragma unroll
        for (int k = 0; k < 2; ++k)
          exponents[k] = *reinterpret_cast<const u32x4*>(exponents_of(tile, 16 * k + 4 * g4));
        const u32x4 grown = *reinterpret_cast<const u32x4*>(lds.grown[before & 1]);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          a[d] = __builtin_bit_cast(u32x2, transposed((const lds_i32x2*)(tile + (place ^ d * 16))));
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) fetch_weights(i);
        fence();
        const auto next = source(unit + kAheadUnits);      // (while these reads go on)
        fence();
        // Weights times the keys' scales for these columns: powers of two, so that nothing is
        // rounded (or only below 2^-126).
        float scales[8];
        auto scaled = [&](const u32x4& w) {
          u32x4 y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(w[i] << 16) * scales[2 * i];
            const float hi = __uint_as_float(w[i] & 0xffff0000u) * scales[2 * i + 1];
            y[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
          }
          return as_bf16x8(y);
        };
        if (__builtin_amdgcn_readfirstlane(grown[0] | grown[1] | grown[2] | grown[3])) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float f = lds.factor[before & 1][16 * t + l16];
#pragma unroll
            for (int d = 0; d < 8; ++d) o[t][d] *= f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) scales[i] = scale_of(exponents[i >> 2][i & 3], wave);
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = widen(a[d][0], a[d][1], 1.0f);
        fence();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t + kAhead - 1 < NT) fetch_weights(t + kAhead - 1);
          // (at once the loads would wait for one another)
#pragma unroll
          for (int i = t * kLoads / NT; i < (t + 1) * kLoads / NT; ++i) tokens.load(next, i);
          const bf16x8 y = scaled(w[t % kAhead]);
          fence();
#pragma unroll
          for (int d = 0; d < 8; ++d) o[t][d] = mfma16(x[d], y, o[t][d]);
          fence();
        }
      }

      // -------- its rows: finished, or a part
      wait_loads<0>();                                     // (those that brought nothing, too)
      kda::lds_barrier();
      float* part = p.parts + int64_t(slot) * p.tile_rows * kPart;
      auto total = [&](int r) { return kSplit == 2 ? lds.sum[0][r] + lds.sum[kSplit - 1][r] : lds.sum[0][r]; };
      const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 16 * t + l16, col = 128 * wave + 4 * g4;
        if (whole) {
          if (r >= rows) continue;
          const int64_t out = int64_t(n) * p.rows + row0 + r;
          const float sum = total(r), f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const f32x4 x = o[t][d] * f;
            *reinterpret_cast<u32x2*>(p.o + out * R + col + 16 * d) =
                (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
          }
          if (p.lse && wave == 0 && g4 == 0) p.lse[out] = lds.top[r] * p.scale + __logf(sum);
        } else if (16 * t < rows) {
#pragma unroll
          for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(part + in_part(t, 8 * wave + d, lane)) = o[t][d];
          if (wave == 0 && g4 == 0)
            *reinterpret_cast<float2*>(part + p.tile_rows * R + 2 * r) = make_float2(lds.top[r], total(r));
        }
      }
    }
    left -= last - first + kExtra;
    first = 0;
    begun = true;
    if (++seg == p.row_tiles) {
      seg = 0;
      if (++n < p.N) len = length(p, n), units = units_of<kUnit>(len);
    }
  }
}

// ---------------------------------------------------------------- the walk, up to 32 rows of many segments

// Four waves, which go through scores, weights and output together; of a unit's scores
// a wave has 16 keys and 16 rows.  Two workgroups on a compute unit: one has its pauses,
// and its segments' beginnings and ends, while the other computes.  With segments this
// is the faster one from about 512 on (latent_decode_kernel and this one, 16 heads, up to 1000
// tokens: 300 sequences 45.2 and 44.8 us; 32 heads: 2000 of up to 2000 339 and 329, 4096 of up to 300
// 228 and 192; and the other way 64 of up to 16384 88 and 91, one of 30000 21 and 26).
constexpr int kManyThreads = 64 * kWaves, kPerCu = 2, kManyRing = 3;
// As kExtra: 4096 sequences of up to 300 tokens with 0, 4, 6 and 8 222, 193, 191 and 195 us, 2000 of up
// to 2000 344, 331, 332 and 337.
constexpr int kManyExtra = 6;
constexpr int kRowTiles = 2;

__global__ __launch_bounds__(kManyThreads, kPerCu) void latent_decode_many_kernel(Params p) {
  // (One object: between two the compiler tells apart what loads to LDS write, and
  // has reads wait for all those that are on their way to the same one.)
  __shared__ __align__(1024) struct {
    unsigned char ring[kManyRing][kBytes];
    unsigned char weights[kBlocks][kRowTiles][1024];
    float scales[kUnit][kBlocks];
    float top[2][16 * kRowTiles];                          // maxima of a unit, and in the end sums
    int there[kManyRing][kWaves];                              // whether a wave's tokens have a page
  } lds;
  auto &ring = lds.ring;
  auto &weights = lds.weights;
  auto &scales = lds.scales;
  auto &top = lds.top;
  auto &there = lds.there;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave & 1, mine = wave >> 1;             // the wave's key tile, and its row tile

  const Piece piece = kda::line::find_piece<kUnit, 1, kManyExtra>(p, 0, p.row_tiles);
  if (threadIdx.x == 0) p.cut[blockIdx.x] = -1;
  int64_t left = piece.to - piece.from;
  int n = piece.n, len = piece.len, units = units_of<kUnit>(len);
  const int64_t inside = piece.from - piece.before;
  int seg = p.row_tiles == 1 ? 0 : __builtin_amdgcn_readfirstlane(int(inside / (units + kManyExtra)));
  int first = __builtin_amdgcn_readfirstlane(int(inside - int64_t(seg) * (units + kManyExtra)) - kManyExtra);
  left += min(first, 0);                                   // (the extra units are before the first)
  first = max(first, 0);
  bool begun = false;                                      // the piece's first segment is done
  const float c = p.scale * kLog2e;

  while (left > 0) {
    // -------- one segment: sequence n, rows row0 .. row0 + tile_rows - 1
    const int row0 = seg * p.tile_rows;
    const int last = int(min(int64_t(units), first + left));
    const int rows = min(p.rows - row0, p.tile_rows);

    Tokens tokens{p.table + n * p.table_stride, min(len, last * kUnit), wave, 0, -1};
    auto load = [&](int unit) {
      const auto next = tokens.source(p, unit, ring[unit % kManyRing], there[unit % kManyRing]);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) tokens.load(next, i);
    };
    if (begun) wait_loads<0>();                            // (stores, that would count among the loads)
    tokens.look(p, first);
    // Rows of Q as operands.  Along a key the order is what lanes of 16 codes make it:
    // steps 2 i and 2 i + 1 are the first and second 8 of lane group g4's 16.
    bf16x8 q[18];
    int limit;                                             // tokens that the lane's row sees
    {
      const int r = row0 + min(16 * mine + l16, rows - 1), i = r / p.H;
      const uint16_t* src = p.q + (int64_t(n) * p.Q + i) * p.q_stride + (r - i * p.H) * (R + S);
#pragma unroll
      for (int s = 0; s < 16; ++s)
        q[s] = *reinterpret_cast<const bf16x8*>(src + 64 * (s >> 1) + 16 * g4 + 8 * (s & 1));
#pragma unroll
      for (int s = 0; s < 2; ++s) q[16 + s] = *reinterpret_cast<const bf16x8*>(src + R + 32 * s + 8 * g4);
      limit = len - p.Q + i + 1;
    }
    fence();
#pragma unroll
    for (int i = 0; i < kManyRing - 1; ++i)
      if (first + i < last) load(first + i);
    // The queries are waited for before the first unit: left to the compiler they would
    // be in every unit, and with them the loads behind them.
    wait_loads<0>();
    f32x4 o[kRowTiles][8];                                       // column 128 wave + 16 d + 4 g4 + e of row 16 t + l16
    float m[kRowTiles], l = 0.0f;                          // m: of all rows; l: own row tile and keys
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      m[t] = -INFINITY;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);
    }

    for (int unit = first; unit < last; ++unit) {
      const int key0 = unit * kUnit;
      const bool edge = key0 + kUnit > len - p.Q + 1;      // some row does not see some key
      unsigned char* tile = ring[unit % kManyRing];
      const int place_lane = lane_now();
      const int p16 = place_lane & 15, p4 = place_lane >> 4;

      // -------- this wave's tokens are there; their scales as factors
      if (unit + 1 < last)
        wait_loads<kLoads>();
      else
        wait_loads<0>();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      if (place_lane < kOwn * kBlocks)
        scales[wave * kOwn + (place_lane >> 2)][place_lane & 3] =
            __uint_as_float(uint32_t(tile[kScale + wave * 256 + place_lane]) << 23);
      if (edge && p.Q > 1) tokens.without_nan(tile);
      kda::lds_barrier();                                  // everybody's; and the unit before is used up
      if (unit + kManyRing - 1 < last) load(unit + kManyRing - 1);

      // -------- scores of 16 keys (rows) and 16 rows (columns)
      f32x4 s = (f32x4)(0.0f);
      {
        float f[2];                                        // the scale of a block, and of the next
        auto fetch_scale = [&](int block) { f[block & 1] = scales[16 * half + p16][block]; };
        fetch_scale(0);
        // Rounds of two pieces of 16 bytes: eight of codes, two steps each, and two of the
        // shared part.
        u32x4 a[2][2];
        auto fetch = [&](int round) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = round * 2 + i, key = 16 * half + p16;
            a[round & 1][i] = *reinterpret_cast<const u32x4*>(
                at < 8 ? tile + key * R + ((p4 ^ p16 ^ half * 8) * 16 ^ at * 64)
                       : tile + kShared + key * 2 * S + ((4 * (at - 8) + p4) ^ swirl2(p16)) * 16);
          }
        };
        fetch(0);
#pragma unroll
        for (int round = 0; round < 5; ++round) {
          fence();
          if (round + 1 < 5) fetch(round + 1);
          if (round < 3) fetch_scale(round + 1);
          fence();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = round * 2 + i;
            const u32x4 x = a[round & 1][i];
            if (at < 8) {
              s = mfma16(widen(x[0], x[1], f[round & 1]), q[2 * at], s);
              s = mfma16(widen(x[2], x[3], f[round & 1]), q[2 * at + 1], s);
            } else {
              s = mfma16(as_bf16x8(x), q[at + 8], s);
            }
          }
        }
        fence();
        const int key = 16 * half + 4 * p4;
        const bool gone = there[unit % kManyRing][key / kOwn] == 0;
        if (edge || __any(gone)) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (gone || key0 + key + e >= limit) s[e] = -INFINITY;
        }
        const float mx = quarter_max(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
        if (p4 == 0) top[half][16 * mine + p16] = mx;
      }
      kda::lds_barrier();

      // -------- the maximum of all rows, the same in all waves; weights of the own ones
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) {
        const float mx = fmaxf(top[0][16 * t + p16], top[1][16 * t + p16]);
        if (__any((mx - m[t]) * c > kSlack)) {
          // (row by row: what a row sees does not change how another one is rounded)
          const float now = (mx - m[t]) * c > kSlack ? mx : m[t];
          const float f = __builtin_amdgcn_exp2f((m[t] - base(now)) * c);
          m[t] = now;
          if (t == mine) l *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) o[t][d] *= f;
        }
      }
      {
        const float b = base(mine == 0 ? m[0] : m[1]) * c;
        f32x4 f[4];                                        // of four keys: their blocks' scales
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const f32x4*>(scales[16 * half + 4 * p4 + e]);
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -b));
          l += x[e];
        }
        // (a key tile is half of a product's 32 keys)
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
          *reinterpret_cast<u32x2*>(weights[d][mine] + place_lane * 16 + half * 8) =
              (u32x2){kda::pack_bf16(x[0] * f[0][d], x[1] * f[1][d]), kda::pack_bf16(x[2] * f[2][d], x[3] * f[3][d])};
      }
      kda::lds_barrier();

      // -------- this wave's 128 columns of all rows: lane l16 takes column l16 of 16 at
      // keys 16 (j / 4) + 4 g4 + j % 4 for j = 0 .. 7, the order in which two key tiles'
      // scores made their weights.  (A transposing read gathers, in every 16 lanes, byte
      // i & 7 of the 8-byte pieces addressed by lanes (i >> 3) + 2 e into byte e of lane i.)
      bf16x8 w[kRowTiles];
      constexpr int kAhead = 4;                            // tiles of 16 columns fetched together
      u32x2 a[2][kAhead];
      const int line = ((p16 >> 1) & 3) + 4 * p4 + (p16 & 8) * 2;
      const int place = line * R + ((8 * wave) ^ swirl(line)) * 16 + (p16 & 1) * 8;
      auto fetch = [&](int round) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
          a[round & 1][d] = __builtin_bit_cast(
              u32x2, transposed((const lds_i32x2*)(tile + (place ^ (kAhead * round + d) * 16))));
      };
      fetch(0);
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) w[t] = *reinterpret_cast<const bf16x8*>(weights[wave][t] + place_lane * 16);
#pragma unroll
      for (int round = 0; round < 8 / kAhead; ++round) {
        fence();
        if (round + 1 < 8 / kAhead) fetch(round + 1);
        fence();
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const bf16x8 x = widen(a[round & 1][d][0], a[round & 1][d][1], 1.0f);
#pragma unroll
          for (int t = 0; t < kRowTiles; ++t) o[t][kAhead * round + d] = mfma16(x, w[t], o[t][kAhead * round + d]);
        }
      }
      fence();
    }

    // -------- its rows: finished, or a part
    l = quarter_sum(l);
    if (g4 == 0) top[half][16 * mine + l16] = l;
    kda::lds_barrier();
    const bool whole = first == 0 && last == units;
    const int64_t segment = int64_t(n) * p.row_tiles + seg;
    const int slot = 2 * piece.w + int(begun);
    if (threadIdx.x == 0) {
      if (first == 0) p.owner[segment] = whole ? -1 : slot;
      if (first != 0 && last == units) p.last_owner[segment] = piece.w;
      if (first == 0 && !whole) p.cut[piece.w] = int(segment);
    }
    float* part = p.parts + int64_t(slot) * p.tile_rows * kPart;
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int r = 16 * t + l16, col = 128 * wave + 4 * g4;
      const float sum = top[0][r] + top[1][r];
      if (whole) {
        if (r >= rows) continue;
        const int64_t out = int64_t(n) * p.rows + row0 + r;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const f32x4 x = o[t][d] * f;
          *reinterpret_cast<u32x2*>(p.o + out * R + col + 16 * d) =
              (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
        }
        if (p.lse && wave == 0 && g4 == 0) p.lse[out] = m[t] * p.scale + __logf(sum);
      } else if (16 * t < rows) {
#pragma unroll
        for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(part + in_part(t, 8 * wave + d, lane)) = o[t][d];
        if (wave == 0 && g4 == 0)
          *reinterpret_cast<float2*>(part + p.tile_rows * R + 2 * r) = make_float2(m[t], sum);
      }
    }
    left -= last - first + kManyExtra;
    first = 0;
    begun = true;
    if (++seg == p.row_tiles) {
      seg = 0;
      if (++n < p.N) len = length(p, n), units = units_of<kUnit>(len);
    }
  }
}

// ---------------------------------------------------------------- joining the parts

// A wave adds up 16 rows x 32 columns, every lane its own row's.  With STREAMS waves
// (a workgroup) each takes every STREAMS-th part of 16 columns (32 or 64 are slower: a
// history of 30000 tokens x 16 heads 25.6, 30.2 and 40.5 us; without streams 16 are: 64
// sequences 96.8, 95.5 and 95.7), and they are brought together in LDS.
template <int STREAMS>
__global__ __launch_bounds__(64 * STREAMS) void latent_decode_join_kernel(Params p) {
  constexpr int kTiles = STREAMS == 1 ? 2 : 1, kAhead = 4;   // column tiles; parts on their way
  __shared__ f32x4 outputs[STREAMS][kTiles][64];
  __shared__ float2 stats[STREAMS][16];
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned row_tiles = unsigned(p.tile_rows) / 16, per = row_tiles * (R / 16 / kTiles);
  const unsigned which = blockIdx.x / per, in = blockIdx.x - which * per;
  const int64_t segment = p.by_piece ? p.cut[which] : int(which);
  if (segment < 0) return;
  const int row_tile = int(in / (R / 16 / kTiles)), column_tile = int(in % (R / 16 / kTiles)) * kTiles;
  const int slot = p.owner[segment], last = p.last_owner[segment];   // (last holds anything unless slot says: cut)
  const int64_t n = segment / p.row_tiles;
  const int r = 16 * row_tile + l16, row = int(segment - n * p.row_tiles) * p.tile_rows + r;
  if (slot < 0 || row - l16 >= p.rows) return; // finished by its workgroup; or no row
  const int w0 = slot >> 1, count = last - w0 + 1;
  const float c = p.scale * kLog2e;
  // part i: the first may be its piece's last segment, the others are their pieces' first
  auto at = [&](int i) { return p.parts + int64_t(i == 0 ? slot : 2 * (w0 + i)) * p.tile_rows * kPart; };
  f32x4 x[kAhead][kTiles], acc[kTiles];
  float2 stat[kAhead];
  float m = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int d = 0; d < kTiles; ++d) acc[d] = (f32x4)(0.0f);
  auto fetch = [&](int i, int k) {
    const float* from = at(min(i, count - 1));
#pragma unroll
    for (int d = 0; d < kTiles; ++d)
      x[k][d] = *reinterpret_cast<const f32x4*>(from + in_part(row_tile, column_tile + d, lane));
    stat[k] = *reinterpret_cast<const float2*>(from + p.tile_rows * R + 2 * r);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(wave + k * STREAMS, k);
  for (int i0 = wave; i0 < count; i0 += kAhead * STREAMS)
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i0 + k * STREAMS >= count) break;
      const float now = fmaxf(m, stat[k].x);
      const float f = __builtin_amdgcn_exp2f((m - base(now)) * c);
      const float g = __builtin_amdgcn_exp2f((stat[k].x - base(now)) * c);
      m = now;
      sum = sum * f + stat[k].y * g;
#pragma unroll
      for (int d = 0; d < kTiles; ++d) acc[d] = acc[d] * f + x[k][d] * g;
      fetch(i0 + (k + kAhead) * STREAMS, k);
    }
  if (STREAMS > 1) {
#pragma unroll
    for (int d = 0; d < kTiles; ++d) outputs[wave][d][lane] = acc[d];
    if (g4 == 0) stats[wave][l16] = make_float2(m, sum);
    __syncthreads();
    if (wave != 0) return;
    float part[STREAMS];
#pragma unroll
    for (int i = 1; i < STREAMS; ++i) m = fmaxf(m, stats[i][l16].x);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < STREAMS; ++i) {
      const float2 other = stats[i][l16];
      part[i] = __builtin_amdgcn_exp2f((other.x - base(m)) * c);
      sum += other.y * part[i];
    }
#pragma unroll
    for (int d = 0; d < kTiles; ++d) acc[d] *= part[0];
#pragma unroll
    for (int i = 1; i < STREAMS; ++i)
#pragma unroll
      for (int d = 0; d < kTiles; ++d) acc[d] += outputs[i][d][lane] * part[i];
  }
  if (row >= p.rows) return;
  const int64_t out = n * p.rows + row;
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int d = 0; d < kTiles; ++d) {
    const f32x4 y = acc[d] * f;
    *reinterpret_cast<u32x2*>(p.o + out * R + 16 * (column_tile + d) + 4 * g4) =
        (u32x2){kda::pack_bf16(y[0], y[1]), kda::pack_bf16(y[2], y[3])};
  }
  if (p.lse && column_tile == 0 && g4 == 0) p.lse[out] = m * p.scale + __logf(sum);
}

struct Plan {
  int rows, tile_rows, row_tiles, pieces;
  int64_t segments;
  bool many;
  size_t parts, bytes;
};

// Rows in equal tiles of up to 96, which is what eight waves' registers hold.  Many
// segments of up to 32 rows go to the kernel of four waves.
Plan plan_for(int64_t N, int64_t Q, int H) {
  Plan x;
  x.rows = int(Q * H);
  x.row_tiles = (x.rows + 95) / 96;
  x.tile_rows = ((x.rows + x.row_tiles - 1) / x.row_tiles + 15) / 16 * 16;
  x.segments = N * x.row_tiles;
  x.many = x.tile_rows <= 32 && x.segments > 2 * kda::device_cus();
  x.pieces = kda::device_cus() * (x.many ? kPerCu : 1);
  x.parts = size_t(2 * x.pieces) * x.tile_rows * kPart * sizeof(float);
  x.bytes = x.parts + (size_t(x.segments) * 2 + x.pieces) * sizeof(int);
  return x;
}

int sizes(int32_t N, int32_t Q, int32_t H) {
  if (N < 0 || Q < 1 || Q > 1024 || H < 1 || H > 65535) return KDA_ERR_SHAPE;
  return int64_t(N) * Q * H > (1 << 24) ? KDA_ERR_SHAPE : KDA_OK;
}

}  // namespace

extern "C" size_t kda_latent_decode_workspace_size(int32_t N, int32_t Q, int32_t H) {
  return sizes(N, Q, H) == KDA_OK && N > 0 ? plan_for(N, Q, H).bytes : 0;
}

extern "C" int kda_latent_decode(const void* q, int64_t q_stride, const void* c_cache, const void* c_scale,
                                 const void* k_cache, int32_t page_size, int64_t c_page, int64_t scale_page,
                                 int64_t k_page, int32_t num_pages, const int32_t* page_table, int64_t table_stride,
                                 int32_t table_width, const int32_t* kv_lens, int32_t N, int32_t Q, int32_t H,
                                 float scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const kda::LatentCache cache{page_size, num_pages, c_page, scale_page, k_page};
  int e = sizes(N, Q, H);
  if (e == KDA_OK) e = kda::attn_scale(scale);
  if (e == KDA_OK) e = kda::latent_cache(cache);
  if (e != KDA_OK) return e;
  if (q_stride < int64_t(H) * (R + S) || q_stride > (int64_t(1) << 31)) return KDA_ERR_SHAPE;
  if (q_stride % 8) return KDA_ERR_ALIGN;
  if (num_pages < 1 || table_width < 1 || table_stride < table_width) return KDA_ERR_SHAPE;
  if (int64_t(table_width) * page_size > (1 << 30)) return KDA_ERR_SHAPE;   // token numbers and a unit or two fit int32
  if (N == 0) return KDA_OK;
  if (!q || !c_cache || !c_scale || !k_cache || !page_table || !kv_lens || !o || !workspace) return KDA_ERR_NULL;
  for (const void* y : {q, c_cache, k_cache, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (!kda::aligned16(y)) return KDA_ERR_ALIGN;
  for (const void* y : {c_scale, static_cast<const void*>(page_table), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(lse)})
    if (!kda::aligned4(y)) return KDA_ERR_ALIGN;
  const Plan x = plan_for(N, Q, H);
  if (workspace_bytes < x.bytes) return KDA_ERR_WORKSPACE;
  int* owner = reinterpret_cast<int*>(static_cast<char*>(workspace) + x.parts);
  const Params p{static_cast<const uint16_t*>(q), q_stride, static_cast<const uint8_t*>(c_cache),
                 static_cast<const uint8_t*>(c_scale), static_cast<const uint16_t*>(k_cache), uint32_t(c_page),
                 uint32_t(scale_page), uint32_t(k_page), page_table, table_stride, kv_lens, N, Q, H, table_width,
                 __builtin_ctz(page_size), num_pages, scale, static_cast<uint16_t*>(o), lse, x.rows, x.tile_rows,
                 x.row_tiles, x.pieces, static_cast<float*>(workspace), owner, owner + x.segments,
                 owner + 2 * x.segments, x.segments > x.pieces};
  const hipStream_t st = kda::as_stream(stream);
  // No more pieces than units that the tables could hold.
  const int64_t units = (int64_t(table_width) * page_size + kUnit - 1) / kUnit;
  const int64_t most = x.segments * (units + (x.many ? kManyExtra : kExtra));
  const int pieces = int(x.pieces < most ? x.pieces : most);
  const dim3 grid{unsigned(pieces)};
  if (x.many)
    hipLaunchKernelGGL(latent_decode_many_kernel, grid, dim3(kManyThreads), 0, st, p);
  else if (x.tile_rows <= 32)
    hipLaunchKernelGGL(latent_decode_kernel<2>, grid, dim3(kThreads), 0, st, p);
  else if (x.tile_rows <= 64)
    hipLaunchKernelGGL(latent_decode_kernel<4>, grid, dim3(kThreads), 0, st, p);
  else
    hipLaunchKernelGGL(latent_decode_kernel<6>, grid, dim3(kThreads), 0, st, p);
  // By the parts of a segment, about; 1, 4 and 16 streams in us: with 12 (20 sequences of up to
  // 8000 tokens, 96 heads) 64.8 and 66.2, with 16 (32 of 16 heads) 39.4 and 37.6, with 64 (8 of
  // them) 25.4 for 4 and 24.9 for 16, with 128 (4) 24.1 and 19.7.
  const unsigned joins = unsigned(p.by_piece ? pieces : x.segments) * unsigned(x.tile_rows / 16) * (R / 16);
  const int64_t each = pieces / x.segments;
  if (each < 16)
    hipLaunchKernelGGL(latent_decode_join_kernel<1>, dim3(joins / 2), dim3(64), 0, st, p);
  else if (each < 64)
    hipLaunchKernelGGL(latent_decode_join_kernel<4>, dim3(joins), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL(latent_decode_join_kernel<16>, dim3(joins), dim3(1024), 0, st, p);
  return kda::launch_status();
}
