// Attention of a few new tokens per sequence over the paged 8-bit cache of
// latents, in the absorbed form (export kda_latent_decode).
//
// A token's key is its latent and its shared part, 576 wide, and its value the
// latent, 512 wide, the same for all heads.  For query token i of Q (its position is
// len - Q + i) and head h, over the tokens j <= len - Q + i of the sequence:
//     z_j = scale q . [c_j s_j],   o = sum_j softmax(z)_j c_j.
// The Q queries of all heads are rows of one matrix, in tiles of at most 128.
//
// All (sequence, row tile) segments in order, in units of tokens, form one line
// that is cut into equal pieces, one per workgroup (attn_line.h); a segment that
// lies in several leaves float32 parts, which latent_decode_join_kernel adds up.
//
// A workgroup holds a unit in LDS as bfloat16, codes times their scales (exact),
// and uses it twice: S^T = [C s] Q^T, with 32 rows of Q in a wave's registers, and
// O^T += C^T P^T, where each wave has 128 of the 512 columns for all rows, so that
// a column is read (transposed) by one wave only.  Weights go from the waves that
// made them to all through LDS, as operands; the running maximum is common to the
// waves, sum and output are float32.  With up to 32 rows the four waves split a
// unit's keys, with more they split the rows.  The next unit's bytes are in flight
// in registers meanwhile.
#include "attn_line.h"
#include "kda_host.h"
#include "latent_device.h"

namespace {

using namespace kda::latent;
using kda::line::Piece;
using kda::line::length;
using kda::line::units_of;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kLine = 2 * (R + S);           // bytes of a token in LDS
constexpr int kMostRows = 96;                // of a row tile: the output of 96 is 192 of a wave's registers
constexpr int kPart = R + 4;                 // floats of a part's row: output, maximum, sum

struct Params {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *codes, *exponents;
  const uint16_t* shared;
  int64_t c_stride, scale_stride, s_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int N, Q, H, width, shift, num_pages;
  float scale;
  uint16_t* o;
  float* lse;
  int rows, tile_rows, row_tiles, join_rows; // Q x H; rows of one tile; tiles; rows of a joining workgroup
  int waves;                                 // pieces
  float* parts;                              // [2 x pieces][tile_rows][kPart]: a piece has one of its first segment, one of its last
  int *owner, *last_owner;                   // [segments]: first part and last piece of those cut, -1 for the others
};

// A word of four codes, times a power of two, as bfloat16 pairs.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 widen(uint32_t w, float f) {
  const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, false);
  const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, true);
  return (u32x2){__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

constexpr int kUnit = 64;                    // tokens of a unit
constexpr int kOwn = kUnit / kWaves;         // of which a wave brings 16, all in one page
constexpr int kSteps = (R + S) / 32;         // matrix instructions along a key

// As they come from the cache, 16 tokens of a wave: codes, shared parts, exponents.
constexpr int kRawShared = kOwn * R, kRawScale = kRawShared + kOwn * 2 * S, kRaw = kRawScale + 256;

// The order of a line's pieces of 16 bytes, as latent_device.h's turn, for reads of 16
// lines (16 different places, whatever the order of these bits) and of 16 columns:
// of 8 successive lines 32 bytes each, in the eight places that there are.
__device__ __forceinline__ int turn16(int line) {
  return ((line & 2) << 1) | ((line >> 1) & 2) | ((line >> 3) & 1);
}
// Where lane (l16, g4) reads lines 0 .. 15 as an operand of a 16 x 16 product,
// contraction indices 32 s + 8 g4 .. + 7 for s = 0; further ones are 64 bytes (s odd)
// beside that in the turned order, and 128 for each two on.
__device__ __forceinline__ int key_place(int l16, int g4) { return l16 * kLine + (g4 ^ turn16(l16)) * 16; }
__device__ __forceinline__ bf16x8 keys_at(const unsigned char* tile, int place, int r, int s) {
  return *reinterpret_cast<const bf16x8*>(tile + (place ^ (s & 1) * 64) + r * kLine + (s >> 1) * 128);
}
// Where lane (l16, g4) reads the transpose of lines 0 .. 31 at columns 0 .. 15: it takes
// column l16 at lines 16 (j / 4) + 4 g4 + j % 4 for j = 0 .. 7, which is the order in
// which the accumulators of two 16 x 16 products hold their rows.  Further columns are
// 32 bytes for each 16 beside that in the turned order, and 128 for each 64.
__device__ __forceinline__ int column_place(int l16, int g4) {
  const int line = 4 * g4 + (l16 >> 2);
  return line * kLine + (((l16 >> 1) & 1) ^ turn16(line)) * 16 + (l16 & 1) * 8;
}
__device__ __forceinline__ bf16x8 columns_at(const unsigned char* tile, int place, int r, int c) {
  const unsigned char* p = tile + (place ^ (c >> 4 & 3) * 32) + r * kLine + (c >> 6) * 128;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * kLine));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// Nothing moves across: operands are fetched in groups, one group ahead of the
// products that use the other.  (Left alone, the compiler reads each operand right
// before its product, and the one wave of a SIMD waits for every one of them.)
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Sum and maximum over the four lanes that hold a row.
__device__ __forceinline__ float quarter_max(float x) { return half_max(fmaxf(x, __shfl_xor(x, 16, 64))); }
__device__ __forceinline__ float quarter_sum(float x) { return half_sum(x + __shfl_xor(x, 16, 64)); }

// NT: row tiles of 16, in groups of two.
template <int NT>
__global__ __launch_bounds__(kThreads, 1) void latent_decode_kernel(Params p) {
  constexpr int kShare = NT == 2 ? 4 : NT == 4 ? 2 : 1;    // waves that split the keys of a group's rows
  constexpr int kKeys = kUnit / 16 / kShare;               // key tiles of 16 for each of them
  constexpr int kAhead = kKeys == 1 ? 6 : kKeys == 2 ? 2 : 1;   // steps of which operands are fetched together
  __shared__ __align__(1024) unsigned char tile[kUnit * kLine];
  __shared__ __align__(1024) unsigned char raw[kWaves][kRaw];
  __shared__ __align__(16) unsigned char weights[NT * 2048];
  __shared__ float top[kShare][16 * NT], sums[kShare][16 * NT];
  __shared__ int there[kUnit / 16];                        // pages of the key tiles, -1: none
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = NT == 2 ? 0 : NT == 4 ? (wave & 1) : wave; // the wave's 32 rows
  const int share = NT == 2 ? wave : NT == 4 ? (wave >> 1) : 0;
  const bool scores = 2 * g < NT;                          // of three groups the fourth wave has none

  const Piece piece = kda::line::find_piece<kUnit, 1>(p, 0, p.row_tiles);
  int64_t left = piece.to - piece.from;
  int n = piece.n, len = piece.len, units = units_of<kUnit>(len);
  const int64_t inside = piece.from - piece.before;
  int seg = int(inside / units), first = int(inside - int64_t(seg) * units);
  bool begun = false;                                      // the piece's first segment is done
  const float c = p.scale * kLog2e;

  while (left > 0) {
    // -------- one segment: sequence n, rows row0 .. row0 + tile_rows - 1
    const int row0 = seg * p.tile_rows;
    const int last = int(min(int64_t(units), first + left));
    const int rows = min(min(p.rows - row0, p.tile_rows), 16 * NT);

    // Pages of this wave's tokens in 64 units, one per lane; -1: no tokens there.
    const int32_t* table = p.table + n * p.table_stride;
    int pages = -1, pages_from = 0, id = -1;
    auto look = [&](int unit) {
      pages_from = unit;
      pages = -1;
      const int64_t token = int64_t(unit + lane) * kUnit + wave * kOwn;
      if (token < len) {
        const int x = table[token >> p.shift];
        if (x >= 0 && x < p.num_pages) pages = x;
      }
    };
    // This wave's 16 tokens of a unit as buffers that end behind the sequence, or
    // are empty: what is not there is zero in LDS.
    auto load = [&](int unit) {
      if (unit - pages_from >= 64) look(unit);
      id = __builtin_amdgcn_readlane(pages, unit - pages_from);
      const int token = unit * kUnit + wave * kOwn;
      const int exist = id < 0 ? 0 : min(len - token, kOwn);
      const int64_t page = max(id, 0);
      const int at = token & ((1 << p.shift) - 1);
      const auto cs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.codes + page * p.c_stride + at * R), 0,
                                                        exist * R, 0x00020000);
      const auto ss = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.shared + page * p.s_stride + at * S), 0,
                                                        exist * 2 * S, 0x00020000);
      const auto es = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(p.exponents + page * p.scale_stride + at * kBlocks), 0, exist * kBlocks, 0x00020000);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(cs, (lds_ptr*)(raw[wave] + j * 1024), 16, lane * 16, j * 1024, 0, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ss, (lds_ptr*)(raw[wave] + kRawShared + j * 1024), 16, lane * 16,
                                                 j * 1024, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(es, (lds_ptr*)(raw[wave] + kRawScale), 4, lane * 4, 0, 0, 0);
    };

    look(first);
    load(first);
    bf16x8 q[2][kSteps];
    int limit[2];                                          // tokens that the lane's rows see
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = row0 + min(32 * g + 16 * t + l16, rows - 1), i = r / p.H;
      const uint16_t* src = p.q + (int64_t(n) * p.Q + i) * p.q_stride + (r - i * p.H) * (R + S) + 8 * g4;
      if (scores)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[t][s] = *reinterpret_cast<const bf16x8*>(src + 32 * s);
      limit[t] = len - p.Q + i + 1;
    }
    f32x4 o[NT][8];                                        // column 128 wave + 16 d + 4 g4 + e of row 16 t + l16
    float m[NT], l[2] = {0.0f, 0.0f};                      // m: of all rows; l: own rows and keys
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);
    }

    for (int unit = first; unit < last; ++unit) {
      const int key0 = unit * kUnit;
      const bool edge = key0 + kUnit > len - p.Q + 1;      // some row does not see some key

      // -------- this wave's tokens, from codes to bfloat16
      // (Places are made anew for every unit: kept, they would take registers that
      // the queries and the output need.)
      int place_lane = lane;
      asm volatile("" : "+v"(place_lane));
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
      u32x2 code[kOwn];
      uint32_t exponent[kOwn];
      u32x4 part[2];
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        code[i] = *reinterpret_cast<const u32x2*>(raw[wave] + i * R + lane * 8);
        exponent[i] = raw[wave][kRawScale + i * kBlocks + g4];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        part[j] = *reinterpret_cast<const u32x4*>(raw[wave] + kRawShared + j * 1024 + lane * 16);
      const int from = id;
      kda::lds_barrier();                                  // the unit before is used up, and this wave has its tokens
      if (unit + 1 < last) load(unit + 1);
      // A token that only some of the queries see may hold codes of NaN, which a
      // weight of zero would not keep out of the others' products: its latent becomes
      // zero and its shared part NaN, which gives the same to those that see it (their
      // scores are NaN) and nothing to the others.
      if (edge && p.Q > 1) {
        uint32_t bad = 0;                                  // one bit for each token
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const uint32_t nan = ((code[i][0] & 0x7f7f7f7fu) + 0x01010101u) | ((code[i][1] & 0x7f7f7f7fu) + 0x01010101u);
          if (__any(nan & 0x80808080u)) {
            bad |= 1u << i;
            code[i] = (u32x2){0, 0};
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (bad >> (8 * j + (lane >> 3)) & 1) part[j] = (u32x4)(0x7fc07fc0u);
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const float f = __uint_as_float(exponent[i] << 23);
        const u32x2 a = widen(code[i][0], f), b = widen(code[i][1], f);
        *reinterpret_cast<u32x4*>(tile + (wave * kOwn + i) * kLine + (place_lane ^ turn16(i)) * 16) =
            (u32x4){a[0], a[1], b[0], b[1]};
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int line = 8 * j + (place_lane >> 3);
        *reinterpret_cast<u32x4*>(tile + (wave * kOwn + line) * kLine + ((R / 8 + (place_lane & 7)) ^ turn16(line)) * 16) =
            part[j];
      }
      if (lane == 0) there[wave] = from;
      kda::lds_barrier();

      // -------- scores of two row tiles and kKeys key tiles (rows = keys)
      f32x4 s[2][kKeys];
      if (scores) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int k = 0; k < kKeys; ++k) s[t][k] = (f32x4)(0.0f);
        bf16x8 a[2][kAhead][kKeys];
        const int place = key_place(place_lane & 15, place_lane >> 4);
        auto fetch = [&](int group) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
              a[group & 1][i][k] = keys_at(tile, place, 16 * (share * kKeys + k), group * kAhead + i);
        };
        fetch(0);
#pragma unroll
        for (int group = 0; group < kSteps / kAhead; ++group) {
          fence();
          if (group + 1 < kSteps / kAhead) fetch(group + 1);
          fence();
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int k = 0; k < kKeys; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) s[t][k] = mfma16(a[group & 1][i][k], q[t][group * kAhead + i], s[t][k]);
        }
        fence();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
          const bool gone = there[share * kKeys + k] < 0;
          if (edge || gone) {
            const int key = key0 + 16 * (share * kKeys + k) + 4 * g4;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (gone || key + e >= limit[t]) s[t][k][e] = -INFINITY;
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float mx = s[t][0][0];
#pragma unroll
          for (int k = 0; k < kKeys; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[t][k][e]);
          mx = quarter_max(mx);
          if (g4 == 0) top[share][32 * g + 16 * t + l16] = mx;
        }
      }
      kda::lds_barrier();

      // -------- the maximum of all rows, the same in all waves; weights of the own ones
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx = top[0][16 * t + l16];
#pragma unroll
        for (int i = 1; i < kShare; ++i) mx = fmaxf(mx, top[i][16 * t + l16]);
        if (__any((mx - m[t]) * c > kSlack)) {
          const float now = fmaxf(m[t], mx);
          const float f = __builtin_amdgcn_exp2f((m[t] - base(now)) * c);
          m[t] = now;
          if ((t >> 1) == g) l[t & 1] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) o[t][d] *= f;
        }
      }
      if (scores) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float b = base(m[t]);
#pragma unroll
          for (int i = 1; i < NT / 2; ++i) b = i == g ? base(m[2 * i + t]) : b;
          b *= c;
#pragma unroll
          for (int k = 0; k < kKeys; ++k) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][k][e], c, -b));
              l[t] += x[e];
            }
            const int key = share * kKeys + k;             // tile: half of a product's 32 keys
            *reinterpret_cast<u32x2*>(weights + (((2 * g + t) * 2 + (key >> 1)) * 64 + lane) * 16 + (key & 1) * 8) =
                (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
          }
        }
      }
      kda::lds_barrier();

      // -------- this wave's 128 columns of all rows
      bf16x8 w[NT], a[2][4];
      const int place = column_place(place_lane & 15, place_lane >> 4);
      auto fetch = [&](int group) {                        // 32 keys, four tiles of 16 columns
#pragma unroll
        for (int d = 0; d < 4; ++d)
          a[group & 1][d] = columns_at(tile, place, 32 * (group >> 1), 128 * wave + 64 * (group & 1) + 16 * d);
      };
      fetch(0);
#pragma unroll
      for (int group = 0; group < 4; ++group) {
        fence();
        if ((group & 1) == 0) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            w[t] = *reinterpret_cast<const bf16x8*>(weights + ((t * 2 + (group >> 1)) * 64 + lane) * 16);
        }
        if (group + 1 < 4) fetch(group + 1);
        fence();
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t][4 * (group & 1) + d] = mfma16(a[group & 1][d], w[t], o[t][4 * (group & 1) + d]);
      }
      fence();
    }

    // -------- its rows: finished, or a part
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      l[t] = quarter_sum(l[t]);
      if (scores && g4 == 0) sums[share][32 * g + 16 * t + l16] = l[t];
    }
    kda::lds_barrier();
    const bool whole = first == 0 && last == units;
    const int64_t segment = int64_t(n) * p.row_tiles + seg;
    const int slot = 2 * piece.w + int(begun);
    if (threadIdx.x == 0) {
      if (first == 0) p.owner[segment] = whole ? -1 : slot;
      if (first != 0 && last == units) p.last_owner[segment] = piece.w;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 16 * t + l16, col = 128 * wave + 4 * g4;
      float sum = sums[0][r];
#pragma unroll
      for (int i = 1; i < kShare; ++i) sum += sums[i][r];
      if (r >= rows) continue;
      if (whole) {
        const int64_t out = int64_t(n) * p.rows + row0 + r;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const f32x4 x = o[t][d] * f;
          *reinterpret_cast<u32x2*>(p.o + out * R + col + 16 * d) =
              (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
        }
        if (p.lse && wave == 0 && g4 == 0) p.lse[out] = m[t] * p.scale + __logf(sum);
      } else {
        float* to = p.parts + (int64_t(slot) * p.tile_rows + r) * kPart;
#pragma unroll
        for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(to + col + 16 * d) = o[t][d];
        if (wave == 0 && g4 == 0) to[R] = m[t], to[R + 1] = sum;
      }
    }
    left -= last - first;
    first = 0;
    begun = true;
    if (++seg == p.row_tiles) {
      seg = 0;
      if (++n < p.N) len = length(p, n), units = units_of<kUnit>(len);
    }
  }
}

// ---------------------------------------------------------------- joining the parts

// A workgroup takes join_rows rows of a segment, one after another: two streams of
// 128 lanes, four columns to a lane.
__global__ __launch_bounds__(256) void latent_decode_join_kernel(Params p) {
  __shared__ float weights[256], red[R], stat[4];
  const int tile = min(p.rows, p.tile_rows), groups = (tile + p.join_rows - 1) / p.join_rows;
  const int64_t segment = blockIdx.x / unsigned(groups);
  const int slot = p.owner[segment];
  if (slot < 0) return;                        // finished by its workgroup
  const int w0 = slot >> 1, count = p.last_owner[segment] - w0 + 1;
  const int64_t n = segment / p.row_tiles;
  const int row0 = int(segment - n * p.row_tiles) * p.tile_rows;
  const int from = int(blockIdx.x % unsigned(groups)) * p.join_rows;
  const int limit = min(min(from + p.join_rows, tile), p.rows - row0);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto over_all = [&](float x, bool most) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const float y = __shfl_xor(x, d, 64);
      x = most ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if (lane == 0) stat[wave] = x;
    __syncthreads();
    x = stat[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) x = most ? fmaxf(x, stat[i]) : x + stat[i];
    return x;
  };
  for (int r = from; r < limit; ++r) {
    // part i: the first may be its piece's last segment, the others are their pieces' first
    auto at = [&](int i) {
      return p.parts + (int64_t(i == 0 ? slot : 2 * (w0 + i)) * p.tile_rows + r) * kPart;
    };
    float m = -INFINITY;
    for (int i = tid; i < count; i += 256) m = fmaxf(m, at(i)[R]);
    m = over_all(m, true);
    const int stream = tid >> 7, col = (tid & 127) * 4;
    f32x4 acc = (f32x4)(0.0f);
    float sum = 0.0f;
    for (int i0 = 0; i0 < count; i0 += 256) {
      const int here = min(count - i0, 256);
      __syncthreads();
      if (tid < here) {
        const float f = __builtin_amdgcn_exp2f((at(i0 + tid)[R] - base(m)) * (p.scale * kLog2e));
        weights[tid] = f;
        sum += f * at(i0 + tid)[R + 1];
      }
      __syncthreads();
#pragma unroll 4
      for (int k = stream; k < here; k += 2) acc += *reinterpret_cast<const f32x4*>(at(i0 + k) + col) * weights[k];
    }
    sum = over_all(sum, false);
    if (stream == 1) *reinterpret_cast<f32x4*>(&red[col]) = acc;
    __syncthreads();
    if (stream == 0) {
      const int64_t out = n * p.rows + row0 + r;
      acc += *reinterpret_cast<const f32x4*>(&red[col]);
      acc *= sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<u32x2*>(p.o + out * R + col) =
          (u32x2){kda::pack_bf16(acc[0], acc[1]), kda::pack_bf16(acc[2], acc[3])};
      if (p.lse && tid == 0) p.lse[out] = m * p.scale + __logf(sum);
    }
  }
}

struct Plan {
  int rows, tile_rows, row_tiles, pieces;
  int64_t segments;
  size_t parts, bytes;
};

// Rows in as few tiles of at most kMostRows as they need, of equal size, in steps of
// 32.
Plan plan_for(int64_t N, int64_t Q, int H) {
  Plan x;
  x.rows = int(Q * H);
  x.row_tiles = (x.rows + kMostRows - 1) / kMostRows;
  x.tile_rows = ((x.rows + x.row_tiles - 1) / x.row_tiles + 31) / 32 * 32;
  x.pieces = kda::device_cus();
  x.segments = N * x.row_tiles;
  x.parts = size_t(2 * x.pieces) * x.tile_rows * kPart * sizeof(float);
  x.bytes = x.parts + size_t(x.segments) * 2 * sizeof(int);
  return x;
}

int sizes(int32_t N, int32_t Q, int32_t H) {
  if (N < 0 || Q < 1 || Q > 1024 || H < 1 || H > 65535) return KDA_ERR_SHAPE;
  return int64_t(N) * Q * H > (1 << 24) ? KDA_ERR_SHAPE : KDA_OK;
}

template <int NT>
void launch(const Params& p, int pieces, hipStream_t stream) {
  hipLaunchKernelGGL(latent_decode_kernel<NT>, dim3(unsigned(pieces)), dim3(kThreads), 0, stream, p);
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
  // Rows of a joining workgroup: one, or more where there would be over 4096
  // workgroups; one that finds nothing to join is not free.
  const int tile = x.rows < x.tile_rows ? x.rows : x.tile_rows;
  const int64_t share = (x.segments * tile + 4095) / 4096;
  const int join_rows = int(share < tile ? share : tile);
  int* owner = reinterpret_cast<int*>(static_cast<char*>(workspace) + x.parts);
  const Params p{static_cast<const uint16_t*>(q), q_stride, static_cast<const uint8_t*>(c_cache),
                 static_cast<const uint8_t*>(c_scale), static_cast<const uint16_t*>(k_cache), c_page, scale_page,
                 k_page, page_table, table_stride, kv_lens, N, Q, H, table_width, __builtin_ctz(page_size), num_pages,
                 scale, static_cast<uint16_t*>(o), lse, x.rows, x.tile_rows, x.row_tiles, join_rows, x.pieces,
                 static_cast<float*>(workspace), owner, owner + x.segments};
  const hipStream_t st = kda::as_stream(stream);
  if (x.tile_rows == 32)
    launch<2>(p, x.pieces, st);
  else if (x.tile_rows == 64)
    launch<4>(p, x.pieces, st);
  else
    launch<6>(p, x.pieces, st);
  const unsigned joins = unsigned(x.segments * ((tile + join_rows - 1) / join_rows));
  hipLaunchKernelGGL(latent_decode_join_kernel, dim3(joins), dim3(256), 0, st, p);
  return kda::launch_status();
}
