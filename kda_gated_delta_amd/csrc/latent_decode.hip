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
// A unit lies in LDS as it came, in codes, and is used twice: S^T = [C s] Q^T, with Q
// in registers, and O^T += C^T P^T, where each wave has 128 of the 512 columns for all
// rows, so that a column is read (transposed) by one wave only.  Codes become
// bfloat16 on their way from LDS into the operands.  A token's 128 values under one
// scale are one wave's columns: a key's scales enter as it is widened, a value's
// enter the weights, which go from the waves that made them to all through LDS, as
// operands, in four versions.  The running maximum is common to the waves, sum and
// output are float32.  The next units are on their way to LDS meanwhile.
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

// Eight codes as an operand.
__device__ __forceinline__ bf16x8 widen(uint32_t x, uint32_t y, float f) {
  const u32x2 a = widen(x, f), b = widen(y, f);
  return as_bf16x8((u32x4){a[0], a[1], b[0], b[1]});
}

constexpr int kUnit = 32;                    // tokens of a unit
constexpr int kRing = 3;                     // units in LDS
constexpr int kPerCu = 2;                    // workgroups of a compute unit
constexpr int kOwn = kUnit / kWaves;         // tokens that a wave brings, all in one page
constexpr int kLoads = kOwn / 2 + 2;         // of a wave for a unit
// A unit in LDS: codes [kUnit][512], shared parts [kUnit][128 bytes], exponents.
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

// The lane, made anew: what is made of it again for every unit takes no register from
// the queries and the output meanwhile.
__device__ __forceinline__ int lane_now() {
  int x;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
  return x;
}

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

// NT: row tiles of 16.
template <int NT>
__global__ __launch_bounds__(kThreads, kPerCu) void latent_decode_kernel(Params p) {
  constexpr int kShare = kWaves / NT, kKeys = 2 / kShare;  // waves that split a row's keys; key tiles of 16 for each
  // (One object: between two the compiler tells apart what loads to LDS write, and
  // has reads wait for all those that are on their way to the same one.)
  __shared__ __align__(1024) struct {
    unsigned char ring[kRing][kBytes];
    unsigned char weights[kBlocks][NT][1024];
    float scales[kUnit][kBlocks];
    float top[kShare][16 * NT];                            // maxima of a unit, and in the end sums
    int there[kRing][kWaves];                              // whether a wave's tokens have a page
  } lds;
  auto &ring = lds.ring;
  auto &weights = lds.weights;
  auto &scales = lds.scales;
  auto &top = lds.top;
  auto &there = lds.there;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int share = wave % kShare, mine = wave / kShare;   // the wave's keys, and its row tile

  const Piece piece = kda::line::find_piece<kUnit, 1>(p, 0, p.row_tiles);
  int64_t left = piece.to - piece.from;
  int n = piece.n, len = piece.len, units = units_of<kUnit>(len);
  const int64_t inside = piece.from - piece.before;
  int seg = __builtin_amdgcn_readfirstlane(int(inside / units));
  int first = __builtin_amdgcn_readfirstlane(int(inside - int64_t(seg) * units));
  bool begun = false;                                      // the piece's first segment is done
  const float c = p.scale * kLog2e;

  while (left > 0) {
    // -------- one segment: sequence n, rows row0 .. row0 + tile_rows - 1
    const int row0 = seg * p.tile_rows;
    const int last = int(min(int64_t(units), first + left));
    const int rows = min(min(p.rows - row0, p.tile_rows), 16 * NT);

    // The slots of this wave's first tokens in 64 units, one to a lane; -1: no page.
    const int32_t* table = p.table + n * p.table_stride;
    int from = 0, slots = -1;
    auto look = [&](int unit) {
      from = unit;
      slots = -1;
      const int64_t token = int64_t(unit + lane_now()) * kUnit + wave * kOwn;
      if (token < len) {
        const int id = table[token >> p.shift];
        if (id >= 0 && id < p.num_pages) slots = (id << p.shift) + (int(token) & ((1 << p.shift) - 1));
      }
    };
    // They come as buffers that end behind the sequence, or are empty: what is not
    // there is zero in LDS.
    auto load = [&](int unit) {
      if (unit - from >= 64) look(unit);
      const int slot = __builtin_amdgcn_readlane(slots, unit - from);
      const int some = slot < 0 ? 0 : min(len - (unit * kUnit + wave * kOwn), kOwn);
      const int64_t page = max(slot, 0) >> p.shift;
      const int at = max(slot, 0) & ((1 << p.shift) - 1);
      const auto cs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.codes + page * p.c_stride + at * R), 0,
                                                        some * R, 0x00020000);
      const auto ss = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.shared + page * p.s_stride + at * S), 0,
                                                        some * 2 * S, 0x00020000);
      const auto es = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(p.exponents + page * p.scale_stride + at * kBlocks), 0, some * kBlocks, 0x00020000);
      const int lane = lane_now();
      if (lane == 0) there[unit % kRing][wave] = some;
      unsigned char* to = ring[unit % kRing];
      const int r0 = wave * kOwn;
      const int piece0 = (lane & 31) ^ swirl(r0) ^ (lane >> 5);
#pragma unroll
      for (int j = 0; j < kOwn / 2; ++j)                   // two lines each
        __builtin_amdgcn_raw_ptr_buffer_load_lds(cs, (lds_ptr*)(to + r0 * R + j * 1024), 16,
                                                 (lane >> 5) * R + (piece0 ^ 2 * j) * 16, j * 1024, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(            // eight lines
          ss, (lds_ptr*)(to + kShared + r0 * 2 * S), 16,
          (lane >> 3) * 2 * S + ((lane & 7) ^ swirl2(r0 + (lane >> 3))) * 16, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(es, (lds_ptr*)(to + kScale + wave * 256), 4, lane * 4, 0, 0, 0);
    };

    if (begun) wait_loads<0>();                            // (stores, that would count among the loads)
    look(first);
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
    for (int i = 0; i < kRing - 1; ++i)
      if (first + i < last) load(first + i);
    // The queries are waited for before the first unit: left to the compiler they would
    // be in every unit, and with them the loads behind them.
    wait_loads<0>();
    f32x4 o[NT][8];                                        // column 128 wave + 16 d + 4 g4 + e of row 16 t + l16
    float m[NT], l = 0.0f;                                 // m: of all rows; l: own row tile and keys
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);
    }

    for (int unit = first; unit < last; ++unit) {
      const int key0 = unit * kUnit;
      const bool edge = key0 + kUnit > len - p.Q + 1;      // some row does not see some key
      unsigned char* tile = ring[unit % kRing];
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
      // A token that only some of the queries see may hold codes of NaN, which a
      // weight of zero would not keep out of the others' products: its latent becomes
      // zero and its shared part NaN, which gives the same to those that see it (their
      // scores are NaN) and nothing to the others.
      if (edge && p.Q > 1) {
#pragma unroll 1
        for (int i = 0; i < kOwn; ++i) {
          u32x2* code = reinterpret_cast<u32x2*>(tile + (wave * kOwn + i) * R) + place_lane;
          const u32x2 x = *code;
          const uint32_t nan = ((x[0] & 0x7f7f7f7fu) + 0x01010101u) | ((x[1] & 0x7f7f7f7fu) + 0x01010101u);
          if (!__any(nan & 0x80808080u)) continue;
          *code = (u32x2){0, 0};
          if (place_lane < 32)
            reinterpret_cast<uint32_t*>(tile + kShared + (wave * kOwn + i) * 2 * S)[place_lane] = 0x7fc07fc0u;
        }
      }
      kda::lds_barrier();                                  // everybody's; and the unit before is used up
      if (unit + kRing - 1 < last) load(unit + kRing - 1);

      // -------- scores of the row tile and kKeys key tiles (rows = keys)
      f32x4 s[kKeys];
      {
        float f[2][kKeys];                                 // the scales of a block, and of the next
        auto fetch_scale = [&](int block) {
#pragma unroll
          for (int k = 0; k < kKeys; ++k) f[block & 1][k] = scales[16 * (share * kKeys + k) + p16][block];
        };
        fetch_scale(0);
#pragma unroll
        for (int k = 0; k < kKeys; ++k) s[k] = (f32x4)(0.0f);
        // Rounds of kAhead pieces of 16 bytes: eight of codes, two steps each, and two of
        // the shared part.
        constexpr int kAhead = 2 / kKeys, kRounds = 10 / kAhead;
        u32x4 a[2][kAhead][kKeys];
        auto fetch = [&](int round) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
              const int at = round * kAhead + i, key = 16 * (share * kKeys + k) + p16;
              const unsigned char* from =
                  at < 8 ? tile + key * R + ((p4 ^ p16 ^ (share * kKeys + k) * 8) * 16 ^ at * 64)
                         : tile + kShared + key * 2 * S + ((4 * (at - 8) + p4) ^ swirl2(p16)) * 16;
              a[round & 1][i][k] = *reinterpret_cast<const u32x4*>(from);
            }
        };
        fetch(0);
#pragma unroll
        for (int round = 0; round < kRounds; ++round) {
          fence();
          if (round + 1 < kRounds) fetch(round + 1);
          if (round * kAhead % 2 == 0 && round * kAhead < 6) fetch_scale(round * kAhead / 2 + 1);
          fence();
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int k = 0; k < kKeys; ++k) {
                const int at = round * kAhead + i;
                const u32x4 x = a[round & 1][i][k];
                if (at < 8)
                  s[k] = mfma16(widen(x[2 * half], x[2 * half + 1], f[at >> 1 & 1][k]), q[2 * at + half], s[k]);
                else if (half == 0)
                  s[k] = mfma16(as_bf16x8(x), q[at + 8], s[k]);
              }
        }
        fence();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
          const int key = 16 * (share * kKeys + k) + 4 * p4;
          const bool gone = there[unit % kRing][key / kOwn] == 0;
          if (edge || __any(gone)) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gone || key0 + key + e >= limit) s[k][e] = -INFINITY;
          }
        }
        float mx = s[0][0];
#pragma unroll
        for (int k = 0; k < kKeys; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[k][e]);
        mx = quarter_max(mx);
        if (p4 == 0) top[share][16 * mine + p16] = mx;
      }
      kda::lds_barrier();

      // -------- the maximum of all rows, the same in all waves; weights of the own ones
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx = top[0][16 * t + p16];
#pragma unroll
        for (int i = 1; i < kShare; ++i) mx = fmaxf(mx, top[i][16 * t + p16]);
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
        float b = base(m[0]);
#pragma unroll
        for (int t = 1; t < NT; ++t) b = t == mine ? base(m[t]) : b;
        b *= c;
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
          const int key = share * kKeys + k;               // tile: half of a product's 32 keys
          f32x4 f[4];                                      // of four keys: their blocks' scales
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const f32x4*>(scales[16 * key + 4 * p4 + e]);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][e], c, -b));
            l += x[e];
          }
#pragma unroll
          for (int d = 0; d < kBlocks; ++d)
            *reinterpret_cast<u32x2*>(weights[d][mine] + place_lane * 16 + key * 8) =
                (u32x2){kda::pack_bf16(x[0] * f[0][d], x[1] * f[1][d]), kda::pack_bf16(x[2] * f[2][d], x[3] * f[3][d])};
        }
      }
      kda::lds_barrier();

      // -------- this wave's 128 columns of all rows: lane l16 takes column l16 of 16 at
      // keys 16 (j / 4) + 4 g4 + j % 4 for j = 0 .. 7, the order in which two key tiles'
      // scores made their weights.  (A transposing read gathers, in every 16 lanes, byte
      // i & 7 of the 8-byte pieces addressed by lanes (i >> 3) + 2 e into byte e of lane i.)
      bf16x8 w[NT];
      constexpr int kAhead = 8 / NT;                       // tiles of 16 columns fetched together
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
      for (int t = 0; t < NT; ++t) w[t] = *reinterpret_cast<const bf16x8*>(weights[wave][t] + place_lane * 16);
#pragma unroll
      for (int round = 0; round < 8 / kAhead; ++round) {
        fence();
        if (round + 1 < 8 / kAhead) fetch(round + 1);
        fence();
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const bf16x8 x = widen(a[round & 1][d][0], a[round & 1][d][1], 1.0f);
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t][kAhead * round + d] = mfma16(x, w[t], o[t][kAhead * round + d]);
        }
      }
      fence();
    }

    // -------- its rows: finished, or a part
    l = quarter_sum(l);
    if (g4 == 0) top[share][16 * mine + l16] = l;
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
      float sum = top[0][r];
#pragma unroll
      for (int i = 1; i < kShare; ++i) sum += top[i][r];
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

// ---------------------------------------------------------------- over 32 rows

// Eight waves, in pairs of one that makes weights and one that uses them (a unit
// later), one of each kind on every SIMD: of the scores a wave has all 32 keys of one
// or two row tiles, so that maxima and sums are its own, of the output 128 columns of
// all row tiles, which are one block of every token's scales.  The output's waves also
// bring the tokens.
constexpr int kWideThreads = 512;

// A scale: byte `block` of a token's four exponents, as a factor.
__device__ __forceinline__ float scale_of(uint32_t exponents, int block) {
  return __uint_as_float((exponents >> (8 * block) & 255u) << 23);
}

// NT: row tiles of 16.
template <int NT>
__global__ __launch_bounds__(kWideThreads, 2) void latent_decode_wide_kernel(Params p) {
  constexpr int kOwnRows = NT <= 4 ? 1 : 2;                // row tiles of a wave's scores
  constexpr int kWideRing = 4;                             // units in LDS
  constexpr int kWideBytes = kScale + kUnit * kBlocks;
  __shared__ __align__(1024) struct {
    unsigned char ring[kWideRing][kWideBytes];
    unsigned char weights[2][kBlocks][NT][1024];
    float factor[2][16 * NT];                              // of the output so far
    int grown[2][kWaves];                                  // whether a wave has factors that are not 1
    float sum[16 * NT], top[16 * NT];
    int there[kWideRing][kWaves];                          // whether a wave's tokens have a page
  } lds;
  auto &ring = lds.ring;
  auto &weights = lds.weights;
  auto &there = lds.there;
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int role = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);

  const Piece piece = kda::line::find_piece<kUnit, 1>(p, 0, p.row_tiles);
  int64_t left = piece.to - piece.from;
  int n = piece.n, len = piece.len, units = units_of<kUnit>(len);
  const int64_t inside = piece.from - piece.before;
  int seg = __builtin_amdgcn_readfirstlane(int(inside / units));
  int first = __builtin_amdgcn_readfirstlane(int(inside - int64_t(seg) * units));
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
      const int mine = wave * kOwnRows;
      const bool busy = 16 * mine < rows;
      // Rows of Q as operands.  Along a key the order is what lanes of 16 codes make it:
      // steps 2 i and 2 i + 1 are the first and second 8 of lane group g4's 16.
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

      for (int unit = first; unit < last; ++unit) {
        kda::lds_barrier();                                // the unit is there
        if (!busy) {
          if (lane == 0) lds.grown[unit & 1][wave] = 0;
          continue;
        }
        unsigned char* tile = ring[unit % kWideRing];
        const int key0 = unit * kUnit;
        const bool edge = key0 + kUnit > len - p.Q + 1;    // some row does not see some key
        const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
        f32x4 s[2][kOwnRows];
        u32x4 own[2];                                      // the exponents of this lane's keys, 16 k + 4 g4 + e
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
            scales[k] = *reinterpret_cast<const uint32_t*>(tile + kScale + (16 * k + l16) * kBlocks);
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
            if (i >= 18) own[k] = *reinterpret_cast<const u32x4*>(tile + kScale + (16 * k + 4 * g4) * kBlocks);
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
        for (int k = 0; k < 2; ++k) gone[k] = there[unit % kWideRing][2 * k + (g4 >> 1)] == 0;
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
        for (int d = 0; d < kBlocks; ++d) {                // as operands, times each block's scales
          float f[8];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * k + e] = scale_of(own[k][e], d);
#pragma unroll
          for (int t = 0; t < kOwnRows; ++t) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[4 * k + e] = s[k][t][e] * f[4 * k + e];
            *reinterpret_cast<bf16x8*>(weights[unit & 1][d][mine + t] + lane * 16) = pack8(x);
          }
        }
      }
      kda::lds_barrier();                                  // the last weights are there
      if (busy) {
#pragma unroll
        for (int t = 0; t < kOwnRows; ++t) {
          l[t] = quarter_sum(l[t]);
          if (g4 == 0) {
            lds.sum[16 * (mine + t) + l16] = l[t];
            lds.top[16 * (mine + t) + l16] = m[t];
          }
        }
      }
      kda::lds_barrier();                                  // and sums and maxima
      if (threadIdx.x == 0) {
        if (first == 0) p.owner[segment] = whole ? -1 : slot;
        if (first != 0 && last == units) p.last_owner[segment] = piece.w;
      }
    } else {
      // ======== columns 128 wave ..
      // The slots of this wave's first tokens in 64 units, one to a lane; -1: no page.
      const int32_t* table = p.table + n * p.table_stride;
      int from = 0, slots = -1;
      auto look = [&](int unit) {
        from = unit;
        slots = -1;
        const int64_t token = int64_t(unit + lane_now()) * kUnit + wave * kOwn;
        if (token < len) {
          const int id = table[token >> p.shift];
          if (id >= 0 && id < p.num_pages) slots = (id << p.shift) + (int(token) & ((1 << p.shift) - 1));
        }
      };
      // They come as buffers that end behind the sequence, or are empty: what is not
      // there is zero in LDS.  (Behind the last unit nothing comes.)
      auto load = [&](int unit) {
        if (unit - from >= 64) look(unit);
        const int slot = __builtin_amdgcn_readlane(slots, unit - from);
        const int some = slot < 0 ? 0 : min(len - (unit * kUnit + wave * kOwn), kOwn);
        const int64_t page = max(slot, 0) >> p.shift;
        const int at = max(slot, 0) & ((1 << p.shift) - 1);
        const int lane = lane_now();
        if (lane == 0) there[unit % kWideRing][wave] = some;
        unsigned char* to = ring[unit % kWideRing];
        const int r0 = wave * kOwn;
        const int piece0 = (lane & 31) ^ swirl(r0) ^ (lane >> 5);
#pragma unroll
        for (int j = 0; j < kOwn / 2; ++j)                 // two lines each
          load_lds<16>(p.codes + page * p.c_stride + at * R, some * R, to + r0 * R + j * 1024,
                       (lane >> 5) * R + (piece0 ^ 2 * j) * 16, j * 1024);
        load_lds<16>(p.shared + page * p.s_stride + at * S, some * 2 * S, to + kShared + r0 * 2 * S,  // eight lines
                     (lane >> 3) * 2 * S + ((lane & 7) ^ swirl2(r0 + (lane >> 3))) * 16, 0);
        if (lane < kOwn)
          load_lds<4>(p.exponents + page * p.scale_stride + at * kBlocks, some * kBlocks, to + kScale + r0 * kBlocks,
                      lane * 4, 0);
      };
      if (begun) wait_loads<0>();                          // (stores, that would count among the loads)
      look(first);
#pragma unroll
      for (int i = 0; i < kWideRing - 2; ++i) load(first + i);
      f32x4 o[NT][8];                                      // column 128 wave + 16 d + 4 g4 + e of row 16 t + l16
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);

      for (int unit = first; unit <= last; ++unit) {
        // this wave's tokens of the unit are there
        wait_loads<(kWideRing - 3) * kLoads>();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        // A token that only some of the queries see may hold codes of NaN, which a
        // weight of zero would not keep out of the others' products: its latent becomes
        // zero and its shared part NaN, which gives the same to those that see it (their
        // scores are NaN) and nothing to the others.
        if (p.Q > 1 && unit < last && unit * kUnit + kUnit > len - p.Q + 1) {
          unsigned char* tile = ring[unit % kWideRing];
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
        kda::lds_barrier();                                // and the weights of the unit before
        if (unit < last) load(unit + kWideRing - 2);
        if (unit == first) continue;

        // -------- the unit before: lane l16 takes column l16 of 16 at keys 16 (j / 4) + 4 g4 +
        // j % 4 for j = 0 .. 7, the order in which the scores hold them.  (A transposing
        // read gathers, in every 16 lanes, byte i & 7 of the 8-byte pieces addressed by
        // lanes (i >> 3) + 2 e into byte e of lane i.)
        const int before = unit - 1;
        unsigned char* tile = ring[before % kWideRing];
        const int lane = lane_now(), l16 = lane & 15, g4 = lane >> 4;
        const int line = ((l16 >> 1) & 3) + 4 * g4 + (l16 & 8) * 2;
        const int place = line * R + ((8 * wave) ^ swirl(line)) * 16 + (l16 & 1) * 8;
        constexpr int kTiles = 4, kAhead = 3;              // tiles of 16 columns at once; row tiles ahead
        bf16x8 w[kAhead], x[kTiles];
        u32x2 a[kTiles];
        auto fetch = [&](int group) {
#pragma unroll
          for (int d = 0; d < kTiles; ++d)
            a[d] = __builtin_bit_cast(u32x2,
                                      transposed((const lds_i32x2*)(tile + (place ^ (kTiles * group + d) * 16))));
        };
        auto fetch_weights = [&](int i) {
          w[i % kAhead] = *reinterpret_cast<const bf16x8*>(weights[before & 1][wave][i % NT] + lane * 16);
        };
        const u32x4 grown = *reinterpret_cast<const u32x4*>(lds.grown[before & 1]);
        fetch(0);
        if (__builtin_amdgcn_readfirstlane(grown[0] | grown[1] | grown[2] | grown[3])) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float f = lds.factor[before & 1][16 * t + l16];
#pragma unroll
            for (int d = 0; d < 8; ++d) o[t][d] *= f;
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) fetch_weights(i);
#pragma unroll
        for (int group = 0; group < 8 / kTiles; ++group) {
#pragma unroll
          for (int d = 0; d < kTiles; ++d) x[d] = widen(a[d][0], a[d][1], 1.0f);
          fence();
          if (group + 1 < 8 / kTiles) fetch(group + 1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int i = group * NT + t;
            if (i + kAhead - 1 < 8 / kTiles * NT) fetch_weights(i + kAhead - 1);
            fence();
#pragma unroll
            for (int d = 0; d < kTiles; ++d)
              o[t][kTiles * group + d] = mfma16(x[d], w[i % kAhead], o[t][kTiles * group + d]);
            fence();
          }
        }
      }

      // -------- its rows: finished, or a part
      wait_loads<0>();                                     // (those that brought nothing, too)
      kda::lds_barrier();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 16 * t + l16, col = 128 * wave + 4 * g4;
        if (r >= rows) continue;
        if (whole) {
          const int64_t out = int64_t(n) * p.rows + row0 + r;
          const float sum = lds.sum[r], f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const f32x4 x = o[t][d] * f;
            *reinterpret_cast<u32x2*>(p.o + out * R + col + 16 * d) =
                (u32x2){kda::pack_bf16(x[0], x[1]), kda::pack_bf16(x[2], x[3])};
          }
          if (p.lse && wave == 0 && g4 == 0) p.lse[out] = lds.top[r] * p.scale + __logf(sum);
        } else {
          float* to = p.parts + (int64_t(slot) * p.tile_rows + r) * kPart;
#pragma unroll
          for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(to + col + 16 * d) = o[t][d];
          if (wave == 0 && g4 == 0) to[R] = lds.top[r], to[R + 1] = lds.sum[r];
        }
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

// Up to 32 rows go to the kernel of four waves, more, in equal tiles of up to 128, to
// the one of eight.
Plan plan_for(int64_t N, int64_t Q, int H) {
  Plan x;
  x.rows = int(Q * H);
  x.row_tiles = (x.rows + 95) / 96;
  x.tile_rows = ((x.rows + x.row_tiles - 1) / x.row_tiles + 15) / 16 * 16;
  x.pieces = kda::device_cus() * (x.tile_rows <= 32 ? kPerCu : 1);
  x.segments = N * x.row_tiles;
  x.parts = size_t(2 * x.pieces) * x.tile_rows * kPart * sizeof(float);
  x.bytes = x.parts + size_t(x.segments) * 2 * sizeof(int);
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
  const dim3 grid(unsigned(x.pieces));
  if (x.tile_rows <= 32)
    hipLaunchKernelGGL(latent_decode_kernel<2>, grid, dim3(kThreads), 0, st, p);
  else if (x.tile_rows <= 64)
    hipLaunchKernelGGL(latent_decode_wide_kernel<4>, grid, dim3(kWideThreads), 0, st, p);
  else
    hipLaunchKernelGGL(latent_decode_wide_kernel<6>, grid, dim3(kWideThreads), 0, st, p);
  const unsigned joins = unsigned(x.segments * ((tile + join_rows - 1) / join_rows));
  hipLaunchKernelGGL(latent_decode_join_kernel, dim3(joins), dim3(256), 0, st, p);
  return kda::launch_status();
}
