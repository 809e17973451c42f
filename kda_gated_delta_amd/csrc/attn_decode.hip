// Attention of a few new tokens per sequence over the paged 8-bit cache
// (export kda_attn_decode).
//
// For query token i of Q (its position is len - Q + i) and query head h, over
// the tokens j <= len - Q + i of the sequence:
//     z_j = scale q . (kc_j ks_page(j)),   o = sum_j softmax(z)_j vc_j vs_page(j).
// The Q queries of the HQ / HKV heads that share a key/value head are rows of
// one matrix, so each byte of the cache is read once for all of them.
//
// The cache's bytes bound it: 256 per token and key/value head.  The work is
// therefore dealt out by tokens: all (sequence, head, row tile) segments in
// order, in units of 64 tokens, form one line of U units that is cut into
// equal pieces, one per wave, whatever the sequences' lengths are -- which only
// the device knows.  Waves never meet: each keeps its own running maximum, sum
// and output in registers and its loads in flight.  A segment that lies in one
// wave's piece is finished there; otherwise its waves leave float32 parts that
// attn_decode_join_kernel brings together in order.  Where the tables are short
// and the segments few, a workgroup takes a segment alone instead.
//
// S^T = K Q^T and O^T += V^T P^T on 16x16x32 matrix instructions, codes widened
// to bfloat16 (exact).  (The instructions that take e4m3 codes as they are add
// their products with fewer bits than float32 has: with each query split into
// two e4m3 terms, exactly, a score was off by 1e-5 of its products' magnitudes,
// and the kernel no faster.)  Contraction orders are chosen so that no data
// moves between lanes: K's columns as a lane loads 32 bytes of a row, V's rows
// in the order in which the accumulator of S^T holds the keys, and V's 8-byte
// loads (one key, 8 columns) turned into 8 operands by byte permutes inside the
// lane.  Weights (times the page's scale of the values) are rounded to bfloat16;
// of up to 16 rows what that left is a second term, in products of its own: the
// roundings of few rows do not average out, and there the matrix unit has time
// (64 sequences of up to 16384 tokens 174.5 and 174.7 us without and with it; with
// 32 rows it would cost 15%).  Maximum, sum and output are float32.
//
// 64 sequences of up to 16384 tokens, 32 heads on 8: 1.03 GB of codes in 165 us,
// 6.2 TB/s, and 5 us of joining; three or four waves per SIMD, or twice as
// many pieces, are slower.  2 sequences of up to 131072 tokens, 4 queries of 16
// heads on 2: 68 MB in 22.5 us and 10 of joining.  There, and the more for one
// sequence of 1000 tokens (10.7 us in one launch), the chain lengths -> table ->
// scales and codes -> products is what it takes, not the bytes.
#include "attn_line.h"
#include "kda_host.h"

namespace {

using namespace kda::attn;
using kda::line::Piece;
using kda::line::length;
using kda::line::units_of;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kAloneWaves = 8;               // of a workgroup that takes a segment alone
constexpr int kUnit = 64;                    // tokens

struct Params {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int N, Q, HQ, HKV, width, shift, num_pages;
  int64_t page_stride;
  float scale;
  uint16_t* o;
  float* lse;
  int rows, tile_rows, row_tiles, join_rows; // Q x group; rows of one tile; tiles; rows of a joining workgroup
  int waves;
  float* parts;                              // [waves + segments][tile_rows][D + 4]: output, maximum, sum
  int *owner, *last_owner;                   // [segments]: first and last wave of those cut, -1 for the others
};

// ---------------------------------------------------------------- codes to operands

// Eight codes (two words) as eight bfloat16 values.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
  const bf16x2 w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2 w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2 w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2 w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return (bf16x8){w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
}

// Pages of up to 64 successive tiles of 16 tokens, one per lane.
struct Pages {
  int id;            // -1: no tokens there
  float ks, vs;
};

// kAlone: a workgroup of eight waves takes a segment alone, an eighth of its
// units each, and finishes it: no parts, no second launch (alone says when).
// kStream: codes are loaded past the last cache level (streams says when).
template <int NT, bool kAlone, bool kStream>
__global__ __launch_bounds__(kAlone ? 64 * kAloneWaves : kThreads, 2) void attn_decode_kernel(Params p) {
  constexpr int kGroup = kAlone ? kAloneWaves : kWaves;
  constexpr int kHint = kStream ? 2 : 0;     // non-temporal
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  __shared__ __align__(16) float merged[kGroup][16 * NT][D + 4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = p.HKV * p.row_tiles;
  int64_t left = 1;                          // units of the wave's piece that are still to do
  int w = 0, n, len, units, seg, first;
  bool merge = kAlone;                       // all waves of the workgroup inside one segment: one part for them
  if constexpr (kAlone) {
    n = int(blockIdx.x / unsigned(per));
    seg = int(blockIdx.x - unsigned(n) * unsigned(per));
    len = length(p, n);
    units = units_of<kUnit>(len);
    first = units * wave / kGroup;
  } else {
    const Piece piece = kda::line::find_piece<kUnit, kWaves>(p, wave, per);
    w = piece.w;
    left = piece.to - piece.from;
    n = piece.n;
    len = piece.len;
    units = units_of<kUnit>(len);
    const int64_t inside = piece.from - piece.before;
    seg = int(inside <= 0x7fffffff ? int64_t(unsigned(inside) / unsigned(units)) : inside / units);
    first = int(inside - int64_t(seg) * units);
    const int64_t start = piece.from - first;                     // the segment's first unit in the line
    merge = piece.lo < piece.hi && start <= piece.lo && piece.hi <= start + units;
  }
  const int G = p.HQ / p.HKV;
  const float c = p.scale * kLog2e;

  // The arguments are read anew for each segment: kept over the walk of the one
  // before, they would take scalar registers that it has not got.
  typedef const __attribute__((address_space(4))) Params Arguments;
  Arguments* arguments = (Arguments*)__builtin_amdgcn_kernarg_segment_ptr();
  while (left > 0) {
    asm volatile("" : "+s"(arguments));
    Arguments& args = *arguments;
    // -------- one segment: sequence n, head hkv, rows row0 .. row0 + tile_rows - 1
    const int hkv = seg / args.row_tiles, row0 = (seg - hkv * args.row_tiles) * args.tile_rows;
    const int last = kAlone ? units * (wave + 1) / kGroup         // units first .. last - 1, none perhaps
                            : int(min(int64_t(units), first + left));
    const int rows = min(args.rows - row0, 16 * NT);

    f32x4 o[NT][8];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY, l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[t][d] = (f32x4)(0.0f);
    }

    const int32_t* table = args.table + n * args.table_stride;
    auto pages_at = [&](int unit) {          // of the 64 tiles from `unit` on, as far as the piece goes
      Pages x{-1, 0.0f, 0.0f};
      const int64_t token = int64_t(unit) * kUnit + lane * 16;
      if (token < min(int64_t(len), int64_t(last) * kUnit)) {
        const int id = table[token >> args.shift];
        if (id >= 0 && id < args.num_pages) {
          x.id = id;
          x.ks = args.k_scale[int64_t(id) * args.HKV + hkv] * c;
          x.vs = args.v_scale[int64_t(id) * args.HKV + hkv];
        }
      }
      return x;
    };
    // Tile j (0 .. 3) of a unit whose pages start at lane `from`, as a buffer of
    // 2 KB (its address stays in scalar registers); a tile without tokens reads
    // page 0, and is masked.
    auto tile_at = [&](const uint8_t* cache, const Pages& x, int unit, int from, int j) {
      const int id = max(__builtin_amdgcn_readlane(x.id, from + j), 0);
      const int inside = (unit * kUnit + 16 * j) & ((1 << args.shift) - 1);
      const int64_t at = int64_t(id) * args.page_stride + ((int64_t(hkv) << args.shift) + inside) * D;
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(cache) + at, 0, 16 * D, 0x00020000);
    };
    const int k_off = l16 * D + 32 * g4, v_off = 4 * g4 * D + 8 * l16;
    u32x4 kr[4][2];                          // tile j: 32 bytes of row l16 from byte 32 g4
    u32x2 vr[4][4];                          // tile j: bytes 8 l16 .. + 7 of rows 4 g4 .. + 3
    auto load_k = [&](const Pages& x, int unit, int from) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto tile = tile_at(args.k_cache, x, unit, from, j);
#pragma unroll
        for (int i = 0; i < 2; ++i) kr[j][i] = __builtin_amdgcn_raw_buffer_load_b128(tile, k_off + 16 * i, 0, kHint);
      }
    };
    auto load_v = [&](const Pages& x, int unit, int from) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto tile = tile_at(args.v_cache, x, unit, from, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[j][i] = __builtin_amdgcn_raw_buffer_load_b64(tile, v_off + i * D, 0, kHint);
      }
    };

    // the chain table -> codes is the longest: it starts before the queries
    Pages now = pages_at(first);
    load_k(now, first, 0);
    load_v(now, first, 0);
    bf16x8 q[NT][4];
    int limit[NT];                           // tokens that the lane's row sees
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = row0 + min(16 * t + l16, rows - 1), i = r / G;
      const uint16_t* src = args.q + (int64_t(n) * args.Q + i) * args.q_stride + (hkv * G + r - i * G) * D + 32 * g4;
#pragma unroll
      for (int s = 0; s < 4; ++s) q[t][s] = *reinterpret_cast<const bf16x8*>(src + 8 * s);
      limit[t] = len - args.Q + i + 1;
    }
    int from = 0;                            // the unit's first tile in `now`
    uint32_t late = 0;                       // units left for the end, from that of token len - Q + 1 on
    for (int unit = first; unit < last; ++unit) {
      const int key0 = unit * kUnit;
      const bool masked = key0 + kUnit > len - args.Q + 1 || (__ballot(now.id < 0) >> from & 15) != 0;
      f32x4 s[NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][j] = (f32x4)(0.0f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x8 a = widen(kr[j][k >> 1][2 * (k & 1)], kr[j][k >> 1][2 * (k & 1) + 1]);
#pragma unroll
          for (int t = 0; t < NT; ++t) s[t][j] = mfma16(a, q[t][k], s[t][j]);
        }
      }
      float ks[4], vs[4];
      bool none[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ks[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now.ks), from + j));
        vs[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now.vs), from + j));
        none[j] = __builtin_amdgcn_readlane(now.id, from + j) < 0;
      }
      // the next unit's keys, in flight over the softmax and the second product
      const bool more = unit + 1 < last;
      Pages then = now;
      int then_from = from + 4;
      if (more) {
        if (then_from == 64) then = pages_at(unit + 1), then_from = 0;
        load_k(then, unit + 1, then_from);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[t][j] *= ks[j];
        if (masked) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (none[j] || key0 + 16 * j + 4 * g4 + e >= limit[t]) s[t][j][e] = -INFINITY;
        }
        float mx = s[t][0][0];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[t][j][e]);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = half_max(mx);
        if (__any(mx - m[t] > kSlack)) {
          const float top = fmaxf(m[t], mx);
          const float f = __builtin_amdgcn_exp2f(m[t] - (top == -INFINITY ? 0.0f : top));
          m[t] = top;
          l[t] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) o[t][d] *= f;
        }
        const float b = m[t] == -INFINITY ? 0.0f : m[t];    // a row that has seen nothing stays at zero
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __builtin_amdgcn_exp2f(s[t][j][e] - b);
            l[t] += x;
            s[t][j][e] = x * vs[j];
          }
      }
      // What lies behind the end may be anything, NaN codes too, which a weight of
      // zero does not keep out of a product.  Nor would it keep a NaN among the
      // last Q - 1 tokens out of the queries before it: such a unit's are left for
      // the end of the segment.
      if (masked) {
        auto clear = [&](int from_key) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (none[j] || key0 + 16 * j + 4 * g4 + i >= from_key) vr[j][i] = (u32x2){0, 0};
        };
        clear(len);
        if (args.Q > 1) {
          const int some = len - args.Q + 1;    // the first token that not all queries see
          uint32_t nan = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 16 * j + 4 * g4 + i >= some)
                nan |= ((vr[j][i][0] & 0x7f7f7f7fu) + 0x01010101u) | ((vr[j][i][1] & 0x7f7f7f7fu) + 0x01010101u);
          if (__any(nan & 0x80808080u)) {
            clear(some);
            late |= 1u << (unit - max(some, 0) / kUnit);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        bf16x8 pb[NT], rest;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = s[t][j][e], x[4 + e] = s[t][j + 1][e];
          pb[t] = pack8(x);
          if constexpr (NT == 1) rest = pack8_rest(x, pb[t]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)          // columns 8 l16 + 4 b + 0 .. 3
#pragma unroll
          for (int d = 0; d < 4; d += 2) {
            // bytes d and d + 1 of eight keys -> the codes of column d, then of column d + 1
            uint32_t two[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int jj = j + (e >> 1), i = 2 * (e & 1);
              two[e] = __builtin_amdgcn_perm(vr[jj][i + 1][b], vr[jj][i][b], d ? 0x07030602u : 0x05010400u);
            }
            bf16x2 lo[4], hi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(two[e], 1.0f, false);
              hi[e] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(two[e], 1.0f, true);
            }
            const bf16x8 a0 = {lo[0][0], lo[0][1], lo[1][0], lo[1][1], lo[2][0], lo[2][1], lo[3][0], lo[3][1]};
            const bf16x8 a1 = {hi[0][0], hi[0][1], hi[1][0], hi[1][1], hi[2][0], hi[2][1], hi[3][0], hi[3][1]};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              o[t][4 * b + d] = mfma16(a0, pb[t], o[t][4 * b + d]);
              o[t][4 * b + d + 1] = mfma16(a1, pb[t], o[t][4 * b + d + 1]);
            }
            if constexpr (NT == 1) {
              o[0][4 * b + d] = mfma16(a0, rest, o[0][4 * b + d]);
              o[0][4 * b + d + 1] = mfma16(a1, rest, o[0][4 * b + d + 1]);
            }
          }
      }
      if (more) load_v(then, unit + 1, then_from);
      now = then;
      from = then_from;
    }

    // -------- the tokens that were left: one by one, each to the queries that see it
    while (late) {
      const int unit = max(len - args.Q + 1, 0) / kUnit + __builtin_ctz(late);
      late &= late - 1;
#pragma unroll 1
      for (int key = max(unit * kUnit, max(len - args.Q + 1, 0)); key < min((unit + 1) * kUnit, len); ++key) {
        const int id = table[key >> args.shift];
        if (id < 0 || id >= args.num_pages) continue;
        const int64_t scale = int64_t(id) * args.HKV + hkv, inside = key & ((1 << args.shift) - 1);
        const float ks = args.k_scale[scale] * c, vs = args.v_scale[scale];
        const int64_t at = int64_t(id) * args.page_stride + ((int64_t(hkv) << args.shift) + inside) * D;
        const u32x4* kp = reinterpret_cast<const u32x4*>(args.k_cache + at + 32 * g4);
        const u32x4* vp = reinterpret_cast<const u32x4*>(args.v_cache + at + 32 * g4);
        float kx[32], vx[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 a = widen(kp[i >> 1][2 * (i & 1)], kp[i >> 1][2 * (i & 1) + 1]);
          const bf16x8 b = widen(vp[i >> 1][2 * (i & 1)], vp[i >> 1][2 * (i & 1) + 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) kx[8 * i + j] = float(a[j]), vx[8 * i + j] = float(b[j]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i) x = __builtin_fmaf(float(q[t][i >> 3][i & 7]), kx[i], x);
          x += __shfl_xor(x, 16, 64);
          x = __builtin_amdgcn_exp2f(half_sum(x) * ks - (m[t] == -INFINITY ? 0.0f : m[t])) * vs;
          if (key >= limit[t]) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int d = 0; d < 8; ++d) o[t][d][e] = __builtin_fmaf(x, vx[8 * e + d], o[t][d][e]);
        }
      }
    }

    // -------- its rows: finished, or a part.  Lane (l16, g4) holds row l16,
    // columns 8 (4 g4 + e) + d in o[d][e].
    const bool whole = !kAlone && first == 0 && last == units;
    const int64_t segment = int64_t(n) * per + seg;
    if (!kAlone && first == 0 && lane == 0) args.owner[segment] = whole ? -1 : w;
    if (!kAlone && first != 0 && last == units && lane == 0) args.last_owner[segment] = w;
    float* parts = args.parts + (segment + w) * args.tile_rows * (D + 4);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float sum = l[t] + __shfl_xor(l[t], 16, 64);
      sum = half_sum(sum);
      const int r = 16 * t + l16;
      if (r >= rows) continue;
      if (whole) {
        const int i = (row0 + r) / G, head = hkv * G + row0 + r - i * G;
        const int64_t out = (int64_t(n) * args.Q + i) * args.HQ + head;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[8];
#pragma unroll
          for (int d = 0; d < 8; ++d) x[d] = o[t][d][e] * f;
          *reinterpret_cast<bf16x8*>(args.o + out * D + 8 * (4 * g4 + e)) = pack8(x);
        }
        if (args.lse && g4 == 0) args.lse[out] = (m[t] + __log2f(sum)) * kLn2;
      } else {
        auto put = [&](auto* part) {         // LDS or global memory
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int d = 0; d < 8; d += 4)
              *reinterpret_cast<f32x4*>(part + 8 * (4 * g4 + e) + d) =
                  (f32x4){o[t][d][e], o[t][d + 1][e], o[t][d + 2][e], o[t][d + 3][e]};
          if (g4 == 0) part[D] = m[t], part[D + 1] = sum;
        };
        if (merge)
          put(&merged[wave][r][0]);
        else
          put(parts + r * (D + 4));
      }
    }
    if (merge) {                             // the same for all the waves, and each one's only segment
      __syncthreads();
      // 32 threads per row; the first wave's slot takes the sum, the others' say that they are empty
      const int col = (threadIdx.x & 31) * 4;
      for (int r = threadIdx.x >> 5; r < rows; r += kGroup * 2) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) top = fmaxf(top, merged[i][r][D]);
        const float base = top == -INFINITY ? 0.0f : top;
        f32x4 acc = (f32x4)(0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float f = __builtin_amdgcn_exp2f(merged[i][r][D] - base);
          acc += *reinterpret_cast<const f32x4*>(&merged[i][r][col]) * f;
          sum += merged[i][r][D + 1] * f;
        }
        if constexpr (kAlone) {
          const int i = (row0 + r) / G;
          const int64_t out = (int64_t(n) * args.Q + i) * args.HQ + hkv * G + row0 + r - i * G;
          acc *= sum == 0.0f ? 0.0f : 1.0f / sum;
          *reinterpret_cast<u32x2*>(args.o + out * D + col) =
              (u32x2){kda::pack_bf16(acc[0], acc[1]), kda::pack_bf16(acc[2], acc[3])};
          if (args.lse && col == 0) args.lse[out] = (top + __log2f(sum)) * kLn2;
          continue;
        }
        float* part = args.parts + ((segment + w - wave) * args.tile_rows + r) * (D + 4);
        *reinterpret_cast<f32x4*>(part + col) = acc;
        if (col == 0) {
          part[D] = top, part[D + 1] = sum;
          for (int i = 1; i < kWaves; ++i) {
            part[i * args.tile_rows * (D + 4) + D] = -INFINITY;
            part[i * args.tile_rows * (D + 4) + D + 1] = 0.0f;
          }
        }
      }
      return;
    }
    left -= last - first;
    first = 0;
    if (++seg == per) {
      seg = 0;
      if (++n < args.N) len = length(args, n), units = units_of<kUnit>(len);
    }
  }
}

// ---------------------------------------------------------------- joining the parts

// A workgroup takes join_rows rows of a segment.  Of few parts (at most 64) a
// wave adds up a row's alone, without a barrier, two columns to a lane; of many,
// THREADS / 32 streams of 32 lanes do, row after row, four columns to a lane.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void attn_decode_join_kernel(Params p) {
  constexpr int kStreams = THREADS / 32, kW = THREADS / 64;
  __shared__ float weights[THREADS], red[kStreams][D], stat[kW];
  __shared__ int places[THREADS], counts[kW];
  const int per = p.HKV * p.row_tiles, tile = min(p.rows, p.tile_rows);
  const int groups = (tile + p.join_rows - 1) / p.join_rows;
  const int64_t segment = blockIdx.x / unsigned(groups);
  const int w0 = p.owner[segment];
  if (w0 < 0) return;                        // finished by its wave
  const int w1 = p.last_owner[segment];
  const int n = int(segment / per), seg = int(segment - int64_t(n) * per);
  const int hkv = seg / p.row_tiles, row0 = (seg - hkv * p.row_tiles) * p.tile_rows;
  const int first = int(blockIdx.x % unsigned(groups)) * p.join_rows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t step = int64_t(p.tile_rows) * (D + 4);
  const int count = w1 - w0 + 1;             // slots of successive waves follow one another

  const int limit = min(min(first + p.join_rows, tile), p.rows - row0), G = p.HQ / p.HKV;
  if (count <= 64) {
    for (int r = first + wave; r < limit; r += kW) {
      const float* part = p.parts + ((segment + w0) * p.tile_rows + r) * (D + 4);
      float mine = -INFINITY, of = 0.0f;
      if (lane < count) mine = part[lane * step + D], of = part[lane * step + D + 1];
      float m = mine;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d, 64));
      const float f = __builtin_amdgcn_exp2f(mine - (m == -INFINITY ? 0.0f : m));
      const bool some = f != 0.0f || of != of; // a part whose scores are all NaN has no maximum
      float sum = some ? f * of : 0.0f;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
      float x = 0.0f, y = 0.0f;
      uint64_t have = __ballot(some);
      while (have) {                         // eight at a time: their loads go out together
        int i[8];
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          i[k] = have ? __builtin_ctzll(have) : -1;
          v[k] = reinterpret_cast<const float2*>(part + (have ? i[k] : i[0]) * step)[lane];
          have &= have - 1;                  // 0 stays 0
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i[k] >= 0) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i[k]));
            x = __builtin_fmaf(v[k].x, w, x), y = __builtin_fmaf(v[k].y, w, y);
          }
      }
      const int row = row0 + r, i = row / G;
      const int64_t out = (int64_t(n) * p.Q + i) * p.HQ + hkv * G + row - i * G;
      const float g = sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<uint32_t*>(p.o + out * D + 2 * lane) = kda::pack_bf16(x * g, y * g);
      if (p.lse && lane == 0) p.lse[out] = (m + __log2f(sum)) * kLn2;
    }
    return;
  }

  auto over_all = [&](float x, bool top) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const float y = __shfl_xor(x, d, 64);
      x = top ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if (lane == 0) stat[wave] = x;
    __syncthreads();
    x = stat[0];
#pragma unroll
    for (int i = 1; i < kW; ++i) x = top ? fmaxf(x, stat[i]) : x + stat[i];
    return x;
  };
  for (int r = first; r < limit; ++r) {
    const int row = row0 + r;
    const float* part = p.parts + ((segment + w0) * p.tile_rows + r) * (D + 4);
    float m = -INFINITY;
    for (int i = tid; i < count; i += THREADS) m = fmaxf(m, part[i * step + D]);
    m = over_all(m, true);
    const float base = m == -INFINITY ? 0.0f : m;
    const int stream = tid >> 5, col = (tid & 31) * 4;
    f32x4 acc = (f32x4)(0.0f);
    float sum = 0.0f;
    for (int i0 = 0; i0 < count; i0 += THREADS) {
      const int i = i0 + tid;
      float f = 0.0f, of = 0.0f;
      if (i < count) f = __builtin_amdgcn_exp2f(part[i * step + D] - base), of = part[i * step + D + 1];
      const bool some = f != 0.0f || of != of; // a part whose scores are all NaN has no maximum
      if (some) sum += f * of;
      const uint64_t have = __ballot(some);
      __syncthreads();
      if (lane == 0) counts[wave] = __builtin_popcountll(have);
      __syncthreads();
      int at = __builtin_popcountll(have & ((uint64_t(1) << lane) - 1)), here = 0;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        if (k < wave) at += counts[k];
        here += counts[k];
      }
      if (some) places[at] = i, weights[at] = f;
      __syncthreads();
#pragma unroll 8
      for (int k = stream; k < here; k += kStreams)
        acc += *reinterpret_cast<const f32x4*>(part + places[k] * step + col) * weights[k];
    }
    sum = over_all(sum, false);
    *reinterpret_cast<f32x4*>(&red[stream][col]) = acc;
    __syncthreads();
    if (tid < 32) {
#pragma unroll
      for (int s = 1; s < kStreams; ++s) acc += *reinterpret_cast<const f32x4*>(&red[s][col]);
      const int i = row / G;
      const int64_t out = (int64_t(n) * p.Q + i) * p.HQ + hkv * G + row - i * G;
      const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
      acc *= f;
      *reinterpret_cast<u32x2*>(p.o + out * D + col) =
          (u32x2){kda::pack_bf16(acc[0], acc[1]), kda::pack_bf16(acc[2], acc[3])};
      if (p.lse && tid == 0) p.lse[out] = (m + __log2f(sum)) * kLn2;
    }
  }
}

struct Plan {
  int rows, tile_rows, row_tiles, waves;
  int64_t segments;
  size_t parts, bytes;
};

// Rows in tiles of 16 (one matrix instruction) or 32.  Eight waves per compute
// unit, two per SIMD: with 16 KB of a unit in flight in each they cover the
// memory's latency.
Plan plan_for(int64_t N, int64_t Q, int HQ, int HKV) {
  Plan x;
  x.rows = int(Q * (HQ / HKV));
  x.tile_rows = x.rows <= 16 ? 16 : 32;
  x.row_tiles = (x.rows + x.tile_rows - 1) / x.tile_rows;
  x.waves = kda::device_cus() * 8;
  x.segments = N * HKV * x.row_tiles;
  x.parts = size_t(x.waves + x.segments) * x.tile_rows * (D + 4) * sizeof(float);
  x.bytes = x.parts + size_t(x.segments) * 2 * sizeof(int);
  return x;
}

// Whether every segment has a workgroup alone.  The host knows what the tables
// can hold, not the lengths.  A wave then walks up to an eighth of a segment, at
// 2.6 us per unit where little else runs; the line balances that, for a second
// launch and the parts' way through memory.  32 heads on 8, lengths up to the
// stated one and tables as wide as the longest, line and alone in us:
//   1 sequence: 1000 tokens 12.5 and 10.8, 2000 12.9 and 16.0, 4096 13.0 and 26.7
//   16: 1000 tokens 15.1 and 11.5, 1536 15.8 and 14.5, 3000 20.7 and 22.3, 4096 24.2 and 27.9
//   24: 1000 tokens 15.5 and 11.9, 2000 20.6 and 17.6, 3000 24.5 and 22.9, 4096 29.9 and 31.6
//   64: 250 tokens 15.9 and 13.2, 1000 23.8 and 22.1, 2000 37.8 and 39.7, 4096 60.0 and 60.7
//   128: 60 tokens 12.6 and 19.2 (a workgroup fills a compute unit, and four wait for each)
// From 2000 tokens on the two are near each other; either may be faster by a tenth.
bool alone(int64_t segments, int64_t tokens) {
  const int64_t cus = kda::device_cus();
  if (segments > 2 * cus) return false;
  return tokens <= 24 * kUnit || (tokens <= 64 * kUnit && 4 * segments >= 3 * cus);
}

// Whether a call may read so many codes that little of them is left in the last
// cache level (256 MB) when it comes again, after other layers': then loading
// past it is faster.  What fits should stay there.  Through it against past it,
// us, by the bytes read, three caches in turn (32 heads on 8; the 68 MB: 4
// queries of 16 heads on 2):
//   1029 MB 198 and 175, 500 MB 117 and 105, 200 MB 46.6 and 41.3, 134 MB 44.3 and 41.8, 107 MB 39.7 and 38.0,
//   68 MB 33.3 and 35.1, 61 MB 21.9 and 22.5, 35 MB 22.5 and 24.7
bool streams(int64_t N, int64_t table_width, int64_t num_pages, int64_t page_size, int64_t HKV) {
  const int64_t pages = N * table_width < num_pages ? N * table_width : num_pages;
  return pages * page_size * HKV * 2 * D > int64_t(96) << 20;
}

int sizes(int32_t N, int32_t Q, int32_t HQ, int32_t HKV, int32_t Dh) {
  const int e = kda::attn_heads(HQ, HKV, Dh);
  if (e != KDA_OK) return e;
  if (N < 0 || Q < 1 || Q > 1024 || int64_t(N) * HKV * Q * (HQ / HKV) > (1 << 26)) return KDA_ERR_SHAPE;
  if (int64_t(N) * HKV > kda::kMostBlocks) return KDA_ERR_SHAPE;   // joining workgroups: with more rows there are fewer
  return KDA_OK;
}

}  // namespace

extern "C" size_t kda_attn_decode_workspace_size(int32_t N, int32_t Q, int32_t HQ, int32_t HKV, int32_t Dh) {
  return sizes(N, Q, HQ, HKV, Dh) == KDA_OK && N > 0 ? plan_for(N, Q, HQ, HKV).bytes : 0;
}

extern "C" int kda_attn_decode(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, int32_t page_size, int64_t page_stride,
                               int32_t num_pages, const int32_t* page_table, int64_t table_stride,
                               int32_t table_width, const int32_t* kv_lens, int32_t N, int32_t Q, int32_t HQ,
                               int32_t HKV, int32_t Dh, float scale, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  int e = sizes(N, Q, HQ, HKV, Dh);
  if (e == KDA_OK) e = kda::attn_scale(scale);
  if (e == KDA_OK) e = kda::attn_stride(q_stride, HQ);
  if (e == KDA_OK) e = kda::attn_cache(HKV, page_size, page_stride, num_pages);
  if (e != KDA_OK) return e;
  if (num_pages < 1 || table_width < 1 || table_stride < table_width) return KDA_ERR_SHAPE;
  if (int64_t(table_width) * page_size > (1 << 30)) return KDA_ERR_SHAPE;   // token numbers and a unit or two fit int32
  if (N == 0) return KDA_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !page_table || !kv_lens || !o || !workspace)
    return KDA_ERR_NULL;
  for (const void* x : {q, k_cache, v_cache, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (!kda::aligned16(x)) return KDA_ERR_ALIGN;
  const Plan x = plan_for(N, Q, HQ, HKV);
  if (workspace_bytes < x.bytes) return KDA_ERR_WORKSPACE;
  // Rows of a joining workgroup: one where segments are few and have many parts
  // each, four (a wave each) otherwise, and more where there would be over 4096
  // workgroups: most segments of a large batch are finished by one wave, and a
  // workgroup that finds nothing to join is not free.
  const int tile = x.rows < x.tile_rows ? x.rows : x.tile_rows;
  const bool many = x.waves / x.segments >= 64;
  int64_t share = (x.segments * tile + 4095) / 4096;
  if (!many && share < 4) share = 4;
  const int join_rows = int(share < tile ? share : tile);
  int* owner = reinterpret_cast<int*>(static_cast<char*>(workspace) + x.parts);
  const Params p{static_cast<const uint16_t*>(q), q_stride, static_cast<const uint8_t*>(k_cache),
                 static_cast<const uint8_t*>(v_cache), k_scale, v_scale, page_table, table_stride, kv_lens,
                 N, Q, HQ, HKV, table_width, __builtin_ctz(page_size), num_pages, page_stride, scale,
                 static_cast<uint16_t*>(o), lse, x.rows, x.tile_rows, x.row_tiles, join_rows, x.waves,
                 static_cast<float*>(workspace), owner, owner + x.segments};
  const hipStream_t st = kda::as_stream(stream);
  if (alone(x.segments, int64_t(table_width) * page_size)) {
    const dim3 grid(unsigned(x.segments));
    if (x.tile_rows == 16)
      hipLaunchKernelGGL((attn_decode_kernel<1, true, false>), grid, dim3(64 * kAloneWaves), 0, st, p);
    else
      hipLaunchKernelGGL((attn_decode_kernel<2, true, false>), grid, dim3(64 * kAloneWaves), 0, st, p);
    return kda::launch_status();
  }
  const dim3 grid(unsigned(x.waves / kWaves));
  const bool stream_past = streams(N, table_width, num_pages, page_size, HKV);
  if (x.tile_rows == 16 && stream_past)
    hipLaunchKernelGGL((attn_decode_kernel<1, false, true>), grid, dim3(kThreads), 0, st, p);
  else if (x.tile_rows == 16)
    hipLaunchKernelGGL((attn_decode_kernel<1, false, false>), grid, dim3(kThreads), 0, st, p);
  else if (stream_past)
    hipLaunchKernelGGL((attn_decode_kernel<2, false, true>), grid, dim3(kThreads), 0, st, p);
  else
    hipLaunchKernelGGL((attn_decode_kernel<2, false, false>), grid, dim3(kThreads), 0, st, p);
  const dim3 joins(unsigned(x.segments * ((tile + join_rows - 1) / join_rows)));
  if (many)
    hipLaunchKernelGGL(attn_decode_join_kernel<1024>, joins, dim3(1024), 0, st, p);
  else
    hipLaunchKernelGGL(attn_decode_join_kernel<256>, joins, dim3(256), 0, st, p);
  return kda::launch_status();
}
