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

template <int NT>
constexpr int unit_tokens() { return NT == 1 ? 128 : 64; }

// NT: row tiles of 32.
template <int NT>
__global__ __launch_bounds__(kThreads, 1) void latent_decode_kernel(Params p) {
  constexpr int kUnit = unit_tokens<NT>();
  constexpr int kShare = NT == 1 ? 4 : NT == 2 ? 2 : 1;    // waves that split the keys of 32 rows
  constexpr int kKeys = kUnit / kShare / 32;               // blocks of 32 keys for each of them
  constexpr int kOwn = kUnit / kWaves;                     // tokens that a wave brings
  constexpr int kGroups = kOwn / 16;                       // the same in groups of 16, each within a page
  __shared__ __align__(1024) unsigned char tile[kUnit * kLine];
  __shared__ __align__(16) unsigned char weights[NT * (kUnit / 32) * 2048];
  __shared__ float top[kShare][32 * NT], sums[kShare][32 * NT];
  __shared__ int there[kUnit / 16];                        // whether a group's page exists
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = NT == 1 ? 0 : NT == 2 ? (wave & 1) : wave; // the wave's 32 rows
  const int share = NT == 1 ? wave : NT == 2 ? (wave >> 1) : 0;
  const bool scores = g < NT;                              // of three row tiles the fourth wave has none

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
    const int rows = min(min(p.rows - row0, p.tile_rows), 32 * NT);

    f32x16 o[NT][4];
    float m[NT], l = 0.0f;                                 // m: of all rows; l: own rows and keys
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[t][d] = (f32x16)(0.0f);
    }

    // Pages of this wave's next groups, one per lane; -1: no tokens there.
    const int32_t* table = p.table + n * p.table_stride;
    int pages = -1, pages_from = 0;
    auto look = [&](int unit) {
      pages_from = unit;
      pages = -1;
      const int64_t token = int64_t(unit + lane / kGroups) * kUnit + wave * kOwn + lane % kGroups * 16;
      if (token < len) {
        const int id = table[token >> p.shift];
        if (id >= 0 && id < p.num_pages) pages = id;
      }
    };
    // A group's 16 tokens as buffers that end behind the sequence, or are empty:
    // what is not there reads as zero.
    u32x4 code[kGroups][8], part[kGroups][2];
    uint32_t exponent[kGroups];
    int ids[kGroups];
    auto load = [&](int unit) {
      if (unit - pages_from >= 64 / kGroups) look(unit);
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        ids[i] = __builtin_amdgcn_readlane(pages, (unit - pages_from) * kGroups + i);
        const int token = unit * kUnit + wave * kOwn + 16 * i;
        const int exist = ids[i] < 0 ? 0 : min(len - token, 16);
        const int64_t page = max(ids[i], 0);
        const int at = token & ((1 << p.shift) - 1);
        const auto cs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(p.codes + page * p.c_stride + at * R), 0, exist * R, 0x00020000);
        const auto ss = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.shared + page * p.s_stride + at * S), 0, exist * 2 * S, 0x00020000);
        const auto es = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(p.exponents + page * p.scale_stride + at * kBlocks), 0, exist * kBlocks, 0x00020000);
#pragma unroll
        for (int j = 0; j < 8; ++j) code[i][j] = __builtin_amdgcn_raw_buffer_load_b128(cs, lane * 16 + j * 1024, 0, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j) part[i][j] = __builtin_amdgcn_raw_buffer_load_b128(ss, lane * 16 + j * 1024, 0, 0);
        exponent[i] = __builtin_amdgcn_raw_buffer_load_b32(es, lane * 4, 0, 0);
      }
    };
    // What was loaded, to LDS.  Lanes of 16 codes: 32 are a token's.  A token that
    // only some of the queries see may hold codes of NaN, which a weight of zero would
    // not keep out of the others' products: its latent becomes zero and its shared part
    // NaN, which gives the same to those that see it (their scores are NaN) and
    // nothing to the others.
    auto stage = [&](int unit, bool check) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int line0 = wave * kOwn + 16 * i;
        uint32_t bad = 0;                                  // one bit for each token
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t e0 = __builtin_amdgcn_readlane(exponent[i], 2 * j);
          const uint32_t e1 = __builtin_amdgcn_readlane(exponent[i], 2 * j + 1);
          const float f = __uint_as_float(((h ? e1 : e0) >> (l32 & 24) & 255u) << 23);
          if (check) {
            uint32_t nan = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) nan |= (code[i][j][k] & 0x7f7f7f7fu) + 0x01010101u;
            const uint64_t any = __ballot(nan & 0x80808080u);
            const bool lo = uint32_t(any) != 0, hi = uint32_t(any >> 32) != 0;
            bad |= uint32_t(lo) << (2 * j) | uint32_t(hi) << (2 * j + 1);
            if (h ? hi : lo) code[i][j] = (u32x4)(0u);
          }
          unsigned char* line = tile + (line0 + 2 * j + h) * kLine;
          const int turned = turn(2 * j);                  // of both lines
          const u32x2 a = widen(code[i][j][0], f), b = widen(code[i][j][1], f);
          const u32x2 x = widen(code[i][j][2], f), y = widen(code[i][j][3], f);
          *reinterpret_cast<u32x4*>(line + ((2 * l32) ^ turned) * 16) = (u32x4){a[0], a[1], b[0], b[1]};
          *reinterpret_cast<u32x4*>(line + ((2 * l32 + 1) ^ turned) * 16) = (u32x4){x[0], x[1], y[0], y[1]};
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = 8 * j + (lane >> 3);
          u32x4 x = part[i][j];
          if (check && (bad >> row & 1)) x = (u32x4)(0x7fc07fc0u);
          *reinterpret_cast<u32x4*>(tile + (line0 + row) * kLine + ((2 * R / 16 + (lane & 7)) ^ turn(row)) * 16) = x;
        }
        if (lane == 0) there[line0 / 16] = ids[i];
      }
    };

    look(first);
    load(first);
    bf16x8 q[2 * (R + S) / 32];
    int limit = 0;                                         // tokens that the lane's row sees
    if (scores) {
      const int r = row0 + min(32 * g + l32, rows - 1), i = r / p.H;
      const uint16_t* src = p.q + (int64_t(n) * p.Q + i) * p.q_stride + (r - i * p.H) * (R + S) + 8 * h;
#pragma unroll
      for (int s = 0; s < 36; ++s) q[s] = *reinterpret_cast<const bf16x8*>(src + 16 * s);
      limit = len - p.Q + i + 1;
    }

    for (int unit = first; unit < last; ++unit) {
      const int key0 = unit * kUnit;
      const bool edge = key0 + kUnit > len - p.Q + 1;      // some row does not see some key
      kda::lds_barrier();                                  // the unit before is used up
      stage(unit, edge && p.Q > 1);
      if (unit + 1 < last) load(unit + 1);
      kda::lds_barrier();
      f32x16 s[kKeys];
      if (scores) {
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
          const int line = 32 * (share * kKeys + u);
          s[u] = (f32x16)(0.0f);
#pragma unroll
          for (int k = 0; k < 36; ++k) s[u] = mfma32(rows_of<kLine>(tile, line, l32, h, k), q[k], s[u]);
          const bool here = there[line / 16] >= 0, next = there[line / 16 + 1] >= 0;
          if (edge || !here || !next) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!(e < 8 ? here : next) || key0 + line + 8 * (e >> 2) + 4 * h + (e & 3) >= limit) s[u][e] = -INFINITY;
          }
        }
        float mx = s[0][0];
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[u][e]);
        mx = half_max(mx);
        if (h == 0) top[share][32 * g + l32] = mx;
      }
      kda::lds_barrier();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx = top[0][32 * t + l32];
#pragma unroll
        for (int i = 1; i < kShare; ++i) mx = fmaxf(mx, top[i][32 * t + l32]);
        if (__any((mx - m[t]) * c > kSlack)) {             // the same in all waves
          const float now = fmaxf(m[t], mx);
          const float f = __builtin_amdgcn_exp2f((m[t] - base(now)) * c);
          m[t] = now;
          if (t == g) l *= f;
#pragma unroll
          for (int d = 0; d < 4; ++d) o[t][d] *= f;
        }
      }
      if (scores) {
        float b = base(m[0]);
#pragma unroll
        for (int t = 1; t < NT; ++t) b = t == g ? base(m[t]) : b;
        b *= c;
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              x[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * k + j], c, -b));
              l += x[j];
            }
            *reinterpret_cast<bf16x8*>(weights + (((g * (kUnit / 32) + share * kKeys + u) * 2 + k) * 64 + lane) * 16) =
                pack8(x);
          }
      }
      kda::lds_barrier();
#pragma unroll
      for (int u = 0; u < kUnit / 32; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          bf16x8 w[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t)
            w[t] = *reinterpret_cast<const bf16x8*>(weights + (((t * (kUnit / 32) + u) * 2 + k) * 64 + lane) * 16);
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const bf16x8 a = columns_of<kLine>(tile, 32 * u, k, 128 * wave + 32 * d, lane);
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t][d] = mfma32(a, w[t], o[t][d]);
          }
        }
    }

    // -------- its rows: finished, or a part
    l = half_sum(l);
    if (scores && h == 0) sums[share][32 * g + l32] = l;
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
      const int r = 32 * t + l32;
      float sum = sums[0][r];
#pragma unroll
      for (int i = 1; i < kShare; ++i) sum += sums[i][r];
      if (r >= rows) continue;
      if (whole) {
        const int64_t out = int64_t(n) * p.rows + row0 + r;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int d = 0; d < 4; ++d) store_row32(p.o + out * R + 128 * wave + 32 * d, o[t][d], f, h);
        if (p.lse && wave == 0 && h == 0) p.lse[out] = m[t] * p.scale + __logf(sum);
      } else {
        float* to = p.parts + (int64_t(slot) * p.tile_rows + r) * kPart;
#pragma unroll
        for (int d = 0; d < 4; ++d) store_row32(to + 128 * wave + 32 * d, o[t][d], 1.0f, h);
        if (wave == 0 && h == 0) to[R] = m[t], to[R + 1] = sum;
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

// Rows in as few tiles of at most 128 as they need, of equal size, in steps of 32.
Plan plan_for(int64_t N, int64_t Q, int H) {
  Plan x;
  x.rows = int(Q * H);
  x.row_tiles = (x.rows + 127) / 128;
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
    launch<1>(p, x.pieces, st);
  else if (x.tile_rows == 64)
    launch<2>(p, x.pieces, st);
  else if (x.tile_rows == 96)
    launch<3>(p, x.pieces, st);
  else
    launch<4>(p, x.pieces, st);
  const unsigned joins = unsigned(x.segments * ((tile + join_rows - 1) / join_rows));
  hipLaunchKernelGGL(latent_decode_join_kernel, dim3(joins), dim3(256), 0, st, p);
  return kda::launch_status();
}
