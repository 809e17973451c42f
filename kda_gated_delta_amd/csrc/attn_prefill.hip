// Causal attention over whole prompts (export kda_attn_prefill).
//
// For every query head h and token i of a sequence, with key/value head
// h / (HQ / HKV), z_ij = scale q_i . k_j for j <= i:
//     lse_i = log sum_j exp(z_ij),   o_i = sum_j exp(z_ij - lse_i) v_j.
//
// One pass over the keys with a running maximum and sum.  A wave owns 32
// query rows and keeps their output transposed, O^T [128][32], in its
// registers.  Per tile of 64 keys (K and V in LDS, two buffers, loaded
// straight from memory while the previous tile is used):
//     S^T = K Q^T          (rows = keys, so a query's scores lie in one lane pair)
//     P^T = exp2(c S^T - c m)
//     O^T += V^T P^T       (V^T by transposing LDS reads)
// The accumulator of S^T holds, in each lane, exactly the contraction indices
// that the next product wants of its B operand (in the order read_columns
// takes V's rows), so P never leaves its registers: no exchange, no LDS.
// P is rounded to bfloat16 for its product; maximum, sum and output are float32.
//
// The matrix unit and the chip's power bound it.  8192 tokens, 32 query heads on
// 8: 512 us, 1074 TFLOP/s, where a large library product reaches 1170 on the same
// card; matrix unit 55% busy, vector unit about 50%, LDS 10% and without bank
// conflicts, at 1.8 GHz (with inputs of zeros the clock stays up and it takes
// 20 to 25% less).  16 packed sequences of up to 4096 tokens, 16 heads on 2: 410
// us.  129 tokens, 8 heads: 7 us, the latency of one walk.  64 query rows per
// wave (half the LDS reads, one wave per SIMD) reach 798 TFLOP/s; the scores of
// the next tile formed beside the weights of this one were 3% slower.
#include "attn_device.h"
#include "kda_host.h"

#include <type_traits>

namespace {

using namespace kda::attn;

constexpr int kWaves = 4;
constexpr int BM = 32 * kWaves;            // query rows of a workgroup
static_assert(BM == kda::kAttnRows);

struct Params {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;    // elements from token to token
  const int32_t* cu;
  int N, T, HQ, HKV, slots;
  float scale;
  uint16_t* o;
  float* lse;
};

// kSplit = 2: a second set of four waves takes every other key tile of the same
// rows, and the two halves of a row are joined at the end (attn_split says when):
// the walk over the keys is a chain, and two waves per SIMD halve it.
template <int kSplit>
__global__ __launch_bounds__(64 * kWaves * kSplit, 2) void attn_prefill_kernel(Params p) {
  constexpr int kHalf = 4 * kTileBytes;    // two buffers of K and V
  __shared__ __align__(1024) unsigned char all[kSplit * kHalf];
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int half = kSplit == 1 ? 0 : id / kWaves, wave = id - half * kWaves;
  unsigned char* lds = all + half * kHalf;
  const int l32 = lane & 31, h = lane >> 5;

  int slot, hkv, hq;
  if (!find_head(blockIdx.x, p.slots, p.HQ, p.HKV, slot, hkv, hq)) return;
  const Rows rows = find_rows<false>(p.cu, p.N, p.T, slot, p.slots, BM);
  if (rows.row0 >= rows.len) return;

  const int r0 = rows.row0 + wave * 32;                   // this wave's first row
  const int r = min(r0 + l32, rows.len - 1);              // this lane's; rows behind the end repeat the last one
  bf16x8 q[8];                                            // as B operands
  const uint16_t* src = p.q + (rows.first + r) * p.q_stride + hq * D + 8 * h;
#pragma unroll
  for (int s = 0; s < 8; ++s) q[s] = *reinterpret_cast<const bf16x8*>(src + 16 * s);
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = (f32x16)(0.0f);
  float m = -INFINITY, l = 0.0f;                          // l: this lane's keys only, until the end
  const float c = p.scale * kLog2e;

  const int keys = min(rows.len, rows.row0 + BM);         // keys that the last row of the tile sees
  const int tiles = (keys + kTile - 1) / kTile;
  TileLoad<kWaves> kload, vload;
  kload.init(wave, lane, p.k_stride);
  vload.init(wave, lane, p.v_stride);
  const uint16_t* kb = p.k + rows.first * p.k_stride + hkv * D;
  const uint16_t* vb = p.v + rows.first * p.v_stride + hkv * D;
  auto issue = [&](int t, int buf) {
    unsigned char* to = lds + buf * 2 * kTileBytes;
    const int64_t at = int64_t(t) * kTile;
    kload.issue(kb + at * p.k_stride, p.k_stride, rows.len - int(at), to, wave);
    vload.issue(vb + at * p.v_stride, p.v_stride, rows.len - int(at), to + kTileBytes, wave);
  };
  int late = -1;                                          // first key of a tile left for the end
  auto tile = [&](const unsigned char* kt, const unsigned char* vt, int key0, auto diagonal) {
    // where the diagonal crosses the first half of a tile the second is not seen
    const int halves_seen = decltype(diagonal)::value && r0 == key0 ? 1 : 2;
    f32x16 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = (f32x16)(0.0f);
      if (u >= halves_seen) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) s[u] = mfma32(read_rows(kt, 32 * u, l32, h, k), q[k], s[u]);
    }
    if constexpr (decltype(diagonal)::value) {
      const int last = r0 + l32 - key0;                   // the last key of the tile that the row sees
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * u + 8 * (e >> 2) + 4 * h + (e & 3) > last) s[u][e] = -INFINITY;
      if (any_not_finite(vt, halves_seen, lane)) late = key0;
    }
    float mx = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[u][e]);
    mx = half_max(mx);
    if (__any((mx - m) * c > kSlack)) {
      const float now = fmaxf(m, mx);
      const float f = __builtin_amdgcn_exp2f((m - base(now)) * c);
      m = now;
      l *= f;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= f;
    }
    const float b = base(m) * c;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[u][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], c, -b));
        sum += s[u][e];
      }
    l += sum;
    if (decltype(diagonal)::value && late >= 0) return;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u >= halves_seen) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[u][8 * k + j];
        const bf16x8 w = pack8(x);
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = mfma32(read_columns(vt, 32 * u, k, 32 * d, lane), w, o[d]);
      }
    }
  };

  // The i-th tile of this half is there, the next on its way.  All waves pass as
  // often.
  const int rounds = (tiles + kSplit - 1) / kSplit;
  auto arrive = [&](int i) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    kda::lds_barrier();
    if ((i + 1) * kSplit + half < tiles) issue((i + 1) * kSplit + half, (i + 1) & 1);
  };
  auto take = [&](int i, auto diagonal) {
    const unsigned char* kt = lds + (i & 1) * 2 * kTileBytes;
    tile(kt, kt + kTileBytes, (i * kSplit + half) * kTile, diagonal);
  };
  if (half < tiles) issue(half, 0);
  // Tiles before the diagonal, the one that it crosses (if it is this half's),
  // and those that other waves of the workgroup still take.
  const int whole = min(r0 / kTile, tiles);               // tiles that all rows of the wave see
  int i = 0;
  for (; i * kSplit + half < whole; ++i) {
    arrive(i);
    take(i, std::false_type{});
  }
  if (i < rounds) {
    arrive(i);
    if (i * kSplit + half == r0 / kTile) take(i, std::true_type{});
    ++i;
  }
  for (; i < rounds; ++i) arrive(i);

  // A weight of zero does not keep an infinity or NaN of a later row of V out of a
  // product.  If the tile that the diagonal crosses, a wave's last, holds one, its
  // keys are added here one by one, from memory, each to the rows that see it.
  if (late >= 0) {
#pragma unroll 1
    for (int key = late; key < min(r0 + 32, rows.len); ++key) {
      const uint16_t* kr = kb + key * p.k_stride + 8 * h;
      const uint16_t* vr = vb + key * p.v_stride + 4 * h;
      float x = 0.0f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const bf16x8 y = *reinterpret_cast<const bf16x8*>(kr + 16 * s);
#pragma unroll
        for (int j = 0; j < 8; ++j) x = __builtin_fmaf(float(q[s][j]), float(y[j]), x);
      }
      x = __builtin_amdgcn_exp2f(__builtin_fmaf(half_sum(x), c, -base(m) * c));
      if (key > r0 + l32) continue;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u32x2 y = *reinterpret_cast<const u32x2*>(vr + 32 * d + 8 * e);
          o[d][4 * e] = __builtin_fmaf(x, kda::bf16lo(y[0]), o[d][4 * e]);
          o[d][4 * e + 1] = __builtin_fmaf(x, kda::bf16hi(y[0]), o[d][4 * e + 1]);
          o[d][4 * e + 2] = __builtin_fmaf(x, kda::bf16lo(y[1]), o[d][4 * e + 2]);
          o[d][4 * e + 3] = __builtin_fmaf(x, kda::bf16hi(y[1]), o[d][4 * e + 3]);
        }
    }
  }

  float total = half_sum(l);
  if constexpr (kSplit == 2) {
    // The second half's output, maximum and sum, 66 floats per lane, through LDS.
    // Its rows may have seen no key there (maximum -inf, output and sum 0).
    kda::lds_barrier();
    float* place = reinterpret_cast<float*>(all) + wave * 66 * 64 + lane;
    if (half == 1) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) place[(16 * d + e) * 64] = o[d][e];
      place[64 * 64] = m;
      place[65 * 64] = total;
    }
    kda::lds_barrier();
    if (half == 1) return;
    const float m2 = place[64 * 64], top = fmaxf(m, m2);
    const float f1 = __builtin_amdgcn_exp2f((m - base(top)) * c), f2 = __builtin_amdgcn_exp2f((m2 - base(top)) * c);
    total = total * f1 + place[65 * 64] * f2;
    m = top;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = o[d][e] * f1 + place[(16 * d + e) * 64] * f2;
  }
  if (r0 + l32 >= rows.len) return;                       // both lanes of a pair alike
  const float f = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* dst = p.o + ((rows.first + r) * p.HQ + hq) * D;
#pragma unroll
  for (int d = 0; d < 4; ++d) store_row32(dst + 32 * d, o[d], f, h);
  if (p.lse && h == 0)
    p.lse[(int64_t(rows.b) * p.HQ + hq) * p.T + rows.start + r] = m * p.scale + __logf(total);
}

}  // namespace

extern "C" int kda_attn_prefill(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, const int32_t* cu_seqlens, int32_t num_seqs, int32_t B, int32_t T,
                                int32_t HQ, int32_t HKV, int32_t Dh, float scale, void* o, float* lse,
                                void* stream) {
  const int e = kda::attn_check(cu_seqlens, num_seqs, B, T, HQ, HKV, Dh, scale, q_stride, k_stride, v_stride);
  if (e != KDA_OK) return e;
  if (T == 0) return KDA_OK;
  if (!q || !k || !v || !o) return KDA_ERR_NULL;
  for (const void* x : {q, k, v, static_cast<const void*>(o), static_cast<const void*>(lse)})
    if (!kda::aligned16(x)) return KDA_ERR_ALIGN;            // no lse: a null pointer passes
  const int64_t slots = kda::attn_slots(B, T, cu_seqlens ? num_seqs : 0);
  if (slots > kda::kMostBlocks) return KDA_ERR_SHAPE;
  const int64_t blocks = head_blocks(slots, HQ, HKV);
  if (blocks > kda::kMostBlocks) return KDA_ERR_SHAPE;
  const Params p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                 q_stride, k_stride, v_stride, cu_seqlens, cu_seqlens ? num_seqs : B, T, HQ, HKV, int(slots), scale,
                 static_cast<uint16_t*>(o), lse};
  if (kda::attn_split(blocks, T, p.N, cu_seqlens != nullptr))
    hipLaunchKernelGGL(attn_prefill_kernel<2>, dim3(unsigned(blocks)), dim3(128 * kWaves), 0,
                       kda::as_stream(stream), p);
  else
    hipLaunchKernelGGL(attn_prefill_kernel<1>, dim3(unsigned(blocks)), dim3(64 * kWaves), 0,
                       kda::as_stream(stream), p);
  return kda::launch_status();
}
