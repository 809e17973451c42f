// Causal attention in latent attention's expanded form (export
// kda_latent_prefill): every head has a key and a value of 128 of its own, and a
// key part of 64 is shared by all.
//
// For every head and query i of a sequence with Tq queries and Tk keys, over the
// keys j <= i + Tk - Tq (the last query stands at the last key):
//     z_ij = scale (qn_i . k_j + qs_i . s_j),  lse_i = log sum_j exp(z_ij),
//     o_i = sum_j exp(z_ij - lse_i) v_j.
//
// The walk is attn_prefill.hip's: a wave owns 32 query rows, S^T = [K s] Q^T, the
// weights stay in the registers that the scores came in, O^T += V^T P^T.  A tile of
// 64 keys is three pieces in LDS: K and V of the head (lines of 256 bytes) and the
// shared part (lines of 128), 40 KB; two buffers, and so two workgroups per compute
// unit.  The shared part is read for every head, from the caches: it is a fifth of
// a tile and never stored 32-fold as a concatenated key would be.
//
// What bounds it: the products, at the power limit (8192 tokens x 32 heads 626 to 669 us by
// the card, 1030 to 1090 TFLOP/s, the matrix units 57% busy at 1.75 to 1.8 GHz; a large
// matrix product reaches 1224 on the faster cards), and with few rows a walk's latency (129
// tokens x 8 heads: 8.4 us).  Parts of prompts over long caches end unevenly (6 of up to 1500
// tokens over up to 6000: 765 to 840 TFLOP/s; 10% of the tiles' pairs are masked, 9% of the
// time waits for the last).
#include "kda_host.h"
#include "latent_device.h"

#include <type_traits>

namespace {

using namespace kda::latent;

constexpr int kWaves = 4;
constexpr int BM = 32 * kWaves;                      // query rows of a workgroup
static_assert(BM == kda::kAttnRows);
constexpr int kBuffer = 2 * kTileBytes + kThinBytes; // K, V, the shared part

struct Params {
  const uint16_t *q, *k, *v, *s;
  int64_t q_stride, k_stride, v_stride, s_stride;    // elements from token to token
  int64_t k_head, v_head;                            // and from head to head
  const int32_t *cu, *cu_kv;
  int N, T, K, H, slots;
  float scale;
  uint16_t* o;
  float* lse;
};

// A tile that all rows of a wave see, one that the diagonal crosses, and such a one of
// whose values some are not finite.
constexpr int kWhole = 0, kDiagonal = 1, kPartly = 2;

// Eight bfloat16 values, zero for those that are not finite.
__device__ __forceinline__ bf16x8 finite_or_zero(bf16x8 x) {
  u32x4 y = __builtin_bit_cast(u32x4, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (y[i] & 0x7f80u) == 0x7f80u ? 0u : y[i] & 0xffffu;
    y[i] = lo | ((y[i] & 0x7f800000u) == 0x7f800000u ? 0u : y[i] & 0xffff0000u);
  }
  return as_bf16x8(y);
}

// kSplit = 2: a second set of four waves takes every other key tile of the same
// rows, and the two halves of a row are joined at the end (attn_split says when).
template <int kSplit>
__global__ __launch_bounds__(64 * kWaves * kSplit, 2) void latent_prefill_kernel(Params p) {
  __shared__ __align__(1024) unsigned char all[kSplit * 2 * kBuffer];
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int half = kSplit == 1 ? 0 : id / kWaves, wave = id - half * kWaves;
  unsigned char* lds = all + half * 2 * kBuffer;
  const int l32 = lane & 31, h = lane >> 5;

  const int slot = int(blockIdx.x / unsigned(p.H)), head = int(blockIdx.x % unsigned(p.H));
  const Rows rows = find_rows<false>(p.cu, p.N, p.T, slot, p.slots, BM);
  if (rows.row0 >= rows.len) return;
  const Keys keys = find_keys(p.cu_kv, p.K, rows.n, rows.len);

  const int r0 = rows.row0 + wave * 32;                   // this wave's first row
  const int r = min(r0 + l32, rows.len - 1);              // this lane's; rows behind the end repeat the last one
  bf16x8 q[12];                                           // as B operands
  const uint16_t* src = p.q + (rows.first + r) * p.q_stride + head * DQ + 8 * h;
#pragma unroll
  for (int s = 0; s < 12; ++s) q[s] = *reinterpret_cast<const bf16x8*>(src + 16 * s);
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = (f32x16)(0.0f);
  float m = -INFINITY, l = 0.0f;                          // l: this lane's keys only, until the end
  const float c = p.scale * kLog2e;

  const int see0 = r0 + keys.shift;                       // the last key that the wave's first row sees (below 0: none)
  const int seen = min(rows.row0 + BM, rows.len) + keys.shift;   // keys that the tile's last row sees
  const int tiles = max(seen + kTile - 1, 0) / kTile;
  TileLoad<kWaves> kload, vload;
  ThinLoad<kWaves> sload;
  kload.init(wave, lane, p.k_stride);
  vload.init(wave, lane, p.v_stride);
  sload.init(wave, lane, p.s_stride);
  const uint16_t* kb = p.k + keys.first * p.k_stride + head * p.k_head;
  const uint16_t* vb = p.v + keys.first * p.v_stride + head * p.v_head;
  const uint16_t* sb = p.s + keys.first * p.s_stride;
  auto issue = [&](int t, int buf) {
    unsigned char* to = lds + buf * kBuffer;
    const int64_t at = int64_t(t) * kTile;
    kload.issue(kb + at * p.k_stride, p.k_stride, keys.len - int(at), to, wave);
    sload.issue(sb + at * p.s_stride, p.s_stride, keys.len - int(at), to + 2 * kTileBytes, wave);
    vload.issue(vb + at * p.v_stride, p.v_stride, keys.len - int(at), to + kTileBytes, wave);
  };
  int late = -1;                                          // first key of a tile with values left for the end
  // False, and nothing done, if the diagonal crosses the tile and some of its values are
  // not finite.
  auto tile = [&](const unsigned char* kt, int key0, auto kind_of) {
    constexpr int kind = decltype(kind_of)::value;
    // (made anew, what follows from the lane is not kept, and with the rest in scratch;
    // where it fits, keeping it saves a short prompt 0.5 of 8.9 us)
    constexpr bool anew = kind == kPartly || (kind == kDiagonal && kSplit == 2);
    const int lane = anew ? lane_now() : int(threadIdx.x & 63), l32 = lane & 31, h = lane >> 5;
    const unsigned char *vt = kt + kTileBytes, *st = vt + kTileBytes;
    // where no row of the wave sees the tile's second half it is left out
    const int halves_seen = kind != kWhole && see0 + 31 < key0 + 32 ? 1 : 2;
    f32x16 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = (f32x16)(0.0f);
      if (u >= halves_seen) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) s[u] = mfma32(read_rows(kt, 32 * u, l32, h, k), q[k], s[u]);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[u] = mfma32(rows_of<2 * S>(st, 32 * u, l32, h, k), q[8 + k], s[u]);
    }
    if constexpr (kind != kWhole) {
      const int last = see0 + l32 - key0;                 // the last key of the tile that the row sees
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * u + 8 * (e >> 2) + 4 * h + (e & 3) > last) s[u][e] = -INFINITY;
      if (kind == kDiagonal && any_not_finite(vt, halves_seen, lane)) return false;
    }
    float mx = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[u][e]);
    mx = half_max(mx);
    if (__any((mx - m) * c > kSlack)) {
      // (row by row: what a row sees does not change how another one is rounded)
      const float now = (mx - m) * c > kSlack ? mx : m;
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
        for (int d = 0; d < 4; ++d) {
          const bf16x8 v = columns_of<256>(vt, 32 * u, k, 32 * d, lane);
          o[d] = mfma32(kind == kPartly ? finite_or_zero(v) : v, w, o[d]);
          if (kind == kPartly) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    return true;
  };

  // The i-th tile of this half is there, the next on its way.  All waves pass as
  // often.
  const int rounds = (tiles + kSplit - 1) / kSplit;
  auto arrive = [&](int i) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    kda::lds_barrier();
    if ((i + 1) * kSplit + half < tiles) issue((i + 1) * kSplit + half, (i + 1) & 1);
  };
  auto take = [&](int i, auto kind) { return tile(lds + (i & 1) * kBuffer, (i * kSplit + half) * kTile, kind); };
  if (half < tiles) issue(half, 0);
  // Tiles that all rows of the wave see, those that the diagonal crosses (two at
  // most, since 32 rows end within 32 keys; none perhaps, or none of this half's),
  // and those that other waves of the workgroup still take.
  const int whole = min(max(see0 + 1, 0) / kTile, tiles);
  const int some = see0 + 31 < 0 ? 0 : min((see0 + 31) / kTile + 1, tiles);
  int i = 0;
  for (; i * kSplit + half < whole; ++i) {
    arrive(i);
    take(i, std::integral_constant<int, kWhole>{});
  }
  bool finite = true;
#pragma unroll 1
  while (finite && i * kSplit + half < some) {
    arrive(i);
    finite = take(i, std::integral_constant<int, kDiagonal>{});
    i += finite;
  }
  // A weight of zero does not keep an infinity or NaN of a later row of V out of a
  // product.  From the first tile on that the diagonal crosses and that holds one, they
  // are left out of the products.
  if (!finite) {
    late = (i * kSplit + half) * kTile;
    bool there = true;
#pragma unroll 1
    for (; i * kSplit + half < some; ++i) {
      if (!there) arrive(i);
      there = false;
      take(i, std::integral_constant<int, kPartly>{});
    }
  }
  for (; i < rounds; ++i) arrive(i);

  // Those values are added here, from memory, each to the rows that see it: nothing that
  // is finite is rounded otherwise than without them.
  const int now = lane_now(), now32 = now & 31, now_h = now >> 5;
  if (late >= 0) {
    const int end = min(see0 + 32, keys.len);
#pragma unroll 1
    for (int key = late; key < (kSplit == 1 ? end : min(end, late + kTile)); ++key) {
      const uint16_t* kr = kb + key * p.k_stride + 8 * now_h;
      const uint16_t* sr = sb + key * p.s_stride + 8 * now_h;
      const uint16_t* vr = vb + key * p.v_stride + 4 * now_h;
      float x = 0.0f;
#pragma unroll
      for (int s = 0; s < 12; ++s) {
        const bf16x8 y = *reinterpret_cast<const bf16x8*>(s < 8 ? kr + 16 * s : sr + 16 * (s - 8));
#pragma unroll
        for (int j = 0; j < 8; ++j) x = __builtin_fmaf(float(q[s][j]), float(y[j]), x);
      }
      x = __builtin_amdgcn_exp2f(__builtin_fmaf(half_sum(x), c, -base(m) * c));
      if (key > see0 + now32) continue;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u32x2 y = *reinterpret_cast<const u32x2*>(vr + 32 * d + 8 * e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = j & 1 ? kda::bf16hi(y[j >> 1]) : kda::bf16lo(y[j >> 1]), sum = o[d][4 * e + j];
            o[d][4 * e + j] = __builtin_fabsf(f) < INFINITY ? sum : __builtin_fmaf(x, f, sum);
          }
        }
    }
  }

  float total = half_sum(l);
  if constexpr (kSplit == 2) {
    // The second half's output, maximum and sum, 66 floats per lane, through LDS.
    // Its rows may have seen no key there (maximum -inf, output and sum 0).
    kda::lds_barrier();
    float* place = reinterpret_cast<float*>(all) + wave * 66 * 64 + now;
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
  const int row = r0 + now32;
  if (row >= rows.len) return;                            // both lanes of a pair alike
  const float f = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* dst = p.o + ((rows.first + row) * p.H + head) * D;
#pragma unroll
  for (int d = 0; d < 4; ++d) store_row32(dst + 32 * d, o[d], f, now_h);
  if (p.lse && now_h == 0)
    p.lse[(int64_t(rows.b) * p.H + head) * p.T + rows.start + row] = m * p.scale + __logf(total);
}

}  // namespace

extern "C" int kda_latent_prefill(const void* q, const void* k, const void* k_shared, const void* v, int64_t q_stride,
                                  int64_t k_stride, int64_t k_head, int64_t s_stride, int64_t v_stride,
                                  int64_t v_head, const int32_t* cu_seqlens, const int32_t* cu_seqlens_kv,
                                  int32_t num_seqs, int32_t B, int32_t T, int32_t T_kv, int32_t H, float scale, void* o,
                                  float* lse, void* stream) {
  const kda::LatentLayout x{q_stride, k_stride, k_head, s_stride, v_stride, v_head};
  const int e = kda::latent_check(x, cu_seqlens, cu_seqlens_kv, num_seqs, B, T, T_kv, H, scale);
  if (e != KDA_OK) return e;
  if (T == 0) return KDA_OK;
  if (!q || !o || (T_kv && (!k || !k_shared || !v))) return KDA_ERR_NULL;
  for (const void* y : {q, k, k_shared, v, static_cast<const void*>(o), static_cast<const void*>(lse)})
    if (!kda::aligned16(y)) return KDA_ERR_ALIGN;            // no lse: a null pointer passes
  const int64_t slots = kda::attn_slots(B, T, cu_seqlens ? num_seqs : 0);
  const int64_t blocks = slots * H;
  if (slots > kda::kMostBlocks || blocks > kda::kMostBlocks) return KDA_ERR_SHAPE;
  const Params p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                 static_cast<const uint16_t*>(k_shared), q_stride, k_stride, v_stride, s_stride, k_head, v_head,
                 cu_seqlens, cu_seqlens_kv, cu_seqlens ? num_seqs : B, T, T_kv, H, int(slots), scale,
                 static_cast<uint16_t*>(o), lse};
  if (kda::attn_split(blocks, T_kv, p.N, cu_seqlens != nullptr))
    hipLaunchKernelGGL(latent_prefill_kernel<2>, dim3(unsigned(blocks)), dim3(128 * kWaves), 0,
                       kda::as_stream(stream), p);
  else
    hipLaunchKernelGGL(latent_prefill_kernel<1>, dim3(unsigned(blocks)), dim3(64 * kWaves), 0,
                       kda::as_stream(stream), p);
  return kda::launch_status();
}
