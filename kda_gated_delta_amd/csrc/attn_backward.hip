// Gradients of causal attention (export kda_attn_backward).
//
// With P_ij = exp(scale q_i . k_j - lse_i) for j <= i, delta_i = do_i . o_i:
//     dV = P^T dO,   dS = P o (dO V^T - delta),
//     dQ = scale dS K,   dK = scale dS^T Q,
// dK and dV summed over the query heads that share a key/value head.
//
// attn_stats_kernel writes, per row, lse in powers of two and delta.  In
// attn_grads_kernel workgroups of 128 query rows walk the keys as the forward
// does, for dQ, and workgroups of 128 keys walk the query rows at and after them,
// head after head of the group, for dK and dV, so every sum has one order.  Where
// there are too few (key tile, head) units to fill the device, several workgroups
// share one: each takes an equal part of its query tiles and writes float32 parts
// that attn_sum_kernel adds in order.  P is formed twice (seven products instead
// of five): the alternative, adding dQ with atomics, would make the result depend
// on the order of workgroups.
//
// Every product takes its left operand from LDS (rows, or columns through
// transposing reads) and its right one from registers; P and dS go from the
// accumulator of one product into the operand of the next without leaving the
// lane, rounded once to bfloat16 (in small calls to two terms of it, see
// both_terms).  Sums are float32 throughout.
//
// Matrix unit and power bound the walks, as in the forward.  8192 tokens, 16
// query heads on 4: 14 us of statistics, 950 of gradients (seven products, 1010
// TFLOP/s; dK and dV's 256 registers leave 24 in scratch: with one wave per SIMD
// and none there they are 5% slower), the parts' sum 22 us (151 MB, 6.9 TB/s).  7
// packed sequences of up to 2011 tokens, 12 heads on 4: 16, 240 and 21 us: there
// the longest sequence's first keys are the chain that the others wait for.
#include "attn_device.h"
#include "kda_host.h"

namespace {

using namespace kda::attn;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int BM = 32 * kWaves;
static_assert(BM == kda::kAttnRows);

struct Params {
  const uint16_t *q, *k, *v, *o, *d_out;
  int64_t q_stride, k_stride, v_stride;
  const float* lse;
  const int32_t* cu;
  int N, B, T, HQ, HKV, slots;
  float scale;
  void *dq, *dk, *dv;
  float *lse2, *delta;       // workspace, [B, HQ, T] each
  int parts;                 // workgroups that share a key tile
  float *dk_part, *dv_part;  // workspace, [parts, B, T, HKV, D] each, if parts > 1
  unsigned key_blocks;       // workgroups of dK and dV
  bool keys_first;           // in the launch, before dQ's
};

// ---------------------------------------------------------------- dQ

// What a workgroup of 128 query rows does.  kStats: it writes lse2 and delta, for
// all that follow; otherwise it reads them and makes dQ.
template <typename Out, bool kBoth, bool kStats>
__device__ __forceinline__ void rows_of_dq(const Params& p, unsigned block, unsigned char* lds) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, h = lane >> 5;
  int slot, hkv, hq;
  if (!find_head(block, p.slots, p.HQ, p.HKV, slot, hkv, hq)) return;
  const Rows rows = find_rows<kStats>(p.cu, p.N, p.T, slot, p.slots, BM);   // a sequence's first take longest there
  if (rows.row0 >= rows.len) return;

  const int r0 = rows.row0 + wave * 32;
  const int r = min(r0 + l32, rows.len - 1);
  bf16x8 q[8], u[8];                                       // rows of Q and dO as B operands
  {
    const uint16_t* qs = p.q + (rows.first + r) * p.q_stride + hq * D + 8 * h;
    const uint16_t* us = p.d_out + ((rows.first + r) * p.HQ + hq) * D + 8 * h;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      q[s] = *reinterpret_cast<const bf16x8*>(qs + 16 * s);
      u[s] = *reinterpret_cast<const bf16x8*>(us + 16 * s);
    }
  }
  const int64_t stat = (int64_t(rows.b) * p.HQ + hq) * p.T + rows.start + r;
  float lse2 = kStats ? p.lse[stat] * kLog2e : p.lse2[stat];
  if (kStats && lse2 == -INFINITY) lse2 = INFINITY;        // all scores -inf: weights of zero
  const float c = p.scale * kLog2e;
  f32x16 dq[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) dq[d] = (f32x16)(0.0f);

  const int keys = min(rows.len, rows.row0 + BM);
  const int tiles = (keys + kTile - 1) / kTile;
  TileLoad<kWaves> kload, vload;
  kload.init(wave, lane, p.k_stride);
  vload.init(wave, lane, p.v_stride);
  const uint16_t* kb = p.k + rows.first * p.k_stride + hkv * D;
  const uint16_t* vb = p.v + rows.first * p.v_stride + hkv * D;
  auto issue = [&](int t, int at_buf) {
    unsigned char* buf = lds + at_buf * 2 * kTileBytes;
    const int64_t at = int64_t(t) * kTile;
    kload.issue(kb + at * p.k_stride, p.k_stride, rows.len - int(at), buf, wave);
    vload.issue(vb + at * p.v_stride, p.v_stride, rows.len - int(at), buf + kTileBytes, wave);
  };
  // P^T and (dO V^T)^T (rows = keys) of 32 keys from key0; P is zero after the diagonal.
  auto scores = [&](const unsigned char* kt, int w, int key0, f32x16& s, f32x16& g) {
    s = g = (f32x16)(0.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) s = mfma32(read_rows(kt, 32 * w, l32, h, k), q[k], s);
#pragma unroll
    for (int k = 0; k < 8; ++k) g = mfma32(read_rows(kt + kTileBytes, 32 * w, l32, h, k), u[k], g);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -lse2));
    if (key0 + 31 > r0) {
      const int last = r0 + l32 - key0;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (8 * (e >> 2) + 4 * h + (e & 3) > last) s[e] = g[e] = 0.0f;
    }
  };

  // delta.  The rounding of o to bfloat16 enters it, and with it every score's
  // gradient of the row.  Where o is a mean of many values it is small beside
  // them and so is its rounding; in a sequence's first rows it is not, and would
  // make a third of the error of dQ and dK.  There (two tiles of keys at most)
  // delta is made as sum_j P_ij (dO V^T)_ij, to which it is equal.
  float delta = 0.0f;
  if constexpr (!kStats) {
    issue(0, 0);
    delta = p.delta[stat];
  } else if (rows.row0 == 0) {
    for (int t = 0; t < tiles; ++t) {                      // one buffer: two tiles at most, and more workgroups
      if (t > 0) kda::lds_barrier();
      issue(t, 0);
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
      kda::lds_barrier();
      for (int w = 0; w < 2; ++w) {
        const int key0 = t * kTile + 32 * w;
        if (key0 > r0 + 31) break;
        f32x16 s, g;
        scores(lds, w, key0, s, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) delta = __builtin_fmaf(s[e], g[e], delta);
      }
    }
  } else {
    const uint16_t* os = p.o + ((rows.first + r) * p.HQ + hq) * D + 8 * h;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const bf16x8 x = *reinterpret_cast<const bf16x8*>(os + 16 * s);
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = __builtin_fmaf(float(x[j]), float(u[s][j]), delta);
    }
  }
  if constexpr (kStats) {
    delta = half_sum(delta);
    if (r0 + l32 < rows.len && h == 0) {
      p.lse2[stat] = lse2;
      p.delta[stat] = delta;
    }
    return;
  }

  for (int t = 0; t < tiles; ++t) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    kda::lds_barrier();
    const unsigned char* kt = lds + (t & 1) * 2 * kTileBytes;
    if (t + 1 < tiles) issue(t + 1, (t + 1) & 1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int key0 = t * kTile + 32 * w;
      if (key0 > r0 + 31) continue;
      f32x16 s, g;
      scores(kt, w, key0, s, g);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] *= g[e] - delta;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[8 * k + j];
        const bf16x8 b = pack8(x);
#pragma unroll
        for (int d = 0; d < 4; ++d) dq[d] = mfma32(read_columns(kt, 32 * w, k, 32 * d, lane), b, dq[d]);
        if constexpr (kBoth) {
          const bf16x8 rest = pack8_rest(x, b);
#pragma unroll
          for (int d = 0; d < 4; ++d) dq[d] = mfma32(read_columns(kt, 32 * w, k, 32 * d, lane), rest, dq[d]);
        }
      }
    }
  }
  if (r0 + l32 >= rows.len) return;
  Out* dst = static_cast<Out*>(p.dq) + ((rows.first + r) * p.HQ + hq) * D;
#pragma unroll
  for (int d = 0; d < 4; ++d) store_row32(dst + 32 * d, dq[d], p.scale, h);
}

// Memory bounds it (o and dO once); three workgroups to a compute unit.
__global__ __launch_bounds__(kThreads, 3) void attn_stats_kernel(Params p) {
  __shared__ __align__(1024) unsigned char lds[2 * kTileBytes];
  rows_of_dq<float, false, true>(p, blockIdx.x, lds);
}

// ---------------------------------------------------------------- dK and dV

constexpr int kBuffer = 2 * kTileBytes + 512;              // Q, dO, lse2, delta

template <typename Out, bool kBoth>
__device__ __forceinline__ void keys_of_dkv(const Params& p, unsigned id, unsigned char* lds) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, h = lane >> 5;
  const unsigned kv_heads = p.HKV;
  const int G = p.HQ / p.HKV;
  const int hkv = int(id % kv_heads);
  const int part = int((id / kv_heads) % unsigned(p.parts));
  const Rows rows = find_rows<true>(p.cu, p.N, p.T, int(id / (kv_heads * p.parts)), p.slots, BM);
  if (rows.row0 >= rows.len) return;

  const int k0 = rows.row0 + wave * 32;                    // this wave's first key
  const int key = min(k0 + l32, rows.len - 1);
  bf16x8 kk[8], vv[8];                                     // rows of K and V as B operands
  {
    const uint16_t* ks = p.k + (rows.first + key) * p.k_stride + hkv * D + 8 * h;
    const uint16_t* vs = p.v + (rows.first + key) * p.v_stride + hkv * D + 8 * h;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      kk[s] = *reinterpret_cast<const bf16x8*>(ks + 16 * s);
      vv[s] = *reinterpret_cast<const bf16x8*>(vs + 16 * s);
    }
  }
  const float c = p.scale * kLog2e;
  f32x16 dk[4], dv[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) dk[d] = dv[d] = (f32x16)(0.0f);

  // Query tiles from the one that holds the first key (row0 is a multiple of 64).
  const int t0 = rows.row0 / kTile, per_head = (rows.len + kTile - 1) / kTile - t0;
  const int begin = int(int64_t(per_head) * G * part / p.parts);
  const int end = int(int64_t(per_head) * G * (part + 1) / p.parts);
  TileLoad<kWaves> qload, uload;
  const int64_t u_stride = int64_t(p.HQ) * D;
  qload.init(wave, lane, p.q_stride);
  uload.init(wave, lane, u_stride);
  auto issue = [&](int n, unsigned char* buf) {
    const int g = n / per_head, row = (t0 + n - g * per_head) * kTile, hq = hkv * G + g;
    const int64_t at = rows.first + row;
    qload.issue(p.q + at * p.q_stride + hq * D, p.q_stride, rows.len - row, buf, wave);
    uload.issue(p.d_out + at * u_stride + hq * D, u_stride, rows.len - row, buf + kTileBytes, wave);
    const int64_t stat = (int64_t(rows.b) * p.HQ + hq) * p.T + rows.start + row;
    if (wave == 0) load_floats(p.lse2 + stat, rows.len - row, buf + 2 * kTileBytes, lane);
    if (wave == 1) load_floats(p.delta + stat, rows.len - row, buf + 2 * kTileBytes + 256, lane);
  };
  if (begin < end) issue(begin, lds);

  for (int n = begin; n < end; ++n) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    kda::lds_barrier();
    const unsigned char* qt = lds + ((n - begin) & 1) * kBuffer;
    const unsigned char* ut = qt + kTileBytes;
    const float* stats = reinterpret_cast<const float*>(ut + kTileBytes);
    if (n + 1 < end) issue(n + 1, lds + ((n + 1 - begin) & 1) * kBuffer);
    const int tile0 = (t0 + n % per_head) * kTile;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      const int row0 = tile0 + 32 * w;
      if (row0 + 31 < k0) continue;                        // wholly before this wave's keys
      f32x16 s = (f32x16)(0.0f), g = (f32x16)(0.0f);       // S and dO V^T, rows = query rows
#pragma unroll
      for (int k = 0; k < 8; ++k) s = mfma32(read_rows(qt, 32 * w, l32, h, k), kk[k], s);
#pragma unroll
      for (int k = 0; k < 8; ++k) g = mfma32(read_rows(ut, 32 * w, l32, h, k), vv[k], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(stats + 32 * w + 8 * i + 4 * h);
        const f32x4 b = *reinterpret_cast<const f32x4*>(stats + 64 + 32 * w + 8 * i + 4 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * i + j], c, -a[j]));
          s[4 * i + j] = x;
          g[4 * i + j] = x * (g[4 * i + j] - b[j]);
        }
      }
      if (row0 < k0 + 31 || row0 + 32 > rows.len) {        // pairs before the diagonal, rows behind the end
        const int first = k0 + l32 - row0, behind = rows.len - row0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = 8 * (e >> 2) + 4 * h + (e & 3);
          if (row < first || row >= behind) s[e] = g[e] = 0.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[8 * k + j], y[j] = g[8 * k + j];
        const bf16x8 pb = pack8(x), gb = pack8(y);
#pragma unroll
        for (int d = 0; d < 4; ++d) dv[d] = mfma32(read_columns(ut, 32 * w, k, 32 * d, lane), pb, dv[d]);
#pragma unroll
        for (int d = 0; d < 4; ++d) dk[d] = mfma32(read_columns(qt, 32 * w, k, 32 * d, lane), gb, dk[d]);
        if constexpr (kBoth) {
          const bf16x8 pr = pack8_rest(x, pb), gr = pack8_rest(y, gb);
#pragma unroll
          for (int d = 0; d < 4; ++d) dv[d] = mfma32(read_columns(ut, 32 * w, k, 32 * d, lane), pr, dv[d]);
#pragma unroll
          for (int d = 0; d < 4; ++d) dk[d] = mfma32(read_columns(qt, 32 * w, k, 32 * d, lane), gr, dk[d]);
        }
      }
    }
  }
  if (k0 + l32 >= rows.len) return;
  // (with parts, Out is float and dk, dv are the parts' buffers)
  const int64_t at = (((int64_t(part) * p.B * p.T + rows.first + key) * p.HKV) + hkv) * D;
  Out* dkd = static_cast<Out*>(p.parts > 1 ? p.dk_part : p.dk) + at;
  Out* dvd = static_cast<Out*>(p.parts > 1 ? p.dv_part : p.dv) + at;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    store_row32(dkd + 32 * d, dk[d], p.scale, h);
    store_row32(dvd + 32 * d, dv[d], 1.0f, h);
  }
}

// All gradients in one launch: what is left open behind the longest walks of the
// ones fills up with the others.
template <typename Out, typename Part, bool kBoth>
__global__ __launch_bounds__(kThreads, 2) void attn_grads_kernel(Params p) {
  __shared__ __align__(1024) unsigned char lds[2 * kBuffer];
  const unsigned second = p.keys_first ? p.key_blocks : gridDim.x - p.key_blocks;
  const bool first = blockIdx.x < second;
  const unsigned block = first ? blockIdx.x : blockIdx.x - second;
  if (first == p.keys_first)
    keys_of_dkv<Part, kBoth>(p, block, lds);
  else
    rows_of_dq<Out, kBoth, false>(p, block, lds);
}

// ---------------------------------------------------------------- the parts' sum

// Four elements of dK or dV (blockIdx.y) per thread.
template <typename Out>
__global__ __launch_bounds__(256) void attn_sum_kernel(Params p) {
  const int64_t size = int64_t(p.B) * p.T * p.HKV * D, at = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (p.cu) {                                              // rows outside the sequences are left as they are
    // From the first offset to the last one every row is passed by some sequence;
    // other rows lie in one only where offsets decrease.
    const int row = int(at / (int64_t(p.HKV) * D));
    bool in = row >= p.cu[0] && row < p.cu[p.N];
    if (!__all(in)) {                                      // a wave's 256 elements lie in one row or two
      const int t = __builtin_amdgcn_readfirstlane(row);
      const bool here = in_sequence(p.cu, p.N, t), next = in_sequence(p.cu, p.N, t + 1);
      in = row == t ? here : next;
    }
    if (!in) return;
  }
  if (at >= size) return;
  const float* src = (blockIdx.y ? p.dv_part : p.dk_part) + at;
  f32x4 sum = *reinterpret_cast<const f32x4*>(src);
  for (int i = 1; i < p.parts; ++i) sum += *reinterpret_cast<const f32x4*>(src + i * size);
  store4(static_cast<Out*>(blockIdx.y ? p.dv : p.dk) + at, sum);
}

// Workgroups that share a key tile, and which gradients come first.  A unit is
// one (key tile, key/value head); two workgroups fit a compute unit, and units of
// early keys have many times the work of late ones, so the device wants three or
// four per compute unit.  With sequences of different lengths the first keys of
// the longest make the longest walk, and come first; with one length both kinds
// have many long walks, dQ's of a length that no parts shorten, and come first.
// Training pass in us, in two launches / dK and dV first, 3 per unit / dQ first, 4:
//   8192 tokens, 16 heads on 4    1300  1325  1294      7 of up to 2011, 12 on 4   360  350  361
//   4096 tokens, 16 on 2           416   408   395      8 of up to 2000, 16 on 2   423  410  429
//   1500 tokens, 8 on 1            115    94    89      3 of up to 1000, 64 on 8   289  268  293
//   700 tokens, 8 on 2              68    55    55      20 of up to 500, 12 on 4   143  128  142
// A part should still walk two query tiles: with one the parts' sum costs more
// than the walk (2000 tokens, 4 heads: 127 us with two, 148 with one, 150 with
// eight).
bool one_length(int N, bool packed) { return !packed || N == 1; }
int parts_for(int64_t slots, int T, int N, bool packed, int HQ, int HKV) {
  const int64_t units = slots * HKV, cus = kda::device_cus(), want = (one_length(N, packed) ? 4 : 3) * cus;
  if (units >= want || slots > kda::kMostBlocks) return 1;   // (of more slots units may have overflowed)
  const int64_t len = kda::attn_typical(T, N, packed);
  const int64_t walk = (len / kTile / 2 + 1) * (HQ / HKV);
  const int64_t most = walk / 2 < 1 ? 1 : (walk / 2 > 16 ? 16 : walk / 2);
  const int64_t parts = (want + units - 1) / units;
  return int(parts < most ? parts : most);
}

// Whether a launch takes the workgroups.  (The parts' sum, of few units, has fewer.)
bool fits(int64_t slots, int parts, int HQ, int HKV) {
  return slots <= kda::kMostBlocks && head_blocks(slots, HQ, HKV) + slots * HKV * parts <= kda::kMostBlocks;
}

// Whether weights and score gradients are carried as two bfloat16 terms.  One
// rounding of each adds as much error to a gradient as rounding the gradient
// itself, and where there are few of them, by chance more: 10 sequences of 3
// tokens, 2 heads: dQ and dK off by 0.0028 of their norm with one term, 0.0017
// with two, as rounded exact ones are.  There the launch's time is latency, and a
// second product with what the rounding left costs little (28.3 us there with
// either, 31.2 for 60 tokens of 8 heads, 36.7 for 32.9 for 128 tokens of 2).  With
// more of them chance is averaged out, and the products are what bounds the walk.
bool both_terms(int64_t rows, int64_t len) { return rows * len <= 1 << 15; }

template <typename Out, bool kBoth>
void launch_grads(const Params& p, unsigned blocks, hipStream_t stream) {
  const dim3 grid(p.key_blocks + blocks);
  if (p.parts == 1) {
    hipLaunchKernelGGL((attn_grads_kernel<Out, Out, kBoth>), grid, dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((attn_grads_kernel<Out, float, kBoth>), grid, dim3(kThreads), 0, stream, p);
    const int64_t quads = int64_t(p.B) * p.T * p.HKV * (D / 4);
    hipLaunchKernelGGL(attn_sum_kernel<Out>, dim3(unsigned((quads + 255) / 256), 2), dim3(256), 0, stream, p);
  }
}

template <typename Out>
int launch(const Params& p, hipStream_t stream) {
  const unsigned blocks = unsigned(head_blocks(p.slots, p.HQ, p.HKV));
  hipLaunchKernelGGL(attn_stats_kernel, dim3(blocks), dim3(kThreads), 0, stream, p);
  if (both_terms(int64_t(p.B) * p.T * p.HQ, kda::attn_typical(p.T, p.N, p.cu != nullptr)))
    launch_grads<Out, true>(p, blocks, stream);
  else
    launch_grads<Out, false>(p, blocks, stream);
  return kda::launch_status();
}

}  // namespace

extern "C" size_t kda_attn_backward_workspace_size(int32_t B, int32_t T, int32_t HQ, int32_t HKV, int32_t Dh,
                                                   int32_t num_seqs) {
  if (B < 1 || T < 0 || num_seqs < 0 || (num_seqs && B != 1) || kda::attn_heads(HQ, HKV, Dh) != KDA_OK) return 0;
  if (T == 0) return 0;
  const int64_t slots = kda::attn_slots(B, T, num_seqs);
  const int parts = parts_for(slots, T, num_seqs ? num_seqs : B, num_seqs > 0, HQ, HKV);
  if (!fits(slots, parts, HQ, HKV)) return 0;
  const size_t sums = parts > 1 ? size_t(parts) * 2 * B * T * HKV * D : 0;
  return (2 * kda::attn_stat_floats(B, T, HQ) + sums) * sizeof(float);
}

extern "C" int kda_attn_backward(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, const void* o, const float* lse, const void* d_out,
                                 const int32_t* cu_seqlens, int32_t num_seqs, int32_t B, int32_t T, int32_t HQ,
                                 int32_t HKV, int32_t Dh, float scale, void* dq, void* dk, void* dv,
                                 int32_t grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const int e = kda::attn_check(cu_seqlens, num_seqs, B, T, HQ, HKV, Dh, scale, q_stride, k_stride, v_stride);
  if (e != KDA_OK) return e;
  if (grad_dtype != KDA_GRAD_FLOAT32 && grad_dtype != KDA_GRAD_INPUT_DTYPE) return KDA_ERR_UNSUPPORTED;
  if (T == 0) return KDA_OK;
  if (!q || !k || !v || !o || !lse || !d_out || !dq || !dk || !dv || !workspace) return KDA_ERR_NULL;
  for (const void* x : {q, k, v, o, static_cast<const void*>(lse), d_out, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv),
                        static_cast<const void*>(workspace)})
    if (!kda::aligned16(x)) return KDA_ERR_ALIGN;
  const int seqs = cu_seqlens ? num_seqs : 0, N = cu_seqlens ? num_seqs : B;
  const int64_t slots = kda::attn_slots(B, T, seqs);
  const int parts = parts_for(slots, T, N, seqs > 0, HQ, HKV);
  if (!fits(slots, parts, HQ, HKV)) return KDA_ERR_SHAPE;
  if (workspace_bytes < kda_attn_backward_workspace_size(B, T, HQ, HKV, Dh, seqs)) return KDA_ERR_WORKSPACE;
  float* ws = static_cast<float*>(workspace);
  const size_t stats = kda::attn_stat_floats(B, T, HQ), grads = size_t(parts) * B * T * HKV * D;
  const Params p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                 static_cast<const uint16_t*>(o), static_cast<const uint16_t*>(d_out), q_stride, k_stride, v_stride,
                 lse, cu_seqlens, N, B, T, HQ, HKV, int(slots), scale, dq, dk, dv,
                 ws, ws + stats, parts, ws + 2 * stats, ws + 2 * stats + grads,
                 unsigned(slots * HKV * parts), !one_length(N, seqs > 0)};
  return grad_dtype == KDA_GRAD_FLOAT32 ? launch<float>(p, kda::as_stream(stream))
                                        : launch<uint16_t>(p, kda::as_stream(stream));
}
