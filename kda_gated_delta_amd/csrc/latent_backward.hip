// Gradients of latent attention's expanded form (export kda_latent_backward).
//
// With k_j = [kn_j s_j] (192 wide), P_ij = exp(scale q_i . k_j - lse_i) for
// j <= i + Tk - Tq, delta_i = do_i . o_i, per head:
//     dV = P^T dO,   dS = P o (dO V^T - delta),
//     dQ = scale dS K,   [dKn dS_shared] = scale dS^T Q,
// the shared part's summed over all heads.
//
// Workgroups of 128 query rows walk the keys for dQ (and first make lse in powers of
// two and delta), then workgroups of 128 keys walk the query rows for dK and dV.  Every
// head has keys of its own, so a walk belongs to one head; only the shared part's
// gradient crosses heads.  Its terms are written in float32 per head and added in order
// by latent_sum_kernel, as the parts of a key tile that several workgroups share are.
//
// Weights and score gradients are made in both walks: 1152 products of a pair's numbers
// where the formulas have 832.  One walk for all would add dQ up across workgroups, in
// float32 through memory and in order (attn_backward.hip has no such sums either).
// What bounds the walks are the products, at the power limit (8192 tokens x 16 heads:
// dK and dV 609 to 646 us, 0.69 TFLOP, 1070 TFLOP/s; dQ 476 to 512 us, 0.55 TFLOP, 1120;
// sum 8; a large matrix product reaches 1224 on this card).  lse2 and delta in a launch of
// their own cost 7 to 13 us (6 samples of up to 500 tokens x 16 heads 89 to 82).  With all
// of a walk in one wave and both walks in one launch of one workgroup to a compute
// unit, dK, dV and dQ took 1422 us: nothing ran while a SIMD's one wave made weights.
#include "kda_host.h"
#include "latent_device.h"

namespace {

using namespace kda::latent;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int BM = 32 * kWaves;
static_assert(BM == kda::kAttnRows);

struct Params {
  const uint16_t *q, *k, *v, *s, *o, *d_out;
  int64_t q_stride, k_stride, v_stride, s_stride, k_head, v_head;
  const float* lse;
  const int32_t *cu, *cu_kv;
  int N, B, T, K, H, slots, key_slots;
  float scale;
  void *dq, *dkv, *ds;       // dkv: [B, K, H, 256], a head's dK and dV
  float *lse2, *delta;       // workspace, [B, H, T] each
  int parts;                 // workgroups that share a key tile
  float* dkv_part;           // workspace, [parts, B, K, H, 256], if parts > 1
  float* ds_part;            // workspace, [H, parts, B, K, 64]
};

// ---------------------------------------------------------------- dQ

constexpr int kKeyBuffer = 2 * kTileBytes + kThinBytes;    // K, V, the shared part

// A workgroup has 128 query rows.  It also writes their lse2 and delta, for the walks
// over query rows that follow.
template <typename Out, bool kBoth>
__global__ __launch_bounds__(kThreads, 2) void latent_dq_kernel(Params p) {
  __shared__ __align__(1024) unsigned char lds[2 * kKeyBuffer];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, h = lane >> 5;
  const int slot = int(blockIdx.x / unsigned(p.H)), head = int(blockIdx.x % unsigned(p.H));
  const Rows rows = find_rows<false>(p.cu, p.N, p.T, slot, p.slots, BM);
  if (rows.row0 >= rows.len) return;
  const Keys keys = find_keys(p.cu_kv, p.K, rows.n, rows.len);

  const int r0 = rows.row0 + wave * 32;
  const int r = min(r0 + l32, rows.len - 1);
  bf16x8 q[12], u[8];                                      // rows of Q and dO as B operands
  {
    const uint16_t* qs = p.q + (rows.first + r) * p.q_stride + head * DQ + 8 * h;
    const uint16_t* us = p.d_out + ((rows.first + r) * p.H + head) * D + 8 * h;
#pragma unroll
    for (int s = 0; s < 12; ++s) q[s] = *reinterpret_cast<const bf16x8*>(qs + 16 * s);
#pragma unroll
    for (int s = 0; s < 8; ++s) u[s] = *reinterpret_cast<const bf16x8*>(us + 16 * s);
  }
  const int64_t stat = (int64_t(rows.b) * p.H + head) * p.T + rows.start + r;
  float lse2 = p.lse[stat] * kLog2e;
  if (lse2 == -INFINITY) lse2 = INFINITY;                  // all scores -inf, or no keys: weights of zero
  const float c = p.scale * kLog2e;
  f32x16 dq[6];
#pragma unroll
  for (int d = 0; d < 6; ++d) dq[d] = (f32x16)(0.0f);

  const int see0 = r0 + keys.shift;                        // the last key that the wave's first row sees
  const int seen = min(rows.row0 + BM, rows.len) + keys.shift;
  const int tiles = max(seen + kTile - 1, 0) / kTile;
  TileLoad<kWaves> kload, vload;
  ThinLoad<kWaves> sload;
  kload.init(wave, lane, p.k_stride);
  vload.init(wave, lane, p.v_stride);
  sload.init(wave, lane, p.s_stride);
  const uint16_t* kb = p.k + keys.first * p.k_stride + head * p.k_head;
  const uint16_t* vb = p.v + keys.first * p.v_stride + head * p.v_head;
  const uint16_t* sb = p.s + keys.first * p.s_stride;
  auto issue = [&](int t, int at_buf) {
    unsigned char* buf = lds + at_buf * kKeyBuffer;
    const int64_t at = int64_t(t) * kTile;
    kload.issue(kb + at * p.k_stride, p.k_stride, keys.len - int(at), buf, wave);
    vload.issue(vb + at * p.v_stride, p.v_stride, keys.len - int(at), buf + kTileBytes, wave);
    sload.issue(sb + at * p.s_stride, p.s_stride, keys.len - int(at), buf + 2 * kTileBytes, wave);
  };
  // P^T and (dO V^T)^T (rows = keys) of 32 keys from key0; P is zero after the diagonal.
  auto scores = [&](const unsigned char* kt, int w, int key0, f32x16& s, f32x16& g) {
    s = g = (f32x16)(0.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) s = mfma32(read_rows(kt, 32 * w, l32, h, k), q[k], s);
#pragma unroll
    for (int k = 0; k < 4; ++k) s = mfma32(rows_of<2 * S>(kt + 2 * kTileBytes, 32 * w, l32, h, k), q[8 + k], s);
#pragma unroll
    for (int k = 0; k < 8; ++k) g = mfma32(read_rows(kt + kTileBytes, 32 * w, l32, h, k), u[k], g);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -lse2));
    if (key0 + 31 > see0) {
      const int last = see0 + l32 - key0;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (8 * (e >> 2) + 4 * h + (e & 3) > last) s[e] = g[e] = 0.0f;
    }
  };

  // delta.  The rounding of o to bfloat16 enters it, and with it every score's
  // gradient of the row (see attn_backward.hip).  Where few keys are seen (four tiles at
  // most, by the workgroup's last row; the walk is one for all its rows) it is made as
  // sum_j P_ij (dO V^T)_ij, to which it is equal: dQ's error, in halves of a rounding's, is
  // 1.54 with none or two tiles so, 1.43 with four and 1.42 with all (4 sequences of up to 690
  // tokens, 2 heads); four cost 5 us where no row sees more and nothing elsewhere, eight 15 of
  // 570.
  float delta = 0.0f;
  if (tiles <= 4) {
    if (tiles > 0) issue(0, 0);
    for (int t = 0; t < tiles; ++t) {
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
      kda::lds_barrier();
      if (t + 1 < tiles) issue(t + 1, (t + 1) & 1);
      for (int w = 0; w < 2; ++w) {
        const int key0 = t * kTile + 32 * w;
        if (key0 > see0 + 31) break;
        f32x16 s, g;
        scores(lds + (t & 1) * kKeyBuffer, w, key0, s, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) delta = __builtin_fmaf(s[e], g[e], delta);
      }
    }
    kda::lds_barrier();
  } else {
    const uint16_t* os = p.o + ((rows.first + r) * p.H + head) * D + 8 * h;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const bf16x8 x = *reinterpret_cast<const bf16x8*>(os + 16 * s);
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = __builtin_fmaf(float(x[j]), float(u[s][j]), delta);
    }
  }
  delta = half_sum(delta);
  if (r0 + l32 < rows.len && h == 0) {
    p.lse2[stat] = lse2;
    p.delta[stat] = delta;
  }

  if (tiles > 0) issue(0, 0);
  for (int t = 0; t < tiles; ++t) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    kda::lds_barrier();
    const unsigned char* kt = lds + (t & 1) * kKeyBuffer;
    const unsigned char* st = kt + 2 * kTileBytes;
    if (t + 1 < tiles) issue(t + 1, (t + 1) & 1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int key0 = t * kTile + 32 * w;
      if (key0 > see0 + 31) continue;
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
        bf16x8 rest;
        if constexpr (kBoth) rest = pack8_rest(x, b);
#pragma unroll
        for (int d = 0; d < 6; ++d) {
          const bf16x8 a = d < 4 ? columns_of<256>(kt, 32 * w, k, 32 * d, lane)
                                 : columns_of<2 * S>(st, 32 * w, k, 32 * (d - 4), lane);
          dq[d] = mfma32(a, b, dq[d]);
          if constexpr (kBoth) dq[d] = mfma32(a, rest, dq[d]);
        }
      }
    }
  }
  if (r0 + l32 >= rows.len) return;
  Out* dst = static_cast<Out*>(p.dq) + ((rows.first + r) * p.H + head) * DQ;
#pragma unroll
  for (int d = 0; d < 6; ++d) store_row32(dst + 32 * d, dq[d], p.scale, h);
}

// ---------------------------------------------------------------- dK and dV

constexpr int kRowBuffer = kTileBytes + kThinBytes + kTileBytes + 512;     // Q (128 and 64 wide), dO, lse2, delta

// Nothing moves across.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Two waves to 32 keys: one makes P and dS of 32 query rows, the other adds the
// products with those of the 32 rows before them to dK and dV.  Each has 20 of the 40
// products; together they are what a SIMD's registers hold, and while one computes
// weights the other's products go on.
template <typename Out, bool kBoth>
__global__ __launch_bounds__(2 * kThreads, 2) void latent_dkv_kernel(Params p) {
  constexpr int kLoadWaves = 2 * kWaves, kRing = kBoth ? 2 : 3, kTerms = kBoth ? 4 : 2;
  __shared__ __align__(1024) struct {
    unsigned char ring[kRing][kRowBuffer];
    unsigned char terms[2][kWaves][kTerms][2][1024];       // P, dS (and what their rounding left) as operands
  } lds;
  auto &ring = lds.ring;
  auto &terms = lds.terms;
  const unsigned id = blockIdx.x;
  const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wave = all_waves & (kWaves - 1), role = all_waves / kWaves;
  const int l32 = lane & 31, h = lane >> 5;
  const unsigned heads = p.H;
  const int head = int(id % heads);
  const int part = int((id / heads) % unsigned(p.parts));
  const Rows keys = find_rows<true>(p.cu_kv, p.N, p.K, int(id / (heads * p.parts)), p.key_slots, BM);
  if (keys.row0 >= keys.len) return;
  const Keys rows = find_keys(p.cu, p.T, keys.n, 0);       // the sequence's query rows
  const int shift = keys.len - rows.len;                   // key j is seen from row j - shift on

  const int k0 = keys.row0 + wave * 32;                    // this wave's first key
  const int key = min(k0 + l32, keys.len - 1);
  // Query tiles from the one that holds the first row that sees the first key.
  const int t0 = max(keys.row0 - shift, 0) / kTile, walk = max((rows.len + kTile - 1) / kTile - t0, 0);
  const int begin = t0 + int(int64_t(walk) * part / p.parts), end = t0 + int(int64_t(walk) * (part + 1) / p.parts);
  const int steps = 2 * max(end - begin, 0);               // of 32 rows
  TileLoad<kLoadWaves> qload, uload;
  ThinLoad<kLoadWaves> q2load;
  const int64_t u_stride = int64_t(p.H) * D;
  qload.init(all_waves, lane, p.q_stride);
  q2load.init(all_waves, lane, p.q_stride);
  uload.init(all_waves, lane, u_stride);
  const uint16_t* qb = p.q + rows.first * p.q_stride + head * DQ;
  const uint16_t* ub = p.d_out + rows.first * u_stride + head * D;
  const int64_t b = p.cu ? 0 : keys.n, start = rows.first - b * p.T;
  const int64_t stat0 = (b * p.H + head) * p.T + start;
  constexpr int kLoads = 5;                                // of a wave for a tile (two have one more)
  auto issue = [&](int i) {                                // tile begin + i; behind the last nothing comes
    const int row = min(begin + i, end) * kTile, left = begin + i < end ? rows.len - row : 0;
    const int64_t at = row;
    unsigned char* buf = ring[i % kRing];
    qload.issue(qb + at * p.q_stride, p.q_stride, left, buf, all_waves);
    q2load.issue(qb + at * p.q_stride + D, p.q_stride, left, buf + kTileBytes, all_waves);
    uload.issue(ub + at * u_stride, u_stride, left, buf + kTileBytes + kThinBytes, all_waves);
    if (all_waves == 0) load_floats(p.lse2 + stat0 + at, left, buf + 2 * kTileBytes + kThinBytes, lane);
    if (all_waves == 1) load_floats(p.delta + stat0 + at, left, buf + 2 * kTileBytes + kThinBytes + 256, lane);
  };
  // Before step i: its rows are there, and the terms of the step before.
  auto arrive = [&](int i) {
    if (i % 2 == 0) __builtin_amdgcn_s_waitcnt(kWaitLoads | (kRing == 3 ? kLoads : 0));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    kda::lds_barrier();
    if (i % 2 == 1) issue(i / 2 + kRing - 1);              // (the tile in its place was used a step before)
  };
  auto skipped = [&](int i) {                              // none of the rows sees this wave's keys
    return begin * kTile + 32 * i + 31 < k0 - shift;
  };

  if (role == 0) {
    bf16x8 kk[12], vv[8];                                    // rows of [K s] and V as B operands
    {
      const uint16_t* ks = p.k + (keys.first + key) * p.k_stride + head * p.k_head + 8 * h;
      const uint16_t* ss = p.s + (keys.first + key) * p.s_stride + 8 * h;
      const uint16_t* vs = p.v + (keys.first + key) * p.v_stride + head * p.v_head + 8 * h;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        kk[s] = *reinterpret_cast<const bf16x8*>(ks + 16 * s);
        vv[s] = *reinterpret_cast<const bf16x8*>(vs + 16 * s);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) kk[8 + s] = *reinterpret_cast<const bf16x8*>(ss + 16 * s);
    }
    const float c = p.scale * kLog2e;
    if (steps > 0) {
#pragma unroll
      for (int i = 0; i < kRing - 1; ++i) issue(i);
    }
    // The keys are waited for before the first step: left to the compiler they would be
    // in every step, and with them the loads behind them.
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    for (int i = 0; i < steps; ++i) {
      arrive(i);
      if (skipped(i)) continue;
      const unsigned char* qt = ring[i / 2 % kRing];
      const unsigned char *q2t = qt + kTileBytes, *ut = q2t + kThinBytes;
      const float* stats = reinterpret_cast<const float*>(ut + kTileBytes);
      const int w = i & 1, row0 = begin * kTile + 32 * i;
      f32x16 s = (f32x16)(0.0f), g = (f32x16)(0.0f);       // S and dO V^T, rows = query rows
      // Operands are read kAhead products before they are used, and what follows from S
      // is made while the products of dO V^T go on.
      constexpr int kAhead = 4;
      bf16x8 a[kAhead];
      f32x4 stat[4], del[4];
      auto fetch = [&](int j) {
        a[j % kAhead] = j < 8    ? read_rows(qt, 32 * w, l32, h, j)
                        : j < 12 ? rows_of<2 * S>(q2t, 32 * w, l32, h, j - 8)
                                 : read_rows(ut, 32 * w, l32, h, j - 12);
      };
#pragma unroll
      for (int j = 0; j < kAhead - 1; ++j) fetch(j);
#pragma unroll
      for (int j = 0; j < 20; ++j) {
        fence();
        if (j + kAhead - 1 < 20) fetch(j + kAhead - 1);
        if (j >= 6 && j < 10) stat[j - 6] = *reinterpret_cast<const f32x4*>(stats + 32 * w + 8 * (j - 6) + 4 * h);
        if (j >= 14 && j < 18)
          del[j - 14] = *reinterpret_cast<const f32x4*>(stats + 64 + 32 * w + 8 * (j - 14) + 4 * h);
        fence();
        if (j < 12) {
          s = mfma32(a[j % kAhead], kk[j], s);
        } else {
          g = mfma32(a[j % kAhead], vv[j - 12], g);
#pragma unroll
          for (int e = 2 * (j - 12); e < 2 * (j - 12) + 2; ++e)
            s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -stat[e >> 2][e & 3]));
        }
      }
      fence();
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] = s[e] * (g[e] - del[e >> 2][e & 3]);
      if (row0 + shift < k0 + 31 || row0 + 32 > rows.len) { // pairs behind the diagonal, rows behind the end
        fence();                                           // (or it is done for all pairs, with selects)
        const int first = k0 + l32 - shift - row0, behind = rows.len - row0;
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
        auto put = [&](int term, bf16x8 z) {
          *reinterpret_cast<bf16x8*>(terms[i & 1][wave][term][k] + lane * 16) = z;
        };
        const bf16x8 pb = pack8(x), gb = pack8(y);
        put(0, pb);
        put(1, gb);
        if constexpr (kBoth) put(2, pack8_rest(x, pb)), put(3, pack8_rest(y, gb));
      }
    }
    if (steps > 0) arrive(steps);
    __builtin_amdgcn_s_waitcnt(kWaitLoads);                // (those that brought nothing)
    return;
  }

  f32x16 dk[6], dv[4];
#pragma unroll
  for (int d = 0; d < 6; ++d) dk[d] = (f32x16)(0.0f);
#pragma unroll
  for (int d = 0; d < 4; ++d) dv[d] = (f32x16)(0.0f);
  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue(i);
    arrive(0);
  }
  for (int i = 1; i <= steps; ++i) {
    arrive(i);
    const int before = i - 1;
    if (skipped(before)) continue;
    const unsigned char* qt = ring[before / 2 % kRing];
    const unsigned char *q2t = qt + kTileBytes, *ut = q2t + kThinBytes;
    const int w = before & 1;
    bf16x8 term[2][kTerms];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < kTerms; ++x)
        term[k][x] = *reinterpret_cast<const bf16x8*>(terms[before & 1][wave][x][k] + lane * 16);
    constexpr int kAhead = 3;                              // as above
    bf16x8 a[kAhead];
    auto fetch = [&](int j) {
      const int k = j / 10, d = j % 10;
      a[j % kAhead] = d < 4   ? columns_of<256>(ut, 32 * w, k, 32 * d, lane)
                      : d < 8 ? columns_of<256>(qt, 32 * w, k, 32 * (d - 4), lane)
                              : columns_of<2 * S>(q2t, 32 * w, k, 32 * (d - 8), lane);
    };
#pragma unroll
    for (int j = 0; j < kAhead - 1; ++j) fetch(j);
#pragma unroll
    for (int j = 0; j < 20; ++j) {
      const int k = j / 10, d = j % 10, x = d < 4 ? 0 : 1;
      fence();
      if (j + kAhead - 1 < 20) fetch(j + kAhead - 1);
      fence();
      f32x16& sum = d < 4 ? dv[d & 3] : dk[d < 4 ? 0 : d - 4];
      sum = mfma32(a[j % kAhead], term[k][x], sum);
      if constexpr (kBoth) sum = mfma32(a[j % kAhead], term[k][x + 2], sum);
    }
    fence();
  }
  __builtin_amdgcn_s_waitcnt(kWaitLoads);                  // (those that brought nothing)
  if (k0 + l32 >= keys.len) return;
  // (with parts, Out is float and dkv is the parts' buffer)
  const int64_t all = int64_t(p.B) * p.K, at = keys.first + key;
  Out* dst = static_cast<Out*>(p.parts > 1 ? p.dkv_part : p.dkv) + ((part * all + at) * p.H + head) * (2 * D);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    store_row32(dst + 32 * d, dk[d], p.scale, h);
    store_row32(dst + D + 32 * d, dv[d], 1.0f, h);
  }
  float* ds = p.ds_part + ((int64_t(head) * p.parts + part) * all + at) * S;
#pragma unroll
  for (int d = 0; d < 2; ++d) store_row32(ds + 32 * d, dk[4 + d], p.scale, h);
}

// ---------------------------------------------------------------- the parts' sums

// `parts` arrays of rows of WIDTH floats added up in order, four elements per
// thread.  Rows outside the sequences are left as they are.
template <typename Out>
__device__ __forceinline__ void sum_parts(const float* src, int64_t rows, int64_t width, int parts, Out* dst,
                                          const int32_t* cu, int N, int64_t at) {
  const int64_t size = rows * width;
  if (cu) {
    // From the first offset to the last one every row is passed by some sequence;
    // other rows lie in one only where offsets decrease.
    const int row = int(min(at, size - 1) / width);
    bool in = row >= cu[0] && row < cu[N];
    uint64_t open = __ballot(!in);
    while (open) {                                         // a wave's 256 elements lie in four rows at most
      const int t = __builtin_amdgcn_readlane(row, __builtin_ctzll(open));
      if (in_sequence(cu, N, t)) in |= row == t;
      open &= ~__ballot(row == t);
    }
    if (!in) return;
  }
  if (at >= size) return;
  f32x4 sum = *reinterpret_cast<const f32x4*>(src + at);
#pragma unroll 4
  for (int i = 1; i < parts; ++i) sum += *reinterpret_cast<const f32x4*>(src + i * size + at);
  store4(dst + at, sum);
}

template <typename Out>
__global__ __launch_bounds__(256) void latent_sum_kernel(Params p, unsigned shared_blocks) {
  const int64_t rows = int64_t(p.B) * p.K;
  if (blockIdx.x < shared_blocks)
    sum_parts<Out>(p.ds_part, rows, S, p.H * p.parts, static_cast<Out*>(p.ds), p.cu_kv, p.N,
                       (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4);
  else
    sum_parts<Out>(p.dkv_part, rows, int64_t(p.H) * 2 * D, p.parts, static_cast<Out*>(p.dkv), p.cu_kv, p.N,
                       (int64_t(blockIdx.x - shared_blocks) * 256 + threadIdx.x) * 4);
}

// Workgroups that share a key tile: enough for every compute unit to have one, or two
// where all walks but the longest are shorter (one length, from the diagonal on) and long
// enough to be cut.  For one and for two, a training pass in us:
//   one length: 8 heads x 4096 tokens 367 and 347, 4 x 8192 695 and 636, 16 x 2048 204 and 205,
//     16 x 1000 111 and 123
//   packed: 8 heads x 8 of up to 1000 134 and 169, 4 x 5 of 2000 196 and 214, 12 x 6 of 1200 150 and 194
int parts_for(int64_t key_slots, int T, int N, bool packed, int H) {
  const int64_t len = kda::attn_typical(T, N, packed), cus = kda::device_cus();
  const int64_t units = key_slots * H, want = (!packed || N == 1) && len > 2048 ? 2 * cus : cus;
  if (units == 0 || units >= want) return 1;
  const int64_t walk = len / kTile / 2 + 1;
  const int64_t most = walk / 2 < 1 ? 1 : (walk / 2 > 16 ? 16 : walk / 2);
  const int64_t parts = (want + units - 1) / units;
  return int(parts < most ? parts : most);
}

// Whether weights and score gradients are carried as two bfloat16 terms, which leaves a
// gradient the error of its own rounding instead of 1.41 times that (by chance more
// where there are few of them, 1.46 with 300 rows x 5 heads) and there costs little: 48.5 to
// 52.5 us for 2 sequences of up to 201 tokens, 5 heads, 53.5 to 57.3 for 4 of up to 228, 12 heads.
bool both_terms(int64_t rows, int64_t len) { return rows * len <= 1 << 19; }

struct Plan {
  int64_t slots, key_slots;
  int parts;
  size_t stats, dkv, ds;     // floats
  int64_t sums, shared;      // workgroups of the sums
  bool fits;
  size_t bytes() const { return (2 * stats + dkv + ds) * sizeof(float); }
};
Plan plan_for(int64_t B, int T, int T_kv, int H, int num_seqs) {
  Plan x{};
  x.slots = kda::attn_slots(B, T, num_seqs);
  x.key_slots = kda::attn_slots(B, T_kv, num_seqs);
  if (x.slots > kda::kMostBlocks || x.key_slots > kda::kMostBlocks) return x;   // (what follows fits 64 bits then)
  x.parts = parts_for(x.key_slots, T, num_seqs ? num_seqs : int(B), num_seqs > 0, H);
  x.stats = kda::attn_stat_floats(B, T, H);
  const int64_t rows = B * T_kv;
  x.dkv = x.parts > 1 ? size_t(x.parts) * rows * H * 2 * D : 0;
  x.ds = size_t(x.parts) * H * rows * S;
  x.shared = (rows * S / 4 + 255) / 256;
  x.sums = x.shared + (x.parts > 1 ? (rows * H * 2 * D / 4 + 255) / 256 : 0);
  const int64_t keys = x.key_slots * x.parts * H;          // of twice as many threads
  x.fits = x.slots * H + keys <= kda::kMostBlocks && keys <= kda::kMostBlocks / 2 && x.sums <= kda::kMostBlocks;
  return x;
}

template <typename Out, bool kBoth>
void launch_grads(const Params& p, unsigned key_blocks, unsigned blocks, hipStream_t stream) {
  if (blocks) hipLaunchKernelGGL((latent_dq_kernel<Out, kBoth>), dim3(blocks), dim3(kThreads), 0, stream, p);
  const dim3 keys(key_blocks);
  if (key_blocks && p.parts == 1)
    hipLaunchKernelGGL((latent_dkv_kernel<Out, kBoth>), keys, dim3(2 * kThreads), 0, stream, p);
  else if (key_blocks)
    hipLaunchKernelGGL((latent_dkv_kernel<float, kBoth>), keys, dim3(2 * kThreads), 0, stream, p);
}

template <typename Out>
int launch(const Params& p, const Plan& x, hipStream_t stream) {
  const unsigned blocks = unsigned(x.slots * p.H), key_blocks = unsigned(x.key_slots * p.H * p.parts);
  if (both_terms(int64_t(p.B) * p.T * p.H, kda::attn_typical(p.K, p.N, p.cu != nullptr)))
    launch_grads<Out, true>(p, key_blocks, blocks, stream);
  else
    launch_grads<Out, false>(p, key_blocks, blocks, stream);
  if (x.sums)
    hipLaunchKernelGGL(latent_sum_kernel<Out>, dim3(unsigned(x.sums)), dim3(256), 0, stream, p, unsigned(x.shared));
  return kda::launch_status();
}

}  // namespace

extern "C" size_t kda_latent_backward_workspace_size(int32_t B, int32_t T, int32_t T_kv, int32_t H, int32_t num_seqs) {
  if (B < 1 || T < 0 || T_kv < 0 || H < 1 || H > kda::kLatentHeads || num_seqs < 0 || (num_seqs && B != 1)) return 0;
  if (T == 0 && T_kv == 0) return 0;
  const Plan x = plan_for(B, T, T_kv, H, num_seqs);
  return x.fits ? x.bytes() : 0;
}

extern "C" int kda_latent_backward(const void* q, const void* k, const void* k_shared, const void* v, int64_t q_stride,
                                   int64_t k_stride, int64_t k_head, int64_t s_stride, int64_t v_stride,
                                   int64_t v_head, const void* o, const float* lse, const void* d_out,
                                   const int32_t* cu_seqlens, const int32_t* cu_seqlens_kv, int32_t num_seqs,
                                   int32_t B, int32_t T, int32_t T_kv, int32_t H, float scale, void* dq, void* d_kv,
                                   void* dk_shared, int32_t grad_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const kda::LatentLayout l{q_stride, k_stride, k_head, s_stride, v_stride, v_head};
  const int e = kda::latent_check(l, cu_seqlens, cu_seqlens_kv, num_seqs, B, T, T_kv, H, scale);
  if (e != KDA_OK) return e;
  if (grad_dtype != KDA_GRAD_FLOAT32 && grad_dtype != KDA_GRAD_INPUT_DTYPE) return KDA_ERR_UNSUPPORTED;
  if (T == 0 && T_kv == 0) return KDA_OK;
  if ((T && (!q || !o || !lse || !d_out || !dq)) || (T_kv && (!k || !k_shared || !v || !d_kv || !dk_shared)) ||
      !workspace)
    return KDA_ERR_NULL;
  for (const void* y : {q, k, k_shared, v, o, static_cast<const void*>(lse), d_out, static_cast<const void*>(dq),
                        static_cast<const void*>(d_kv), static_cast<const void*>(dk_shared),
                        static_cast<const void*>(workspace)})
    if (!kda::aligned16(y)) return KDA_ERR_ALIGN;
  const int seqs = cu_seqlens ? num_seqs : 0;
  const Plan x = plan_for(B, T, T_kv, H, seqs);
  if (!x.fits) return KDA_ERR_SHAPE;
  if (workspace_bytes < x.bytes()) return KDA_ERR_WORKSPACE;
  float* ws = static_cast<float*>(workspace);
  const int N = cu_seqlens ? num_seqs : B;
  const Params p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                 static_cast<const uint16_t*>(k_shared), static_cast<const uint16_t*>(o),
                 static_cast<const uint16_t*>(d_out), q_stride, k_stride, v_stride, s_stride, k_head, v_head, lse,
                 cu_seqlens, cu_seqlens_kv, N, B, T, T_kv, H, int(x.slots), int(x.key_slots), scale, dq, d_kv,
                 dk_shared, ws, ws + x.stats, x.parts, ws + 2 * x.stats, ws + 2 * x.stats + x.dkv};
  return grad_dtype == KDA_GRAD_FLOAT32 ? launch<float>(p, x, kda::as_stream(stream))
                                        : launch<uint16_t>(p, x, kda::as_stream(stream));
}
