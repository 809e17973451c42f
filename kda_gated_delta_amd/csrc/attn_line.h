// Decode's line of work (gfx950 / CDNA4, wave64): all segments, which are a
// sequence's (head, row tile) walks over its tokens, one after another in units of
// tokens, cut into equal pieces whatever the sequences' lengths are.
#pragma once

#include "attn_device.h"

namespace kda {
namespace line {

template <typename P>
__device__ __forceinline__ int length(P& p, int n) { return min(max(p.lens[n], 0), p.width << p.shift); }
// An empty sequence has one unit too: somebody writes its zeros.
template <int UNIT>
__device__ __forceinline__ int units_of(int len) { return max((len + UNIT - 1) / UNIT, 1); }

// A lane's value for the whole wave, in scalar registers.
__device__ __forceinline__ int64_t lane_value(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(uint64_t(x)), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(uint64_t(x) >> 32), lane);
  return int64_t(uint64_t(hi) << 32 | lo);
}

// x plus what CTRL's lane holds, in the rows of 16 lanes that ROWS names and have one.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t plus_lane(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(uint64_t(x))), CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(uint64_t(x) >> 32)), CTRL, ROWS, 0xf, false);
  return x + int64_t(uint64_t(hi) << 32 | lo);
}
// Sum over the lanes up to each.  (Shuffles through LDS would cost every workgroup half
// a microsecond of its start.)
__device__ __forceinline__ int64_t sum_upto(int64_t x) {
  x = plus_lane<0x111, 0xf>(x);                  // 1, 2, 4, 8 lanes before, within rows
  x = plus_lane<0x112, 0xf>(x);
  x = plus_lane<0x114, 0xf>(x);
  x = plus_lane<0x118, 0xf>(x);
  x = plus_lane<0x142, 0xa>(x);                  // the row before's last lane
  return plus_lane<0x143, 0xc>(x);               // lane 31
}

// Where a piece of the line begins.  WAVES successive pieces belong to a workgroup,
// one to each wave (or one to all of it, with WAVES = 1).
struct Piece {
  int w;             // its place in the line
  int64_t from, to;  // its units
  int64_t lo, hi;    // its workgroup's units, if all its pieces have some; else empty
  int n, len;        // the sequence that holds the first, and its length
  int64_t before;    // units of the sequences before it
};

// The line has U = per x (units of all sequences) units, per = heads x row
// tiles; place w of W = min(waves, U) takes floor(U w / W) .. floor(U (w + 1) / W) - 1.
// With EXTRA every segment counts as many units more, before its own: what it costs to
// begin and end one, so that a piece that does so in its middle is shorter.
// A 64-way search: each lane sums a stretch of sequences, the wave adds up and
// picks the stretch that holds the unit, down to one sequence.
template <int UNIT, int WAVES, int EXTRA = 0, typename P>
__device__ __forceinline__ Piece find_piece(const P& p, int wave, int per) {
  const int lane = threadIdx.x & 63;
  Piece x{};
  int lo = 0, hi = p.N;
  bool top = true;
  do {
    const int step = (hi - lo + 63) / 64;
    const int a = min(lo + lane * step, hi), b = min(a + step, hi);
    int64_t own = 0;
    int len = 0;
#pragma unroll 8
    for (int n = a; n < b; ++n) len = length(p, n), own += units_of<UNIT>(len) + EXTRA;
    own *= per;
    const int64_t end = sum_upto(own);
    if (top) {
      const int64_t total = lane_value(end, 63), waves = min(total, int64_t(p.waves));
      // floor(total i / waves) without a long division for each i
      const unsigned parts = unsigned(waves);
      const int64_t each = total <= 0x7fffffff ? int64_t(unsigned(total) / parts) : total / waves;
      const unsigned left = unsigned(total - each * waves);
      auto cut = [&](int i) { return each * i + int64_t(left * unsigned(i) / parts); };
      x.w = int(blockIdx.x) * WAVES + wave;
      if (x.w >= waves) return x;            // nothing for this wave
      if (x.w - wave + WAVES <= waves) {
        x.lo = cut(x.w - wave);
        x.hi = cut(x.w - wave + WAVES);
      }
      x.from = cut(x.w);
      x.to = cut(x.w + 1);
      top = false;
    }
    const uint64_t upto = __ballot(x.before + end <= x.from);   // lanes whose sequences all end before it
    const int k = min(int(__builtin_popcountll(upto)), (hi - lo + step - 1) / step - 1);
    x.before += lane_value(end - own, k);
    x.len = __builtin_amdgcn_readlane(len, k);     // in the last round a stretch is one sequence
    lo += k * step;
    hi = min(lo + step, hi);
  } while (hi - lo > 1);
  x.n = lo;
  return x;
}

}  // namespace line
}  // namespace kda
