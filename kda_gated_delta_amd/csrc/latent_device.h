// Device helpers shared by the latent-attention kernels (gfx950 / CDNA4,
// wave64): widths, and tiles in LDS whose lines are an odd multiple of 128 bytes.
#pragma once

#include "attn_device.h"

namespace kda {
namespace latent {

using namespace kda::attn;

constexpr int R = 512;                   // the latent
constexpr int S = 64;                    // the key part that all heads share
constexpr int DQ = D + S;                // an expanded query
constexpr int kBlocks = R / 128;         // scales of a token

// The lane, made anew: what is made of it again for every unit or tile takes no
// register from the queries and the output meanwhile.
__device__ __forceinline__ int lane_now() {
  int x;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
  return x;
}

// Lines of 128 bytes, or of an odd multiple: successive lines begin in the two
// halves of the banks' 256 bytes by turns.  Piece c (16 bytes) of line r is stored
// at place c ^ turn(r): 16 successive lines hold one piece in 16 different places,
// and 4 successive lines hold one 64-byte block in the four quarters, so neither
// rows nor transposed columns meet a bank twice.
__device__ __forceinline__ int turn(int line) { return ((line & 2) << 1) | ((line >> 2) & 3); }

// As attn_device.h's read_rows, of a tile with lines of BYTES.
template <int BYTES>
__device__ __forceinline__ bf16x8 rows_of(const unsigned char* tile, int r, int l32, int h, int s) {
  const int line = r + l32;
  return *reinterpret_cast<const bf16x8*>(tile + line * BYTES + (((2 * s + h) ^ turn(line)) * 16));
}

// Transposing reads.  What they read was waited for by whoever calls them: as calls
// with a pointer of their own (restrict) the compiler does not take them to read what
// loads to LDS that are still on their way will write, and does not wait for those.
__device__ __forceinline__ s16x4 transposed(const lds_s16x4* __restrict p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_s16x4*>(p));
}
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
__device__ __forceinline__ i32x2 transposed(const lds_i32x2* __restrict p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32(const_cast<lds_i32x2*>(p));
}

// As attn_device.h's read_columns, of a tile with lines of BYTES in the order `turn`.
template <int BYTES>
__device__ __forceinline__ bf16x8 columns_of(const unsigned char* tile, int r, int m, int c, int lane) {
  const int j = lane & 15, h = lane >> 5;
  const int line = r + 16 * m + 4 * h + (j >> 2);
  const int col = c + (lane & 16) + 4 * (j & 3);
  const int piece = col >> 3, half = (col & 4) * 2;
  const unsigned char* p = tile + line * BYTES + half;
  auto place = [](int line) { return BYTES == 256 ? swizzle(line) : turn(line); };
  const s16x4 a = transposed((const lds_s16x4*)(p + (piece ^ place(line)) * 16));
  const s16x4 b = transposed((const lds_s16x4*)(p + 8 * BYTES + (piece ^ place(line + 8)) * 16));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// A tile of 64 rows of 64 bf16 (lines of 128 bytes), loaded as TileLoad's.
constexpr int kThinBytes = kTile * 2 * S;
template <int WAVES>
struct ThinLoad {
  uint32_t lane_off, step;
  static_assert(8 % WAVES == 0 && WAVES % 4 == 0, "the turn must be the same in all blocks of a wave");

  __device__ __forceinline__ void init(int wave, int lane, int64_t stride) {
    const int line = 8 * wave + (lane >> 3);
    lane_off = uint32_t(line * stride * 2) + ((lane & 7) ^ turn(line)) * 16;
    step = uint32_t(8 * WAVES * stride * 2);
  }
  __device__ __forceinline__ void issue(const uint16_t* base, int64_t stride, int rows, unsigned char* lds,
                                        int wave) const {
    const uint32_t bytes = uint32_t(min(rows, kTile)) * uint32_t(stride * 2);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, bytes, 0x00020000);
#pragma unroll
    for (int j = 0; j < 8 / WAVES; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr*)(lds + (wave + j * WAVES) * 1024), 16, lane_off,
                                               j * step, 0, 0);
  }
};

// The keys that go with the rows of a sequence.
struct Keys {
  int64_t first;   // the first, counted over the whole batch
  int len;
  int shift;       // row i sees keys 0 .. i + shift
};
__device__ __forceinline__ Keys find_keys(const int32_t* cu, int K, int n, int rows) {
  Keys x;
  if (cu) {
    const int c0 = offset_of(cu, n, K), c1 = offset_of(cu, n + 1, K);
    x.first = c0;
    x.len = max(c1 - c0, 0);
  } else {
    x.first = int64_t(n) * K;
    x.len = K;
  }
  x.shift = x.len - rows;
  return x;
}

}  // namespace latent
}  // namespace kda
