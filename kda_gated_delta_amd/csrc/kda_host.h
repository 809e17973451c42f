// Host-side helpers shared by the entry points: status handling and
// metadata checks.  No allocation, no synchronisation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda.h"

namespace kda {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// Compute units of the current device, cached per device (256, MI355X's
// count, when the runtime reports no device).  Launch shapes and the choice
// between kernels follow it.
inline int device_cus() {
  constexpr int kDevices = 64;
  static std::atomic<int> cache[kDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return 256;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Map the runtime's view of the most recent launch to a status.
inline int launch_status() {
  hipError_t e = hipGetLastError();
  return e == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

// Sizes shared by the full-attention entry points: heads 128 wide, query
// heads in equal groups, packed sequences in one batch row, strides that keep
// every row 16-byte aligned and a 64-row tile's offsets within 31 bits.
inline int attn_heads(int32_t HQ, int32_t HKV, int32_t D) {
  if (HQ < 1 || HKV < 1 || HQ > 65535 || HQ % HKV != 0) return KDA_ERR_SHAPE;
  return D == 128 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
inline int attn_stride(int64_t stride, int32_t heads) {
  if (stride < int64_t(heads) * 128 || stride > (int64_t(1) << 23)) return KDA_ERR_SHAPE;
  return stride % 8 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}
// Workgroups (of 256 threads) that a launch takes: the runtime counts its threads
// in 32 bits.
constexpr int64_t kMostBlocks = (int64_t(1) << 24) - 1;
// Pages of 16 to 256 tokens, a power of two; slot numbers (page x page_size +
// offset) fit int32.
inline bool attn_page(int32_t page_size) {
  return page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0;
}
inline int attn_cache(int32_t HKV, int32_t page_size, int64_t page_stride, int32_t num_pages) {
  if (!attn_page(page_size)) return KDA_ERR_UNSUPPORTED;
  if (num_pages < 0 || int64_t(num_pages) * page_size > 0x7fffffff) return KDA_ERR_SHAPE;
  if (page_stride < int64_t(HKV) * page_size * 128 || page_stride > (int64_t(1) << 32)) return KDA_ERR_SHAPE;
  return page_stride % 16 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}
inline int attn_scale(float scale) { return scale > 0.0f && scale < 1e30f ? KDA_OK : KDA_ERR_SHAPE; }
inline int attn_check(const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T, int32_t HQ, int32_t HKV, int32_t D,
                      float scale, int64_t q_stride, int64_t k_stride, int64_t v_stride) {
  if (B < 1 || T < 0 || (cu && (B != 1 || num_seqs < 1))) return KDA_ERR_SHAPE;
  int e = attn_heads(HQ, HKV, D);
  if (e == KDA_OK) e = attn_scale(scale);
  if (e == KDA_OK) e = attn_stride(q_stride, HQ);
  if (e == KDA_OK) e = attn_stride(k_stride, HKV);
  if (e == KDA_OK) e = attn_stride(v_stride, HKV);
  return e;
}

// Row tiles that a prompt call may have (num_seqs: 0 without packed sequences), and the
// floats that a statistic of every row and head takes.
constexpr int kAttnRows = 128;
inline int64_t attn_slots(int64_t B, int64_t T, int64_t num_seqs) {
  return num_seqs ? T / kAttnRows + num_seqs : B * ((T + kAttnRows - 1) / kAttnRows);
}
inline size_t attn_stat_floats(int64_t B, int64_t T, int64_t heads) { return size_t((B * T * heads + 3) / 4 * 4); }

// Length of a typical sequence of a prompt call.
inline int64_t attn_typical(int T, int num_seqs, bool packed) { return packed ? T / num_seqs : T; }
// Whether the forward walks a row tile's keys with two sets of waves, which halves
// the chain that the longest walk is but costs a join and, with an odd number of
// tiles, a pause.  It pays where one workgroup per compute unit leaves half of
// the wave slots empty, or where two of them are all there are, so that nothing
// is left to fill the device behind the longest.  One set against two, us:
//   one workgroup per unit (8 heads on 2; 400, 600, 1000, 2000 tokens): 11.2, 14.8, 21.7, 37.6 and 11.3,
//     13.8, 18.9, 31.7
//   two (2000 x 32 heads, 2500 x 24, 4096 x 16, 8192 x 8): 47.5, 55.5, 88.4, 170 and 48.7, 52.2, 79, 143
//   three (12000 x 8): 284 and 303
inline bool attn_split(int64_t blocks, int T, int num_seqs, bool packed) {
  const int64_t len = attn_typical(T, num_seqs, packed), cus = device_cus();
  return (blocks <= cus && len >= 512) || (blocks <= 2 * cus && len >= 2048);
}

// Sizes shared by the latent-attention entry points.  Keys and values are read
// through a token's and a head's stride (heads may be slices of one projection's
// rows, or the outer axis); strides keep every row 16-byte aligned and a 64-row
// tile's offsets within 31 bits.
struct LatentLayout {
  int64_t q_stride, k_stride, k_head, s_stride, v_stride, v_head;
};
inline int latent_stride(int64_t stride, int64_t least) {
  if (stride < least || stride > (int64_t(1) << 23)) return KDA_ERR_SHAPE;
  return stride % 8 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}
inline int latent_head(int64_t stride) {
  if (stride < 0 || stride > (int64_t(1) << 40)) return KDA_ERR_SHAPE;
  return stride % 8 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}
// (a row of queries is heads x 192 of at most 2^23)
constexpr int32_t kLatentHeads = (1 << 23) / 192;
inline int latent_check(const LatentLayout& x, const int32_t* cu, const int32_t* cu_kv, int32_t num_seqs, int32_t B,
                        int32_t T, int32_t T_kv, int32_t H, float scale) {
  if (B < 1 || T < 0 || T_kv < 0 || (!cu) != (!cu_kv) || (cu && (B != 1 || num_seqs < 1))) return KDA_ERR_SHAPE;
  if (H < 1 || H > kLatentHeads) return KDA_ERR_SHAPE;
  int e = attn_scale(scale);
  if (e == KDA_OK) e = latent_stride(x.q_stride, int64_t(H) * 192);
  if (e == KDA_OK) e = latent_stride(x.k_stride, 128);
  if (e == KDA_OK) e = latent_stride(x.v_stride, 128);
  if (e == KDA_OK) e = latent_stride(x.s_stride, 64);
  if (e == KDA_OK) e = latent_head(x.k_head);
  if (e == KDA_OK) e = latent_head(x.v_head);
  return e;
}
// The latent cache: pages as the attention cache's, each of its three parts with a
// page stride of its own (in elements), of which a row keeps its alignment.
struct LatentCache {
  int32_t page_size, num_pages;
  int64_t c_stride, scale_stride, s_stride;
};
inline int latent_cache(const LatentCache& x) {
  if (!attn_page(x.page_size)) return KDA_ERR_UNSUPPORTED;
  if (x.num_pages < 0 || int64_t(x.num_pages) * x.page_size > 0x7fffffff) return KDA_ERR_SHAPE;
  if (x.c_stride < int64_t(x.page_size) * 512 || x.c_stride >= (int64_t(1) << 32)) return KDA_ERR_SHAPE;
  if (x.scale_stride < int64_t(x.page_size) * 4 || x.scale_stride >= (int64_t(1) << 32)) return KDA_ERR_SHAPE;
  if (x.s_stride < int64_t(x.page_size) * 64 || x.s_stride >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
  return x.c_stride % 16 == 0 && x.scale_stride % 4 == 0 && x.s_stride % 8 == 0 ? KDA_OK : KDA_ERR_ALIGN;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace kda
