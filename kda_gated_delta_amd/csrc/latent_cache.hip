// The paged 8-bit cache of latents: what fills it (export
// kda_latent_cache_store) and what reads it back (export
// kda_latent_cache_load).
//
// A page holds page_size successive tokens of one sequence: the latents' codes
// [page_size][512] in e4m3, an exponent for each 128 of them [page_size][4], and the
// shared key parts [page_size][64] in bfloat16.  A value is code x 2^(exponent -
// 127).  Every token has scales of its own, so that appending one leaves the others
// as they are; the shared part, an eighth of the values, is what positions are
// told by, and stays as it came.
#include "kda_host.h"
#include "latent_device.h"

namespace {

using namespace kda::latent;

constexpr int kWaves = 4;
constexpr int kLeast = -64, kMost = 119;   // exponents of a scale: 448 x 2^119 is the last that bfloat16 holds

struct Cache {
  uint8_t *codes, *exponents;
  uint16_t* shared;
  int64_t c_stride, scale_stride, s_stride;
  int page_size, shift, num_pages;
};

// ---------------------------------------------------------------- store

struct StoreParams {
  const uint16_t *c, *s;
  int64_t c_stride, s_stride;
  const int32_t* slots;
  int T;
  Cache cache;
};

// Larger of the finite magnitudes in eight bf16 values (bits).
__device__ __forceinline__ uint32_t finite_top(const u32x4 x) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = x[i] & 0x7fffu, hi = (x[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) top = max(top, lo);
    if (hi < 0x7f80u) top = max(top, hi);
  }
  return top;
}

// Finite values to at most 448 (above it only under the largest scale); infinities
// and NaN stay, and have the code of NaN.
__device__ __forceinline__ float fit(float x) {
  return __builtin_fabsf(x) < INFINITY ? __builtin_amdgcn_fmed3f(x, -448.0f, 448.0f) : x;
}

// A wave takes kTokens successive tokens, all their rows on the way at once: 64 lanes
// of 8 values are a latent, 16 lanes one block.  Bound by memory where there are many
// (75000 tokens, 135 MB, 28.1 us, 4.8 TB/s, the copy's rate; with 1, 4 and 8 tokens
// to a wave 29.2, 29.3 and 31.2), by the launch where there are few.
constexpr int kTokens = 2;
__global__ __launch_bounds__(64 * kWaves) void latent_cache_store_kernel(StoreParams p) {
  const int lane = threadIdx.x & 63;
  const int t0 = (int(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kTokens;
  const int n = min(p.T - t0, kTokens);
  if (n <= 0) return;
  int slot[kTokens];
  u32x4 x[kTokens], s;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = t0 + min(i, n - 1);
    slot[i] = i < n ? p.slots[t] : -1;
    x[i] = *reinterpret_cast<const u32x4*>(p.c + t * p.c_stride + 8 * lane);
  }
  const int row = min(lane >> 3, n - 1);                   // the shared parts: eight lanes a token
  if (lane < 8 * kTokens) s = *reinterpret_cast<const u32x4*>(p.s + (t0 + row) * p.s_stride + 8 * (lane & 7));
  int mine = -1;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    uint32_t top = finite_top(x[i]);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
    // least e with 448 x 2^e >= top, 448 = 1.75 x 2^8
    const int e = min(max(int(top >> 7) - 127 - 8 + int((top & 127) > 96), kLeast), kMost);
    const float f = __uint_as_float(uint32_t(127 - e) << 23);
    u32x2 codes;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int w = 0;
      w = __builtin_amdgcn_cvt_pk_fp8_f32(fit(kda::bf16lo(x[i][2 * j]) * f), fit(kda::bf16hi(x[i][2 * j]) * f), w,
                                          false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(fit(kda::bf16lo(x[i][2 * j + 1]) * f),
                                          fit(kda::bf16hi(x[i][2 * j + 1]) * f), w, true);
      codes[j] = uint32_t(w);
    }
    if (slot[i] < 0 || (slot[i] >> p.cache.shift) >= p.cache.num_pages) continue;
    if ((lane >> 3) == i) mine = slot[i];
    const int64_t page = slot[i] >> p.cache.shift;
    const int off = slot[i] & (p.cache.page_size - 1);
    *reinterpret_cast<u32x2*>(p.cache.codes + page * p.cache.c_stride + off * R + 8 * lane) = codes;
    if ((lane & 15) == 0)
      p.cache.exponents[page * p.cache.scale_stride + off * kBlocks + (lane >> 4)] = uint8_t(127 + e);
  }
  if (mine >= 0) {
    const int64_t page = mine >> p.cache.shift;
    const int off = mine & (p.cache.page_size - 1);
    *reinterpret_cast<u32x4*>(p.cache.shared + page * p.cache.s_stride + off * S + 8 * (lane & 7)) = s;
  }
}

// ---------------------------------------------------------------- load

struct LoadParams {
  Cache cache;
  const int32_t* table;
  int64_t table_stride;
  int width, N, T;
  const int32_t* cu;
  uint16_t *c, *s;
};

// A wave takes kRun successive rows of the output; lane i < kRun finds out where
// row i comes from.  Bound by memory (131000 tokens, 236 MB: 43 us, 5.4 TB/s, into
// outputs that the caches hold, 53 into others).
constexpr int kRun = 8;
__global__ __launch_bounds__(64 * kWaves) void latent_cache_load_kernel(LoadParams p) {
  const int lane = threadIdx.x & 63;
  const int t0 = (int(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kRun;
  if (t0 >= p.T) return;
  int from = -2;                           // slot; -1: a token without a page, zeros; -2: none, left as it is
  {
    const int t = t0 + (lane & (kRun - 1));
    int lo = 0, hi = p.N;                  // the last n with cu[n] <= t, if the first has
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int at = p.cu[lo];
    if (t < p.T && at <= t && t < p.cu[lo + 1]) {
      const int64_t pos = int64_t(t) - at;
      const int64_t col = pos >> p.cache.shift;
      const int id = col < p.width ? p.table[lo * p.table_stride + col] : -1;
      from = id >= 0 && id < p.cache.num_pages ? (id << p.cache.shift) + int(pos & (p.cache.page_size - 1)) : -1;
    }
  }
  u32x2 codes[kRun];
  uint32_t exponent[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int slot = __builtin_amdgcn_readlane(from, i);
    const int64_t page = max(slot, 0) >> p.cache.shift;
    const int off = max(slot, 0) & (p.cache.page_size - 1);
    codes[i] = (u32x2){0, 0};
    exponent[i] = 127;
    if (slot >= 0) {
      codes[i] = *reinterpret_cast<const u32x2*>(p.cache.codes + page * p.cache.c_stride + off * R + 8 * lane);
      exponent[i] = p.cache.exponents[page * p.cache.scale_stride + off * kBlocks + (lane >> 4)];
    }
  }
  const int own = __shfl(from, lane >> 3, 64);             // the shared parts: eight lanes a token
  u32x4 s = (u32x4)(0u);
  if (own >= 0)
    s = *reinterpret_cast<const u32x4*>(p.cache.shared + int64_t(own >> p.cache.shift) * p.cache.s_stride +
                                        (own & (p.cache.page_size - 1)) * S + 8 * (lane & 7));
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    if (__builtin_amdgcn_readlane(from, i) < -1) continue;
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const float f = __uint_as_float(exponent[i] << 23);
    u32x4 y;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i][j], f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i][j], f, true);
      y[2 * j] = __builtin_bit_cast(uint32_t, lo);
      y[2 * j + 1] = __builtin_bit_cast(uint32_t, hi);
    }
    *reinterpret_cast<u32x4*>(p.c + int64_t(t0 + i) * R + 8 * lane) = y;
  }
  if (own >= -1) *reinterpret_cast<u32x4*>(p.s + int64_t(t0 + (lane >> 3)) * S + 8 * (lane & 7)) = s;
}

Cache as_cache(void* c, void* scale, void* s, const kda::LatentCache& x) {
  return Cache{static_cast<uint8_t*>(c), static_cast<uint8_t*>(scale), static_cast<uint16_t*>(s), x.c_stride,
               x.scale_stride, x.s_stride, x.page_size, __builtin_ctz(x.page_size), x.num_pages};
}

}  // namespace

extern "C" int kda_latent_cache_store(const void* c, const void* k_shared, int64_t c_stride, int64_t s_stride,
                                      const int32_t* slots, int32_t T, void* c_cache, void* c_scale, void* k_cache,
                                      int32_t page_size, int64_t c_page, int64_t scale_page, int64_t k_page,
                                      int32_t num_pages, void* stream) {
  const kda::LatentCache x{page_size, num_pages, c_page, scale_page, k_page};
  int e = kda::latent_cache(x);
  if (e == KDA_OK) e = kda::latent_stride(c_stride, R);
  if (e == KDA_OK) e = kda::latent_stride(s_stride, S);
  if (e == KDA_OK && T < 0) e = KDA_ERR_SHAPE;
  if (e != KDA_OK) return e;
  const int64_t most = int64_t(kda::kMostBlocks) * kWaves * kTokens;
  if (T > most) return KDA_ERR_SHAPE;
  if (T == 0 || num_pages == 0) return KDA_OK;
  if (!c || !k_shared || !slots || !c_cache || !c_scale || !k_cache) return KDA_ERR_NULL;
  for (const void* y : {c, k_shared, static_cast<const void*>(c_cache), static_cast<const void*>(k_cache)})
    if (!kda::aligned16(y)) return KDA_ERR_ALIGN;
  if (!kda::aligned4(c_scale) || !kda::aligned4(slots)) return KDA_ERR_ALIGN;
  const StoreParams p{static_cast<const uint16_t*>(c), static_cast<const uint16_t*>(k_shared), c_stride, s_stride,
                      slots, T, as_cache(c_cache, c_scale, k_cache, x)};
  const unsigned blocks = unsigned((int64_t(T) + kWaves * kTokens - 1) / (kWaves * kTokens));
  hipLaunchKernelGGL(latent_cache_store_kernel, dim3(blocks), dim3(64 * kWaves), 0, kda::as_stream(stream), p);
  return kda::launch_status();
}

extern "C" int kda_latent_cache_load(const void* c_cache, const void* c_scale, const void* k_cache,
                                     int32_t page_size, int64_t c_page, int64_t scale_page, int64_t k_page,
                                     int32_t num_pages, const int32_t* page_table, int64_t table_stride,
                                     int32_t table_width, const int32_t* cu_seqlens, int32_t num_seqs,
                                     int32_t num_tokens, void* c, void* k_shared, void* stream) {
  const kda::LatentCache x{page_size, num_pages, c_page, scale_page, k_page};
  const int e = kda::latent_cache(x);
  if (e != KDA_OK) return e;
  if (num_pages < 1 || num_seqs < 1 || num_tokens < 0 || table_width < 1 || table_stride < table_width)
    return KDA_ERR_SHAPE;
  if (num_tokens == 0) return KDA_OK;
  if (!c_cache || !c_scale || !k_cache || !page_table || !cu_seqlens || !c || !k_shared) return KDA_ERR_NULL;
  for (const void* y : {c_cache, k_cache, static_cast<const void*>(c), static_cast<const void*>(k_shared)})
    if (!kda::aligned16(y)) return KDA_ERR_ALIGN;
  if (!kda::aligned4(c_scale) || !kda::aligned4(page_table) || !kda::aligned4(cu_seqlens)) return KDA_ERR_ALIGN;
  const LoadParams p{as_cache(const_cast<void*>(c_cache), const_cast<void*>(c_scale), const_cast<void*>(k_cache), x),
                     page_table, table_stride, table_width, num_seqs, num_tokens, cu_seqlens,
                     static_cast<uint16_t*>(c), static_cast<uint16_t*>(k_shared)};
  const int64_t blocks = (int64_t(num_tokens) + kWaves * kRun - 1) / (kWaves * kRun);
  if (blocks > kda::kMostBlocks) return KDA_ERR_SHAPE;
  hipLaunchKernelGGL(latent_cache_load_kernel, dim3(unsigned(blocks)), dim3(64 * kWaves), 0, kda::as_stream(stream),
                     p);
  return kda::launch_status();
}
