// The paged 8-bit cache of the full-attention layers: what fills it (export
// kda_attn_cache_store) and the tables that say where (export
// kda_attn_tables).
//
// A page holds page_size successive tokens of one sequence, for every
// key/value head [page_size][128] codes in e4m3 and one float32 scale; keys
// and values apart.  A value is code x scale.  Scales made here are powers of
// two: e4m3 codes have the same relative step at every power of two, so a
// finer scale would buy nothing, and a page whose scale has to grow when a
// larger token is appended only shifts the exponents of what it holds (exact
// but for codes that fall below e4m3's normal range).
#include "attn_device.h"
#include "kda_host.h"

namespace {

using namespace kda::attn;

// ---------------------------------------------------------------- store

constexpr int kStoreWaves = 4;
constexpr int kLeast = -64;        // smallest exponent of a scale

struct StoreParams {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  int T, HKV, page_size, shift, wshift;
  unsigned items, waves;
  int64_t num_slots, page_stride;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
};

// Larger of the finite magnitudes in eight bf16 values and `top` (bits).
__device__ __forceinline__ uint32_t finite_top(const u32x4 x, uint32_t top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = x[i] & 0x7fffu, hi = (x[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) top = max(top, lo);
    if (hi < 0x7f80u) top = max(top, hi);
  }
  return top;
}

// Two words of codes from eight values, each rounded to nearest even once;
// infinities and NaN become NaN.
__device__ __forceinline__ u32x2 to_codes(const u32x4 x, float f) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(kda::bf16lo(x[2 * i]) * f, kda::bf16hi(x[2 * i]) * f, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(kda::bf16lo(x[2 * i + 1]) * f, kda::bf16hi(x[2 * i + 1]) * f, w, true);
    r[i] = uint32_t(w);
  }
  return r;
}

// Four codes times f, rounded again.
__device__ __forceinline__ uint32_t rescale(uint32_t w, float f) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_cvt_f32_fp8(int(w), 0) * f,
                                      __builtin_amdgcn_cvt_f32_fp8(int(w), 1) * f, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_cvt_f32_fp8(int(w), 2) * f,
                                      __builtin_amdgcn_cvt_f32_fp8(int(w), 3) * f, r, true);
  return uint32_t(r);
}

// Rows of a run as a buffer that ends behind the last one: rows past it read as
// zero and are not written, so a wave handles groups of four rows without a branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t as_buffer(const void* at, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, int(bytes), 0x00020000);
}

// One wave stores `n` tokens of one head, keys or values, the first of them at
// offset `off` of a page.  rows: the first token's row; page: the (page, head)'s
// codes.  GROUPS x 4 tokens are read once and kept in registers between the
// maximum and the codes; what is over (pages of 128 and 256) is read twice.
template <int GROUPS>
__device__ __forceinline__ void store_run(const uint16_t* rows, int64_t stride, int n, uint8_t* page, int off,
                                          float* scale, int lane) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const int row = lane >> 4, at = (lane & 15) * 8, here = min(n, 4 * GROUPS);
  const auto src = as_buffer(rows, ((here - 1) * stride + D) * 2);
  const float was = off ? *scale : 0.0f;
  u32x4 kept[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; ++i)
    kept[i] = __builtin_amdgcn_raw_buffer_load_b128(src, int((4 * i + row) * stride + at) * 2, 0, 0);
  u16x2 most = {0, 0};
#pragma unroll
  for (int i = 0; i < GROUPS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, kept[i][j] & 0x7fff7fffu));
  uint32_t top = max(most[0], most[1]);
  if (__any(top >= 0x7f80u)) {                 // an infinity or NaN: only finite values count
    top = 0;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) top = finite_top(kept[i], top);
  }
#pragma unroll 4
  for (int i = 4 * GROUPS + row; i < n; i += 4)
    top = finite_top(*reinterpret_cast<const u32x4*>(rows + i * stride + at), top);
#pragma unroll
  for (int i = 1; i < 64; i *= 2) top = max(top, uint32_t(__shfl_xor(int(top), i, 64)));
  // least e with 448 x 2^e >= top, 448 = 1.75 x 2^8
  const int e = max(int(top >> 7) - 127 - 8 + int((top & 127) > 96), kLeast);
  const float fits = __uint_as_float(uint32_t(127 + e) << 23);
  const float now = fmaxf(was, fits);
  if (off && now != was) {                     // the page's earlier tokens take the new scale
    const float f = was / now;
    const int pieces = off * (D / 16);         // 16 codes each
    for (int i = lane; i < pieces; i += 64) {
      u32x4* p = reinterpret_cast<u32x4*>(page) + i;
      u32x4 w = *p;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = rescale(w[j], f);
      *p = w;
    }
  }
  if (lane == 0) *scale = now;
  const float f = 1.0f / now;
  const auto dst = as_buffer(page + off * D, here * D);
#pragma unroll
  for (int i = 0; i < GROUPS; ++i)
    __builtin_amdgcn_raw_buffer_store_b64(to_codes(kept[i], f), dst, (4 * i + row) * D + at, 0, 0);
#pragma unroll 4
  for (int i = 4 * GROUPS + row; i < n; i += 4)
    *reinterpret_cast<u32x2*>(page + (off + i) * D + at) =
        to_codes(*reinterpret_cast<const u32x4*>(rows + i * stride + at), f);
}

// A run is a stretch of tokens whose slots follow one another within a page.
// One wave takes the keys or the values of one run of one head, so a page's
// scale has one writer.  An item is (window of 2^wshift tokens, head, keys or
// values): the wave looks there for the runs that begin.  Waves go from item to
// item, the next one's slots already on their way.
// Memory bounds it where there is much to store: 35000 tokens x 8 heads, 215 MB,
// take 36 us (6 TB/s, keys and values fresh in the last cache level), 54 of
// prompts over three caches in turn, which no cache level holds.  256 single
// tokens x 8 heads take 5 us, the latency of slots, rows, scale and codes one
// after another.  With a branch for each four rows, and loads that waited for
// them, one page took 13 us instead of 5.
__global__ __launch_bounds__(64 * kStoreWaves, 4) void attn_cache_store_kernel(StoreParams p) {
  const int lane = threadIdx.x & 63, window = 1 << p.wshift;
  const unsigned waves = p.waves;
  unsigned item = __builtin_amdgcn_readfirstlane(blockIdx.x * kStoreWaves + (threadIdx.x >> 6));
  if (item >= waves) return;
  auto slot_at = [&](int64_t t) -> int {       // -1: no such token, or not stored
    const int s = t >= 0 && t < p.T ? p.slots[t] : -1;
    return s >= 0 && s < p.num_slots ? s : -1;
  };
  auto begin_of = [&](unsigned i) { return int64_t(i / (2u * unsigned(p.HKV))) << p.wshift; };
  int mine = -1, before = -1;
  auto look = [&](unsigned i) {
    mine = before = -1;
    if (i < p.items && lane < window) mine = slot_at(begin_of(i) + lane), before = slot_at(begin_of(i) + lane - 1);
  };
  look(item);
  while (item < p.items) {
    const int64_t t0 = begin_of(item);
    const unsigned part = item % (2u * unsigned(p.HKV));
    const int head = int(part >> 1);
    const bool leads = mine >= 0 && ((mine & (p.page_size - 1)) == 0 || before < 0 || before != mine - 1);
    uint64_t runs = __ballot(leads);
    const int slots = mine;
    item = item + waves < item ? p.items : item + waves;
    look(item);
    while (runs) {
      const int i = __builtin_ctzll(runs);
      runs &= runs - 1;
      const int64_t t = t0 + i;
      const int slot = __builtin_amdgcn_readlane(slots, i);
      const int off = slot & (p.page_size - 1), most = p.page_size - off;
      int n = 0;
      for (bool whole = true; whole && n < most; ) {
        const uint64_t same = __ballot(n + lane < most && slot_at(t + n + lane) == slot + n + lane);
        whole = same == ~uint64_t(0);
        n += whole ? 64 : __builtin_ctzll(~same);
      }
      const int64_t page = slot >> p.shift;
      const bool v = part & 1;
      const int64_t stride = v ? p.v_stride : p.k_stride;
      const uint16_t* rows = (v ? p.v : p.k) + t * stride + head * D;
      uint8_t* codes = (v ? p.v_cache : p.k_cache) + page * p.page_stride + int64_t(head) * p.page_size * D;
      float* scale = (v ? p.v_scale : p.k_scale) + page * p.HKV + head;
      if (n <= 4)
        store_run<1>(rows, stride, n, codes, off, scale, lane);
      else if (n <= 16)
        store_run<4>(rows, stride, n, codes, off, scale, lane);
      else
        store_run<16>(rows, stride, n, codes, off, scale, lane);
    }
  }
}

// ---------------------------------------------------------------- tables

constexpr int kTableThreads = 512;
constexpr int kMostRequests = 8192;
constexpr int kTokensPerBlock = 2048;

struct TableParams {
  const int32_t *cached, *fresh;
  int32_t* table;
  int64_t table_stride;
  int width, N, page_size, shift, tokens, num_free;
  const int32_t *free_pages, *free_head;
  int32_t *cu, *slots, *lens, *next_head;
};

// Every workgroup makes the two prefix sums (new tokens, new pages) over all
// requests for itself in LDS, then looks up its share of the tokens and of the
// new pages: one launch, no word passed between workgroups.  Latency bounds it:
// 256 requests of one token 4.2 us, 32 prompts of up to 8192 tokens 6.3 us.
__global__ __launch_bounds__(kTableThreads) void attn_tables_kernel(TableParams p) {
  __shared__ int32_t cu[kMostRequests + 1], pages[kMostRequests + 1];
  __shared__ int32_t wave_sums[2][kTableThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (p.N + kTableThreads - 1) / kTableThreads;

  auto old_len = [&](int n) { return max(p.cached[n], 0); };
  auto new_len = [&](int n) { return max(p.fresh[n], 0); };
  auto pages_of = [&](int64_t tokens) { return int(min((tokens + p.page_size - 1) >> p.shift, int64_t(p.width))); };

  int tok = 0, pg = 0;
  for (int i = 0; i < per; ++i) {
    const int n = tid * per + i;
    if (n >= p.N) break;
    const int64_t a = old_len(n), b = a + new_len(n);
    tok += int(b - a);
    pg += pages_of(b) - pages_of(a);
  }
  int tok_at = tok, pg_at = pg;                // inclusive sums over the wave, then over the workgroup
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(tok_at, d, 64), y = __shfl_up(pg_at, d, 64);
    if (lane >= d) tok_at += x, pg_at += y;
  }
  if (lane == 63) wave_sums[0][wave] = tok_at, wave_sums[1][wave] = pg_at;
  __syncthreads();
  tok_at -= tok, pg_at -= pg;
  for (int w = 0; w < wave; ++w) tok_at += wave_sums[0][w], pg_at += wave_sums[1][w];
  for (int i = 0; i < per; ++i) {
    const int n = tid * per + i;
    if (n >= p.N) break;
    const int64_t a = old_len(n), b = a + new_len(n);
    cu[n] = tok_at, pages[n] = pg_at;
    tok_at += int(b - a);
    pg_at += pages_of(b) - pages_of(a);
    if (n == p.N - 1) cu[p.N] = tok_at, pages[p.N] = pg_at;
  }
  __syncthreads();

  const int head = p.free_head ? max(*p.free_head, 0) : 0;
  const int total_tokens = cu[p.N], total_pages = pages[p.N];
  auto free_page = [&](int j) -> int {         // the j-th page that this call takes, -1 if there is none
    const int64_t at = int64_t(head) + j;
    return j >= 0 && at < p.num_free ? p.free_pages[at] : -1;
  };
  auto find = [&](const int32_t* sums, int x) {   // the request n with sums[n] <= x < sums[n + 1]
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };

  const int first = blockIdx.x * kTokensPerBlock, last = min(first + kTokensPerBlock, p.tokens);
  for (int t = first + tid; t < last; t += kTableThreads) {
    int slot = -1;
    if (t < total_tokens) {
      const int n = find(cu, t);
      const int64_t pos = int64_t(old_len(n)) + t - cu[n];
      const int64_t c = pos >> p.shift;
      if (c >= 0 && c < p.width) {
        const int held = pages_of(old_len(n));
        const int id = c < held ? p.table[n * p.table_stride + c] : free_page(pages[n] + int(c) - held);
        if (id >= 0 && id <= (0x7fffffff >> p.shift)) slot = int((uint32_t(id) << p.shift) + (pos & (p.page_size - 1)));
      }
    }
    p.slots[t] = slot;
  }
  const int threads = gridDim.x * kTableThreads, me = blockIdx.x * kTableThreads + tid;
  for (int j = me; j < total_pages; j += threads) {
    const int n = find(pages, j);
    const int c = pages_of(old_len(n)) + j - pages[n];
    if (c >= 0 && c < p.width) p.table[n * p.table_stride + c] = free_page(j);
  }
  for (int n = me; n <= p.N; n += threads) {
    p.cu[n] = cu[n];
    if (n < p.N) p.lens[n] = int(min(int64_t(old_len(n)) + new_len(n), int64_t(0x7fffffff)));
  }
  if (me == 0) *p.next_head = int(min(int64_t(head) + total_pages, int64_t(0x7fffffff)));
}

}  // namespace

extern "C" int kda_attn_cache_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                    const int32_t* slots, int32_t T, int32_t HKV, int32_t Dh, void* k_cache,
                                    void* v_cache, float* k_scale, float* v_scale, int32_t page_size,
                                    int64_t page_stride, int32_t num_pages, void* stream) {
  if (T < 0) return KDA_ERR_SHAPE;
  int e = kda::attn_heads(HKV, HKV, Dh);
  if (e == KDA_OK) e = kda::attn_stride(k_stride, HKV);
  if (e == KDA_OK) e = kda::attn_stride(v_stride, HKV);
  if (e == KDA_OK) e = kda::attn_cache(HKV, page_size, page_stride, num_pages);
  if (e != KDA_OK) return e;
  if (T == 0 || num_pages == 0) return KDA_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale) return KDA_ERR_NULL;
  for (const void* x : {k, v, static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
    if (!kda::aligned16(x)) return KDA_ERR_ALIGN;
  // Every run costs a wave its latency, every empty window a look.  A decode
  // step's tokens are a run each and want a window each; in prompts a run is a
  // page.  Windows grow until two items are left for a wave, up to 16 tokens.
  // From one item to its next a wave passes an odd number of windows: runs begin
  // a page apart, and an even step would give all of them to the same few waves
  // (one sequence of 35000 tokens x 8 heads: 58 us with 256 windows, 36 with 255).
  const int64_t each = 2 * int64_t(HKV), most = 16 * int64_t(kda::device_cus());
  const int64_t step = most / each < 3 ? 1 : (most / each - 1) | 1;
  int wshift = 0;
  while (wshift < 4 && (int64_t(T) >> wshift) * each > 2 * most) ++wshift;
  const int64_t items = ((int64_t(T) + (1 << wshift) - 1) >> wshift) * each;
  if (items > 0x7fffffff) return KDA_ERR_SHAPE;
  const int64_t waves = items < step * each ? items : step * each;
  const StoreParams p{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride, slots,
                      T, HKV, page_size, __builtin_ctz(page_size), wshift, unsigned(items), unsigned(waves),
                      int64_t(num_pages) * page_size, page_stride,
                      static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scale, v_scale};
  const int64_t blocks = (waves + kStoreWaves - 1) / kStoreWaves;
  hipLaunchKernelGGL(attn_cache_store_kernel, dim3(unsigned(blocks)), dim3(64 * kStoreWaves), 0,
                     kda::as_stream(stream), p);
  return kda::launch_status();
}

extern "C" int kda_attn_tables(const int32_t* cached_lens, const int32_t* new_lens, int32_t N, int32_t* page_table,
                               int64_t table_stride, int32_t table_width, const int32_t* free_pages,
                               int32_t num_free, const int32_t* free_head, int32_t page_size, int32_t num_tokens,
                               int32_t* cu_seqlens, int32_t* slots, int32_t* kv_lens, int32_t* next_head,
                               void* stream) {
  if (N < 1 || N > kMostRequests || table_width < 1 || table_stride < table_width || num_free < 0 || num_tokens < 0)
    return KDA_ERR_SHAPE;
  if (!kda::attn_page(page_size)) return KDA_ERR_UNSUPPORTED;
  if (!cached_lens || !new_lens || !page_table || !cu_seqlens || !kv_lens || !next_head || (num_tokens && !slots) ||
      (num_free && !free_pages))
    return KDA_ERR_NULL;
  // read by every workgroup, written by one
  if (kv_lens == cached_lens || kv_lens == new_lens || next_head == free_head) return KDA_ERR_SHAPE;
  const TableParams p{cached_lens, new_lens, page_table, table_stride, table_width, N, page_size,
                      __builtin_ctz(page_size), num_tokens, num_free, free_pages, free_head,
                      cu_seqlens, slots, kv_lens, next_head};
  const unsigned blocks = unsigned((int64_t(num_tokens) + kTokensPerBlock - 1) / kTokensPerBlock);
  hipLaunchKernelGGL(attn_tables_kernel, dim3(blocks ? blocks : 1), dim3(kTableThreads), 0, kda::as_stream(stream), p);
  return kda::launch_status();
}
