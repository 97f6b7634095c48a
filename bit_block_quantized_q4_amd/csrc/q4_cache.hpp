// Shared by the kernels of the paged Q4_0 cache and of the attention over it
// (gfx950).  Internal header; the layout is stated in the public one.
#pragma once

#include "q4_fused.hpp"

namespace q4 {

constexpr int kGranule = 16;  // positions per granule

// A cache and a batch as kernels take them, by value.
struct Cache {
  uint8_t* data = nullptr;
  int pages = 0;
  int per_page = 0;      // granules per page
  uint32_t inverse = 0;  // floor(2^32 / per_page), 2^32 - 1 for one
  int kv_heads = 0;
  int dim = 0;
  int64_t page_bytes = 0;
  int64_t head_bytes = 0;  // keys and values of a kv head's page
};

struct Batch {
  const int* tables = nullptr;
  const int* lengths = nullptr;
  const int* offsets = nullptr;  // null: one row each
  int seqs = 0, tokens = 0, max_pages = 0;
  int max_length = 0;  // max_pages page_size
};

// A sequence: its first row, its rows, its positions and its first row's position.
struct Seq {
  int row, rows, length, first;
};

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ int offset_of(const Batch& b, int s) {
  return b.offsets == nullptr ? s : clamp_int(b.offsets[s], 0, b.tokens);
}

__device__ __forceinline__ Seq seq_of(const Batch& b, int s) {
  Seq q;
  q.row = offset_of(b, s);
  const int end = offset_of(b, s + 1);
  q.rows = end > q.row ? end - q.row : 0;
  q.length = clamp_int(b.lengths[s], 0, b.max_length);
  q.first = q.length - q.rows;
  return q;
}

// The last s of 0 .. count - 1 whose f(s), which does not fall, is at most key (0 if
// none is).  A wavefront takes it together: each round 64 candidates.
template <typename F>
__device__ __forceinline__ int last_not_above(int count, int64_t key, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = count;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave;
    const bool below = static_cast<int64_t>(lane) * step < n && f(lo + lane * step) <= key;
    const uint64_t mask = __ballot(below);
    const int k = mask == 0 ? 0 : 63 - __builtin_clzll(mask);
    lo += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The sequences' granules that hold their rows, as places of a grid: sequence s has
// the places from granule_place(s) on.  n rows lie in at most n / 16 + 2 granules, so
// no two sequences' places meet, and a place behind a sequence's last granule is idle.
__device__ __forceinline__ int64_t granule_place(const Batch& b, int s) {
  return static_cast<int64_t>(offset_of(b, s) / kGranule) + 2 * static_cast<int64_t>(s);
}
inline int64_t granule_places(const Batch& b) {
  return b.offsets == nullptr ? b.seqs : b.tokens / kGranule + 2 * static_cast<int64_t>(b.seqs);
}

// Granule g of a sequence (positions 16 g on): its bytes of kv head h's keys, or null
// where no page is named.  The values' lie per_page 9 dim bytes on.
__device__ __forceinline__ uint8_t* granule_at(const Cache& c, const Batch& b, int s, int g, int h) {
  const uint32_t u = static_cast<uint32_t>(g), per = static_cast<uint32_t>(c.per_page);
  uint32_t slot = __umulhi(u, c.inverse);  // g / per_page, or one less
  uint32_t in = u - slot * per;
  if (in >= per) {
    ++slot;
    in -= per;
  }
  if (slot >= static_cast<uint32_t>(b.max_pages)) return nullptr;
  const int id = b.tables[static_cast<int64_t>(s) * b.max_pages + slot];
  if (id < 0 || id >= c.pages) return nullptr;
  return c.data + id * c.page_bytes + h * c.head_bytes + static_cast<int64_t>(in) * (9 * c.dim);
}

inline Cache make_cache(void* data, int64_t pages, int64_t page_size, int64_t kv_heads, int64_t dim) {
  Cache c;
  c.data = static_cast<uint8_t*>(data);
  c.pages = static_cast<int>(pages);
  c.per_page = static_cast<int>(page_size / kGranule);
  c.inverse = c.per_page == 1 ? 0xFFFFFFFFu
                              : static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint32_t>(c.per_page));
  c.kv_heads = static_cast<int>(kv_heads);
  c.dim = static_cast<int>(dim);
  c.head_bytes = 2 * c.per_page * 9 * dim;
  c.page_bytes = kv_heads * c.head_bytes;
  return c;
}

struct Attention {
  Cache cache;
  Batch batch;
  const void* q = nullptr;
  int64_t q_stride = 0;
  DType qt = DType::F16;
  int heads = 0;
  int group = 0;  // heads per kv head
  float scale = 0.f, softcap = 0.f;
  int causal = 1;
  int window = 0;  // 0: none
  void* y = nullptr;
  int y_dt = 0;
  float* lse = nullptr;
};

// The positions lo .. hi - 1 that a row at position p of a sequence sees.
__device__ __forceinline__ void seen_by(const Attention& a, int length, int p, int* lo, int* hi) {
  *hi = a.causal && p + 1 < length ? p + 1 : length;
  if (*hi < 0) *hi = 0;
  *lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  if (*lo > *hi) *lo = *hi;
}

hipError_t launch_cache_write(const Cache& c, const Batch& b, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, DType dt, Queue q);
hipError_t launch_cache_read(const Cache& c, const Batch& b, void* k, void* v, DType dt, Queue q);

size_t attention_workspace_bytes(const Attention& a);
hipError_t launch_attention(const Attention& a, void* workspace, Queue q);

}  // namespace q4
