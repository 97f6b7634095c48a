// Writing and reading the paged Q4_0 cache of keys and values.
//
// A workgroup takes one granule (sixteen positions) of one sequence and kv head,
// keys and values.  Grids are sized from the numbers of rows and sequences alone
// (granule_places); what a place holds is found on the device.
#include "q4_cache.hpp"
#include "q4_quantize_block.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;

// Four consecutive elements, as fp32 (exact).
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&v)[4]) {
  const float4_t t = *reinterpret_cast<const float4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = t[i];
}
template <>
__device__ __forceinline__ void load4<half_t>(const half_t* p, float (&v)[4]) {
  const half4_t t = *reinterpret_cast<const half4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(t[i]);
}
template <>
__device__ __forceinline__ void load4<bf16_t>(const bf16_t* p, float (&v)[4]) {
  const uint2 t = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_bits_to_float(t.x & 0xFFFFu);
  v[1] = bf16_bits_to_float(t.x >> 16);
  v[2] = bf16_bits_to_float(t.y & 0xFFFFu);
  v[3] = bf16_bits_to_float(t.y >> 16);
}

// Finite, of at most fp16's largest magnitude: NaN counts as 0.
__device__ __forceinline__ float storable(float v) {
  return v != v ? 0.f : fminf(fmaxf(v, -65504.f), 65504.f);
}

// What a workgroup of the granule grid takes: positions [from, to) of granule g of
// sequence s, the rows from `row` on.  False: nothing.
struct Granule {
  int s, g, from, to, row;
};
__device__ __forceinline__ bool granule_of(const Batch& b, int64_t place, Granule* out) {
  const int s = b.offsets == nullptr
                    ? static_cast<int>(place)
                    : last_not_above(b.seqs, place, [&](int i) { return granule_place(b, i); });
  const Seq q = seq_of(b, s);
  const int first = q.first < 0 ? 0 : q.first;  // the first position with a row
  const int64_t g = first / kGranule + (b.offsets == nullptr ? 0 : place - granule_place(b, s));
  if (q.rows == 0 || g * kGranule >= q.length) return false;
  out->s = s;
  out->g = static_cast<int>(g);
  const int base = out->g * kGranule;
  out->from = first > base ? first - base : 0;
  out->to = q.length - base < kGranule ? q.length - base : kGranule;
  out->row = q.row + base + out->from - q.first;
  return out->from < out->to;
}

// Eight lanes to a block of 32 values.  Keys' code bytes leave as words of a
// position, values' as single bytes, sixteen positions apart.
template <typename T>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(Cache c, Batch b, const T* __restrict__ k,
                                                               int64_t k_stride, const T* __restrict__ v,
                                                               int64_t v_stride) {
  const int64_t place = blockIdx.x / c.kv_heads;
  const int h = static_cast<int>(blockIdx.x - place * c.kv_heads);
  Granule gr;
  if (!granule_of(b, place, &gr)) return;
  uint8_t* const keys = granule_at(c, b, gr.s, gr.g, h);
  if (keys == nullptr) return;
  uint8_t* const values = keys + static_cast<int64_t>(c.per_page) * (9 * c.dim);
  const int nb = c.dim / kQK, part = threadIdx.x & 7;
  const int n = gr.to - gr.from, tasks = 2 * n * nb;
  for (int t = threadIdx.x >> 3; t < tasks; t += kThreads / 8) {
    const bool value = t >= n * nb;
    const int u = value ? t - n * nb : t;
    const int i = u / nb, blk = u - i * nb, at = gr.from + i;
    const int64_t row = gr.row + i;
    float x[4];
    load4(value ? v + row * v_stride + h * c.dim + blk * kQK + part * 4
                : k + row * k_stride + h * c.dim + blk * kQK + part * 4, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = storable(x[e]);
    uint32_t bytes;
    const half_t d = quantize_lanes(part, x, &bytes);
    const uint16_t bits = __builtin_bit_cast(uint16_t, d);
    if (value) {
      if (part < 4) {
        uint8_t* p = values + (blk * 16 + part * 4) * 16 + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[16 * e] = static_cast<uint8_t>(bytes >> (8 * e));
      }
      const int quarter = at & 3, place4 = (quarter & 1) * 2 + (quarter >> 1);
      if (part == 0)
        reinterpret_cast<uint16_t*>(values + 8 * c.dim)[blk * 16 + (at & ~3) + place4] = bits;
    } else {
      if (part < 4) *reinterpret_cast<uint32_t*>(keys + at * (c.dim / 2) + (part * nb + blk) * 4) = bytes;
      if (part == 0) reinterpret_cast<uint16_t*>(keys + 8 * c.dim)[((at >> 2) * nb + blk) * 4 + (at & 3)] = bits;
    }
  }
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ half_t narrow<half_t>(float v) { return static_cast<half_t>(v); }
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float v) {
  return bf16_t{__builtin_bit_cast(uint16_t, static_cast<__bf16>(v))};
}

// One value of a granule in LDS.
__device__ __forceinline__ float decoded(const uint8_t* g, bool value, int nb, int at, int e) {
  const int blk = e / kQK, i = e & 15, high = (e >> 4) & 1;
  const int quarter = at & 3;
  const int code_at = value ? (blk * 16 + i) * 16 + at : at * nb * 16 + ((i >> 2) * nb + blk) * 4 + (i & 3);
  const int scale_at = value ? blk * 16 + (at & ~3) + (quarter & 1) * 2 + (quarter >> 1)
                             : ((at >> 2) * nb + blk) * 4 + quarter;
  const int code = (g[code_at] >> (4 * high)) & 15;
  const float d = half_bits_to_float(reinterpret_cast<const uint16_t*>(g + nb * 256)[scale_at]);
  return static_cast<float>(code - 8) * d;
}

// A granule's bytes go through LDS; a thread gives eight values of a row at a time.
template <typename T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(Cache c, Batch b, T* __restrict__ k,
                                                              T* __restrict__ v) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][9 * 256];
  const int64_t place = blockIdx.x / c.kv_heads;
  const int h = static_cast<int>(blockIdx.x - place * c.kv_heads);
  Granule gr;
  if (!granule_of(b, place, &gr)) return;
  const uint8_t* const keys = granule_at(c, b, gr.s, gr.g, h);
  const int nb = c.dim / kQK, pieces = 9 * c.dim / 16;
  if (keys != nullptr) {
    const uint8_t* const values = keys + static_cast<int64_t>(c.per_page) * (9 * c.dim);
    for (int i = threadIdx.x; i < 2 * pieces; i += kThreads) {
      const int w = i >= pieces, j = i - w * pieces;
      *reinterpret_cast<uint4*>(lds[w] + 16 * j) = *reinterpret_cast<const uint4*>((w ? values : keys) + 16 * j);
    }
  }
  __syncthreads();
  const int n = gr.to - gr.from, per_row = c.dim / 8;
  const int64_t row_elems = static_cast<int64_t>(c.kv_heads) * c.dim;
  for (int t = threadIdx.x; t < 2 * n * per_row; t += kThreads) {
    const bool value = t >= n * per_row;
    const int u = value ? t - n * per_row : t;
    const int i = u / per_row, e = (u - i * per_row) * 8;
    T out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      out[j] = narrow<T>(keys == nullptr ? 0.f : decoded(lds[value], value, nb, gr.from + i, e + j));
    T* const p = (value ? v : k) + (gr.row + i) * row_elems + h * c.dim + e;
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = out[j];
  }
}

// Rows of a sequence whose position is negative (fewer positions than rows).
template <typename T>
__global__ __launch_bounds__(kThreads) void cache_read_none_kernel(Batch b, int64_t row_elems, T* __restrict__ k,
                                                                   T* __restrict__ v) {
  for (int s = blockIdx.x; s < b.seqs; s += gridDim.x) {
    const Seq q = seq_of(b, s);
    const int64_t n = q.first < 0 ? (-q.first < q.rows ? -q.first : q.rows) * row_elems : 0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads)
      k[q.row * row_elems + i] = v[q.row * row_elems + i] = narrow<T>(0.f);
  }
}

template <typename T>
hipError_t write_as(const Cache& c, const Batch& b, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, Queue q) {
  Cache ca = c;
  Batch ba = b;
  const T *kp = static_cast<const T*>(k), *vp = static_cast<const T*>(v);
  void* argv[] = {&ca, &ba, &kp, &k_stride, &vp, &v_stride};
  return launch_blocks(reinterpret_cast<const void*>(&cache_write_kernel<T>), granule_places(b) * c.kv_heads,
                       kThreads, argv, 0, q);
}

template <typename T>
hipError_t read_as(const Cache& c, const Batch& b, void* k, void* v, Queue q) {
  Cache ca = c;
  Batch ba = b;
  T *kp = static_cast<T*>(k), *vp = static_cast<T*>(v);
  void* argv[] = {&ca, &ba, &kp, &vp};
  const hipError_t e = launch_blocks(reinterpret_cast<const void*>(&cache_read_kernel<T>),
                                     granule_places(b) * c.kv_heads, kThreads, argv, 0, q);
  if (e != hipSuccess) return e;
  int64_t row_elems = static_cast<int64_t>(c.kv_heads) * c.dim;
  void* none[] = {&ba, &row_elems, &kp, &vp};
  return launch_blocks(reinterpret_cast<const void*>(&cache_read_none_kernel<T>), b.seqs < 1024 ? b.seqs : 1024,
                       kThreads, none, 0, q);
}

}  // namespace

hipError_t launch_cache_write(const Cache& c, const Batch& b, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, DType dt, Queue q) {
  if (dt == DType::F32) return write_as<float>(c, b, k, k_stride, v, v_stride, q);
  if (dt == DType::F16) return write_as<half_t>(c, b, k, k_stride, v, v_stride, q);
  return write_as<bf16_t>(c, b, k, k_stride, v, v_stride, q);
}

hipError_t launch_cache_read(const Cache& c, const Batch& b, void* k, void* v, DType dt, Queue q) {
  if (dt == DType::F32) return read_as<float>(c, b, k, v, q);
  if (dt == DType::F16) return read_as<half_t>(c, b, k, v, q);
  return read_as<bf16_t>(c, b, k, v, q);
}

}  // namespace q4
