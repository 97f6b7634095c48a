// Shared by the fused linear layer, the expert products and the routing
// (gfx950).  Internal header.
#pragma once

#include "q4_device.hpp"

namespace q4 {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluErf = 3, kActSilu = 4 };

// What follows a product, and where its outputs go (see q4_epilogue in the
// public header).  Passed to kernels by value.
struct Epi {
  const void* bias = nullptr;  // [n], or [experts][n]
  const void* residual = nullptr;
  void* y = nullptr;
  int64_t ldy = 0;   // output columns
  int64_t half = 0;  // gated: the "up" row of output column c is weight row half + c; 0: no gate
  int bias_dt = 0, act = 0, y_dt = 0;
};

// Which rows of x a product takes.  recs == nullptr: one group, rows 0 .. m - 1
// of x and y.  Otherwise tile t is the plan's record t: {expert, first place,
// rows, 0} and then its pairs; pair p reads row p / xdiv of x and writes row p
// of y.
struct Rows {
  const int* recs = nullptr;
  const int* ntiles = nullptr;  // tiles in use (the grid is an upper bound)
  int rec_words = 0;
  int xdiv = 1;
  int64_t wstride = 0;  // packed bytes per expert
  int64_t nbias = 0;    // bias values per expert
};

// ------------------------------------------------------------------ plan
//
// Device layout of a plan in int32 words: offsets[experts + 1], order[pairs],
// pos[pairs] (the place of a pair in `order`, -1 without an expert), {ntiles,
// rows per tile, 0, 0}, and the tiles' records: {expert, first place, rows, 0}
// and `tile_rows` pairs (a product's workgroup finds all it needs to start in
// one place).  Every part starts at a multiple of four words.
struct PlanLayout {
  int64_t order, pos, head, tiles, words;
  int64_t max_tiles;
  int tile_rows, rec_words;
};

// Rows per tile of the expert products, by the mean number of rows per
// expert alone, so that one plan serves every product over it: 16 (one
// activation tile of the matrix-core decode kernel) up to 12 rows, 32 up to
// 40, then the 128-row tiles of the prefill kernel, and from 80 on the experts'
// own tile of 192 rows.  Tiles of 16 and 32 rows multiply exact codes, the higher
// ones weights rounded to fp16.  Experts chosen evenly, gated, fp16, us with tiles
// of 16 / 32 / 128 / 192 rows, device time of the product:
//   mean          10               14               24               40
//   128 x 4096 x 2048   240/242/-/-   235/250/387/-   323/274/369/273   380/459/383/284
//   32 x 4096 x 4096    83/102/-/-    95/105/176/-    144/118/178/132   196/191/180/138
//   mean          64               80               96               128
//   128 x 4096 x 2048   -/605/401/338  -/730/411/378  -/856/408/388  -/1080/579/447
//   32 x 4096 x 4096    -/252/188/165  -/294/189/177  -/340/196/178  -/428/283/211
// The borders are older than this table: 192 rows take less time than 128 at every
// mean of it, and than 32 from about 24 to 32 on.
constexpr int kGroupRows = 192;

inline int expert_tile_rows(int64_t m, int64_t topk, int64_t experts) {
  const double mean = static_cast<double>(m) * static_cast<double>(topk) / static_cast<double>(experts);
  return mean <= 12.0 || m <= 16 ? 16 : mean <= 40.0 || m <= 32 ? 32 : mean <= 80.0 ? 128 : kGroupRows;
}

inline PlanLayout plan_layout(int64_t m, int64_t topk, int64_t experts) {
  PlanLayout p;
  const int64_t pairs = m * topk;
  auto up4 = [](int64_t v) { return (v + 3) / 4 * 4; };
  p.tile_rows = expert_tile_rows(m, topk, experts);
  // whole tiles, plus one partial tile for every expert that has rows
  p.max_tiles = pairs / p.tile_rows + (pairs < experts ? pairs : experts);
  p.order = up4(experts + 1);
  p.pos = p.order + up4(pairs);
  p.head = p.pos + up4(pairs);
  p.tiles = p.head + 4;
  p.rec_words = 4 + p.tile_rows;
  p.words = p.tiles + p.rec_words * p.max_tiles;
  return p;
}

// ------------------------------------------------------------------ values

// Element i of a dtype-coded array, as fp32 (exact).
__device__ __forceinline__ float load_f32(const void* p, int dt, int64_t i) {
  if (dt == static_cast<int>(DType::F32)) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return dt == static_cast<int>(DType::F16) ? half_bits_to_float(b) : bf16_bits_to_float(b);
}

// fp32 -> 16 bits, to nearest even.
__device__ __forceinline__ uint16_t f32_to_16(float v, int dt) {
  if (dt == static_cast<int>(DType::F16)) return __builtin_bit_cast(uint16_t, static_cast<half_t>(v));
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

__device__ __forceinline__ void store_as(void* p, int dt, int64_t i, float v) {
  if (dt == static_cast<int>(DType::F32)) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = f32_to_16(v, dt);
}

// Staging a bf16 row as fp16: the largest magnitude (as bf16 bits) so far, the
// power of two that brings it to [2^15, 2^16) (at most 2^126; none for rows of
// zeros), and two values times that power, rounded to nearest even.  A row with
// an infinity or NaN takes 2^-112, which brings every finite value into fp16:
// its outputs are infinite or NaN by that element alone.
__device__ __forceinline__ uint32_t max_magnitude_bf16(uint32_t top, uint32_t v) {
  const uint32_t lo = v & 0x7FFFu, hi = (v >> 16) & 0x7FFFu;
  const uint32_t b = lo > hi ? lo : hi;
  return b > top ? b : top;
}
__device__ __forceinline__ int bf16_row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 7);  // top = 1.f 2^(e - 127)
  const int shift = e == 0xFF ? -112 : top == 0 ? 0 : 142 - e;
  return shift > 126 ? 126 : shift;
}
__device__ __forceinline__ float power_of_two(int s) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(127 + s) << 23);
}
__device__ __forceinline__ uint32_t bf16x2_scaled_to_f16x2(uint32_t v, float f) {
  const half2_t h = {static_cast<half_t>(bf16_bits_to_float(v & 0xFFFFu) * f),
                     static_cast<half_t>(__builtin_bit_cast(float, v & 0xFFFF0000u) * f)};
  return __builtin_bit_cast(uint32_t, h);
}

// dma16_sbase (NT: the non-temporal one) with five wait states in place of the
// scalar move (see dma16): the form for kernels whose scalar registers spill.  (A
// build without either read a spilled address too early, and faulted.)
template <bool NT>
__device__ __forceinline__ void copy16(uint32_t voff, const void* sbase, uint32_t lds) {
  if constexpr (NT)
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
  else
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
}

// silu and the tanh form of gelu as z / (1 + exp(-t)): no cancellation for
// negative z, and 0 (not NaN) where exp overflows.
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f || z != z ? z : 0.f;
    case kActSilu: return z / (1.f + expf(-z));
    case kActGelu: return z / (1.f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    case kActGeluErf: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    default: return z;
  }
}

// Output column c of one row from its weight row sums (z1: the "up" row's,
// read with a gate only), without the residual.  e: expert (0 without).
__device__ __forceinline__ float finish(const Epi& ep, int64_t boff, int64_t c, float z0, float z1) {
  if (ep.bias != nullptr) {
    z0 += load_f32(ep.bias, ep.bias_dt, boff + c);
    if (ep.half != 0) z1 += load_f32(ep.bias, ep.bias_dt, boff + ep.half + c);
  }
  const float a = activate(z0, ep.act);
  return ep.half != 0 ? a * z1 : a;
}

// As finish, with the residual, stored to row `row` of y.
__device__ __forceinline__ void finish_store(const Epi& ep, int64_t boff, int64_t row, int64_t c,
                                             float z0, float z1) {
  float v = finish(ep, boff, c, z0, z1);
  const int64_t at = row * ep.ldy + c;
  if (ep.residual != nullptr) v += load_f32(ep.residual, ep.y_dt, at);
  store_as(ep.y, ep.y_dt, at, v);
}

// ------------------------------------------------------------------ launchers

// Where launches go.  A dry run of a call makes none, reads no pointer and asks no
// device for anything but its compute units: it says whether a grid holds every one
// of the call's launches, before the first.
struct Queue {
  hipStream_t s = nullptr;
  bool dry = false;
};

// A launch of x * y * z workgroups.  One that a grid does not hold (2^32 threads
// along x, 65535 workgroups along y or z) is refused here instead of cut short.
// dynamic: bytes of dynamic LDS that the kernel has to be allowed, noted in `allowed`.
inline hipError_t launch_blocks(const void* fn, int64_t x, int threads, void** argv, size_t lds, Queue q,
                                int64_t y = 1, int64_t z = 1, int dynamic = 0,
                                std::atomic<uint64_t>* allowed = nullptr) {
  if (x < 1 || x > ((int64_t{1} << 32) - 1) / threads || y < 1 || y > 65535 || z < 1 || z > 65535)
    return hipErrorInvalidConfiguration;
  if (q.dry) return hipSuccess;
  if (allowed != nullptr) {
    const hipError_t e = allow_dynamic_lds(fn, dynamic, *allowed);
    if (e != hipSuccess) return e;
  }
  return hipLaunchKernel(fn, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y), static_cast<unsigned>(z)),
                         dim3(static_cast<unsigned>(threads)), argv, lds, q.s);
}

// p + n bytes; of a null pointer (dry runs have no buffers) itself.
inline uint8_t* behind(void* p, size_t n) { return p != nullptr ? static_cast<uint8_t*>(p) + n : nullptr; }

// A product as the launchers take it.
struct Product {
  const void* x = nullptr;
  DType xt;
  int64_t x_rows;
  const uint8_t* W = nullptr;
  int64_t m;  // rows of one group (dense), or tokens
  int64_t n, k;
  int64_t topk = 1, experts = 0;  // experts == 0: dense
  const int* plan = nullptr;      // experts: the plan's words
  bool combine = false;           // experts: rows summed by `weights`
  const float* weights = nullptr;
  Epi ep;
};

size_t product_workspace_bytes(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k,
                               int64_t x_rows, DType xt, bool gated, bool combine);
hipError_t launch_product(const Product& p, void* workspace, Queue q);

// Matrix-core products of many rows (16-bit x, and fp32 x on the exact route).
size_t stage_bytes(int64_t rows, int64_t k);
hipError_t launch_stage(const void* x, int64_t rows, int64_t k, void* ws, const half_t** xs,
                        const float** scale, Queue q);
size_t fused_gemm_bytes(int64_t m, int64_t n, int64_t k, DType xt, bool gated, bool grouped);
hipError_t launch_fused_gemm(const Product& p, const Epi& ep, const Rows& rows, const half_t* xs,
                             const float* xscale, int64_t row_tiles, void* workspace, Queue q);

// Matrix-core products of few rows (16-bit x as fp16).
bool fused_gemv_supports(int64_t n, int64_t k, int64_t x_rows, int64_t experts);
hipError_t launch_fused_gemv(const Product& p, const Epi& ep, const Rows& rows, const half_t* xs,
                             const float* xscale, int64_t max_tiles, int tile_rows, Queue q);

// Expert products of at most 16 rows per tile, streamed by single wavefronts.
// They take bf16 x as it is.
bool fused_wave_supports(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k, int64_t x_rows);
hipError_t launch_fused_wave(const Product& p, const Epi& ep, const Rows& rows, int64_t max_tiles, Queue q);

// Dense products of few rows and few row tiles (bf16 x, xb, as it is).
bool fused_split_supports(int64_t m, int64_t nout, int64_t n, int64_t k, bool xb);
hipError_t launch_fused_split(const Product& p, const Epi& ep, Queue q);

struct RouteArgs {
  const void* logits;
  DType dt;
  int64_t m, experts, topk;
  const float* bias;
  int sigmoid, groups, group_topk, top2, renormalise;
  float scale;
  int* ids;
  float* weights;
  int* plan;  // may be null
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_plan(const int* ids, int64_t m, int64_t topk, int64_t experts, int* plan,
                             hipStream_t s);

// An expert layer of one token (r.plan unused; up.ep.y is down.x).
bool moe_one_supports(const RouteArgs& r, const Product& up, const Product& down);
hipError_t launch_moe_one(const RouteArgs& r, const Product& up, const Product& down, Queue q);

}  // namespace q4
