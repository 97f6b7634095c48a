// Fused linear layer and expert products for many rows: the prefill GEMM's
// tiles (q4_gemm_tile.hpp) with the epilogue in their stores.
//
// Bound by the matrix cores: 2 m n k flops.  A gated layer needs gate row c
// and up row n / 2 + c in one lane at the store, so the weight rows enter the
// tile interleaved by 32 (tile column c: row (c / 64) 32 + c % 32 of the gate
// for c / 32 even, of the up half for odd): the two 32-column products of a
// wave are then the two factors of its outputs, register by register, and the
// loop over k is the plain GEMM's.  An expert's tile gathers its rows of x by
// per-row addresses in the same copies (no gathered copy of x is made) and
// scatters its outputs by row.
//
// The dequantised weights are fp16, rounded once (2^-11 relative), as q4_gemm's:
// the codes kept exact and the block scale applied to the sums in fp32 take 16
// vector FMAs per two matrix products, as many cycles as those have.  The error of a
// fp16 output grows from its own rounding's 2.1e-4 of the norm to 2.6e-4, with a gate,
// where two such sums are multiplied, to 3.2e-4.
//
// bf16 rows are staged once as fp16, each multiplied by the power of two that
// brings its largest magnitude to [2^15, 2^16), which the store takes back:
// exact for every value from 2^-32 of that magnitude on, below that rounded to
// multiples of 2^-39 of it (finer than what the fp32 sums keep of the row).
#include "q4_fused.hpp"
#include "q4_gemm_plan.hpp"
#include "q4_gemm_group.hpp"

namespace q4 {
namespace {

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ half_t to_out<half_t>(float v) { return static_cast<half_t>(v); }
template <>
__device__ __forceinline__ __bf16 to_out<__bf16>(float v) { return static_cast<__bf16>(v); }

template <typename T>
struct alignas(16) Vec8 {
  T v[8];
};

// activate() on eight values, one branch for all.
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f(v[i]);
  };
  switch (act) {
    case kActRelu: each([](float z) { return activate(z, kActRelu); }); break;
    case kActSilu: each([](float z) { return activate(z, kActSilu); }); break;
    case kActGelu: each([](float z) { return activate(z, kActGelu); }); break;
    case kActGeluErf: each([](float z) { return activate(z, kActGeluErf); }); break;
    default: break;
  }
}

// What a fused tile needs beside the tile code's own arguments.
struct FusedArgs {
  Epi ep;
  Rows rows;
  const float* xscale;  // [x rows], or nullptr
  int64_t m;            // dense: rows
  int64_t cols;         // tile columns: n, or gated n / 2 rounded up to 32, times two
  int64_t c0;           // first tile column of this launch
  float* part;          // PART: split-K partials, [z][m][ldp]
  int64_t ldp, zstride;
  int parts;            // experts: kernel tiles per tile of the plan
};

enum Mode { kDense = 0, kGrouped = 1, kPart = 2 };

template <int BM, bool GATED, int MODE, bool DEALT = false>
struct FusedIO {
  static constexpr bool kPlain = false, kDealt = DEALT;
  static constexpr bool kPairs = GATED && MODE != kPart;
  FusedArgs a;
  int* prow;      // LDS: row of y of every tile row
  float* pscale;  // LDS: factor of its sums
  uint32_t* votes;  // LDS: chunks of rows with a sum that is not finite
  int64_t n0 = 0, m0 = 0, boff = 0, woff = 0;
  const int* rec = nullptr;  // kGrouped: the tile's pairs
  int count = 0;

  // A thread's eight output columns.
  struct Cols {
    int64_t c;    // the first one (PART: of the partials)
    int valid;    // how many of them exist
    bool wide;    // one wide access covers them
    float b0[8], b1[8];
  };

  // The output column (GATED: of the pair) of tile column c of this launch.
  __device__ __forceinline__ int64_t unit(int64_t g) const { return 32 * (g >> 6) + (g & 31); }

  template <int TM, int TN>
  __device__ __forceinline__ bool begin() {
    static_assert(TM == BM, "tile rows");
    n0 = a.c0 + static_cast<int64_t>(blockIdx.x) * TN;
    if constexpr (MODE == kGrouped) {
      const int t = blockIdx.y / a.parts;
      rec = a.rows.recs + static_cast<int64_t>(t) * a.rows.rec_words;
      const int4 tile = *reinterpret_cast<const int4*>(rec);
      const int used = *a.rows.ntiles;  // (both loads in flight)
      const int skip = (blockIdx.y - t * a.parts) * BM, left = tile.z - skip;
      if (t >= used || left <= 0) return false;
      rec += 4 + skip;
      count = left < BM ? left : BM;
      woff = tile.x * a.rows.wstride;
      boff = tile.x * a.rows.nbias;
    } else {
      m0 = static_cast<int64_t>(blockIdx.y) * BM;
      const int64_t left = a.m - m0;
      count = left < BM ? static_cast<int>(left) : BM;
    }
    if (threadIdx.x < 4) votes[threadIdx.x] = 0u;
    for (int r = threadIdx.x; r < BM; r += blockDim.x) {
      const int64_t x = xrow(r);
      if constexpr (MODE == kGrouped) prow[r] = rec[r < count ? r : 0];
      pscale[r] = a.xscale != nullptr ? a.xscale[x] : 1.0f;
    }
    return true;  // (read after the tile loop's barriers)
  }
  __device__ __forceinline__ const uint8_t* weights(const uint8_t* W) const { return W + woff; }
  __device__ __forceinline__ int64_t xrow(int r) const {
    if constexpr (MODE == kGrouped) return rec[r < count ? r : 0] / a.rows.xdiv;
    return m0 + (r < count ? r : count - 1);
  }
  __device__ __forceinline__ int64_t wrow(int c) const {
    const int64_t g = n0 + c;
    if constexpr (GATED) {
      const int64_t u = unit(g);
      return (u < a.ep.half ? u : a.ep.half - 1) + ((g >> 5) & 1) * a.ep.half;
    }
    return g < a.cols ? g : a.cols - 1;
  }
  __device__ __forceinline__ int fragments(int rows) const {
    return __builtin_amdgcn_readfirstlane((count + rows - 1) / rows);
  }
  __device__ __forceinline__ bool row_in(int r) const { return r < count; }
  __device__ __forceinline__ bool col_in(int c) const {
    return GATED ? unit(n0 + c) < a.ep.half : n0 + c < a.cols;
  }
  __device__ __forceinline__ int64_t xrow_in(int r) const { return xrow(r); }
  __device__ __forceinline__ int64_t wrow_in(int c) const { return wrow(c); }
  __device__ __forceinline__ int64_t xbase() const { return MODE == kGrouped ? 0 : m0; }
  __device__ __forceinline__ int64_t wbase() const { return GATED ? 0 : n0; }
  __device__ __forceinline__ int64_t yrow(int r) const {
    if constexpr (MODE == kGrouped) return prow[r];
    return m0 + r;
  }
  template <int W>
  __device__ __forceinline__ Cols columns(int c0, int g) const {
    Cols col;
    int64_t end;
    if constexpr (kPairs) {
      col.c = unit(n0 + c0) + 32 * (g >> 2) + 8 * (g & 3);
      end = a.ep.half;
    } else {
      col.c = n0 + c0 + 8 * g;
      end = a.cols;
      if constexpr (MODE == kPart) {
        col.c -= a.c0;
        end -= a.c0;
      }
    }
    col.valid = end - col.c >= 8 ? 8 : end > col.c ? static_cast<int>(end - col.c) : 0;
    col.wide = col.valid == 8 && (MODE == kPart ? (a.ldp & 3) == 0 : (a.ep.ldy & 7) == 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      col.b0[i] = col.b1[i] = 0.f;
      if constexpr (MODE != kPart) {
        if (a.ep.bias != nullptr && i < col.valid) {
          col.b0[i] = load_f32(a.ep.bias, a.ep.bias_dt, boff + col.c + i);
          if constexpr (GATED) col.b1[i] = load_f32(a.ep.bias, a.ep.bias_dt, boff + a.ep.half + col.c + i);
        }
      }
    }
    return col;
  }
  template <bool SCALED>
  __device__ __forceinline__ void emit(const Cols& col, const float* sums, int r) const {
    if (r >= count || col.valid == 0) return;
    const float sc = SCALED ? pscale[r] : 1.0f;
    float v[8];
    auto read8 = [&](const float* p, float (&o)[8]) {
      const float4_t lo = *reinterpret_cast<const float4_t*>(p), hi = *reinterpret_cast<const float4_t*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = lo[i] * sc;
        o[4 + i] = hi[i] * sc;
      }
    };
    read8(sums, v);
    if constexpr (MODE == kPart) {
      float* p = a.part + static_cast<int64_t>(blockIdx.z) * a.zstride + (m0 + r) * a.ldp + col.c;
      if (col.wide) {
        *reinterpret_cast<float4_t*>(p) = float4_t{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<float4_t*>(p + 4) = float4_t{v[4], v[5], v[6], v[7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < col.valid) p[i] = v[i];
      }
    } else {
      if (a.ep.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += col.b0[i];
      }
      activate8(v, a.ep.act);
      if constexpr (GATED) {
        float u[8];
        read8(sums + 32, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= u[i] + col.b1[i];
      }
      const int64_t at = yrow(r) * a.ep.ldy + col.c;
      if (a.ep.y_dt == static_cast<int>(DType::F32)) put8<float>(col, at, v);
      else if (a.ep.y_dt == static_cast<int>(DType::F16)) put8<half_t>(col, at, v);
      else put8<__bf16>(col, at, v);
    }
  }
  template <typename T>
  __device__ __forceinline__ void put8(const Cols& col, int64_t at, float (&v)[8]) const {
    T* y = static_cast<T*>(a.ep.y) + at;
    const T* res = static_cast<const T*>(a.ep.residual) + at;
    if (col.wide) {
      if (a.ep.residual != nullptr) {
        const Vec8<T> q = *reinterpret_cast<const Vec8<T>*>(res);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += static_cast<float>(q.v[i]);
      }
      Vec8<T> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = to_out<T>(v[i]);
      *reinterpret_cast<Vec8<T>*>(y) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < col.valid) {
          if (a.ep.residual != nullptr) v[i] += static_cast<float>(res[i]);
          y[i] = to_out<T>(v[i]);
        }
    }
  }
};

template <int BM, int BN, int WVM, int WVN, bool GATED, int MODE>
__global__ __launch_bounds__(WVM * WVN * 64, 1) void fused_mfma_kernel(const half_t* __restrict__ x,
                                                                       const uint8_t* __restrict__ W,
                                                                       int64_t k, int kps, FusedArgs a,
                                                                       const void* __restrict__ xe, int xet) {
  __shared__ int prow[BM];
  __shared__ float pscale[BM];
  __shared__ uint32_t votes[4];
  gemm_mfma_body<BM, BN, WVM, WVN>(FusedIO<BM, GATED, MODE>{a, prow, pscale, votes}, x, W, k, kps, xe, xet);
}

template <bool GATED>
__global__ __launch_bounds__(512, 1) void fused_group_kernel(const half_t* __restrict__ x,
                                                             const uint8_t* __restrict__ W, int64_t k, int,
                                                             FusedArgs a, const void* __restrict__ xe,
                                                             int xet) {
  __shared__ int prow[kGroupRows];
  __shared__ float pscale[kGroupRows];
  __shared__ uint32_t votes[4];
  gemm_group_body<kGroupRows, 256, 2, 4>(
      FusedIO<kGroupRows, GATED, kGrouped, true>{a, prow, pscale, votes}, x, W, k, xe, xet);
}

template <bool GATED, int MODE>
__global__ __launch_bounds__(256, 1) void fused_slicek_kernel(const half_t* __restrict__ x,
                                                              const uint8_t* __restrict__ W, int64_t k,
                                                              int kps, FusedArgs a,
                                                              const void* __restrict__ xe, int xet) {
  __shared__ int prow[128];
  __shared__ float pscale[128];
  __shared__ uint32_t votes[4];
  gemm_slicek_body(FusedIO<128, GATED, MODE>{a, prow, pscale, votes}, x, W, k, kps, xe, xet);
}

template <bool GATED, int MODE>
__global__ __launch_bounds__(256) void fused_tile_kernel(const half_t* __restrict__ x,
                                                         const uint8_t* __restrict__ W, int64_t k, int,
                                                         FusedArgs a, const void* __restrict__ xe, int xet) {
  __shared__ int prow[128];
  __shared__ float pscale[128];
  __shared__ uint32_t votes[4];
  gemm_tile_body(FusedIO<128, GATED, MODE>{a, prow, pscale, votes}, x, W, k, xe, xet);
}

// The exact route for every tile (fp32 activations).
template <bool GATED, int MODE>
__global__ __launch_bounds__(256) void fused_exact_kernel(const half_t* __restrict__,
                                                          const uint8_t* __restrict__ W, int64_t k, int,
                                                          FusedArgs a, const void* __restrict__ xe, int xet) {
  __shared__ __attribute__((aligned(16))) float lds[64 * 132];
  __shared__ int prow[128];
  __shared__ float pscale[128];
  __shared__ uint32_t votes[4];
  FusedIO<128, GATED, MODE> io{a, prow, pscale, votes};
  if (!io.template begin<128, 128>()) return;
  exact_tile128<256>(io, xe, static_cast<DType>(xet), k, io.weights(W), (k / kQK) * kBlockBytes, 0, 0, 0,
                     k / kQK, lds);
}

// y = epilogue(sum over z of part[z]) for the outputs of the split columns,
// four columns per thread, in split order.
template <bool GATED>
__global__ __launch_bounds__(256) void fused_reduce_kernel(FusedArgs a, int splits, int64_t quads) {
  const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (q >= a.m * quads) return;
  const int64_t r = q / quads, c = 4 * (q - r * quads);           // output column, from the first one here
  const int64_t pc = GATED ? 64 * (c >> 5) + (c & 31) : c;        // partial column
  const int64_t out0 = GATED ? a.c0 / 2 : a.c0, nout = GATED ? a.ep.half : a.cols;
  float4_t s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
  for (int z = 0; z < splits; ++z) {
    const float* p = a.part + z * a.zstride + r * a.ldp + pc;
    s0 += *reinterpret_cast<const float4_t*>(p);
    if constexpr (GATED) s1 += *reinterpret_cast<const float4_t*>(p + 32);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (out0 + c + i < nout) finish_store(a.ep, 0, r, out0 + c + i, s0[i], s1[i]);
}

// bf16 rows -> fp16 rows and the inverse of their power-of-two factors.  WIDE:
// one workgroup per row, read twice; else one wavefront per row of at most
// kStagePieces x 64 16-byte pieces, which stay in registers (16384 rows of 768:
// 13.2 us against 16.9).  The sums of a row with an infinity or a NaN are not
// finite, so its tiles take the exact route.
constexpr int kStagePieces = 4;
template <bool WIDE>
__global__ __launch_bounds__(256) void stage_bf16_kernel(const uint16_t* __restrict__ x,
                                                         uint16_t* __restrict__ out,
                                                         float* __restrict__ inv, int64_t rows, int64_t k) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t row = WIDE ? blockIdx.x : blockIdx.x * int64_t{4} + wave;
  if (row >= rows) return;  // whole wavefront (WIDE: none)
  const u32x4* src = reinterpret_cast<const u32x4*>(x + row * k);
  u32x4* dst = reinterpret_cast<u32x4*>(out + row * k);
  const int64_t np = k / 8;
  uint32_t top = 0;  // largest magnitude, as bf16 bits
  auto look = [&](const u32x4& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max_magnitude_bf16(top, v[e]);
  };
  auto over_wave = [&]() {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const uint32_t o = __shfl_xor(top, off);
      top = o > top ? o : top;
    }
  };
  auto put = [&](int64_t p, u32x4 v, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = bf16x2_scaled_to_f16x2(v[e], f);
    dst[p] = v;
  };
  if constexpr (WIDE) {
    __shared__ uint32_t top_s[4];
    for (int64_t p = threadIdx.x; p < np; p += 256) look(src[p]);
    over_wave();
    if (lane == 0) top_s[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = top_s[w] > top ? top_s[w] : top;
    const int shift = bf16_row_shift(top);
    const float f = power_of_two(shift);
    if (threadIdx.x == 0) inv[row] = power_of_two(-shift);
    for (int64_t p = threadIdx.x; p < np; p += 256) put(p, src[p], f);
  } else {
    u32x4 v[kStagePieces];
#pragma unroll
    for (int i = 0; i < kStagePieces; ++i) {
      const int64_t p = lane + i * kWave;
      v[i] = src[p < np ? p : np - 1];
    }
#pragma unroll
    for (int i = 0; i < kStagePieces; ++i) look(v[i]);
    over_wave();
    const int shift = bf16_row_shift(top);
    const float f = power_of_two(shift);
    if (lane == 0) inv[row] = power_of_two(-shift);
#pragma unroll
    for (int i = 0; i < kStagePieces; ++i) {
      const int64_t p = lane + i * kWave;
      if (p < np) put(p, v[i], f);
    }
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Tile columns of a product.
int64_t tile_cols(int64_t n, bool gated) { return gated ? (n / 2 + 31) / 32 * 64 : n; }

// The slice-K tile reaches a gate's up rows by 32-bit offsets from the gate's.
bool slice_k(int64_t n, int64_t k, bool gated) {
  return !gated || n * (k / kQK * kBlockBytes) < (int64_t{1} << 32);
}

using KernelFn = const void*;

template <bool GATED, int MODE>
KernelFn kernel_of(Tile t) {
  if constexpr (MODE != kGrouped) {
    if (t == Tile::Big) return reinterpret_cast<KernelFn>(&fused_mfma_kernel<256, 256, 2, 4, GATED, MODE>);
    if (t == Tile::SliceK) return reinterpret_cast<KernelFn>(&fused_slicek_kernel<GATED, MODE>);
  }
  return reinterpret_cast<KernelFn>(&fused_mfma_kernel<128, 128, 2, 2, GATED, MODE>);
}

template <bool GATED>
KernelFn kernel_in(Tile t, int mode) {
  return mode == kDense ? kernel_of<GATED, kDense>(t)
                        : mode == kGrouped ? kernel_of<GATED, kGrouped>(t) : kernel_of<GATED, kPart>(t);
}

hipError_t launch_tiles(KernelFn fn, int tile, int threads, const half_t* x, const uint8_t* W, int64_t k,
                        int kps, const FusedArgs& a0, int64_t cols, int64_t row_tiles, int splits,
                        const void* xe, int xet, Queue q) {
  FusedArgs a = a0;
  void* argv[] = {&x, &W, &k, &kps, &a, &xe, &xet};
  return launch_blocks(fn, (cols + tile - 1) / tile, threads, argv, 0, q, row_tiles, splits);
}

}  // namespace

size_t stage_bytes(int64_t rows, int64_t k) {
  return up256(static_cast<size_t>(rows) * static_cast<size_t>(k) * 2) + up256(static_cast<size_t>(rows) * 4);
}

hipError_t launch_stage(const void* x, int64_t rows, int64_t k, void* ws, const half_t** xs,
                        const float** scale, Queue q) {
  const uint16_t* src = static_cast<const uint16_t*>(x);
  uint16_t* dst = static_cast<uint16_t*>(ws);
  float* inv = reinterpret_cast<float*>(behind(ws, up256(static_cast<size_t>(rows) * static_cast<size_t>(k) * 2)));
  *xs = reinterpret_cast<const half_t*>(dst);
  *scale = inv;
  void* argv[] = {&src, &dst, &inv, &rows, &k};
  if (k > kStagePieces * kWave * 8)
    return launch_blocks(reinterpret_cast<const void*>(&stage_bf16_kernel<true>), rows, 256, argv, 0, q);
  return launch_blocks(reinterpret_cast<const void*>(&stage_bf16_kernel<false>), (rows + 3) / 4, 256, argv, 0, q);
}

size_t fused_gemm_bytes(int64_t m, int64_t n, int64_t k, DType xt, bool gated, bool grouped) {
  if (grouped || xt == DType::F32) return 0;
  return up256(gemm_plan(m, tile_cols(n, gated), k, slice_k(n, k, gated)).ws_bytes);
}

hipError_t launch_fused_gemm(const Product& p, const Epi& ep, const Rows& rows, const half_t* xs,
                             const float* xscale, int64_t row_tiles, void* workspace, Queue q) {
  const bool gated = ep.half != 0, grouped = p.experts != 0;
  FusedArgs a{ep, rows, xscale, p.m, tile_cols(p.n, gated), 0, nullptr, 0, 0, 1};
  const int xet = static_cast<int>(p.xt);
  const int plan_rows = grouped ? plan_layout(p.m, p.topk, p.experts).tile_rows : 128;
  a.parts = (plan_rows + 127) / 128;  // of the kernels of 128-row tiles
  if (grouped) row_tiles *= a.parts;
  const int mode = grouped ? kGrouped : kDense;
  if (p.xt == DType::F32) {
    const KernelFn fn =
        gated ? (grouped ? reinterpret_cast<KernelFn>(&fused_exact_kernel<true, kGrouped>)
                         : reinterpret_cast<KernelFn>(&fused_exact_kernel<true, kDense>))
              : (grouped ? reinterpret_cast<KernelFn>(&fused_exact_kernel<false, kGrouped>)
                         : reinterpret_cast<KernelFn>(&fused_exact_kernel<false, kDense>));
    return launch_tiles(fn, 128, 256, xs, p.W, p.k, 0, a, a.cols, grouped ? row_tiles : (p.m + 127) / 128, 1,
                        p.x, xet, q);
  }
  if (p.k % kBK != 0) {
    const KernelFn fn =
        gated ? (grouped ? reinterpret_cast<KernelFn>(&fused_tile_kernel<true, kGrouped>)
                         : reinterpret_cast<KernelFn>(&fused_tile_kernel<true, kDense>))
              : (grouped ? reinterpret_cast<KernelFn>(&fused_tile_kernel<false, kGrouped>)
                         : reinterpret_cast<KernelFn>(&fused_tile_kernel<false, kDense>));
    return launch_tiles(fn, 128, 256, xs, p.W, p.k, 0, a, a.cols, grouped ? row_tiles : (p.m + 127) / 128, 1,
                        p.x, xet, q);
  }
  const int nks = static_cast<int>(p.k / kBK);
  if (grouped) {
    if (plan_rows == kGroupRows) {
      row_tiles /= a.parts;
      a.parts = 1;
      return launch_tiles(gated ? reinterpret_cast<KernelFn>(&fused_group_kernel<true>)
                                : reinterpret_cast<KernelFn>(&fused_group_kernel<false>),
                          256, 512, xs, p.W, p.k, nks, a, a.cols, row_tiles, 1, p.x, xet, q);
    }
    return launch_tiles(gated ? kernel_in<true>(Tile::Out128, mode) : kernel_in<false>(Tile::Out128, mode), 128,
                        256, xs, p.W, p.k, nks, a, a.cols, row_tiles, 1, p.x, xet, q);
  }
  const GemmPlan g = gemm_plan(p.m, a.cols, p.k, slice_k(p.n, p.k, gated));
  auto threads = [](Tile t) { return t == Tile::Big ? 512 : 256; };
  hipError_t e = hipSuccess;
  if (g.n_main > 0) {
    const int bt = tile_rows(g.main);
    FusedArgs b = a;
    const int64_t cols = g.n_main < a.cols ? g.n_main : a.cols;
    e = launch_tiles(gated ? kernel_in<true>(g.main, kDense) : kernel_in<false>(g.main, kDense), bt,
                     threads(g.main), xs, p.W, p.k, nks, b, cols, (p.m + bt - 1) / bt, 1, p.x, xet, q);
    if (e != hipSuccess || g.n_main == a.cols) return e;
  }
  const int bt = tile_rows(g.tail);
  a.c0 = g.n_main;
  a.part = static_cast<float*>(workspace);
  a.ldp = a.cols - g.n_main;
  a.zstride = p.m * a.ldp;
  e = launch_tiles(gated ? kernel_in<true>(g.tail, kPart) : kernel_in<false>(g.tail, kPart), bt,
                   threads(g.tail), xs, p.W, p.k, g.kps, a, a.ldp, (p.m + bt - 1) / bt, g.splits, p.x, xet, q);
  if (e != hipSuccess) return e;
  int splits = g.splits;
  int64_t quads = (gated ? a.ldp / 2 : a.ldp) / 4;
  void* argv[] = {&a, &splits, &quads};
  const KernelFn fn = gated ? reinterpret_cast<KernelFn>(&fused_reduce_kernel<true>)
                            : reinterpret_cast<KernelFn>(&fused_reduce_kernel<false>);
  return launch_blocks(fn, (p.m * quads + 255) / 256, 256, argv, 0, q);
}

}  // namespace q4
