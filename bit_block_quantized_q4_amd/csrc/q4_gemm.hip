// Q4_0 prefill GEMM for gfx950: y[m][n] = x[m][k] . dequant(W)^T on fp16 MFMA.
//
// The GPU path from Q4_0 weights onto matrix cores of the vertical-disaggregation page
// (section "Every cycle counts: custom kernels"): long prompts are dense
// computation, so weights are dequantised once per workgroup to fp16
// w = (q - 8) * d (one rounding) and contracted with the fp16 activations on
// v_mfma_f32_32x32x16_f16 with fp32 accumulation.  Every output is summed in a
// fixed order (k order within one lane; for slice-K tiles the four slice
// partials then in wave order; for split-K tails the splits in split order),
// so results are bit-reproducible.
//
// Kernels
// -------
//   - gemm_mfma_kernel (k % 64 == 0): a BM x BN output tile per workgroup
//     (256 x 256 with 8 waves, each 128 x 64, for m >= 1024; else 128 x 128
//     with 4 waves of 64 x 64), k steps of 64 (two Q4_0 blocks), two LDS
//     stages.  Activations arrive by direct global->LDS copies
//     (global_load_lds_dwordx4) into an XOR swizzle (piece c of row r at
//     r*8 + (c ^ key(r)), key(r) = (r & 7) ^ ((r >> 3) & 1)) under which the
//     16-byte operand reads have no bank conflicts.  Each
//     thread owns weight units (one whole block of one row), loads them two
//     steps ahead, dequantises them with byte permutes, the 1024+q / 64+q
//     exponent trick, an exact packed subtraction and one packed multiply by
//     d, and writes them into the other stage in the same swizzle, interleaved
//     with the step's matrix products.  One barrier per step.
//   - gemm_slicek_kernel (m < 1024, k % 256 == 0, k >= 1024): 128 x 128 tiles
//     whose four waves each own the whole tile for one k16 slice of every
//     step, with packed weights copied into LDS and dequantised in registers
//     by the one wave that uses them; see its own comment.
//   - gemm_tile_kernel: the generic LDS-tiled kernel for k % 64 != 0.
//   - gemm_exact_kernel: the exact route (fp32 activations; see exact_tile128).
// Launches run whole rounds of tiles on the compute units; a partial round's
// columns run the same tiles with K split across workgroups (fp32 partials,
// then splitk_reduce_kernel in split order).
//
// The fp16 tiles are exact up to fp32 summation only while every dequantised
// weight and every activation is an fp16 value.  A block scale |d| > 8188
// breaks the first (its largest element, code 0, dequantises to 8 |d| >
// 65504, i.e. to +-inf), and bf16 activations outside fp16's range or off
// its subnormal grid break the second (the bf16 staging pass writes such a
// row as NaN).  Either makes the tile's fp32 accumulators non-finite, so
// every fp16 kernel checks its accumulators once at the end and a workgroup
// that finds a non-finite one recomputes its tile (and K range) on the exact
// route from the original activations.  In-domain results are finite, so the
// check never fires on them.
#include <initializer_list>

#include "q4_gemm_plan.hpp"
#include "q4_gemm_tile.hpp"

namespace q4 {
namespace {

// Rows and columns of a plain product: tile (blockIdx.y, blockIdx.x) of x
// [m][k] against n weight rows, outputs at row stride ldy (final outputs or,
// zstride apart by blockIdx.z, fp32 split-K partials).
template <typename YT>
struct PlainIO {
  static constexpr bool kPlain = true, kPairs = false;
  YT* y;
  int64_t m, n, ldy, zstride;
  int64_t m0 = 0, n0 = 0;

  template <int BM, int BN>
  __device__ __forceinline__ bool begin() {
    m0 = static_cast<int64_t>(blockIdx.y) * BM;
    n0 = static_cast<int64_t>(blockIdx.x) * BN;
    y += static_cast<int64_t>(blockIdx.z) * zstride;
    return true;
  }
  __device__ __forceinline__ const uint8_t* weights(const uint8_t* W) const { return W; }
  __device__ __forceinline__ int64_t xrow(int r) const { return m0 + r < m ? m0 + r : m - 1; }
  __device__ __forceinline__ int64_t wrow(int c) const { return n0 + c < n ? n0 + c : n - 1; }
  __device__ __forceinline__ bool row_in(int r) const { return m0 + r < m; }
  __device__ __forceinline__ bool col_in(int c) const { return n0 + c < n; }
  __device__ __forceinline__ int64_t xbase() const { return m0; }
  __device__ __forceinline__ int64_t wbase() const { return n0; }
  __device__ __forceinline__ int64_t xrow_in(int r) const { return m0 + r; }
  __device__ __forceinline__ int64_t wrow_in(int c) const { return n0 + c; }
  __device__ __forceinline__ void store1(int r, int c, float v) const {
    const int64_t row = m0 + r, col = n0 + c;
    if (row < m && col < n) y[row * ldy + col] = static_cast<YT>(v);
  }
  __device__ __forceinline__ void store4x4(int r4, int c4, const float4_t (&sc)[4]) const {
    const int64_t col = n0 + c4;
    const bool vec_ok = (ldy & 3) == 0 && col + 3 < n;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = m0 + r4 + r;
      if (row >= m) continue;
      YT* dst = y + row * ldy + col;
      if (vec_ok) {
        if constexpr (sizeof(YT) == 2) {
          const half4_t h = {static_cast<half_t>(sc[0][r]), static_cast<half_t>(sc[1][r]),
                             static_cast<half_t>(sc[2][r]), static_cast<half_t>(sc[3][r])};
          *reinterpret_cast<half4_t*>(dst) = h;
        } else {
          *reinterpret_cast<float4_t*>(dst) = float4_t{sc[0][r], sc[1][r], sc[2][r], sc[3][r]};
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col + c < n) dst[c] = static_cast<YT>(sc[c][r]);
      }
    }
  }
};

template <int BM, int BN, int WVM, int WVN, typename YT>
__global__ __launch_bounds__(WVM * WVN * 64, 1) void gemm_mfma_kernel(
    const half_t* __restrict__ x, const uint8_t* __restrict__ W, YT* __restrict__ y,
    int64_t m, int64_t n, int64_t k, int64_t ldy, int kps, int64_t zstride,
    const void* __restrict__ xe, int xet) {
  gemm_mfma_body<BM, BN, WVM, WVN>(PlainIO<YT>{y, m, n, ldy, zstride}, x, W, k, kps, xe, xet);
}

template <typename YT>
__global__ __launch_bounds__(256, 1) void gemm_slicek_kernel(
    const half_t* __restrict__ x, const uint8_t* __restrict__ W, YT* __restrict__ y,
    int64_t m, int64_t n, int64_t k, int64_t ldy, int kps, int64_t zstride,
    const void* __restrict__ xe, int xet) {
  gemm_slicek_body(PlainIO<YT>{y, m, n, ldy, zstride}, x, W, k, kps, xe, xet);
}

template <typename YT>
__global__ __launch_bounds__(256) void gemm_tile_kernel(
    const half_t* __restrict__ x, const uint8_t* __restrict__ W, YT* __restrict__ y,
    int64_t m, int64_t n, int64_t k, const void* __restrict__ xe, int xet) {
  gemm_tile_body(PlainIO<YT>{y, m, n, n, 0}, x, W, k, xe, xet);
}

// Exact route as a kernel: one 128 x 128 tile per workgroup over all of K
// (fp32 activations).
template <typename YT>
__global__ __launch_bounds__(256) void gemm_exact_kernel(const void* __restrict__ x, int xt,
                                                         const uint8_t* __restrict__ W,
                                                         YT* __restrict__ y, int64_t m, int64_t n,
                                                         int64_t k) {
  __shared__ __attribute__((aligned(16))) float lds[kExLdsBytes / 4];
  PlainIO<YT> io{y, m, n, n, 0};
  io.template begin<128, 128>();
  exact_tile128<256>(io, x, static_cast<DType>(xt), k, W, (k / kQK) * kBlockBytes, 0, 0, 0, k / kQK, lds);
}



// Output columns c0 .. c0 + nc - 1 (weight rows c0 ..) into yc (their first
// column, row stride ldy); with splits > 1, split z of K goes to yc + z zstride.
// The original activations (the exact route's input): a pointer and dtype.
struct XSrc {
  const void* p;
  int dt;
};

template <int BM, int BN, int WVM, int WVN, typename YT>
hipError_t launch_tiled(const half_t* x, const uint8_t* packed, int64_t c0, int64_t nc, YT* yc,
                        int64_t m, int64_t k, int64_t ldy, int splits, int kps, int64_t zstride,
                        XSrc xe, hipStream_t s) {
  const uint8_t* w = packed + c0 * ((k / kQK) * kBlockBytes);
  void* argv[] = {const_cast<const half_t**>(&x), const_cast<const uint8_t**>(&w), &yc, &m,
                  &nc, &k, &ldy, &kps, &zstride, &xe.p, &xe.dt};
  const dim3 grid(static_cast<unsigned>((nc + BN - 1) / BN), static_cast<unsigned>((m + BM - 1) / BM),
                  static_cast<unsigned>(splits));
  return hipLaunchKernel(reinterpret_cast<const void*>(&gemm_mfma_kernel<BM, BN, WVM, WVN, YT>),
                         grid, dim3(WVM * WVN * 64), argv, 0, s);
}

template <typename YT>
hipError_t launch_slicek(const half_t* x, const uint8_t* packed, int64_t c0, int64_t nc, YT* yc,
                         int64_t m, int64_t k, int64_t ldy, int splits, int kps, int64_t zstride,
                         XSrc xe, hipStream_t s) {
  const uint8_t* w = packed + c0 * ((k / kQK) * kBlockBytes);
  void* argv[] = {const_cast<const half_t**>(&x), const_cast<const uint8_t**>(&w), &yc, &m,
                  &nc, &k, &ldy, &kps, &zstride, &xe.p, &xe.dt};
  const dim3 grid(static_cast<unsigned>((nc + 127) / 128), static_cast<unsigned>((m + 127) / 128),
                  static_cast<unsigned>(splits));
  return hipLaunchKernel(reinterpret_cast<const void*>(&gemm_slicek_kernel<YT>), grid, dim3(256),
                         argv, 0, s);
}

// y[r][c] = sum over z of part[z][r][c] (fixed order), 4 columns per thread.
template <typename YT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ part, YT* __restrict__ y,
                                                           int64_t m, int64_t nc, int64_t ldy, int splits) {
  const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // quad index
  const int64_t quads = m * nc / 4;
  if (q >= quads) return;
  const int64_t e = 4 * q, r = e / nc, c = e - r * nc;
  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int z = 0; z < splits; ++z) acc += *reinterpret_cast<const float4_t*>(part + z * m * nc + e);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[r * ldy + c + i] = static_cast<YT>(acc[i]);
}

template <typename YT>
hipError_t launch_tile_type(Tile t, const half_t* x, const uint8_t* packed, int64_t c0, int64_t nc,
                            YT* yc, int64_t m, int64_t k, int64_t ldy, int splits, int kps,
                            int64_t zstride, XSrc xe, hipStream_t s) {
  if (t == Tile::Big)
    return launch_tiled<256, 256, 2, 4, YT>(x, packed, c0, nc, yc, m, k, ldy, splits, kps, zstride, xe, s);
  if (t == Tile::SliceK)
    return launch_slicek<YT>(x, packed, c0, nc, yc, m, k, ldy, splits, kps, zstride, xe, s);
  return launch_tiled<128, 128, 2, 2, YT>(x, packed, c0, nc, yc, m, k, ldy, splits, kps, zstride, xe, s);
}

template <typename YT>
hipError_t dispatch_tiled(const half_t* x, const uint8_t* packed, YT* y, int64_t m, int64_t n,
                          int64_t k, void* workspace, XSrc xe, hipStream_t s) {
  const GemmPlan p = gemm_plan(m, n, k);
  const int nks = static_cast<int>(k / kBK);
  hipError_t e = hipSuccess;
  if (p.n_main > 0) {
    e = launch_tile_type<YT>(p.main, x, packed, 0, p.n_main, y, m, k, n, 1, nks, 0, xe, s);
    if (e != hipSuccess || p.n_main == n) return e;
  }
  // Split columns: split z of K writes part[z], m x nt with row stride nt.
  const int64_t nt = n - p.n_main;
  float* part = static_cast<float*>(workspace);
  e = launch_tile_type<float>(p.tail, x, packed, p.n_main, nt, part, m, k, nt, p.splits, p.kps,
                              m * nt, xe, s);
  if (e != hipSuccess) return e;
  const int64_t quads = m * nt / 4;
  YT* yt = y + p.n_main;
  int sp = p.splits;
  int64_t ldy = n, mm = m, ntt = nt;
  void* argv[] = {&part, &yt, &mm, &ntt, &ldy, &sp};
  return hipLaunchKernel(reinterpret_cast<const void*>(&splitk_reduce_kernel<YT>),
                         dim3(static_cast<unsigned>((quads + 255) / 256)), dim3(256), argv, 0, s);
}

}  // namespace

namespace {

// Converted bf16 activations occupy the workspace's first bytes.
int64_t bf16_stage_bytes(int64_t m, int64_t k) { return (m * k * 2 + 255) / 256 * 256; }

// bf16 activations -> fp16 rows (round to nearest even), one workgroup of
// 256 threads per row (a 256-row chunk still fills the chip).  A row that
// holds any value fp16 cannot represent exactly (beyond its range, or off its
// subnormal grid) is written entirely as NaN instead: every tile and K split
// that reads it then ends with non-finite accumulators and is recomputed on
// the exact route from the bf16 original.  Both buffers are 16-byte aligned
// and k % 32 == 0.
__global__ __launch_bounds__(256) void bf16_rows_to_f16_kernel(const uint16_t* __restrict__ x,
                                                               uint16_t* __restrict__ out,
                                                               int64_t m, int64_t k) {
  const int64_t row = blockIdx.x;  // < m: one workgroup per row
  const u32x4* src = reinterpret_cast<const u32x4*>(x + row * k);
  u32x4* dst = reinterpret_cast<u32x4*>(out + row * k);
  const int64_t np = k / 8;  // 16-byte pieces
  bool inexact = false;
  for (int64_t p = threadIdx.x; p < np; p += 256) {
    u32x4 v = src[p];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t h = bf16x2_to_f16x2(v[e]);
      inexact |= !f16x2_holds_bf16x2(h, v[e]);
      v[e] = h;
    }
    dst[p] = v;
  }
  // (a separate kernel with no dynamic LDS: __syncthreads_or's own LDS is fine)
  if (__syncthreads_or(inexact)) {
    const u32x4 qnan = {0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
    for (int64_t p = threadIdx.x; p < np; p += 256) dst[p] = qnan;  // after this thread's own stores
  }
}

}  // namespace

size_t gemm_workspace_bytes(int64_t m, int64_t n, int64_t k, DType xt) {
  if (xt == DType::F32) return 0;  // the exact route needs no workspace
  const size_t tiles = gemm_plan(m, n, k).ws_bytes;
  return xt == DType::BF16 ? static_cast<size_t>(bf16_stage_bytes(m, k)) + tiles : tiles;
}

hipError_t launch_gemm(const void* x, DType xt, const uint8_t* packed, void* y,
                       DType yt, int64_t m, int64_t n, int64_t k, void* workspace,
                       hipStream_t s) {
  const dim3 grid128(static_cast<unsigned>((n + 127) / 128), static_cast<unsigned>((m + 127) / 128));
  if (xt == DType::F32) {
    // fp32 activations: the exact route (fp32 matrix cores) for every tile.
    int xti = static_cast<int>(xt);
    void* argv[] = {const_cast<void**>(&x), &xti, const_cast<const uint8_t**>(&packed), &y,
                    &m, &n, &k};
    const void* fn = yt == DType::F16 ? reinterpret_cast<const void*>(&gemm_exact_kernel<half_t>)
                                      : reinterpret_cast<const void*>(&gemm_exact_kernel<float>);
    return hipLaunchKernel(fn, grid128, dim3(256), argv, 0, s);
  }
  const half_t* xp = static_cast<const half_t*>(x);
  const XSrc xe{x, static_cast<int>(xt)};
  if (xt == DType::BF16) {
    // Stage the activations as fp16 rows in the workspace (NaN rows where
    // fp16 cannot hold them exactly), then run the fp16 path on them with the
    // rest of the workspace; the exact route reads the bf16 original.
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const uint16_t* src = static_cast<const uint16_t*>(x);
    uint16_t* dst = reinterpret_cast<uint16_t*>(ws);
    int64_t mm = m, kk = k;
    void* argv[] = {&src, &dst, &mm, &kk};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&bf16_rows_to_f16_kernel),
                                         dim3(static_cast<unsigned>(m)), dim3(256), argv, 0, s);
    if (e != hipSuccess) return e;
    xp = reinterpret_cast<const half_t*>(ws);
    workspace = gemm_plan(m, n, k).ws_bytes > 0 ? ws + bf16_stage_bytes(m, k) : nullptr;
  }
  if (k % kBK == 0) {
    if (yt == DType::F16)
      return dispatch_tiled(xp, packed, static_cast<half_t*>(y), m, n, k, workspace, xe, s);
    return dispatch_tiled(xp, packed, static_cast<float*>(y), m, n, k, workspace, xe, s);
  }
  const void* xev = xe.p;
  int xet = xe.dt;
  if (yt == DType::F16) {
    half_t* yp = static_cast<half_t*>(y);
    void* argv[] = {&xp, const_cast<const uint8_t**>(&packed), &yp, &m, &n, &k, &xev, &xet};
    return hipLaunchKernel(reinterpret_cast<const void*>(&gemm_tile_kernel<half_t>),
                           grid128, dim3(256), argv, 0, s);
  }
  float* yp = static_cast<float*>(y);
  void* argv[] = {&xp, const_cast<const uint8_t**>(&packed), &yp, &m, &n, &k, &xev, &xet};
  return hipLaunchKernel(reinterpret_cast<const void*>(&gemm_tile_kernel<float>),
                         grid128, dim3(256), argv, 0, s);
}

}  // namespace q4
