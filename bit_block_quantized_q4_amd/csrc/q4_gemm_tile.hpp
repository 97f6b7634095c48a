// The prefill GEMM's tiles, shared by the plain GEMM and the fused products
// (gfx950).  Internal header.
//
// A tile kernel computes one BM x BN output tile; where its rows and columns
// come from and where its outputs go is the IO's:
//   begin<BM, BN>()    picks the workgroup's tile (false: it has none)
//   weights(W)         the tile's weight matrix
//   xrow(r), wrow(c)   x row / weight row of tile row r / column c, clamped to
//                      ones that exist; row_in(r), col_in(c): it does exist;
//                      xrow_in(r), wrow_in(c): the same for those, unclamped
//   xbase(), wbase()   a row near those (uniform)
// and, with kPlain (the plain GEMM, no epilogue),
//   store1(r, c, v)    one output
//   store4x4(r, c, s)  rows r .. r + 3 (float4 elements) of columns c .. c + 3
// or else
//   columns<W>(c0)     what this thread needs of its 8 columns of W from c0
//   emit<SCALED>(cols, sums, r)  the outputs of tile row r in those columns
//   votes              LDS words, one per chunk of rows, zero at the end of K
// kDealt: fragment i of wave row w holds tile rows 32 (i WVM + w) .. instead of
//   32 (w TM + i) ..; fragments(n) says how many fragments of n rows hold rows.
// kPairs: tile columns c and c + 32 (c / 32 even) make one output.
#pragma once

#include "q4_device.hpp"

namespace q4 {
namespace {

template <int V>
struct IC {
  static constexpr int value = V;
};

constexpr int BM = 128;       // rows of x per workgroup
constexpr int BN = 128;       // output features per workgroup
constexpr int BK = kQK;       // one Q4_0 block per k step
constexpr int LDK = BK + 8;   // padded LDS row (halves)

// ------------------------------------------------------------------ exact route
//
// y = sum over blocks of sum_j x[j] (q_j - 8) d with the activations widened
// exactly to fp32 (from fp32, fp16 or bf16) and the weights dequantised
// exactly to fp32, contracted on v_mfma_f32_32x32x2_f32 (fp32 operands, fp32
// accumulation): every product is formed from the exact operands, so the
// error is fp32 summation error relative to sum |x w|, for every in-domain
// input.  It is several times slower than the fp16 tiles.
constexpr int kExLd = 17;                        // floats per LDS row (16 k + 1 pad)
constexpr int kExLdsBytes = 2 * 128 * kExLd * 4;  // 17408

__device__ __forceinline__ float load_x_f32(const void* x, DType xt, int64_t i) {
  if (xt == DType::F32) return static_cast<const float*>(x)[i];
  if (xt == DType::F16) return static_cast<float>(static_cast<const half_t*>(x)[i]);
  return bf16_bits_to_float(static_cast<const uint16_t*>(x)[i]);
}

// f(IC<0>{}), ..., f(IC<N - 1>{}).
template <int I, int N, typename F>
__device__ __forceinline__ void each_chunk(F&& f) {
  if constexpr (I < N) {
    f(IC<I>{});
    each_chunk<I + 1, N>(f);
  }
}

// The fused products' way out: the sums of a tile go through LDS one chunk of
// RCH rows at a time, so that a thread stores eight neighbouring columns of a
// row with one wide store (and reads its residual, bias and the gate's other
// factor the same way) in a loop that is not unrolled.  write(IC<i>) puts the
// sums of chunk i into buf ([RCH][BN + 4] floats) and says whether one of them
// is not finite; tile_row(i, r) is the tile row of its row r.  A chunk with
// such a sum is not stored (the residual may be the output, which the exact
// route must find unchanged): its bit is set in the result, uniform over the
// workgroup.  live: chunks that hold rows.
template <int CHUNKS, int NTH, int BN, int RCH, bool SCALED, typename IO, typename W, typename R>
__device__ __forceinline__ uint32_t fused_epilogue(const IO& io, float* buf, int c0, W write, R tile_row,
                                                   int live = CHUNKS) {
  constexpr int kGroups = IO::kPairs ? BN / 16 : BN / 8;  // threads per row
  constexpr int kStep = NTH / kGroups;
  const int g = threadIdx.x % kGroups;
  const auto cols = io.template columns<BN>(c0, g);
  const int at = IO::kPairs ? 64 * (g >> 2) + 8 * (g & 3) : 8 * g;
  uint32_t skipped = 0;
  each_chunk<0, CHUNKS>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    if (i >= live) return;  // no rows
    __syncthreads();  // the buffer's previous readers are done
    if (write(ic)) io.votes[i] = 1u;  // every writer writes the same value
    __syncthreads();
    if (io.votes[i] != 0u) {
      skipped |= 1u << i;
    } else {
#pragma unroll 1
      for (int r = threadIdx.x / kGroups; r < RCH; r += kStep)
        io.template emit<SCALED>(cols, buf + r * (BN + 4) + at, tile_row(i, r));
    }
  });
  return skipped;
}

// One 128 x 128 sub-tile of the tile `io` describes: its rows r0 .. r0 + 127
// against its columns c0 .. c0 + 127 (tile-local), over the Q4_0 blocks
// b0 .. b1 - 1 of K.  NTH threads (4 or 8 waves) stage each half block (16 k)
// of x and of the dequantised weights in LDS; the waves split the tile 2 x 2
// (64 x 64 each, 2 x 2 products of 32 x 32) or, with eight waves, 4 x 2
// (32 x 64 each, 1 x 2 products), which keeps the fallback's registers few
// where it is inlined into a large kernel.
template <int NTH, typename IO>
__device__ __forceinline__ void exact_tile128(const IO& io, const void* x, DType xt, int64_t ldx,
                                              const uint8_t* W, int64_t rb, int r0, int c0, int64_t b0,
                                              int64_t b1, float* lds, int chunk_rows = 128,
                                              int chunk_mask = 0, uint32_t chunks = ~0u) {
  static_assert(NTH == 256 || NTH == 512, "four or eight waves");
  constexpr int WVM = NTH == 512 ? 4 : 2;  // waves along the rows
  constexpr int TI = 4 / WVM;              // 32-row products per wave
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  float* As = lds;
  float* Bs = lds + 128 * kExLd;
  float16_t acc[TI][2];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
#pragma unroll 1
  for (int64_t b = b0; b < b1; ++b) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      __syncthreads();  // the previous half's operand reads are done
      for (int e = tid; e < 128 * 16; e += NTH) {
        const int r = e >> 4, j = e & 15;
        As[r * kExLd + j] =
            io.row_in(r0 + r) ? load_x_f32(x, xt, io.xrow_in(r0 + r) * ldx + kQK * b + 16 * h + j) : 0.0f;
        float w = 0.0f;
        if (io.col_in(c0 + r)) {
          const uint8_t* blk = W + io.wrow_in(c0 + r) * rb + b * kBlockBytes;
          const float d = half_bits_to_float(static_cast<uint16_t>(blk[0] | (blk[1] << 8)));
          const int q = (blk[2 + j] >> (4 * h)) & 0xF;
          w = static_cast<float>(q - 8) * d;
        }
        Bs[r * kExLd + j] = w;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int kc = 2 * kk + (lane >> 5);  // lane l supplies k = l / 32 of the pair
        float a[TI], bv[2];
#pragma unroll
        for (int i = 0; i < TI; ++i)
          a[i] = As[(wm * 32 * TI + 32 * i + (lane & 31)) * kExLd + kc];
#pragma unroll
        for (int j = 0; j < 2; ++j) bv[j] = Bs[(wn * 64 + 32 * j + (lane & 31)) * kExLd + kc];
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], bv[j], acc[i][j], 0, 0, 0);
      }
    }
  }
  // 32 x 32 accumulator layout: lane l holds column l % 32; register r holds
  // row 8 (r / 4) + 4 (l / 32) + r % 4.
  if constexpr (IO::kPlain) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          io.store1(r0 + wm * 32 * TI + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + (r & 3),
                    c0 + wn * 64 + 32 * j + (lane & 31), acc[i][j][r]);
  } else {
    // Stores the rows whose chunk (row / chunk_rows & chunk_mask) is asked for.
    const auto cols = io.template columns<128>(c0, threadIdx.x % (IO::kPairs ? 8 : 16));
    constexpr int kGroups = IO::kPairs ? 8 : 16;
    const int g = threadIdx.x % kGroups, at = IO::kPairs ? 64 * (g >> 2) + 8 * (g & 3) : 8 * g;
    each_chunk<0, TI>([&](auto ic) {
      constexpr int q = decltype(ic)::value;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          lds[(wm * 32 + 8 * (r / 4) + 4 * (lane >> 5) + (r & 3)) * 132 + wn * 64 + 32 * j + (lane & 31)] =
              acc[q][j][r];
      __syncthreads();
#pragma unroll 1
      for (int r = tid / kGroups; r < 32 * WVM; r += NTH / kGroups) {
        const int row = r0 + (r >> 5) * 32 * TI + 32 * q + (r & 31);
        if ((chunks >> ((row / chunk_rows) & chunk_mask)) & 1) io.template emit<false>(cols, lds + r * 132 + at, row);
      }
    });
  }
}

// A BMT x BNT tile (BNT a multiple of 128) on the exact route, 128 x 128 at a time.
template <int NTH, int BMT, int BNT, typename IO>
__device__ __forceinline__ void exact_tile(const IO& io, const void* x, DType xt, int64_t ldx,
                                           const uint8_t* W, int64_t rb, int64_t b0, int64_t b1,
                                           float* lds, int chunk_rows, int chunk_mask,
                                           uint32_t chunks) {
#pragma unroll 1
  for (int ti = 0; ti < (BMT + 127) / 128; ++ti)
#pragma unroll 1
    for (int tj = 0; tj < BNT / 128; ++tj)
      exact_tile128<NTH>(io, x, xt, ldx, W, rb, 128 * ti, 128 * tj, b0, b1, lds, chunk_rows,
                         chunk_mask, chunks);
}

// Stores the workgroup's WVM x WVN waves' TM x TN products of 32 x 32.  32 x 32
// accumulator layout: lane l holds column l % 32; register r holds row
// 8 * (r / 4) + 4 * (l / 32) + r % 4.  A non-finite accumulator anywhere in the
// workgroup: exact(chunks) writes the tile's outputs; a plain product overwrites
// what it stored, a fused one has left out the chunks asked for.
template <int WVM, int WVN, int TM, int TN, typename IO, typename F>
__device__ __forceinline__ void store_tile(const IO& io, const float16_t (&acc)[TM][TN], uint8_t* lds,
                                           F exact, int live = TM) {
  const int wave = threadIdx.x >> 6;
  const int wm = wave / WVN, wn = wave % WVN;
  const int r0 = wm * 32 * TM, c0 = wn * 32 * TN;
  const int lane = threadIdx.x & 63, kg = lane >> 5;
  if constexpr (IO::kPlain) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float v = acc[i][j][r];
          bad |= !__builtin_isfinite(v);
          io.store1(r0 + 32 * i + 8 * (r / 4) + 4 * kg + (r & 3), c0 + 32 * j + (lane & 31), v);
        }
    if (workgroup_any_flag(bad, reinterpret_cast<uint32_t*>(lds))) exact(~0u);
  } else {
    constexpr int LD = 32 * TN * WVN + 4;
    float* buf = reinterpret_cast<float*>(lds);
    const uint32_t skipped = fused_epilogue<TM, WVM * WVN * 64, 32 * TN * WVN, 32 * WVM, true>(
        io, buf, 0,
        [&](auto ic) {
          bool odd = false;
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const float v = acc[decltype(ic)::value][j][r];
              odd |= !__builtin_isfinite(v);
              buf[(wm * 32 + 8 * (r / 4) + 4 * kg + (r & 3)) * LD + c0 + 32 * j + (lane & 31)] = v;
            }
          return odd;
        },
        [&](int i, int r) {
          return IO::kDealt ? 32 * WVM * i + r : (r >> 5) * 32 * TM + 32 * i + (r & 31);
        },
        live);
    if (skipped != 0) exact(skipped);
  }
}

// The generic tile for k % 64 != 0: 128 x 128, both operands staged as fp16 in
// padded LDS rows, one block of k per step, two barriers per step.
template <typename IO>
__device__ __forceinline__ void gemm_tile_body(IO io, const half_t* __restrict__ x,
                                               const uint8_t* __restrict__ W, int64_t k,
                                               const void* __restrict__ xe, int xet) {
  // xe / xet: the original activations, for the exact route.
  constexpr int kTileLds = IO::kPlain ? (2 * BM * LDK * 2 > kExLdsBytes ? 2 * BM * LDK * 2 : kExLdsBytes)
                                      : 64 * 132 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t tsm[kTileLds];
  half_t (*As)[LDK] = reinterpret_cast<half_t (*)[LDK]>(tsm);
  half_t (*Bs)[LDK] = reinterpret_cast<half_t (*)[LDK]>(tsm + BM * LDK * 2);

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wid = t >> 6;
  const int wm = wid >> 1;  // 2 x 2 waves, 64 x 64 each
  const int wn = wid & 1;
  if (!io.template begin<BM, BN>()) return;
  W = io.weights(W);
  const int64_t nb = k / kQK;

  float16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int lr = t >> 1;          // tile row this thread stages
  const int lh = t & 1;           // which half of the 32-wide k step
  const bool lrow = io.row_in(lr), lcol = io.col_in(lr);
  const half_t* const lx = x + io.xrow(lr) * k;
  const uint8_t* const lw = W + io.wrow(lr) * nb * kBlockBytes;

  for (int64_t kb = 0; kb < nb; ++kb) {
    // Activations: 16 halves per thread.
    {
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (lrow) {
        const uint4* src = reinterpret_cast<const uint4*>(lx + kb * kQK + lh * 16);
        v0 = src[0];
        v1 = src[1];
      }
      *reinterpret_cast<uint4*>(&As[lr][lh * 16]) = v0;
      *reinterpret_cast<uint4*>(&As[lr][lh * 16 + 8]) = v1;
    }
    // Weights: half a block per thread, dequantised to fp16.
    {
      half_t lo[8], hi[8];
      if (lcol) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(lw + kb * kBlockBytes);
        const float d = half_bits_to_float(p[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t c = p[1 + 4 * lh + i];  // code bytes 8lh+2i, 8lh+2i+1
          lo[2 * i] = static_cast<half_t>(static_cast<float>(static_cast<int>(c & 0xFu) - 8) * d);
          lo[2 * i + 1] = static_cast<half_t>(static_cast<float>(static_cast<int>((c >> 8) & 0xFu) - 8) * d);
          hi[2 * i] = static_cast<half_t>(static_cast<float>(static_cast<int>((c >> 4) & 0xFu) - 8) * d);
          hi[2 * i + 1] = static_cast<half_t>(static_cast<float>(static_cast<int>((c >> 12) & 0xFu) - 8) * d);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) { lo[i] = 0; hi[i] = 0; }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Bs[lr][8 * lh + i] = lo[i];
        Bs[lr][16 + 8 * lh + i] = hi[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      half8_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[i] = *reinterpret_cast<const half8_t*>(&As[wm * 64 + i * 32 + (lane & 31)][ks + 8 * (lane >> 5)]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b[j] = *reinterpret_cast<const half8_t*>(&Bs[wn * 64 + j * 32 + (lane & 31)][ks + 8 * (lane >> 5)]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }

  store_tile<2, 2>(io, acc, tsm, [&](uint32_t chunks) {
    exact_tile128<256>(io, xe, static_cast<DType>(xet), k, W, nb * kBlockBytes, 0, 0, 0, nb,
                       reinterpret_cast<float*>(tsm), 32, 1, chunks);
  });
}

// ------------------------------------------------------------------ tiled

constexpr int kBK = 64;            // k per step: two Q4_0 blocks
constexpr int kRowBytes16 = 128;   // one tile row of 64 fp16 = 8 pieces of 16 bytes

// Swizzle key of LDS row r (128-byte rows of eight 16-byte pieces): piece c
// of row r sits at r * 8 + (c ^ key(r)).  Sixteen consecutive rows reading
// one piece column land in sixteen distinct 16-byte bank groups of a 256-byte
// bank window (rows r and r + 8 differ in the key's low bit), and any eight
// consecutive rows in eight distinct groups of a 128-byte window.
__device__ __forceinline__ int swz_key(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz(int r, int c) { return r * 8 + (c ^ swz_key(r)); }

// One weight unit: one block of a row (scale and 16 code bytes) as the
// 20-byte aligned window w0..w4 that contains it.
struct WUnit {
  u32x4 w;     // w0 .. w3
  uint32_t w4;
};

template <int BM, int BN, int WVM, int WVN, typename IO>
__device__ __forceinline__ void gemm_mfma_body(IO io, const half_t* __restrict__ x,
                                               const uint8_t* __restrict__ W, int64_t k, int kps,
                                               const void* __restrict__ xe, int xet) {
  // k: full K (row strides).  Workgroups with blockIdx.z = z take the K steps
  // z kps .. min((z + 1) kps, k / 64) - 1 (a split-K partial when
  // gridDim.z > 1).  xe / xet: the original activations, for the exact route.
  constexpr int NTH = WVM * WVN * 64;       // threads
  constexpr int WM = BM / WVM, WN = BN / WVN;  // wave tile
  constexpr int TM = WM / 32, TN = WN / 32; // 32 x 32 products per wave
  constexpr int A_STAGE = BM * kRowBytes16;
  constexpr int B_STAGE = BN * kRowBytes16;
  constexpr int STAGE = A_STAGE + B_STAGE;
  constexpr int A_COPIES = BM * 8 / NTH;    // 16-byte copies per thread per step
  constexpr int UNITS = BN * 2 / NTH;       // weight units (blocks) per thread per step
  static_assert(A_COPIES >= 1 && UNITS >= 1, "tile too small");
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave / WVN, wn = wave % WVN;
  if (!io.template begin<BM, BN>()) return;
  W = io.weights(W);
  const int64_t rb = (k / kQK) * kBlockBytes;
  const int ks0 = static_cast<int>(blockIdx.z) * kps;
  const int nks_all = static_cast<int>(k / kBK);
  const int nks = nks_all - ks0 < kps ? nks_all - ks0 : kps;
  const uint8_t* const W0 = W;
  x += static_cast<int64_t>(ks0) * kBK;
  W += static_cast<int64_t>(ks0) * 2 * kBlockBytes;

  // Activation copies: copy i of this thread is LDS piece P = NTH i + tid
  // (row P / 8, swizzled column P % 8); the source column undoes the swizzle.
  const half_t* asrc[A_COPIES];
#pragma unroll
  for (int i = 0; i < A_COPIES; ++i) {
    const int P = NTH * i + tid;
    const int r = P >> 3;
    const int c = (P & 7) ^ swz_key(r);
    asrc[i] = x + io.xrow(r) * k + 8 * c;
  }
  auto issue_a = [&](int ks, int stage) {
    uint8_t* dst = smem + stage * STAGE;
#pragma unroll
    for (int i = 0; i < A_COPIES; ++i)
      dma16(asrc[i] + static_cast<int64_t>(ks) * kBK, dst + (NTH * i + 64 * wave) * 16);
  };

  // Weight units: unit u of this thread is U = NTH u + tid: row U / 2, block
  // U % 2 of the step.  A step is 36 bytes of the row starting 4-byte aligned
  // (rows are 36-byte multiples here); block 0's window is its first 20
  // bytes, block 1's the last 20, so both stay inside the step.  In the window
  // the scale is at byte 2b and code byte c at 2 + 2b + c.
  const uint8_t* wsrc[UNITS];
  uint32_t sel_even[UNITS], sel_odd[UNITS], dshift[UNITS];
  int wrow[UNITS], wblk[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int U = NTH * u + tid;
    const int r = U >> 1;
    const int b = U & 1;
    wsrc[u] = W + io.wrow(r) * rb + 16 * b;  // + 36 per step
    // code pair i' (bytes 8h + 2i', +1) sits at byte 2 + 2b + 2 (i' & 1) of
    // the dword pair {w[2h + i'/2 + 1] : w[2h + i'/2]}; selectors give [c, 0, c', 0]
    const uint32_t s0 = static_cast<uint32_t>(2 + 2 * b);
    const uint32_t s1 = s0 + 2;
    sel_even[u] = s0 | (0x0cu << 8) | ((s0 + 1) << 16) | (0x0cu << 24);
    sel_odd[u] = s1 | (0x0cu << 8) | ((s1 + 1) << 16) | (0x0cu << 24);
    dshift[u] = 16u * b;
    wrow[u] = r;
    wblk[u] = b;
  }
  // Untracked loads of the packed bytes of step ks (see load_dwordx4_untracked).
  struct Units {
    WUnit v[UNITS];
  };
  auto load_units = [&](int ks) {
    Units r;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint8_t* src = wsrc[u] + static_cast<int64_t>(ks) * 2 * kBlockBytes;
      r.v[u].w = load_dwordx4_untracked(src);
      r.v[u].w4 = load_dword_untracked(src + 16);
    }
    return r;
  };
  auto tie_units = [&](Units& r) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      tie_after(r.v[u].w);
      tie_after(r.v[u].w4);
    }
  };

  const UnpackConsts kc = make_unpack_consts();
  // Dequantise half h of unit u (16 weights) and store its two pieces into
  // `stage`: codes 8h .. 8h+7 give k 8h .. 8h+7 (low nibbles, piece 4b + h)
  // and k 16 + 8h .. (high nibbles, piece 4b + h + 2).
  auto dequant_half = [&](const WUnit& un, int u, int h, int stage) {
    const uint32_t w[5] = {un.w[0], un.w[1], un.w[2], un.w[3], un.w4};
    const uint32_t dbits = (w[0] >> dshift[u]) & 0xFFFFu;
    const half2_t d2 = __builtin_bit_cast(half2_t, dbits | (dbits << 16));
    const half2_t klo = {static_cast<half_t>(-1032.0f), static_cast<half_t>(-1032.0f)};
    const half2_t khi = {static_cast<half_t>(-72.0f), static_cast<half_t>(-72.0f)};
    uint8_t* bs = smem + stage * STAGE + A_STAGE;
    u32x4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = __builtin_amdgcn_perm(w[2 * h + i / 2 + 1], w[2 * h + i / 2],
                                               (i & 1) ? sel_odd[u] : sel_even[u]);
      const half2_t ql = __builtin_bit_cast(half2_t, (t & kc.mask_lo) | kc.exp_lo) + klo;
      const half2_t qh = __builtin_bit_cast(half2_t, (t & kc.mask_hi) | kc.exp_hi) + khi;
      lo[i] = __builtin_bit_cast(uint32_t, ql * d2);
      hi[i] = __builtin_bit_cast(uint32_t, qh * d2);
    }
    *reinterpret_cast<u32x4*>(bs + swz(wrow[u], 4 * wblk[u] + h) * 16) = lo;
    *reinterpret_cast<u32x4*>(bs + swz(wrow[u], 4 * wblk[u] + h + 2) * 16) = hi;
  };

  float16_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Every vector-memory operation in the loop is untracked by the compiler
  // (LDS copies and register loads); each step ends with one explicit drain.
  // Prologue: stage 0 complete, packed weights of step 1 in registers.
  issue_a(0, 0);
  {
    Units u0 = load_units(0);
    wait_vm<0>();
    tie_units(u0);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      dequant_half(u0.v[u], u, 0, 0);
      dequant_half(u0.v[u], u, 1, 0);
    }
  }
  Units nxt = load_units(nks > 1 ? 1 : 0);
  wait_vm<0>();
  tie_units(nxt);
  __syncthreads();

  const int arow = wm * WM + (lane & 31);
  const int brow = wn * WN + (lane & 31);
  const int kg = lane >> 5;

  // Operand fragments of k16 sub-step kk of a stage (lane: row arow / brow,
  // 8 k-values 8 kg .. 8 kg + 7 of the sub-step).
  auto read_frags = [&](const uint8_t* as, int kk, half8_t (&af)[TM], half8_t (&bf)[TN]) {
    const uint8_t* bs = as + A_STAGE;
#pragma unroll
    for (int i = 0; i < TM; ++i)
      af[i] = *reinterpret_cast<const half8_t*>(as + swz(arow + 32 * i, 2 * kk + kg) * 16);
#pragma unroll
    for (int j = 0; j < TN; ++j)
      bf[j] = *reinterpret_cast<const half8_t*>(bs + swz(brow + 32 * j, 2 * kk + kg) * 16);
  };
  // Interleave the matrix products of a sub-step with the next sub-step's
  // operand reads and the dequantisation (one MFMA, one LDS read, two VALU).
  auto interleave = [](auto with_reads) {
    constexpr bool R = decltype(with_reads)::value;
#pragma unroll
    for (int i = 0; i < TM * TN; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      if (R && i < TM + TN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // VALU
    }
  };

  if constexpr (TM * TN <= 4) {
    // Small wave tiles (one wave per SIMD): few products per k16 sub-step
    // cannot cover an LDS read, so all four sub-steps' fragments of a stage
    // are read right after its barrier and the products then run back to
    // back, with the dequantisation interleaved.
    half8_t fa[4][TM], fb[4][TN];
    auto read_all = [&](const uint8_t* as) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) read_frags(as, kk, fa[kk], fb[kk]);
    };
    auto interleave_valu = []() {
#pragma unroll
      for (int i = 0; i < TM * TN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // VALU
      }
    };
    read_all(smem);
    for (int ks = 0; ks < nks; ++ks) {
      const int st = ks & 1;
      issue_a(ks + 1 < nks ? ks + 1 : ks, st ^ 1);
      const Units cur = nxt;
      nxt = load_units(ks + 2 < nks ? ks + 2 : nks - 1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[kk][i], fb[kk][j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
          for (int h = 0; h < 2; ++h)
            if ((2 * u + h) % 4 == kk) dequant_half(cur.v[u], u, h, st ^ 1);
        interleave_valu();
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vm<0>();
      tie_units(nxt);
      __syncthreads();
      read_all(smem + (st ^ 1) * STAGE);
    }
  } else {
    half8_t af[2][TM], bf[2][TN];
    read_frags(smem, 0, af[0], bf[0]);
    for (int ks = 0; ks < nks; ++ks) {
      const int st = ks & 1;
      // Activations of step ks + 1 into the other stage (the last step copies
      // its own again: that stage is no longer read).
      issue_a(ks + 1 < nks ? ks + 1 : ks, st ^ 1);
      const Units cur = nxt;
      nxt = load_units(ks + 2 < nks ? ks + 2 : nks - 1);
      const uint8_t* as = smem + st * STAGE;
  #pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // 16-wide k sub-steps
        const int c = kk & 1;
        if (kk < 3) read_frags(as, kk + 1, af[c ^ 1], bf[c ^ 1]);
  #pragma unroll
        for (int i = 0; i < TM; ++i)
  #pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[c][i], bf[c][j], acc[i][j], 0, 0, 0);
        // The next step's weights (on the last step: a harmless rewrite of the
        // stage no longer read).
  #pragma unroll
        for (int u = 0; u < UNITS; ++u)
          for (int h = 0; h < 2; ++h)
            if ((2 * u + h) % 4 == kk) dequant_half(cur.v[u], u, h, st ^ 1);
        if (kk < 3) interleave(IC<true>{});
        else interleave(IC<false>{});
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vm<0>();
      tie_units(nxt);
      __syncthreads();
      read_frags(smem + (st ^ 1) * STAGE, 0, af[0], bf[0]);
    }
  }

  // (Storing y transposed from swapped operands, four columns per 8-byte
  // store, measured slower: each store then touches 32 rows.)
  store_tile<WVM, WVN>(io, acc, smem, [&](uint32_t chunks) {
    exact_tile<NTH, BM, BN>(io, xe, static_cast<DType>(xet), k, W0, rb, 2 * static_cast<int64_t>(ks0),
                            2 * static_cast<int64_t>(ks0 + nks), reinterpret_cast<float*>(smem), 32, TM - 1,
                            chunks);
  });
}

// ------------------------------------------------------------------ slice-K
//
// 128 x 128 output tile, four waves, k % 256 == 0.  Wave w owns the whole
// tile for the k16 slice w of every 64-wide k step: k 16w .. 16w+15, which is
// one nibble half (w & 1) of block w >> 1 of the step.  Every activation and
// weight element is therefore read from LDS by one wave only and dequantised
// once, and a wave's operand fragments per step are four of each (against
// eight for a 2 x 2 split of the tile).  The four partial tiles are summed in
// wave order at the end.
//
// Copies (global -> LDS, 16-byte pieces, issued by all waves):
//   - activations: a ring of six 64-wide k stages, stage of step ks = ks % 6,
//     refilled five steps ahead;
//   - packed weights: the 144 bytes of each row that cover four steps (256 k,
//     16-byte aligned because k % 256 == 0), a ring of three, refilled three
//     segments ahead.
// Per step: issue copies, read the next step's activation fragments and the
// raw weights of the step after, run this step's 16 matrix products
// interleaved with those reads and with the dequantisation of the next
// step's weights (read one step earlier, so no arithmetic waits on a fresh
// LDS read), then one barrier once the copies the next step reads have
// landed.
constexpr int kSkAStage = 128 * kRowBytes16;        // 16 KB
constexpr int kSkSeg = 4 * 2 * kBlockBytes;         // 144 packed bytes per row and 4 steps
constexpr int kSkWStage = 128 * kSkSeg;             // 18 KB
constexpr int kSkAStages = 6;
constexpr int kSkWOff = kSkAStages * kSkAStage;     // weight ring after the activation ring
constexpr int kSkLds = kSkWOff + 3 * kSkWStage;     // 150 KB
constexpr int kSkRedCol = 36;                       // floats per column of a partial (32 rows + pad)
constexpr int kSkRedBytes = 4 * 128 * kSkRedCol * 4;
static_assert(kSkRedBytes <= kSkLds, "reduction buffer");

template <typename IO>
__device__ __forceinline__ void gemm_slicek_body(IO io, const half_t* __restrict__ x,
                                                 const uint8_t* __restrict__ W, int64_t k, int kps,
                                                 const void* __restrict__ xe, int xet) {
  // k: full K (row strides).  Workgroups with blockIdx.z = z take the k steps
  // z kps .. min((z + 1) kps, k / 64) - 1 (kps % 4 == 0).
  // xe / xet: the original activations, for the exact route.
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSkLds];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = lane >> 5, lc = lane & 31;
  if (!io.template begin<128, 128>()) return;
  W = io.weights(W);
  const int64_t rb = (k / kQK) * kBlockBytes;
  const int ks0 = static_cast<int>(blockIdx.z) * kps;
  const int nks_all = static_cast<int>(k / kBK);
  const int nks = nks_all - ks0 < kps ? nks_all - ks0 : kps;  // a multiple of 4
  const int nss = nks >> 2;
  const uint8_t* const W0 = W;
  x += static_cast<int64_t>(ks0) * kBK;
  W += static_cast<int64_t>(ks0) * 2 * kBlockBytes;

  // Copies take a wave-uniform base (step ks of x's row xbase, or segment ss of
  // weight row wbase) plus a 32-bit per-lane byte offset.
  // Activation copy i of this thread: LDS piece P = 256 i + tid of a stage
  // (row P / 8, swizzled column P % 8).
  const uint32_t lds0 = lds_addr(smem);
  uint32_t aoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int P = 256 * i + tid;
    const int r = P >> 3;
    const int c = (P & 7) ^ swz_key(r);
    const int64_t rr = io.xrow(r) - io.xbase();
    aoff[i] = static_cast<uint32_t>((rr * k + 8 * c) * 2);
  }
  const half_t* const xt = x + io.xbase() * k;
  auto issue_a = [&](int ks, int stage) {
    const half_t* base = xt + static_cast<int64_t>(ks) * kBK;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dma16_sbase(aoff[i], base, lds0 + stage * kSkAStage + (256 * i + 64 * wave) * 16);
  };
  // Weight copy i of this thread: piece p of a weight stage (row p / 9, piece
  // p % 9 of its 144 bytes); 1152 pieces = four full rounds of 256 plus a
  // fifth in which each wave copies 32.
  uint32_t woff[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int p = i < 4 ? 256 * i + tid : 1024 + 32 * wave + lc;
    const int r = p / 9;
    const int c = p - 9 * r;
    const int64_t rr = io.wrow(r) - io.wbase();
    woff[i] = static_cast<uint32_t>(rr * rb + 16 * c);
  }
  const uint8_t* const wt = W + io.wbase() * rb;
  auto issue_w = [&](int ss, int buf) {
    const uint8_t* base = wt + static_cast<int64_t>(ss) * kSkSeg;
    const uint32_t dst = lds0 + kSkWOff + buf * kSkWStage;
#pragma unroll
    for (int i = 0; i < 4; ++i) dma16_sbase(woff[i], base, dst + (256 * i + 64 * wave) * 16);
    if (lane < 32) dma16_sbase(woff[4], base, dst + (1024 + 32 * wave) * 16);
  };

  // This wave's share of a step: block b = w >> 1 of the step and its code
  // bytes 8h .. 8h + 7 (h = w & 1), both nibbles.  The k order inside a
  // matrix product is free as long as both operands follow it: lane (lc, kg)
  // takes the low nibbles (kg = 0, block elements 8h .. 8h + 7) or the high
  // nibbles (kg = 1, elements 16 + 8h ..) of those bytes, and its activation
  // fragment is the matching 8 halves, piece 4b + 2kg + h of the step.  Both
  // halves of the wave read the same weight bytes (one LDS broadcast): the
  // aligned 12-byte window at step byte 16b + 8h (code byte 8h + e at window
  // byte O + e, O = 2 + 2b) and the scale as the dword at 16b (its low half
  // for b = 0, high half for b = 1).
  const int b = wave >> 1, h = wave & 1;
  const uint32_t O = 2u + 2u * static_cast<uint32_t>(b);
  const uint32_t sel_a = O | (0x0cu << 8) | ((O + 1) << 16) | (0x0cu << 24);
  const uint32_t sel_b = (O + 2) | (0x0cu << 8) | ((O + 3) << 16) | (0x0cu << 24);
  const uint32_t nib_mask = kg ? 0x00F000F0u : 0x000F000Fu;
  const uint32_t nib_exp = kg ? 0x54005400u : 0x64006400u;  // fp16 64 + q / 1024 + q
  const half_t sub1 = static_cast<half_t>(kg ? -72.0f : -1032.0f);
  const half2_t nib_sub = {sub1, sub1};
  const uint32_t dshift = 16u * static_cast<uint32_t>(b);
  const int apiece = 4 * b + 2 * kg + h;

  struct Raw {
    uint32_t w[4][3];
    uint32_t d[4];
  };
  // Fragment reads from a lane base plus compile-time offsets (stage, buffer,
  // step within the segment, fragment).  Reads past the last step are of
  // valid LDS addresses and unused.
  const uint8_t* const abase = smem + swz(lc, apiece) * 16;  // + 32 i rows: swz(32 i + lc, apiece)
  const uint8_t* const wbase = smem + kSkWOff + lc * kSkSeg + 16 * b;
  auto read_a = [&](auto stage_c, half8_t (&fa)[4]) {
    constexpr int stage = decltype(stage_c)::value;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fa[i] = *reinterpret_cast<const half8_t*>(abase + stage * kSkAStage + i * 4096);
  };
  auto read_w = [&](const uint8_t* wb, auto j_c, Raw& raw) {
    constexpr int off = 36 * decltype(j_c)::value;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const uint8_t* rp = wb + off + jj * 32 * kSkSeg;
      const uint32_t* win = reinterpret_cast<const uint32_t*>(rp + 8 * h);
      raw.w[jj][0] = win[0];
      raw.w[jj][1] = win[1];
      raw.w[jj][2] = win[2];
      raw.d[jj] = *reinterpret_cast<const uint32_t*>(rp);
    }
  };
  auto dequant = [&](const Raw& raw, half8_t (&fb)[4]) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const uint32_t db = (raw.d[jj] >> dshift) & 0xFFFFu;
      const half2_t d2 = __builtin_bit_cast(half2_t, db | (db << 16));
      const uint32_t w0 = raw.w[jj][0], w1 = raw.w[jj][1], w2 = raw.w[jj][2];
      const uint32_t t[4] = {__builtin_amdgcn_perm(w1, w0, sel_a), __builtin_amdgcn_perm(w1, w0, sel_b),
                             __builtin_amdgcn_perm(w2, w1, sel_a), __builtin_amdgcn_perm(w2, w1, sel_b)};
      u32x4 r;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const half2_t v = __builtin_bit_cast(half2_t, (t[q] & nib_mask) | nib_exp) + nib_sub;
        r[q] = __builtin_bit_cast(uint32_t, v * d2);
      }
      fb[jj] = __builtin_bit_cast(half8_t, r);
    }
  };

  float16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Prologue: copies in the order the loop's waits assume (W0 A0 W1 A1 A2
  // A3 A4 W2, as if steps -5 .. -1 had run); once A0, W0 and A1 have landed:
  // step 0's operands and step 1's raw weights.
  const int last = nks - 1;
  issue_w(0, 0);
  issue_a(0, 0);
  issue_w(1 < nss - 1 ? 1 : nss - 1, 1);
  issue_a(1 < last ? 1 : last, 1);
  issue_a(2 < last ? 2 : last, 2);
  issue_a(3 < last ? 3 : last, 3);
  issue_a(4 < last ? 4 : last, 4);
  issue_w(2 < nss - 1 ? 2 : nss - 1, 2);
  wait_vm_lgkm0<17>();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
  half8_t fa[4], fb[4];
  Raw rc;  // raw weights of step ks + 1
  {
    Raw r0;
    read_a(IC<0>{}, fa);
    read_w(wbase, IC<0>{}, r0);
    read_w(wbase, IC<1>{}, rc);
    dequant(r0, fb);
  }
  // (step 0 refills stage 5, which nothing has read: no barrier needed here)

  // Step ks = 4 ss + j works on operands in registers and, for the steps
  // ahead, reads step ks + 1's activation fragments and step ks + 2's raw
  // weights and dequantises step ks + 1's.  Copies: A(ks + 5) into stage
  // (ks - 1) % 6, and at j = 3, after it, weight segment ss + 3 into buffer
  // ss % 3.  Both were last read a step before this one and those reads were
  // consumed (by step ks - 1's products, by this step's predecessor's
  // dequantisation) before the last barrier, so no wave waits for its LDS
  // reads at a barrier.  The wait is for A(ks + 2), which step ks + 1 reads:
  // issued at step ks - 3, it has the three later activation copies and
  // exactly one weight segment (every four steps issue one) behind it, 17
  // copies.  Copies retire in order, so every weight segment older than it
  // (among them the one step ks + 1 reads) has landed too; an activation
  // copy issued right after a weight segment is due four steps later.
  // Twelve steps (three segments) per loop trip, so that every stage and
  // buffer index is a constant: with ss = 3 q + sr, step ks = 4 ss + j has
  // stage (4 sr + j) % 6 and reads weight buffers sr and (sr + 1) % 3.
  auto step = [&](auto j_c, auto sr_c, int ss) {
    constexpr int j = decltype(j_c)::value;
    constexpr int sr = decltype(sr_c)::value;
    constexpr int sa = (4 * sr + j) % kSkAStages;                   // stage of step ks
    constexpr int sn = (sa + 1) % kSkAStages;                       // of step ks + 1
    constexpr int sp = (sa + kSkAStages - 1) % kSkAStages;          // of step ks - 1
    constexpr int wcur = sr, wnext = (sr + 1) % 3;
    const int ks = 4 * ss + j;
    issue_a(ks + 5 < last ? ks + 5 : last, sp);
    if constexpr (j == 3) issue_w(ss + 3 < nss - 1 ? ss + 3 : nss - 1, wcur);
    half8_t na[4], nb[4];
    Raw rn;
    read_a(IC<sn>{}, na);
    read_w(wbase + (j < 2 ? wcur : wnext) * kSkWStage, IC<(j + 2) & 3>{}, rn);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        acc[i][jj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[jj], acc[i][jj], 0, 0, 0);
    dequant(rc, nb);
    // each product followed by one fragment read and a share of the
    // dequantisation
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);  // VALU
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tie_after(nb[i]);  // dequantised within this step, not sunk into the next
      fa[i] = na[i];
      fb[i] = nb[i];
    }
    rc = rn;
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<17>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    compiler_fence();
  };
  auto segment = [&](auto sr_c, int ss) {
    step(IC<0>{}, sr_c, ss);
    step(IC<1>{}, sr_c, ss);
    step(IC<2>{}, sr_c, ss);
    step(IC<3>{}, sr_c, ss);
  };
  int ss = 0;
  for (; ss + 3 <= nss; ss += 3) {
    segment(IC<0>{}, ss);
    segment(IC<1>{}, ss + 1);
    segment(IC<2>{}, ss + 2);
  }
  if (ss < nss) segment(IC<0>{}, ss);
  if (ss + 1 < nss) segment(IC<1>{}, ss + 1);
  wait_vm_lgkm0<0>();
  __syncthreads();

  // Sum the four partial tiles, one 32-row fragment row at a time: each wave
  // writes its partial column-major (column stride kSkRedCol floats), then
  // thread t sums the 4 x 4 block of rows 4 (t % 8) .. + 3 and columns
  // 4 (t / 8) .. + 3 in wave order and stores each row's 4 columns with one
  // 8-byte (fp16) or 16-byte (fp32) store; a store instruction costs about
  // as much as a copy, so per-element stores made this epilogue several
  // microseconds long.
  float* red = reinterpret_cast<float*>(smem);
  const int rb4 = tid & 7, cb4 = tid >> 3;
  auto exact = [&](uint32_t chunks) {
    exact_tile128<256>(io, xe, static_cast<DType>(xet), k, W0, rb, 0, 0, 2 * static_cast<int64_t>(ks0),
                       2 * static_cast<int64_t>(ks0 + nks), reinterpret_cast<float*>(smem), 32, 3, chunks);
  };
  // One 32-row chunk: the waves' partials column-major, then their sums
  // (columns 4 cb4 .. + 3, rows 4 rb4 .. + 3 of the chunk).
  auto put = [&](const float16_t (&a)[4]) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float4_t v = {a[jj][4 * q], a[jj][4 * q + 1], a[jj][4 * q + 2], a[jj][4 * q + 3]};
        *reinterpret_cast<float4_t*>(red + (wave * 128 + 32 * jj + lc) * kSkRedCol + 8 * q + 4 * kg) = v;
      }
  };
  auto sum4 = [&](float4_t (&sc)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) sc[c] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        sc[c] += *reinterpret_cast<const float4_t*>(red + (w * 128 + 4 * cb4 + c) * kSkRedCol + 4 * rb4);
  };
  if constexpr (IO::kPlain) {
    bool bad = false;  // a non-finite sum (then the exact route rewrites the tile)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      put(acc[i]);
      __syncthreads();
      float4_t sc[4];
      sum4(sc);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) bad |= !__builtin_isfinite(sc[c][r]);
      io.store4x4(32 * i + 4 * rb4, 4 * cb4, sc);
      __syncthreads();
    }
    if (workgroup_any_flag(bad, reinterpret_cast<uint32_t*>(smem))) exact(~0u);
  } else {
    static_assert(kSkRedBytes + 32 * 132 * 4 <= kSkLds, "sums behind the partials");
    float* buf = red + kSkRedBytes / 4;
    const uint32_t skipped = fused_epilogue<4, 256, 128, 32, true>(
        io, buf, 0,
        [&](auto ic) {
          put(acc[decltype(ic)::value]);
          __syncthreads();
          float4_t sc[4];
          sum4(sc);
          bool odd = false;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) odd |= !__builtin_isfinite(sc[c][r]);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *reinterpret_cast<float4_t*>(buf + (4 * rb4 + r) * 132 + 4 * cb4) =
                float4_t{sc[0][r], sc[1][r], sc[2][r], sc[3][r]};
          return odd;
        },
        [&](int i, int r) { return 32 * i + r; });
    if (skipped != 0) exact(skipped);
  }
}

}  // namespace
}  // namespace q4
