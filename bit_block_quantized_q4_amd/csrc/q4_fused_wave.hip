// Products of up to 16 rows of which every wavefront streams weight rows by
// itself: those of experts, and dense ones of few weight rows.
//
// An expert's matrix is small (a few MB) and a batch reaches many, so a
// workgroup that fills, drains and reduces for every few rows of one spends
// its time starting and stopping.  Here a workgroup stages its tile's rows of
// x in LDS once, and each wavefront then takes 16 weight rows over all of K
// (with a gate 8 gate rows and their 8 up rows in turn) after another through
// a private ring of LDS slots, one chunk of 8 blocks (144 bytes a row) each:
// no barrier, no sum between wavefronts, and the copies of the next rows are
// under way while the last chunks of these are multiplied.  Per block one
// v_mfma_f32_16x16x32_f16 with up to 16 rows of x against 16 weight rows, the
// codes as exact fp16 q - 8 and the block scale d applied in fp32, as in the
// decode GEMV (bound by the packed weights; at most about 7 TB/s by the 18
// vector instructions per block).  64 tokens over 128 experts of 1536 x 2048 and
// 2048 x 768, eight each: 54.6 + 31.6 us, 3.9 TB/s.
#include <cmath>

#include "q4_wave_stream.hpp"

namespace q4 {
namespace {

constexpr int kLdsMax = 160 * 1024;

struct WaveArgs {
  Epi ep;
  Rows rows;
  int64_t nout;   // output columns
  int blocks_per; // workgroups per tile
  int cap;        // rows staged at a time (a tile of more takes several passes)
};

// kNW wavefronts, each with kRing chunks in flight.  XB: x is bf16; a staged
// row is turned into fp16 in LDS, multiplied by the power of two that brings
// its largest magnitude to [2^15, 2^16) (as stage_bf16_kernel does).
template <int kNW, int kRing, bool GATED, bool SHIFT, bool XB>
__global__ __launch_bounds__(kNW * kWave) void fused_wave_kernel(const half_t* __restrict__ x,
                                                                 const uint8_t* __restrict__ W, int64_t k,
                                                                 WaveArgs a) {
  constexpr int kCols = GATED ? 8 : 16;  // output columns per row tile
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tile = blockIdx.x / a.blocks_per;
  const int part = blockIdx.x - tile * a.blocks_per;
  const int* const rec = a.rows.recs + static_cast<int64_t>(tile) * a.rows.rec_words;
  const int4 head = *reinterpret_cast<const int4*>(rec);
  const int pairs = rec[4 + (lane & 15)];  // (all three loads in flight)
  if (tile >= *a.rows.ntiles) return;
  const int count = head.z;
  W += head.x * a.rows.wstride;
  const int64_t boff = head.x * a.rows.nbias;
  // This wavefront's row tiles: t, t + kNW, ... of the workgroup's share.
  const int64_t all = (a.nout + kCols - 1) / kCols;
  const int64_t t_end = all * (part + 1) / a.blocks_per;
  const int64_t t_begin = all * part / a.blocks_per + wave;
  const int ntiles = t_begin < t_end ? static_cast<int>((t_end - t_begin + kNW - 1) / kNW) : 0;
  // LDS: staged rows, their factors, the wavefronts' rings.
  const int xpieces = static_cast<int>(k / 8), xstride = xpieces + 1;
  const int xbytes = a.cap * xstride * 16;
  float* const factors = reinterpret_cast<float*>(smem + xbytes);
  const int ring_at = xbytes + 64 + wave * (kRing * slot_bytes<SHIFT>);
  const int r = lane & 15, g = lane >> 4;

#pragma unroll 1
  for (int r0 = 0; r0 < count; r0 += a.cap) {  // one pass but for a token that names an expert often
    const int m = count - r0 < a.cap ? count - r0 : a.cap;
    if (r0 > 0) __syncthreads();  // the rows staged before have been read
    // Lane l < 16 knows row l: its pair and x row.
    const int pair = __shfl(pairs, (r0 + lane) & 15);
    const int xrow = lane < m ? pair / a.rows.xdiv : 0;
    // Stage x: position i of the area is piece i % xstride of row i / xstride.
    const int positions = m * xstride;
    for (int i0 = wave * kWave; i0 < positions; i0 += kNW * kWave) {
      const int i = i0 + lane;
      const int ar = i / xstride;
      const int pc = i - ar * xstride;
      const int64_t row = __shfl(xrow, ar & 15);
      if (i < positions && pc < xpieces) dma16(x + row * k + 8 * pc, smem + static_cast<int64_t>(i0) * 16);
    }
    int yr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) yr[e] = __shfl(pair, 4 * g + e);
    RowStream<kRing, GATED, SHIFT> stream;
    stream.begin(smem, ring_at, W, k, a.nout, a.ep.half, t_begin, kNW, ntiles);
    // x (issued before the ring's copies) has landed; the barrier extends that to
    // every wavefront.
    wait_vm_upto<kCopies * kRing>(stream.prologue());
    __builtin_amdgcn_s_barrier();
    compiler_fence();
    float sc[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (XB) {
      for (int row = wave; row < m; row += kNW) {
        const float f = stage_row_bf16(reinterpret_cast<u32x4*>(smem + row * xstride * 16), xpieces);
        if (lane == 0) factors[row] = f;
      }
      wait_lgkm0();
      __builtin_amdgcn_s_barrier();
      compiler_fence();
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[e] = factors[4 * g + e < m ? 4 * g + e : 0];
    }
    // Rows past m read row m - 1 (their sums are not stored).
    stream.run(smem + (r < m ? r : m - 1) * xstride * 16 + 8 * g, [&](int64_t t, const float4_t& acc) {
      const int64_t c = t * kCols + (GATED ? r >> 1 : r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = acc[e] * sc[e];
        const float u = GATED ? __shfl_xor(z, 1) : 0.f;
        if (4 * g + e < m && c < a.nout && (!GATED || (r & 1) == 0)) finish_store(a.ep, boff, yr[e], c, z, u);
      }
    });
  }
}

// Dense products whose row tiles are few (a decode layer's narrower linears): a
// workgroup takes one row tile, its wavefronts a part of k each (whole chunks),
// with the part's pieces of x, and their sums are added in the order of the
// parts.  Nearly the whole matrix is then in flight at once, and no phase waits
// for the slowest wavefront.  bf16: every wavefront scales its part of a row.
constexpr int kSplitWaves = 8, kSplitRing = 3;

struct SplitArgs {
  Epi ep;
  int m;
};

template <bool GATED, bool SHIFT, bool XB>
__global__ __launch_bounds__(kSplitWaves * kWave) void fused_split_kernel(const half_t* __restrict__ x,
                                                                          const uint8_t* __restrict__ W,
                                                                          int64_t k, SplitArgs a) {
  constexpr int kCols = GATED ? 8 : 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int waves = blockDim.x / kWave;
  const int nch = static_cast<int>((k / kQK + kChunk - 1) / kChunk);
  const int c0 = nch * wave / waves, c1 = nch * (wave + 1) / waves;
  constexpr int kChunkPieces = kChunk * kQK / 8;  // of x
  const int first = c0 * kChunkPieces;
  const int np = (c1 < nch ? c1 * kChunkPieces : static_cast<int>(k / 8)) - first;
  // LDS: every wavefront's rows and ring, then the sums [wave][row][16].
  const int xstride = ((nch + waves - 1) / waves * kChunkPieces + 1) * 16;
  const int own = a.m * xstride + kSplitRing * slot_bytes<SHIFT>;
  uint8_t* const mine = smem + wave * own;
  float* const sums = reinterpret_cast<float*>(smem + waves * own);
  for (int row = 0; row < a.m; ++row)
    for (int i0 = 0; i0 < np; i0 += kWave)
      if (i0 + lane < np) dma16(x + row * k + 8 * (first + i0 + lane), mine + row * xstride + i0 * 16);
  RowStream<kSplitRing, GATED, SHIFT> stream;
  stream.begin(smem, wave * own + a.m * xstride, W, k, a.ep.ldy, a.ep.half, blockIdx.x, 1, 1);
  stream.limit(c0, c1, 1);
  wait_vm_upto<kCopies * kSplitRing>(stream.prologue());  // x, issued first, has landed
  compiler_fence();
  const int r = lane & 15, g = lane >> 4;
  float sc[4] = {1.f, 1.f, 1.f, 1.f};
  if constexpr (XB) {
    for (int row = 0; row < a.m; ++row) {
      const float f = stage_row_bf16(reinterpret_cast<u32x4*>(mine + row * xstride), np);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (row == 4 * g + e) sc[e] = f;
    }
    wait_lgkm0();
    compiler_fence();
  }
  stream.run(mine + (r < a.m ? r : a.m - 1) * xstride + 8 * g, [&](int64_t, const float4_t& acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * g + e < a.m) sums[(wave * a.m + 4 * g + e) * 16 + r] = acc[e] * sc[e];
  });
  __syncthreads();
  for (int o = threadIdx.x; o < a.m * kCols; o += blockDim.x) {
    const int row = o / kCols, c = o - row * kCols;
    const int64_t col = blockIdx.x * int64_t{kCols} + c;
    if (col >= a.ep.ldy) continue;
    float z = 0.f, u = 0.f;
    for (int w = 0; w < waves; ++w) {
      const float* p = sums + (w * a.m + row) * 16 + (GATED ? 2 * c : c);
      z += p[0];
      if constexpr (GATED) u += p[1];
    }
    finish_store(a.ep, 0, row, col, z, u);
  }
}

using KernelFn = const void*;

// Wavefronts of a row tile: as many as there are chunks, up to eight.
int split_waves(int64_t k) {
  const int64_t nch = (k / kQK + kChunk - 1) / kChunk;
  return static_cast<int>(nch < kSplitWaves ? nch : kSplitWaves);
}
int64_t split_lds(int64_t m, int64_t k, int waves) {
  const int64_t nch = (k / kQK + kChunk - 1) / kChunk;
  const int64_t xstride = ((nch + waves - 1) / waves * (kChunk * kQK / 8) + 1) * 16;
  const int64_t slot = k % 256 != 0 ? slot_bytes<true> : slot_bytes<false>;
  return waves * (m * xstride + kSplitRing * slot + m * 64);
}

// Rows staged at a time: no tile of distinct tokens has more.  (Fewer, with a
// second pass for the fuller tiles, doubles the time of the whole launch.)
int cap_rows(int64_t m) { return static_cast<int>(m < 16 ? m : 16); }

int lds_bytes(int cap, int64_t k, int nw, int ring, bool shift) {
  return static_cast<int>(cap * staged_bytes(k)) + 64 + nw * ring * (shift ? slot_bytes<true> : slot_bytes<false>);
}

template <int NW, int R>
hipError_t launch_form(const half_t* x, bool xb, const uint8_t* W, int64_t k, WaveArgs a, bool gated,
                       bool shift, int lds, int64_t grid, Queue q) {
  static const KernelFn fns[8] = {
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, false, false, false>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, false, false, true>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, false, true, false>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, false, true, true>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, true, false, false>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, true, false, true>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, true, true, false>),
      reinterpret_cast<KernelFn>(&fused_wave_kernel<NW, R, true, true, true>)};
  static std::atomic<uint64_t> allowed[8];
  const int f = (gated ? 4 : 0) + (shift ? 2 : 0) + (xb ? 1 : 0);
  void* argv[] = {&x, &W, &k, &a};
  return launch_blocks(fns[f], grid, NW * kWave, argv, static_cast<size_t>(lds), q, 1, 1, kLdsMax, &allowed[f]);
}

}  // namespace

bool fused_wave_supports(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k, int64_t x_rows) {
  if (experts == 0 || expert_tile_rows(m, topk, experts) != 16 || k > (1 << 15) ||
      !fused_gemv_supports(n, k, x_rows, experts))
    return false;
  return lds_bytes(cap_rows(m), k, 8, 3, k % 256 != 0) <= kLdsMax;
}

hipError_t launch_fused_wave(const Product& p, const Epi& ep, const Rows& rows, int64_t max_tiles,
                             Queue q) {
  const bool gated = ep.half != 0, shift = p.k % 256 != 0, xb = p.xt == DType::BF16;
  const int64_t pairs = p.m * p.topk, cu = device_cu_count();
  WaveArgs a{ep, rows, ep.ldy, 1, cap_rows(p.m)};
  // Workgroups per tile: one round of the resident workgroups over the tiles
  // that have rows (their number is only known on the device; here its mean for
  // experts chosen at random, and a tenth more: a second round for the last few
  // costs as much as a first), and no more than one row tile per wavefront.
  const double mean = static_cast<double>(p.experts) *
                      (1.0 - std::pow(1.0 - static_cast<double>(p.topk < p.experts ? p.topk : p.experts) /
                                                static_cast<double>(p.experts),
                                      static_cast<double>(p.m)));
  int64_t reached = static_cast<int64_t>(1.1 * mean) + 1;
  if (reached > pairs) reached = pairs;
  if (reached > p.experts) reached = p.experts;
  const int64_t row_tiles = (ep.ldy + (gated ? 7 : 15)) / (gated ? 8 : 16);
  const half_t* x = static_cast<const half_t*>(p.x);
  auto lds = [&](int nw, int ring) { return lds_bytes(a.cap, p.k, nw, ring, shift); };
  auto grid = [&](int nw, int resident) {
    int64_t per = cu * resident / reached;
    const int64_t most = (row_tiles + nw - 1) / nw;
    if (per > most) per = most;
    a.blocks_per = static_cast<int>(per < 1 ? 1 : per);
    return a.blocks_per * max_tiles;
  };
  // Few row tiles in all: workgroups of four wavefronts reach more compute units
  // (one token, eight experts of 1536 x 2048: 9.6 us against 12.7 us).  Else
  // twelve with three chunks each in flight, or where the staged rows leave
  // less room eight (64 tokens over 128 experts of 1536 x 2048: 54.7 us with
  // twelve, 56.4 with eight of four chunks, 81 with two workgroups of eight of
  // two chunks, which do not cover the memory's latency).
  if (reached * row_tiles <= 4 * cu && lds(4, 4) <= kLdsMax / 2) {
    const int64_t n = grid(4, 2);
    return launch_form<4, 4>(x, xb, p.W, p.k, a, gated, shift, lds(4, 4), n, q);
  }
  if (lds(12, 3) <= kLdsMax) {
    const int64_t n = grid(12, 1);
    return launch_form<12, 3>(x, xb, p.W, p.k, a, gated, shift, lds(12, 3), n, q);
  }
  const int64_t n = grid(8, 1);
  return launch_form<8, 3>(x, xb, p.W, p.k, a, gated, shift, lds(8, 3), n, q);
}

// Up to eight rows (fp16) or four (bf16, whose rows every wavefront turns into
// fp16 one after another), and row tiles for at most two workgroups per compute
// unit at once.  Against the phase ring of q4_fused_gemv.hip (us, fp16 / bf16 with its
// staging): 4096 x 4096, one row 5.8 and 6.9 / 6.1 and 9.3, four rows 6.1 and 6.8 /
// 8.0 and 9.4; 7168 x 5120, one row 8.6 and 9.9 / 9.5 and 12.4.  Not taken:
// 512 x 1024, 16 rows 5.3 and 4.7 / 12.5 and 7.0; 16384 x 2048 gated (four row tiles
// per compute unit), one row 9.3 and 8.8.
bool fused_split_supports(int64_t m, int64_t nout, int64_t n, int64_t k, bool xb) {
  const int64_t tiles = (nout + (nout < n ? 7 : 15)) / (nout < n ? 8 : 16), cu = device_cu_count();
  if (m > (xb ? 4 : 8) || k > (1 << 15) || tiles > 2 * cu || !fused_gemv_supports(n, k, m, 0)) return false;
  return split_lds(m, k, split_waves(k)) <= (tiles <= cu ? kLdsMax : kLdsMax / 2);
}

hipError_t launch_fused_split(const Product& p, const Epi& ep, Queue q) {
  static const KernelFn fns[8] = {reinterpret_cast<KernelFn>(&fused_split_kernel<false, false, false>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<false, false, true>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<false, true, false>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<false, true, true>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<true, false, false>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<true, false, true>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<true, true, false>),
                                  reinterpret_cast<KernelFn>(&fused_split_kernel<true, true, true>)};
  static std::atomic<uint64_t> allowed[8];
  const bool gated = ep.half != 0;
  const int f = (gated ? 4 : 0) + (p.k % 256 != 0 ? 2 : 0) + (p.xt == DType::BF16 ? 1 : 0);
  const int waves = split_waves(p.k);
  const half_t* x = static_cast<const half_t*>(p.x);
  const uint8_t* W = p.W;
  int64_t k = p.k;
  SplitArgs a{ep, static_cast<int>(p.m)};
  void* argv[] = {&x, &W, &k, &a};
  return launch_blocks(fns[f], (ep.ldy + (gated ? 7 : 15)) / (gated ? 8 : 16), waves * kWave, argv,
                       static_cast<size_t>(split_lds(p.m, p.k, waves)), q, 1, 1, kLdsMax, &allowed[f]);
}

}  // namespace q4
