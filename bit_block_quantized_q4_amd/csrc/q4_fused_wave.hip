// Expert products for up to 16 rows per expert: every wavefront streams weight
// rows by itself.
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
// vector instructions per block).
#include <cmath>

#include "q4_fused.hpp"

namespace q4 {
namespace {

constexpr int kLdsMax = 160 * 1024;
constexpr int kChunk = 8;     // blocks per chunk
constexpr int kSeg = kChunk * kBlockBytes;  // 144 bytes of a row
constexpr int kCopies = 3;    // copy instructions per chunk

struct WaveArgs {
  Epi ep;
  Rows rows;
  int64_t nout;   // output columns
  int blocks_per; // workgroups per tile
  int cap;        // rows staged at a time (a tile of more takes several passes)
};

// Row stride of a slot in 16-byte pieces.  9 (the segment itself) and 11 both
// put the 16 rows of one dword column and its neighbours into 64 banks.
// SHIFT: rows start at any multiple of 4 bytes (k % 256 != 0); a segment is
// then copied as the up to 10 pieces that hold it.
template <bool SHIFT>
constexpr int stride_pc = SHIFT ? 11 : 9;
template <bool SHIFT>
constexpr int slot_bytes = 16 * 16 * stride_pc<SHIFT>;

template <int I, int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<I + 1, N>(f);
  }
}

// kNW wavefronts, each with kRing chunks in flight.  XB: x is bf16; a staged
// row is turned into fp16 in LDS, multiplied by the power of two that brings
// its largest magnitude to [2^15, 2^16) (as stage_bf16_kernel does).
template <int kNW, int kRing, bool GATED, bool SHIFT, bool XB>
__global__ __launch_bounds__(kNW * kWave) void fused_wave_kernel(const half_t* __restrict__ x,
                                                                 const uint8_t* __restrict__ W, int64_t k,
                                                                 WaveArgs a) {
  constexpr int kPc = stride_pc<SHIFT>;
  constexpr int kCols = GATED ? 8 : 16;  // output columns per 16 weight rows
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
  const int nb = static_cast<int>(k / kQK);
  const int64_t rb = static_cast<int64_t>(nb) * kBlockBytes;
  const int nch = (nb + kChunk - 1) / kChunk;
  const int last = nb - (nch - 1) * kChunk;  // blocks of a row's last chunk
  // This wavefront's row tiles: t, t + kNW, ... of the workgroup's share.
  const int64_t all = (a.nout + kCols - 1) / kCols;
  const int64_t t_end = all * (part + 1) / a.blocks_per;
  const int64_t t_begin = all * part / a.blocks_per + wave;
  const int ntiles = t_begin < t_end ? static_cast<int>((t_end - t_begin + kNW - 1) / kNW) : 0;
  // LDS: staged rows, their factors, the wavefronts' rings.
  // A staged row takes one 16-byte piece more than it has, so that the 16 rows
  // that an operand read touches lie in different banks.
  const int xpieces = static_cast<int>(k / 8), xstride = xpieces + 1;
  const int xbytes = a.cap * xstride * 16;
  float* const factors = reinterpret_cast<float*>(smem + xbytes);
  const uint32_t lds0 = lds_addr(smem);
  const int ring_at = xbytes + 64 + wave * (kRing * slot_bytes<SHIFT>);

  // Copies of a chunk: slot piece 64 q + lane is piece c of row r's segment,
  // from the piece that holds its first byte on.
  const uint32_t ring = lds0 + ring_at;
  int pr[kCopies], pcx[kCopies];
  uint32_t src[kCopies];
  int need[kCopies];  // bytes of the segment from which the piece holds some
  const uint32_t wlow = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(W) & 15);
  const uint8_t* const wbase = W - wlow;
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int i = q * kWave + lane;
    pr[q] = i / kPc;
    pcx[q] = i - pr[q] * kPc;
  }
  // Weight row of slot row r of row tile t (columns past the last repeat it).
  auto wrow = [&](int64_t t, int r) -> int64_t {
    int64_t c = t * kCols + (GATED ? r >> 1 : r);
    if (c >= a.nout) c = a.nout - 1;
    return GATED ? c + (r & 1) * a.ep.half : c;
  };
  auto set_tile = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const uint32_t off = wlow + static_cast<uint32_t>(wrow(t, pr[q] & 15) * rb);
      const int sh = static_cast<int>(off & 15u);
      src[q] = off - sh + 16 * pcx[q];
      need[q] = pr[q] < 16 ? 16 * pcx[q] - sh : 1 << 20;
    }
  };
  auto issue = [&](int ch, int slot) {
    const uint8_t* base = wbase + static_cast<int64_t>(ch) * kSeg;
    const int bytes = ch == nch - 1 ? last * kBlockBytes : kSeg;
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      if (need[q] < bytes) dma16_sbase(src[q], base, ring + slot * slot_bytes<SHIFT> + q * (kWave * 16));
  };

  const int r = lane & 15, g = lane >> 4;
  const uint8_t* const slots = smem + ring_at + r * (16 * kPc);
  const UnpackConsts kc = make_unpack_consts();

#pragma unroll 1
  for (int r0 = 0; r0 < count; r0 += a.cap) {  // one pass but for a token that names an expert often
  const int m = count - r0 < a.cap ? count - r0 : a.cap;
  if (r0 > 0) __syncthreads();  // the rows staged before have been read
  // Lane l < 16 knows row l: its pair and x row.
  const int pair = __shfl(pairs, (r0 + lane) & 15);
  const int xrow = lane < m ? pair / a.rows.xdiv : 0;
  // Stage x: position i of the area is piece i % xstride of row i / xstride.
  {
    const int positions = m * xstride;
    for (int i0 = wave * kWave; i0 < positions; i0 += kNW * kWave) {
      const int i = i0 + lane;
      const int ar = i / xstride;
      const int pc = i - ar * xstride;
      const int64_t row = __shfl(xrow, ar & 15);
      if (i < positions && pc < xpieces) dma16(x + row * k + 8 * pc, smem + static_cast<int64_t>(i0) * 16);
    }
  }
  // Lane roles: B side slot row r = lane % 16 and code dword g = lane / 16; A side
  // row lane % 16 of x (rows past m read row m - 1), the same g: its operand
  // halves are the elements 4 g .. and 16 + 4 g .. of a block.
  const int ar = r < m ? r : m - 1;
  const uint8_t* const xl = smem + ar * xstride * 16 + 8 * g;
  int yr[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) yr[e] = __shfl(pair, 4 * g + e);

  const int total = ntiles * nch;
  int64_t tl = t_begin;  // the row tile being copied
  int cl = 0, issued = 0;
  if (total > 0) set_tile(tl);
  auto next_copy = [&]() {
    issue(cl, issued % kRing);
    ++issued;
    if (++cl == nch) {
      cl = 0;
      tl += kNW;
      if (issued < total) set_tile(tl);
    }
  };
  const int npro = total < kRing ? total : kRing;
  for (int i = 0; i < npro; ++i) next_copy();
  // x (issued before the npro chunks) has landed; the barrier extends that to
  // every wavefront.
  wait_vm_upto<kCopies * kRing>(kCopies * npro);
  __builtin_amdgcn_s_barrier();
  compiler_fence();
  float sc[4] = {1.f, 1.f, 1.f, 1.f};
  if constexpr (XB) {
    for (int row = wave; row < m; row += kNW) {
      u32x4* p = reinterpret_cast<u32x4*>(smem + row * xstride * 16);
      uint32_t top = 0;  // largest magnitude, as bf16 bits
      for (int i = lane; i < xpieces; i += kWave) {
        const u32x4 v = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max_magnitude_bf16(top, v[e]);
      }
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t o = __shfl_xor(top, off);
        top = o > top ? o : top;
      }
      const int shift = bf16_row_shift(top);
      const float f = power_of_two(shift);
      for (int i = lane; i < xpieces; i += kWave) {
        u32x4 v = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = bf16x2_scaled_to_f16x2(v[e], f);
        p[i] = v;
      }
      if (lane == 0) factors[row] = power_of_two(-shift);
    }
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    compiler_fence();
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = factors[4 * g + e < m ? 4 * g + e : 0];
  }

  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  int64_t tc = t_begin;
  int cc = 0;
  int sh = 0;
  if constexpr (SHIFT) sh = static_cast<int>((wlow + static_cast<uint32_t>(wrow(tc < all ? tc : all - 1, r) * rb)) & 15u);
  auto compute = [&](int slot) {
    const uint8_t* sl = slots + slot * slot_bytes<SHIFT> + sh;
    const int blocks = cc == nch - 1 ? last : kChunk;
    const uint8_t* xc = xl + cc * (kChunk * kQK * 2);
    uint32_t dw[kChunk], c0[kChunk], c1[kChunk];
    half8_t A[kChunk];
    float4_t D[kChunk];
    auto load = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const uint8_t* p = sl + j * kBlockBytes;
      dw[j] = *reinterpret_cast<const uint16_t*>(p);
      if constexpr ((j & 1) == 0) {
        c0[j] = *reinterpret_cast<const uint32_t*>(p + 4 * g);
        c1[j] = *reinterpret_cast<const uint32_t*>(p + 4 * g + 4);
      } else {
        c0[j] = *reinterpret_cast<const uint32_t*>(p + 4 * g + 2);
        c1[j] = c0[j];
      }
      const u32x2 lo = *reinterpret_cast<const u32x2*>(xc + 64 * j);
      const u32x2 hi = *reinterpret_cast<const u32x2*>(xc + 64 * j + 32);
      A[j] = __builtin_bit_cast(half8_t, u32x4{lo[0], lo[1], hi[0], hi[1]});
    };
    auto multiply = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      half8_t bw;
      if constexpr ((j & 1) == 0) bw = unpack8<2>(c0[j], c1[j], kc);
      else bw = unpack8<0>(c0[j], c0[j], kc);
      D[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A[j], bw, float4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
    };
    auto scale = [&](auto jj) {
      constexpr int j = decltype(jj)::value;
      const float d = half_bits_to_float(static_cast<uint16_t>(dw[j]));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = d * D[j][e] + acc[e];
    };
    if (blocks == kChunk) {
      each<0, kChunk>(load);
      // Block j is scaled after block j + 1 is unpacked: its product is done then.
      each<0, kChunk>([&](auto jj) {
        constexpr int j = decltype(jj)::value;
        multiply(jj);
        if constexpr (j > 0) scale(std::integral_constant<int, j - 1>{});
        __builtin_amdgcn_sched_barrier(0x308);  // (matrix and LDS instructions may cross)
      });
      scale(std::integral_constant<int, kChunk - 1>{});
    } else {  // a row's short last chunk: whole pairs of blocks
      each<0, kChunk / 2>([&](auto pp) {
        constexpr int j = 2 * decltype(pp)::value;
        if (j < blocks) {
          load(std::integral_constant<int, j>{});
          load(std::integral_constant<int, j + 1>{});
          multiply(std::integral_constant<int, j>{});
          multiply(std::integral_constant<int, j + 1>{});
          scale(std::integral_constant<int, j>{});
          scale(std::integral_constant<int, j + 1>{});
        }
      });
    }
    wait_lgkm0();  // the slot's reads are complete before it is refilled
  };
  auto finish_chunk = [&](int slot) {
    compute(slot);
    if (++cc < nch) return;
    // The rows' sums are whole: lane l holds weight row l % 16 and rows
    // 4 (l / 16) .. + 3 of x.
    cc = 0;
    const int64_t c = tc * kCols + (GATED ? r >> 1 : r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float z = acc[e] * sc[e];
      const float u = GATED ? __shfl_xor(z, 1) : 0.f;
      if (4 * g + e < m && c < a.nout && (!GATED || (r & 1) == 0)) finish_store(a.ep, boff, yr[e], c, z, u);
    }
    acc = float4_t{0.f, 0.f, 0.f, 0.f};
    tc += kNW;
    if constexpr (SHIFT) {
      if (tc < all) sh = static_cast<int>((wlow + static_cast<uint32_t>(wrow(tc, r) * rb)) & 15u);
    }
  };
  // Chunk t has landed when at most the chunks after it are in flight (copies
  // retire in order; stores and loads of finish_store only make the wait longer).
  int t = 0;
  for (; t + kRing < total; ++t) {
    wait_vm<kCopies * (kRing - 1)>();
    compiler_fence();
    finish_chunk(t % kRing);
    compiler_fence();
    next_copy();
  }
  for (; t < total; ++t) {
    wait_vm_upto<kCopies * (kRing - 1)>(kCopies * (total - 1 - t));
    compiler_fence();
    finish_chunk(t % kRing);
  }
  }  // passes
}

using KernelFn = const void*;

// Rows staged at a time: no tile of distinct tokens has more.  (Fewer, with a
// second pass for the fuller tiles, doubles the time of the whole launch.)
int cap_rows(int64_t m) { return static_cast<int>(m < 16 ? m : 16); }

int lds_bytes(int cap, int64_t k, int nw, int ring, bool shift) {
  return static_cast<int>(cap * (k * 2 + 16)) + 64 + nw * ring * (shift ? slot_bytes<true> : slot_bytes<false>);
}

template <int NW, int R>
hipError_t launch_form(const half_t* x, bool xb, const uint8_t* W, int64_t k, WaveArgs a, bool gated,
                       bool shift, int lds, int64_t grid, hipStream_t s) {
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
  const hipError_t e = allow_dynamic_lds(fns[f], kLdsMax, allowed[f]);
  if (e != hipSuccess) return e;
  void* argv[] = {&x, &W, &k, &a};
  return hipLaunchKernel(fns[f], dim3(static_cast<unsigned>(grid)), dim3(NW * kWave), argv,
                         static_cast<size_t>(lds), s);
}

}  // namespace

bool fused_wave_supports(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k, int64_t x_rows) {
  if (experts == 0 || expert_tile_rows(m, topk, experts) != 16 || k > (1 << 15) ||
      !fused_gemv_supports(n, k, x_rows, experts))
    return false;
  return lds_bytes(cap_rows(m), k, 8, 3, k % 256 != 0) <= kLdsMax;
}

hipError_t launch_fused_wave(const Product& p, const Epi& ep, const Rows& rows, int64_t max_tiles,
                             hipStream_t s) {
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
    return launch_form<4, 4>(x, xb, p.W, p.k, a, gated, shift, lds(4, 4), n, s);
  }
  if (lds(12, 3) <= kLdsMax) {
    const int64_t n = grid(12, 1);
    return launch_form<12, 3>(x, xb, p.W, p.k, a, gated, shift, lds(12, 3), n, s);
  }
  const int64_t n = grid(8, 1);
  return launch_form<8, 3>(x, xb, p.W, p.k, a, gated, shift, lds(8, 3), n, s);
}

}  // namespace q4
