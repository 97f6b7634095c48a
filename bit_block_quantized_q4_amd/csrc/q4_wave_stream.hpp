// One wavefront's stream of packed weight rows (gfx950).  Internal header.
//
// A wavefront takes row tiles of 16 weight rows (with a gate 8 gate rows and
// their 8 up rows in turn) over all of K, one after another, through a private
// ring of kRing LDS slots, a chunk of 8 blocks (144 bytes a row) each: the
// copies of the next rows are under way while the last chunks of these are
// multiplied, and no other wavefront is waited for.  Per block one
// v_mfma_f32_16x16x32_f16 of up to 16 staged rows of x (fp16, in LDS) against
// the 16 weight rows, the codes as exact fp16 q - 8; the block scale d is
// applied in fp32.
#pragma once

#include "q4_fused.hpp"

namespace q4 {
namespace {

constexpr int kChunk = 8;                   // blocks per chunk
constexpr int kSeg = kChunk * kBlockBytes;  // 144 bytes of a row
constexpr int kCopies = 3;                  // copy instructions per chunk

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

// A staged row of x takes one 16-byte piece more than it has, so that the 16
// rows that an operand read touches lie in different banks.
__host__ __device__ inline int64_t staged_bytes(int64_t k) { return k * 2 + 16; }

// A staged bf16 row (np pieces at p) -> fp16 times a power of two, by one
// wavefront; returns the inverse of that power.
__device__ __forceinline__ float stage_row_bf16(u32x4* p, int np) {
  const int lane = threadIdx.x & (kWave - 1);
  uint32_t top = 0;  // largest magnitude, as bf16 bits
  for (int i = lane; i < np; i += kWave) {
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
  for (int i = lane; i < np; i += kWave) {
    u32x4 v = p[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = bf16x2_scaled_to_f16x2(v[e], f);
    p[i] = v;
  }
  return power_of_two(-shift);
}

template <int kRing, bool GATED, bool SHIFT>
struct RowStream {
  static constexpr int kPc = stride_pc<SHIFT>;
  static constexpr int kCols = GATED ? 8 : 16;  // output columns per row tile
  const uint8_t* wbase;  // the matrix, from the 16-byte piece that holds its first byte
  uint32_t wlow;         // its offset in that piece
  int64_t rb, nout, half, all;
  int nch, last, total, step;
  uint32_t ring;
  const uint8_t* slots;
  int pr[kCopies], pcx[kCopies];
  uint32_t src[kCopies];
  int need[kCopies];  // bytes of the segment from which the piece holds some
  int64_t tl, tc;     // row tile being copied, being multiplied
  int cl, issued;

  // Row tiles t, t + step, ... (ntiles of them) of W ([n][k], nout output
  // columns, with a gate half = nout), through the ring at smem + ring_at.
  __device__ __forceinline__ void begin(uint8_t* smem, int ring_at, const uint8_t* W, int64_t k,
                                        int64_t nout_, int64_t half_, int64_t t, int step_, int ntiles) {
    const int lane = threadIdx.x & (kWave - 1);
    const int nb = static_cast<int>(k / kQK);
    rb = static_cast<int64_t>(nb) * kBlockBytes;
    nout = nout_;
    half = half_;
    all = (nout + kCols - 1) / kCols;
    nch = (nb + kChunk - 1) / kChunk;
    last = nb - (nch - 1) * kChunk;
    total = ntiles * nch;
    step = step_;
    ring = lds_addr(smem) + ring_at;
    slots = smem + ring_at + (lane & 15) * (16 * kPc);
    wlow = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(W) & 15);
    wbase = W - wlow;
    // Slot piece 64 q + lane is piece pcx of row pr's segment.
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int i = q * kWave + lane;
      pr[q] = i / kPc;
      pcx[q] = i - pr[q] * kPc;
    }
    tl = tc = t;
    cl = issued = 0;
    if (total > 0) set_tile();
  }
  // Of every row only the chunks c0 .. c1 - 1 (before the prologue).
  __device__ __forceinline__ void limit(int c0, int c1, int ntiles) {
    wbase += c0 * kSeg;
    if (c1 < nch) last = kChunk;
    nch = c1 - c0;
    total = ntiles * nch;
  }
  // Weight row of slot row r of row tile t (columns past the last repeat it).
  __device__ __forceinline__ int64_t wrow(int64_t t, int r) const {
    int64_t c = t * kCols + (GATED ? r >> 1 : r);
    if (c >= nout) c = nout - 1;
    return GATED ? c + (r & 1) * half : c;
  }
  __device__ __forceinline__ void set_tile() {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const uint32_t off = wlow + static_cast<uint32_t>(wrow(tl, pr[q] & 15) * rb);
      const int sh = static_cast<int>(off & 15u);
      src[q] = off - sh + 16 * pcx[q];
      need[q] = pr[q] < 16 ? 16 * pcx[q] - sh : 1 << 20;
    }
  }
  __device__ __forceinline__ void next_copy() {
    const uint8_t* base = wbase + static_cast<int64_t>(cl) * kSeg;
    const int bytes = cl == nch - 1 ? last * kBlockBytes : kSeg;
    const int slot = issued % kRing;
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      if (need[q] < bytes) copy16<false>(src[q], base, ring + slot * slot_bytes<SHIFT> + q * (kWave * 16));
    ++issued;
    if (++cl == nch) {
      cl = 0;
      tl += step;
      if (issued < total) set_tile();
    }
  }
  // Fills the ring; the copies then in flight.
  __device__ __forceinline__ int prologue() {
    const int n = total < kRing ? total : kRing;
    for (int i = 0; i < n; ++i) next_copy();
    return kCopies * n;
  }
  // Streams every chunk; xl: this lane's operand in the staged rows (row lane %
  // 16, + 8 (lane / 16) bytes).  fin(t, acc) takes row tile t's sums: lane l holds
  // weight row l % 16 and rows 4 (l / 16) .. + 3 of x.
  template <typename F>
  __device__ __forceinline__ void run(const uint8_t* xl, F fin) {
    const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
    const UnpackConsts kc = make_unpack_consts();
    float4_t acc = {0.f, 0.f, 0.f, 0.f};
    int cc = 0, sh = 0;
    auto set_shift = [&]() {
      if constexpr (SHIFT)
        sh = static_cast<int>((wlow + static_cast<uint32_t>(wrow(tc < all ? tc : all - 1, r) * rb)) & 15u);
    };
    set_shift();
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
      cc = 0;
      fin(tc, acc);
      acc = float4_t{0.f, 0.f, 0.f, 0.f};
      tc += step;
      set_shift();
    };
    // Chunk t has landed when at most the chunks after it are in flight (copies
    // retire in order; what fin loads and stores only makes the wait longer).
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
  }
};

}  // namespace
}  // namespace q4
