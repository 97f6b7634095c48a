// Geometry of the matrix-core decode kernels' LDS ring (gfx950), shared by the
// plain and the fused decode product.  Internal header.
#pragma once

#include "q4_device.hpp"

namespace q4 {
namespace {

constexpr int kTLdsMax = 160 * 1024;
// Phases resident in LDS.  (Deeper rings of smaller phases, 16 blocks in up
// to seven slots, measured slower than three slots of 32 blocks at
// 5120 x 5120: the per-phase barrier and fixed costs outweigh the extra
// copies in flight.)
constexpr int kTSlots = 3;

template <int V>
struct TC {
  static constexpr int value = V;
};

// Unrolled loop over a compile-time range: f(TC<0>{}), ..., f(TC<N - 1>{}).
template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F&& f) {
  if constexpr (I < N) {
    f(TC<I>{});
    unroll<I + 1, N>(f);
  }
}

// Geometry of one phase slot for T row tiles, AT activation tiles, PB blocks
// per phase, NW computing waves and NP copying waves (NP = 0: the computing
// waves copy too).  WR (<= 16 T) is the weight rows a slot holds: below 16 T
// the last tile's rows past WR read bytes of the slot's activation area
// (in bounds; they feed only outputs that are never stored), which lets
// three slots of 5 tiles x 2 activation tiles fit the LDS.  XR (<= 16 AT)
// is the activation rows a slot holds: a launch needs m <= XR, and operand
// rows past m read row m - 1, so a smaller area (nine tiles with m <= 10)
// leaves the LDS to weight rows.
template <int T, int AT, int PB, int NW, int NP, int WR = 16 * T, int XR = 16 * AT>
struct TileGeo {
  static constexpr int nw = NW;
  static constexpr int lanes = (NW + NP) * kWave;         // threads of the workgroup
  static constexpr int cwaves = NP > 0 ? NP : NW;         // copying waves
  static constexpr int clanes = cwaves * kWave;
  static constexpr int jb = PB / NW;                      // blocks per wave per phase
  static constexpr int row_pc = PB * kBlockBytes / 16;    // weight pieces per row
  static constexpr int wstride_pc = row_pc + 1;           // odd row stride (pieces)
  static constexpr int wstride = 16 * wstride_pc;
  static_assert(WR >= 1 && WR <= 16 * T, "weight rows of a slot");
  static constexpr int wpos = WR * wstride_pc;             // weight pieces per slot
  static constexpr int niw = (wpos + clanes - 1) / clanes;  // copy rounds (max per wave)
  static constexpr int wbytes = (16 * wpos + 255) / 256 * 256;
  static constexpr int xp = PB * kQK * 2 / 16;            // 16-byte pieces per activation row
  static_assert(XR >= 1 && XR <= 16 * AT, "activation rows of a slot");
  static constexpr int nix_max = (XR * xp + clanes - 1) / clanes;
  static constexpr int xbytes = XR * xp * 16;
  static constexpr int slot = wbytes + xbytes;
  static constexpr int red = T * AT * NW * kWave * 16;
  static constexpr int lds = kTSlots * slot > red ? kTSlots * slot : red;
  static constexpr int phase_k = PB * kQK;
  static constexpr int ndma = niw + nix_max;              // copy instructions per phase (max)
  static constexpr int tiles = T * jb;                    // (row tile, block) pairs per wave
  static constexpr int dma_per_tile = (ndma + tiles - 1) / tiles;
  static_assert(PB % (2 * NW) == 0, "blocks per wave must be even");
  static_assert((PB * kBlockBytes) % 16 == 0, "row segments of whole pieces");
  static_assert(xp >= 16, "swizzle needs 16 pieces per row");
};

}  // namespace
}  // namespace q4
