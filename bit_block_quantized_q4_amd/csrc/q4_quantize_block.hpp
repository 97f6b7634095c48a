// The Q4_0 rule for one block on eight lanes (gfx950): what the quantiser of
// weights and the cache's writer share.  Internal header.
#pragma once

#include "q4_internal.hpp"

namespace q4 {

// Lane exchange inside a group of eight (DPP, no LDS round trip).
constexpr int kDppXor1 = 0xB1;      // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;      // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;  // lane i <-> 7 - i within each 8 lanes
constexpr int kDppShl4 = 0x104;     // lane i reads lane i + 4 (row_shl:4)

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __builtin_bit_cast(float, dpp_i<CTRL>(__builtin_bit_cast(int, v)));
}

// Keep the (value, index) of larger magnitude, the smaller index on a tie.
template <int CTRL>
__device__ __forceinline__ void amax_step(float& best, float& bmag, int& bidx) {
  const float ob = dpp_f<CTRL>(best);
  const int oi = dpp_i<CTRL>(bidx);
  const float om = fabsf(ob);
  if (om > bmag || (om == bmag && oi < bidx)) { best = ob; bmag = om; bidx = oi; }
}

// Code q = min(15, trunc(fl(fl(x / D) + 8.5))) (negative truncations clamp to
// 0).  Fast path: r ~ 1/D (v_rcp_f32, 1 ulp), u = x r refined by one
// residual step e = fma(-u, D, x), u += e r, which leaves u within 2 ulp of
// the correctly rounded quotient (|u| <= 12 here, so 2^-19), and t = u + 8.5
// within 2^-18 of the rule's t.  Only a t within 2^-16 of an integer can
// truncate differently; those lanes redo the correctly rounded division.
__device__ __forceinline__ int code_of(float x, float D, float r) {
  float u = x * r;
  const float e = fmaf(-u, D, x);
  u = fmaf(e, r, u);
  float t = u + 8.5f;
  if (fabsf(t - __builtin_rintf(t)) < 0x1p-16f) {
    const float ue = x / D;
    asm volatile("" : "+v"(t));
    t = ue + 8.5f;
  }
  const int q = static_cast<int>(t);  // truncation
  return q < 0 ? 0 : (q > 15 ? 15 : q);
}

// One block: the eight lanes of a group hold its elements 4p .. 4p + 3 in v.
// Returns the scale (on every lane) and, on lanes 0 .. 3, the finished code bytes
// 4p .. 4p + 3.
__device__ __forceinline__ half_t quantize_lanes(int part, const float (&v)[4], uint32_t* bytes) {
  // Largest magnitude inside this lane, first index on ties.
  float best = v[0];
  float bmag = fabsf(v[0]);
  int bidx = part * 4;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const float a = fabsf(v[i]);
    if (a > bmag) { bmag = a; best = v[i]; bidx = part * 4 + i; }
  }
  // Across the eight lanes: both quads, then the other quad (the mirror pairs
  // lanes whose quads already agree), so every lane ends with the same pair.
  amax_step<kDppXor1>(best, bmag, bidx);
  amax_step<kDppXor2>(best, bmag, bidx);
  amax_step<kDppHalfMirror>(best, bmag, bidx);

  // The quotient is exact in fp32 (a power-of-two scaling), then rounded once
  // to fp16.  The empty asm keeps the compiler from fusing the two steps into a
  // mixed-precision fma with a +0 addend, which would turn a -0 scale into +0
  // (an all +0 block must get d = fp16(+0 / -8) = -0).
  float t = best / -8.0f;
  asm volatile("" : "+v"(t));
  const half_t dh = static_cast<half_t>(t);
  const float D = static_cast<float>(dh);

  uint32_t nib = 0x08080808u;  // every q is 8 when d is zero
  if (D != 0.0f) {
    const float r = __builtin_amdgcn_rcpf(D);
    nib = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) nib |= static_cast<uint32_t>(code_of(v[i], D, r)) << (8 * i);
  }
  // Lane p (< 4) holds low nibbles of code bytes 4p..4p+3; lane p+4 holds the
  // matching high nibbles (elements 16 + 4p ..).
  const uint32_t hi = static_cast<uint32_t>(dpp_i<kDppShl4>(static_cast<int>(nib)));
  *bytes = nib | (hi << 4);
  return dh;
}

}  // namespace q4
