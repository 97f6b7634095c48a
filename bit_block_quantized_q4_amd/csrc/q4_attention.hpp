// Shared by the matrix-core kernels of the attention over the paged Q4_0 cache
// (gfx950).  Internal header.
//
// Scores are kept in units of log2: x = s log2 e, weights exp2(x - m).  A weight is
// held times 2^12 (kLift): fp16 then keeps its full 11 bits down to 2^-26 of the
// largest, and a single weight of 2^12 stays far below fp16's range.
#pragma once

#include "q4_cache.hpp"

namespace q4 {

constexpr int kTile = 64;  // positions
constexpr int kWaves = 4;  // wavefronts of a workgroup
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLift = 12.f;

// c tanh(z), z = s / c, from s: in units of log2 (LOG2) or natural, with an error of some
// 5 2^-24 of the result whatever c is.
//   |z| <= kNear: s times an even polynomial, tanh(z) / z = 1 + z^2 (..), fitted to 2^-27.
//   above: t = exp(-2 |z|), 1 - 2 t / (1 + t), exp and reciprocal of the hardware (1 ulp).
// (The second form alone leaves an error of 2^-24 c, which for a c of 10^6 is 0.1.)  Scores
// of a tile that are all near, as they mostly are, take the polynomial alone: two
// transcendental instructions less each.  (6 ragged prompts, 16 heads of 64, window 512: a cap
// of 50 81 us, as with the second form alone, one of 1, which few scores are near, 115, not 81;
// without a cap 62.)
template <bool LOG2>
struct Cap {
  static constexpr float kNear = 0.625f, kUnit = LOG2 ? kLog2e : 1.f;
  float top, in;
  // (both the same on all lanes, kept in scalar registers; a c below 2^-128 has no
  // reciprocal in fp32)
  __device__ __forceinline__ explicit Cap(float c)
      : top(uniform(c * kUnit)), in(uniform(fminf(1.f / c, 3.4028234e38f))) {}
  static __device__ __forceinline__ float uniform(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
  }
  // Whether scores of up to this magnitude are near.
  __device__ __forceinline__ bool near(float most) const { return most * in <= kNear; }
  __device__ __forceinline__ float of_near(float s) const {
    const float z = s * in, u = z * z;
    float p = fmaf(u, -0.00570498f * kUnit, 0.02063908f * kUnit);
    p = fmaf(u, p, -0.05373971f * kUnit);
    p = fmaf(u, p, 0.13331442f * kUnit);
    p = fmaf(u, p, -0.33333282f * kUnit);
    return s * fmaf(u, p, kUnit);
  }
  __device__ __forceinline__ float of(float s) const {
    const float z = fabsf(s * in), t = __builtin_amdgcn_exp2f(-2.f * kLog2e * z);
    const float far = __builtin_copysignf(fmaf(-2.f * t, __builtin_amdgcn_rcpf(1.f + t), 1.f), s) * top;
    return z <= kNear ? of_near(s) : far;
  }
};

// f q (f 0 or +-1) of two values of q; NaN of an infinite one, so that every product with it
// is NaN, also with a code or a scale of 0.
__device__ __forceinline__ uint32_t query_pair(uint32_t q, float f) {
  const half2_t v = __builtin_bit_cast(half2_t, q);
  const half_t h = static_cast<half_t>(f), z = static_cast<half_t>(0.f);
  return __builtin_bit_cast(uint32_t, v * half2_t{h, h} + v * half2_t{z, z});
}

// The larger / the sum of the values that the lanes of the same l % 16 hold.
__device__ __forceinline__ float max_over_groups(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(p[0])), __builtin_bit_cast(float, static_cast<uint32_t>(p[1])));
  const uint32_t c = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = __builtin_bit_cast(float, static_cast<uint32_t>(p[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(p[1]));
  const uint32_t c = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return __builtin_bit_cast(float, static_cast<uint32_t>(r[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(r[1]));
}

// As those, over the lanes l and l + 32.
__device__ __forceinline__ float max_over_halves(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(p[0])), __builtin_bit_cast(float, static_cast<uint32_t>(p[1])));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __builtin_bit_cast(float, static_cast<uint32_t>(p[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(p[1]));
}

// The exact q - 8 of a dword's eight codes, as fp16 pairs of bytes (0, 2) and (1, 3):
// low nibbles l02, l13, high nibbles h02, h13.  (A nibble in the low bits of a fixed
// exponent is 1024 + q or 64 + q.)
struct Codes {
  half2_t l02, l13, h02, h13;
};
__device__ __forceinline__ Codes codes_of(uint32_t w, const UnpackConsts& k) {
  const uint32_t v = w >> 8;
  const half2_t klo = {static_cast<half_t>(-1032.0f), static_cast<half_t>(-1032.0f)};
  const half2_t khi = {static_cast<half_t>(-72.0f), static_cast<half_t>(-72.0f)};
  Codes c;
  c.l02 = __builtin_bit_cast(half2_t, (w & k.mask_lo) | k.exp_lo) + klo;
  c.l13 = __builtin_bit_cast(half2_t, (v & k.mask_lo) | k.exp_lo) + klo;
  c.h02 = __builtin_bit_cast(half2_t, (w & k.mask_hi) | k.exp_hi) + khi;
  c.h13 = __builtin_bit_cast(half2_t, (v & k.mask_hi) | k.exp_hi) + khi;
  return c;
}

__device__ __forceinline__ half8_t join(half2_t a, half2_t b, half2_t c, half2_t d) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, a);
  r[1] = __builtin_bit_cast(uint32_t, b);
  r[2] = __builtin_bit_cast(uint32_t, c);
  r[3] = __builtin_bit_cast(uint32_t, d);
  return __builtin_bit_cast(half8_t, r);
}

// Four consecutive outputs from column `at` on (a multiple of four).
__device__ __forceinline__ void store4(void* y, int dt, int64_t at, const float (&v)[4]) {
  if (dt == static_cast<int>(DType::F32)) {
    float4_t r = {v[0], v[1], v[2], v[3]};
    *reinterpret_cast<float4_t*>(static_cast<float*>(y) + at) = r;
  } else {
    uint2 r;
    r.x = f32_to_16(v[0], dt) | static_cast<uint32_t>(f32_to_16(v[1], dt)) << 16;
    r.y = f32_to_16(v[2], dt) | static_cast<uint32_t>(f32_to_16(v[3], dt)) << 16;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = r;
  }
}

// Every sequence one row (no offsets), and any numbers of rows.
size_t attention_few_bytes(const Attention& a);
hipError_t launch_attention_few(const Attention& a, void* workspace, Queue q);
size_t attention_mixed_bytes(const Attention& a);
hipError_t launch_attention_mixed(const Attention& a, void* workspace, Queue q);

}  // namespace q4
