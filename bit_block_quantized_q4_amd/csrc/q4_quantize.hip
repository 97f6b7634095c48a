// Q4_0 quantiser for gfx950.
//
// One weight copy serves every backend (vertical-disaggregation page, section
// "Every cycle counts: custom kernels"), so this kernel must reproduce the
// format rule bit for bit: per 32-wide block along K, m is the element of
// largest magnitude (first index on a tie), d = fp16(m / -8) rounded to
// nearest even with subnormals kept, q = min(15, trunc(x / d + 8.5)) with a
// correctly rounded fp32 division by d widened to fp32 and an fp32 add; every
// q is 8 when d is zero.  Bytes: d little-endian, then byte i = q[i] | q[i+16]<<4.
//
// Mapping: eight lanes per block, lane p holds elements 4p..4p+3, so a wave
// reads 64 x 16 contiguous bytes (fp32) per load instruction.  The block
// maximum is a 3-step DPP reduction inside each group of eight; the
// high-nibble codes of elements 16..31 (lanes 4..7) are moved down onto
// lanes 0..3, which then own four finished code bytes each.  The kernel
// reads 4 (fp32) or 2 (fp16, bf16; both widened exactly to fp32) bytes and
// writes 0.5625 bytes per weight.  The
// codes follow the correctly rounded fp32 division exactly: a reciprocal with
// one residual step decides every code whose t is not within 2^-16 of an
// integer, the rest redo the IEEE division (the library is built without
// fast-math).
#include "q4_quantize_block.hpp"

namespace q4 {
namespace {

constexpr int kQuantUF32 = 4;  // blocks in flight per lane group (16-byte loads)
constexpr int kQuantUF16 = 2;  // (8-byte loads; the kernel is VALU-bound, so more
                                // workgroups beat more loads in flight: 8 -> 2 took
                                // 5120 x 5120 fp16 from 30.2 to 23.0 us)

template <typename T>
struct Load4;

// fp32 weights are read with non-temporal loads: each byte is read once, and
// keeping the 4-byte input out of the caches measured 4 % faster (5120 x 5120:
// 24.5 -> 23.4 us; 17408 x 5120: 74.2 -> 71.0 us).  The 2-byte inputs gain
// nothing from it (their kernel is bound by its arithmetic), so they keep
// ordinary loads.
template <>
struct Load4<float> {
  static __device__ __forceinline__ void run(const float* p, float v[4]) {
    typedef float f32x4_t __attribute__((ext_vector_type(4)));
    const f32x4_t t = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
    v[0] = t[0]; v[1] = t[1]; v[2] = t[2]; v[3] = t[3];
  }
};

template <>
struct Load4<bf16_t> {
  static __device__ __forceinline__ void run(const bf16_t* p, float v[4]) {
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    const u32x2_t t = *reinterpret_cast<const u32x2_t*>(p);
    v[0] = bf16_bits_to_float(t[0] & 0xFFFFu); v[1] = bf16_bits_to_float(t[0] >> 16);
    v[2] = bf16_bits_to_float(t[1] & 0xFFFFu); v[3] = bf16_bits_to_float(t[1] >> 16);
  }
};

template <>
struct Load4<half_t> {
  static __device__ __forceinline__ void run(const half_t* p, float v[4]) {
    const half4_t t = *reinterpret_cast<const half4_t*>(p);
    v[0] = static_cast<float>(t[0]); v[1] = static_cast<float>(t[1]);
    v[2] = static_cast<float>(t[2]); v[3] = static_cast<float>(t[3]);
  }
};

// One block: the eight lanes of a group share `blk` and hold its elements
// 4p .. 4p + 3 in v.
__device__ __forceinline__ void quantize_block(int64_t blk, int part, const float (&v)[4],
                                               uint8_t* __restrict__ out) {
  uint32_t bytes;
  const half_t dh = quantize_lanes(part, v, &bytes);
  uint8_t* ob = out + blk * kBlockBytes;
  if (part < 4) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(ob + 2 + 4 * part);  // 2-byte aligned
    dst[0] = static_cast<uint16_t>(bytes & 0xFFFFu);
    dst[1] = static_cast<uint16_t>(bytes >> 16);
  }
  if (part == 0) {
    *reinterpret_cast<uint16_t*>(ob) = __builtin_bit_cast(uint16_t, dh);
  }
}

// Each group of eight lanes takes U blocks per sweep, blk0 + u * stride, and
// issues all U loads before quantising any: one load in flight per lane would
// leave about 32 KB in flight per CU, which at HBM latency caps the stream
// near 4 TB/s.
template <typename T, int U>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ w,
                                                       uint8_t* __restrict__ out,
                                                       int64_t nblocks) {
  const int part = threadIdx.x & 7;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 3);
  // The eight lanes of a group always share their blocks, so they take every
  // branch together (the shuffles stay within active groups).
  for (int64_t blk0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
       blk0 < nblocks; blk0 += U * stride) {
    float v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t blk = blk0 + u * stride;
      if (blk < nblocks) Load4<T>::run(w + blk * kQK + part * 4, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t blk = blk0 + u * stride;
      if (blk < nblocks) quantize_block(blk, part, v[u], out);
    }
  }
}

}  // namespace

hipError_t launch_quantize(const void* w, DType wt, int64_t n, int64_t k,
                           uint8_t* packed, hipStream_t s) {
  const int64_t nblocks = n * (k / kQK);
  const int U = wt == DType::F32 ? kQuantUF32 : kQuantUF16;
  const int64_t groups = (nblocks + 32 * U - 1) / (32 * U);  // 32 blocks per workgroup per sweep
  const dim3 grid(static_cast<unsigned>(groups < 65535 ? groups : 65535));
  const dim3 block(256);
  if (wt == DType::F32) {
    const float* p = static_cast<const float*>(w);
    void* argv[] = {&p, &packed, const_cast<int64_t*>(&nblocks)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&quantize_kernel<float, kQuantUF32>),
                           grid, block, argv, 0, s);
  }
  if (wt == DType::BF16) {
    const bf16_t* p = static_cast<const bf16_t*>(w);
    void* argv[] = {&p, &packed, const_cast<int64_t*>(&nblocks)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&quantize_kernel<bf16_t, kQuantUF16>),
                           grid, block, argv, 0, s);
  }
  const half_t* p = static_cast<const half_t*>(w);
  void* argv[] = {&p, &packed, const_cast<int64_t*>(&nblocks)};
  return hipLaunchKernel(reinterpret_cast<const void*>(&quantize_kernel<half_t, kQuantUF16>),
                         grid, block, argv, 0, s);
}

}  // namespace q4
