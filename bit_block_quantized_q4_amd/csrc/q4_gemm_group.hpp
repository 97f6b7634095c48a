// The expert products' tile (gfx950): up to BM rows of one expert, gathered,
// against BN of its weight rows.  Internal header, see q4_gemm_tile.hpp for the
// IO's part.
//
// The 256 x 256 tile of the prefill GEMM with two differences that an expert's
// row count asks for:
//   - Fragments are dealt to the wave rows in turn, and only those that hold rows
//     are copied, read and multiplied (a loop for each count): the time of a
//     tile follows its rows in steps of 32 WVM.
//   - A short tile computes for less than a load takes, so activations are copied
//     two steps ahead (three LDS stages) and packed weights loaded three steps
//     ahead (three register sets, which is why the step is unrolled by three:
//     a set in flight is never moved).  192 rows leave the LDS to both.
// Per step ks: issue A(ks + 2) and W(ks + 3); multiply stage ks while W(ks + 1) is
// dequantised into the other B stage; wait until only this step's own issues are
// in flight (loads retire in order), which are NF copies and 2 UNITS loads.
// Bound by dequantisation and barriers at the rows an expert has: 128 experts of
// 128 rows on average, 2048 x 2048 gated: 227 us, 605 TFLOP/s; 2048 x 1024: 145 us.
#pragma once

#include "q4_gemm_tile.hpp"

namespace q4 {
namespace {

template <int BM, int BN, int WVM, int WVN, typename IO>
__device__ __forceinline__ void gemm_group_body(IO io, const half_t* __restrict__ x,
                                                const uint8_t* __restrict__ W, int64_t k,
                                                const void* __restrict__ xe, int xet) {
  // xe / xet: the original activations, for the exact route.
  constexpr int NTH = WVM * WVN * 64;          // threads
  constexpr int WM = BM / WVM, WN = BN / WVN;  // wave tile
  constexpr int TM = WM / 32, TN = WN / 32;    // 32 x 32 products per wave
  constexpr int A_STAGE = BM * kRowBytes16;
  constexpr int B_STAGE = BN * kRowBytes16;
  constexpr int kAStages = 3;
  constexpr int A_COPIES = BM * 8 / NTH;       // 16-byte copies per thread per step
  constexpr int UNITS = BN * 2 / NTH;          // weight units (blocks) per thread per step
  static_assert(TM <= 3 && UNITS >= 1, "tile");
  static_assert(NTH / 8 == 32 * WVM, "a copy round is a fragment of every wave row");
  __shared__ __attribute__((aligned(16))) uint8_t smem[kAStages * A_STAGE + 2 * B_STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave / WVN, wn = wave % WVN;
  if (!io.template begin<BM, BN>()) return;
  W = io.weights(W);
  const int64_t rb = (k / kQK) * kBlockBytes;
  const int nks = static_cast<int>(k / kBK);
  const int last = nks - 1;

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
  auto load_units = [&](int ks, Units& r) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint8_t* src = wsrc[u] + static_cast<int64_t>(ks) * 2 * kBlockBytes;
      r.v[u].w = load_dwordx4_untracked(src);
      r.v[u].w4 = load_dword_untracked(src + 16);
    }
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
    uint8_t* bs = smem + kAStages * A_STAGE + stage * B_STAGE;
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

  // Fragment i of wave row wm: tile rows 32 (i WVM + wm) ..
  const int arow = wm * 32 + (lane & 31);
  const int brow = wn * WN + (lane & 31);
  const int kg = lane >> 5;

  auto main_loop = [&](auto nf_c) {
    constexpr int NF = decltype(nf_c)::value;
    auto issue_a = [&](int ks, int stage) {
      uint8_t* dst = smem + stage * A_STAGE;
#pragma unroll
      for (int i = 0; i < NF; ++i)
        dma16(asrc[i] + static_cast<int64_t>(ks) * kBK, dst + (NTH * i + 64 * wave) * 16);
    };
    // Operand fragments of k16 sub-step kk (lane: row arow / brow, 8 k-values
    // 8 kg .. 8 kg + 7 of the sub-step).
    auto read_frags = [&](const uint8_t* as, const uint8_t* bs, int kk, half8_t (&af)[NF], half8_t (&bf)[TN]) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
        af[i] = *reinterpret_cast<const half8_t*>(as + swz(arow + 32 * WVM * i, 2 * kk + kg) * 16);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        bf[j] = *reinterpret_cast<const half8_t*>(bs + swz(brow + 32 * j, 2 * kk + kg) * 16);
    };
    const uint8_t* const b0 = smem + kAStages * A_STAGE;
    Units U[3];  // W(ks) in U[ks % 3]
    issue_a(0, 0);
    load_units(0, U[0]);
    wait_vm<0>();
    tie_units(U[0]);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      dequant_half(U[0].v[u], u, 0, 0);
      dequant_half(U[0].v[u], u, 1, 0);
    }
    issue_a(1 < last ? 1 : last, 1);
    load_units(1 < last ? 1 : last, U[1]);
    load_units(2 < last ? 2 : last, U[2]);
    wait_vm_lgkm0<2 * UNITS>();  // A(1) and W(1)
    tie_units(U[1]);
    __builtin_amdgcn_s_barrier();
    compiler_fence();
    half8_t af[2][NF], bf[2][TN];
    read_frags(smem, b0, 0, af[0], bf[0]);
    auto step = [&](auto s_c, int ks) {
      constexpr int s = decltype(s_c)::value;  // ks % 3
      const int st = ks & 1;
      // (Past the last step: copies of it into stages that are no longer read.)
      issue_a(ks + 2 < last ? ks + 2 : last, (s + 2) % 3);
      load_units(ks + 3 < last ? ks + 3 : last, U[s]);
      const uint8_t* as = smem + s * A_STAGE;
      const uint8_t* bs = b0 + st * B_STAGE;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // 16-wide k sub-steps
        const int c = kk & 1;
        if (kk < 3) read_frags(as, bs, kk + 1, af[c ^ 1], bf[c ^ 1]);
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[c][i], bf[c][j], acc[i][j], 0, 0, 0);
        // The next step's weights (on the last step: a rewrite of the stage that
        // is no longer read).
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
          for (int h = 0; h < 2; ++h)
            if ((2 * u + h) % 4 == kk) dequant_half(U[(s + 1) % 3].v[u], u, h, st ^ 1);
        // one product, one operand read, a share of the dequantisation
#pragma unroll
        for (int i = 0; i < NF * TN; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
          if (kk < 3 && i < NF + TN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
          __builtin_amdgcn_sched_group_barrier(0x002, NF > 1 ? 2 : 6, 0);  // VALU
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vm_lgkm0<NF + 2 * UNITS>();  // A(ks + 1) and W(ks + 2) have landed
      tie_units(U[(s + 2) % 3]);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      compiler_fence();
      read_frags(smem + (s + 1) % 3 * A_STAGE, b0 + (st ^ 1) * B_STAGE, 0, af[0], bf[0]);
    };
    int ks = 0;
    for (; ks + 3 <= nks; ks += 3) {
      step(IC<0>{}, ks);
      step(IC<1>{}, ks + 1);
      step(IC<2>{}, ks + 2);
    }
    if (ks < nks) {
      step(IC<0>{}, ks);
      if (ks + 1 < nks) step(IC<1>{}, ks + 1);
    }
    wait_vm_lgkm0<0>();  // nothing may land in the LDS that the epilogue reuses
#pragma unroll
    for (int i = 0; i < 3; ++i) tie_units(U[i]);
  };
  const int live = io.fragments(32 * WVM);
  if (live >= TM) main_loop(IC<TM>{});
  else if (TM > 2 && live == 2) main_loop(IC<(TM > 2 ? 2 : 1)>{});
  else main_loop(IC<1>{});

  store_tile<WVM, WVN>(io, acc, smem, [&](uint32_t chunks) {
    exact_tile<NTH, BM, BN>(io, xe, static_cast<DType>(xet), k, W, rb, 0, k / kQK,
                            reinterpret_cast<float*>(smem), 32 * WVM, 3, chunks);
  }, live);
}

}  // namespace
}  // namespace q4
