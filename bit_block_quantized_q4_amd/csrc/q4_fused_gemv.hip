// Fused linear layer and expert products for few rows (up to 32 per product)
// on 16 x 16 x 32 matrix cores.
//
// Bound by the packed weights: n k 0.5625 bytes are read once.  The kernel is
// the decode GEMV's: a workgroup owns some weight rows over all of K, copying
// waves stream the phases of its rows and of x's columns global -> LDS into a
// ring of three slots, computing waves turn the codes into exact fp16 q - 8,
// multiply, and apply the block scale d in fp32.  What differs:
//   - A gate: slot row 2 c is the gate row of output column c, slot row 2 c + 1
//     its up row, so both sums of an output lie in neighbouring lanes and any
//     even number of rows can be dealt to a workgroup.
//   - Experts: a workgroup takes one tile of the plan (up to 16 or 32 rows of one
//     expert), gathers its rows of x by per-lane addresses in the same copies
//     and scatters its outputs by row.
//   - k need only be a multiple of 64: a row's segment is copied as the
//     16-byte pieces that contain it (the row's offset in its first piece, 0, 4,
//     8 or 12 bytes, is the same in every phase and for every 8th row, so it is
//     a constant of the lane), and the last phase may be short; its copies and
//     its waves' blocks stop at the row's end.
// Ten rows of 5120 against 34816 gated weight rows: 23.7 us a call among others,
// 4.25 TB/s (a large copy moves 4.8); a traced launch, which overlaps no other,
// takes 25.7.  Narrow layers of few rows: see fused_split_kernel.
#include "q4_fused.hpp"
#include "q4_tile_geo.hpp"

namespace q4 {
namespace {

struct FewArgs {
  Epi ep;
  Rows rows;
  const float* xscale;  // [x rows], or nullptr
  int64_t nout;         // output columns
  int m;                // dense: rows
  int cols;             // output columns per workgroup
  int cblocks;          // workgroups per tile
};

template <int T, int AT, int PB, int NW, int NP, int WR, int XR, bool GATED>
__global__ __launch_bounds__((NW + NP) * kWave, 1) void fused_gemv_kernel(const half_t* __restrict__ x,
                                                                          const uint8_t* __restrict__ W,
                                                                          int64_t k, FewArgs a) {
  using G = TileGeo<T, AT, PB, NW, NP, WR, XR>;
  constexpr int CW = G::cwaves;
  static_assert(NP > 0 && G::niw <= 32 && G::nix_max <= 32, "copy masks");
  extern __shared__ __attribute__((aligned(16))) uint8_t tsm[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tile = blockIdx.x / a.cblocks;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x - tile * a.cblocks) * a.cols;
  int64_t boff = 0;
  int m = a.m;
  // Rows of y and factors of the tile's rows, behind the ring (thread r keeps
  // row r's until the end).
  int* const yrows = reinterpret_cast<int*>(tsm + G::lds);
  float* const factors = reinterpret_cast<float*>(yrows + 16 * AT);
  const int* const rec = a.rows.recs != nullptr ? a.rows.recs + static_cast<int64_t>(tile) * a.rows.rec_words : nullptr;
  int pair = threadIdx.x;
  if (rec != nullptr) {
    const int4 t = *reinterpret_cast<const int4*>(rec);
    if (threadIdx.x < 16 * AT) pair = rec[4 + threadIdx.x];  // (all three loads in flight)
    if (tile >= *a.rows.ntiles) return;
    m = t.z;
    W += t.x * a.rows.wstride;
    boff = t.x * a.rows.nbias;
  }
  if (static_cast<int>(threadIdx.x) < m) {
    yrows[threadIdx.x] = pair;
    const int64_t row = rec != nullptr ? pair / a.rows.xdiv : pair;
    factors[threadIdx.x] = a.xscale != nullptr ? a.xscale[row] : 1.0f;
  }
  const int nc = static_cast<int>(a.nout - col0 < a.cols ? a.nout - col0 : a.cols);  // columns stored
  const int rv = GATED ? 2 * nc : nc;                                               // weight rows copied
  const int nb = static_cast<int>(k / kQK);
  const int64_t rb = static_cast<int64_t>(nb) * kBlockBytes;  // bytes per weight row
  const int nph = (nb + PB - 1) / PB;
  const int last = nb - (nph - 1) * PB;  // blocks of the last phase
  const uint32_t smem = lds_addr(tsm);

  // Weight row of slot row r, from row col0.
  auto wrow = [&](int r) -> int64_t { return GATED ? (r >> 1) + (r & 1) * a.ep.half : r; };

  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(x);
  // Row col0, from the 16-byte piece that holds its first byte (the packed
  // weights start at one, so it lies in them).
  const uint32_t shift0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(W + col0 * rb) & 15);
  const uint8_t* const wbase = W + col0 * rb - shift0;

  float4_t acc[T][AT];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int t = 0; t < AT; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};

  if (wave >= NW) {
    // Copying waves.  Slot piece i = (q CW + cwave) 64 + lane is piece
    // i % wstride_pc of the segment of slot row i / wstride_pc, from the piece
    // that holds the segment's first byte on.  A lane copies piece c of a phase
    // if it holds any byte of the segment (bit q of `full`, or of `fin` in the
    // last phase); a wave issues the copies that any of its lanes makes (the
    // same bits of the uniform masks).
    const int cwave = wave - NW;
    uint32_t wsrc[G::niw], wfull = 0, wfin = 0, wfull_any = 0, wfin_any = 0;
#pragma unroll
    for (int q = 0; q < G::niw; ++q) {
      const int i = (q * CW + cwave) * kWave + lane;
      const int r = i / G::wstride_pc, c = i - r * G::wstride_pc;
      const uint32_t off = shift0 + static_cast<uint32_t>(wrow(r < rv ? r : 0) * rb);
      const int sh = static_cast<int>(off & 15u);
      wsrc[q] = off - sh + 16 * c;
      const bool f = r < rv && 16 * c < sh + PB * kBlockBytes;
      const bool l = r < rv && 16 * c < sh + last * kBlockBytes;
      wfull |= f ? 1u << q : 0u;
      wfin |= l ? 1u << q : 0u;
      wfull_any |= __ballot(f) != 0 ? 1u << q : 0u;
      wfin_any |= __ballot(l) != 0 ? 1u << q : 0u;
    }
    // Activation copies: position i of the slot's activation area holds piece
    // (i % xp) ^ (row & 15) of row i / xp of the phase's columns.
    uint32_t xsrc[G::nix_max], xfull = 0, xfin = 0, xfull_any = 0, xfin_any = 0;
#pragma unroll
    for (int q = 0; q < G::nix_max; ++q) {
      const int i = (q * CW + cwave) * kWave + lane;
      const int ar = i / G::xp;
      const int pc = (i - ar * G::xp) ^ (ar & 15);
      const int at = ar < m ? ar : 0;
      const int64_t row = rec != nullptr ? rec[4 + at] / a.rows.xdiv : at;
      xsrc[q] = static_cast<uint32_t>((row * k + 8 * pc) * 2);
      const bool f = ar < m, l = f && pc < 4 * last;
      xfull |= f ? 1u << q : 0u;
      xfin |= l ? 1u << q : 0u;
      xfull_any |= __ballot(f) != 0 ? 1u << q : 0u;
      xfin_any |= __ballot(l) != 0 ? 1u << q : 0u;
    }
    // (uniform: kept in scalar registers)
    wfull_any = __builtin_amdgcn_readfirstlane(wfull_any);
    wfin_any = __builtin_amdgcn_readfirstlane(wfin_any);
    xfull_any = __builtin_amdgcn_readfirstlane(xfull_any);
    xfin_any = __builtin_amdgcn_readfirstlane(xfin_any);
    auto issue = [&](int p) {
      const bool fin = p == nph - 1;
      const uint32_t wa = fin ? wfin_any : wfull_any, xa = fin ? xfin_any : xfull_any;
      const uint32_t wl = fin ? wfin : wfull, xl = fin ? xfin : xfull;
      const uint32_t sb = smem + (p % kTSlots) * G::slot;
      const uint8_t* ws = wbase + static_cast<int64_t>(p) * (PB * kBlockBytes);
      const uint8_t* xs = xbase + static_cast<int64_t>(p) * (G::phase_k * 2);
      unroll<0, G::niw>([&](auto cc) {
        constexpr int q = decltype(cc)::value;
        if ((wa >> q) & 1u) {
          if ((wl >> q) & 1u) {
            copy16<T <= 2>(wsrc[q], ws, sb + (q * CW + cwave) * (kWave * 16));
          }
        }
      });
      unroll<0, G::nix_max>([&](auto cc) {
        constexpr int q = decltype(cc)::value;
        if ((xa >> q) & 1u) {
          if ((xl >> q) & 1u) copy16<false>(xsrc[q], xs, sb + G::wbytes + (q * CW + cwave) * (kWave * 16));
        }
      });
    };
    const int per_full = __popc(wfull_any) + __popc(xfull_any);
    const int per_fin = __popc(wfin_any) + __popc(xfin_any);
    issue(0);
    if (nph > 1) issue(1);
    for (int p = 0; p < nph; ++p) {
      // Only phase p + 1's copies may still be in flight.
      wait_vm_upto<G::niw + G::nix_max>(p + 1 >= nph ? 0 : p + 1 == nph - 1 ? per_fin : per_full);
      __builtin_amdgcn_s_barrier();
      compiler_fence();
      if (p + 2 < nph) issue(p + 2);  // the slot of phase p - 1, which every wave is done with
    }
  } else {
    // Lane roles: B side weight row r = lane % 16 and code dword g = lane / 16;
    // A side activation row lane % 16 (rows past m read row m - 1), the same g.
    const int r = lane & 15, g = lane >> 4;
    const int sh = static_cast<int>((shift0 + static_cast<uint32_t>(wrow(r) * rb)) & 15u);
    const uint32_t rs0 = r * G::wstride + sh + wave * (G::jb * kBlockBytes);  // scale of block 0
    const uint32_t rg0 = rs0 + 4 * g;                                          // code dword g
    uint32_t xa[G::jb][2][AT];  // activation operand halves (elements 4g.. and 16 + 4g..)
#pragma unroll
    for (int t = 0; t < AT; ++t) {
      int ar = r + 16 * t;
      if (ar > m - 1) ar = m - 1;
      const int sw = ar & 15;
#pragma unroll
      for (int j = 0; j < G::jb; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int pc = 4 * (wave * G::jb + j) + 2 * h + (g >> 1);
          xa[j][h][t] = G::wbytes + ar * (G::xp * 16) + 16 * (pc ^ sw) + 8 * (g & 1);
        }
    }
    const UnpackConsts kc = make_unpack_consts();
    for (int p = 0; p < nph; ++p) {
      __builtin_amdgcn_s_barrier();
      compiler_fence();
      // (blocks come in pairs, and a wave's are whole pairs)
      if (p == nph - 1 && wave * G::jb >= last) continue;
      const uint8_t* slot = tsm + (p % kTSlots) * G::slot;
      half8_t A[G::jb][AT];
#pragma unroll
      for (int j = 0; j < G::jb; ++j)
#pragma unroll
        for (int t = 0; t < AT; ++t) {
          const u32x2 lo = *reinterpret_cast<const u32x2*>(slot + xa[j][0][t]);
          const u32x2 hi = *reinterpret_cast<const u32x2*>(slot + xa[j][1][t]);
          A[j][t] = __builtin_bit_cast(half8_t, u32x4{lo[0], lo[1], hi[0], hi[1]});
        }
      // With one activation tile every pair's words are read before the first
      // product, with two each pair's next to it (as the decode GEMV does).
      uint32_t dw[T][G::jb], c0[T][G::jb], c1[T][G::jb];
      auto load_pair = [&](auto ii, auto jj) {
        constexpr int i = decltype(ii)::value;
        constexpr int j = decltype(jj)::value;
        constexpr int bo = i * 16 * G::wstride + j * kBlockBytes;
        dw[i][j] = *reinterpret_cast<const uint16_t*>(slot + rs0 + bo);
        if constexpr ((j & 1) == 0) {
          c0[i][j] = *reinterpret_cast<const uint32_t*>(slot + rg0 + bo);
          c1[i][j] = *reinterpret_cast<const uint32_t*>(slot + rg0 + bo + 4);
        } else {
          c0[i][j] = *reinterpret_cast<const uint32_t*>(slot + rg0 + bo + 2);
          c1[i][j] = c0[i][j];
        }
      };
      if constexpr (AT == 1)
        unroll<0, T>([&](auto ii) { unroll<0, G::jb>([&](auto jj) { load_pair(ii, jj); }); });
      unroll<0, T>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        unroll<0, G::jb>([&](auto jj) {
          constexpr int j = decltype(jj)::value;
          if constexpr (AT != 1) load_pair(ii, jj);
          const float d = half_bits_to_float(static_cast<uint16_t>(dw[i][j]));
          half8_t bw;
          if constexpr ((j & 1) == 0) bw = unpack8<2>(c0[i][j], c1[i][j], kc);
          else bw = unpack8<0>(c0[i][j], c0[i][j], kc);
#pragma unroll
          for (int t = 0; t < AT; ++t) {
            const float4_t D = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                A[j][t], bw, float4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][t][e] = d * D[e] + acc[i][t][e];
          }
        });
      });
      wait_lgkm0();  // this phase's reads are complete before its slot is refilled
    }
  }

  // Sum the computing waves' partial tiles, each output in wave order, and
  // finish it.  Lane l of a tile holds activation rows 4 (l / 16) .. + 3 of
  // weight row l % 16.
  __syncthreads();
  float4_t* red = reinterpret_cast<float4_t*>(tsm);
  if (wave < NW) {
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int t = 0; t < AT; ++t)
        if (16 * t + 4 * (lane >> 4) < m) red[((i * AT + t) * NW + wave) * kWave + lane] = acc[i][t];
  }
  __syncthreads();
  const float* rf = reinterpret_cast<const float*>(tsm);
  for (int o = threadIdx.x; o < nc * m; o += G::lanes) {
    const int ar = o / nc, c = o - ar * nc;
    const int64_t row = yrows[ar];
    const float sc = factors[ar];
    auto sum = [&](int r) {
      const float* q = rf + ((((r >> 4) * AT + (ar >> 4)) * NW) * kWave + (r & 15) + 16 * ((ar >> 2) & 3)) * 4 + (ar & 3);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += q[w * kWave * 4];
      return s * sc;
    };
    const float z0 = sum(GATED ? 2 * c : c);
    finish_store(a.ep, boff, row, col0 + c, z0, GATED ? sum(2 * c + 1) : 0.f);
  }
}

using KernelFn = const void*;

// One way to run: kernel, and the geometry the launch needs.
struct Form {
  KernelFn fn[2];  // plain, gated
  int rows, lds, threads;
  std::atomic<uint64_t>* allowed;  // [2]
};

template <int T, int AT, int PB, int NW = 8, int NP = 4, int WR = 16 * T, int XR = 16 * AT>
Form form() {
  using G = TileGeo<T, AT, PB, NW, NP, WR, XR>;
  constexpr int kLds = G::lds + 16 * AT * 8;  // the ring, and the rows' table
  static_assert(kLds <= kTLdsMax, "LDS budget");
  static std::atomic<uint64_t> allowed[2];
  return Form{{reinterpret_cast<KernelFn>(&fused_gemv_kernel<T, AT, PB, NW, NP, WR, XR, false>),
               reinterpret_cast<KernelFn>(&fused_gemv_kernel<T, AT, PB, NW, NP, WR, XR, true>)},
              WR, kLds, G::lanes, allowed};
}

// Two workgroups per compute unit: 8-block phases, four computing and two
// copying waves, up to 112 weight rows (64 with two activation tiles).
template <int T, int AT>
Form pair_form() {
  using G = TileGeo<T, AT, 8, 4, 2>;
  static_assert(2 * (G::lds + 16 * AT * 8) <= kTLdsMax, "two workgroups per compute unit");
  return form<T, AT, 8, 4, 2>();
}

Form pick_pair(int t, int at) {
  if (at == 2) {
    switch (t) {
      case 1: return pair_form<1, 2>();
      case 2: return pair_form<2, 2>();
      case 3: return pair_form<3, 2>();
      default: return pair_form<4, 2>();
    }
  }
  switch (t) {
    case 1: return pair_form<1, 1>();
    case 2: return pair_form<2, 1>();
    case 3: return pair_form<3, 1>();
    case 4: return pair_form<4, 1>();
    case 5: return pair_form<5, 1>();
    case 6: return pair_form<6, 1>();
    default: return pair_form<7, 1>();
  }
}

// One workgroup per compute unit.
Form pick_one(int t, int at, bool wide_phase) {
  if (at == 2) {
    switch (t) {
      case 1: return form<1, 2, 16>();
      case 2: return form<2, 2, 16>();
      case 3: return form<3, 2, 16>();
      case 4: return form<4, 2, 16>();
      default: return form<5, 2, 16, 8, 4, 68>();
    }
  }
  if (wide_phase) return t == 1 ? form<1, 1, 32>() : form<2, 1, 32>();
  switch (t) {
    case 1: return form<1, 1, 16>();
    case 2: return form<2, 1, 16>();
    case 3: return form<3, 1, 16>();
    case 4: return form<4, 1, 16>();
    case 5: return form<5, 1, 16>();
    case 6:
    case 7: return form<7, 1, 16>();
    default: return form<9, 1, 16, 8, 4, 144, 10>();
  }
}

struct FewPlan {
  Form form;
  int rows;  // weight rows per workgroup
};

// Weight rows per workgroup.  One product (dense): as the decode GEMV deals
// them, whole 16-row tiles or, with eight or more phases, spread evenly over
// the compute units, up to 144 rows (m <= 10), 112 (m <= 16) or 68 in one
// round; past one round two workgroups per compute unit.  Experts: every
// reached expert's rows in equal parts over workgroups of which two run on a
// compute unit.
FewPlan few_plan(int m, int64_t n, int64_t k, int64_t tiles, int at) {
  const int64_t cu = device_cu_count();
  FewPlan p;
  if (tiles > 1) {
    const int64_t most = at == 2 ? 64 : 112;
    int64_t rows = (n * tiles + 2 * cu - 1) / (2 * cu);
    rows = (rows + 15) / 16 * 16;
    if (rows > most) {
      // equal parts of one expert's rows
      const int64_t parts = (n + most - 1) / most;
      rows = (n + parts - 1) / parts;
    }
    rows = (rows + 1) / 2 * 2;
    p.rows = static_cast<int>(rows);
    p.form = pick_pair(static_cast<int>((rows + 15) / 16), at);
    return p;
  }
  int64_t tfull = ((n + 15) / 16 + cu - 1) / cu;
  if (tfull < 1) tfull = 1;
  int tmax = 5;
  if (at == 2) tmax = 4;
  else if (tfull <= 7) tmax = 7;
  else if (m <= 10) tmax = 9;
  if (tmax == 9 && tfull > 9) {
    int64_t rows = (n + 2 * cu - 1) / (2 * cu);
    rows = (rows + 3) / 4 * 4;
    if (rows <= 112) {
      p.rows = static_cast<int>(rows);
      p.form = pick_pair(static_cast<int>((rows + 15) / 16), 1);
      return p;
    }
  }
  const bool wide = tfull > tmax;
  if (tfull > tmax) tfull = tmax;
  const bool wide_phase = at == 1 && tfull <= 2 && k % 1024 == 0;
  int64_t rows = 16 * tfull;
  const int64_t spread = ((n + cu - 1) / cu + 1) / 2 * 2;
  if (k / ((wide_phase ? 32 : 16) * kQK) >= 8 && spread < rows) rows = spread;
  if (at == 2 && wide) rows = spread < 68 ? spread : 68;
  p.rows = static_cast<int>(rows);
  p.form = pick_one(static_cast<int>((rows + 15) / 16), at, wide_phase);
  return p;
}

}  // namespace

bool fused_gemv_supports(int64_t n, int64_t k, int64_t x_rows, int64_t experts) {
  // Whole 16-byte pieces to the end of the packed weights, 32-bit offsets of
  // a gate's up rows and of x's rows.  (A matrix is reached from the piece that
  // holds its first byte, up to 12 bytes before it, and to the end of its last.)
  const int64_t rb = k / kQK * kBlockBytes;
  return k % 64 == 0 && (n * (experts > 0 ? experts : 1) * rb) % 16 == 0 && n * rb <= (int64_t{1} << 32) - 16 &&
         x_rows * k * 2 < (int64_t{1} << 32);
}

hipError_t launch_fused_gemv(const Product& p, const Epi& ep, const Rows& rows, const half_t* xs,
                             const float* xscale, int64_t max_tiles, int tile_rows, Queue q) {
  const bool gated = ep.half != 0, grouped = p.experts != 0;
  const int64_t pairs = p.m * p.topk;
  const int at = (grouped ? tile_rows : p.m) > 16 ? 2 : 1;
  const int64_t tiles = grouped ? (pairs < p.experts ? pairs : p.experts) : 1;
  const int mrows = grouped ? tile_rows : static_cast<int>(p.m);
  const FewPlan f = few_plan(mrows, p.n, p.k, tiles, at);
  if (f.rows < 1 || f.rows > f.form.rows) return hipErrorInvalidValue;
  FewArgs a{ep, rows, xscale, ep.ldy, static_cast<int>(grouped ? 0 : p.m), gated ? f.rows / 2 : f.rows, 0};
  if (a.cols < 1) return hipErrorInvalidValue;
  a.cblocks = static_cast<int>((a.nout + a.cols - 1) / a.cols);
  const KernelFn fn = f.form.fn[gated ? 1 : 0];
  const uint8_t* W = p.W;
  int64_t k = p.k;
  void* argv[] = {&xs, &W, &k, &a};
  const int64_t grid = static_cast<int64_t>(a.cblocks) * (grouped ? max_tiles : 1);
  return launch_blocks(fn, grid, f.form.threads, argv, static_cast<size_t>(f.form.lds), q, 1, 1, kTLdsMax,
                       &f.form.allowed[gated ? 1 : 0]);
}

}  // namespace q4
