// The fused linear layer and the expert products: launch rules, and the
// kernels that are right for every shape and type.
//
//   z[i, r] = sum_j x[i, j] (q[r, j] - 8) d[r, j / 32]
//   y = act(z + b) (x the gated half) + residual
//
// fused_row_kernel: one wavefront per output column and up to eight rows of
// x; a lane takes every 64th Q4_0 block of the column's weight row (of both
// rows with a gate), sums x (q - 8) in fp32 and applies d per block, and the
// wave adds its lanes' sums by xor shuffles, a fixed order.  Bound by latency and
// the fp32 products: 512 x 512, one fp32 row: 4.6 us a call, a launch's own time.
#include "q4_fused.hpp"

namespace q4 {
namespace {

constexpr int kRowMT = 8;
constexpr int kFewRows = 32;  // most rows per product of the decode kernels

template <typename XT>
__device__ __forceinline__ float widen(const XT* x, int64_t i);
template <>
__device__ __forceinline__ float widen<float>(const float* x, int64_t i) { return x[i]; }
template <>
__device__ __forceinline__ float widen<half_t>(const half_t* x, int64_t i) {
  return static_cast<float>(x[i]);
}
template <>
__device__ __forceinline__ float widen<bf16_t>(const bf16_t* x, int64_t i) {
  return bf16_bits_to_float(x[i].bits);
}

// The 32 exact q - 8 of a block at p (2-byte aligned) and its scale.
__device__ __forceinline__ float block_codes(const uint8_t* blk, float (&w)[kQK]) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(blk);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = p[1 + i];
    w[2 * i] = static_cast<float>(static_cast<int>(c & 0xFu) - 8);
    w[2 * i + 16] = static_cast<float>(static_cast<int>((c >> 4) & 0xFu) - 8);
    w[2 * i + 1] = static_cast<float>(static_cast<int>((c >> 8) & 0xFu) - 8);
    w[2 * i + 17] = static_cast<float>(static_cast<int>((c >> 12) & 0xFu) - 8);
  }
  return half_bits_to_float(p[0]);
}

// Workgroup = four output columns of one tile of rows (dense: all m rows).
template <typename XT, int G>
__global__ __launch_bounds__(256) void fused_row_kernel(const XT* __restrict__ x,
                                                        const uint8_t* __restrict__ W, int64_t m,
                                                        int64_t nout, int64_t k, int64_t cblocks,
                                                        Epi ep, Rows rows) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = blockIdx.x / cblocks;
  const int64_t c = (blockIdx.x - t * cblocks) * 4 + threadIdx.x / kWave;
  if (c >= nout) return;  // whole wavefront
  int64_t count = m, boff = 0;
  const int* rec = nullptr;
  if (rows.recs != nullptr) {
    if (t >= *rows.ntiles) return;
    rec = rows.recs + t * rows.rec_words;
    const int4 tile = *reinterpret_cast<const int4*>(rec);
    rec += 4;
    count = tile.z;
    W += tile.x * rows.wstride;
    boff = tile.x * rows.nbias;
  }
  const int64_t nb = k / kQK, rb = nb * kBlockBytes;
  const uint8_t* wr[G];
#pragma unroll
  for (int g = 0; g < G; ++g) wr[g] = W + (c + g * ep.half) * rb;
  for (int64_t r0 = 0; r0 < count; r0 += kRowMT) {
    const int mt = static_cast<int>(count - r0 < kRowMT ? count - r0 : kRowMT);
    const XT* xr[kRowMT];
    int64_t yrow[kRowMT];
#pragma unroll
    for (int i = 0; i < kRowMT; ++i) {
      const int64_t at = r0 + (i < mt ? i : mt - 1);  // rows past the last repeat it
      yrow[i] = at;
      int64_t from = at;
      if (rec != nullptr) {
        const int p = rec[at];
        yrow[i] = p;
        from = p / rows.xdiv;
      }
      xr[i] = x + from * k;
    }
    float acc[G][kRowMT];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < kRowMT; ++i) acc[g][i] = 0.f;
    for (int64_t b = lane; b < nb; b += kWave) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float w[kQK];
        const float d = block_codes(wr[g] + b * kBlockBytes, w);
#pragma unroll
        for (int i = 0; i < kRowMT; ++i) {
          if (i < mt) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kQK; ++j) s = fmaf(widen<XT>(xr[i], b * kQK + j), w[j], s);
            acc[g][i] = fmaf(d, s, acc[g][i]);
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < kRowMT; ++i)
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) acc[g][i] += __shfl_xor(acc[g][i], off);
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kRowMT; ++i)
        if (i < mt) finish_store(ep, boff, yrow[i], c, acc[0][i], acc[G - 1][i]);
    }
  }
}

// y[i] = sum_j weights[i, j] rows[i topk + j] + residual[i] in the order of j;
// a pair whose pos is negative has no expert and counts 0.  A workgroup takes
// 256 V columns of one token, so weights and places are uniform, and the loads
// of up to eight rows are in flight together.  Bound by HBM: 2048 tokens of eight
// rows of 2048: 26.6 us, 5.4 TB/s.
template <int V>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ part,
                                                      const float* __restrict__ weights,
                                                      const int* __restrict__ pos, int topk,
                                                      int64_t nout, int cblocks, Epi ep) {
  const int64_t i = blockIdx.x / cblocks;
  const int64_t c = (static_cast<int64_t>(blockIdx.x - i * cblocks) * 256 + threadIdx.x) * V;
  if (c >= nout) return;
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
  const float* p0 = part + i * topk * nout + c;
  for (int j0 = 0; j0 < topk; j0 += 8) {
    float r[8][V];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = j0 + j;
      const bool live = at < topk && pos[i * topk + (at < topk ? at : 0)] >= 0;
#pragma unroll
      for (int e = 0; e < V; ++e) r[j][e] = 0.f;
      if (live) {
        if constexpr (V == 4) {
          const float4_t q = *reinterpret_cast<const float4_t*>(p0 + at * nout);
#pragma unroll
          for (int e = 0; e < 4; ++e) r[j][e] = q[e];
        } else {
          r[j][0] = p0[at * nout];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = j0 + j;
      if (at < topk && pos[i * topk + at] >= 0) {
        const float w = weights[i * topk + at];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(w, r[j][e], v[e]);
      }
    }
  }
  const int64_t at = i * nout + c;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (ep.residual != nullptr) v[e] += load_f32(ep.residual, ep.y_dt, at + e);
    store_as(ep.y, ep.y_dt, at + e, v[e]);
  }
}

Rows plan_rows(const Product& p) {
  Rows r;
  if (p.experts == 0) return r;
  const PlanLayout L = plan_layout(p.m, p.topk, p.experts);
  if (p.plan != nullptr) {
    r.recs = p.plan + L.tiles;
    r.ntiles = p.plan + L.head;
  }
  r.rec_words = L.rec_words;
  r.xdiv = p.x_rows == p.m ? static_cast<int>(p.topk) : 1;
  r.wstride = p.n * (p.k / kQK) * kBlockBytes;
  r.nbias = p.n;
  return r;
}

template <typename XT>
hipError_t launch_row(const Product& p, const Epi& ep0, Queue q) {
  Epi ep = ep0;
  Rows rows = plan_rows(p);
  const XT* x = static_cast<const XT*>(p.x);
  const uint8_t* W = p.W;
  int64_t m = p.m, nout = ep.ldy, k = p.k, cblocks = (nout + 3) / 4;
  const int64_t tiles = p.experts == 0 ? 1 : plan_layout(p.m, p.topk, p.experts).max_tiles;
  void* argv[] = {&x, &W, &m, &nout, &k, &cblocks, &ep, &rows};
  const void* fn = ep.half != 0 ? reinterpret_cast<const void*>(&fused_row_kernel<XT, 2>)
                                : reinterpret_cast<const void*>(&fused_row_kernel<XT, 1>);
  return launch_blocks(fn, cblocks * tiles, 256, argv, 0, q);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Whether the decode GEMV takes a plain product of few fp16 rows in less time than
// the kernels here, whose addresses and masks for gates, gathered rows and any k
// take longer to set up (device us, GEMV / here, rows of x in front):
//   k % 512 == 0, its matrix-core kernels: always (5120 x 5120: 1 row 6.1 / 8.3,
//     10 rows 7.1 / 9.6, 32 rows 9.8 / 11.8);
//   k % 256 == 0, its streaming kernel: up to 16 rows and one row tile per compute
//     unit (4096 x 11008: 1 row 9.2 / 10.0, 16 rows 12.7 / 14.5; but 17 rows 18.2 /
//     16.9, 12288 x 3328: 1 row 11.4 / 9.4, 8192 x 1280: 16 rows 7.5 / 5.9);
//   other k % 64 == 0, its general kernel: one or two rows of a small layer (2048 x
//     1408: 1 row 3.2 / 4.4, 2 rows 3.5 / 4.4; 2048 x 8640: 1 row 6.9 / 8.6; but
//     10 rows of 2048 x 1408 9.2 / 4.8, 4096 x 4160: 1 row 7.3 / 6.3);
//   what only the row kernel here takes: always (5120 x 1056: 1 row 3.8 / 6.9, 32
//     rows 39 / 44).
bool gemv_is_faster(int64_t m, int64_t n, int64_t k) {
  if (k % 512 == 0 || !fused_gemv_supports(n, k, m, 0)) return true;
  const int64_t cu = device_cu_count();
  if (k % 256 == 0) return m <= 16 && n <= 16 * cu;
  return m <= 2 && m * n <= (k <= 2048 ? 20 : 8) * cu;
}

}  // namespace

// Rows of a product from which it runs on the prefill tiles.
bool many_rows(int64_t m, int64_t topk, int64_t experts) {
  return experts == 0 ? m > kFewRows : expert_tile_rows(m, topk, experts) > kFewRows;
}

size_t product_workspace_bytes(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k,
                               int64_t x_rows, DType xt, bool gated, bool combine) {
  size_t b = 0;
  const bool many = many_rows(m, topk, experts);
  if (xt == DType::BF16 && !fused_wave_supports(m, topk, experts, n, k, x_rows) &&
      !(experts == 0 && fused_split_supports(m, gated ? n / 2 : n, n, k, true)) &&
      (many || fused_gemv_supports(n, k, x_rows, experts)))
    b += stage_bytes(x_rows, k);
  if (many) b += fused_gemm_bytes(m, n, k, xt, gated, experts != 0);
  if (combine) b += up256(static_cast<size_t>(m * topk) * static_cast<size_t>(gated ? n / 2 : n) * 4);
  return b;
}

hipError_t launch_product(const Product& p, void* workspace, Queue q) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Epi ep = p.ep;
  const float* part = reinterpret_cast<const float*>(ws);
  if (p.combine) {  // fp32 rows first, then their sums
    ep.y = ws;
    ep.y_dt = static_cast<int>(DType::F32);
    ep.residual = nullptr;
    ws = behind(ws, up256(static_cast<size_t>(p.m * p.topk) * static_cast<size_t>(ep.ldy) * 4));
  }
  hipError_t e = hipSuccess;
  const bool many = many_rows(p.m, p.topk, p.experts);
  const bool plain = p.experts == 0 && ep.half == 0 && ep.act == kActNone && ep.bias == nullptr &&
                     ep.residual == nullptr && ep.y_dt != static_cast<int>(DType::BF16);
  if (plain && !many && p.xt == DType::F16 && gemv_is_faster(p.m, p.n, p.k)) {
    if (!q.dry)  // (one launch)
      e = launch_gemv(p.x, p.xt, p.W, ep.y, static_cast<DType>(ep.y_dt), static_cast<int>(p.m), p.n, p.k, q.s);
  } else if (p.xt != DType::F32 && fused_wave_supports(p.m, p.topk, p.experts, p.n, p.k, p.x_rows)) {
    e = launch_fused_wave(p, ep, plan_rows(p), plan_layout(p.m, p.topk, p.experts).max_tiles, q);
  } else if (p.xt != DType::F32 && p.experts == 0 &&
             fused_split_supports(p.m, ep.ldy, p.n, p.k, p.xt == DType::BF16)) {
    e = launch_fused_split(p, ep, q);
  } else if (many || (p.xt != DType::F32 && fused_gemv_supports(p.n, p.k, p.x_rows, p.experts))) {
    const half_t* xs = static_cast<const half_t*>(p.x);
    const float* scale = nullptr;
    if (p.xt == DType::BF16) {
      e = launch_stage(p.x, p.x_rows, p.k, ws, &xs, &scale, q);
      if (e != hipSuccess) return e;
      ws = behind(ws, stage_bytes(p.x_rows, p.k));
    }
    PlanLayout L{};
    if (p.experts != 0) L = plan_layout(p.m, p.topk, p.experts);
    if (many) e = launch_fused_gemm(p, ep, plan_rows(p), xs, scale, L.max_tiles, ws, q);
    else e = launch_fused_gemv(p, ep, plan_rows(p), xs, scale, L.max_tiles, L.tile_rows, q);
  } else if (p.xt == DType::F32) {
    e = launch_row<float>(p, ep, q);
  } else if (p.xt == DType::F16) {
    e = launch_row<half_t>(p, ep, q);
  } else {
    e = launch_row<bf16_t>(p, ep, q);
  }
  if (e != hipSuccess || !p.combine) return e;
  const PlanLayout L = plan_layout(p.m, p.topk, p.experts);
  const float* w = p.weights;
  const int* pos = p.plan != nullptr ? p.plan + L.pos : nullptr;
  int64_t nout = ep.ldy;
  const int v = nout % 4 == 0 ? 4 : 1;
  int topk = static_cast<int>(p.topk), cblocks = static_cast<int>((nout + 256 * v - 1) / (256 * v));
  Epi out = p.ep;
  void* argv[] = {&part, &w, &pos, &topk, &nout, &cblocks, &out};
  const void* fn = v == 4 ? reinterpret_cast<const void*>(&combine_kernel<4>)
                          : reinterpret_cast<const void*>(&combine_kernel<1>);
  return launch_blocks(fn, p.m * cblocks, 256, argv, 0, q);
}

}  // namespace q4
