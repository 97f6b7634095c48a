// An expert layer of one token in two launches.
//
// With one token each launch and each round trip to memory counts: the layer's
// reached weights (8 experts of 1536 x 2048 and 2048 x 768: 21 MB) take 4 us at
// 5 TB/s, four launches (routing and plan, gate and up, down, sum) took 25.7 us,
// these two take 19.2 (11.7 and 6.8 of the device's).
//   moe_one_up_kernel: every workgroup chooses the token's experts itself (one
//     wavefront, while another stages the row of x), takes the expert of its
//     place in the choice and streams its share of that expert's rows.
//   moe_one_down_kernel: wavefront j of a workgroup streams the j-th expert's rows
//     for the workgroup's 16 output columns; their sum, weighted in the order of
//     j, is formed in LDS, so no rows of single experts are written.
// The same sums in the same order as the four launches: the same bits.
#include "q4_route_token.hpp"
#include "q4_wave_stream.hpp"

namespace q4 {
namespace {

constexpr int kLdsMax = 160 * 1024;
constexpr int kUpWaves = 4, kRing = 4;
constexpr int kPerLane = 4;  // experts per lane: up to 256
constexpr int kOneTopk = 16;

struct OneUp {
  const void* logits;
  int dt;
  RouteParams route;
  int* ids;        // of the choice, for the second launch
  float* weights;
  Epi ep;          // y: [topk][nout]
  int64_t wstride, nbias;
  int parts;       // workgroups per chosen expert
};

template <typename K, bool GATED, bool SHIFT, bool XB>
__global__ __launch_bounds__(kUpWaves * kWave) void moe_one_up_kernel(const half_t* __restrict__ x,
                                                                      const uint8_t* __restrict__ W,
                                                                      int64_t k, OneUp a) {
  constexpr int kCols = GATED ? 8 : 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int place = blockIdx.x / a.parts, part = blockIdx.x - place * a.parts;
  // LDS: the row, {its factor, the expert}, scores and keys of the choice, rings.
  const int xpieces = static_cast<int>(k / 8);
  const int xbytes = (xpieces + 1) * 16;
  float* const factor_s = reinterpret_cast<float*>(smem + xbytes);
  int* const expert_s = reinterpret_cast<int*>(factor_s + 1);
  double* const scores = reinterpret_cast<double*>(smem + xbytes + 16);
  K* const keys = reinterpret_cast<K*>(scores + kPerLane * kWave);
  const int ring_at = xbytes + 16 + kPerLane * kWave * 16 + wave * (kRing * slot_bytes<SHIFT>);
  if (wave == 0) {
    const Choice c = route_token<kPerLane, K>(a.logits, a.dt, 0, a.route, scores, keys);
    if (lane == place) *expert_s = c.id;
    if (blockIdx.x == 0 && lane < a.route.topk) {
      a.ids[lane] = c.id;
      a.weights[lane] = c.weight;
    }
  } else if (wave == 1) {
    for (int i0 = 0; i0 < xpieces; i0 += kWave)
      if (i0 + lane < xpieces) dma16(x + 8 * (i0 + lane), smem + i0 * 16);
    wait_vm<0>();
    float f = 1.0f;
    if constexpr (XB) f = stage_row_bf16(reinterpret_cast<u32x4*>(smem), xpieces);
    if (lane == 0) *factor_s = f;
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(*expert_s);
  if (e < 0) return;  // no expert in this place (uniform)
  const float factor = *factor_s;
  const int64_t all = (a.ep.ldy + kCols - 1) / kCols;
  const int64_t t_end = all * (part + 1) / a.parts, t_begin = all * part / a.parts + wave;
  const int ntiles = t_begin < t_end ? static_cast<int>((t_end - t_begin + kUpWaves - 1) / kUpWaves) : 0;
  const int r = lane & 15, g = lane >> 4;
  RowStream<kRing, GATED, SHIFT> stream;
  stream.begin(smem, ring_at, W + e * a.wstride, k, a.ep.ldy, a.ep.half, t_begin, kUpWaves, ntiles);
  stream.prologue();
  stream.run(smem + 8 * g, [&](int64_t t, const float4_t& acc) {  // (every operand row is the token's)
    const int64_t c = t * kCols + (GATED ? r >> 1 : r);
    const float z = acc[0] * factor;
    const float u = GATED ? __shfl_xor(z, 1) : 0.f;
    if (g == 0 && c < a.ep.ldy && (!GATED || (r & 1) == 0))
      finish_store(a.ep, e * a.nbias, place, c, z, u);
  });
}

struct OneDown {
  const int* ids;
  const float* weights;
  Epi ep;  // y: [nout]
  int64_t wstride, nbias;
  int tiles;  // row tiles per workgroup
};

// One wavefront per chosen expert.
template <bool SHIFT, bool XB>
__global__ __launch_bounds__(kOneTopk * kWave) void moe_one_down_kernel(const half_t* __restrict__ h,
                                                                        const uint8_t* __restrict__ W,
                                                                        int64_t k, OneDown a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int topk = blockDim.x / kWave;
  const int xpieces = static_cast<int>(k / 8);
  // LDS: every wavefront's row and ring, then the rows' results [wave][16 tiles].
  const int own = (xpieces + 1) * 16 + kRing * slot_bytes<SHIFT>;
  uint8_t* const mine = smem + wave * own;
  float* const results = reinterpret_cast<float*>(smem + topk * own);
  const int64_t all = (a.ep.ldy + 15) / 16;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tiles;
  const int ntiles = static_cast<int>(all - t0 < a.tiles ? all - t0 : a.tiles);
  const int e = a.ids[wave];
  const int r = lane & 15, g = lane >> 4;
  if (e >= 0) {
    const half_t* const row = h + wave * k;
    for (int i0 = 0; i0 < xpieces; i0 += kWave)
      if (i0 + lane < xpieces) dma16(row + 8 * (i0 + lane), mine + i0 * 16);
    RowStream<kRing, false, SHIFT> stream;
    stream.begin(smem, wave * own + (xpieces + 1) * 16, W + e * a.wstride, k, a.ep.ldy, 0, t0, 1, ntiles);
    wait_vm_upto<kCopies * kRing>(stream.prologue());
    compiler_fence();
    float factor = 1.0f;
    if constexpr (XB) {
      factor = stage_row_bf16(reinterpret_cast<u32x4*>(mine), xpieces);
      wait_lgkm0();
    }
    stream.run(mine + 8 * g, [&](int64_t t, const float4_t& acc) {
      const int64_t c = t * 16 + r;
      if (g == 0 && c < a.ep.ldy)
        results[(wave * a.tiles + static_cast<int>(t - t0)) * 16 + r] =
            finish(a.ep, e * a.nbias, c, acc[0] * factor, 0.f);
    });
  }
  __syncthreads();
  for (int o = threadIdx.x; o < ntiles * 16; o += blockDim.x) {
    const int64_t c = t0 * 16 + o;
    if (c >= a.ep.ldy) continue;
    float v = 0.f;
    for (int j = 0; j < topk; ++j)
      if (a.ids[j] >= 0) v = fmaf(a.weights[j], results[j * a.tiles * 16 + o], v);
    if (a.ep.residual != nullptr) v += load_f32(a.ep.residual, a.ep.y_dt, c);
    store_as(a.ep.y, a.ep.y_dt, c, v);
  }
}

using KernelFn = const void*;

int up_lds(int64_t k, bool shift) {
  return static_cast<int>(staged_bytes(k)) + 16 + kPerLane * kWave * 16 +
         kUpWaves * kRing * (shift ? slot_bytes<true> : slot_bytes<false>);
}
int down_lds(int64_t k, bool shift, int64_t topk, int tiles) {
  return static_cast<int>(topk * (staged_bytes(k) + kRing * (shift ? slot_bytes<true> : slot_bytes<false>) +
                                  tiles * 64));
}

// Row tiles per workgroup of the second launch: one workgroup per compute unit
// where there are more.
int down_tiles(int64_t nout) {
  const int64_t cu = device_cu_count(), all = (nout + 15) / 16;
  return static_cast<int>((all + cu - 1) / cu);
}

hipError_t launch(KernelFn fn, std::atomic<uint64_t>& allowed, int64_t grid, int threads, int lds, void** argv,
                  Queue q) {
  return launch_blocks(fn, grid, threads, argv, static_cast<size_t>(lds), q, 1, 1, kLdsMax, &allowed);
}

template <typename K>
KernelFn up_kernel(bool gated, bool shift, bool xb) {
  static const KernelFn fns[8] = {reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, false, false, false>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, false, false, true>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, false, true, false>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, false, true, true>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, true, false, false>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, true, false, true>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, true, true, false>),
                                  reinterpret_cast<KernelFn>(&moe_one_up_kernel<K, true, true, true>)};
  return fns[(gated ? 4 : 0) + (shift ? 2 : 0) + (xb ? 1 : 0)];
}

}  // namespace

bool moe_one_supports(const RouteArgs& r, const Product& up, const Product& down) {
  if (r.m != 1 || r.topk > kOneTopk || r.experts > kPerLane * kWave || up.xt == DType::F32 ||
      up.k > (1 << 15) || down.k > (1 << 15) || !fused_gemv_supports(up.n, up.k, 1, r.experts) ||
      !fused_gemv_supports(down.n, down.k, r.topk, r.experts))
    return false;
  return up_lds(up.k, up.k % 256 != 0) <= kLdsMax &&
         down_lds(down.k, down.k % 256 != 0, r.topk, down_tiles(down.n)) <= kLdsMax;
}

hipError_t launch_moe_one(const RouteArgs& r, const Product& up, const Product& down, Queue q) {
  const bool xb = up.xt == DType::BF16, gated = up.ep.half != 0;
  const int64_t cu = device_cu_count();
  {
    const bool shift = up.k % 256 != 0;
    const int64_t row_tiles = (up.ep.ldy + (gated ? 7 : 15)) / (gated ? 8 : 16);
    // Three or four workgroups of four wavefronts fit a compute unit; two each
    // already have every row tile of an ordinary expert on a wavefront of its own.
    const int64_t want = (2 * cu + r.topk - 1) / r.topk, most = (row_tiles + kUpWaves - 1) / kUpWaves;
    OneUp a{r.logits, static_cast<int>(r.dt), route_params(r), r.ids, r.weights, up.ep,
            up.n * (up.k / kQK) * kBlockBytes, up.n, static_cast<int>(want < most ? want : most)};
    const half_t* x = static_cast<const half_t*>(up.x);
    const uint8_t* W = up.W;
    int64_t k = up.k;
    void* argv[] = {&x, &W, &k, &a};
    const bool sums = sum_keys(r);
    static std::atomic<uint64_t> allowed[16];
    const int at = (sums ? 8 : 0) + (gated ? 4 : 0) + (shift ? 2 : 0) + (xb ? 1 : 0);
    const hipError_t e =
        launch(sums ? up_kernel<uint64_t>(gated, shift, xb) : up_kernel<uint32_t>(gated, shift, xb), allowed[at],
               r.topk * a.parts, kUpWaves * kWave, up_lds(k, shift), argv, q);
    if (e != hipSuccess) return e;
  }
  const bool shift = down.k % 256 != 0;
  OneDown a{r.ids, r.weights, down.ep, down.n * (down.k / kQK) * kBlockBytes, down.n, down_tiles(down.n)};
  const half_t* h = static_cast<const half_t*>(down.x);
  const uint8_t* W = down.W;
  int64_t k = down.k;
  void* argv[] = {&h, &W, &k, &a};
  const KernelFn fn = shift ? (xb ? reinterpret_cast<KernelFn>(&moe_one_down_kernel<true, true>)
                                  : reinterpret_cast<KernelFn>(&moe_one_down_kernel<true, false>))
                            : (xb ? reinterpret_cast<KernelFn>(&moe_one_down_kernel<false, true>)
                                  : reinterpret_cast<KernelFn>(&moe_one_down_kernel<false, false>));
  static std::atomic<uint64_t> allowed[4];
  const int64_t grid = ((down.n + 15) / 16 + a.tiles - 1) / a.tiles;
  return launch(fn, allowed[(shift ? 2 : 0) + (xb ? 1 : 0)], grid, static_cast<int>(r.topk) * kWave,
                down_lds(k, shift, r.topk, a.tiles), argv, q);
}

}  // namespace q4
