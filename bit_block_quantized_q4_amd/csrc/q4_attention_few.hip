// Attention over the paged Q4_0 cache for one row a sequence: no offsets to look at.
#include "q4_attention_few.hpp"

namespace q4 {
namespace {

// Workgroups of a compute unit: registers for two wavefronts on a SIMD, or for one.
constexpr int per_unit(int nb, int nt) { return nb * nt > 8 || nb == 8 ? 1 : 2; }

template <int NB, int NT, bool BF16>
__global__ __launch_bounds__(kWaves* kWave, per_unit(NB, NT)) void attention_few_kernel(Attention a, Few f) {
  __shared__ __attribute__((aligned(16))) FewLds<NB, NT> lds;
  attention_few<NB, NT, BF16>(a, f, blockIdx.x, gridDim.x, lds);
}

template <int NB, int NT>
__global__ __launch_bounds__(kWaves* kWave) void attention_join_kernel(Attention a, Parts parts) {
  attention_join<NB, NT>(a, parts, blockIdx.x, blockIdx.y >> 1, blockIdx.y & 1);
}

template <int NB, int NT>
__global__ __launch_bounds__(kWaves* kWave) void attention_join_wide_kernel(Attention a, Parts parts) {
  __shared__ __attribute__((aligned(16))) JoinLds lds;
  const int y = blockIdx.y;
  attention_join_wide<NB, NT>(a, parts, blockIdx.x, y / (2 * NB), y / NB % 2, y % NB, lds);
}

// Notes up to which their parts are spread over workgroups.
constexpr int kWideNotes = 64;

int workgroups(const Attention& a) {
  return per_unit(a.cache.dim / kQK, few_row_tiles(a)) * device_cu_count();
}

template <int NB, int NT, bool BF16>
hipError_t launch_as(const Attention& a, Few& f, int n, Queue q) {
  Attention args = a;
  void* argv[] = {&args, &f};
  const hipError_t e = launch_blocks(reinterpret_cast<const void*>(&attention_few_kernel<NB, NT, BF16>), n,
                                     kWaves * kWave, argv, 0, q);
  if (e != hipSuccess || f.whole) return e;
  void* joined[] = {&args, &f.parts};
  const int notes = f.parts.jobs ? f.parts.jobs : n;
  if (notes <= kWideNotes)
    return launch_blocks(reinterpret_cast<const void*>(&attention_join_wide_kernel<NB, NT>), notes, kWaves * kWave,
                         joined, 0, q, 2 * NT * NB);
  return launch_blocks(reinterpret_cast<const void*>(&attention_join_kernel<NB, NT>), notes, kWaves * kWave, joined, 0,
                       q, 2 * NT);
}

template <int NB>
hipError_t launch_dim(const Attention& a, Few& f, int n, Queue q) {
  const bool bf = a.qt == DType::BF16;
  if constexpr (NB <= 6) {
    if (few_row_tiles(a) == 2) return bf ? launch_as<NB, 2, true>(a, f, n, q) : launch_as<NB, 2, false>(a, f, n, q);
  }
  return bf ? launch_as<NB, 1, true>(a, f, n, q) : launch_as<NB, 1, false>(a, f, n, q);
}

}  // namespace

size_t attention_few_bytes(const Attention& a) { return few_bytes(a, workgroups(a)); }

hipError_t launch_attention_few(const Attention& a, void* workspace, Queue q) {
  const int n = workgroups(a);
  Few f = make_few(a, n, INT32_MAX, workspace);
  switch (a.cache.dim / kQK) {
    case 1: return launch_dim<1>(a, f, n, q);
    case 2: return launch_dim<2>(a, f, n, q);
    case 3: return launch_dim<3>(a, f, n, q);
    case 4: return launch_dim<4>(a, f, n, q);
    case 5: return launch_dim<5>(a, f, n, q);
    case 6: return launch_dim<6>(a, f, n, q);
    case 7: return launch_dim<7>(a, f, n, q);
    default: return launch_dim<8>(a, f, n, q);
  }
}

}  // namespace q4
