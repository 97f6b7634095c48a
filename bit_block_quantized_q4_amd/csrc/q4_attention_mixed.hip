// Attention over the paged Q4_0 cache where offsets say how many rows a sequence has,
// which the host does not know: one launch whose first workgroups take the sequences
// of few rows and whose others those of many, and one that joins what either left in
// parts.  (Four launches in a row, two of them for nothing, were 9 us longer.)
#include "q4_attention_few.hpp"
#include "q4_attention_many.hpp"

namespace q4 {
namespace {

// Most rows (query rows times heads per kv head) of a sequence of few.  16 sequences within
// a window of 4096, by this way and by that of many rows: 15 rows 33 and 59 us, 25 rows 44 and
// 61, 35 rows 59 and 67, 50 rows 61 and 75, 65 rows 78 either way; 64 sequences of 4096, 30
// rows 90 and 282, 40 rows 160 and 183.  (Up to 64 would be no worse, and some 15% better from
// 33 on.)
constexpr int kFewRows = 32;

template <int NB, int NT>
union Lds {
  FewLds<NB, NT> few;
  ManyLds<NB> many;
};

template <int NB, int NT, bool BF16>
__global__ __launch_bounds__(kWaves* kWave, NB > 4 ? 1 : NB > 2 ? 2 : 3) void attention_mixed_kernel(Attention a, Few f, Many y,
                                                                                          int few) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dynamic[];
  Lds<NB, NT>& lds = *reinterpret_cast<Lds<NB, NT>*>(dynamic);
  if (static_cast<int>(blockIdx.x) < few) attention_few<NB, NT, BF16>(a, f, blockIdx.x, few, lds.few);
  else attention_many<NB, BF16>(a, y, blockIdx.x - few, lds.many);
}

template <int NB, int NT>
__global__ __launch_bounds__(kWaves* kWave) void attention_finish_kernel(Attention a, Parts parts, Many y, int joins) {
  const int block = blockIdx.x;
  if (block < joins) attention_join<NB, NT>(a, parts, block / (2 * NT), block / 2 % NT, block & 1);
  else attention_splits<NB>(a, y, (block - joins) / kWaves, (block - joins) % kWaves);
}

int few_workgroups(const Attention& a) { return many_per_unit(a.cache.dim) * device_cu_count(); }

std::atomic<uint64_t> g_allowed[8][2][2];

template <int NB, int NT, bool BF16>
hipError_t launch_as(const Attention& a, Few& f, Many& y, int few, Queue q) {
  constexpr int kLds = sizeof(Lds<NB, NT>);
  Attention args = a;
  void* argv[] = {&args, &f, &y, &few};
  const int64_t rows = y.places * a.cache.kv_heads;
  const hipError_t e = launch_blocks(reinterpret_cast<const void*>(&attention_mixed_kernel<NB, NT, BF16>),
                                     few + rows * y.splits, kWaves * kWave, argv, kLds, q, 1, 1, kLds,
                                     &g_allowed[NB - 1][NT - 1][BF16]);
  int joins = f.whole ? 0 : 2 * NT * few;
  const int64_t blocks = joins + (y.splits > 1 ? rows * kWaves : 0);
  if (e != hipSuccess || blocks == 0) return e;
  void* finish[] = {&args, &f.parts, &y, &joins};
  return launch_blocks(reinterpret_cast<const void*>(&attention_finish_kernel<NB, NT>), blocks, kWaves * kWave, finish,
                       0, q);
}

template <int NB>
hipError_t launch_dim(const Attention& a, Few& f, Many& y, int few, Queue q) {
  const bool bf = a.qt == DType::BF16;
  if constexpr (NB > 2 && NB <= 6) {
    if (few_row_tiles(a) == 2)
      return bf ? launch_as<NB, 2, true>(a, f, y, few, q) : launch_as<NB, 2, false>(a, f, y, few, q);
  }
  return bf ? launch_as<NB, 1, true>(a, f, y, few, q) : launch_as<NB, 1, false>(a, f, y, few, q);
}

size_t first_bytes(const Attention& a) { return (few_bytes(a, few_workgroups(a)) + 255) / 256 * 256; }

}  // namespace

size_t attention_mixed_bytes(const Attention& a) { return first_bytes(a) + many_bytes(a); }

hipError_t launch_attention_mixed(const Attention& a, void* workspace, Queue q) {
  const int few = few_workgroups(a);
  Few f = make_few(a, few, kFewRows, workspace);
  Many y = make_many(a, kFewRows + 1, behind(workspace, first_bytes(a)));
  switch (a.cache.dim / kQK) {
    case 1: return launch_dim<1>(a, f, y, few, q);
    case 2: return launch_dim<2>(a, f, y, few, q);
    case 3: return launch_dim<3>(a, f, y, few, q);
    case 4: return launch_dim<4>(a, f, y, few, q);
    case 5: return launch_dim<5>(a, f, y, few, q);
    case 6: return launch_dim<6>(a, f, y, few, q);
    case 7: return launch_dim<7>(a, f, y, few, q);
    default: return launch_dim<8>(a, f, y, few, q);
  }
}

}  // namespace q4
