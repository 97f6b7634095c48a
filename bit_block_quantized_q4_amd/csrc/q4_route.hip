// Routing of tokens to experts, and the order of the chosen pairs by expert.
//
// Choice: one wavefront per token, see q4_route_token.hpp.
//
// Plan: a stable counting sort of the pairs by expert, in one launch: every
// workgroup counts all pairs in LDS (integer adds: their order does not matter)
// and places its own, ranked by ballots.  Up to 16 tokens run as one workgroup
// and one launch with their choice.
//
// Bound by latency and by the instructions of the choice: 4096 tokens of 256
// experts are 2 MB of logits (0.4 us at 5 TB/s) and 0.6 MB of outputs; with groups,
// a bias and eight chosen the choice takes 12.9 us and the plan 8.0.  16 tokens of
// 128 experts: 8.0 us with the call.
#include "q4_route_token.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 1024;
constexpr int kOneTokens = 16;  // most tokens of a single-workgroup routing,
constexpr int kOnePerLane = 4;  // and most experts per lane (its waves' LDS)

// Lane j's choice as the j-th of token t.
__device__ __forceinline__ void write_choice(const Choice& c, int64_t t, const RouteParams& a, int* ids,
                                             float* weights) {
  const int lane = threadIdx.x & (kWave - 1);
  if (lane >= a.topk) return;
  ids[t * a.topk + lane] = c.id;
  weights[t * a.topk + lane] = c.weight;
}

// ------------------------------------------------------------------ plan

struct PlanLds {
  int base[kMaxExperts + 1];  // next place of an expert's pairs; at the end: of those without one
  int tile0[kMaxExperts];     // first tile
  int wave_pairs[kWaves], wave_tiles[kWaves];
  int ids[kThreads];
  uint16_t count[kWaves][kMaxExperts + 1];  // pairs per wavefront and expert (the last entry: without one)
};

// Clears the counts of `pairs` pairs; plan_one's first barrier is behind it.
__device__ __forceinline__ void clear_counts(PlanLds& s, int pairs, int experts) {
  const int waves = (pairs + kWave - 1) / kWave;
  for (int w = 0; w < waves; ++w)
    for (int e = threadIdx.x; e <= experts; e += kThreads) s.count[w][e] = 0;
}

// The earlier lanes of this wavefront with the same id (-1: none); its count by
// their first lane into s.count.
__device__ __forceinline__ int rank_in_wave(PlanLds& s, int id) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  uint64_t same = ~uint64_t{0};  // agreement in every bit of id + 1
#pragma unroll
  for (int b = 0; b < 11; ++b) {  // (id + 1 <= kMaxExperts + 1 < 2^11)
    const bool set = (((id + 1) >> b) & 1) != 0;
    const uint64_t who = __ballot(set);
    same &= set ? who : ~who;
  }
  const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
  if (id >= 0 && rank == 0) s.count[wave][id] = static_cast<uint16_t>(__popcll(same));
  return rank;
}

// Thread e < experts has expert e's pairs c and tiles tc, also in p and t; these
// become the sums up to and with e.  First places and tiles into s, behind a
// barrier.
__device__ __forceinline__ void scan_experts(PlanLds& s, int experts, int c, int tc, int& p, int& t) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int op = __shfl_up(p, off), ot = __shfl_up(t, off);
    if (lane >= off) {
      p += op;
      t += ot;
    }
  }
  if (lane == kWave - 1) {
    s.wave_pairs[wave] = p;
    s.wave_tiles[wave] = t;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int op = s.wave_pairs[w], ot = s.wave_tiles[w];
    if (w < wave) {
      p += op;
      t += ot;
    }
  }
  if (tid < experts) {
    s.base[tid] = p - c;
    s.tile0[tid] = t - tc;
    if (tid == experts - 1) s.base[experts] = p;
  }
  __syncthreads();
}

// Tile i of expert e, which has c pairs from place `first` on.
__device__ __forceinline__ void write_tile(int e, int i, int first, int c, int tile0, const PlanLayout& L,
                                           int* plan) {
  const int left = c - i * L.tile_rows;
  *reinterpret_cast<int4*>(plan + L.tiles + static_cast<int64_t>(tile0 + i) * L.rec_words) =
      int4{e, first + i * L.tile_rows, left < L.tile_rows ? left : L.tile_rows, 0};
}

// Pair p is the r-th of its expert, whose places start at `first` and whose
// tiles at tile0.
__device__ __forceinline__ void place_pair(int p, int r, int first, int tile0, const PlanLayout& L,
                                           int* plan) {
  plan[L.order + first + r] = p;
  plan[L.pos + p] = first + r;
  const int t = r / L.tile_rows;
  plan[L.tiles + static_cast<int64_t>(tile0 + t) * L.rec_words + 4 + (r - t * L.tile_rows)] = p;
}

// The whole plan of at most kThreads pairs by one workgroup, one pair per
// thread.  Their ids are in s.ids (`experts` for a pair without one), the counts
// cleared.  A pair's rank among its expert's is the count of the earlier
// wavefronts and of the earlier lanes.  Nothing goes to memory before the last
// barrier, which would wait for it.
__device__ __forceinline__ void plan_one(PlanLds& s, int pairs, int experts, const PlanLayout& L, int* plan) {
  const int tid = threadIdx.x, wave = tid / kWave;
  const int waves = (pairs + kWave - 1) / kWave;
  __syncthreads();
  const int id = tid < pairs ? s.ids[tid] : -1;  // (-1 matches no pair)
  int rank = rank_in_wave(s, id);
  __syncthreads();
  int c = 0;
  if (tid < experts)
    for (int w = 0; w < waves; ++w) c += s.count[w][tid];
  if (id >= 0)
    for (int w = 0; w < wave; ++w) rank += s.count[w][id];
  const int tc = (c + L.tile_rows - 1) / L.tile_rows;
  int p = c, t = tc;
  scan_experts(s, experts, c, tc, p, t);
  if (tid < experts) {
    plan[tid] = p - c;
    for (int i = 0; i < tc; ++i) write_tile(tid, i, p - c, c, t - tc, L, plan);
    if (tid == experts - 1) {
      plan[experts] = p;
      plan[L.head] = t;
      plan[L.head + 1] = L.tile_rows;
    }
  }
  if (id >= 0) {
    if (id < experts) {
      place_pair(tid, rank, s.base[id], s.tile0[id], L, plan);
    } else {
      plan[L.order + s.base[id] + rank] = -1;
      plan[L.pos + tid] = -1;
    }
  }
}

// Up to kOneTokens tokens and kThreads pairs: choice and plan in one workgroup.
template <int NPL, typename K>
__global__ __launch_bounds__(kThreads) void route_one_kernel(const void* __restrict__ logits, int dt,
                                                             int m, RouteParams a, int* ids,
                                                             float* weights, PlanLayout L, int* plan) {
  __shared__ PlanLds s;
  __shared__ double scores[sizeof(K) == 8 ? kWaves : 1][NPL * kWave];
  __shared__ K keys[kWaves][NPL * kWave];
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
  if (plan != nullptr) clear_counts(s, m * a.topk, a.experts);
  static_assert(kOneTokens <= kWaves, "one token per wavefront");
  Choice c{-1, 0.0f};
  if (wave < m) {
    c = route_token<NPL, K>(logits, dt, wave, a, scores[sizeof(K) == 8 ? wave : 0], keys[wave]);
    if (lane < a.topk) s.ids[wave * a.topk + lane] = c.id < 0 ? a.experts : c.id;
  }
  if (plan != nullptr) plan_one(s, m * a.topk, a.experts, L, plan);
  if (wave < m) write_choice(c, wave, a, ids, weights);
}

// Choice, one token per wavefront.
template <int NPL, typename K>
__global__ __launch_bounds__(4 * kWave) void route_kernel(const void* __restrict__ logits, int dt,
                                                          int64_t m, RouteParams a,
                                                          int* __restrict__ ids,
                                                          float* __restrict__ weights) {
  __shared__ double scores[sizeof(K) == 8 ? 4 : 1][NPL * kWave];
  __shared__ K keys[4][NPL * kWave];
  const int wave = threadIdx.x / kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t < m)
    write_choice(route_token<NPL, K>(logits, dt, t, a, scores[sizeof(K) == 8 ? wave : 0], keys[wave]), t, a,
                 ids, weights);
}

// The plan of given ids by one workgroup (at most kThreads pairs).
__global__ __launch_bounds__(kThreads) void plan_one_kernel(const int* __restrict__ ids, int pairs,
                                                            int experts, PlanLayout L,
                                                            int* __restrict__ plan) {
  __shared__ PlanLds s;
  const int tid = threadIdx.x;
  if (tid < pairs) {
    const int id = ids[tid];
    s.ids[tid] = id < 0 || id >= experts ? experts : id;
  }
  clear_counts(s, pairs, experts);
  plan_one(s, pairs, experts, L, plan);
}

// Workgroup g places the pairs g span .. (g + 1) span - 1, after counting all
// pairs by expert, those before its own apart: integer adds in LDS, four copies
// by lane so that pairs of one expert meet less often, 32 ids per thread in
// flight.  (Tiles are numbered without gaps: slots left empty between the experts'
// cost the products a quarter of their time.)  32768 pairs of 256 experts: 8.0
// us; with a workgroup per expert that placed that expert's pairs, 17.0.
constexpr int kCopies = 4, kQuads = 8;
__global__ __launch_bounds__(kThreads) void plan_kernel(const int* __restrict__ ids, int pairs, int experts,
                                                        int span, PlanLayout L, int* __restrict__ plan) {
  __shared__ PlanLds s;
  __shared__ int hist[2][kCopies][kMaxExperts + 1];  // before this workgroup's pairs, and from them on
  __shared__ int before[kMaxExperts + 1];
  const int tid = threadIdx.x, wave = tid / kWave;
  const int begin = blockIdx.x * span;
  const int end = pairs - begin < span ? pairs : begin + span;
  for (int e = tid; e <= experts; e += kThreads)
#pragma unroll
    for (int i = 0; i < kCopies; ++i) hist[0][i][e] = hist[1][i][e] = 0;
  __syncthreads();
  auto expert = [&](int id) { return id < 0 || id >= experts ? experts : id; };
  auto add = [&](int p, int id) { atomicAdd(&hist[p < begin ? 0 : 1][tid % kCopies][expert(id)], 1); };
  const int quads = pairs / 4;
  for (int q0 = 0; q0 < quads; q0 += kThreads * kQuads) {
    int4 v[kQuads];
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int q = q0 + u * kThreads + tid;
      v[u] = reinterpret_cast<const int4*>(ids)[q < quads ? q : quads - 1];
    }
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int q = q0 + u * kThreads + tid;
      if (q < quads) {
        add(4 * q, v[u].x);
        add(4 * q, v[u].y);
        add(4 * q, v[u].z);
        add(4 * q, v[u].w);
      }
    }
  }
  if (tid < pairs - 4 * quads) add(4 * quads + tid, ids[4 * quads + tid]);
  __syncthreads();
  int c = 0;
  for (int e = tid; e <= experts; e += kThreads) {
    int b = 0, n = 0;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      b += hist[0][i][e];
      n += hist[1][i][e];
    }
    before[e] = b;
    if (e == tid && e < experts) c = b + n;
  }
  const int tc = (c + L.tile_rows - 1) / L.tile_rows;
  int p = c, t = tc;
  scan_experts(s, experts, c, tc, p, t);
  if (tid < experts) {
    for (int i = blockIdx.x; i < tc; i += gridDim.x) write_tile(tid, i, p - c, c, t - tc, L, plan);
    if (blockIdx.x == 0) {
      plan[tid] = p - c;
      if (tid == experts - 1) {
        plan[experts] = p;
        plan[L.head] = t;
        plan[L.head + 1] = L.tile_rows;
      }
    }
  }
  for (int p0 = begin; p0 < end; p0 += kThreads) {
    const int at = p0 + tid;
    const int id = at < end ? expert(ids[at]) : -1;
    clear_counts(s, kThreads, experts);
    __syncthreads();
    int rank = rank_in_wave(s, id);
    __syncthreads();
    if (id >= 0) {
      for (int w = 0; w < wave; ++w) rank += s.count[w][id];
      rank += before[id];
      if (id < experts) {
        place_pair(at, rank, s.base[id], s.tile0[id], L, plan);
      } else {
        plan[L.order + s.base[id] + rank] = -1;
        plan[L.pos + at] = -1;
      }
    }
    if (p0 + kThreads >= end) break;
    __syncthreads();
    for (int e = tid; e <= experts; e += kThreads)
      for (int w = 0; w < kWaves; ++w) before[e] += s.count[w][e];
    __syncthreads();
  }
}

template <int NPL, typename K>
hipError_t launch_route_k(const RouteArgs& a, hipStream_t s) {
  const void* logits = a.logits;
  int dt = static_cast<int>(a.dt);
  RouteParams r = route_params(a);
  int* ids = a.ids;
  float* weights = a.weights;
  int* plan = a.plan;
  if constexpr (NPL <= kOnePerLane) {
    if (a.m <= kOneTokens && a.m * a.topk <= kThreads) {
      PlanLayout L = plan_layout(a.m, a.topk, a.experts);
      int m = static_cast<int>(a.m);
      void* argv[] = {&logits, &dt, &m, &r, &ids, &weights, &L, &plan};
      return hipLaunchKernel(reinterpret_cast<const void*>(&route_one_kernel<NPL, K>), dim3(1),
                             dim3(kThreads), argv, 0, s);
    }
  }
  int64_t m = a.m;
  void* argv[] = {&logits, &dt, &m, &r, &ids, &weights};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&route_kernel<NPL, K>),
                                       dim3(static_cast<unsigned>((m + 3) / 4)), dim3(4 * kWave), argv, 0, s);
  if (e != hipSuccess || plan == nullptr) return e;
  return launch_route_plan(ids, a.m, a.topk, a.experts, plan, s);
}

template <int NPL>
hipError_t launch_route_n(const RouteArgs& a, hipStream_t s) {
  if (sum_keys(a)) return launch_route_k<NPL, uint64_t>(a, s);
  return launch_route_k<NPL, uint32_t>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.experts <= 64) return launch_route_n<1>(a, s);
  if (a.experts <= 128) return launch_route_n<2>(a, s);
  if (a.experts <= 256) return launch_route_n<4>(a, s);
  if (a.experts <= 512) return launch_route_n<8>(a, s);
  return launch_route_n<16>(a, s);
}

hipError_t launch_route_plan(const int* ids, int64_t m, int64_t topk, int64_t experts, int* plan,
                             hipStream_t s) {
  PlanLayout L = plan_layout(m, topk, experts);
  int pairs = static_cast<int>(m * topk), ne = static_cast<int>(experts);
  void* argv[] = {&ids, &pairs, &ne, &L, &plan};
  if (pairs <= kThreads)
    return hipLaunchKernel(reinterpret_cast<const void*>(&plan_one_kernel), dim3(1), dim3(kThreads), argv, 0, s);
  // A workgroup per 1024 pairs, up to one per compute unit (each reads all ids).
  const int64_t chunks = (m * topk + kThreads - 1) / kThreads, cu = device_cu_count();
  int span = static_cast<int>((chunks + cu - 1) / cu) * kThreads;
  void* argl[] = {&ids, &pairs, &ne, &span, &L, &plan};
  return launch_blocks(reinterpret_cast<const void*>(&plan_kernel), (pairs + span - 1) / span, kThreads, argl, 0, Queue{s});
}

}  // namespace q4
