// Routing of tokens to experts, and the order of the chosen pairs by expert.
//
// Choice: one wavefront per token, see q4_route_token.hpp.
//
// Plan: a stable counting sort of the pairs by expert.  One workgroup per
// expert counts the earlier experts' pairs in an LDS histogram (integer adds:
// their order does not matter) and places its own in ascending order by
// ballots.  Up to 16 tokens run as one workgroup and one launch.
//
// Bound by latency and by the instructions of the choice: 4096 tokens of 256
// experts are 2 MB of logits (0.4 us at 5 TB/s) and 0.6 MB of outputs.
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
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int waves = (pairs + kWave - 1) / kWave;
  __syncthreads();
  const int id = tid < pairs ? s.ids[tid] : -1;  // (-1 matches no pair)
  // Lanes of this wavefront with the same id: agreement in every bit of id + 1.
  uint64_t same = ~uint64_t{0};
#pragma unroll
  for (int b = 0; b < 11; ++b) {  // (id + 1 <= kMaxExperts + 1 < 2^11)
    const bool set = (((id + 1) >> b) & 1) != 0;
    const uint64_t who = __ballot(set);
    same &= set ? who : ~who;
  }
  int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
  if (id >= 0 && rank == 0) s.count[wave][id] = static_cast<uint16_t>(__popcll(same));
  __syncthreads();
  // Thread e: expert e's pairs and tiles, and those of the experts before it.
  int c = 0;
  if (tid < experts)
    for (int w = 0; w < waves; ++w) c += s.count[w][tid];
  const int tc = (c + L.tile_rows - 1) / L.tile_rows;
  int p = c, t = tc;  // inclusive sums over the wave
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
  if (id >= 0)
    for (int w = 0; w < wave; ++w) rank += s.count[w][id];
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

// Workgroup e < experts places expert e's pairs, workgroup `experts` what is
// left: the order behind the last pair, the pairs without an expert, the totals.
// Wavefront w takes the w-th sixteenth of the ids, 64 at a time: the earlier
// experts' counts go into an LDS histogram (their tiles come before its own,
// without gaps: tile slots left empty between the experts' cost the products a
// quarter of their time), its own are counted and placed by ballots.
__global__ __launch_bounds__(kThreads) void plan_kernel(const int* __restrict__ ids, int pairs, int experts,
                                                        PlanLayout L, int* __restrict__ plan) {
  __shared__ int hist[kMaxExperts + 1];
  __shared__ int mine_s[kWaves], first_s, tile_s;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int me = blockIdx.x;
  for (int e = tid; e < me; e += kThreads) hist[e] = 0;
  __syncthreads();
  const int chunks = (pairs + kThreads - 1) / kThreads;
  const int p0 = wave * chunks * kWave;
  constexpr int kAhead = 8;  // loads in flight
  // Ids of chunks c0 .. c0 + 7; experts + 1 (which counts nowhere) past the end.
  auto load = [&](int c0, int (&id)[kAhead]) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int p = p0 + (c0 + u) * kWave + lane;
      id[u] = ids[p < pairs ? p : pairs - 1];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = c0 + u < chunks && p0 + (c0 + u) * kWave + lane < pairs;
      id[u] = !in ? experts + 1 : id[u] < 0 || id[u] >= experts ? experts : id[u];
    }
  };
  int mine = 0;
  for (int c0 = 0; c0 < chunks; c0 += kAhead) {
    int id[kAhead];
    load(c0, id);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      mine += __popcll(__ballot(id[u] == me));
      if (id[u] < me) atomicAdd(&hist[id[u]], 1);
    }
  }
  if (lane == 0) mine_s[wave] = mine;
  __syncthreads();
  if (wave == 0) {
    int f = 0, t = 0;
    for (int e = lane; e < me; e += kWave) {
      f += hist[e];
      t += (hist[e] + L.tile_rows - 1) / L.tile_rows;
    }
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      f += __shfl_xor(f, off);
      t += __shfl_xor(t, off);
    }
    if (lane == 0) {
      first_s = f;
      tile_s = t;
    }
  }
  __syncthreads();
  const int first = first_s, tile0 = tile_s;
  int count = 0, before = 0;  // before: in the earlier wavefronts' shares
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int n = mine_s[w];
    count += n;
    if (w < wave) before += n;
  }
  const bool rest = me == experts;
  if (tid == 0) {
    plan[me] = first;
    if (rest) {
      plan[L.head] = tile0;
      plan[L.head + 1] = L.tile_rows;
    }
  }
  if (!rest && wave == 0)
    for (int i = lane; i * L.tile_rows < count; i += kWave) write_tile(me, i, first, count, tile0, L, plan);
  int at = before;
  for (int c0 = 0; c0 < chunks; c0 += kAhead) {
    int id[kAhead];
    load(c0, id);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint64_t mask = __ballot(id[u] == me);
      if (id[u] == me) {
        const int p = p0 + (c0 + u) * kWave + lane;
        const int r = at + __popcll(mask & ((uint64_t{1} << lane) - 1));
        if (rest) {
          plan[L.order + first + r] = -1;
          plan[L.pos + p] = -1;
        } else {
          place_pair(p, r, first, tile0, L, plan);
        }
      }
      at += __popcll(mask);
    }
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
  return hipLaunchKernel(reinterpret_cast<const void*>(&plan_kernel), dim3(static_cast<unsigned>(experts + 1)),
                         dim3(kThreads), argv, 0, s);
}

}  // namespace q4
