// Routing of tokens to experts, and the order of the chosen pairs by expert.
//
// Choice (one wavefront per token): lane l holds experts l, l + 64, ...
//   s = softmax(l) or sigmoid(l);  key = s + bias, or the logit itself
// The keys are unsigned integers in their order: 32 bits where a logit is the
// key, else 64 (of the double s + bias, so that the order of near ties is that
// of the exact values).  The topk largest are taken one by one: every lane's
// best, the wave's largest upper word (DPP row shifts and broadcasts, no LDS),
// and only where several lanes hold it the lower word and then the index.
// Scores are formed in 64 bits, and where the logit is the key only for the
// chosen (and, for a softmax that is not renormalised, its sum).  With groups
// the keys pass through LDS once, where 64 / groups lanes per group find its
// two best.
//
// Plan: a stable counting sort of the pairs by expert.  One workgroup per
// expert counts the earlier experts' pairs in an LDS histogram (integer adds:
// their order does not matter) and places its own in ascending order by
// ballots.  Up to 16 tokens run as one workgroup and one launch.
//
// Bound by latency and by the instructions of the choice: 4096 tokens of 256
// experts are 2 MB of logits (0.4 us at 5 TB/s) and 0.6 MB of outputs.
#include "q4_fused.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 1024;
constexpr int kOneTokens = 16;  // most tokens of a single-workgroup routing,
constexpr int kOnePerLane = 4;  // and most experts per lane (its waves' LDS)

struct RouteParams {
  const float* bias;
  int experts, topk, sigmoid, groups, group_topk, top2, renormalise;
  float scale;
};

// ------------------------------------------------------------------ choice

// The largest value of the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint32_t o = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), decltype(ctrl)::value,
                                                   decltype(rows)::value, 0xF, false);
    v = o > v ? o : v;
  };
  step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // row_shr:1
  step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});  // row_shr:2
  step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});  // row_shr:4
  step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});  // row_shr:8
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast:15
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row_bcast:31
  return __builtin_amdgcn_readlane(v, 63);
}

// Unsigned integers in the order of the values (-0 as +0; NaN never comes
// here); 0 stands for "none".
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return (b >> 63) != 0 ? ~b : b | (uint64_t{1} << 63);
}
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (b >> 31) != 0 ? ~b : b | (1u << 31);
}

// Index (64 i + lane) of the wave's largest key[i], the lowest among equal
// ones; -1 if every key is 0.  Uniform.
template <int NPL, typename K>
__device__ __forceinline__ int wave_first(const K (&key)[NPL]) {
  const int lane = threadIdx.x & (kWave - 1);
  K k = key[0];
  int at = lane;
#pragma unroll
  for (int i = 1; i < NPL; ++i)
    if (key[i] > k) {
      k = key[i];
      at = lane + kWave * i;
    }
  const uint32_t hi = static_cast<uint32_t>(sizeof(K) == 8 ? static_cast<uint64_t>(k) >> 32 : k);
  const uint32_t most = wave_max(hi);
  uint64_t who = __ballot(hi == most);
  if constexpr (sizeof(K) == 8) {
    if ((who & (who - 1)) != 0) {
      const uint32_t lo = hi == most ? static_cast<uint32_t>(k) : 0u;
      const uint32_t least = wave_max(lo);
      if (most == 0 && least == 0) return -1;
      who = __ballot(hi == most && lo == least);
    }
  } else {
    if (most == 0) return -1;
  }
  if constexpr (NPL > 1) {
    if ((who & (who - 1)) != 0) {  // equal keys: the lowest index
      const bool mine = ((who >> lane) & 1) != 0;
      const uint32_t best = wave_max(mine ? ~static_cast<uint32_t>(at) : 0u);
      return static_cast<int>(~best);
    }
  }
  return __builtin_amdgcn_readlane(at, __builtin_ctzll(who));
}

// Chooses token t's experts; every lane of the wave calls it.  K: uint64_t
// where keys are sums with the score, else uint32_t.  `scores`, `keys`: LDS of
// this wave, 64 NPL entries each (scores for sums and softmax totals only, keys
// with groups only).
template <int NPL, typename K>
__device__ __forceinline__ void route_token(const void* logits, int dt, int64_t t, const RouteParams& a,
                                            double* scores, K* keys, int* ids, float* weights, int* hist) {
  constexpr bool kSum = sizeof(K) == 8;
  const int lane = threadIdx.x & (kWave - 1);
  const double ninf = -__builtin_inf();
  const int E = a.experts;
  constexpr float kMax = 3.4028234663852886e38f;

  float l[NPL];  // -infinity: not to be chosen
  float top = -kMax;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + kWave * i;
    l[i] = -__builtin_inff();
    if (e < E) {
      const float v = load_f32(logits, dt, t * E + e);
      if (v > -__builtin_inff()) l[i] = fminf(v, kMax);  // (false for NaN)
    }
    top = fmaxf(top, l[i]);
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
  }
  auto raw = [&](float v) {  // the score, a softmax's without its sum
    if (!(v > -__builtin_inff())) return 0.0;
    return a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v)))
                     : exp(static_cast<double>(v) - static_cast<double>(top));
  };
  K rank[NPL];
  double inv = 1.0;  // 1 / sum of a softmax
  if (kSum || (!a.sigmoid && !a.renormalise)) {
    double score[NPL], sum = 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      score[i] = raw(l[i]);
      sum += score[i];
    }
    if (!a.sigmoid) {
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) sum += __shfl_xor(sum, off);
      inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    if constexpr (kSum) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + kWave * i;
        double k = score[i] * inv;
        scores[e] = k;
        if (a.bias != nullptr && e < E) k += static_cast<double>(a.bias[e]);
        rank[i] = l[i] > -__builtin_inff() && k > ninf ? ordered(k) : 0;  // (no NaN bias either)
      }
    }
  }
  if constexpr (!kSum) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) rank[i] = l[i] > -__builtin_inff() ? ordered(l[i]) : 0;
  }

  if (a.groups > 1) {
    const int per = E / a.groups;
    int lpg = kWave;  // lanes per group: a power of two
    while (lpg * a.groups > kWave) lpg >>= 1;
#pragma unroll
    for (int i = 0; i < NPL; ++i) keys[lane + kWave * i] = rank[i];
    wait_lgkm0();  // this wave's own writes, complete
    const int g = lane / lpg, sub = lane % lpg;
    K b0 = 0, b1 = 0;
    if (g < a.groups)
      for (int j = sub; j < per; j += lpg) {
        const K v = keys[g * per + j];
        const K lo = v < b0 ? v : b0;
        b0 = v > b0 ? v : b0;
        b1 = lo > b1 ? lo : b1;
      }
    for (int off = 1; off < lpg; off <<= 1) {
      const K o0 = __shfl_xor(b0, off), o1 = __shfl_xor(b1, off);
      const K lo = o0 < b0 ? o0 : b0, hi1 = o1 > b1 ? o1 : b1;
      b0 = o0 > b0 ? o0 : b0;
      b1 = lo > hi1 ? lo : hi1;
    }
    K gk[1] = {sub == 0 && g < a.groups ? b0 : 0};
    if constexpr (kSum) {
      // The sum of the two, from their integers back.
      auto value = [](uint64_t k) {
        return __builtin_bit_cast(double, (k >> 63) != 0 ? k & ~(uint64_t{1} << 63) : ~k);
      };
      if (a.top2 && gk[0] != 0 && b1 != 0) gk[0] = ordered(value(b0) + value(b1));
    }
    uint64_t open = 0;  // bit: a lane that stands for a chosen group
    for (int r = 0; r < a.group_topk; ++r) {
      const int at = wave_first<1>(gk);
      if (at < 0) break;
      open |= uint64_t{1} << at;
      if (lane == at) gk[0] = 0;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + kWave * i;
      if (e < E && ((open >> (e / per * lpg)) & 1) == 0) rank[i] = 0;
    }
  }

  // The chosen, one by one; lane j keeps the j-th.
  int my_id = -1;
  for (int j = 0; j < a.topk; ++j) {
    const int e = wave_first<NPL>(rank);
    if (e < 0) break;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e == lane + kWave * i) rank[i] = 0;
    if (lane == j) my_id = e;
  }
  if constexpr (kSum) wait_lgkm0();  // the scores' writes
  double w = 0.0;
  if (my_id >= 0) {
    if constexpr (kSum) {
      w = scores[my_id];
    } else {
      w = raw(fminf(load_f32(logits, dt, t * E + my_id), kMax)) * inv;
    }
  }
  if (a.renormalise) {
    double total = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) total += __shfl_xor(total, off);  // (topk <= 32 lanes)
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < a.topk) {
    ids[t * a.topk + lane] = my_id;
    weights[t * a.topk + lane] = static_cast<float>(w * static_cast<double>(a.scale));
    if (hist != nullptr) atomicAdd(&hist[my_id < 0 ? E : my_id], 1);
  }
}

// ------------------------------------------------------------------ plan

struct PlanLds {
  int total[kMaxExperts + 1];  // pairs per expert; the last entry: without one
  int base[kMaxExperts + 1];   // next place of an expert's pairs
  int tile0[kMaxExperts];      // first tile
  int wave_pairs[kWaves], wave_tiles[kWaves];
  alignas(16) int ids[kThreads];
};

// Offsets (into base[]) and first tiles from the totals: thread e scans expert e.
__device__ __forceinline__ void scan_experts(PlanLds& s, int experts, int tile_rows) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int c = tid < experts ? s.total[tid] : 0;
  const int tc = (c + tile_rows - 1) / tile_rows;
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

// Tiles of expert e (c pairs from place `first`), written by one wavefront.
__device__ __forceinline__ void write_tiles(int e, int first, int c, int tile0, const PlanLayout& L,
                                            int* plan) {
  for (int i = threadIdx.x & (kWave - 1); i * L.tile_rows < c; i += kWave) {
    const int left = c - i * L.tile_rows;
    *reinterpret_cast<int4*>(plan + L.tiles + static_cast<int64_t>(tile0 + i) * L.rec_words) =
        int4{e, first + i * L.tile_rows, left < L.tile_rows ? left : L.tile_rows, 0};
  }
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

// The whole plan of at most kThreads pairs whose counts are in s.total, by one
// workgroup.
__device__ __forceinline__ void plan_one(PlanLds& s, const int* ids, int pairs, int experts,
                                         const PlanLayout& L, int* plan) {
  const int tid = threadIdx.x, wave = tid / kWave;
  scan_experts(s, experts, L.tile_rows);
  if (tid <= experts) plan[tid] = s.base[tid];
  if (experts == kThreads && tid == 0) plan[experts] = s.base[experts];
  if (tid == 0) {
    plan[L.head] = s.tile0[experts - 1] + (s.total[experts - 1] + L.tile_rows - 1) / L.tile_rows;
    plan[L.head + 1] = L.tile_rows;
  }
  for (int e = wave; e < experts; e += kWaves) write_tiles(e, s.base[e], s.total[e], s.tile0[e], L, plan);
  int id = -1;  // (behind the end: matches no pair)
  if (tid < pairs) {
    id = ids[tid];
    if (id < 0 || id >= experts) id = experts;
  }
  s.ids[tid] = id;
  // Lanes of this wavefront with the same id: agreement in every bit of id + 1.
  uint64_t same = ~uint64_t{0};
#pragma unroll
  for (int b = 0; b < 11; ++b) {  // (id + 1 <= kMaxExperts + 1 < 2^11)
    const bool set = (((id + 1) >> b) & 1) != 0;
    const uint64_t who = __ballot(set);
    same &= set ? who : ~who;
  }
  __syncthreads();
  if (id >= 0) {
    int rank = 0;  // earlier pairs of the same expert
    const int4* v4 = reinterpret_cast<const int4*>(s.ids);
#pragma unroll 4
    for (int j = 0; j < wave * (kWave / 4); ++j) {
      const int4 v = v4[j];
      rank += (v.x == id) + (v.y == id) + (v.z == id) + (v.w == id);
    }
    rank += __popcll(same & ((uint64_t{1} << (tid & (kWave - 1))) - 1));
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
  const int tid = threadIdx.x, wave = tid / kWave;
  for (int e = tid; e <= a.experts; e += kThreads) s.total[e] = 0;
  __syncthreads();
  for (int t = wave; t < m; t += kWaves)
    route_token<NPL, K>(logits, dt, t, a, scores[sizeof(K) == 8 ? wave : 0], keys[wave], ids, weights,
                        s.total);
  if (plan == nullptr) return;
  __syncthreads();
  plan_one(s, ids, m * a.topk, a.experts, L, plan);
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
    route_token<NPL, K>(logits, dt, t, a, scores[sizeof(K) == 8 ? wave : 0], keys[wave], ids, weights,
                        nullptr);
}

// The plan of given ids by one workgroup (at most kThreads pairs).
__global__ __launch_bounds__(kThreads) void plan_one_kernel(const int* __restrict__ ids, int pairs,
                                                            int experts, PlanLayout L,
                                                            int* __restrict__ plan) {
  __shared__ PlanLds s;
  const int tid = threadIdx.x;
  for (int e = tid; e <= experts; e += kThreads) s.total[e] = 0;
  __syncthreads();
  if (tid < pairs) {
    const int id = ids[tid];
    atomicAdd(&s.total[id < 0 || id >= experts ? experts : id], 1);
  }
  __syncthreads();
  plan_one(s, ids, pairs, experts, L, plan);
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
  if (!rest && wave == 0) write_tiles(me, first, count, tile0, L, plan);
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
  RouteParams r{a.bias, static_cast<int>(a.experts), static_cast<int>(a.topk), a.sigmoid, a.groups,
                a.group_topk, a.top2, a.renormalise, a.scale};
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
  if (a.bias != nullptr || (a.groups > 1 && a.top2)) return launch_route_k<NPL, uint64_t>(a, s);
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
