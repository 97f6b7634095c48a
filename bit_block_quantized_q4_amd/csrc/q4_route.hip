// Routing of tokens to experts, and the order of the chosen pairs by expert.
//
// route_kernel: one wavefront per token.  Lane l holds experts l, l + 64, ...
//   s = softmax(l) or sigmoid(l);  key = s + bias, or the logit itself
// in 64 bits, so that the order of near ties is that of the exact values.
// The topk largest keys are taken one by one: every lane's best, then the
// wave's by xor shuffles, (key, index) compared with the lower index first.
//
// plan_kernel: one workgroup per expert.  Each counts all ids in an LDS
// histogram (integer adds: the result does not depend on their order), scans
// it, and places its own expert's pairs in ascending order by ballots.
#include "q4_fused.hpp"

namespace q4 {
namespace {

constexpr int kRouteWaves = 4;  // tokens per workgroup

struct RouteParams {
  const float* bias;
  int experts, topk, sigmoid, groups, group_topk, top2, renormalise;
  float scale;
};

// The wave's best (key, index): the largest key, the lowest index among equal
// ones; every lane returns it.  Keys are never NaN.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const double ok = __shfl_xor(key, off);
    const int oi = __shfl_xor(idx, off);
    if (ok > key || (ok == key && oi < idx)) {
      key = ok;
      idx = oi;
    }
  }
}

template <int NPL>
__device__ __forceinline__ void lane_best(const double (&key)[NPL], double& k, int& idx) {
  const int lane = threadIdx.x & (kWave - 1);
  k = key[0];
  idx = lane;
#pragma unroll
  for (int i = 1; i < NPL; ++i)
    if (key[i] > k) {
      k = key[i];
      idx = lane + kWave * i;
    }
}

template <int NPL>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(const void* __restrict__ logits,
                                                                    int dt, int64_t m, RouteParams a,
                                                                    int* __restrict__ ids,
                                                                    float* __restrict__ weights) {
  __shared__ double keys[kRouteWaves][NPL * kWave];  // groups only
  __shared__ uint8_t open[kRouteWaves][NPL * kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave;
  if (t >= m) return;  // whole wavefront; only wave-local exchange below
  const double ninf = -__builtin_inf();
  const int E = a.experts;

  float l[NPL];
  bool live[NPL];
  float top = -3.4028234663852886e38f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + kWave * i;
    l[i] = 0.f;
    live[i] = false;
    if (e < E) {
      const float v = load_f32(logits, dt, t * E + e);
      live[i] = v > -__builtin_inff();  // false for NaN
      l[i] = fminf(v, 3.4028234663852886e38f);
      if (live[i]) top = fmaxf(top, l[i]);
    }
  }
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));

  double score[NPL], key[NPL];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const double v = l[i];
    if (a.sigmoid) score[i] = live[i] ? 1.0 / (1.0 + exp(-v)) : 0.0;
    else score[i] = live[i] ? exp(v - static_cast<double>(top)) : 0.0;
    sum += score[i];
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) sum += __shfl_xor(sum, off);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) score[i] *= inv;
  }
  const bool additive = a.bias != nullptr || (a.groups > 1 && a.top2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + kWave * i;
    double k = additive ? score[i] : static_cast<double>(l[i]);
    if (a.bias != nullptr && e < E) k += static_cast<double>(a.bias[e]);
    key[i] = live[i] && k > ninf ? k : ninf;  // (a NaN bias too)
  }

  if (a.groups > 1) {
    const int per = E / a.groups;
    double* kw = keys[wave];
    uint8_t* ow = open[wave];
#pragma unroll
    for (int i = 0; i < NPL; ++i) kw[lane + kWave * i] = key[i];
    wait_lgkm0();  // one wavefront: its own writes are visible once complete
    double gk[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int g = lane + kWave * i;
      double b0 = ninf, b1 = ninf;
      if (g < a.groups) {
        for (int j = 0; j < per; ++j) {
          const double v = kw[g * per + j];
          if (v > b0) {
            b1 = b0;
            b0 = v;
          } else if (v > b1) {
            b1 = v;
          }
        }
      }
      gk[i] = a.top2 && b1 > ninf ? b0 + b1 : b0;
      ow[g] = 0;
    }
    wait_lgkm0();
    for (int r = 0; r < a.group_topk; ++r) {
      double k;
      int g;
      lane_best<NPL>(gk, k, g);
      wave_best(k, g);
      if (!(k > ninf)) break;  // uniform
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (g == lane + kWave * i) {
          gk[i] = ninf;
          ow[g] = 1;
        }
    }
    wait_lgkm0();
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + kWave * i;
      if (e < E && !ow[e / per]) key[i] = ninf;
    }
  }

  // The chosen, one by one; lane j keeps the j-th.
  int my_id = -1;
  double my_w = 0.0, total = 0.0;
  for (int j = 0; j < a.topk; ++j) {
    double k;
    int e;
    lane_best<NPL>(key, k, e);
    wave_best(k, e);
    if (!(k > ninf)) break;  // uniform
    double w = 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e == lane + kWave * i) {
        w = score[i];
        key[i] = ninf;
      }
    w = __shfl(w, e & (kWave - 1));
    total += w;
    if (lane == j) {
      my_id = e;
      my_w = w;
    }
  }
  if (lane < a.topk) {
    if (a.renormalise) my_w = total > 0.0 ? my_w / total : 0.0;
    ids[t * a.topk + lane] = my_id;
    weights[t * a.topk + lane] = static_cast<float>(my_w * static_cast<double>(a.scale));
  }
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kMaxExperts = 1024;

// Workgroup e < experts places expert e's pairs and writes its tiles and
// offset; workgroup `experts` fills what is left: the order behind the last
// pair, the places of the pairs without an expert, and the totals.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int* __restrict__ ids, int64_t pairs,
                                                            int experts, PlanLayout L,
                                                            int* __restrict__ plan) {
  __shared__ int hist[kMaxExperts + 1];
  __shared__ int before[kPlanWaves];
  __shared__ int first_s, tile_s;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int me = blockIdx.x;
  for (int i = tid; i <= experts; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  for (int64_t p = tid; p < pairs; p += kPlanThreads) {
    const int id = ids[p];
    const int at = id >= 0 && id < experts ? id : experts;
    if (at <= me) atomicAdd(&hist[at], 1);
  }
  __syncthreads();
  // Pairs and tiles of the experts before this one.
  if (wave == 0) {
    int f = 0, t = 0;
    for (int i = lane; i < me; i += kWave) {
      f += hist[i];
      t += (hist[i] + L.tile_rows - 1) / L.tile_rows;
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
  const int first = first_s, tile0 = tile_s, count = hist[me];
  int* order = plan + L.order;
  int* pos = plan + L.pos;
  if (tid == 0) {
    plan[me] = first;
    if (me == experts) {
      plan[L.head] = tile0;
      plan[L.head + 1] = L.tile_rows;
    }
  }
  const bool rest = me == experts;
  if (!rest) {
    int4* tiles = reinterpret_cast<int4*>(plan + L.tiles);
    for (int i = tid; i * L.tile_rows < count; i += kPlanThreads) {
      const int left = count - i * L.tile_rows;
      tiles[tile0 + i] = int4{me, first + i * L.tile_rows, left < L.tile_rows ? left : L.tile_rows, 0};
    }
  }
  // This expert's pairs in ascending order.
  int at = first;
  for (int64_t p0 = 0; p0 < pairs; p0 += kPlanThreads) {
    const int64_t p = p0 + tid;
    bool mine = false;
    if (p < pairs) {
      const int id = ids[p];
      mine = (id >= 0 && id < experts ? id : experts) == me;
    }
    const uint64_t mask = __ballot(mine);
    if (lane == 0) before[wave] = __popcll(mask);
    __syncthreads();
    int mine_at = at + __popcll(mask & ((uint64_t{1} << lane) - 1));
    int all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w < wave) mine_at += before[w];
      all += before[w];
    }
    if (mine) {
      order[mine_at] = rest ? -1 : static_cast<int>(p);
      pos[p] = rest ? -1 : mine_at;
    }
    at += all;
    __syncthreads();
  }
}

template <int NPL>
hipError_t launch_route_n(const RouteArgs& a, hipStream_t s) {
  const void* logits = a.logits;
  int dt = static_cast<int>(a.dt);
  int64_t m = a.m;
  RouteParams r{a.bias, static_cast<int>(a.experts), static_cast<int>(a.topk), a.sigmoid, a.groups,
                a.group_topk, a.top2, a.renormalise, a.scale};
  int* ids = a.ids;
  float* weights = a.weights;
  void* argv[] = {&logits, &dt, &m, &r, &ids, &weights};
  return hipLaunchKernel(reinterpret_cast<const void*>(&route_kernel<NPL>),
                         dim3(static_cast<unsigned>((m + kRouteWaves - 1) / kRouteWaves)),
                         dim3(kRouteWaves * kWave), argv, 0, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.experts <= 64) e = launch_route_n<1>(a, s);
  else if (a.experts <= 128) e = launch_route_n<2>(a, s);
  else if (a.experts <= 256) e = launch_route_n<4>(a, s);
  else if (a.experts <= 512) e = launch_route_n<8>(a, s);
  else e = launch_route_n<16>(a, s);
  if (e != hipSuccess || a.plan == nullptr) return e;
  return launch_route_plan(a.ids, a.m, a.topk, a.experts, a.plan, s);
}

hipError_t launch_route_plan(const int* ids, int64_t m, int64_t topk, int64_t experts, int* plan,
                             hipStream_t s) {
  PlanLayout L = plan_layout(m, topk, experts);
  int64_t pairs = m * topk;
  int ne = static_cast<int>(experts);
  void* argv[] = {&ids, &pairs, &ne, &L, &plan};
  return hipLaunchKernel(reinterpret_cast<const void*>(&plan_kernel),
                         dim3(static_cast<unsigned>(experts + 1)), dim3(kPlanThreads), argv, 0, s);
}

}  // namespace q4
