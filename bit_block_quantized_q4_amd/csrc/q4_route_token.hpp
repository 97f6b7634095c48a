// The choice of one token's experts by one wavefront (gfx950).  Internal header.
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
#pragma once

#include "q4_fused.hpp"

namespace q4 {
namespace {

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

// Chooses token t's experts; every lane of the wave calls it.  Lane j <
// topk gets the j-th: its id (-1: none) and weight.  K: uint64_t where keys are
// sums with the score, else uint32_t.  `scores`, `keys`: LDS of this wave, 64 NPL
// entries each (scores for sums only, keys with groups only).
struct Choice {
  int id;
  float weight;
};
template <int NPL, typename K>
__device__ __forceinline__ Choice route_token(const void* logits, int dt, int64_t t, const RouteParams& a,
                                              double* scores, K* keys) {
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
  return Choice{my_id, static_cast<float>(w * static_cast<double>(a.scale))};
}

inline RouteParams route_params(const RouteArgs& a) {
  return RouteParams{a.bias, static_cast<int>(a.experts), static_cast<int>(a.topk), a.sigmoid, a.groups,
                     a.group_topk, a.top2, a.renormalise, a.scale};
}

// Whether keys are sums with the score (see route_token).
inline bool sum_keys(const RouteArgs& a) { return a.bias != nullptr || (a.groups > 1 && a.top2); }

}  // namespace
}  // namespace q4
