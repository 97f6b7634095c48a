// Attention over the paged Q4_0 cache for sequences of few rows: single tokens and
// drafts.  Internal header.
//
//   s = scale sum_b dk[t, b] sum_j (ck[t, b, j] - 8) q_bj;  m, l running;
//   O = sum_t exp2(x_t - m) (cv[t, j] - 8) dv[t, b]
//
// A kv head's heads and a sequence's rows together are the rows of one product, so a
// position's keys and values are read once for all of them.  Products are transposed
// (positions or columns by rows): S^T = K Q^T leaves a lane the scores of one row, and
// for positions in the order below they are, rounded to fp16, the right operand of
// O^T = V^T P^T as they stand: no exchange between lanes, no LDS.
//
// A tile is 64 positions, four granules.  Lane l, with m = l % 16, g = l / 16:
//   K  product u (0 .. 3) has position 16 (m / 4) + 4 u + m % 4 in row m, so that the
//      scores of lane group g are the sixteen positions of granule g.  The lane's codes
//      are word g of each block: product (u, b) is block b alone, its codes exact
//      integers, the scale an fp32 factor of the result;
//   V  the lane holds columns m and m + 16 of each block for granule g's positions, as
//      16 bytes; scales multiply in fp16 (one rounding of the decoded value).
//
// Work is cut evenly by tiles: a workgroup takes a run of them over sequences, heads
// and rows as they come, its four wavefronts every fourth tile, and adds up the
// wavefronts' parts in LDS.  A sequence's head that lies in one workgroup is finished
// there; the others' parts go through the workspace to a second launch.  All orders are
// fixed by the lengths.
//
// Bound by memory where rows are few: 64 sequences of 2048 to 8192 positions (380 MB of
// cache, 40 heads of 128 on 8) take 94 us, 4.0 TB/s of a large copy's 4.65, of which 5 are
// the joining; one of 131072 (151 MB) 43.5, 5 of them the joining; one of 1000 12.5, three
// quarters of it the two launches and the wait for the first bytes.  With 32 rows (five
// tokens of five heads each, 16 sequences within a window of 4096: 43 us) vector
// instructions issue in 55% of the busy cycles, beside 1 TB/s: a code is still taken apart once,
// but exp, maximum and conversion are each row's.  The rest is waiting at both ends of a
// workgroup's run of some 15 tiles, and 5 us of joining.
#pragma once

#include "q4_attention.hpp"

namespace q4 {

// Parts of rows in the workspace: for each slot NT x 16 rows of (maximum, sum), then
// their columns as the lanes hold them.
struct Parts {
  // What is noted of the rows whose first part lies with a workgroup as its last one:
  // {parts (0: there are none), workgroup, sequence, kv head << 16 | first row / 16}; a note
  // per workgroup, or (jobs) one for each head and 16 NT rows of it.
  int* notes = nullptr;
  int jobs = 0;
  float* stats = nullptr;   // [slots][16 NT][2]
  float4_t* cols = nullptr; // [slots][NT][2][NB][64]
};

struct Few {
  int max_rows = 0;  // sequences of more rows are left out
  int least = 1;     // units that a workgroup takes at least
  int whole = 0;     // heads are not cut: nothing is left to join
  Parts parts;
};

struct Work {
  Seq q;
  int tile0, tiles, row_tiles;
};

template <int R>
__device__ __forceinline__ Work work_of(const Attention& a, int max_rows, int s) {
  Work w;
  w.q = seq_of(a.batch, s);
  const int64_t rows = static_cast<int64_t>(w.q.rows) * a.group;
  int lo, hi;
  seen_by(a, w.q.length, w.q.first < 0 ? 0 : w.q.first, &lo, &hi);  // the first row's first
  w.tile0 = lo / kTile;
  w.tiles = (w.q.length + kTile - 1) / kTile - w.tile0;
  if (w.tiles < 1) w.tiles = 1;
  w.row_tiles = rows > max_rows ? 0 : static_cast<int>((rows + R - 1) / R);
  return w;
}
// Units that are dealt out: tiles, or with `whole` all of a head's and its rows' at once.
__device__ __forceinline__ int64_t units_of(const Attention& a, const Work& w, int whole) {
  return static_cast<int64_t>(whole ? 1 : w.tiles) * w.row_tiles * a.cache.kv_heads;
}

// A tile's bytes in registers.  Sixteen lanes want the same scales, so a lane fetches
// a share of its granule's (words m + 16 i), and they are spread through LDS.
template <int NB>
struct Keys {
  uint32_t codes[4][NB];
  uint32_t scales[(NB + 1) / 2];
};
template <int NB>
struct Values {
  u32x4 codes[NB];
  uint32_t scales[(NB + 1) / 2];
};

// A granule's page number and place, and its address (of page 0 where it names none).
struct Place {
  int id, in;
};
__device__ __forceinline__ Place place_of(const Cache& c, const Batch& b, const int* table, int g) {
  const uint32_t u = static_cast<uint32_t>(g), per = static_cast<uint32_t>(c.per_page);
  uint32_t slot = __umulhi(u, c.inverse), in = u - slot * per;
  if (in >= per) {
    ++slot;
    in -= per;
  }
  Place p;
  p.id = slot < static_cast<uint32_t>(b.max_pages) ? table[slot] : -1;
  p.in = static_cast<int>(in);
  return p;
}
template <int NB>
__device__ __forceinline__ const uint8_t* address_of(const Cache& c, const Place& p, const uint8_t* head, bool* named) {
  *named = static_cast<uint32_t>(p.id) < static_cast<uint32_t>(c.pages);
  return head + (*named ? p.id : 0) * c.page_bytes + static_cast<int64_t>(p.in) * (288 * NB);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = q[i];
}

// The LDS of a workgroup.
template <int NB, int NT>
struct FewLds {
  static constexpr int kScales = 8 * NB + 4;  // words of a granule's scales, padded
  float4_t cols[kWaves][NB][kWave];
  uint32_t spread[kWaves][2][4 * kScales];
  float stats[kWaves][16 * NT][2];
  int64_t sums[kWaves];
  int64_t found[2];
};

// Workgroup `block` of `blocks`.
template <int NB, int NT, bool BF16>
__device__ __forceinline__ void attention_few(const Attention& a, const Few& f, int block, int blocks,
                                              FewLds<NB, NT>& lds) {
  constexpr int R = 16 * NT;
  constexpr bool kTwo = !BF16 && NT == 1;  // weights in two fp16 parts (for 32 rows registers do not suffice)
  constexpr int kStep = NB * NT > 4 ? 2 : 4;  // blocks whose products wait for their scales together
  constexpr int kScales = FewLds<NB, NT>::kScales;
  auto& sums = lds.sums;
  auto& found = lds.found;
  auto& stats = lds.stats;
  auto& cols = lds.cols;
  auto& spread = lds.spread;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int m16 = lane & 15, g = lane >> 4;
  const Batch& b = a.batch;
  const Cache& c = a.cache;

  // The whole work, and the sequence where this workgroup's run begins.
  const int chunk = (b.seqs + kWaves * kWave - 1) / (kWaves * kWave);
  const int s0 = threadIdx.x * chunk;
  int64_t mine = 0;
  for (int s = s0; s < s0 + chunk && s < b.seqs; ++s) mine += units_of(a, work_of<R>(a, f.max_rows, s), f.whole);
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int64_t v = __shfl_up(upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == kWave - 1) sums[wave] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) upto += sums[w];
    total += sums[w];
  }
  int64_t per = (total + blocks - 1) / blocks;
  if (per < f.least) per = f.least;
  int64_t unit = block * per;
  const int64_t end = unit + per < total ? unit + per : total;
  int4* const notes = reinterpret_cast<int4*>(f.parts.notes);
  bool noted = false;
  if (unit < end) {
    if (upto - mine <= unit && unit < upto) {
      found[0] = s0;
      found[1] = upto - mine;
    }
    __syncthreads();
    int s = static_cast<int>(found[0]);
    int64_t base = found[1];
    s = __builtin_amdgcn_readfirstlane(s);
    Work w = work_of<R>(a, f.max_rows, s);
    int64_t units = units_of(a, w, f.whole);
    while (unit >= base + units) {
      base += units;
      w = work_of<R>(a, f.max_rows, ++s);
      units = units_of(a, w, f.whole);
    }
    // The sequence's rows and heads in turn (heads outside): the first one, and its tile.
    int64_t job = f.whole ? unit - base : (unit - base) / w.tiles;
    int t0 = f.whole ? 0 : static_cast<int>(unit - base - job * w.tiles);
    const UnpackConsts uc = make_unpack_consts();
    const Cap<true> cap(a.softcap);

    while (unit < end) {
      while (job >= static_cast<int64_t>(w.row_tiles) * c.kv_heads) {
        w = work_of<R>(a, f.max_rows, ++s);
        job = 0;
      }
      const int64_t left = f.whole ? w.tiles : end - unit;
      const int t1 = left < w.tiles - t0 ? t0 + static_cast<int>(left) : w.tiles;
      const int h = w.row_tiles == 1 ? static_cast<int>(job) : static_cast<int>(job / w.row_tiles);
      const int r0 = static_cast<int>(job - static_cast<int64_t>(h) * w.row_tiles) * R;
      const Seq q = w.q;

      // This lane's rows: what they see, and their parts of q as the right operand.
      const int rows = q.rows * a.group;
      const int last_row = r0 + R < rows ? r0 + R - 1 : rows - 1;
      int lo[NT], hi[NT];
      float mul[NT];
      half8_t qf[NT][NB];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 16 + m16;
        const int at = r < rows ? r : rows - 1;
        const int i = at / a.group;
        seen_by(a, q.length, q.first + i, &lo[nt], &hi[nt]);
        if (r >= rows) lo[nt] = hi[nt] = 0;
        const uint16_t* x = static_cast<const uint16_t*>(a.q) + (q.row + i) * a.q_stride +
                            static_cast<int64_t>(h * a.group + at - i * a.group) * (NB * kQK) + 4 * g;
        uint2 part[NB][2];
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          part[blk][0] = *reinterpret_cast<const uint2*>(x + blk * kQK);
          part[blk][1] = *reinterpret_cast<const uint2*>(x + blk * kQK + 16);
        }
        mul[nt] = a.softcap > 0.f ? a.scale : a.scale * kLog2e;
        if constexpr (BF16) {
          uint32_t top = 0;
#pragma unroll
          for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              top = max_magnitude_bf16(top, part[blk][e].x);
              top = max_magnitude_bf16(top, part[blk][e].y);
            }
          // (as positive floats, magnitudes compare as their bits do)
          const float big = max_over_groups(__builtin_bit_cast(float, top << 16));
          const int shift = bf16_row_shift(__builtin_bit_cast(uint32_t, big) >> 16);
          const float by = power_of_two(shift);
          mul[nt] *= power_of_two(-shift);
#pragma unroll
          for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              part[blk][e].x = bf16x2_scaled_to_f16x2(part[blk][e].x, by);
              part[blk][e].y = bf16x2_scaled_to_f16x2(part[blk][e].y, by);
            }
        }
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          u32x4 v;  // elements (0, 2), (1, 3), (16, 18), (17, 19) from 4 g on
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[2 * e] = query_pair(__builtin_amdgcn_perm(part[blk][e].y, part[blk][e].x, 0x05040100), 1.f);
            v[2 * e + 1] = query_pair(__builtin_amdgcn_perm(part[blk][e].y, part[blk][e].x, 0x07060302), 1.f);
          }
          qf[nt][blk] = __builtin_bit_cast(half8_t, v);
        }
      }
      // Tiles from full0 on and before full1 are seen whole by every row.
      int lo_first, hi_first, lo_last, hi_last;
      seen_by(a, q.length, q.first + r0 / a.group, &lo_first, &hi_first);
      seen_by(a, q.length, q.first + last_row / a.group, &lo_last, &hi_last);

      float m[NT], l[NT];
      float4_t o[NT][2][NB];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY;
        l[nt] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) o[nt][e][blk] = float4_t{0.f, 0.f, 0.f, 0.f};
      }

      const int* table = b.tables + static_cast<int64_t>(s) * b.max_pages;
      const uint8_t* head = c.data + h * c.head_bytes;
      const int64_t to_values = static_cast<int64_t>(c.per_page) * (288 * NB);
      Keys<NB> keys;
      Values<NB> values;
      Place pk, pv;
      bool named_v = false, next_named = false;
      const uint8_t* at_v = nullptr;
      auto places = [&](int t) {
        pk = place_of(c, b, table, (w.tile0 + t) * 4 + (m16 >> 2));
        pv = place_of(c, b, table, (w.tile0 + t) * 4 + g);
      };
      auto load_scales = [&](const uint8_t* granule, uint32_t(&w)[(NB + 1) / 2]) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(granule + 256 * NB);
#pragma unroll
        for (int i = 0; i < (NB + 1) / 2; ++i)
          if (16 * i + 16 <= 8 * NB || m16 < 8) w[i] = p[16 * i + m16];
      };
      auto spread_scales = [&](const uint32_t(&w)[(NB + 1) / 2], uint32_t* at) {
#pragma unroll
        for (int i = 0; i < (NB + 1) / 2; ++i)
          if (16 * i + 16 <= 8 * NB || m16 < 8) at[16 * i + m16] = w[i];
      };
      auto load_keys = [&]() {
        bool named;
        const uint8_t* pk_at = address_of<NB>(c, pk, head, &named);
        at_v = address_of<NB>(c, pv, head, &next_named);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          load_words(pk_at + (4 * u + (m16 & 3)) * (16 * NB) + g * (4 * NB), keys.codes[u]);
        load_scales(at_v, keys.scales);
      };
      auto load_values = [&]() {
        const uint8_t* p = at_v + to_values;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
          values.codes[blk] = *reinterpret_cast<const u32x4*>(p + blk * 256 + m16 * 16);
        load_scales(p, values.scales);
      };
      uint32_t* const ks = spread[wave][0] + g * kScales;
      uint32_t* const vs = spread[wave][1] + g * kScales;

      int t = t0 + wave;
      if (t < t1) {
        places(t);
        load_keys();
        load_values();
        named_v = next_named;
        if (t + kWaves < t1) places(t + kWaves);
      }
      for (; t < t1; t += kWaves) {
        const int first = (w.tile0 + t) * kTile;  // the tile's first position
        const bool more = t + kWaves < t1;
        // Scores.
        float x[NT][16];
        spread_scales(keys.scales, ks);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][4 * u + i] = 0.f;
#pragma unroll
          for (int b0 = 0; b0 < NB; b0 += kStep) {
            float4_t r[NT][kStep];
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
              if (b0 + j >= NB) break;
              const Codes k = codes_of(keys.codes[u][b0 + j], uc);
              const half8_t kf = join(k.l02, k.l13, k.h02, k.h13);
              const float4_t z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                r[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[nt][b0 + j], z, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
              if (b0 + j >= NB) break;
              const half4_t d = *reinterpret_cast<const half4_t*>(ks + (u * NB + b0 + j) * 2);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[nt][4 * u + i] = fmaf(static_cast<float>(d[i]), r[nt][j][i], x[nt][4 * u + i]);
            }
            // The sums are formed here, not where they are used: their parts would all
            // wait in registers.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) tie_after(x[nt][4 * u + i]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (more) load_keys();

        const bool whole = first >= lo_last && first + kTile <= hi_first && __all(named_v);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[nt][e] *= mul[nt];
          if (__builtin_expect(a.softcap > 0.f, 0)) {
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(x[nt][e]));
            if (__all(cap.near(most))) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[nt][e] = cap.of_near(x[nt][e]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[nt][e] = cap.of(x[nt][e]);
            }
          }
          if (!whole) {
            const int from = lo[nt] - first - 16 * g, to = named_v ? hi[nt] - first - 16 * g : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[nt][e] = e >= from && e < to ? x[nt][e] : -INFINITY;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        // Weights.
        half8_t p[NT][2], p2[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float top = x[nt][0];
#pragma unroll
          for (int e = 1; e < 16; ++e) top = fmaxf(top, x[nt][e]);
          top = max_over_groups(top);
          if (__any(top > m[nt])) {
            const float next = fmaxf(m[nt], top);
            const float old = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[nt] - next);
            m[nt] = next;
            l[nt] *= old;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][e][blk][i] *= old;
          }
          const float from = (m[nt] == -INFINITY ? 0.f : m[nt]) - kLift;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[nt][e] = __builtin_amdgcn_exp2f(x[nt][e] - from);
            l[nt] += x[nt][e];
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            half_t hi16[8];
            constexpr int kOrder[8] = {0, 2, 1, 3, 4, 6, 5, 7};
#pragma unroll
            for (int e = 0; e < 8; ++e) hi16[e] = static_cast<half_t>(x[nt][8 * st + kOrder[e]]);
            p[nt][st] = half8_t{hi16[0], hi16[1], hi16[2], hi16[3], hi16[4], hi16[5], hi16[6], hi16[7]};
            if constexpr (kTwo) {
              half_t lo16[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                lo16[e] = static_cast<half_t>(x[nt][8 * st + kOrder[e]] - static_cast<float>(hi16[e]));
              p2[nt][st] = half8_t{lo16[0], lo16[1], lo16[2], lo16[3], lo16[4], lo16[5], lo16[6], lo16[7]};
            }
          }
        }
        spread_scales(values.scales, vs);
        if (!whole) {  // unseen places may hold anything: their scales become 0
          const int to = named_v ? hi_last - first - 16 * g : 0, from = lo_first - first - 16 * g;
          // word i of a block's scales holds positions 4 (i / 2) + i % 2 and two further on
          for (int i = m16; i < 8 * NB; i += 16) {
            const int at = (i & 7) / 2 * 4 + (i & 1);
            const uint32_t keep = (at >= from && at < to ? 0xFFFFu : 0u) |
                                  (at + 2 >= from && at + 2 < to ? 0xFFFF0000u : 0u);
            vs[i] &= keep;
          }
        }
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const Codes v0 = codes_of(values.codes[blk][2 * st], uc), v1 = codes_of(values.codes[blk][2 * st + 1], uc);
            const u32x4 sc = *reinterpret_cast<const u32x4*>(vs + blk * 8 + st * 4);
            const half2_t d0 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(sc[0]));
            const half2_t d1 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(sc[1]));
            const half2_t d2 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(sc[2]));
            const half2_t d3 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(sc[3]));
            const half8_t low = join(v0.l02 * d0, v0.l13 * d1, v1.l02 * d2, v1.l13 * d3);
            const half8_t high = join(v0.h02 * d0, v0.h13 * d1, v1.h02 * d2, v1.h13 * d3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              o[nt][0][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(low, p[nt][st], o[nt][0][blk], 0, 0, 0);
              o[nt][1][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(high, p[nt][st], o[nt][1][blk], 0, 0, 0);
              if constexpr (kTwo) {
                o[nt][0][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(low, p2[nt][st], o[nt][0][blk], 0, 0, 0);
                o[nt][1][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(high, p2[nt][st], o[nt][1][blk], 0, 0, 0);
              }
            }
            if (st == 1) __builtin_amdgcn_sched_barrier(0);
          }
        if (more) {
          named_v = next_named;
          load_values();
          if (t + 2 * kWaves < t1) places(t + 2 * kWaves);
        }
      }

      // The wavefronts' parts together, then the rows or their part.
      const bool done = t0 == 0 && t1 == w.tiles;
      const int64_t slot = 2 * static_cast<int64_t>(block) + (t0 == 0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt] = sum_over_groups(l[nt]);
        if (g == 0) {
          stats[wave][nt * 16 + m16][0] = m[nt];
          stats[wave][nt * 16 + m16][1] = l[nt];
        }
      }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) top = fmaxf(top, stats[v][nt * 16 + m16][0]);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
          sum = fmaf(stats[v][nt * 16 + m16][1], __builtin_amdgcn_exp2f(stats[v][nt * 16 + m16][0] - ref), sum);
        const float by = __builtin_amdgcn_exp2f(m[nt] - ref);
        const int r = r0 + nt * 16 + m16;
        const int i = r / a.group;
        const int64_t at = static_cast<int64_t>(q.row + i) * a.heads + h * a.group + (r - i * a.group);
        const float inverse = sum != 0.f ? 1.f / sum : 0.f;
        if (wave == 0 && g == 0) {
          if (!done) {
            float* st = f.parts.stats + (slot * R + nt * 16 + m16) * 2;
            st[0] = top;
            st[1] = sum;
          } else if (r < rows && a.lse != nullptr) {
            a.lse[at] = sum != 0.f ? (top - kLift + log2f(sum)) * kLn2 : -INFINITY;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) cols[wave][blk][lane] = o[nt][e][blk] * by;
          __syncthreads();
          for (int blk = wave; blk < NB; blk += kWaves) {
            float4_t v = cols[0][blk][lane];
#pragma unroll
            for (int x = 1; x < kWaves; ++x) v += cols[x][blk][lane];
            if (!done) {
              f.parts.cols[((slot * NT + nt) * 2 + e) * (NB * kWave) + blk * kWave + lane] = v;
            } else if (r < rows) {
              const float out[4] = {v[0] * inverse, v[1] * inverse, v[2] * inverse, v[3] * inverse};
              store4(a.y, a.y_dt, at * (NB * kQK) + blk * kQK + e * 16 + 4 * g, out);
            }
          }
          __syncthreads();
        }
      }
      if (t0 == 0 && !f.whole && (!done || f.parts.jobs)) {
        // done, or this run ends inside the rows' tiles
        const int64_t last = unit + w.tiles - 1;
        const int count = done ? 0 : static_cast<int>(last / per - block) + 1;
        const int64_t at = f.parts.jobs ? s * static_cast<int64_t>(w.row_tiles) * c.kv_heads + job : block;
        noted = true;
        if (threadIdx.x == 0) notes[at] = int4{count, block, s, static_cast<int>(static_cast<uint32_t>(h) << 16 | r0 / 16)};
      }
      unit += f.whole ? 1 : t1 - t0;
      ++job;
      t0 = 0;
    }
  }
  if (!noted && !f.whole && !f.parts.jobs && threadIdx.x == 0) notes[block] = int4{0, 0, 0, 0};
}

// Rows whose parts lie with several workgroups: part 0 is the noting workgroup's last
// (slot 2 w + 1), part i the first one of the i-th behind it (slot 2 (w + i)).

// What 16 rows of 16 columns (block blk, half e) have in parts first, first + step, ..,
// FLIGHT of them at once.
struct Joined {
  float top = -INFINITY, sum = 0.f;
  float4_t v = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float2& st, const float4_t& part) {
    const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.f : next;
    const float old = __builtin_amdgcn_exp2f(top - ref), by = __builtin_amdgcn_exp2f(st.x - ref);
    top = next;
    sum = sum * old + st.y * by;
    v = v * old + part * by;
  }
};
template <int NB, int NT, int FLIGHT>
__device__ __forceinline__ Joined join_parts(const Parts& parts, int count, int w, int nt, int e, int blk, int first,
                                             int step) {
  const int lane = threadIdx.x & (kWave - 1), m16 = lane & 15;
  Joined o;
  for (int i0 = first; i0 < count; i0 += FLIGHT * step) {
    float2 st[FLIGHT];
    float4_t part[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {  // (behind the last one: the first again, and not added)
      const int i = i0 + j * step < count ? i0 + j * step : i0;
      const int64_t slot = 2 * (static_cast<int64_t>(w) + i) + (i == 0);
      st[j] = reinterpret_cast<const float2*>(parts.stats)[slot * (16 * NT) + nt * 16 + m16];
      part[j] = parts.cols[((slot * NT + nt) * 2 + e) * (NB * kWave) + blk * kWave + lane];
    }
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
      if (i0 + j * step < count) o.add(st[j], part[j]);
  }
  return o;
}
template <int NB>
__device__ __forceinline__ void store_joined(const Attention& a, const int4& note, const Joined& o, int nt, int e,
                                             int blk) {
  const int lane = threadIdx.x & (kWave - 1), m16 = lane & 15, g = lane >> 4;
  const Seq q = seq_of(a.batch, note.z);
  const int r = (note.w & 0xFFFF) * 16 + nt * 16 + m16;
  if (r >= q.rows * a.group) return;
  const int token = r / a.group, h = static_cast<int>(static_cast<uint32_t>(note.w) >> 16);
  const int64_t at = static_cast<int64_t>(q.row + token) * a.heads + h * a.group + (r - token * a.group);
  const float inverse = o.sum != 0.f ? 1.f / o.sum : 0.f;
  const float out[4] = {o.v[0] * inverse, o.v[1] * inverse, o.v[2] * inverse, o.v[3] * inverse};
  store4(a.y, a.y_dt, at * (NB * kQK) + blk * kQK + e * 16 + 4 * g, out);
  if (a.lse != nullptr && g == 0 && e == 0 && blk == 0)
    a.lse[at] = o.sum != 0.f ? (o.top - kLift + log2f(o.sum)) * kLn2 : -INFINITY;
}

// Many notes, few parts each: a workgroup takes 16 rows of half the columns (e) of a note,
// a wavefront every fourth block.
template <int NB, int NT>
__device__ __forceinline__ void attention_join(const Attention& a, const Parts& parts, int note_at, int nt, int e) {
  const int4 note = reinterpret_cast<const int4*>(parts.notes)[note_at];
  if (note.x == 0) return;
  for (int blk = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); blk < NB; blk += kWaves)
    store_joined<NB>(a, note, join_parts<NB, NT, 8>(parts, note.x, note.y, nt, e, blk, 0, 1), nt, e, blk);
}

// Few notes of many parts: a workgroup takes 16 rows of 16 columns, a wavefront every fourth
// part.  (For many notes that are mostly empty starting so many workgroups takes 9 us.)
struct JoinLds {
  float4_t cols[kWaves][kWave];
  float2 stats[kWaves][16];
};
template <int NB, int NT>
__device__ __forceinline__ void attention_join_wide(const Attention& a, const Parts& parts, int note_at, int nt, int e,
                                                    int blk, JoinLds& lds) {
  const int4 note = reinterpret_cast<const int4*>(parts.notes)[note_at];
  if (note.x == 0) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const Joined mine = join_parts<NB, NT, 16>(parts, note.x, note.y, nt, e, blk, wave, kWaves);
  if (lane < 16) lds.stats[wave][lane] = float2{mine.top, mine.sum};
  lds.cols[wave][lane] = mine.v;
  __syncthreads();
  if (wave != 0) return;
  Joined o;
#pragma unroll
  for (int x = 0; x < kWaves; ++x) o.add(lds.stats[x][lane & 15], lds.cols[x][lane]);
  store_joined<NB>(a, note, o, nt, e, blk);
}

// ------------------------------------------------------------------ host

// Rows per product: 16 rows, or 32 where the sequences have more on average and registers
// hold their sums: of up to 192 columns, and beside sequences of many rows (which take
// three workgroups a compute unit for up to 64) of more than 64.  (The average is all that the
// host knows: one long chunk raises it for single tokens beside it, whose products then have
// rows that are none.)
inline int few_row_tiles(const Attention& a) {
  const int64_t rows = static_cast<int64_t>(a.batch.tokens) * a.group;
  const bool room = a.cache.dim <= 192 && (a.batch.offsets == nullptr || a.cache.dim > 64);
  return room && rows > static_cast<int64_t>(a.batch.seqs) * 16 ? 2 : 1;
}

// Whether a head's tiles are few enough for one workgroup: as many as its wavefronts take
// in two turns.  (A turn more is 1.6 us, the second launch 4: one token of 1000 positions,
// four turns, 12.3 us cut and joined, 13.6 whole.)
inline bool few_whole(const Attention& a) {
  int64_t most = a.batch.max_length;
  const int64_t within = static_cast<int64_t>(a.window) + 32 + kTile;  // of 32 rows, from any place of a tile on
  if (a.window > 0 && within < most) most = within;
  return most <= 8 * kTile;
}

// The parts of n workgroups in the workspace.
inline size_t notes_bytes(int n) { return static_cast<size_t>(n) * 16; }
inline size_t few_stats_bytes(int n, int nt) { return static_cast<size_t>(n) * 2 * 16 * nt * 8; }
inline size_t few_bytes(const Attention& a, int n) {
  const int nt = few_row_tiles(a);
  return notes_bytes(n) + few_stats_bytes(n, nt) + static_cast<size_t>(n) * 2 * nt * 16 * a.cache.dim * 4;
}
// (notes: as many as there are workgroups, also where they go by jobs: those are no more.)
inline Few make_few(const Attention& a, int n, int max_rows, void* workspace) {
  Few f;
  f.max_rows = max_rows;
  f.whole = few_whole(a);
  f.least = f.whole ? 1 : kWaves;
  if (a.batch.offsets == nullptr) {  // all sequences have the rows of one token
    const int rows = 16 * few_row_tiles(a);
    const int64_t jobs = static_cast<int64_t>(a.batch.seqs) * a.cache.kv_heads * ((a.group + rows - 1) / rows);
    f.parts.jobs = jobs <= n ? static_cast<int>(jobs) : 0;
  }
  f.parts.notes = static_cast<int*>(workspace);
  f.parts.stats = reinterpret_cast<float*>(behind(workspace, notes_bytes(n)));
  f.parts.cols = reinterpret_cast<float4_t*>(behind(workspace, notes_bytes(n) + few_stats_bytes(n, few_row_tiles(a))));
  return f;
}

}  // namespace q4
