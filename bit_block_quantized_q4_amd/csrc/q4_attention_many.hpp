// Attention over the paged Q4_0 cache for sequences of many rows: prompts and chunks
// of them.
//
//   S^T = K Q^T,  P = exp2(x - m),  O^T = V^T P^T
//
// with keys and values rounded to fp16 as they are decoded, once for all the rows of a
// workgroup.  A kv head's heads and a sequence's rows together are the rows; a
// wavefront takes 32 of them, a workgroup 128, and walks over the positions in tiles of
// 64.  Each tile is decoded into one of two LDS buffers, a granule by each wavefront,
// while the other is multiplied; the next tile's bytes are on their way in registers
// meanwhile.
//
// LDS holds 16-byte pieces, the operands of v_mfma_f32_32x32x16_f16 as they are read:
//   K  position t, piece 4 b + g: elements 4 g + {0, 2, 1, 3, 16, 18, 17, 19} of block
//      b (the order in which a code word comes apart; q is held in the same order)
//   V  column c, piece 2 k + h: positions 16 k + 4 h + {0, 2, 1, 3, 8, 10, 9, 11}, which
//      is what lane half h holds of the scores' rows: the weights are the right operand
//      of the second product where they are
// The piece number is exclusive-ored with the row's so that rows lie in other banks.
//
// Three things are rounded to fp16, each once: a decoded key, a weight and a decoded value
// (a code times its scale has up to 15 bits).  For fp16 outputs over random keys and values
// that makes 4.0e-4 of y (2-norms), where rounding y alone makes 2.1e-4; bf16 outputs hide
// it (1.7e-3 either way).  Exact codes with the scales as fp32 factors of each block's
// scores, and weights in two parts, bring it to 2.7e-4, but for 128 more vector
// instructions and half as many products again a tile: 512 rows behind 32488 positions 623
// us, not 411.  (q of 32 bits goes another way, with no rounding.)
//
// Where there are fewer workgroups than compute units hold the positions are split as
// well, and the parts joined in a second launch; less so beside sequences of few rows, which
// take places too (many_splits).
//
// Bound by issuing vector instructions (taking codes apart, exp, the maximum) beside the
// matrix products: of 730 us for a prompt of 8000 (40 heads of 128 on 8, bf16) the products
// alone take 436, the softmax alone 256; without decoding it is 627, without the softmax
// 575.  That is 890 TFLOP/s of products, 71% of a large library product's rate.  So
// what counts is that other wavefronts have products ready: two workgroups share a compute
// unit (three for heads of up to 64), each SIMD with two wavefronts that no barrier ties to
// one another.  Rows by wavefronts, for that prompt, 512 rows behind 32488 positions, and
// six ragged prompts with heads of 64 (us):
//   32 x 4, two workgroups a unit    730  411   80
//   32 x 8, opposite halves' phases  735  505  127
//   32 x 8                           774  553  121
//   16 x 8                           774  436   81
//   16 x 16, opposite phases         790  603  117
#pragma once

#include "q4_attention.hpp"

namespace q4 {

constexpr int kManyRows = 32 * kWaves;
constexpr float kLift2 = 8.f;   // weights are held times 2^8 ..
constexpr float kSlack = 7.f;   // .. of a maximum that may have grown by 2^7 since

struct Many {
  int min_rows = 0;   // sequences of fewer rows are left out
  int splits = 1;
  int64_t places = 0;
  float* stats = nullptr;   // [workgroups][rows][2]
  float4_t* cols = nullptr; // [workgroups][wavefronts][NB][4][64]
};

// Row tiles of R rows, as places of a grid: sequence s has the places from row_place(s)
// on, at least as many as it has tiles; without offsets exactly as many.
__device__ __forceinline__ int64_t row_place(const Batch& b, int group, int rows, int s) {
  return static_cast<int64_t>(offset_of(b, s)) * group / rows + s;
}

// What workgroup `at` takes: heads inside (neighbours, which lie on other dies, then
// read other keys), the last rows, which see most, first.
template <int R>
__device__ __forceinline__ bool job_of(const Attention& a, const Many& y, int64_t at, int* s, int* h,
                                       int* r0, int* rows, int* split, Seq* q) {
  const int kv = a.cache.kv_heads;
  *h = static_cast<int>(at % kv);
  at /= kv;
  *split = static_cast<int>(at % y.splits);
  const int64_t place = y.places - 1 - at / y.splits;
  const bool alike = a.batch.offsets == nullptr;  // one token each
  const int per = (a.group + R - 1) / R;
  *s = alike ? static_cast<int>(place / per) : last_not_above(a.batch.seqs, place, [&](int i) {
    return row_place(a.batch, a.group, R, i);
  });
  *q = seq_of(a.batch, *s);
  const int64_t n = static_cast<int64_t>(q->rows) * a.group;
  const int64_t first = (place - (alike ? static_cast<int64_t>(*s) * per : row_place(a.batch, a.group, R, *s))) * R;
  if (n < y.min_rows || first < 0 || first >= n) return false;
  *r0 = static_cast<int>(first);
  *rows = static_cast<int>(n);
  return true;
}

// What position t's piece numbers are exclusive-ored with.  LDS serves sixteen lanes at
// a time from 256 bytes of banks; rows are 64 NB bytes.  Read are sixteen positions'
// pieces of one number, written four positions' of four.
template <int NB>
__device__ __forceinline__ int turn_key(int t) {
  if constexpr (NB % 4 == 0) return (t & 15) ^ (t & 1) << 2;
  else if constexpr (NB % 2 == 0) return (t >> 1 & 3) | ((t ^ t >> 3) & 1) << 2;
  else return t >> 2 & 3;
}
// As that for column c's, of 128 bytes.
__device__ __forceinline__ int turn_value(int c) { return (c & 7) ^ (c >> 3 & 1); }

template <int NB>
struct Bytes {
  uint32_t k[NB];
  uint16_t ks[NB];
  u32x4 v[(NB + 3) / 4], vs[(NB + 3) / 4][2];
};

// The order of N LDS reads and as many matrix products behind it: kAhead reads go ahead
// (left alone the compiler reads two pieces, waits, and multiplies).
template <int N, int AHEAD>
__device__ __forceinline__ void feed() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

template <int NB>
struct ManyLds {
  u32x4 tiles[2][kTile * 4 * NB + NB * kQK * 8];  // keys and values, in two buffers
  int named[2][4];                                // whether a granule has a page
};

// Workgroup `block`.
template <int NB, bool BF16>
__device__ __forceinline__ void attention_many(const Attention& a, const Many& y, int64_t block, ManyLds<NB>& shared) {
  constexpr int R = kManyRows;
  constexpr int kAhead = NB > 6 ? 2 : 4;          // LDS reads before the first product
  constexpr int kPieces = 4 * NB;                 // of a position's key
  constexpr int kKeys = kTile * kPieces, kValues = NB * kQK * 8;
  u32x4* const lds = shared.tiles[0];
  int* const named = shared.named[0];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n = lane & 31, half = lane >> 5;
  int s, h, r0, rows, split;
  Seq q;
  if (!job_of<R>(a, y, block, &s, &h, &r0, &rows, &split, &q)) return;
  const Cache& c = a.cache;
  const UnpackConsts uc = make_unpack_consts();
  const Cap<true> cap(a.softcap);

  // The tiles of all the workgroup's rows, and of this part of them.
  const int end_row = r0 + R < rows ? r0 + R : rows;
  int lo_first, hi_first, lo_last, hi_last;
  seen_by(a, q.length, q.first + r0 / a.group, &lo_first, &hi_first);
  seen_by(a, q.length, q.first + (end_row - 1) / a.group, &lo_last, &hi_last);
  const int tile0 = lo_first / kTile, tiles = hi_last > lo_first ? (hi_last + kTile - 1) / kTile - tile0 : 0;
  const int t0 = tile0 + static_cast<int>(static_cast<int64_t>(tiles) * split / y.splits);
  const int t1 = tile0 + static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / y.splits);

  // This wavefront's rows, and what this lane's row sees.
  const int w0 = r0 + 32 * wave, w1 = w0 + 32 < end_row ? w0 + 32 : end_row;
  int wlo = 0, whi = 0, wlo_last = 0, whi_first = 0;
  if (w0 < w1) {
    seen_by(a, q.length, q.first + w0 / a.group, &wlo, &whi_first);
    seen_by(a, q.length, q.first + (w1 - 1) / a.group, &wlo_last, &whi);
  }
  const int row = w0 + n < end_row ? w0 + n : end_row - 1;
  const int token = row / a.group, hq = h * a.group + row - token * a.group;
  int lo, hi;
  seen_by(a, q.length, q.first + token, &lo, &hi);
  if (w0 + n >= end_row) lo = hi = 0;

  // q as the right operand: pieces 4 b + g for g = half, half + 2.
  half8_t qf[2 * NB];
  float mul = fabsf(a.scale) * (a.softcap > 0.f ? 1.f : kLog2e);
  {
    const uint16_t* x = static_cast<const uint16_t*>(a.q) + (q.row + token) * a.q_stride +
                        static_cast<int64_t>(hq) * (NB * kQK) + 4 * half;
    uint2 part[2 * NB][2];
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      part[i][0] = *reinterpret_cast<const uint2*>(x + i / 2 * kQK + 8 * (i % 2));
      part[i][1] = *reinterpret_cast<const uint2*>(x + i / 2 * kQK + 8 * (i % 2) + 16);
    }
    if constexpr (BF16) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top = max_magnitude_bf16(top, part[i][e].x);
          top = max_magnitude_bf16(top, part[i][e].y);
        }
      top = __builtin_bit_cast(uint32_t, max_over_halves(__builtin_bit_cast(float, top << 16))) >> 16;
      const int shift = bf16_row_shift(top);
      const float by = power_of_two(shift);
      mul *= power_of_two(-shift);
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          part[i][e].x = bf16x2_scaled_to_f16x2(part[i][e].x, by);
          part[i][e].y = bf16x2_scaled_to_f16x2(part[i][e].y, by);
        }
    }
    // The factor is positive, so that the largest score is the largest product's: a
    // negative scale turns q, one of 0 clears it (but what is no number).
    const float sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
    mul = fmaxf(mul, 1.17549435e-38f);
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[2 * e] = query_pair(__builtin_amdgcn_perm(part[i][e].y, part[i][e].x, 0x05040100), sign);
        v[2 * e + 1] = query_pair(__builtin_amdgcn_perm(part[i][e].y, part[i][e].x, 0x07060302), sign);
      }
      qf[i] = __builtin_bit_cast(half8_t, v);
    }
  }

  // Fetching and decoding: a wavefront has a granule of a tile, keys and values.
  const int mine = wave;
  const int* table = a.batch.tables + static_cast<int64_t>(s) * a.batch.max_pages;
  const int64_t to_values = static_cast<int64_t>(c.per_page) * (288 * NB);
  Bytes<NB> bytes;
  int fetched_named = 0;
  // Where the granule of a tile lies, for 64 tiles at a time, one a lane (its upper half
  // all ones: nowhere).
  uint32_t at_lo = 0, at_hi = 0;
  auto look_up = [&](int tile) __attribute__((always_inline)) {
    const uint32_t gi = static_cast<uint32_t>((tile + lane) * 4 + mine), per = static_cast<uint32_t>(c.per_page);
    uint32_t slot = __umulhi(gi, c.inverse), inside = gi - slot * per;
    if (inside >= per) {
      ++slot;
      inside -= per;
    }
    int id = -1;
    if (tile + lane < t1 && slot < static_cast<uint32_t>(a.batch.max_pages)) id = table[slot];
    const uint64_t at = static_cast<uint64_t>(id) * c.page_bytes + static_cast<uint64_t>(inside) * (288 * NB);
    const bool some = static_cast<uint32_t>(id) < static_cast<uint32_t>(c.pages);
    at_lo = static_cast<uint32_t>(at);
    at_hi = some ? static_cast<uint32_t>(at >> 32) : ~0u;
  };
  const uint8_t* const head = c.data + h * c.head_bytes;
  auto fetch = [&](int tile) __attribute__((always_inline)) {
    const int i = (tile - t0) & 63;
    if (i == 0) look_up(tile);
    const uint32_t high = __builtin_amdgcn_readlane(at_hi, i), low = __builtin_amdgcn_readlane(at_lo, i);
    fetched_named = high != ~0u;
    const uint8_t* p = head + (fetched_named ? static_cast<uint64_t>(high) << 32 | low : 0);
    {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(p) + lane * NB;
#pragma unroll
      for (int b = 0; b < NB; ++b) bytes.k[b] = w[b];
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(p + 256 * NB) + (lane >> 4) * (4 * NB) + ((lane >> 2) & 3);
#pragma unroll
      for (int b = 0; b < NB; ++b) bytes.ks[b] = sc[4 * b];
    }
    {
      p += to_values;
#pragma unroll
      for (int i = 0; i < (NB + 3) / 4; ++i) {
        // Block at / 16, byte at % 16.  Lanes beyond the last one load it again: without a
        // branch here.  (At one in the kernel of 192 columns, which is short of registers,
        // the compiler moved values that all lanes need while some did not take part.)
        const int at = 64 * i + lane < 16 * NB ? 64 * i + lane : 16 * NB - 1;
        bytes.v[i] = *reinterpret_cast<const u32x4*>(p + at * 16);
        bytes.vs[i][0] = *reinterpret_cast<const u32x4*>(p + 256 * NB + at / 16 * 32);
        bytes.vs[i][1] = *reinterpret_cast<const u32x4*>(p + 256 * NB + at / 16 * 32 + 16);
      }
    }
  };
  auto decode = [&](int tile, int buffer) __attribute__((always_inline)) {
    u32x4* const keys = lds + buffer * (kKeys + kValues);
    u32x4* const values = keys + kKeys;
    {
      const int t = 16 * mine + (lane >> 2), g = lane & 3;
      int turn = turn_key<NB>(t);
      if constexpr (NB > 6) tie_after(turn);  // (addresses formed anew: there are too many to keep)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const Codes k = codes_of(bytes.k[b], uc);
        const half_t d = __builtin_bit_cast(half_t, bytes.ks[b]);
        const half2_t dd = {d, d};
        const half8_t piece = join(k.l02 * dd, k.l13 * dd, k.h02 * dd, k.h13 * dd);
        keys[t * kPieces + ((4 * b + g) ^ turn)] = __builtin_bit_cast(u32x4, piece);
      }
      if (lane == 0) named[buffer * 4 + mine] = fetched_named;
    }
    {
      const int first = tile * kTile + 16 * mine;
      const int from = lo_first - first, to = fetched_named ? hi_last - first : 0;
      const bool whole = from <= 0 && to >= 16;  // unseen places may hold anything
#pragma unroll
      for (int i = 0; i < (NB + 3) / 4; ++i) {
        const int at = 64 * i + lane;
        if (64 * i + 64 > 16 * NB && at >= 16 * NB) break;
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int p = e / 2 * 4 + e % 2;
            const uint32_t keep = (p >= from && p < to ? 0xFFFFu : 0u) |
                                  (p + 2 >= from && p + 2 < to ? 0xFFFF0000u : 0u);
            bytes.vs[i][e >> 2][e & 3] &= keep;
          }
        }
        const int col = at / 16 * 32 + at % 16;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const Codes v0 = codes_of(bytes.v[i][hf], uc), v1 = codes_of(bytes.v[i][hf + 2], uc);
          const half2_t d0 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(bytes.vs[i][0][2 * hf]));
          const half2_t d1 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(bytes.vs[i][0][2 * hf + 1]));
          const half2_t d2 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(bytes.vs[i][1][2 * hf]));
          const half2_t d3 = __builtin_bit_cast(half2_t, static_cast<uint32_t>(bytes.vs[i][1][2 * hf + 1]));
          const half8_t low = join(v0.l02 * d0, v0.l13 * d1, v1.l02 * d2, v1.l13 * d3);
          const half8_t high = join(v0.h02 * d0, v0.h13 * d1, v1.h02 * d2, v1.h13 * d3);
          values[col * 8 + ((2 * mine + hf) ^ turn_value(col))] = __builtin_bit_cast(u32x4, low);
          values[(col + 16) * 8 + ((2 * mine + hf) ^ turn_value(col))] = __builtin_bit_cast(u32x4, high);
        }
      }
    }
  };

  float m = -INFINITY, l = 0.f;  // m: what weights are taken against, at most kSlack below the maximum
  float16_t o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[b][i] = 0.f;

  half8_t p[4];
  float16_t x[2];
  int4 there = {0, 0, 0, 0};  // whether the tile's granules have pages
  // The tiles that the wavefront's rows see some of, and those that each sees whole.
  const int some0 = w0 < w1 ? wlo / kTile : t1, some1 = w0 < w1 ? (whi + kTile - 1) / kTile : 0;
  const int whole0 = (wlo_last + kTile - 1) / kTile, whole1 = w1 == w0 + 32 ? whi_first / kTile : 0;
  auto scores = [&](int buffer) __attribute__((always_inline)) {
    const u32x4* const keys = lds + buffer * (kKeys + kValues);
    int turn = turn_key<NB>(n);
    if constexpr (NB > 6) tie_after(turn);  // (addresses formed anew: there are too many to keep)
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[mt][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const half8_t kf = __builtin_bit_cast(
            half8_t, keys[(32 * mt + n) * kPieces + ((2 * ks + half) ^ turn)]);
        x[mt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[ks], x[mt], 0, 0, 0);
      }
  };
  auto products = [&](int buffer) __attribute__((always_inline)) {
    const u32x4* const values = lds + buffer * (kKeys + kValues) + kKeys;
    int turn = turn_value(n);
    if constexpr (NB > 6) tie_after(turn);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const half8_t vf = __builtin_bit_cast(half8_t, values[(32 * b + n) * 8 + ((2 * k + half) ^ turn)]);
        o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[k], o[b], 0, 0, 0);
      }
  };
  auto weights = [&](int t) __attribute__((always_inline)) {
    const bool all = __builtin_amdgcn_readfirstlane(there.x & there.y & there.z & there.w) != 0;
    float by = mul;
    // (As an unlikely way: with its code in line a prompt of 4000, 32 heads of 256 on 8, takes
    // 493 us, so 478; of 192 407 and 401.)
    if (__builtin_expect(a.softcap > 0.f, 0)) {
      by = 1.f;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[mt][i] *= mul;
          most = fmaxf(most, fabsf(x[mt][i]));
        }
        if (__all(cap.near(most))) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[mt][i] = cap.of_near(x[mt][i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[mt][i] = cap.of(x[mt][i]);
        }
      }
    }
    if (!(t >= whole0 && t < whole1 && all)) {
      const int first = t * kTile;
      const int from = lo - first - 4 * half, to = hi - first - 4 * half;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = 32 * mt + 8 * (i / 4) + i % 4;
          const int page = e / 16 == 0 ? there.x : e / 16 == 1 ? there.y : e / 16 == 2 ? there.z : there.w;
          x[mt][i] = page && e >= from && e < to ? x[mt][i] : -INFINITY;
        }
    }
    float top = fmaxf(x[0][0], x[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(x[0][i], x[1][i]), top);
    top = max_over_halves(top) * by;
    if (__any(top > m + kSlack)) {
      const float next = fmaxf(m, top);
      const float old = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= old;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= old;
    }
    const float from = kLift2 - (m == -INFINITY ? 0.f : m);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[mt][i] = __builtin_amdgcn_exp2f(fmaf(x[mt][i], by, from));
        l += x[mt][i];
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        constexpr int kOrder[8] = {0, 2, 1, 3, 4, 6, 5, 7};
        half_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = static_cast<half_t>(x[mt][8 * ks + kOrder[e]]);
        p[2 * mt + ks] = half8_t{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
      }
    }
  };
  // A barrier that waits for this wavefront's LDS accesses alone: fetches stay in flight.
  auto meet = [&]() __attribute__((always_inline)) {
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    compiler_fence();
  };

  // A tile: its scores, the decoding of the next tile into the other buffers (which the
  // barrier behind the tile before has freed), its weights, its products.  The two
  // workgroups of a compute unit are in different places of this, so that matrix and
  // vector units work at the same time.
  if (t0 < t1) {
    fetch(t0);
    decode(t0, 0);
    if (t0 + 1 < t1) fetch(t0 + 1);
    meet();
    auto step = [&](int t, int buffer) __attribute__((always_inline)) {
      const bool seen = t >= some0 && t < some1;
      there = *reinterpret_cast<const int4*>(named + 4 * buffer);
      if (seen) {
        scores(buffer);
        feed<4 * NB, kAhead>();
      }
      if (t + 1 < t1) {
        decode(t + 1, buffer ^ 1);
        if (t + 2 < t1) fetch(t + 2);
      }
      if (seen) {
        weights(t);
        products(buffer);
        feed<4 * NB, kAhead>();
      }
      meet();
    };
    if constexpr (NB > 6) {
      for (int t = t0; t < t1; ++t) step(t, (t - t0) & 1);
    } else {  // (each buffer's addresses are then constants away from the other's)
      for (int t = t0; t < t1; t += 2) {
        step(t, 0);
        if (t + 1 < t1) step(t + 1, 1);
      }
    }
  }

  l = sum_over_halves(l);
  if (y.splits > 1) {
    const int64_t at = block * kWaves + wave;
    if (half == 0) *reinterpret_cast<float2*>(y.stats + (at * 32 + n) * 2) = float2{m, l};
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y.cols[((at * NB + b) * 4 + i) * kWave + lane] =
            float4_t{o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]};
    return;
  }
  if (w0 + n >= end_row) return;
  const int64_t at = static_cast<int64_t>(q.row + token) * a.heads + hq;
  const float inverse = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float out[4] = {o[b][4 * i] * inverse, o[b][4 * i + 1] * inverse, o[b][4 * i + 2] * inverse,
                            o[b][4 * i + 3] * inverse};
      store4(a.y, a.y_dt, at * (NB * kQK) + b * kQK + 8 * i + 4 * half, out);
    }
  if (a.lse != nullptr && half == 0) a.lse[at] = l != 0.f ? (m - kLift2 + log2f(l)) * kLn2 : -INFINITY;
}

// The splits' parts of a row tile, in their order; a wavefront takes 32 rows (of
// the first launch's wavefront `wave`) of a block's columns.
template <int NB>
__device__ __forceinline__ void attention_splits(const Attention& a, const Many& y, int64_t block, int wave) {
  constexpr int R = kManyRows;
  const int lane = threadIdx.x & (kWave - 1), n = lane & 31, half = lane >> 5;
  const int kv = a.cache.kv_heads;
  const int64_t place = block / kv;  // as the first launch counts them, without its splits
  const int64_t block0 = place * y.splits * kv + block % kv;
  int s, h, r0, rows, split;
  Seq q;
  if (!job_of<R>(a, y, block0, &s, &h, &r0, &rows, &split, &q)) return;
  const int row = r0 + 32 * wave + n;
  for (int b = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); b < NB; b += kWaves) {
    float m = -INFINITY, l = 0.f;
    float4_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < y.splits; ++i) {
      const int64_t at = (block0 + static_cast<int64_t>(i) * kv) * kWaves + wave;
      const float2 st = *reinterpret_cast<const float2*>(y.stats + (at * 32 + n) * 2);
      const float next = fmaxf(m, st.x), ref = next == -INFINITY ? 0.f : next;
      const float old = __builtin_amdgcn_exp2f(m - ref), by = __builtin_amdgcn_exp2f(st.x - ref);
      m = next;
      l = l * old + st.y * by;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = v[j] * old + y.cols[((at * NB + b) * 4 + j) * kWave + lane] * by;
    }
    if (row >= rows) continue;
    const int token = row / a.group;
    const int64_t at = static_cast<int64_t>(q.row + token) * a.heads + h * a.group + row - token * a.group;
    const float inverse = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float out[4] = {v[j][0] * inverse, v[j][1] * inverse, v[j][2] * inverse, v[j][3] * inverse};
      store4(a.y, a.y_dt, at * (NB * kQK) + b * kQK + 8 * j + 4 * half, out);
    }
    if (a.lse != nullptr && half == 0 && b == 0) a.lse[at] = l != 0.f ? (m - kLift2 + log2f(l)) * kLn2 : -INFINITY;
  }
}

// ------------------------------------------------------------------ host

inline int64_t many_places(const Attention& a) {
  return static_cast<int64_t>(a.batch.tokens) * a.group / kManyRows + a.batch.seqs;
}

// Workgroups that a compute unit holds, by their registers.
inline int many_per_unit(int dim) { return dim > 128 ? 1 : dim > 64 ? 2 : 3; }

// Parts of the positions where there are fewer row tiles than workgroups at once: the
// number that lets the fewest turns of all workgroups do, the smallest such.  Places of
// sequences without a tile start workgroups too, of which a quarter more than at once is
// enough.  (256 rows of each of two sequences behind 16128 positions, heads of 256: whole
// 955 us, in two parts 509; heads of 128 215 and 174.)
//
// At most 32.  What that costs either way, with one kv head (16, 32, 64 parts): 40 rows
// behind 131072 positions 202, 120, 95 us, behind 8000 29, 30, 40; a prompt of 280 rows and
// one head of 256, most of whose parts have no positions, 31, 43, 72.
//
// A place for every sequence leaves few parts to a chunk beside many of them: 512 rows
// behind 32488 positions are cut in three alone, 417 us, and not at all beside the next tokens
// of 64 sequences (106 us alone): 1021 us together.
inline int many_splits(const Attention& a) {
  const int64_t room = device_cu_count() * static_cast<int64_t>(many_per_unit(a.cache.dim));
  const int64_t rows = static_cast<int64_t>(a.batch.tokens) * a.group;
  const int64_t n = (rows + kManyRows - 1) / kManyRows * a.cache.kv_heads;
  if (n >= room) return 1;
  const int64_t most = 5 * room / (4 * many_places(a) * a.cache.kv_heads);
  int best = 1;
  int64_t turns = 1;  // of best, each the best-th part of the positions
  for (int s = 2; s <= most && s <= 32; ++s) {
    const int64_t mine = (n * s + room - 1) / room;
    if (mine * best < turns * s) {
      best = s;
      turns = mine;
    }
  }
  return best;
}

inline size_t many_stats_bytes(const Attention& a, int splits) {
  return static_cast<size_t>(many_places(a)) * a.cache.kv_heads * splits * kManyRows * 8;
}
inline size_t many_bytes(const Attention& a) {
  const int splits = many_splits(a);
  if (splits == 1) return 0;
  return many_stats_bytes(a, splits) +
         static_cast<size_t>(many_places(a)) * a.cache.kv_heads * splits * kManyRows * a.cache.dim * 4;
}
inline Many make_many(const Attention& a, int min_rows, void* workspace) {
  Many y;
  y.min_rows = min_rows;
  y.splits = many_splits(a);
  y.places = many_places(a);
  y.stats = static_cast<float*>(workspace);
  y.cols = reinterpret_cast<float4_t*>(behind(workspace, many_stats_bytes(a, y.splits)));
  return y;
}

}  // namespace q4
