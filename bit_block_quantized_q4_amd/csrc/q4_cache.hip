// Writing and reading the paged Q4_0 cache of keys and values.
//
// A workgroup takes one granule (sixteen positions) of one sequence and kv head,
// keys and values, of some kv heads in turn.  Grids are sized from the numbers of rows and
// sequences alone (granule_places); what a place holds is found on the device.
//
// Both only move bytes: reading 401 MB of cache to 1.4 GB of fp16 takes 426 us, 4.3 TB/s
// (a large copy: 4.65).  Writing 44 MB from 156 MB of bf16 takes 54 us, 3.7 TB/s: the 16
// codes of a lane are some 300 vector instructions, which at four wavefronts to a SIMD take
// as long as its bytes do.  Reading that back at once takes 36 us.  (312 MB of fp32 take 94
// us to write, 3.8 TB/s, and 95 to read back.)
#include <type_traits>

#include "q4_cache.hpp"
#include "q4_quantize_block.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;

using u16x2 = uint16_t __attribute__((ext_vector_type(2)));

// What a workgroup of the granule grid takes: positions [from, to) of granule g of
// sequence s, the rows from `row` on.  False: nothing.
struct Granule {
  int s, g, from, to, row;
  int none, none_row;  // at a sequence's first place: its rows without a position
};
__device__ __forceinline__ bool granule_of(const Batch& b, int64_t place, Granule* out) {
  const int s = b.offsets == nullptr
                    ? static_cast<int>(place)
                    : last_not_above(b.seqs, place, [&](int i) { return granule_place(b, i); });
  const Seq q = seq_of(b, s);
  const int first = q.first < 0 ? 0 : q.first;  // the first position with a row
  const int64_t nth = b.offsets == nullptr ? 0 : place - granule_place(b, s);
  const int64_t g = first / kGranule + nth;
  out->none = q.first < 0 && nth == 0 ? (-q.first < q.rows ? -q.first : q.rows) : 0;
  out->none_row = q.row;
  if (q.rows == 0 || g * kGranule >= q.length) return false;
  out->s = s;
  out->g = static_cast<int>(g);
  const int base = out->g * kGranule;
  out->from = first > base ? first - base : 0;
  out->to = q.length - base < kGranule ? q.length - base : kGranule;
  out->row = q.row + base + out->from - q.first;
  return out->from < out->to;
}

// ------------------------------------------------------------------ writing

// Finite, of at most fp16's largest magnitude: NaN counts as 0.
__device__ __forceinline__ float storable(float v) {
  return v != v ? 0.f : fminf(fmaxf(v, -65504.f), 65504.f);
}

// Sixteen consecutive elements of a row as they lie there.
template <typename T>
struct Raw {
  u32x4 w[sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  // As fp32 (exact), limited to what is stored.  Magnitudes compare as their bits do:
  // rarely is one above the limit (NaN, infinities), and only then is each looked at.
  __device__ __forceinline__ void values(float (&v)[16]) const {
    constexpr bool kWide = sizeof(T) == 4, kHalf = std::is_same<T, half_t>::value;
    uint32_t top = 0;
    if constexpr (kWide) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t m = w[i / 4][i % 4] & 0x7FFFFFFFu;
        top = m > top ? m : top;
      }
    } else {
      u16x2 most = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u16x2 m = __builtin_bit_cast(u16x2, w[i / 4][i % 4] & 0x7FFF7FFFu);
        most = __builtin_elementwise_max(most, m);
      }
      top = most.x > most.y ? most.x : most.y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (kWide) {
        v[i] = __builtin_bit_cast(float, static_cast<uint32_t>(w[i / 4][i % 4]));
      } else {
        const uint32_t two = w[i / 8][i / 2 % 4];
        if constexpr (kHalf) v[i] = half_bits_to_float(static_cast<uint16_t>(i % 2 ? two >> 16 : two));
        else v[i] = __builtin_bit_cast(float, i % 2 ? two & 0xFFFF0000u : two << 16);
      }
    }
    constexpr uint32_t kLimit = kWide ? 0x477FE000u : kHalf ? 0x7BFFu : 0x477Fu;  // (65504; bf16 65280)
    if (top > kLimit) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = storable(v[i]);
    }
  }
};

// The Q4_0 rule on two lanes, 0 and 1 of a pair holding elements 0 .. 15 and 16 .. 31.
// Returns the scale; words[0 .. 1] are this lane's code bytes, 0 .. 7 or 8 .. 15.
//   m: the larger of max and -min; where they are equal the one that comes first.
//   code: trunc(x / d + 8.5).  u = fma(x, 1 / d, 8.5) differs from the rule's t, two
//   roundings, by less than 2^-17 (|x / d| < 16, and a subnormal d is needed for more than
//   8.01; the reciprocal is good to 2^-22).  Below, 2^-16 is added to u.
//   EXACT (x of 16 bits): t is an integer or more than 2^-13 from one.  For x / d to be
//   near k + 1/2, |x| is about d / 2 or more; x and d (k + 1/2) are multiples of 2^-12 d or
//   of larger powers of two, as both have at most 11 bits (15 with the factor 2 k + 1,
//   whose unit is d's, halved).  So u truncates as t does: an integer t to itself.
//   (Such t are common: with bf16, 2 elements of 1000.)
//   Otherwise a t within 2^-16 of an integer can truncate differently; those are the ones
//   where the fraction is below 2^-15 (u's own rounding, 2^-20, fits between).  Their blocks
//   redo the rule's own division, and any other truncates alike with what was added.
template <bool EXACT>
__device__ __forceinline__ half_t quantize_pair(int upper, const float (&v)[16], uint32_t (&words)[2]) {
  float most = v[0], least = v[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    most = fmaxf(most, v[i]);
    least = fminf(least, v[i]);
  }
  most = fmaxf(most, dpp_f<kDppXor1>(most));
  least = fminf(least, dpp_f<kDppXor1>(least));
  float m = most > -least ? most : least;
  if (most == -least) {  // both signs, or zeros
    int at = 99;
    float found = 0.f;
#pragma unroll
    for (int i = 15; i >= 0; --i)
      if (fabsf(v[i]) == most) {
        at = i + 16 * upper;
        found = v[i];
      }
    const int other = dpp_i<kDppXor1>(at);
    const float theirs = dpp_f<kDppXor1>(found);
    m = at < other ? found : theirs;
  }
  float t = m / -8.0f;  // (exact; kept from fusing with the rounding, as in quantize_lanes)
  asm volatile("" : "+v"(t));
  const half_t dh = static_cast<half_t>(t);
  const float D = static_cast<float>(dh);
  uint32_t code[4] = {0x08080808u, 0x08080808u, 0x08080808u, 0x08080808u};
  if (D != 0.f) {
    const float r = __builtin_amdgcn_rcpf(D);
    float near = 1.f;
    uint32_t q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float u = fmaf(v[i], r, 8.5f + 0x1p-16f);
      if constexpr (!EXACT) near = fminf(near, __builtin_amdgcn_fractf(u));
      const int c = static_cast<int>(u);
      q[i] = static_cast<uint32_t>(c < 0 ? 0 : c > 15 ? 15 : c);
    }
    if (!EXACT && near < 0x1p-15f) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float e = v[i] / D;
        asm volatile("" : "+v"(e));
        const int c = static_cast<int>(e + 8.5f);
        q[i] = static_cast<uint32_t>(c < 0 ? 0 : c > 15 ? 15 : c);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) code[i] = q[4 * i] | q[4 * i + 1] << 8 | q[4 * i + 2] << 16 | q[4 * i + 3] << 24;
  }
  // The lower lane keeps words 0 and 1 of the block and gets their high nibbles, the
  // upper lane words 2 and 3 and their low ones.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t mine = upper ? code[2 + i] : code[i], give = upper ? code[i] : code[2 + i];
    const uint32_t theirs = static_cast<uint32_t>(dpp_i<kDppXor1>(static_cast<int>(give)));
    words[i] = upper ? theirs | mine << 4 : mine | theirs << 4;
  }
  return dh;
}

// Pieces of 16 bytes in a granule's image: eight, then one left free, so that the values'
// bytes of a position, sixteen apart, lie in other banks for each block and half.
__device__ __forceinline__ int piece_at(int i) { return 16 * (i + (i >> 3)); }
__device__ __forceinline__ int byte_at(int i) { return i + 16 * (i >> 7); }
constexpr int kImage = 16 * (144 + 144 / 8);

// Two lanes to a block of 32 values.  Code bytes and scales are put together as the
// granule's image in LDS; a whole granule then leaves in 16-byte pieces, a part of one
// as what belongs to its positions: words of a key, single bytes of values.  A workgroup
// takes `per` kv heads in turn, the next one's rows on their way while this one's are
// worked on, images by turns.
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void cache_write_kernel(Cache c, Batch b, const T* __restrict__ k,
                                                              int64_t k_stride, const T* __restrict__ v,
                                                              int64_t v_stride, int per, int chunks) {
  __shared__ __attribute__((aligned(16))) uint8_t images[2][2][kImage];
  const int64_t place = blockIdx.x / chunks;
  const int h0 = static_cast<int>(blockIdx.x - place * chunks) * per;
  const int heads = c.kv_heads - h0 < per ? c.kv_heads - h0 : per;
  Granule gr;
  if (!granule_of(b, place, &gr)) return;
  uint8_t* keys = granule_at(c, b, gr.s, gr.g, h0);
  if (keys == nullptr) return;
  const int64_t to_values = static_cast<int64_t>(c.per_page) * (9 * c.dim);
  const int nb = c.dim / kQK, upper = threadIdx.x & 1;
  const int n = gr.to - gr.from, tasks = 2 * n * nb;
  const auto row_of = [&](int t, int h) __attribute__((always_inline)) {
    const bool value = t >= n * nb;
    const int u = value ? t - n * nb : t, i = u / nb, blk = u - i * nb;
    const int64_t row = gr.row + i;
    return (value ? v + row * v_stride : k + row * k_stride) + h * c.dim + blk * kQK + 16 * upper;
  };
  const int mine = threadIdx.x >> 1;
  const T* const first = mine < tasks ? row_of(mine, h0) : k;
  Raw<T> raw = {};
  if (mine < tasks) raw.load(first);
  for (int h = 0; h < heads; ++h, keys += c.head_bytes) {
    uint8_t(&image)[2][kImage] = images[h & 1];
    for (int t = mine; t < tasks; t += THREADS / 2) {
      if (t != mine) raw.load(row_of(t, h0 + h));
      float x[16];
      raw.values(x);
      if (t + THREADS / 2 >= tasks && h + 1 < heads) raw.load(first + (h + 1) * c.dim);
      const bool value = t >= n * nb;
      const int u = value ? t - n * nb : t, i = u / nb, blk = u - i * nb, at = gr.from + i;
      uint32_t words[2];
      const uint16_t bits = __builtin_bit_cast(uint16_t, quantize_pair<sizeof(T) == 2>(upper, x, words));
      uint8_t* const g = image[value];
      int scale;  // its byte
      if (value) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          g[piece_at(blk * 16 + 8 * upper) + 16 * e + at] = static_cast<uint8_t>(words[e >> 2] >> (8 * (e & 3)));
        const int quarter = at & 3;
        scale = 8 * c.dim + 2 * (blk * 16 + (at & ~3) + (quarter & 1) * 2 + (quarter >> 1));
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint32_t*>(g + byte_at(at * (c.dim / 2) + ((2 * upper + e) * nb + blk) * 4)) = words[e];
        scale = 8 * c.dim + 2 * (((at >> 2) * nb + blk) * 4 + (at & 3));
      }
      if (upper == 0) *reinterpret_cast<uint16_t*>(g + byte_at(scale)) = bits;
    }
    __syncthreads();  // (an image is written again only after the next one's barrier)
    if (n == kGranule) {
      const int pieces = 9 * c.dim / 16;
      for (int i = threadIdx.x; i < 2 * pieces; i += THREADS) {
        const int w = i >= pieces, j = i - w * pieces;
        *reinterpret_cast<u32x4*>(keys + w * to_values + 16 * j) =
            *reinterpret_cast<const u32x4*>(image[w] + piece_at(j));
      }
      continue;
    }
    const int words = n * nb * 4;  // a key's code words lie together
    for (int i = threadIdx.x; i < words; i += THREADS) {
      const int at = gr.from * nb * 4 + i;
      reinterpret_cast<uint32_t*>(keys)[at] = *reinterpret_cast<const uint32_t*>(image[0] + byte_at(4 * at));
    }
    for (int i = threadIdx.x; i < n * nb * 16; i += THREADS) {
      const int byte = i / n, at = byte * 16 + gr.from + i - byte * n;
      keys[to_values + at] = image[1][byte_at(at)];
    }
    for (int i = threadIdx.x; i < 2 * n * nb; i += THREADS) {
      const int w = i >= n * nb, u = i - w * n * nb, t = gr.from + u / nb, blk = u % nb, quarter = t & 3;
      const int at = 8 * c.dim + 2 * (w ? blk * 16 + (t & ~3) + (quarter & 1) * 2 + (quarter >> 1)
                                        : ((t >> 2) * nb + blk) * 4 + quarter);
      *reinterpret_cast<uint16_t*>(keys + w * to_values + at) = *reinterpret_cast<const uint16_t*>(image[w] + byte_at(at));
    }
  }
}

// ------------------------------------------------------------------ reading

// Eight values (q - 8) d, rounded to T, from two dwords whose bytes' low or (high)
// nibbles are the codes; stored as 16-byte pieces.
template <typename T>
__device__ __forceinline__ void give8(T* p, uint32_t w0, uint32_t w1, bool high, float d) {
  const int by = high ? 4 : 0;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? w0 : w1;
    v[i] = static_cast<float>(static_cast<int>((w >> (8 * (i & 3) + by)) & 15u) - 8) * d;
  }
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4_t*>(p)[0] = float4_t{v[0], v[1], v[2], v[3]};
    reinterpret_cast<float4_t*>(p)[1] = float4_t{v[4], v[5], v[6], v[7]};
  } else {
    constexpr int dt = static_cast<int>(std::is_same<T, half_t>::value ? DType::F16 : DType::BF16);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32_to_16(v[2 * i], dt) | static_cast<uint32_t>(f32_to_16(v[2 * i + 1], dt)) << 16;
    *reinterpret_cast<u32x4*>(p) = o;
  }
}

// 4 x 4 bytes turned: byte j of out[i] is byte i of in[j].
__device__ __forceinline__ void turn4(const uint32_t (&in)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400), b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602);
  const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400), d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// A thread takes eight values of a key, or of four positions' values (whose bytes lie
// sixteen apart: eight words of four positions each, turned in registers), for
// `per` kv heads in turn.
template <typename T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(Cache c, Batch b, T* __restrict__ k, T* __restrict__ v,
                                                              int per, int chunks) {
  const int64_t place = blockIdx.x / chunks;
  const int h0 = static_cast<int>(blockIdx.x - place * chunks) * per;
  const int heads = c.kv_heads - h0 < per ? c.kv_heads - h0 : per;
  const int64_t row_elems = static_cast<int64_t>(c.kv_heads) * c.dim;
  Granule gr;
  const bool some = granule_of(b, place, &gr);
  if (gr.none > 0) {  // the sequence's rows without a position, by its first place
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(gr.none) * heads * c.dim; i += kThreads) {
      const int64_t row = i / (heads * c.dim);
      const int64_t at = (gr.none_row + row) * row_elems + h0 * c.dim + (i - row * heads * c.dim);
      k[at] = v[at] = T{};
    }
  }
  if (!some) return;
  const uint8_t* const keys = granule_at(c, b, gr.s, gr.g, h0);
  const int64_t to_values = static_cast<int64_t>(c.per_page) * (9 * c.dim);
  const int nb = c.dim / kQK, n = gr.to - gr.from;
  const int key_tasks = n * nb * 4, value_tasks = nb * 16;  // of a head
  for (int t = threadIdx.x; t < heads * (key_tasks + value_tasks); t += kThreads) {
    if (t < heads * key_tasks) {  // (position, head, block, eight values): as they lie in k
      const int i = t / (heads * nb * 4), e = t - i * (heads * nb * 4), h = e / (nb * 4);
      const int blk = e / 4 - h * nb, part = e & 3, at = gr.from + i;
      T* const p = k + (gr.row + i) * row_elems + h0 * c.dim + e * 8;
      uint32_t w[2] = {0, 0};
      float d = 0.f;
      if (keys != nullptr) {
        const uint8_t* g = keys + h * c.head_bytes;
        const int word = 2 * (part & 1);
        w[0] = *reinterpret_cast<const uint32_t*>(g + at * (c.dim / 2) + (word * nb + blk) * 4);
        w[1] = *reinterpret_cast<const uint32_t*>(g + at * (c.dim / 2) + ((word + 1) * nb + blk) * 4);
        d = half_bits_to_float(reinterpret_cast<const uint16_t*>(g + 8 * c.dim)[((at >> 2) * nb + blk) * 4 + (at & 3)]);
      }
      give8<T>(p, w[0], w[1], part >= 2, d);
    } else {  // (head, block, half of its bytes, nibble, four positions)
      const int r = t - heads * key_tasks, h = r / value_tasks, e = r - h * value_tasks;
      const int u = e & 3, part = (e >> 2) & 3, blk = e >> 4;
      if (4 * u + 4 <= gr.from || 4 * u >= gr.to) continue;
      uint32_t in[2][4] = {}, out[2][4];
      uint2 sc = {0, 0};
      if (keys != nullptr) {
        const uint8_t* g = keys + h * c.head_bytes + to_values;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          in[i / 4][i % 4] = *reinterpret_cast<const uint32_t*>(g + (blk * 16 + 8 * (part & 1) + i) * 16 + 4 * u);
        sc = *reinterpret_cast<const uint2*>(g + 8 * c.dim + blk * 32 + u * 8);  // positions 0, 2, 1, 3
      }
      turn4(in[0], out[0]);
      turn4(in[1], out[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 4 * u + i;
        if (at < gr.from || at >= gr.to) continue;
        const uint32_t two = i & 1 ? sc.y : sc.x;
        const float d = half_bits_to_float(static_cast<uint16_t>(i & 2 ? two >> 16 : two));
        give8<T>(v + (gr.row + at - gr.from) * row_elems + (h0 + h) * c.dim + blk * kQK + part * 8, out[0][i],
                 out[1][i], part >= 2, d);
      }
    }
  }
}

// Kv heads that a workgroup takes in turn, so that the search for its place is made once:
// up to eight, of sixteen workgroups a compute unit or more.  (One, two, four, eight:
// reading 401 MB of cache to fp16 565, 502, 437, 426 us; 44 MB of it to bf16 46, 39, 36
// and 41 us, as so few workgroups do not come out even; writing those 68, 55, 53, 53.)
int heads_in_turn(const Cache& c, int64_t places) {
  const int64_t plenty = places * c.kv_heads / (16 * static_cast<int64_t>(device_cu_count()));
  const int per = plenty < 1 ? 1 : plenty < 8 ? static_cast<int>(plenty) : 8;
  return per < c.kv_heads ? per : c.kv_heads;
}

template <typename T>
hipError_t write_as(const Cache& c, const Batch& b, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, Queue q) {
  Cache ca = c;
  Batch ba = b;
  const T *kp = static_cast<const T*>(k), *vp = static_cast<const T*>(v);
  const int64_t places = granule_places(b);
  // One position each: a wavefront has lanes for a head's, and a head is soon done.
  const bool one = b.offsets == nullptr;
  int per = one ? 1 : heads_in_turn(c, places), chunks = (c.kv_heads + per - 1) / per;
  void* argv[] = {&ca, &ba, &kp, &k_stride, &vp, &v_stride, &per, &chunks};
  if (one) return launch_blocks(reinterpret_cast<const void*>(&cache_write_kernel<T, kWave>), places * chunks, kWave, argv, 0, q);
  return launch_blocks(reinterpret_cast<const void*>(&cache_write_kernel<T, kThreads>), places * chunks, kThreads, argv, 0, q);
}

template <typename T>
hipError_t read_as(const Cache& c, const Batch& b, void* k, void* v, Queue q) {
  Cache ca = c;
  Batch ba = b;
  T *kp = static_cast<T*>(k), *vp = static_cast<T*>(v);
  const int64_t places = granule_places(b);
  int per = heads_in_turn(c, places);
  int chunks = (c.kv_heads + per - 1) / per;
  void* argv[] = {&ca, &ba, &kp, &vp, &per, &chunks};
  return launch_blocks(reinterpret_cast<const void*>(&cache_read_kernel<T>), places * chunks, kThreads, argv, 0, q);
}

}  // namespace

hipError_t launch_cache_write(const Cache& c, const Batch& b, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, DType dt, Queue q) {
  if (dt == DType::F32) return write_as<float>(c, b, k, k_stride, v, v_stride, q);
  if (dt == DType::F16) return write_as<half_t>(c, b, k, k_stride, v, v_stride, q);
  return write_as<bf16_t>(c, b, k, k_stride, v, v_stride, q);
}

hipError_t launch_cache_read(const Cache& c, const Batch& b, void* k, void* v, DType dt, Queue q) {
  if (dt == DType::F32) return read_as<float>(c, b, k, v, q);
  if (dt == DType::F16) return read_as<half_t>(c, b, k, v, q);
  return read_as<bf16_t>(c, b, k, v, q);
}

}  // namespace q4
