// Softmax attention over the paged Q4_0 cache: launch rules, and the kernel that is
// right for every shape and type.
//
//   s_t = scale sum_j q_j k_tj  (capped: c tanh(s_t / c))
//   y   = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  m = max_t s_t
//
// in one pass over the positions that a row sees, with the running maximum and sum.
#include "q4_attention.hpp"

namespace q4 {
namespace {

constexpr int kMaxDim = 256;
// A workgroup per row and head; a wavefront takes every fourth tile of 64 positions:
// first a position a lane (its score), then two pairs of columns a lane.  Everything
// is fp32 on the exactly decoded values.
__global__ __launch_bounds__(kWaves* kWave) void attention_row_kernel(Attention a) {
  __shared__ float qs[kMaxDim];
  __shared__ float weights[kWaves][kWave];
  __shared__ float out[kWaves][kMaxDim];
  __shared__ float stats[kWaves][2];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int row = blockIdx.x / a.heads, head = blockIdx.x - row * a.heads;
  const Batch& b = a.batch;
  const int s = b.offsets == nullptr ? row
                                     : last_not_above(b.seqs, row, [&](int i) {
                                         return static_cast<int64_t>(offset_of(b, i));
                                       });
  const Seq q = seq_of(b, s);
  if (row < q.row || row >= q.row + q.rows) return;  // a row of no sequence
  const int d = a.cache.dim, nb = d / kQK;
  for (int e = threadIdx.x; e < d; e += kWaves * kWave)
    qs[e] = load_f32(a.q, static_cast<int>(a.qt), row * a.q_stride + head * d + e);
  __syncthreads();
  int lo, hi;
  seen_by(a, q.length, q.first + row - q.row, &lo, &hi);
  const int h = head / a.group;
  const int64_t to_values = static_cast<int64_t>(a.cache.per_page) * (9 * d);

  float m = -INFINITY, l = 0.f;
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // columns i and i + 16 of byte column lane + 64 r
  for (int t0 = (lo / kWave + wave) * kWave; t0 < hi; t0 += kWaves * kWave) {
    const int t = t0 + lane, at = t & 15;
    const uint8_t* g = t < hi ? granule_at(a.cache, b, s, t / kGranule, h) : nullptr;
    const bool seen = g != nullptr && t >= lo;
    float score = -INFINITY;
    if (seen) {
      score = 0.f;
      for (int blk = 0; blk < nb; ++blk) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(g + at * (d / 2) + (w * nb + blk) * 4);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int lo4 = static_cast<int>((c >> (8 * r)) & 15) - 8, hi4 = static_cast<int>((c >> (8 * r + 4)) & 15) - 8;
            sum = fmaf(qs[blk * 32 + w * 4 + r], static_cast<float>(lo4), sum);
            sum = fmaf(qs[blk * 32 + 16 + w * 4 + r], static_cast<float>(hi4), sum);
          }
        }
        const uint16_t bits = reinterpret_cast<const uint16_t*>(g + 8 * d)[((at >> 2) * nb + blk) * 4 + (at & 3)];
        score = fmaf(half_bits_to_float(bits), sum, score);
      }
      score *= a.scale;
      if (a.softcap > 0.f) score = capped(score, a.softcap);
    }
    float top = score;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if (top == -INFINITY) continue;  // the whole tile is masked
    const float next = fmaxf(m, top);
    const float old = m == -INFINITY ? 0.f : exp2f((m - next) * kLog2e);
    const float p = seen ? exp2f((score - next) * kLog2e) : 0.f;
    m = next;
    float total = p;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) total += __shfl_xor(total, off);
    l = fmaf(l, old, total);
    weights[wave][lane] = p;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 2; ++r) acc[r][0] *= old, acc[r][1] *= old;
    for (int gi = 0; gi < 4; ++gi) {
      if (t0 + 16 * gi >= hi) break;
      const uint8_t* vg = granule_at(a.cache, b, s, t0 / kGranule + gi, h);
      if (vg == nullptr) continue;
      vg += to_values;
      const int end = hi - t0 - 16 * gi < 16 ? hi - t0 - 16 * gi : 16;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int col = lane + kWave * r;
        if (col >= d / 2) continue;
        const uint8_t* codes = vg + col * 16;
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(vg + 8 * d) + col / 16 * 16;
        for (int e = 0; e < end; ++e) {
          const int quarter = e & 3, place = (e & ~3) + (quarter & 1) * 2 + (quarter >> 1);
          const float pe = weights[wave][16 * gi + e];
          if (pe == 0.f) continue;  // (an unseen place may hold anything)
          const float w = pe * half_bits_to_float(scales[place]);
          acc[r][0] = fmaf(w, static_cast<float>(static_cast<int>(codes[e] & 15) - 8), acc[r][0]);
          acc[r][1] = fmaf(w, static_cast<float>(static_cast<int>(codes[e] >> 4) - 8), acc[r][1]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  // The wavefronts' parts, in their order.
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int col = lane + kWave * r;
    if (col < d / 2) {
      out[wave][col / 16 * 32 + col % 16] = acc[r][0];
      out[wave][col / 16 * 32 + col % 16 + 16] = acc[r][1];
    }
  }
  if (lane == 0) {
    stats[wave][0] = m;
    stats[wave][1] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, part[kWaves];
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[w][0]);
  for (int w = 0; w < kWaves; ++w) {
    part[w] = stats[w][0] == -INFINITY ? 0.f : exp2f((stats[w][0] - top) * kLog2e);
    sum = fmaf(stats[w][1], part[w], sum);
  }
  const float inverse = sum > 0.f ? 1.f / sum : 0.f;
  const int64_t at = static_cast<int64_t>(row) * a.heads + head;
  for (int e = threadIdx.x; e < d; e += kWaves * kWave) {
    float v = 0.f;
    for (int w = 0; w < kWaves; ++w) v = fmaf(out[w][e], part[w], v);
    store_as(a.y, a.y_dt, at * d + e, v * inverse);
  }
  if (a.lse != nullptr && threadIdx.x == 0) a.lse[at] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

hipError_t launch_row(const Attention& a, Queue q) {
  Attention args = a;
  void* argv[] = {&args};
  return launch_blocks(reinterpret_cast<const void*>(&attention_row_kernel),
                       static_cast<int64_t>(a.batch.tokens) * a.heads, kWaves * kWave, argv, 0, q);
}

}  // namespace

size_t attention_workspace_bytes(const Attention& a) {
  if (a.qt == DType::F32) return 0;
  return a.batch.offsets == nullptr ? attention_few_bytes(a) : attention_mixed_bytes(a);
}

hipError_t launch_attention(const Attention& a, void* workspace, Queue q) {
  if (a.qt == DType::F32) return launch_row(a, q);
  return a.batch.offsets == nullptr ? launch_attention_few(a, workspace, q) : launch_attention_mixed(a, workspace, q);
}

}  // namespace q4
