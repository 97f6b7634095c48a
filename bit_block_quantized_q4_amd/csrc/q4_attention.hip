// Softmax attention over the paged Q4_0 cache: launch rules, and the kernel for q of 32
// bits.
//
//   s_t = scale sum_j q_j k_tj  (capped: c tanh(s_t / c))
//   y   = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  m = max_t s_t
//
// in one pass over the positions that a row sees, with the running maximum and sum.
#include "q4_attention_many.hpp"

namespace q4 {
namespace {

// q of 32 bits: everything is fp32 on the exactly decoded values, on the vector units.
//
// A kv head's heads and a sequence's rows together are the rows; a workgroup takes R of
// them, so that a code is taken apart once for R, and a wavefront every fourth tile of 64
// positions: first a position a lane (its R scores), then two columns a lane or four.  q
// and the weights lie in LDS with R beside each other, which all lanes read at once.
// Where there are few workgroups the positions are split over several (every splits-th
// four tiles), and the parts joined in a second launch.
//
// Bound by the vector units: some 6 + 2 R instructions for the two codes of a byte, and the
// LDS reads beside them.  They issue in 81% of the busy cycles over one row of 131072
// positions, in all of them for a prompt of 2000.  32 heads of 128 on 8 kv heads: one row
// of 131072 positions 121 us, 21 of them the joining of 64 parts by eight workgroups
// (a workgroup to a row and head, without splits: 4607), 64 sequences of 4096 196 us (468),
// a prompt of 2000 705 us (2421), 512 rows behind 16384 2.7 ms (9.3).  q of 16 bits, on
// matrix cores, takes 42, 70, 74 and 203 us.
template <int NB, int R>
struct RowLds {
  float q[NB * kQK][R];
  union {
    float weights[kWaves][kTile][R];
    float cols[kWaves][R][NB * kQK];
  };
  float stats[kWaves][R][2];
};

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {  // N: 1 or a multiple of 4
  if constexpr (N == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4_t w = *reinterpret_cast<const float4_t*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = w[j];
    }
  }
}

template <int NB, int R>
__global__ __launch_bounds__(kWaves* kWave) void attention_row_kernel(Attention a, Many y) {
  constexpr int D = NB * kQK, C = NB > 4 ? 2 : 1;  // byte columns of a lane
  __shared__ __attribute__((aligned(16))) RowLds<NB, R> lds;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int s, h, r0, rows, split;
  Seq q;
  if (!job_of<R>(a, y, blockIdx.x, &s, &h, &r0, &rows, &split, &q)) return;
  for (int i = threadIdx.x; i < R * D; i += kWaves * kWave) {
    const int j = i / D, e = i - j * D, r = r0 + j < rows ? r0 + j : rows - 1, token = r / a.group;
    const float v = static_cast<const float*>(a.q)[(q.row + token) * a.q_stride +
                                                   static_cast<int64_t>(h * a.group + r - token * a.group) * D + e];
    lds.q[e][j] = fmaf(v, 0.f, v);  // (NaN of an infinity: see query_pair)
  }
  int lo[R], hi[R], first = 0x7FFFFFFF, end = 0;  // what each row sees, and all together
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = r0 + j < rows ? r0 + j : rows - 1;
    seen_by(a, q.length, q.first + r / a.group, &lo[j], &hi[j]);
    if (lo[j] < hi[j]) {
      first = lo[j] < first ? lo[j] : first;
      end = hi[j] > end ? hi[j] : end;
    }
  }
  __syncthreads();
  const int64_t to_values = static_cast<int64_t>(a.cache.per_page) * (9 * D);
  const Cap<false> cap(a.softcap);

  float m[R], l[R], acc[R][C][2];  // l: this lane's positions; acc: columns i and i + 16 of byte column lane + 64 c
#pragma unroll
  for (int j = 0; j < R; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[j][c][0] = acc[j][c][1] = 0.f;
  }
  for (int64_t tile = static_cast<int64_t>(end > 0 ? first / kTile : 0) + split * kWaves + wave; tile * kTile < end;
       tile += kWaves * y.splits) {
    const int t0 = static_cast<int>(tile) * kTile, t = t0 + lane, at = t & 15;
    const uint8_t* g = t < end ? granule_at(a.cache, a.batch, s, t / kGranule, h) : nullptr;
    float x[R];
#pragma unroll
    for (int j = 0; j < R; ++j) x[j] = 0.f;
    if (g != nullptr && t >= first) {
      const u32x4* words = reinterpret_cast<const u32x4*>(g + at * (D / 2));
      u32x4 w[NB];  // word i of block b is number i NB + b
#pragma unroll
      for (int i = 0; i < NB; ++i) w[i] = words[i];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float sum[R];
#pragma unroll
        for (int j = 0; j < R; ++j) sum[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t c = w[(i * NB + b) / 4][(i * NB + b) % 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float low = static_cast<float>(static_cast<int>((c >> (8 * e)) & 15u) - 8);
            const float high = static_cast<float>(static_cast<int>((c >> (8 * e + 4)) & 15u) - 8);
            float ql[R], qh[R];
            load_floats<R>(lds.q[b * kQK + 4 * i + e], ql);
            load_floats<R>(lds.q[b * kQK + 4 * i + e + 16], qh);
#pragma unroll
            for (int j = 0; j < R; ++j) sum[j] = fmaf(qh[j], high, fmaf(ql[j], low, sum[j]));
          }
        }
        const uint16_t bits = reinterpret_cast<const uint16_t*>(g + 8 * D)[((at >> 2) * NB + b) * 4 + (at & 3)];
        const float d = half_bits_to_float(bits);
#pragma unroll
        for (int j = 0; j < R; ++j) x[j] = fmaf(d, sum[j], x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      x[j] *= a.scale;
      if (a.softcap > 0.f) x[j] = cap.of(x[j]);
      if (g == nullptr || t < lo[j] || t >= hi[j]) x[j] = -INFINITY;
      float top = max_over_groups(x[j]);
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
      const float next = fmaxf(m[j], top), ref = next == -INFINITY ? 0.f : next;
      const float old = exp2f((m[j] - ref) * kLog2e), p = exp2f((x[j] - ref) * kLog2e);
      m[j] = next;
      l[j] = fmaf(l[j], old, p);
      lds.weights[wave][lane][j] = p;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        acc[j][c][0] *= old;
        acc[j][c][1] *= old;
      }
    }
    __builtin_amdgcn_wave_barrier();
    for (int gi = 0; gi < 4; ++gi) {
      const int from = t0 + 16 * gi;
      if (from >= end || from + kGranule <= first) continue;
      const uint8_t* vg = granule_at(a.cache, a.batch, s, from / kGranule, h);
      if (vg == nullptr) continue;
      vg += to_values;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = lane + kWave * c;
        if (col >= D / 2) continue;
        const u32x4 codes = *reinterpret_cast<const u32x4*>(vg + col * 16);
        const u32x4* const scales = reinterpret_cast<const u32x4*>(vg + 8 * D + col / 16 * 32);
        const u32x4 sc[2] = {scales[0], scales[1]};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          // (an unseen place may hold anything); positions 0, 2, 1, 3 of each four
          const uint32_t two = sc[e / 8][e / 4 % 2 * 2 + (e & 1)];
          const bool some = from + e >= first && from + e < end;
          const float d = some ? half_bits_to_float(static_cast<uint16_t>(e & 2 ? two >> 16 : two)) : 0.f;
          const uint32_t code = codes[e / 4] >> (8 * (e & 3));
          const float low = static_cast<float>(static_cast<int>(code & 15u) - 8) * d;
          const float high = static_cast<float>(static_cast<int>((code >> 4) & 15u) - 8) * d;
          float p[R];
          load_floats<R>(lds.weights[wave][16 * gi + e], p);
#pragma unroll
          for (int j = 0; j < R; ++j) {
            acc[j][c][0] = fmaf(p[j], low, acc[j][c][0]);
            acc[j][c][1] = fmaf(p[j], high, acc[j][c][1]);
          }
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  // The wavefronts' parts, in their order.
  __syncthreads();
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float sum = sum_over_groups(l[j]);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) {
      lds.stats[wave][j][0] = m[j];
      lds.stats[wave][j][1] = sum;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = lane + kWave * c;
      if (col >= D / 2) continue;
      lds.cols[wave][j][col / 16 * 32 + col % 16] = acc[j][c][0];
      lds.cols[wave][j][col / 16 * 32 + col % 16 + 16] = acc[j][c][1];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * D; i += kWaves * kWave) {
    const int j = i / D, e = i - j * D, r = r0 + j;
    if (r >= rows) return;
    float top = -INFINITY, sum = 0.f, v = 0.f;
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds.stats[w][j][0]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWaves; ++w) {
      const float by = exp2f((lds.stats[w][j][0] - ref) * kLog2e);
      sum = fmaf(lds.stats[w][j][1], by, sum);
      v = fmaf(lds.cols[w][j][e], by, v);
    }
    if (y.splits > 1) {
      const int64_t part = static_cast<int64_t>(blockIdx.x) * R + j;
      reinterpret_cast<float*>(y.cols)[part * D + e] = v;
      if (e == 0) reinterpret_cast<float2*>(y.stats)[part] = float2{top, sum};
      continue;
    }
    const int token = r / a.group;
    const int64_t out = static_cast<int64_t>(q.row + token) * a.heads + h * a.group + r - token * a.group;
    store_as(a.y, a.y_dt, out * D + e, sum != 0.f ? v / sum : 0.f);
    if (a.lse != nullptr && e == 0) a.lse[out] = sum != 0.f ? top + logf(sum) : -INFINITY;
  }
}

// The splits' parts, in their order: a workgroup takes the R rows of one.
template <int R>
__global__ __launch_bounds__(kWaves* kWave) void attention_row_join_kernel(Attention a, Many y) {
  const int kv = a.cache.kv_heads, dim = a.cache.dim;
  const int64_t block0 = blockIdx.x / kv * y.splits * kv + blockIdx.x % kv;
  int s, h, r0, rows, split;
  Seq q;
  if (!job_of<R>(a, y, block0, &s, &h, &r0, &rows, &split, &q)) return;
  for (int i = threadIdx.x; i < R * dim; i += kWaves * kWave) {
    const int j = i / dim, e = i - j * dim, r = r0 + j;
    if (r >= rows) return;
    float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll 4
    for (int x = 0; x < y.splits; ++x) {
      const int64_t part = (block0 + static_cast<int64_t>(x) * kv) * R + j;
      const float2 st = reinterpret_cast<const float2*>(y.stats)[part];
      const float col = reinterpret_cast<const float*>(y.cols)[part * dim + e];
      const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.f : next;
      const float old = exp2f((top - ref) * kLog2e), by = exp2f((st.x - ref) * kLog2e);
      top = next;
      sum = fmaf(sum, old, st.y * by);
      v = fmaf(v, old, col * by);
    }
    const int token = r / a.group;
    const int64_t out = static_cast<int64_t>(q.row + token) * a.heads + h * a.group + r - token * a.group;
    store_as(a.y, a.y_dt, out * dim + e, sum != 0.f ? v / sum : 0.f);
    if (a.lse != nullptr && e == 0) a.lse[out] = sum != 0.f ? top + logf(sum) : -INFINITY;
  }
}

// Rows of a workgroup: one where sequences have one, else four, or eight where they have
// as many on average.
int row_rows(const Attention& a) {
  const int64_t rows = static_cast<int64_t>(a.batch.tokens) * a.group, seqs = a.batch.seqs;
  return rows <= seqs ? 1 : rows < 8 * seqs ? 4 : 8;
}
int64_t row_places(const Attention& a) {
  const int rows = row_rows(a);
  if (a.batch.offsets == nullptr) return static_cast<int64_t>(a.batch.seqs) * ((a.group + rows - 1) / rows);
  return static_cast<int64_t>(a.batch.tokens) * a.group / rows + a.batch.seqs;
}
// Parts of the positions: as many as give each compute unit two workgroups, at most 64.
// (32, 64, 256 of them, one row of one head: 131072 positions 107, 63, 49 us, 1000 positions
// 15, 18, 40; one row of 32 heads on 8 kv heads, 131072 positions: 184, 122, 122.)
int row_splits(const Attention& a) {
  const int64_t n = row_places(a) * a.cache.kv_heads, room = 2 * static_cast<int64_t>(device_cu_count());
  return n >= room ? 1 : static_cast<int>(room / n < 64 ? room / n : 64);
}
size_t row_stats_bytes(const Attention& a) {
  return (static_cast<size_t>(row_places(a)) * a.cache.kv_heads * row_splits(a) * row_rows(a) * 8 + 15) / 16 * 16;
}
size_t row_bytes(const Attention& a) {
  if (row_splits(a) == 1) return 0;
  return row_stats_bytes(a) +
         static_cast<size_t>(row_places(a)) * a.cache.kv_heads * row_splits(a) * row_rows(a) * a.cache.dim * 4;
}

template <int NB, int R>
hipError_t launch_row_as(const Attention& a, void* workspace, Queue q) {
  Attention args = a;
  Many y;
  y.splits = row_splits(a);
  y.places = row_places(a);
  y.stats = static_cast<float*>(workspace);
  y.cols = reinterpret_cast<float4_t*>(behind(workspace, row_stats_bytes(a)));
  void* argv[] = {&args, &y};
  const int64_t jobs = y.places * a.cache.kv_heads;
  const hipError_t e = launch_blocks(reinterpret_cast<const void*>(&attention_row_kernel<NB, R>), jobs * y.splits,
                                     kWaves * kWave, argv, 0, q);
  if (e != hipSuccess || y.splits == 1) return e;
  return launch_blocks(reinterpret_cast<const void*>(&attention_row_join_kernel<R>), jobs, kWaves * kWave, argv, 0, q);
}
template <int NB>
hipError_t launch_row(const Attention& a, void* workspace, Queue q) {
  switch (row_rows(a)) {
    case 1: return launch_row_as<NB, 1>(a, workspace, q);
    case 4: return launch_row_as<NB, 4>(a, workspace, q);
    default: return launch_row_as<NB, 8>(a, workspace, q);
  }
}

}  // namespace

size_t attention_workspace_bytes(const Attention& a) {
  if (a.qt == DType::F32) return row_bytes(a);
  return a.batch.offsets == nullptr ? attention_few_bytes(a) : attention_mixed_bytes(a);
}

hipError_t launch_attention(const Attention& a, void* workspace, Queue q) {
  if (a.qt != DType::F32)
    return a.batch.offsets == nullptr ? launch_attention_few(a, workspace, q) : launch_attention_mixed(a, workspace, q);
  switch (a.cache.dim / kQK) {
    case 1: return launch_row<1>(a, workspace, q);
    case 2: return launch_row<2>(a, workspace, q);
    case 3: return launch_row<3>(a, workspace, q);
    case 4: return launch_row<4>(a, workspace, q);
    case 5: return launch_row<5>(a, workspace, q);
    case 6: return launch_row<6>(a, workspace, q);
    case 7: return launch_row<7>(a, workspace, q);
    default: return launch_row<8>(a, workspace, q);
  }
}

}  // namespace q4
