// libq4 C ABI: argument validation and dispatch.  Every check runs on the host
// before anything touches the device; the library keeps no state, never
// allocates, frees or synchronises.
#include <mutex>

#include "q4.h"
#include "q4_cache.hpp"

// Workspace of q4_gemm_noalloc: one copy per device that loads the library,
// held until the process ends.  In host code `scratch` names a host-side
// stand-in, never the device memory: the device address is looked up per
// device with hipGetSymbolAddress and only that address reaches a kernel.
static __device__ __align__(256) uint8_t scratch[Q4_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 31;
// Largest k of a matmul: the kernels address a tile's rows of x and of the
// packed weight with 32-bit per-lane byte offsets (up to 128 rows of 2 k
// bytes of activations), which stay below 2^32 for k <= 2^24.
constexpr int64_t kMaxMatmulK = int64_t(1) << 24;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Inputs (weights, activations) may be bf16; outputs are fp32 or fp16.
bool valid_in_dtype(int dt) { return dt == Q4_F32 || dt == Q4_F16 || dt == Q4_BF16; }
bool valid_out_dtype(int dt) { return dt == Q4_F32 || dt == Q4_F16; }

size_t dtype_bytes(int dt) { return dt == Q4_F32 ? 4 : 2; }

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a);
  const uintptr_t pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

bool valid_nk(int64_t n, int64_t k) {
  return n >= 1 && k >= Q4_QK && k % Q4_QK == 0 && n < kMaxRows &&
         k < kMaxElems && n <= kMaxElems / k;
}

q4_status from_hip(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }

// Device address of `scratch` on the current device, looked up once per
// device (each device holds its own copy at its own address).
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_dev[kMaxDevices] = {};

q4_status scratch_address(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return Q4_ERR_HIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_dev[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr)
      return Q4_ERR_HIP;
    g_scratch_dev[dev] = p;
  }
  *out = g_scratch_dev[dev];
  return Q4_OK;
}

q4_status check_matmul(const void* x, int x_dtype, const void* packed, void* y,
                       int y_dtype, int64_t m, int64_t n, int64_t k) {
  if (!x || !packed || !y) return Q4_ERR_INVALID_ARG;
  if (!valid_nk(n, k) || k > kMaxMatmulK || m < 1 || m >= kMaxRows || m > kMaxElems / k ||
      m > kMaxElems / n)
    return Q4_ERR_SHAPE;
  if (!valid_in_dtype(x_dtype) || !valid_out_dtype(y_dtype)) return Q4_ERR_DTYPE;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(y)) return Q4_ERR_ALIGNMENT;
  const size_t ybytes = static_cast<size_t>(m) * n * dtype_bytes(y_dtype);
  const size_t xbytes = static_cast<size_t>(m) * k * dtype_bytes(x_dtype);
  if (overlap(y, ybytes, x, xbytes) || overlap(y, ybytes, packed, q4_packed_size(n, k)))
    return Q4_ERR_INVALID_ARG;
  return Q4_OK;
}

// ------------------------------------------------------------------ fused

// A product without its buffers.  experts == 0: dense.
q4::Product make_product(int x_dtype, int64_t x_rows, int64_t m, int64_t n, int64_t k, int64_t topk = 1,
                         int64_t experts = 0, bool combine = false) {
  q4::Product p;
  p.xt = static_cast<q4::DType>(x_dtype);
  p.x_rows = x_rows;
  p.m = m;
  p.n = n;
  p.k = k;
  p.topk = topk;
  p.experts = experts;
  p.combine = combine;
  return p;
}

// Whether a grid holds every launch of a product: a matter of the shape, settled
// before the first of them.
bool fits(const q4::Product& p) { return q4::launch_product(p, nullptr, q4::Queue{nullptr, true}) == hipSuccess; }

constexpr int64_t kMaxPairs = int64_t(1) << 24;  // tokens x experts each

struct Span {
  const void* p;
  size_t n;
};

// out shares a byte with one of `in` (empty and null spans share none).
template <size_t N>
bool overlaps_any(Span out, const Span (&in)[N]) {
  for (const Span& i : in)
    if (out.p && i.p && out.n && i.n && overlap(out.p, out.n, i.p, i.n)) return true;
  return false;
}

// A checked product: what both q4_linear and q4_experts ask of their
// arguments.  groups: weight matrices in `packed`; y_rows x (n or n / 2) outputs.
q4_status check_product(const void* x, int x_dtype, int64_t x_rows, const void* packed, int64_t groups,
                        const q4_epilogue* ep, void* y, int y_dtype, int64_t y_rows, int64_t n,
                        int64_t k, void* workspace, size_t need, size_t workspace_bytes,
                        Span plan, Span weights) {
  const q4_epilogue none = {nullptr, 0, Q4_ACT_NONE, 0, nullptr};
  if (!ep) ep = &none;
  if (ep->activation < Q4_ACT_NONE || ep->activation > Q4_ACT_SILU || ep->gated < 0 || ep->gated > 1)
    return Q4_ERR_INVALID_ARG;
  if (ep->gated && n % 2 != 0) return Q4_ERR_SHAPE;
  if (!valid_in_dtype(x_dtype) || !valid_in_dtype(y_dtype) ||
      (ep->bias && !valid_in_dtype(ep->bias_dtype)))
    return Q4_ERR_DTYPE;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(y) || !aligned16(ep->bias) ||
      !aligned16(ep->residual))
    return Q4_ERR_ALIGNMENT;
  const int64_t nout = ep->gated ? n / 2 : n;
  const Span ys{y, static_cast<size_t>(y_rows) * nout * dtype_bytes(y_dtype)};
  const Span rs{ep->residual == y ? nullptr : ep->residual, ys.n};  // in place is allowed
  const Span xs{x, static_cast<size_t>(x_rows) * k * dtype_bytes(x_dtype)};
  const Span ws{packed, static_cast<size_t>(groups) * q4_packed_size(n, k)};
  const Span bs{ep->bias, ep->bias ? static_cast<size_t>(groups) * n * dtype_bytes(ep->bias_dtype) : 0};
  if (overlaps_any(ys, {xs, ws, bs, rs, plan, weights})) return Q4_ERR_INVALID_ARG;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q4_ERR_ALIGNMENT;
    if (overlaps_any({workspace, need}, {xs, ws, bs, Span{ep->residual, ys.n}, ys, plan, weights}))
      return Q4_ERR_INVALID_ARG;
  }
  return Q4_OK;
}

// For the sizes: some epilogue, so that the product is none that q4_gemv takes
// (which needs no workspace).
q4::Epi size_epi(int64_t n, bool gate) {
  q4::Epi e;
  e.act = q4::kActRelu;
  e.ldy = gate ? n / 2 : n;
  e.half = gate ? n / 2 : 0;
  return e;
}

q4::Epi make_epi(const q4_epilogue* ep, void* y, int y_dtype, int64_t n) {
  q4::Epi e;
  e.y = y;
  e.y_dt = y_dtype;
  e.ldy = n;
  if (ep) {
    e.bias = ep->bias;
    e.bias_dt = ep->bias_dtype;
    e.residual = ep->residual;
    e.act = ep->activation;
    if (ep->gated) e.ldy = e.half = n / 2;
  }
  return e;
}

bool gated(const q4_epilogue* ep) { return ep && ep->gated == 1; }

bool valid_linear(int64_t m, int64_t n, int64_t k) {
  return valid_nk(n, k) && k <= kMaxMatmulK && m >= 1 && m < kMaxRows && m <= kMaxElems / k &&
         m <= kMaxElems / n;
}

// Token and expert counts of a plan.
bool valid_pairs(int64_t m, int64_t topk, int64_t experts) {
  return experts >= 1 && experts <= Q4_MAX_EXPERTS && topk >= 1 && topk <= Q4_MAX_TOPK && m >= 1 &&
         m <= kMaxPairs && m * topk <= kMaxPairs;
}

bool valid_experts(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k) {
  return valid_pairs(m, topk, experts) && valid_nk(n, k) && k <= kMaxMatmulK && n < kMaxMatmulK &&
         experts <= kMaxElems / (n * k) && m * topk <= (kMaxElems >> 3) / n &&
         m * topk <= (kMaxElems >> 3) / k;
}

q4_status check_routing(const void* logits, int logits_dtype, int64_t m, int64_t experts, int64_t topk,
                        const q4_routing* r) {
  if (!logits || !r) return Q4_ERR_INVALID_ARG;
  if (!valid_pairs(m, topk, experts) || topk > experts) return Q4_ERR_SHAPE;
  if (r->groups < 1 || r->groups > Q4_MAX_GROUPS || experts % r->groups != 0 || r->group_topk < 1 ||
      r->group_topk > r->groups)
    return Q4_ERR_SHAPE;
  if (!valid_in_dtype(logits_dtype)) return Q4_ERR_DTYPE;
  if ((r->score != Q4_SCORE_SOFTMAX && r->score != Q4_SCORE_SIGMOID) ||
      (r->group_score != Q4_GROUP_MAX && r->group_score != Q4_GROUP_TOP2) || r->renormalise < 0 ||
      r->renormalise > 1 || !(r->scale - r->scale == 0.0f))
    return Q4_ERR_INVALID_ARG;
  if (!aligned16(logits) || (reinterpret_cast<uintptr_t>(r->bias) & 3u) != 0) return Q4_ERR_ALIGNMENT;
  return Q4_OK;
}

q4::RouteArgs make_route(const void* logits, int logits_dtype, int64_t m, int64_t experts, int64_t topk,
                         const q4_routing& r, int32_t* ids, float* weights, void* plan) {
  return q4::RouteArgs{logits, static_cast<q4::DType>(logits_dtype), m, experts, topk, r.bias,
                       r.score == Q4_SCORE_SIGMOID, r.groups, r.group_topk,
                       r.group_score == Q4_GROUP_TOP2, r.renormalise, r.scale, ids, weights,
                       static_cast<int*>(plan)};
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

extern "C" {

int q4_abi_version(void) { return Q4_ABI_VERSION; }

const char* q4_status_string(int status) {
  switch (status) {
    case Q4_OK: return "ok";
    case Q4_ERR_INVALID_ARG: return "invalid argument (null pointer, overlapping buffers or an option out of range)";
    case Q4_ERR_SHAPE: return "invalid shape (need m, n >= 1, k >= 32, k % 32 == 0, within size limits)";
    case Q4_ERR_DTYPE: return "unsupported dtype for this call";
    case Q4_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case Q4_ERR_HIP: return "HIP runtime refused the kernel launch";
    case Q4_ERR_WORKSPACE: return "workspace missing or too small";
    case Q4_ERR_UNSUPPORTED: return "the host CPU lacks AVX2, FMA or F16C";
    case Q4_ERR_SCRATCH: return "the call needs more scratch than q4_gemm_noalloc's fixed array holds";
    default: return "unknown q4 status";
  }
}

size_t q4_packed_size(int64_t n, int64_t k) {
  if (!valid_nk(n, k)) return 0;
  return static_cast<size_t>(n) * static_cast<size_t>(k / Q4_QK) * Q4_BLOCK_BYTES;
}

q4_status q4_quantize(const void* w, int w_dtype, int64_t n, int64_t k, void* packed,
                      q4_stream_t stream) {
  if (!w || !packed) return Q4_ERR_INVALID_ARG;
  if (!valid_nk(n, k)) return Q4_ERR_SHAPE;
  if (!valid_in_dtype(w_dtype)) return Q4_ERR_DTYPE;
  if (!aligned16(w) || !aligned16(packed)) return Q4_ERR_ALIGNMENT;
  if (overlap(w, static_cast<size_t>(n) * k * dtype_bytes(w_dtype), packed,
              q4_packed_size(n, k)))
    return Q4_ERR_INVALID_ARG;
  return from_hip(q4::launch_quantize(w, static_cast<q4::DType>(w_dtype), n, k,
                                      static_cast<uint8_t*>(packed),
                                      reinterpret_cast<hipStream_t>(stream)));
}

q4_status q4_gemv(const void* x, int x_dtype, const void* packed, void* y, int y_dtype,
                  int64_t m, int64_t n, int64_t k, q4_stream_t stream) {
  const q4_status st = check_matmul(x, x_dtype, packed, y, y_dtype, m, n, k);
  if (st != Q4_OK) return st;
  if (m > Q4_GEMV_MAX_M) return Q4_ERR_SHAPE;
  return from_hip(q4::launch_gemv(x, static_cast<q4::DType>(x_dtype),
                                  static_cast<const uint8_t*>(packed), y,
                                  static_cast<q4::DType>(y_dtype), static_cast<int>(m),
                                  n, k, reinterpret_cast<hipStream_t>(stream)));
}

size_t q4_gemm_workspace_size(int64_t m, int64_t n, int64_t k) {
  return q4_gemm_workspace_size_dt(m, n, k, Q4_F16);
}

size_t q4_gemm_workspace_size_dt(int64_t m, int64_t n, int64_t k, int x_dtype) {
  if (!valid_nk(n, k) || k > kMaxMatmulK || m < 1 || m >= kMaxRows || m > kMaxElems / k)
    return 0;
  if (!valid_in_dtype(x_dtype)) return 0;
  return q4::gemm_workspace_bytes(m, n, k, static_cast<q4::DType>(x_dtype));
}

q4_status q4_gemm(const void* x, int x_dtype, const void* packed, void* y, int y_dtype,
                  int64_t m, int64_t n, int64_t k, void* workspace,
                  size_t workspace_bytes, q4_stream_t stream) {
  const q4_status st = check_matmul(x, x_dtype, packed, y, y_dtype, m, n, k);
  if (st != Q4_OK) return st;
  const size_t need = q4::gemm_workspace_bytes(m, n, k, static_cast<q4::DType>(x_dtype));
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q4_ERR_ALIGNMENT;
    const size_t xbytes = static_cast<size_t>(m) * k * dtype_bytes(x_dtype);
    if (overlap(workspace, need, x, xbytes) || overlap(workspace, need, y,
                static_cast<size_t>(m) * n * dtype_bytes(y_dtype)) ||
        overlap(workspace, need, packed, q4_packed_size(n, k)))
      return Q4_ERR_INVALID_ARG;
  }
  return from_hip(q4::launch_gemm(x, static_cast<q4::DType>(x_dtype),
                                  static_cast<const uint8_t*>(packed),
                                  y, static_cast<q4::DType>(y_dtype), m, n, k,
                                  need > 0 ? workspace : nullptr,
                                  reinterpret_cast<hipStream_t>(stream)));
}

q4_status q4_gemm_noalloc(const void* x, int x_dtype, const void* packed, void* y,
                          int y_dtype, int64_t m, int64_t n, int64_t k, q4_stream_t stream) {
  const q4_status st = check_matmul(x, x_dtype, packed, y, y_dtype, m, n, k);
  if (st != Q4_OK) return st;
  const size_t need = q4::gemm_workspace_bytes(m, n, k, static_cast<q4::DType>(x_dtype));
  if (need > Q4_NOALLOC_SCRATCH_BYTES) return Q4_ERR_SCRATCH;
  void* ws = nullptr;
  if (need > 0) {
    const q4_status sa = scratch_address(&ws);
    if (sa != Q4_OK) return sa;
  }
  return from_hip(q4::launch_gemm(x, static_cast<q4::DType>(x_dtype),
                                  static_cast<const uint8_t*>(packed),
                                  y, static_cast<q4::DType>(y_dtype), m, n, k, ws,
                                  reinterpret_cast<hipStream_t>(stream)));
}

size_t q4_linear_workspace_size(int64_t m, int64_t n, int64_t k, int x_dtype, int gate) {
  if (!valid_linear(m, n, k) || !valid_in_dtype(x_dtype) || gate < 0 || gate > 1 ||
      (gate && n % 2 != 0))
    return 0;
  q4::Product p = make_product(x_dtype, m, m, n, k);
  p.ep = size_epi(n, gate == 1);
  if (!fits(p)) return 0;
  return q4::product_workspace_bytes(m, 1, 0, n, k, m, p.xt, gate == 1, false);
}

q4_status q4_linear(const void* x, int x_dtype, const void* packed, const q4_epilogue* epilogue,
                    void* y, int y_dtype, int64_t m, int64_t n, int64_t k, void* workspace,
                    size_t workspace_bytes, q4_stream_t stream) {
  if (!x || !packed || !y) return Q4_ERR_INVALID_ARG;
  if (!valid_linear(m, n, k)) return Q4_ERR_SHAPE;
  const size_t need = q4_linear_workspace_size(m, n, k, x_dtype, gated(epilogue));
  const q4_status st = check_product(x, x_dtype, m, packed, 1, epilogue, y, y_dtype, m, n, k, workspace,
                                     need, workspace_bytes, {nullptr, 0}, {nullptr, 0});
  if (st != Q4_OK) return st;
  q4::Product p = make_product(x_dtype, m, m, n, k);
  p.x = x;
  p.W = static_cast<const uint8_t*>(packed);
  p.ep = make_epi(epilogue, y, y_dtype, n);
  if (!fits(p)) return Q4_ERR_SHAPE;
  return from_hip(q4::launch_product(p, workspace, q4::Queue{reinterpret_cast<hipStream_t>(stream)}));
}

size_t q4_route_plan_size(int64_t m, int64_t topk, int64_t experts) {
  if (!valid_pairs(m, topk, experts)) return 0;
  return static_cast<size_t>(q4::plan_layout(m, topk, experts).words) * 4;
}

q4_status q4_route(const void* logits, int logits_dtype, int64_t m, int64_t experts, int64_t topk,
                   const q4_routing* routing, int32_t* ids, float* weights, void* plan,
                   q4_stream_t stream) {
  if (!ids || !weights) return Q4_ERR_INVALID_ARG;
  const q4_status st = check_routing(logits, logits_dtype, m, experts, topk, routing);
  if (st != Q4_OK) return st;
  if (!aligned16(ids) || !aligned16(weights) || !aligned16(plan)) return Q4_ERR_ALIGNMENT;
  const size_t pairs = static_cast<size_t>(m * topk);
  const Span ls{logits, static_cast<size_t>(m) * experts * dtype_bytes(logits_dtype)};
  const Span bs{routing->bias, static_cast<size_t>(experts) * 4};
  const Span is{ids, pairs * 4}, ws{weights, pairs * 4}, ps{plan, q4_route_plan_size(m, topk, experts)};
  if (overlaps_any(is, {ls, bs, ws, ps}) || overlaps_any(ws, {ls, bs, ps}) || overlaps_any(ps, {ls, bs}))
    return Q4_ERR_INVALID_ARG;
  return from_hip(q4::launch_route(
      make_route(logits, logits_dtype, m, experts, topk, *routing, ids, weights, plan),
      reinterpret_cast<hipStream_t>(stream)));
}

q4_status q4_route_plan(const int32_t* ids, int64_t m, int64_t topk, int64_t experts, void* plan,
                        q4_stream_t stream) {
  if (!ids || !plan) return Q4_ERR_INVALID_ARG;
  if (!valid_pairs(m, topk, experts)) return Q4_ERR_SHAPE;
  if (!aligned16(ids) || !aligned16(plan)) return Q4_ERR_ALIGNMENT;
  if (overlap(ids, static_cast<size_t>(m * topk) * 4, plan, q4_route_plan_size(m, topk, experts)))
    return Q4_ERR_INVALID_ARG;
  return from_hip(q4::launch_route_plan(ids, m, topk, experts, static_cast<int*>(plan),
                                        reinterpret_cast<hipStream_t>(stream)));
}

size_t q4_experts_workspace_size(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k,
                                 int64_t x_rows, int x_dtype, int gate, int combine) {
  if (!valid_experts(m, topk, experts, n, k) || (x_rows != m && x_rows != m * topk) ||
      !valid_in_dtype(x_dtype) || gate < 0 || gate > 1 || (gate && n % 2 != 0))
    return 0;
  q4::Product p = make_product(x_dtype, x_rows, m, n, k, topk, experts, combine != 0);
  p.ep = size_epi(n, gate == 1);
  if (!fits(p)) return 0;
  return q4::product_workspace_bytes(m, topk, experts, n, k, x_rows, p.xt, gate == 1, combine != 0);
}

q4_status q4_experts(const void* x, int x_dtype, int64_t x_rows, const void* packed,
                     const q4_epilogue* epilogue, const void* plan, const float* weights, void* y,
                     int y_dtype, int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k,
                     void* workspace, size_t workspace_bytes, q4_stream_t stream) {
  if (!x || !packed || !y || !plan) return Q4_ERR_INVALID_ARG;
  if (!valid_experts(m, topk, experts, n, k) || (x_rows != m && x_rows != m * topk)) return Q4_ERR_SHAPE;
  if (!aligned16(plan) || !aligned16(weights)) return Q4_ERR_ALIGNMENT;
  const size_t need = q4_experts_workspace_size(m, topk, experts, n, k, x_rows, x_dtype,
                                                gated(epilogue), weights != nullptr);
  const q4_status st = check_product(
      x, x_dtype, x_rows, packed, experts, epilogue, y, y_dtype, weights ? m : m * topk, n, k, workspace,
      need, workspace_bytes, {plan, q4_route_plan_size(m, topk, experts)},
      {weights, weights ? static_cast<size_t>(m * topk) * 4 : 0});
  if (st != Q4_OK) return st;
  q4::Product p = make_product(x_dtype, x_rows, m, n, k, topk, experts, weights != nullptr);
  p.x = x;
  p.W = static_cast<const uint8_t*>(packed);
  p.plan = static_cast<const int*>(plan);
  p.weights = weights;
  p.ep = make_epi(epilogue, y, y_dtype, n);
  if (!fits(p)) return Q4_ERR_SHAPE;
  return from_hip(q4::launch_product(p, workspace, q4::Queue{reinterpret_cast<hipStream_t>(stream)}));
}

}  // extern "C"

namespace {

// Workspace of q4_moe: plan, ids, weights, the rows between the products, and
// the larger of the two products' own.
struct MoeLayout {
  size_t ids, weights, h, product, total;
};

MoeLayout moe_layout(int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter,
                     int x_dtype, bool gate) {
  const int64_t pairs = m * topk;
  MoeLayout L;
  L.ids = up256(q4_route_plan_size(m, topk, experts));
  L.weights = L.ids + up256(static_cast<size_t>(pairs) * 4);
  L.h = L.weights + up256(static_cast<size_t>(pairs) * 4);
  L.product = L.h + up256(static_cast<size_t>(pairs) * inter * dtype_bytes(x_dtype));
  const size_t a = q4_experts_workspace_size(m, topk, experts, gate ? 2 * inter : inter, hidden, m, x_dtype,
                                             gate, 0);
  const size_t b = q4_experts_workspace_size(m, topk, experts, hidden, inter, pairs, x_dtype, 0, 1);
  L.total = L.product + (a > b ? a : b);
  return L;
}

bool valid_moe(int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter, bool gate) {
  return inter >= 1 && inter < kMaxMatmulK &&
         valid_experts(m, topk, experts, gate ? 2 * inter : inter, hidden) &&
         valid_experts(m, topk, experts, hidden, inter);
}

// The two products of a layer, without their buffers.
struct MoeProducts {
  q4::Product up, down;
};

MoeProducts moe_products(int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter, int x_dtype,
                         bool gate) {
  const int64_t nup = gate ? 2 * inter : inter;
  MoeProducts p{make_product(x_dtype, m, m, nup, hidden, topk, experts),
                make_product(x_dtype, m * topk, m, hidden, inter, topk, experts, true)};
  p.up.ep = size_epi(nup, gate);
  p.down.ep = size_epi(hidden, false);
  return p;
}

// As fits, for the launches of a layer.  (The routing's always do.)
bool moe_fits(const MoeProducts& p) {
  q4::RouteArgs r{};
  r.m = p.up.m;
  r.topk = p.up.topk;
  r.experts = p.up.experts;
  if (q4::moe_one_supports(r, p.up, p.down))
    return q4::launch_moe_one(r, p.up, p.down, q4::Queue{nullptr, true}) == hipSuccess;
  return fits(p.up) && fits(p.down);
}

}  // namespace

extern "C" {

size_t q4_moe_workspace_size(int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter,
                             int x_dtype, int gate) {
  if (gate < 0 || gate > 1 || !valid_in_dtype(x_dtype) || topk > experts ||
      !valid_moe(m, topk, experts, hidden, inter, gate == 1) ||
      !moe_fits(moe_products(m, topk, experts, hidden, inter, x_dtype, gate == 1)))
    return 0;
  return moe_layout(m, topk, experts, hidden, inter, x_dtype, gate == 1).total;
}

q4_status q4_moe(const void* x, int x_dtype, const void* logits, int logits_dtype,
                 const q4_routing* routing, const void* up, const q4_epilogue* up_epilogue,
                 const void* down, const q4_epilogue* down_epilogue, void* y, int y_dtype, int64_t m,
                 int64_t topk, int64_t experts, int64_t hidden, int64_t inter, int32_t* ids,
                 float* weights, void* workspace, size_t workspace_bytes, q4_stream_t stream) {
  if (!x || !up || !down || !y || !up_epilogue) return Q4_ERR_INVALID_ARG;
  const q4_status sr = check_routing(logits, logits_dtype, m, experts, topk, routing);
  if (sr != Q4_OK) return sr;
  if (up_epilogue->gated < 0 || up_epilogue->gated > 1 || up_epilogue->residual ||
      (down_epilogue && (down_epilogue->gated != 0 || down_epilogue->activation != Q4_ACT_NONE)))
    return Q4_ERR_INVALID_ARG;
  const bool gate = up_epilogue->gated == 1;
  if (!valid_moe(m, topk, experts, hidden, inter, gate)) return Q4_ERR_SHAPE;
  if (!valid_in_dtype(x_dtype)) return Q4_ERR_DTYPE;
  if (!aligned16(ids) || !aligned16(weights)) return Q4_ERR_ALIGNMENT;
  MoeProducts products = moe_products(m, topk, experts, hidden, inter, x_dtype, gate);
  if (!moe_fits(products)) return Q4_ERR_SHAPE;
  const MoeLayout L = moe_layout(m, topk, experts, hidden, inter, x_dtype, gate);
  if (!workspace || workspace_bytes < L.total) return Q4_ERR_WORKSPACE;
  if (!aligned16(workspace)) return Q4_ERR_ALIGNMENT;
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  const size_t pairs = static_cast<size_t>(m * topk);
  const int64_t nup = gate ? 2 * inter : inter;
  // Every buffer against every output before anything is launched.
  const size_t ybytes = static_cast<size_t>(m) * hidden * dtype_bytes(y_dtype);
  const Span all{workspace, L.total}, ys{y, ybytes}, is{ids, pairs * 4}, ws{weights, pairs * 4};
  const Span xs{x, static_cast<size_t>(m) * hidden * dtype_bytes(x_dtype)};
  const Span ls{logits, static_cast<size_t>(m) * experts * dtype_bytes(logits_dtype)};
  const Span bs{routing->bias, static_cast<size_t>(experts) * 4};
  const Span us{up, static_cast<size_t>(experts) * q4_packed_size(nup, hidden)};
  const Span ds{down, static_cast<size_t>(experts) * q4_packed_size(hidden, inter)};
  const Span ub{up_epilogue->bias, static_cast<size_t>(experts) * nup * dtype_bytes(up_epilogue->bias_dtype)};
  const Span db{down_epilogue ? down_epilogue->bias : nullptr,
                down_epilogue ? static_cast<size_t>(experts) * hidden * dtype_bytes(down_epilogue->bias_dtype) : 0};
  const void* res = down_epilogue ? down_epilogue->residual : nullptr;
  const Span rs{res == y ? nullptr : res, ybytes};
  if (overlaps_any(all, {xs, ls, bs, us, ds, ub, db, ys, is, ws, rs}) ||
      overlaps_any(is, {xs, ls, bs, us, ds, ub, db, ys, ws, rs}) ||
      overlaps_any(ws, {xs, ls, bs, us, ds, ub, db, ys, rs}) ||
      overlaps_any(ys, {ls, bs, ub}))
    return Q4_ERR_INVALID_ARG;
  int32_t* const wids = ids ? ids : reinterpret_cast<int32_t*>(base + L.ids);
  float* const ww = weights ? weights : reinterpret_cast<float*>(base + L.weights);
  void* const h = base + L.h;
  void* const pw = base + L.product;
  const size_t pwb = L.total - L.product;
  // The arguments of both products, checked before the first launch.
  const q4_status s1 = check_product(x, x_dtype, m, up, experts, up_epilogue, h, x_dtype, m * topk, nup,
                                     hidden, pw, pwb, pwb, {base, L.ids}, {nullptr, 0});
  if (s1 != Q4_OK) return s1;
  const q4_status s2 = check_product(h, x_dtype, m * topk, down, experts, down_epilogue, y, y_dtype, m,
                                     hidden, inter, pw, pwb, pwb, {base, L.ids}, {ww, pairs * 4});
  if (s2 != Q4_OK) return s2;
  if (overlaps_any(ys, {xs, us})) return Q4_ERR_INVALID_ARG;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const q4::RouteArgs ra = make_route(logits, logits_dtype, m, experts, topk, *routing, wids, ww, base);
  q4::Product &p = products.up, &d = products.down;
  p.x = x;
  p.W = static_cast<const uint8_t*>(up);
  p.plan = d.plan = reinterpret_cast<const int*>(base);
  p.ep = make_epi(up_epilogue, h, x_dtype, nup);
  d.x = h;
  d.W = static_cast<const uint8_t*>(down);
  d.weights = ww;
  d.ep = make_epi(down_epilogue, y, y_dtype, hidden);
  const q4::Queue q{st};
  if (q4::moe_one_supports(ra, p, d)) return from_hip(q4::launch_moe_one(ra, p, d, q));
  hipError_t e = q4::launch_route(ra, st);
  if (e == hipSuccess) e = q4::launch_product(p, pw, q);
  if (e == hipSuccess) e = q4::launch_product(d, pw, q);
  return from_hip(e);
}

}  // extern "C"

// ------------------------------------------------------------------ cache and attention

namespace {

constexpr int64_t kMaxPositions = int64_t(1) << 30;  // of one sequence, and of one page
constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxHeads = 65536;

bool valid_cache(int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  return pages >= 1 && pages <= kMaxInt && page_size >= Q4_CACHE_GRANULE && page_size <= kMaxPositions &&
         page_size % Q4_CACHE_GRANULE == 0 && kv_heads >= 1 && kv_heads < kMaxHeads && head_dim >= Q4_QK &&
         head_dim <= Q4_CACHE_MAX_HEAD_DIM && head_dim % Q4_QK == 0 &&
         pages <= kMaxElems / (page_size * head_dim) / kv_heads;
}

bool valid_rows(int64_t seqs, int64_t tokens) {
  return seqs >= 1 && seqs <= Q4_CACHE_MAX_SEQS && tokens >= 1 && tokens <= kMaxInt;
}

// What every call asks of its cache and batch.
q4_status check_cache(const q4_cache* c, const q4_batch* b) {
  if (!c || !b || !c->data || !b->tables || !b->lengths) return Q4_ERR_INVALID_ARG;
  if (!valid_cache(c->pages, c->page_size, c->kv_heads, c->head_dim) || !valid_rows(b->seqs, b->tokens) ||
      (!b->offsets && b->tokens != b->seqs) || b->max_pages < 1 || b->max_pages > kMaxPositions / c->page_size)
    return Q4_ERR_SHAPE;
  return Q4_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool aligned_batch(const q4_cache* c, const q4_batch* b) {
  return aligned16(c->data) && aligned4(b->tables) && aligned4(b->lengths) && aligned4(b->offsets);
}

// Rows of `width` elements, `stride` elements apart.
q4_status check_rows(const void* p, int64_t rows, int64_t width, int64_t stride, int dtype, Span* span) {
  if (stride < width || stride > kMaxElems || rows > kMaxElems / stride) return Q4_ERR_SHAPE;
  if (!valid_in_dtype(dtype)) return Q4_ERR_DTYPE;
  const size_t size = dtype_bytes(dtype);
  if (!aligned16(p) || static_cast<size_t>(stride) * size % 16 != 0) return Q4_ERR_ALIGNMENT;
  *span = {p, (static_cast<size_t>(rows - 1) * stride + width) * size};
  return Q4_OK;
}

Span cache_span(const q4_cache* c) {
  return {c->data, q4_cache_size(c->pages, c->page_size, c->kv_heads, c->head_dim)};
}
Span tables_span(const q4_batch* b) { return {b->tables, static_cast<size_t>(b->seqs) * b->max_pages * 4}; }
Span lengths_span(const q4_batch* b) { return {b->lengths, static_cast<size_t>(b->seqs) * 4}; }
Span offsets_span(const q4_batch* b) { return {b->offsets, b->offsets ? static_cast<size_t>(b->seqs + 1) * 4 : 0}; }

q4::Cache device_cache(const q4_cache* c) {
  return q4::make_cache(c->data, c->pages, c->page_size, c->kv_heads, c->head_dim);
}
q4::Batch device_batch(const q4_cache* c, const q4_batch* b) {
  q4::Batch d;
  d.tables = b->tables;
  d.lengths = b->lengths;
  d.offsets = b->offsets;
  d.seqs = static_cast<int>(b->seqs);
  d.tokens = static_cast<int>(b->tokens);
  d.max_pages = static_cast<int>(b->max_pages);
  d.max_length = static_cast<int>(b->max_pages * c->page_size);
  return d;
}

bool valid_heads(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  return heads >= 1 && heads <= kMaxHeads && kv_heads >= 1 && heads % kv_heads == 0 &&
         tokens <= kMaxElems / (heads * head_dim);
}

constexpr q4::Queue kDry{nullptr, true};

}  // namespace

extern "C" {

size_t q4_cache_size(int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  if (!valid_cache(pages, page_size, kv_heads, head_dim)) return 0;
  return static_cast<size_t>(pages) * page_size * kv_heads * 2 * (head_dim / Q4_QK) * Q4_BLOCK_BYTES;
}

q4_status q4_cache_write(const q4_cache* cache, const q4_batch* batch, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int dtype, q4_stream_t stream) {
  if (!k || !v) return Q4_ERR_INVALID_ARG;
  q4_status st = check_cache(cache, batch);
  if (st != Q4_OK) return st;
  const int64_t width = cache->kv_heads * cache->head_dim;
  Span ks, vs;
  if ((st = check_rows(k, batch->tokens, width, k_stride, dtype, &ks)) != Q4_OK) return st;
  if ((st = check_rows(v, batch->tokens, width, v_stride, dtype, &vs)) != Q4_OK) return st;
  if (!aligned_batch(cache, batch)) return Q4_ERR_ALIGNMENT;
  if (overlaps_any(cache_span(cache), {ks, vs, tables_span(batch), lengths_span(batch), offsets_span(batch)}))
    return Q4_ERR_INVALID_ARG;
  const q4::Cache c = device_cache(cache);
  const q4::Batch b = device_batch(cache, batch);
  const q4::DType dt = static_cast<q4::DType>(dtype);
  if (q4::launch_cache_write(c, b, k, k_stride, v, v_stride, dt, kDry) != hipSuccess) return Q4_ERR_SHAPE;
  return from_hip(q4::launch_cache_write(c, b, k, k_stride, v, v_stride, dt,
                                         q4::Queue{reinterpret_cast<hipStream_t>(stream)}));
}

q4_status q4_cache_read(const q4_cache* cache, const q4_batch* batch, void* k, void* v, int dtype,
                        q4_stream_t stream) {
  if (!k || !v) return Q4_ERR_INVALID_ARG;
  q4_status st = check_cache(cache, batch);
  if (st != Q4_OK) return st;
  const int64_t width = cache->kv_heads * cache->head_dim;
  Span ks, vs;
  if ((st = check_rows(k, batch->tokens, width, width, dtype, &ks)) != Q4_OK) return st;
  if ((st = check_rows(v, batch->tokens, width, width, dtype, &vs)) != Q4_OK) return st;
  if (!aligned_batch(cache, batch)) return Q4_ERR_ALIGNMENT;
  const Span cs = cache_span(cache), ts = tables_span(batch), ls = lengths_span(batch), os = offsets_span(batch);
  if (overlaps_any(ks, {vs, cs, ts, ls, os}) || overlaps_any(vs, {cs, ts, ls, os})) return Q4_ERR_INVALID_ARG;
  const q4::Cache c = device_cache(cache);
  const q4::Batch b = device_batch(cache, batch);
  const q4::DType dt = static_cast<q4::DType>(dtype);
  if (q4::launch_cache_read(c, b, k, v, dt, kDry) != hipSuccess) return Q4_ERR_SHAPE;
  return from_hip(q4::launch_cache_read(c, b, k, v, dt, q4::Queue{reinterpret_cast<hipStream_t>(stream)}));
}

size_t q4_attention_workspace_size(int64_t seqs, int64_t tokens, int64_t heads, int64_t kv_heads,
                                   int64_t head_dim, int q_dtype, int with_offsets) {
  if (!valid_rows(seqs, tokens) || !valid_cache(1, Q4_CACHE_GRANULE, kv_heads, head_dim) ||
      !valid_heads(tokens, heads, kv_heads, head_dim) || !valid_in_dtype(q_dtype) || with_offsets < 0 ||
      with_offsets > 1 || (!with_offsets && tokens != seqs))
    return 0;
  q4::Attention a;
  a.cache.kv_heads = static_cast<int>(kv_heads);
  a.cache.dim = static_cast<int>(head_dim);
  a.batch.seqs = static_cast<int>(seqs);
  a.batch.tokens = static_cast<int>(tokens);
  const int some = 0;
  a.batch.offsets = with_offsets ? &some : nullptr;  // (asked for being there alone)
  a.heads = static_cast<int>(heads);
  a.group = static_cast<int>(heads / kv_heads);
  a.qt = static_cast<q4::DType>(q_dtype);
  if (q4::launch_attention(a, nullptr, kDry) != hipSuccess) return 0;
  return q4::attention_workspace_bytes(a);
}

q4_status q4_attention(const q4_cache* cache, const q4_batch* batch, const q4_attention_options* options,
                       const void* q, int64_t q_stride, int q_dtype, int64_t heads, void* y, int y_dtype,
                       float* lse, void* workspace, size_t workspace_bytes, q4_stream_t stream) {
  if (!options || !q || !y) return Q4_ERR_INVALID_ARG;
  q4_status st = check_cache(cache, batch);
  if (st != Q4_OK) return st;
  if (!valid_heads(batch->tokens, heads, cache->kv_heads, cache->head_dim)) return Q4_ERR_SHAPE;
  if (!(fabsf(options->scale) <= 3.4028234e38f) || !(options->softcap >= 0.f && options->softcap <= 3.4028234e38f) ||
      options->causal < 0 || options->causal > 1 || options->window < 0)
    return Q4_ERR_INVALID_ARG;
  Span qs, ys;
  const int64_t width = heads * cache->head_dim;
  if ((st = check_rows(q, batch->tokens, width, q_stride, q_dtype, &qs)) != Q4_OK) return st;
  if ((st = check_rows(y, batch->tokens, width, width, y_dtype, &ys)) != Q4_OK) return st;
  if (!aligned_batch(cache, batch) || !aligned16(lse)) return Q4_ERR_ALIGNMENT;
  const Span es{lse, static_cast<size_t>(batch->tokens) * heads * 4};
  const Span cs = cache_span(cache), ts = tables_span(batch), ls = lengths_span(batch), os = offsets_span(batch);
  if (overlaps_any(ys, {qs, es, cs, ts, ls, os}) || overlaps_any(es, {qs, cs, ts, ls, os}))
    return Q4_ERR_INVALID_ARG;
  q4::Attention a;
  a.cache = device_cache(cache);
  a.batch = device_batch(cache, batch);
  a.q = q;
  a.q_stride = q_stride;
  a.qt = static_cast<q4::DType>(q_dtype);
  a.heads = static_cast<int>(heads);
  a.group = static_cast<int>(heads / cache->kv_heads);
  a.scale = options->scale;
  a.softcap = options->softcap;
  a.causal = options->causal;
  // A window of every position that there can be is none.
  a.window = options->window > kMaxPositions ? 0 : static_cast<int>(options->window);
  a.y = y;
  a.y_dt = y_dtype;
  a.lse = lse;
  if (q4::launch_attention(a, nullptr, kDry) != hipSuccess) return Q4_ERR_SHAPE;
  const size_t need = q4::attention_workspace_bytes(a);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q4_ERR_ALIGNMENT;
    if (overlaps_any({workspace, need}, {qs, ys, es, cs, ts, ls, os})) return Q4_ERR_INVALID_ARG;
  }
  return from_hip(q4::launch_attention(a, workspace, q4::Queue{reinterpret_cast<hipStream_t>(stream)}));
}

}  // extern "C"
