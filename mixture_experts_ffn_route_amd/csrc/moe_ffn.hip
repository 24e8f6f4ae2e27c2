// The BF16 gated feed-forward block with its gradients (moe_ffn_forward,
// moe_ffn_backward).
//
//   g | u = x w13^T, h = silu(g) u, y = h w2^T
//   dh = dy w2, du = dh silu(g), dg = dh u s (1 + g (1 - s)), s = sigmoid(g)
//   dx = (dg | du) w13, dw13 = (dg | du)^T x, dw2 = dy^T h
//
// Sums are FP32.  Rounded to bfloat16 between the products are h and dg | du,
// which the MFMA takes.  g | u stay float32 for the gradients: as bfloat16 they
// would save 8 T I bytes of traffic (1.5 % of a step at T=4096 H=7168 I=2048) and
// double the error that dx and dw13 have beside their own rounding (0.0030 in
// place of 0.0024 of their root mean square, of which that rounding is 0.0017).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "moe_dense_big.h"
#include "moe_dense_few.h"
#include "moe_dense_host.h"
#include "moe_dense_tile.h"
#include "moe_internal.h"

namespace moe {
namespace {

using namespace dense;

constexpr Rates kRates = {{0.075, 0.12, 0.14, 0.17}, 0.8, 0.52, 1.05, 0.88, 1.55};

Plan plan_for(int m, int n, int kbs, bool k_inside) { return choose(m, n, kbs, kRates, k_inside, true, false); }

size_t parts_bytes(int m, int n, int kbs, bool k_inside) {
  const Plan p = plan_for(m, n, kbs, k_inside);
  return p.splits > 1 ? pad256((size_t)p.splits * m * n * 4) : 0;
}

// a.n: columns of the product (SwiGLU: of h).
template <int LL, int LR, int EPI, int BM>
void launch_big(Args a, int splits, hipStream_t s) {
  a.m_tiles = cdiv(a.m, BM);
  a.n_tiles = cdiv(a.n, EPI == kSwiglu ? 128 : 256);
  a.kb_per_split = cdiv(a.kbs, splits);
  const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
  const dim3 grid(tiles < 256 ? tile_grid(tiles) : 256, splits);
  if (a.k % 64 == 0)
    hipLaunchKernelGGL((big_kernel<LL, LR, BM, 256, EPI, false>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((big_kernel<LL, LR, BM, 256, EPI, true>), grid, dim3(256), 0, s, a);
}
template <int LL, int LR, int EPI>
void launch_plan(Args a, const Plan& p, hipStream_t s) {
  if (p.tn == 256)
    return p.tm == 256 ? launch_big<LL, LR, EPI, 256>(a, p.splits, s) : launch_big<LL, LR, EPI, 128>(a, p.splits, s);
  a.m_tiles = cdiv(a.m, 128);
  a.n_tiles = cdiv(a.n, EPI == kSwiglu ? 64 : 128);
  a.kb_per_split = p.splits > 1 ? cdiv(a.kbs, p.splits) : a.kbs;
  launch_tile<false, LL, LR, EPI>(a, p.splits, s);
}

// A product of L (K inside) and R, whose result has n columns, into EPI (SwiGLU:
// h has half of them).
template <int LR, int EPI>
void product(Args a, int n, float* parts, hipStream_t s) {
  const Plan p = plan_for(a.m, n, a.kbs, LR == kKin);
  if constexpr (LR == kKin) {
    if (p.tm == 0) return launch_few<kBf16, EPI>(a, s);
  }
  if (p.splits == 1) return launch_plan<kKin, LR, EPI>(a, p, s);
  Args b = a;
  b.n = b.pitch = n;
  b.outf = parts;
  launch_plan<kKin, LR, kPart>(b, p, s);
  launch_join<EPI>(a, parts, p.splits, n, s);
}

// A weight gradient: K (the tokens) outside both operands; without tokens zero.
template <int EPI>
void gradient(const Args& a, hipStream_t s) {
  const Plan p = a.kbs == 0 ? Plan{128, 128, 1} : choose(a.m, a.n, a.kbs, kRates, false, false, false);
  launch_plan<kKout, kKout, EPI>(a, p, s);
}

moe_status_t check_sizes(int32_t m, int32_t hidden, int32_t inter) {
  if (m < 0 || hidden <= 0 || inter <= 0)
    return fail(MOE_ERR_INVALID_ARG, "num_tokens %d, hidden %d, intermediate %d", m, hidden, inter);
  if (hidden % 8 || inter % 8 || hidden > 65536 || inter > 65536)
    return fail(MOE_ERR_UNSUPPORTED, "hidden (%d) and intermediate (%d) must be multiples of 8, at most 65536", hidden,
                inter);
  return MOE_OK;
}
moe_status_t check_rows(const char* name, const void* p, int64_t stride, int64_t rows, int64_t cols) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "%s must be non-NULL", name);
  if ((uintptr_t)p & 15) return fail(MOE_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (rows > 1 && (stride < cols || stride % 8 || stride > kMaxStride / 2))
    return fail(MOE_ERR_INVALID_ARG, "%s_stride %lld: %lld at least, a multiple of 8, at most %lld", name,
                (long long)stride, (long long)cols, (long long)(kMaxStride / 2));
  return MOE_OK;
}

// Outputs share memory with no other area.
moe_status_t check_apart(const Area* outs, int n_outs, const Area* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i], ins[j]))
        return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(MOE_ERR_INVALID_ARG, "two outputs overlap");
  }
  return MOE_OK;
}

size_t forward_bytes(int m, int hidden, int inter) {
  return std::max(parts_bytes(m, 2 * inter, cdiv(hidden, 64), true), parts_bytes(m, hidden, cdiv(inter, 64), true));
}
// dg | du, then parts
size_t backward_bytes(int m, int hidden, int inter, size_t* first) {
  *first = pad256((size_t)m * 2 * inter * 2);
  return *first +
         std::max(parts_bytes(m, inter, cdiv(hidden, 64), false), parts_bytes(m, hidden, cdiv(2 * inter, 64), false));
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_ffn_workspace_query(int32_t num_tokens, int32_t hidden, int32_t intermediate,
                                                size_t* forward_ws_bytes, size_t* backward_ws_bytes) {
  using namespace moe;
  clear_error();
  if (!forward_ws_bytes || !backward_ws_bytes) return fail(MOE_ERR_INVALID_ARG, "ws_bytes is NULL");
  const moe_status_t st = check_sizes(num_tokens, hidden, intermediate);
  if (st != MOE_OK) return st;
  size_t first;
  *forward_ws_bytes = num_tokens == 0 ? 0 : forward_bytes(num_tokens, hidden, intermediate);
  *backward_ws_bytes = num_tokens == 0 ? 0 : backward_bytes(num_tokens, hidden, intermediate, &first);
  return MOE_OK;
}

extern "C" moe_status_t moe_ffn_forward(const void* x, int64_t x_stride, const void* w13, const void* w2,
                                        int32_t num_tokens, int32_t hidden, int32_t intermediate, void* gate_up,
                                        void* h, void* out, int64_t out_stride, void* workspace, size_t ws_bytes,
                                        void* stream) {
  using namespace moe;
  clear_error();
  const int32_t m = num_tokens;
  moe_status_t st = check_sizes(m, hidden, intermediate);
  if (st != MOE_OK) return st;
  if (m == 0) return MOE_OK;
  if ((st = check_rows("x", x, x_stride, m, hidden)) != MOE_OK) return st;
  if ((st = check_rows("out", out, out_stride, m, hidden)) != MOE_OK) return st;
  if ((st = check_rows("w13", w13, hidden, 1, hidden)) != MOE_OK) return st;
  if ((st = check_rows("w2", w2, intermediate, 1, intermediate)) != MOE_OK) return st;
  if ((st = check_rows("h", h, intermediate, 1, intermediate)) != MOE_OK) return st;
  if ((uintptr_t)gate_up & 15) return fail(MOE_ERR_INVALID_ARG, "gate_up must be 16-byte aligned");
  const int64_t weights = (int64_t)hidden * intermediate, rows = (int64_t)m * intermediate;
  const Area outs[] = {area(out, m, out_stride, hidden, 2), area(h, 1, 0, rows, 2), area(gate_up, 1, 0, 2 * rows, 4)};
  const Area ins[] = {area(x, m, x_stride, hidden, 2), area(w13, 1, 0, 2 * weights, 2), area(w2, 1, 0, weights, 2)};
  if ((st = check_apart(outs, 3, ins, 3)) != MOE_OK) return st;
  if ((st = check_workspace(workspace, ws_bytes, forward_bytes(m, hidden, intermediate))) != MOE_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Args a = {};
  a.l = static_cast<const uint8_t*>(x);
  a.l_stride = m == 1 ? (int64_t)hidden * 2 : x_stride * 2;
  a.r = static_cast<const uint8_t*>(w13);
  a.r_stride = (int64_t)hidden * 2;
  a.m = m;
  a.n = intermediate;
  a.k = hidden;
  a.kbs = cdiv(hidden, 64);
  a.out = static_cast<uint16_t*>(h);
  a.out_stride = intermediate;
  a.gu = static_cast<float*>(gate_up);
  Args b = {};
  b.l = static_cast<const uint8_t*>(h);
  b.l_stride = (int64_t)intermediate * 2;
  b.r = static_cast<const uint8_t*>(w2);
  b.r_stride = (int64_t)intermediate * 2;
  b.m = m;
  b.n = hidden;
  b.k = intermediate;
  b.kbs = cdiv(intermediate, 64);
  set_out(b, nullptr, 0, out, out_stride);
  float* parts = static_cast<float*>(workspace);
  product<kKin, kSwiglu>(a, 2 * intermediate, parts, s);
  product<kKin, kOut>(b, hidden, parts, s);
  return launched("gated ffn");
}

extern "C" moe_status_t moe_ffn_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                         const void* w13, const void* w2, const void* gate_up, const void* h,
                                         int32_t num_tokens, int32_t hidden, int32_t intermediate, void* dx,
                                         int64_t dx_stride, void* dw13, void* dw2, int32_t dw_type, int32_t accumulate,
                                         void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  clear_error();
  const int32_t m = num_tokens;
  moe_status_t st = check_sizes(m, hidden, intermediate);
  if (st != MOE_OK) return st;
  if (dw_type != MOE_TYPE_BF16 && dw_type != MOE_TYPE_F32) return fail(MOE_ERR_INVALID_ARG, "unknown dw_type %d", dw_type);
  if (accumulate != 0 && accumulate != 1) return fail(MOE_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  if (accumulate && dw_type != MOE_TYPE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "accumulate needs float32 weight gradients");
  if ((((uintptr_t)dw13 | (uintptr_t)dw2) & 15)) return fail(MOE_ERR_INVALID_ARG, "dw13 and dw2 must be 16-byte aligned");
  size_t first = 0;
  if (m > 0) {
    if ((st = check_rows("dy", dy, dy_stride, m, hidden)) != MOE_OK) return st;
    if ((dw13 && (st = check_rows("x", x, x_stride, m, hidden)) != MOE_OK)) return st;
    if (dx && (st = check_rows("dx", dx, dx_stride, m, hidden)) != MOE_OK) return st;
    if (dx && (st = check_rows("w13", w13, hidden, 1, hidden)) != MOE_OK) return st;
    if ((dx || dw13) && (st = check_rows("w2", w2, intermediate, 1, intermediate)) != MOE_OK) return st;
    if ((dx || dw13) && (st = check_rows("gate_up", gate_up, intermediate, 1, intermediate)) != MOE_OK) return st;
    if (dw2 && (st = check_rows("h", h, intermediate, 1, intermediate)) != MOE_OK) return st;
    const size_t need = dx || dw13 ? backward_bytes(m, hidden, intermediate, &first) : 0;
    if ((st = check_workspace(workspace, ws_bytes, need)) != MOE_OK) return st;
  }
  const int64_t weights = (int64_t)hidden * intermediate, rows = (int64_t)m * intermediate;
  const int size = dw_type == MOE_TYPE_F32 ? 4 : 2;
  const Area outs[] = {area(dx, m, dx_stride, hidden, 2), area(dw13, 1, 0, 2 * weights, size),
                       area(dw2, 1, 0, weights, size)};
  const Area ins[] = {area(dy, m, dy_stride, hidden, 2),  area(x, m, x_stride, hidden, 2), area(w13, 1, 0, 2 * weights, 2),
                      area(w2, 1, 0, weights, 2), area(gate_up, 1, 0, 2 * rows, 4), area(h, 1, 0, rows, 2)};
  if ((st = check_apart(outs, 3, ins, 6)) != MOE_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* dgu = static_cast<uint8_t*>(workspace);
  float* parts = reinterpret_cast<float*>(dgu + first);
  const int64_t dys = m == 1 ? hidden : dy_stride, xs = m == 1 ? hidden : x_stride;
  if (m > 0 && (dx || dw13)) {
    Args a = {};  // dh, and from it dg | du
    a.l = static_cast<const uint8_t*>(dy);
    a.l_stride = dys * 2;
    a.r = static_cast<const uint8_t*>(w2);
    a.r_stride = (int64_t)intermediate * 2;
    a.m = m;
    a.n = intermediate;
    a.k = hidden;
    a.kbs = cdiv(hidden, 64);
    a.gu = const_cast<float*>(static_cast<const float*>(gate_up));
    a.out = reinterpret_cast<uint16_t*>(dgu);
    a.out_stride = 2 * (int64_t)intermediate;
    product<kKout, kDswiglu>(a, intermediate, parts, s);
  }
  if (m > 0 && dx) {
    Args a = {};
    a.l = dgu;
    a.l_stride = (int64_t)intermediate * 4;
    a.r = static_cast<const uint8_t*>(w13);
    a.r_stride = (int64_t)hidden * 2;
    a.m = m;
    a.n = hidden;
    a.k = 2 * intermediate;
    a.kbs = cdiv(2 * intermediate, 64);
    set_out(a, nullptr, 0, dx, dx_stride);
    product<kKout, kOut>(a, hidden, parts, s);
  }
  for (int which = 0; which < 2; ++which) {  // dw13 [2 I, H], dw2 [H, I]
    void* dw = which ? dw2 : dw13;
    if (!dw) continue;
    Args a = {};
    a.l = which ? static_cast<const uint8_t*>(dy) : dgu;
    a.l_stride = which ? dys * 2 : (int64_t)intermediate * 4;
    a.r = static_cast<const uint8_t*>(which ? h : x);
    a.r_stride = which ? (int64_t)intermediate * 2 : xs * 2;
    a.m = which ? hidden : 2 * intermediate;
    a.n = which ? intermediate : hidden;
    a.k = m;
    a.kbs = cdiv(m, 64);
    a.accumulate = accumulate;
    if (dw_type == MOE_TYPE_F32) {
      a.outf = static_cast<float*>(dw);
      gradient<kOutF32>(a, s);
    } else {
      set_out(a, nullptr, 0, dw, a.n);
      gradient<kOut>(a, s);
    }
  }
  return launched("gated ffn backward");
}
