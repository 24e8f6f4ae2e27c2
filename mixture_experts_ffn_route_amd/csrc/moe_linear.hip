// The e4m3 matrix product with block scales (moe_fp8_matmul) and the shared
// expert on it (moe_ffn_fp8).
//
//   out[m, n] = bf16(sum_kb sx[m, kb] sw[n / 128, kb] sum_{k in kb} x[m, k] w[n, k] + add[m, n])
//   shared expert: g | u = x w13^T in float32, h = silu(g) u, per 128 columns of h
//   hs = max|h| / 448 and e4m3 codes, out = the product of those with w2
#include <hip/hip_runtime.h>

#include "moe_dense_big8.h"
#include "moe_dense_few.h"
#include "moe_dense_host.h"
#include "moe_dense_tile.h"
#include "moe_internal.h"

namespace moe {
namespace {

using namespace dense;

constexpr int kFewQuant = 16;  // up to here the shared expert's second product quantises h as it reads it

constexpr Rates kRates = {{0.13, 0.17, 0.19, 0.21}, 0.6, 0.80, 1.10, 1.00, 1.75};

// Up to 16 rows sums are float32's in any case: few_kernel.
Plan plan_for(int m, int n, int kbs, bool joined = false) {
  if (m <= 16) return Plan{0, 0, 1};
  return choose(m, n, kbs, kRates, true, true, joined);
}

size_t parts_bytes(int m, int n, int kbs) {
  const Plan p = plan_for(m, n, kbs);
  return p.splits > 1 ? pad256((size_t)p.splits * m * pitch_of(n) * 4) : 0;
}

template <int EPI, int BM>
void launch_big(Args a, int splits, hipStream_t s) {
  a.m_tiles = cdiv(a.m, BM);
  a.n_tiles = cdiv(a.n, EPI == kSwigluQ ? 128 : 256);
  a.kb_per_split = cdiv(a.kbs, splits);
  const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
  const dim3 grid(tiles < 256 ? tile_grid(tiles) : 256, splits), block(512);
  const bool cut = a.k % 128 != 0;
  if constexpr (EPI == kSwigluQ) {
    hipLaunchKernelGGL((big8_kernel<EPI, false, true, BM>), grid, block, 0, s, a);
  } else if (EPI == kPart || a.vec == 2) {
    if (cut)
      hipLaunchKernelGGL((big8_kernel<EPI, true, true, BM>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((big8_kernel<EPI, false, true, BM>), grid, block, 0, s, a);
  } else {
    if (cut)
      hipLaunchKernelGGL((big8_kernel<kOut, true, false, BM>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((big8_kernel<kOut, false, false, BM>), grid, block, 0, s, a);
  }
}

template <int EPI>
void launch_plan(Args a, const Plan& p, hipStream_t s) {
  if (p.tn == 256) return p.tm == 256 ? launch_big<EPI, 256>(a, p.splits, s) : launch_big<EPI, 128>(a, p.splits, s);
  a.m_tiles = cdiv(a.m, 128);
  a.n_tiles = cdiv(a.n, 128);
  a.kb_per_split = cdiv(a.kbs, p.splits);
  launch_tile<true, kKin, kKin, EPI>(a, p.splits, s);
}

void product(Args a, float* parts, hipStream_t s) {
  const Plan p = plan_for(a.m, a.n, a.kbs);
  if (p.tm == 0) return launch_few<kCodes, kOut>(a, s);
  if (p.splits == 1) return launch_plan<kOut>(a, p, s);
  Args b = a;
  b.outf = parts;
  b.pitch = pitch_of(a.n);
  launch_plan<kPart>(b, p, s);
  launch_join<kOut>(a, parts, p.splits, b.pitch, s);
}

// h of the shared expert: gate | up of `a` (a.n columns of h), quantised.  Where
// the 2 n columns of gate | up are no plan of one part on tiles of 256 rows of R
// they go through `first`, 2 n float32 a row and part.
bool fused_h(const Plan& p) { return p.tn == 256 && p.splits == 1; }
void product_h(Args a, float* first, hipStream_t s) {
  const Plan p = plan_for(a.m, 2 * a.n, a.kbs, true);
  if (fused_h(p)) return p.tm == 256 ? launch_big<kSwigluQ, 256>(a, 1, s) : launch_big<kSwigluQ, 128>(a, 1, s);
  Args b = a;
  b.n = b.pitch = 2 * a.n;
  b.outf = first;
  if (p.tm == 0)
    launch_few<kCodes, kPart>(b, s);
  else
    launch_plan<kPart>(b, p, s);
  launch_join<kSwigluQ>(a, first, p.splits, b.pitch, s);
}

moe_status_t check_rows(const char* name, const void* x, int64_t stride, int64_t rows, int64_t k) {
  if (!x) return fail(MOE_ERR_INVALID_ARG, "%s must be non-NULL", name);
  if ((uintptr_t)x & 15) return fail(MOE_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (rows > 1 && (stride < k || stride % 16 || stride > kMaxStride))
    return fail(MOE_ERR_INVALID_ARG, "%s_stride %lld: %lld at least, a multiple of 16, at most %lld", name,
                (long long)stride, (long long)k, (long long)kMaxStride);
  return MOE_OK;
}

moe_status_t check_sizes(int32_t m, int32_t n, int32_t k) {
  if (m < 0 || n <= 0 || k <= 0) return fail(MOE_ERR_INVALID_ARG, "m %d, n %d, k %d", m, n, k);
  if (k % 16 || k > 65536 || n > 262144)
    return fail(MOE_ERR_UNSUPPORTED, "k (%d) must be a multiple of 16, at most 65536; n (%d) at most 262144", k, n);
  return MOE_OK;
}
moe_status_t check_ffn(int32_t m, int32_t hidden, int32_t inter) {
  if (m < 0 || hidden <= 0 || inter <= 0)
    return fail(MOE_ERR_INVALID_ARG, "num_tokens %d, hidden %d, intermediate %d", m, hidden, inter);
  if (hidden % 128 || inter % 128 || hidden > 65536 || inter > 65536)
    return fail(MOE_ERR_UNSUPPORTED, "hidden (%d) and intermediate (%d) must be multiples of 128, at most 65536",
                hidden, inter);
  return MOE_OK;
}

// The shared expert's workspace: `first` bytes of float32 h, gate/up or parts,
// then h's codes and scales.
struct FfnLayout {
  size_t first, codes, scales;
  size_t total() const { return first + codes + scales; }
};
FfnLayout ffn_layout(int32_t m, int32_t hidden, int32_t inter) {
  FfnLayout l{0, 0, 0};
  if (m <= kFewQuant) {
    l.first = pad256((size_t)m * inter * 4);
    return l;
  }
  const Plan p = plan_for(m, 2 * inter, hidden / 128, true);
  l.first = fused_h(p) ? 0 : pad256((size_t)p.splits * m * 2 * inter * 4);
  const size_t second = parts_bytes(m, hidden, inter / 128);
  if (second > l.first) l.first = second;
  l.codes = pad256((size_t)m * inter);
  l.scales = pad256((size_t)m * (inter / 128) * 4);
  return l;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_fp8_matmul_workspace_query(int32_t m, int32_t n, int32_t k, size_t* ws_bytes) {
  moe::clear_error();
  if (!ws_bytes) return moe::fail(MOE_ERR_INVALID_ARG, "ws_bytes is NULL");
  const moe_status_t st = moe::check_sizes(m, n, k);
  if (st != MOE_OK) return st;
  *ws_bytes = m == 0 ? 0 : moe::parts_bytes(m, n, moe::cdiv(k, 128));
  return MOE_OK;
}

extern "C" moe_status_t moe_fp8_matmul(const uint8_t* x, int64_t x_stride, const float* x_scale, const uint8_t* w,
                                       int64_t w_stride, const float* w_scale, int32_t m, int32_t n, int32_t k,
                                       const void* add_bf16, int64_t add_stride, void* out_bf16, int64_t out_stride,
                                       void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  clear_error();
  moe_status_t st = check_sizes(m, n, k);
  if (st != MOE_OK) return st;
  if (m == 0) return MOE_OK;  // tensors of no rows have no address
  if ((st = check_rows("x", x, x_stride, m, k)) != MOE_OK) return st;
  if ((st = check_rows("w", w, w_stride, n, k)) != MOE_OK) return st;
  if (!x_scale || !w_scale || (((uintptr_t)x_scale | (uintptr_t)w_scale) & 3))
    return fail(MOE_ERR_INVALID_ARG, "x_scale and w_scale must be non-NULL and 4-byte aligned");
  if ((st = check_out(m, n, add_bf16, add_stride, out_bf16, out_stride)) != MOE_OK) return st;
  const int64_t kbs = cdiv(k, 128);
  const Area to = area(out_bf16, m, out_stride, n, 2);
  if (overlap(to, area(x, m, x_stride, k, 1)) || overlap(to, area(w, n, w_stride, k, 1)) ||
      overlap(to, area(x_scale, 1, 0, m * kbs, 4)) || overlap(to, area(w_scale, 1, 0, cdiv(n, 128) * kbs, 4)))
    return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
  if ((st = check_workspace(workspace, ws_bytes, parts_bytes(m, n, (int)kbs))) != MOE_OK) return st;
  Args a = {};
  a.l = x;
  a.l_stride = m == 1 ? k : x_stride;
  a.r = w;
  a.r_stride = n == 1 ? k : w_stride;
  a.ls = x_scale;
  a.rs = w_scale;
  a.m = m;
  a.n = n;
  a.k = k;
  a.kbs = (int32_t)kbs;
  set_out(a, add_bf16, add_stride, out_bf16, out_stride);
  product(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  return launched("fp8 matmul");
}

extern "C" moe_status_t moe_ffn_fp8_workspace_query(int32_t num_tokens, int32_t hidden, int32_t intermediate,
                                                    size_t* ws_bytes) {
  moe::clear_error();
  if (!ws_bytes) return moe::fail(MOE_ERR_INVALID_ARG, "ws_bytes is NULL");
  const moe_status_t st = moe::check_ffn(num_tokens, hidden, intermediate);
  if (st != MOE_OK) return st;
  *ws_bytes = num_tokens == 0 ? 0 : moe::ffn_layout(num_tokens, hidden, intermediate).total();
  return MOE_OK;
}

extern "C" moe_status_t moe_ffn_fp8(const uint8_t* x, int64_t x_stride, const float* x_scale, const uint8_t* w13,
                                    const float* w13_scale, const uint8_t* w2, const float* w2_scale,
                                    int32_t num_tokens, int32_t hidden, int32_t intermediate, const void* add_bf16,
                                    int64_t add_stride, void* out_bf16, int64_t out_stride, void* workspace,
                                    size_t ws_bytes, void* stream) {
  using namespace moe;
  clear_error();
  const int32_t m = num_tokens;
  moe_status_t st = check_ffn(m, hidden, intermediate);
  if (st != MOE_OK) return st;
  if (m == 0) return MOE_OK;
  if ((st = check_rows("x", x, x_stride, m, hidden)) != MOE_OK) return st;
  if ((st = check_rows("w13", w13, hidden, 2 * intermediate, hidden)) != MOE_OK) return st;
  if ((st = check_rows("w2", w2, intermediate, hidden, intermediate)) != MOE_OK) return st;
  if (!x_scale || !w13_scale || !w2_scale || (((uintptr_t)x_scale | (uintptr_t)w13_scale | (uintptr_t)w2_scale) & 3))
    return fail(MOE_ERR_INVALID_ARG, "the scales must be non-NULL and 4-byte aligned");
  if ((st = check_out(m, hidden, add_bf16, add_stride, out_bf16, out_stride)) != MOE_OK) return st;
  const int64_t weights = (int64_t)hidden * intermediate;
  const Area to = area(out_bf16, m, out_stride, hidden, 2);
  if (overlap(to, area(x, m, x_stride, hidden, 1)) || overlap(to, area(w13, 1, 0, 2 * weights, 1)) ||
      overlap(to, area(w2, 1, 0, weights, 1)) || overlap(to, area(x_scale, 1, 0, (int64_t)m * (hidden / 128), 4)) ||
      overlap(to, area(w13_scale, 1, 0, weights / 8192, 4)) || overlap(to, area(w2_scale, 1, 0, weights / 16384, 4)))
    return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
  const FfnLayout lay = ffn_layout(m, hidden, intermediate);
  if ((st = check_workspace(workspace, ws_bytes, lay.total())) != MOE_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* first = reinterpret_cast<float*>(ws);
  Args a = {};
  a.l = x;
  a.l_stride = m == 1 ? hidden : x_stride;
  a.r = w13;
  a.r_stride = hidden;
  a.ls = x_scale;
  a.rs = w13_scale;
  a.m = m;
  a.n = intermediate;
  a.k = hidden;
  a.kbs = hidden / 128;
  a.hq = ws + lay.first;
  a.hs = reinterpret_cast<float*>(ws + lay.first + lay.codes);
  Args b = a;  // the second product
  b.l = a.hq;
  b.l_stride = intermediate;
  b.ls = a.hs;
  b.r = w2;
  b.r_stride = intermediate;
  b.rs = w2_scale;
  b.n = hidden;
  b.k = intermediate;
  b.kbs = intermediate / 128;
  set_out(b, add_bf16, add_stride, out_bf16, out_stride);
  if (m <= kFewQuant) {
    a.outf = first;
    launch_few<kCodes, kSwigluF32, 1>(a, s);
    b.l = ws;
    b.l_stride = (int64_t)intermediate * 4;
    launch_few<kQuant, kOut, 1>(b, s);
    return launched("shared expert");
  }
  product_h(a, first, s);
  product(b, first, s);
  return launched("shared expert");
}
