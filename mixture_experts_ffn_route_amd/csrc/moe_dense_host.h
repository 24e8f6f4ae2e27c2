// Host side of the dense products: argument checks, parts of K, launches that
// moe_linear.hip and moe_ffn.hip share.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_dense_tile.h"
#include "moe_internal.h"

#ifndef MOE_WN
#define MOE_WN 4
#define MOE_WN2 4
#endif
namespace moe {
namespace dense {

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

// Parts of K for a product whose 128 x 128 tiles would leave CUs idle (two
// tiles a CU): at least 4 K-blocks each.
inline int splits_for(int m, int n, int kbs) {
  const int64_t tiles = (int64_t)cdiv(m, 128) * cdiv(n, 128);
  if (tiles >= 256) return 1;
#ifndef MOE_SLOTS
#define MOE_SLOTS 256
#endif
  int s = (int)(MOE_SLOTS / tiles);
  if (s > kbs / 4) s = kbs / 4;
  if (s > 16) s = 16;
  return s < 2 ? 1 : cdiv(kbs, cdiv(kbs, s));
}

// `a` has its tiles.  One workgroup a CU: four stages; more: two.
template <bool FP8, int LL, int LR, int BM, int BN, int EPI>
void launch_tile(const Args& a, int splits, hipStream_t s) {
  const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
  const dim3 grid(tile_grid(tiles), splits);
  if constexpr (BM + BN > 256)  // one workgroup a CU in any case
    hipLaunchKernelGGL((tile_kernel<FP8, LL, LR, BM, BN, EPI, 3, MOE_WN2>), grid, dim3(MOE_WN2 * 128), 0, s, a);
  else if (tiles * splits <= 256)
    hipLaunchKernelGGL((tile_kernel<FP8, LL, LR, BM, BN, EPI, 4, MOE_WN>), grid, dim3(MOE_WN * 128), 0, s, a);
  else
    hipLaunchKernelGGL((tile_kernel<FP8, LL, LR, BM, BN, EPI, 2, 2>), grid, dim3(256), 0, s, a);
}

template <int EPI>
void launch_join(const Args& a, const float* part, int splits, int cols, hipStream_t s) {
  const int64_t threads = (int64_t)a.m * ((a.n + 3) / 4);
  hipLaunchKernelGGL((join_kernel<EPI>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, part, splits, cols);
}

// Whether two strided areas of rows share memory, by their first and last byte.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
inline int64_t span(int64_t rows, int64_t stride, int64_t cols, int size) {
  return rows > 0 ? ((rows - 1) * stride + cols) * size : 0;
}

// Bytes from one memory line of an operand to the next: offsets in a tile stay
// within 32 bits.
constexpr int64_t kMaxStride = 1 << 21;

inline moe_status_t check_out(int32_t m, int64_t n, const void* add, int64_t add_stride, const void* out, int64_t out_stride) {
  if (!out) return fail(MOE_ERR_INVALID_ARG, "out must be non-NULL");
  if (((uintptr_t)out | (uintptr_t)add) & 1) return fail(MOE_ERR_INVALID_ARG, "add and out must be 2-byte aligned");
  if (m > 1 && (out_stride < n || (add && add_stride < n)))
    return fail(MOE_ERR_INVALID_ARG, "out_stride %lld or add_stride %lld below %lld", (long long)out_stride,
                (long long)add_stride, (long long)n);
  if (add && !(add == out && (m == 1 || add_stride == out_stride)) &&
      overlap(add, span(m, add_stride, n, 2), out, span(m, out_stride, n, 2)))
    return fail(MOE_ERR_INVALID_ARG, "add and out overlap without being the same rows");
  return MOE_OK;
}
inline moe_status_t launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : fail(MOE_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}
inline moe_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (have < need) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", have, need);
  if (need && (!ws || ((uintptr_t)ws & 255)))
    return fail(MOE_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  return MOE_OK;
}

inline void set_out(Args& a, const void* add, int64_t add_stride, void* out, int64_t out_stride) {
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.add = static_cast<const uint16_t*>(add);
  a.add_stride = add_stride;
  const bool strides = a.m == 1 || (out_stride % 4 == 0 && (!add || add_stride % 4 == 0));
  a.vec = strides && !(((uintptr_t)out | (uintptr_t)add) & 7);
}

}  // namespace dense
}  // namespace moe
