// Host side of the dense products: argument checks, parts of K, launches that
// moe_linear.hip and moe_ffn.hip share.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_dense_tile.h"
#include "moe_internal.h"

namespace moe {
namespace dense {

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline size_t pad256(size_t v) { return (v + 255) / 256 * 256; }

inline int pitch_of(int n) { return (n + 3) / 4 * 4; }

// How a product is made: by few_kernel, or on tiles of tm rows of L and tn of R (128
// x 128: tile_kernel, else the large tiles' kernel), K in `splits` parts that
// join_kernel sums.
struct Plan {
  int tm, tn, splits;  // tm 0: few_kernel
};

// us a K-block (128 bytes of K) takes in a workgroup of each form, as measured:
// few_kernel with 1..4 blocks of L rows and 32 columns, and its part of that with
// 16; 128 x 128 tiles, one and two workgroups a CU; 128 x 256; 256 x 256.
struct Rates {
  double few[4], narrow, tile, tile2, wide, large;
};

// The form that is estimated to be fastest, from the sizes alone: rounds of
// workgroups over the CUs (tiles: over the 32 of the XCD with the most), each as many K-blocks long as a part of K has, 4
// us around them (few_kernel 2.8), and with parts of K a join of 3 us and their
// bytes at 6.5 TB/s.  Measured at 16 m from 17 to 4096 for 8 products from N=576
// K=7168 to N=K=7168 and the blocks of H=7168 I=2048 and H=2048 I=768, with few_kernel
// and each tile with K in 1, 2, 4 and 8 parts forced in turn, the choice takes at most
// 1.20 times the fastest form's time (shared expert H=2048 I=768 T=512 24.1 us, 20.0
// with few_kernel), 1.007 times in the mean.
// few: whether few_kernel can make it; split: whether K may be split; joined: a
// join follows in any case but that of one part on tiles of 256 rows of R.
inline Plan choose(int m, int n, int kbs, const Rates& r, bool few, bool split, bool joined) {
  auto rounds = [](int64_t groups, int64_t slots) { return (double)((groups + slots - 1) / slots); };
  auto join = [&](int parts) { return 3.0 + (double)parts * m * n * 8e-6 / 6.5; };
  Plan best{128, 128, 1};
  double least = 1e30;
  auto offer = [&](double us, const Plan& p) {
    if (us < least) {
      least = us;
      best = p;
    }
  };
  if (few) {
    const int blocks = cdiv(m, 16), mt = few_blocks(blocks, cdiv(n, 32)), parts = cdiv(blocks, mt);
    const int64_t groups = (int64_t)cdiv(n, 32) * parts;
    const double us = few_narrow(groups, mt) ? 2.8 + rounds(2 * groups, 256) * (kbs * r.few[mt - 1] * r.narrow + 0.4)
                                   : 2.8 + rounds(groups, 256) * (kbs * r.few[mt - 1] + 0.4);
    if (parts <= 65535)  // the grid's second dimension
      offer(us + (joined ? join(1) : 0.0), Plan{0, 0, 1});
  }
  for (int s = 1; s <= 16 && (s == 1 || (split && kbs >= 2 * s)); ++s) {
    const int kb = cdiv(kbs, s);
    if (cdiv(kbs, kb) != s) continue;  // fewer parts of the same length
    auto per_xcd = [&](int tm, int tn) { return cdiv((int64_t)cdiv(m, tm) * cdiv(n, tn), 8) * (int64_t)s; };
    const int64_t t = per_xcd(128, 128);
    const double tail = s > 1 ? join(s) : 0.0, fused = joined && s == 1 ? join(1) : 0.0;
    offer(4.0 + (t <= 32 ? kb * r.tile : rounds(t, 64) * kb * r.tile2) + tail + fused, Plan{128, 128, s});
    offer(4.0 + rounds(per_xcd(128, 256), 32) * kb * r.wide + tail, Plan{128, 256, s});
    offer(4.0 + rounds(per_xcd(256, 256), 32) * kb * r.large + tail, Plan{256, 256, s});
  }
  return best;
}

// `a` has its tiles.  One workgroup a CU: four stages; more: two.
template <bool FP8, int LL, int LR, int EPI>
void launch_tile(const Args& a, int splits, hipStream_t s) {
  const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
  const dim3 grid(tile_grid(tiles), splits);
  if ((tiles + 7) / 8 * splits <= 32)
    hipLaunchKernelGGL((tile_kernel<FP8, LL, LR, EPI, 4, 4>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((tile_kernel<FP8, LL, LR, EPI, 2, 2>), grid, dim3(256), 0, s, a);
}

template <int EPI>
void launch_join(const Args& a, const float* part, int splits, int pitch, hipStream_t s) {
  const int64_t threads = (int64_t)a.m * ((a.n + 3) / 4);
  hipLaunchKernelGGL((join_kernel<EPI>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, part, splits, pitch);
}

// Rows of `width` bytes, `stride` bytes apart.
struct Area {
  const void* p;
  int64_t rows, stride, width;
};
inline Area area(const void* p, int64_t rows, int64_t stride, int64_t cols, int size) {
  return Area{p, rows, rows > 1 ? stride * size : cols * size, cols * size};
}
// Whether two areas may share memory: by their first and last bytes, but not
// columns of one buffer beside each other.
inline bool overlap(const Area& a, const Area& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y + (uintptr_t)((b.rows - 1) * b.stride + b.width) || y >= x + (uintptr_t)((a.rows - 1) * a.stride + a.width))
    return false;
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
    const int64_t s = a.stride, d = (((int64_t)(y - x)) % s + s) % s;  // b's columns from a's first
    return !(d >= a.width && d + b.width <= s);
  }
  return true;
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
      overlap(area(add, m, add_stride, n, 2), area(out, m, out_stride, n, 2)))
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
  auto pieces = [&](int values) {
    const bool strides = a.m == 1 || (out_stride % values == 0 && (!add || add_stride % values == 0));
    return strides && !(((uintptr_t)out | (uintptr_t)add) & (2 * values - 1));
  };
  a.vec = pieces(8) && a.n % 8 == 0 ? 2 : pieces(4) ? 1 : 0;
}

}  // namespace dense
}  // namespace moe
