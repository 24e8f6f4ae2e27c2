// Residual addition, RMS norm and e4m3 quantisation of activation rows, in
// one pass over them: what a decoder layer does between its attention and
// this layer, with the output in the form moe_stage_inputs and
// moe_layer_decode take.
//
//   s = x + residual                       (FP32)
//   y = s * rsqrt(mean(s^2) + eps) * weight
//   per 128 columns: scale = max|y| / 448, code = e4m3 RNE_sat(y / scale)
//
// Rounding happens once per output: the new residual is s, the BF16 row is y
// and the codes are y / scale, each from the FP32 values (the codes are not
// taken from the rounded BF16 row).  The sum of squares is kept in FP64, so
// that no finite row overflows or vanishes in it; everything else is FP32.
//
// HBM bounds it.  One workgroup per row at a time; a thread owns C chunks of
// 8 consecutive columns (16 bytes of BF16) and keeps s in registers between
// the sum and the output, so every input is read once.  A 128-column block is
// one chunk of 16 consecutive lanes, a DPP row, so the block maximum never
// leaves the wave.  The outputs are stored non-temporally: T=8192 H=2048 24.2
// us against 30.8 with plain stores of codes and BF16 rows, T=4096 H=7168
// 48.3 against 50.8 (before the quotients came from p: 2 to 3 % more now).  At
// T=4096 H=7168 with a BF16 residual and every output a call moves 265 MB in 50.6
// to 51.1 us, 5.2 TB/s (a 2 GiB copy: 4.9); T=32768 without the BF16 rows 1652 MB
// in 314 to 322 us, 5.2 TB/s; T=1 takes 4.2 us.
#include <hip/hip_runtime.h>
#include <math.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_quant_dev.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxWaves = 16;

struct NormArgs {
  const uint16_t* x;
  int64_t x_stride;
  const void* residual;  // null: none
  int64_t residual_stride;
  const void* weight;
  int32_t tokens, hidden;
  float eps;
  uint8_t* codes;
  float* scales;
  uint16_t* y;         // null: not wanted
  void* residual_out;  // null: not wanted
  int64_t residual_out_stride;
};

__device__ __forceinline__ void load8_bf16(const uint16_t* p, float v[8]) {
  const u32x4 r = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(r[i] & 0xffffu);
    v[2 * i + 1] = bf16_to_f32(r[i] >> 16);
  }
}
__device__ __forceinline__ void load8_f32(const float* p, float v[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float v[8]) {
  if constexpr (F32)
    load8_f32(static_cast<const float*>(base) + at, v);
  else
    load8_bf16(static_cast<const uint16_t*>(base) + at, v);
}
template <typename T>
__device__ __forceinline__ void store_nt(void* p, T v) {
  __builtin_nontemporal_store(v, static_cast<T*>(p));
}
__device__ __forceinline__ u32x4 pack8_bf16(const float v[8]) {
  return u32x4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
}

// The row's factor cancels in a code's quotient: y / scale = 448 p / max p with
// p = s w, taken from p 2^k (k: the factor's exponent, so that p is near y),
// where sums and products of short mantissas are exact and a quotient in the
// middle of two codes comes out there (one in 3000 of BF16 rows).
//
// With an FP32 residual the codes are those of 64-bit arithmetic: a quotient
// next to such a middle, where the roundings of p and max p would decide, is
// decided exactly.
//
// from_middle: how far quotient q lies from that middle, in units of its last
// place from kNear units below it on.  Codes are 2^20 units apart (from 2^-6
// up; those below are not looked at: a step is 2^-9 there, beside a maximum of
// 448).  A quotient carries six roundings at most (sum and product of its p and
// of the maximum, 7/8 p, its own): six half steps, 3 to 6 units.
constexpr uint32_t kNear = 12;
__device__ __forceinline__ uint32_t from_middle(float q) {
  return (__float_as_uint(q) - 0x80000u + kNear) & 0xfffffu;
}

// R: 0 no residual, 1 BF16, 2 FP32.  WF32: FP32 weight.
template <int C, int R, bool WF32>
__global__ __launch_bounds__(1024) void rms_norm_quant_kernel(NormArgs a) {
  __shared__ double part[2][kMaxWaves];
  const int nt = blockDim.x, tid = threadIdx.x;
  const int wave = tid >> 6, waves = nt >> 6;
  const int chunks = a.hidden >> 3;
  float w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = c * nt + tid;
    if (j < chunks) load8<WF32>(a.weight, (int64_t)j * 8, w[c]);
  }
  int parity = 0;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x, parity ^= 1) {
    float s[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * nt + tid;
      if (j < chunks) {
        load8_bf16(a.x + t * a.x_stride + j * 8, s[c]);
        if constexpr (R != 0) {
          float r[8];
          load8<R == 2>(a.residual, t * a.residual_stride + j * 8, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[c][i] += r[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[c][i] = 0.0f;
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)s[c][i], (double)s[c][i], sum);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
    if ((tid & 63) == 0) part[parity][wave] = sum;
    __syncthreads();  // the other parity's sums of the last row may still be read
    sum = 0.0;
    for (int i = 0; i < waves; ++i) sum += part[parity][i];
    // 1 / rms = near * rest: a power of two (within float32's range) and the rest
    const double factor = 1.0 / sqrt(sum / a.hidden + (double)a.eps);
    const int k = !(factor >= 0x1p-126) ? -126 : factor >= 0x1p127 ? 127 : ilogb(factor);
    const float near = __uint_as_float((uint32_t)(k + 127) << 23), rest = (float)ldexp(factor, -k);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * nt + tid;
      if (j >= chunks) continue;  // whole DPP rows: chunks and nt are multiples of 16
      float p[8], y[8];
      uint32_t m = 0;  // maximum of |p| as bits: a NaN is larger than every number
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = s[c][i] * near * w[c][i];
        y[i] = p[i] * rest;
        m = max(m, __float_as_uint(p[i]) & 0x7fffffffu);
      }
      // residual_out may be the residual and the BF16 rows x, which are read
      // again below where the sums are not exact
      auto store_rows = [&]() {
        if constexpr (R != 0) {
          if (a.residual_out) {
            if constexpr (R == 2) {
              float* d = static_cast<float*>(a.residual_out) + t * a.residual_out_stride + j * 8;
              store_nt(d, f32x4{s[c][0], s[c][1], s[c][2], s[c][3]});
              store_nt(d + 4, f32x4{s[c][4], s[c][5], s[c][6], s[c][7]});
            } else {
              store_nt(static_cast<uint16_t*>(a.residual_out) + t * a.residual_out_stride + j * 8, pack8_bf16(s[c]));
            }
          }
        }
        if (a.y) store_nt(a.y + t * a.hidden + j * 8, pack8_bf16(y));
      };
      if constexpr (R != 2) store_rows();
      if (a.codes) {
        const float top = __uint_as_float(row16_max(m));
        const float scale = top * rest / kE4m3Max;
        q_u32x2 codes = codes_without_scale(scale);
        const bool scaled = scale != 0.0f && isfinite(scale);
        // p / 512 against max p / 512 * 7 / 8, both exact; blocks of the smallest
        // scales, whose own rounding counts, by their scale
        const bool small = scale < 0x1p-100f;
        float q[8];
        if (scaled) {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = small ? y[i] : 0.875f * p[i];
          quotients8(q, small ? scale : 0x1p-9f * top, q);
        }
        if constexpr (R == 2) {
          uint32_t closest = ~0u;
          if (scaled && !small) {
#pragma unroll
            for (int i = 0; i < 8; ++i) closest = min(closest, from_middle(q[i]));
          }
          if (__ballot(closest <= 2 * kNear)) {
            // Next to a tie of two codes 7/8 |p| is compared with middle / 512 times
            // max|p|, all with the rests of their sums and products, and the
            // quotient becomes the middle or a neighbour of it.
            float low[8];  // |p| is low more
            float x[8], r[8];
            load8_bf16(a.x + t * a.x_stride + j * 8, x);
            load8<true>(a.residual, t * a.residual_stride + j * 8, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float of_x = s[c][i] - r[i], lost = (x[i] - of_x) + (r[i] - (s[c][i] - of_x));
              low[i] = fmaf(fabsf(s[c][i] * near), fabsf(w[c][i]), -fabsf(p[i])) +
                       copysignf(1.0f, s[c][i]) * (lost * near) * fabsf(w[c][i]);
            }
            // The maximum's: that of the largest |p| + low, whose |p| may be a
            // unit below the largest.
            float top_low = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) top_low = fmaxf(top_low, (fabsf(p[i]) - top) + low[i]);
#pragma unroll
            for (int k = 1; k < 16; k <<= 1) top_low = fmaxf(top_low, __shfl_xor(top_low, k, 16));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (!scaled || small || from_middle(q[i]) > 2 * kNear) continue;
              const float middle = __uint_as_float((__float_as_uint(fabsf(q[i])) & 0xfff00000u) | 0x80000u);
              const float part = 0x1p-9f * middle, h = part * top;
              const float d = fmaf(0.875f, fabsf(p[i]), -h) - fmaf(part, top, -h) +
                              fmaf(0.875f, low[i], -part * top_low);
              if (fabsf(q[i]) >= 0x1p-6f)
                q[i] = copysignf(__uint_as_float(__float_as_uint(middle) + (d > 0.0f ? 1 : d < 0.0f ? -1 : 0)), q[i]);
            }
          }
        }
        if (scaled) codes = codes8(q);
        store_nt(a.codes + t * a.hidden + j * 8, codes);
        if ((tid & 15) == 0) a.scales[t * (a.hidden >> 7) + (j >> 4)] = scale;
      }
      if constexpr (R == 2) store_rows();
    }
  }
}

template <int C>
int launch_c(const NormArgs& a, int r, bool wf32, dim3 grid, dim3 block, hipStream_t s) {
#define MOE_NORM(R)                                                                             \
  if (wf32)                                                                                     \
    hipLaunchKernelGGL((rms_norm_quant_kernel<C, R, true>), grid, block, 0, s, a);              \
  else                                                                                          \
    hipLaunchKernelGGL((rms_norm_quant_kernel<C, R, false>), grid, block, 0, s, a)
  if (r == 0) {
    MOE_NORM(0);
  } else if (r == 1) {
    MOE_NORM(1);
  } else {
    MOE_NORM(2);
  }
#undef MOE_NORM
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_norm(const NormArgs& a, int r, bool wf32, hipStream_t s) {
  const int chunks = a.hidden / 8;
  // Chunks per thread: two from H = 4096 up, one below.  With one, a row of
  // H = 7168 takes 14 waves, and two such workgroups leave a CU 4 wave slots
  // idle (T=4096 57.8 us against 48.3; T=32768 399 against 295); with two, a
  // row of H = 2048 has 2 waves (T=512 4.5 us against 4.0, T=8192 24.2
  // against 24.6).  Four chunks were slower at both (51.2, 309; 5.4, 25.9).
  const int c = chunks > 512 ? 2 : 1;
  const int nt = ((chunks + c - 1) / c + 63) / 64 * 64;
  const int grid = a.tokens < 65536 ? a.tokens : 65536;
  return c == 1 ? launch_c<1>(a, r, wf32, dim3(grid), dim3(nt), s) : launch_c<2>(a, r, wf32, dim3(grid), dim3(nt), s);
}

bool valid_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_rms_norm_quant(const moe_norm_config_t* cfg, const void* x, int64_t x_stride,
                                           const void* residual, int64_t residual_stride, const void* weight,
                                           int32_t num_tokens, uint8_t* codes, float* scales, void* y_bf16,
                                           void* residual_out, int64_t residual_out_stride, void* stream) {
  moe::clear_error();
  if (!cfg) return moe::fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
  const int32_t H = cfg->hidden;
  if (H <= 0) return moe::fail(MOE_ERR_INVALID_ARG, "hidden (%d) must be positive", H);
  if (H % 128 || H > 16384)
    return moe::fail(MOE_ERR_UNSUPPORTED, "hidden (%d) must be a multiple of 128, at most 16384", H);
  if (!(cfg->eps >= 0.0f) || !isfinite(cfg->eps))
    return moe::fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!moe::valid_type(cfg->residual_type) || !moe::valid_type(cfg->weight_type))
    return moe::fail(MOE_ERR_INVALID_ARG, "unknown residual_type %d or weight_type %d", cfg->residual_type,
                     cfg->weight_type);
  if (num_tokens < 0) return moe::fail(MOE_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return MOE_OK;  // tensors of no rows have no address
  if (!codes != !scales) return moe::fail(MOE_ERR_INVALID_ARG, "codes and scales come together");
  if (!codes && !y_bf16) return moe::fail(MOE_ERR_INVALID_ARG, "neither codes nor y_bf16 is wanted");
  if (residual_out && !residual) return moe::fail(MOE_ERR_INVALID_ARG, "residual_out without a residual");
  if (!x || !weight) return moe::fail(MOE_ERR_INVALID_ARG, "x and weight must be non-NULL");
  if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)y_bf16 | (uintptr_t)residual_out) & 15)
    return moe::fail(MOE_ERR_INVALID_ARG, "x, residual, weight, y and residual_out must be 16-byte aligned");
  if (((uintptr_t)codes & 7) || ((uintptr_t)scales & 3))
    return moe::fail(MOE_ERR_INVALID_ARG, "codes must be 8-byte and scales 4-byte aligned");
  // rows of 16-byte pieces that do not overlap (a single row needs no stride)
  const int per16 = cfg->residual_type == MOE_TYPE_F32 ? 4 : 8;
  if (num_tokens > 1) {
    if (x_stride < H || x_stride % 8) return moe::fail(MOE_ERR_INVALID_ARG, "x_stride %lld", (long long)x_stride);
    if (residual && (residual_stride < H || residual_stride % per16))
      return moe::fail(MOE_ERR_INVALID_ARG, "residual_stride %lld", (long long)residual_stride);
    if (residual_out && (residual_out_stride < H || residual_out_stride % per16))
      return moe::fail(MOE_ERR_INVALID_ARG, "residual_out_stride %lld", (long long)residual_out_stride);
    // an output over its input: row over row, which the row's workgroup has read
    if (residual_out && residual_out == residual && residual_out_stride != residual_stride)
      return moe::fail(MOE_ERR_INVALID_ARG, "residual_out over residual with strides %lld and %lld",
                       (long long)residual_out_stride, (long long)residual_stride);
    if (y_bf16 && y_bf16 == x && x_stride != H)
      return moe::fail(MOE_ERR_INVALID_ARG, "y over x with x_stride %lld", (long long)x_stride);
  }
  moe::NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.weight = weight;
  a.tokens = num_tokens;
  a.hidden = H;
  a.eps = cfg->eps;
  a.codes = codes;
  a.scales = scales;
  a.y = static_cast<uint16_t*>(y_bf16);
  a.residual_out = residual_out;
  a.residual_out_stride = residual_out_stride;
  const int r = !residual ? 0 : (cfg->residual_type == MOE_TYPE_F32 ? 2 : 1);
  if (moe::launch_norm(a, r, cfg->weight_type == MOE_TYPE_F32, static_cast<hipStream_t>(stream)) != 0) {
    const hipError_t e = hipGetLastError();
    return moe::fail(MOE_ERR_HIP, "norm launch: %s", hipGetErrorString(e));
  }
  return MOE_OK;
}
