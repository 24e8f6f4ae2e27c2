// Dense products for a few tokens, where the weights' bytes are what counts: a
// workgroup takes 16 RB rows of R and all of L, its waves take the K-blocks in
// turn and hold both operands in registers, straight from memory (no LDS: no
// two waves share a weight), and their sums are joined through LDS.
//
// e4m3 products are made on the BF16 MFMA, whose operands hold every code and
// whose sums keep float32: these sizes wait for memory, and the wider product
// costs nothing.
#pragma once

#include "moe_dense_tile.h"

namespace moe {
namespace dense {

enum { kBf16 = 0, kCodes = 1, kQuant = 2 };  // L: bfloat16; e4m3 codes; float32 rows, quantised as they are read

// 8 codes -> 8 bfloat16, exact
__device__ __forceinline__ v8bf widen_fp8(uint32_t lo, uint32_t hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One lane's 32 bytes of a K-block: [at, at + 32) bytes of a row, whose last 16
// are read again past its end (trim makes those zeros).  Weights, which one
// workgroup reads once, are loaded non-temporally.
struct Line {
  u32x4 c[2];
};
template <bool NT>
__device__ __forceinline__ Line load_line(const uint8_t* row, int at, int bytes) {
  Line v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32x4* p = reinterpret_cast<const u32x4*>(row + min(at + 16 * i, bytes - 16));
    v.c[i] = NT ? __builtin_nontemporal_load(p) : *p;
  }
  return v;
}
__device__ __forceinline__ void trim(Line& v, int at, int bytes) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at + 16 * i >= bytes) v.c[i] = u32x4{0, 0, 0, 0};
}

// e4m3 codes and scale of 32 float32 values of a row, the other 96 of whose block
// the lanes l ^ 16, l ^ 32 and l ^ 48 hold.
__device__ __forceinline__ Line quant_line(const float* row, float& scale) {
  float v[32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const v4f f = reinterpret_cast<const v4f*>(row)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[4 * i + e] = f[e];
      top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
    }
  }
  top = max(top, (uint32_t)__shfl_xor((int)top, 16));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  scale = __uint_as_float(top) / kE4m3Max;
  Line r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.c[i >> 2][i & 3] = quant4(v + 4 * i, scale);
  return r;
}

// U: K-blocks in flight per wave.
template <int L, int RB, int MT, int U, int WAVES, int EPI>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(Args a) {
  constexpr bool kPair = EPI == kSwiglu || EPI == kSwigluF32, kFp8 = L != kBf16;
  static_assert(!kPair || RB == 2, "gate and up rows");
  __shared__ __attribute__((aligned(16))) v4f part[WAVES][RB][MT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, n0 = blockIdx.x * (kPair ? 16 : 16 * RB);
  const int bytes = a.k * (kFp8 ? 1 : 2);
  const uint8_t* rp[RB];
  const float* sw[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = kPair ? min(n0 + (lane & 15), a.n - 1) + b * a.n : min(n0 + 16 * b + (lane & 15), a.n - 1);
    rp[b] = a.r + row * a.r_stride;
    // a block of 16 rows lies in one scale block
    const int first = kPair ? n0 + b * a.n : min(n0 + 16 * b, a.n - 1);
    if constexpr (kFp8) sw[b] = a.rs + (int64_t)(first / 128) * a.kbs;
  }
  const uint8_t* lp[MT];
  const float* sx[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = min(t * 16 + (lane & 15), a.m - 1);
    lp[t] = a.l + m * a.l_stride;
    if constexpr (L == kCodes) sx[t] = a.ls + (int64_t)m * a.kbs;
  }
  v4f acc[RB][MT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[b][t] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int kb = wave; kb < a.kbs; kb += WAVES * U) {
    Line w[U][RB], x[U][MT];
    float fw[U][RB], fx[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kb + u * WAVES, at = k * kLine + 32 * g;
      if (u > 0 && k >= a.kbs) break;  // wave-uniform
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        w[u][b] = load_line<true>(rp[b], at, bytes);
        if constexpr (kFp8) fw[u][b] = sw[b][k];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (L != kQuant) x[u][t] = load_line<false>(lp[t], at, bytes);
        if constexpr (L == kCodes) fx[u][t] = sx[t][k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kb + u * WAVES;
      if (u > 0 && k >= a.kbs) break;
      if ((k + 1) * kLine > bytes) {  // the last K-block, cut
#pragma unroll
        for (int b = 0; b < RB; ++b) trim(w[u][b], k * kLine + 32 * g, bytes);
#pragma unroll
        for (int t = 0; t < MT; ++t) trim(x[u][t], k * kLine + 32 * g, bytes);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if constexpr (L == kQuant)
          x[u][t] = quant_line(reinterpret_cast<const float*>(lp[t]) + k * kLine + 32 * g, fx[u][t]);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if constexpr (kFp8) {
            v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  widen_fp8(w[u][b].c[s >> 1][2 * (s & 1)], w[u][b].c[s >> 1][2 * (s & 1) + 1]),
                  widen_fp8(x[u][t].c[s >> 1][2 * (s & 1)], x[u][t].c[s >> 1][2 * (s & 1) + 1]), p, 0, 0, 0);
            const float f = fw[u][b] * fx[u][t];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][t][e] = fmaf(p[e], f, acc[b][t][e]);
          } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
              acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(v8bf, w[u][b].c[s]), __builtin_bit_cast(v8bf, x[u][t].c[s]), acc[b][t], 0, 0, 0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][b][t][lane] = acc[b][t];
  __syncthreads();
  constexpr int kJobs = (kPair ? 1 : RB) * MT;  // blocks of 16 x 16 results, one wave each
  for (int job = wave; job < kJobs; job += WAVES) {
    const int b = job / MT, t = job % MT;
    const int m = t * 16 + (lane & 15), c = n0 + 16 * b + 4 * g;
    if (m >= a.m || c >= a.n) continue;
    float v[kPair ? 2 : 1][4] = {};
#pragma unroll
    for (int h = 0; h < (kPair ? 2 : 1); ++h)
      for (int w = 0; w < WAVES; ++w) {
        const v4f p = part[w][kPair ? h : b][t][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][e] += p[e];
      }
    if constexpr (EPI == kOut) {
      store_out(a, m, c, v[0]);
    } else if constexpr (EPI == kPart) {
      store_f32(a.outf + (int64_t)m * a.n + c, c, a.n, a.vec, false, v[0]);
    } else if constexpr (EPI == kSwiglu) {
      store_swiglu(a, m, c, v[0], v[1]);
    } else {
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = swiglu(v[0][e], v[1][e]);
      store_f32(a.outf + (int64_t)m * a.n + c, c, a.n, 1, false, h);
    }
  }
}

}  // namespace dense
}  // namespace moe
