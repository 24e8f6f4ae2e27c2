// Dense products for a few tokens, where the weights' bytes are what counts: a
// workgroup takes 16 RB rows of R and up to 64 of L, its waves take the K-blocks in
// turn, each through a ring of its own in LDS, filled by DMA (no two waves share a
// weight, so they never wait for each other), and their sums are joined through
// LDS.
//
// Memory bounds it for one row: N=K=7168 (51 MB of e4m3 weights) 10.2 us with the
// weights in no cache, 5.0 TB/s (a 2 GiB copy: 4.8); the BF16 block T=1 H=7168
// I=2048 (88 MB) 17.9 us in two launches.  Those are with non-temporal loads of
// the weights; with plain ones 11.7 and 19.3, though weights that stay in the last
// cache then come faster (N=7168 K=2048 3.9 us against 4.5).  With 64 rows, whose
// 12 KB a K-block the CUs load at 17 bytes a clock, 18 us.  Fragments loaded
// straight into registers, 16 bytes of each of 16 rows four times a line, took
// 14.5 us for one row and 47.8 for 64: the DMA asks for whole lines.
#pragma once

#include "moe_dense_tile.h"

namespace moe {
namespace dense {

enum { kBf16 = 0, kCodes = 1, kQuant = 2 };  // L: bfloat16; e4m3 codes; float32 rows, quantised as they are read (up to 16)

// 8 codes -> 8 bfloat16, exact
__device__ __forceinline__ v8bf widen_fp8(uint32_t lo, uint32_t hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// RB: blocks of 16 rows of R (SwiGLU: 2, gate rows and up rows, or 1, 8 of each);
// MT: blocks of 16 rows of L, blockIdx.y the part of L.  DEPTH: K-blocks in a
// wave's own ring in LDS.
//
// With one block of L rows an e4m3 product is made on the BF16 MFMA, whose
// operands hold every code and whose sums keep float32: the conversions are
// nothing beside the weights' bytes.  With more it is made on the FP8 MFMA.
template <int L, int RB, int MT, int WAVES, int DEPTH, int EPI>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(Args a) {
  constexpr bool kPair = EPI == kSwiglu || EPI == kSwigluF32, kFp8 = L != kBf16, kHalves = kPair && RB == 1;
  static_assert(!kPair || RB <= 2, "gate and up rows");
  constexpr int COLS = kHalves ? 8 : kPair ? 16 : 16 * RB;  // of the result, per workgroup
  constexpr int SLOT = (RB + MT) * 2048 + (kFp8 ? 256 : 0);
  constexpr int LT = L == kQuant ? 0 : MT;                  // blocks of L that DMA fetches
  constexpr int LOADS = 2 * (RB + LT) + (L == kCodes ? 1 : 0);
  constexpr int RING = WAVES * DEPTH * SLOT, PART = WAVES * RB * MT * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > PART ? RING : PART];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, n0 = blockIdx.x * COLS, m0 = blockIdx.y * 16 * MT;
  const int bytes = a.k * (kFp8 ? 1 : 2);
  lds_u8* ring = (lds_u8*)lds + wave * DEPTH * SLOT;

  // DMA instruction h of a block fetches 8 rows; this lane's row and chunk
  const int dr = lane >> 3;
  uint32_t roff[RB][2], loff[LT ? LT : 1][2], soff = 0;
  auto chunk = [&](int h) { return ((lane & 7) ^ swz(8 * h + dr)) * 16; };
  // row r of the workgroup's block b of R
  auto r_row = [&](int b, int r) {
    return kHalves ? min(n0 + (r & 7), a.n - 1) + (r >> 3) * a.n
                   : kPair ? min(n0 + r, a.n - 1) + b * a.n : min(n0 + 16 * b + r, a.n - 1);
  };
  const uint8_t* rbase[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = r_row(b, 8 * h);  // wave-uniform
      rbase[b][h] = a.r + first * a.r_stride;
      roff[b][h] = __umul24(r_row(b, 8 * h + dr) - first, (uint32_t)a.r_stride) + chunk(h);
    }
  const uint8_t* lbase = a.l + m0 * a.l_stride;
  const int rows = min(a.m - m0, 16 * MT);
#pragma unroll
  for (int t = 0; t < LT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      loff[t][h] = __umul24(min(16 * t + 8 * h + dr, rows - 1), (uint32_t)a.l_stride) + chunk(h);
  if constexpr (L == kCodes) soff = __umul24(min(lane, rows - 1), (uint32_t)a.kbs) * 4u;
  const bool once = gridDim.y == 1;  // no other workgroup reads these weights
  auto issue = [&](int kb, int slot) {
    lds_u8* to = ring + slot * SLOT;
    const int64_t at = (int64_t)kb * kLine;
    if ((kb + 1) * kLine <= bytes) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (once)
            dma16_nt(rbase[b][h] + at, roff[b][h], to + b * 2048 + h * 1024);
          else
            dma16(rbase[b][h] + at, roff[b][h], to + b * 2048 + h * 1024);
        }
#pragma unroll
      for (int t = 0; t < LT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) dma16(lbase + at, loff[t][h], to + (RB + t) * 2048 + h * 1024);
    } else {  // the last K-block, cut: zeros beyond K
      auto from = [&](const uint8_t* base, uint32_t off, int h) {
        return chunk(h) < bytes - kb * kLine ? base + at + off : (const uint8_t*)&kZeros;
      };
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) dma16_at(from(rbase[b][h], roff[b][h], h), to + b * 2048 + h * 1024);
#pragma unroll
      for (int t = 0; t < LT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) dma16_at(from(lbase, loff[t][h], h), to + (RB + t) * 2048 + h * 1024);
    }
    if constexpr (L == kCodes) dma4(a.ls + (int64_t)m0 * a.kbs + kb, soff, to + (RB + MT) * 2048);
  };

  // The weight scales of each block of R, which lies in one scale block (kHalves:
  // rows 0-7 and 8-15 in two; a lane's results are rows 4 g and up).
  const float *sw[RB], *sw_up = nullptr;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int first = kPair ? n0 + b * a.n : min(n0 + 16 * b, a.n - 1);
    sw[b] = kFp8 ? a.rs + (int64_t)(first / 128) * a.kbs : nullptr;
  }
  if constexpr (kFp8 && kHalves) sw_up = a.rs + (int64_t)((n0 + a.n) / 128) * a.kbs;
  v4f acc[RB][MT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[b][t] = v4f{0.f, 0.f, 0.f, 0.f};

  const int count = wave < a.kbs ? (a.kbs - wave + WAVES - 1) / WAVES : 0;  // this wave's K-blocks
#pragma unroll
  for (int i = 0; i < DEPTH; ++i)
    if (i < count) issue(wave + i * WAVES, i);
  int slot = 0;
  for (int i = 0; i < count; ++i) {
    const int kb = wave + i * WAVES;
    if constexpr (L == kQuant) {
      // this K-block of L's rows as codes and scales into the slot: four rows at a
      // time, 16 lanes and 8 columns a lane each
      lds_u8* to = ring + slot * SLOT + RB * 2048;
      const int c = lane & 15;
      for (int r0 = 0; r0 < rows; r0 += 4) {
        const int r = r0 + (lane >> 4);
        const float* p = reinterpret_cast<const float*>(a.l + min(m0 + r, a.m - 1) * a.l_stride) + kb * kLine + 8 * c;
        const v4f lo = reinterpret_cast<const v4f*>(p)[0], hi = reinterpret_cast<const v4f*>(p)[1];
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        uint32_t top = 0;  // max |v| as bits: a NaN is larger than every number
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        const float scale = __uint_as_float(row16_max(top)) / kE4m3Max;
        *reinterpret_cast<__attribute__((address_space(3))) q_u32x2*>(to + chunk_at(r, c >> 1) + 8 * (c & 1)) =
            quant8(v, scale);
        if (c == 0) *reinterpret_cast<__attribute__((address_space(3))) float*>(to + MT * 2048 + 4 * r) = scale;
      }
    }
    if (i + DEPTH <= count)
      wait_vm<LOADS * (DEPTH - 1)>();
    else
      wait_vm<0>();
    const lds_u8* st = ring + slot * SLOT;
    if constexpr (kFp8) {
      float fw[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) fw[b] = scalar_f32(sw[b] + kb);
      if constexpr (kHalves) {
        const float up = scalar_f32(sw_up + kb);
        fw[0] = g >= 2 ? up : fw[0];
      }
      v8i w[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) w[b] = frag_fp8(st, b, lane);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const v8i x = frag_fp8(st, RB + t, lane);
        const float fx = ((const __attribute__((address_space(3))) float*)(st + (RB + MT) * 2048))[16 * t + (lane & 15)];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          v4f p = {0.f, 0.f, 0.f, 0.f};
          if constexpr (MT == 1) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp8((uint32_t)w[b][2 * s], (uint32_t)w[b][2 * s + 1]),
                                                          widen_fp8((uint32_t)x[2 * s], (uint32_t)x[2 * s + 1]), p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[b], x, p, 0, 0, 0, 0, 0, 0);
          }
          const float f = fw[b] * fx;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b][t][e] = fmaf(p[e], f, acc[b][t][e]);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        v8bf w[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) w[b] = frag_bf16<kKin>(st, b, s, lane);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const v8bf x = frag_bf16<kKin>(st, RB + t, s, lane);
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[b], x, acc[b][t], 0, 0, 0);
        }
      }
    }
    if (i + DEPTH < count) {
      wait_lds();  // the slot has been read
      issue(kb + DEPTH * WAVES, slot);
    }
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
  }
  __syncthreads();  // every ring has been read
  typedef __attribute__((address_space(3))) v4f lds_v4f;
  lds_v4f* part = (lds_v4f*)lds;  // [WAVES][RB][MT][64]
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[((wave * RB + b) * MT + t) * 64 + lane] = acc[b][t];
  __syncthreads();
  constexpr int kJobs = (kPair ? 1 : RB) * MT;  // blocks of 16 x 16 results (kHalves: 8 x 16), one wave each
  for (int job = wave; job < kJobs; job += WAVES) {
    const int b = job / MT, t = job % MT;
    const int m = m0 + t * 16 + (lane & 15), c = n0 + 16 * b + 4 * g;
    if (m >= a.m || c >= a.n || (kHalves && g >= 2)) continue;
    float v[kPair ? 2 : 1][4] = {};
#pragma unroll
    for (int h = 0; h < (kPair ? 2 : 1); ++h)
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const v4f p = part[((w * RB + (kHalves ? 0 : kPair ? h : b)) * MT + t) * 64 + (kHalves ? lane + 32 * h : lane)];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][e] += p[e];
      }
    if constexpr (EPI == kOut) {
      store_out(a, m, c, v[0]);
    } else if constexpr (EPI == kPart) {
      *reinterpret_cast<v4f*>(a.outf + (int64_t)m * a.pitch + c) = v4f{v[0][0], v[0][1], v[0][2], v[0][3]};
    } else if constexpr (EPI == kSwiglu) {
      store_swiglu(a, m, c, v[0], v[1]);
    } else {
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = swiglu(v[0][e], v[1][e]);
      store_f32(a.outf + (int64_t)m * a.n + c, c, a.n, false, h);
    }
  }
}

template <int L, int EPI, int RB, int MT, int WAVES, int DEPTH>
void launch_few_as(const Args& a, hipStream_t s) {
  constexpr int cols = EPI == kSwiglu || EPI == kSwigluF32 ? 8 * RB : 16 * RB;
  hipLaunchKernelGGL((few_kernel<L, RB, MT, WAVES, DEPTH, EPI>),
                     dim3((a.n + cols - 1) / cols, (a.m + 16 * MT - 1) / (16 * MT)), dim3(WAVES * 64), 0, s, a);
}
// MAX_MT 1: one block of L rows only (a.m <= 16).
template <int L, int EPI, int MAX_MT = 4>
void launch_few(const Args& a, hipStream_t s) {
  // 16 columns a workgroup, 8 with SwiGLU, where twice as many would leave CUs idle
  // (M=64 K=7168: N=7168 18 us with 32, 26 with 16; N=4096 T=1 7.1 with 16)
  const int wide = EPI == kSwiglu || EPI == kSwigluF32 ? 16 : 32, blocks = (a.m + 15) / 16;
  const int64_t cols = (a.n + wide - 1) / wide;
  const int mt = few_blocks(blocks, cols);
  const bool narrow = few_narrow(cols * ((blocks + mt - 1) / mt), mt);
  if constexpr (MAX_MT > 1) {
    if (mt == 2) return narrow ? launch_few_as<L, EPI, 1, 2, 8, 2>(a, s) : launch_few_as<L, EPI, 2, 2, 8, 2>(a, s);
    if (mt == 3) return narrow ? launch_few_as<L, EPI, 1, 3, 4, 3>(a, s) : launch_few_as<L, EPI, 2, 3, 4, 3>(a, s);
    if (mt == 4) return narrow ? launch_few_as<L, EPI, 1, 4, 4, 3>(a, s) : launch_few_as<L, EPI, 2, 4, 6, 2>(a, s);
  }
  // what is quantised first hides behind more waves (shared expert T=1 H=4096 I=8192
  // 23.3 us with 16 waves, 25.6 with 8)
  if constexpr (L == kQuant)
    return narrow ? launch_few_as<L, EPI, 1, 1, 16, 1>(a, s) : launch_few_as<L, EPI, 2, 1, 16, 1>(a, s);
  else
    return narrow ? launch_few_as<L, EPI, 1, 1, 8, 2>(a, s) : launch_few_as<L, EPI, 2, 1, 8, 2>(a, s);
}

}  // namespace dense
}  // namespace moe
