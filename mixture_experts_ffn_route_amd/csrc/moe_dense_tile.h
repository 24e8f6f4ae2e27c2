// Dense products on 128 x 128 tiles, for mid-size batches, and the sums of products
// split over K.
//
// WN (n) x 2 (m) waves; a K-block of 128 bytes is one stage of a ring, of
// four where a CU has one workgroup, of two where it has two, whose loads then
// run beside the other's MFMAs.
//
// Latency bounds it: a K-block takes 0.75 us with one workgroup a CU (LDS reads 0.35,
// MFMAs 0.25, and a barrier between), 1.1 for two.  N=7168 K=2048 M=512 16.4 us;
// with four waves in place of eight 18.6, with two stages in parts of K 25.
// Fragments read one K-block ahead, between the MFMAs, were slower (24 us): with
// branches around the loads the compiler no longer overlaps anything.
#pragma once

#include "moe_dense_dev.h"

namespace moe {
namespace dense {

// What becomes of a tile's results.
enum {
  kOut,       // out = bf16(acc + add)
  kOutF32,    // outf = acc, or outf + acc
  kPart,      // part[split] = acc
  kSwiglu,    // R = gate rows, then up rows: out = h = bf16(silu(g) u), gu = g | u where wanted
  kSwigluQ,   // the same, h as e4m3 with a scale per 128 columns
  kDswiglu,   // acc = dh: out = bf16(dg | du) from gu
  kSwigluF32  // outf = h (few tokens)
};

struct Args {
  const uint8_t* l;  // m side; strides in bytes between memory lines
  int64_t l_stride;
  const uint8_t* r;  // n side
  int64_t r_stride;
  const float* ls;   // e4m3: [m, kbs]
  const float* rs;   // e4m3: [ceil(n / 128), kbs]
  int32_t m, n, k;   // n: columns of the result (SwiGLU: of h)
  int32_t kbs;       // K-blocks of 128 bytes (bfloat16: 64 values)
  int32_t m_tiles, n_tiles, kb_per_split;
  uint16_t* out;
  int64_t out_stride;  // values
  const uint16_t* add;  // null: none
  int64_t add_stride;
  float* outf;  // kOutF32: [m, n]; kPart: [splits, m, pitch]; kSwigluF32: [m, n]
  int32_t pitch;  // kPart: n up to whole 16 bytes
  int32_t accumulate;
  int32_t vec;  // results of 4 columns may be stored at once; 2: of 8, and n is a multiple of 8
  float* gu;  // [m, 2 n]
  uint8_t* hq;
  float* hs;
};

// Whether few_kernel takes half of its columns a workgroup: where the whole would
// be `groups` workgroups, too few for the CUs, and twice as many run at once (two
// a CU with one block of L rows, else one). N=K=5120, 160 groups of whole width:
// M=24 9.7 us with half, 7.0 with whole; M=64 17.1 and 11.2; N=4160 K=2048 M=17 4.9
// and 3.8. With one block of L rows half gains up to 200 groups.
inline bool few_narrow(int64_t groups, int mt) { return mt == 1 ? groups < 200 : groups <= 128; }
// Blocks of 16 L rows a workgroup of few_kernel takes, at most 4: fewer where the
// workgroups of half width still run at once, `cols` of whole width for each part of L
// (N=576 K=7168: M=64 11.5 us with 4, 5.3 with 1, M=128 9.2 and 5.6; BF16 block H=2048
// I=768 T=64 11.3 and 7.3).
inline int few_blocks(int blocks, int64_t cols) {
  const int parts = (blocks + 3) / 4;
  int mt = (blocks + parts - 1) / parts;
  while (mt > 1 && 2 * cols * ((blocks + mt - 2) / (mt - 1)) <= 256) --mt;
  return mt;
}

__device__ __forceinline__ void unpack4(u32x2 v, float f[4]) {
  f[0] = bf16_to_f32(v[0] & 0xffffu);
  f[1] = bf16_to_f32(v[0] >> 16);
  f[2] = bf16_to_f32(v[1] & 0xffffu);
  f[3] = bf16_to_f32(v[1] >> 16);
}
__device__ __forceinline__ u32x2 pack4(const float f[4]) { return u32x2{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])}; }

// Results of two neighbouring blocks of 16 columns as 16 bytes a lane: lane group g
// of 16 lanes holds columns 4 g + [0, 4) of both, and after the exchange of rows
// of lanes columns 8 (g / 2) + [0, 8) of block g % 2; and back.
__device__ __forceinline__ void swap_rows(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ u32x4 join16(u32x2 a, u32x2 b) {
  uint32_t a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1];
  swap_rows(a0, b0);
  swap_rows(a1, b1);
  return u32x4{a0, a1, b0, b1};
}
__device__ __forceinline__ void part16(u32x4 v, u32x2& a, u32x2& b) {
  uint32_t a0 = v[0], a1 = v[1], b0 = v[2], b1 = v[3];
  swap_rows(a0, b0);
  swap_rows(a1, b1);
  a = u32x2{a0, a1};
  b = u32x2{b0, b1};
}

// Four results of row m, columns [c, c + 4) (those below n exist).
__device__ __forceinline__ void store_out(const Args& a, int64_t m, int c, const float v[4]) {
  uint16_t* o = a.out + m * a.out_stride + c;
  const uint16_t* d = a.add ? a.add + m * a.add_stride + c : nullptr;
  if (a.vec && c + 4 <= a.n) {
    float f[4] = {v[0], v[1], v[2], v[3]};
    if (d) {
      float e[4];
      unpack4(*reinterpret_cast<const u32x2*>(d), e);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] += e[i];
    }
    *reinterpret_cast<u32x2*>(o) = pack4(f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < a.n) o[i] = (uint16_t)f32_to_bf16_rne(d ? v[i] + bf16_to_f32(d[i]) : v[i]);
  }
}
// n is a multiple of 4, and o aligned, in these
__device__ __forceinline__ void store_f32(float* o, int c, int n, bool accumulate, const float v[4]) {
  if (c >= n) return;
  v4f f = {v[0], v[1], v[2], v[3]};
  if (accumulate) f += *reinterpret_cast<const v4f*>(o);
  *reinterpret_cast<v4f*>(o) = f;
}
// h, and g | u where wanted
__device__ __forceinline__ void store_swiglu(const Args& a, int64_t m, int c, const float g[4], const float u[4]) {
  if (c >= a.n) return;
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = swiglu(g[i], u[i]);
  *reinterpret_cast<u32x2*>(a.out + m * a.out_stride + c) = pack4(h);
  if (a.gu) {
    float* p = a.gu + m * 2 * (int64_t)a.n + c;
    *reinterpret_cast<v4f*>(p) = v4f{g[0], g[1], g[2], g[3]};
    *reinterpret_cast<v4f*>(p + a.n) = v4f{u[0], u[1], u[2], u[3]};
  }
}
__device__ __forceinline__ void store_dswiglu(const Args& a, int64_t m, int c, const float dh[4]) {
  if (c >= a.n) return;
  const float* p = a.gu + m * 2 * (int64_t)a.n + c;
  const v4f g = *reinterpret_cast<const v4f*>(p), u = *reinterpret_cast<const v4f*>(p + a.n);
  float dg[4], du[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dswiglu(g[i], u[i], dh[i], dg[i], du[i]);
  uint16_t* o = a.out + m * a.out_stride + c;
  *reinterpret_cast<u32x2*>(o) = pack4(dg);
  *reinterpret_cast<u32x2*>(o + a.n) = pack4(du);
}

template <bool FP8, int LL, int LR, int EPI, int STAGES, int WN>
__global__ __launch_bounds__(WN * 128, STAGES == 2 ? 2 : 1) void tile_kernel(Args a) {
  constexpr bool kPair = EPI == kSwiglu;
  static_assert(!FP8 || (LL == kKin && LR == kKin && !kPair), "e4m3: no transposing read here, gate | up through kPart");
  constexpr int BM = 128, BN = 128, WAVES = 2 * WN, NB = BN / 16 / WN, TB = BM / 32, HN = BN / 2;  // blocks of 16 per wave; rows of R in half a tile
  constexpr int NP = (BN + BM) / 8 / WAVES, NPR = BN / 8 / WAVES;  // DMA pieces per wave and K-block, of R
  constexpr int STAGE = (BN + BM) * kLine + (FP8 ? BM * 4 : 0);
  constexpr int LOADS = NP + (FP8 ? 1 : 0);
  __shared__ __attribute__((aligned(1024))) uint8_t ring_lds[STAGES * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave % WN, wm = wave / WN;
  int mt, nt;
  if (!tile_of(blockIdx.x, a.m_tiles, a.n_tiles, 8, mt, nt)) return;
  const int m0 = mt * BM, n0 = nt * (kPair ? HN : BN);
  const int kb0 = blockIdx.y * a.kb_per_split, kb1 = min(kb0 + a.kb_per_split, a.kbs);
  constexpr int ES = FP8 ? 1 : 2;

  // operands: two halves of R (gate and up rows, or rows that follow), L
  Operand op[3];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int row = kPair ? n0 + h * a.n : n0 + h * HN;
    int rows = kPair ? a.n - n0 : a.n - n0 - h * HN;
    if (rows <= 0) {  // nothing there: half 0 again, not stored
      row = n0;
      rows = a.n - n0;
    }
    op[h] = Operand{a.r + (LR == kKin ? row * a.r_stride : (int64_t)row * ES), a.r_stride, min(rows, HN)};
  }
  op[2] = Operand{a.l + (LL == kKin ? m0 * a.l_stride : (int64_t)m0 * ES), a.l_stride, min(a.m - m0, BM)};
  uint32_t off[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = i * WAVES + wave;
    if (i < NPR / 2)
      off[i] = piece_offset<LR>(op[0], p, lane);
    else if (i < NPR)
      off[i] = piece_offset<LR>(op[1], p - HN / 8, lane);
    else
      off[i] = piece_offset<LL>(op[2], p - BN / 8, lane);
  }
  const uint32_t sx_off = FP8 ? __umul24(min(wave * 64 % BM + lane, op[2].rows - 1), (uint32_t)a.kbs) * 4u : 0;
  auto issue = [&](int kb) {
    const lds_u8* st = (const lds_u8*)ring_lds + (kb - kb0) % STAGES * STAGE;
    if constexpr (FP8)  // the rows' scales (the waves behind the first load them again)
      dma4(a.ls + (int64_t)m0 * a.kbs + kb, sx_off, st + (BN + BM) * kLine + wave * 64 % BM * 4);
    const int64_t radv = LR == kKin ? (int64_t)kb * kLine : (int64_t)kb * 64 * a.r_stride;
    const int64_t ladv = LL == kKin ? (int64_t)kb * kLine : (int64_t)kb * 64 * a.l_stride;
    const int kleft = a.k - kb * (kLine / ES);  // values of K from here on
    if (kleft >= kLine / ES) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool is_r = i < NPR;
        dma16(is_r ? op[i < NPR / 2 ? 0 : 1].base + radv : op[2].base + ladv, off[i], st + (i * WAVES + wave) * 1024);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool is_r = i < NPR;
        const int p = i * WAVES + wave - (is_r ? (i < NPR / 2 ? 0 : HN / 8) : BN / 8);
        const uint8_t* src = (is_r ? op[i < NPR / 2 ? 0 : 1].base + radv : op[2].base + ladv) + off[i];
        const bool ok = is_r ? piece_valid<LR>(p, lane, LR == kKin ? kleft * ES : kleft)
                             : piece_valid<LL>(p, lane, LL == kKin ? kleft * ES : kleft);
        dma16_at(ok ? src : (const uint8_t*)&kZeros, st + (i * WAVES + wave) * 1024);
      }
    }
  };

  // e4m3: scales of the two halves' weight blocks
  const float* sw_p[2] = {nullptr, nullptr};
  if constexpr (FP8) {
    const int blocks = (a.n + 127) / 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) sw_p[h] = a.rs + (int64_t)min((n0 + h * HN) / 128, blocks - 1) * a.kbs;
  }

  v4f acc[NB][TB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
  // block of R's fragment i within the half: (half, block)
  auto r_tile = [&](const lds_u8* st, int i) { return st + (i < NB / 2 ? 0 : HN * kLine); };
  auto r_block = [&](int i) { return wn * (NB / 2) + (i < NB / 2 ? i : i - NB / 2); };

#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i)
    if (kb0 + i < kb1) issue(kb0 + i);  // (no tokens: no K-block)
  for (int kb = kb0; kb < kb1; ++kb) {
    if (kb + STAGES - 2 < kb1)
      wait_vm<LOADS * (STAGES - 2)>();
    else
      wait_vm<0>();
    wait_lds();
    barrier();
    const lds_u8* st = (const lds_u8*)ring_lds + (kb - kb0) % STAGES * STAGE;
    const lds_u8* lt = st + BN * kLine;
    if constexpr (FP8) {
      const float sw0 = scalar_f32(sw_p[0] + kb), sw1 = scalar_f32(sw_p[1] + kb);
      const __attribute__((address_space(3))) float* sx =
          (const __attribute__((address_space(3))) float*)(lt + BM * kLine) + wm * (BM / 2) + (lane & 15);
      // every fragment at once: the loads are issued while they come
      v8i rf[NB], lf[TB];
      float s[TB];
#pragma unroll
      for (int i = 0; i < NB; ++i) rf[i] = frag_fp8(r_tile(st, i), r_block(i), lane);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        lf[t] = frag_fp8(lt, wm * TB + t, lane);
        s[t] = sx[t * 16];
      }
      if (kb + STAGES - 1 < kb1) issue(kb + STAGES - 1);
      // the multiply-adds run two MFMAs behind
      v4f p[4];
      auto add = [&](int q) {
        const int t = q / NB, i = q % NB;
        const float f = s[t] * (i < NB / 2 ? sw0 : sw1);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(p[q & 3][e], f, acc[i][t][e]);
      };
#pragma unroll
      for (int q = 0; q < NB * TB; ++q) {
        p[q & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(rf[q % NB], lf[q / NB], v4f{0.f, 0.f, 0.f, 0.f}, 0,
                                                                    0, 0, 0, 0, 0);
        if (q >= 2) add(q - 2);
      }
      add(NB * TB - 2);
      add(NB * TB - 1);
    } else {
      v8bf rf[2][NB], lf[2][TB];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < NB; ++i) rf[s][i] = frag_bf16<LR>(r_tile(st, i), r_block(i), s, lane);
#pragma unroll
        for (int t = 0; t < TB; ++t) lf[s][t] = frag_bf16<LL>(lt, wm * TB + t, s, lane);
      }
      if (kb + STAGES - 1 < kb1) issue(kb + STAGES - 1);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
          for (int i = 0; i < NB; ++i)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(rf[s][i], lf[s][t], acc[i][t], 0, 0, 0);
    }
  }

  const int lm = m0 + wm * (BM / 2) + (lane & 15);  // this lane's row of block t: + 16 t
  const int lc = 4 * (lane >> 4);
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int64_t m = lm + t * 16;
    if (m >= a.m) continue;
#pragma unroll
    for (int i = 0; i < (kPair ? NB / 2 : NB); ++i) {
      const int c = n0 + (i < NB / 2 ? 0 : HN) + r_block(i) * 16 + lc;
      const v4f v = acc[i][t];
      const float f[4] = {v[0], v[1], v[2], v[3]};
      if constexpr (EPI == kOut) {
        store_out(a, m, c, f);
      } else if constexpr (EPI == kOutF32) {
        store_f32(a.outf + m * a.n + c, c, a.n, a.accumulate, f);
      } else if constexpr (EPI == kPart) {
        if (c < a.pitch) *reinterpret_cast<v4f*>(a.outf + ((int64_t)blockIdx.y * a.m + m) * a.pitch + c) = v;
      } else if constexpr (EPI == kSwiglu) {
        const v4f w = acc[NB / 2 + i][t];
        const float u[4] = {w[0], w[1], w[2], w[3]};
        store_swiglu(a, m, c, f, u);
      } else {
        store_dswiglu(a, m, c, f);
      }
    }
  }
}

// Sums of kPart results over the splits, in ascending order, and what becomes
// of them; a thread takes 4 columns of one row.  kSwigluQ: 32 lanes hold a scale
// block.  part: [splits, a.m, pitch].
template <int EPI>
__global__ __launch_bounds__(256) void join_kernel(Args a, const float* part, int splits, int pitch) {
  constexpr bool kPair = EPI == kSwiglu || EPI == kSwigluQ;
  const int quads = (a.n + 3) / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = at / quads;
  const int c = (int)(at - m * quads) * 4;
  if (m >= a.m) return;  // kSwigluQ: whole groups of 32 lanes
  const int64_t plane = (int64_t)a.m * pitch;
  float v[kPair ? 2 : 1][4] = {};
#pragma unroll
  for (int h = 0; h < (kPair ? 2 : 1); ++h) {
    const float* p = part + m * pitch + c + h * a.n;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const v4f w = *reinterpret_cast<const v4f*>(p + s * plane);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h][i] += w[i];
    }
  }
  if constexpr (EPI == kOut) {
    store_out(a, m, c, v[0]);
  } else if constexpr (EPI == kDswiglu) {
    store_dswiglu(a, m, c, v[0]);
  } else if constexpr (EPI == kSwiglu) {
    store_swiglu(a, m, c, v[0], v[1]);
  } else {
    float h[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = swiglu(v[0][i], v[1][i]);
      top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, w, 32));
    const float s = __uint_as_float(top) / kE4m3Max;
    *reinterpret_cast<uint32_t*>(a.hq + m * a.n + c) = quant4(h, s);
    if (c % 128 == 0) a.hs[m * (a.n / 128) + c / 128] = s;
  }
}

}  // namespace dense
}  // namespace moe
