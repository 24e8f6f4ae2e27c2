// BF16 products on tiles of 256 rows of R and BM (256, 128) of L.
//
// Four waves, one a SIMD, 2 (n) x 2 (m), each with a quarter of the tile in its
// accumulators (128 x 128: 256 registers).  A wave that large reads an operand
// value from LDS once for 128 results: 128 KB of reads and 64 KB of DMA a K-block
// of 64, 1536 of LDS's cycles beside 2048 of the MFMA's; with eight waves of 64 x
// 128 the reads alone would take 1536.
//
// With one wave a SIMD nothing but the wave itself hides a latency: the
// fragments are double-buffered in registers (those of half a K-block, 32 k, are
// read while the other half's MFMAs run), the K-blocks in LDS (two stages), and
// reads and DMA are spread between the MFMAs.  One barrier a K-block, between
// its halves: there every wave holds the second half's fragments, so the stage
// can take the next K-block but one, and the next K-block has landed.
//
// R has three stages of 32 KB and L two (with 128 rows of L three of 16 KB): the
// loads of a K-block are issued over all of the one before, half of them two ahead.
// All in the half behind the barrier, they hold up the MFMAs (T=16384 H=7168 I=2048
// FC1 792 us against 776; in the first half of that 822).
//
// Workgroups stay: a tile's last K-blocks already load the next tile's first.
//
// With 256 rows of L every register is taken: up to 3 are spilled around the epilogue,
// 28 to 31 with SwiGLU and float32 results, where the next tile's first fragments live
// over it; none in the K loop.
//
// The card's power bounds it in long runs: FC1 of T=16384 H=7168 I=2048 takes 705 us
// at first (1.36 PFLOP/s) and 770 when the clock has come down to 1.8 GHz, where the
// MFMAs are busy 72 % of the cycles.  Products with K outside run at the same rate
// (dw13 of T=4096 2 I=4096 H=7168 256 us in 1.75 rounds of tiles): their LDS reads
// have no conflicts either.  That step's backward takes 640 us with BF16 and with
// float32 weight gradients, 724 where those are accumulated, which reads 176 MB more.
#pragma once

#include <type_traits>

#include "moe_dense_tile.h"

namespace moe {
namespace dense {

// acc += r l^T in accumulation registers: with 256 of them the compiler, left to
// choose, keeps some in the other half of the file and copies them to and fro.
// What it does not know of an MFMA in asm: results are read only after the wait
// behind the K loop, an accumulator is used again NB TB MFMAs later, and
// operands come from LDS reads, for which it waits.
__device__ __forceinline__ void mfma(v4f& acc, const v8bf& r, const v8bf& l) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(r), "v"(l));
}

// CUT: K is no multiple of 64.  blockIdx.y: the part of K (kPart).
template <int LL, int LR, int BM, int BN, int EPI, bool CUT>
__global__ __launch_bounds__(256, 1) void big_kernel(Args a) {
  constexpr bool kPair = EPI == kSwiglu;
  constexpr int NB = BN / 32, TB = BM / 32, HN = BN / 2;
  constexpr int NPR = BN / 32, NPL = BM / 32;               // DMA pieces per wave and K-block
  constexpr int R_BYTES = BN * kLine, L_BYTES = BM * kLine;  // a K-block of each
  __shared__ __attribute__((aligned(1024))) uint8_t r_lds[3 * R_BYTES];
  constexpr int LST = BM == 256 ? 2 : 3;                     // stages of L
  __shared__ __attribute__((aligned(1024))) uint8_t l_lds[LST * L_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 1, wm = wave >> 1;
  const int total = a.m_tiles * a.n_tiles;
  const int kb0 = blockIdx.y * a.kb_per_split, kbs = min(a.kb_per_split, a.kbs - kb0);

  // The tiles whose loads are being issued, R's and L's: scalars only (a lane's
  // offsets are computed again for each piece, three instructions beside the
  // MFMAs, in place of a register each).
  const uint8_t* base[3];
  int rows[3];
  auto setup_r = [&](int nt) {
    const int n0 = nt * (kPair ? HN : BN);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int row = kPair ? n0 + h * a.n : n0 + h * HN, left = kPair ? a.n - n0 : a.n - n0 - h * HN;
      if (left <= 0) {  // nothing there: half 0 again, not stored
        row = n0;
        left = a.n - n0;
      }
      base[h] = a.r + (LR == kKin ? row * a.r_stride : (int64_t)row * 2);
      rows[h] = min(left, HN);
    }
  };
  auto setup_l = [&](int mt) {
    const int m0 = mt * BM;
    base[2] = a.l + (LL == kKin ? m0 * a.l_stride : (int64_t)m0 * 2);
    rows[2] = min(a.m - m0, BM);
  };
  // Pieces 4 i + wave (see piece_offset): kKin rows 32 i + in_row, chunk in_c;
  // kKout k = 8 (i % 2) + out_k, rows 64 (i / 2) + out_n.
  const int in_row = 8 * wave + (lane >> 3), in_c = ((lane & 7) ^ swz(in_row & 15)) * 16;
  const int out_k = 16 * (2 * (wave & 1) + ((lane >> 3) & 1)) + 4 * (wave >> 1) + ((lane >> 1) & 3);
  const int out_n = 16 * (lane >> 4) + 8 * (lane & 1);
  // Piece i of K-block kb of R or L into a stage of its own.
  auto issue_piece = [&](bool is_r, int stage, int kb_local, int i) {
    const int kb = kb0 + kb_local;
    const lds_u8* to = (is_r ? (const lds_u8*)r_lds + stage * R_BYTES : (const lds_u8*)l_lds + stage * L_BYTES) +
                       (i * 4 + wave) * 1024;
    const int o = is_r ? (i < HN / 32 ? 0 : 1) : 2, j = is_r ? i - o * (HN / 32) : i;
    const int layout = is_r ? LR : LL;
    const int64_t stride = is_r ? a.r_stride : a.l_stride;
    const uint8_t* from = base[o] + (layout == kKin ? (int64_t)kb * kLine : (int64_t)kb * 64 * stride);
    const uint32_t off = layout == kKin
                             ? __umul24(min(32 * j + in_row, rows[o] - 1), (uint32_t)stride) + in_c
                             : __umul24(8 * (j & 1) + out_k, (uint32_t)stride) + 2 * min(64 * (j >> 1) + out_n, rows[o] - 8);
    if constexpr (!CUT) {
      dma16(from, off, to);
    } else {
      const int left = a.k - kb * 64;
      const bool ok = layout == kKin ? in_c < 2 * left : 8 * (j & 1) + out_k < left;
      dma16_at(ok ? from + off : (const uint8_t*)&kZeros, to);
    }
  };

  v8bf rf[2][NB], lf[2][TB];
  // fragment f (R's, then L's) of half s of the K-block in these stages
  auto read = [&](int sr, int sl, int s, int f) {
    if (f < NB)
      rf[s][f] = frag_bf16<LR>((const lds_u8*)r_lds + sr * R_BYTES + (f < NB / 2 ? 0 : HN * kLine),
                               wn * (NB / 2) + (f < NB / 2 ? f : f - NB / 2), s, lane);
    else
      lf[s][f - NB] = frag_bf16<LL>((const lds_u8*)l_lds + sl * L_BYTES, wm * TB + f - NB, s, lane);
  };

  // The K-blocks to load next are r.kb of tile r.v and l.kb of l.v.  After the
  // last tile its last K-block is loaded again, into stages that nothing reads.
  const int ids = (total + 7) / 8 * 8;  // grid is a multiple of 8: a workgroup keeps its XCD
  int mt = 0, nt = 0;
  auto next = [&](int id) {  // the next tile from id on, in mt and nt
    while (id < ids && !tile_of(id, a.m_tiles, a.n_tiles, 8, mt, nt)) id += gridDim.x;
    return id;
  };
  struct Cursor {
    int v, kb;
  };
  int v = next(blockIdx.x);
  if (v >= ids) return;
  int mt_cur = mt, nt_cur = nt;
  setup_r(nt);
  setup_l(mt);
  Cursor cr{v, 0}, cl{v, 0};
  auto advance = [&](Cursor& c) {  // true: another tile, in mt and nt
    if (++c.kb < kbs) return false;
    if (c.v < ids) c.v = next(c.v + gridDim.x);
    c.kb = c.v < ids ? 0 : kbs - 1;
    return c.v < ids;
  };
  auto advance_r = [&]() {
    if (advance(cr)) setup_r(nt);
  };
  auto advance_l = [&]() {
    if (advance(cl)) setup_l(mt);
  };
#pragma unroll
  for (int pre = 0; pre < 2; ++pre) {
#pragma unroll
    for (int i = 0; i < NPR; ++i) issue_piece(true, pre, cr.kb, i);
    advance_r();
  }
#pragma unroll
  for (int pre = 0; pre < LST; ++pre) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) issue_piece(false, pre, cl.kb, i);
    advance_l();
  }
  int sr = 0, sl = 0;  // stages of the K-block at hand
  auto after = [](int stage, int n) { return stage + n >= 3 ? stage + n - 3 : stage + n; };
  wait_vm<0>();
  barrier();
#pragma unroll
  for (int f = 0; f < NB + TB; ++f) read(0, 0, 0, f);

  while (true) {
    v4f acc[NB][TB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
    // written by VALU instructions, and next read by MFMAs that the compiler does not know
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) asm volatile("" : "+a"(acc[i][t]));
    asm volatile("s_nop 7" ::: "memory");
    constexpr int GROUPS = NB * TB / 4, READS = NB + TB;
    // half s of a K-block: its MFMAs; the fragments of half s ^ 1 (of the next
    // K-block if s is 1) from stages fr and fl; the loads of R (s = 0) or L into
    // a stage
    auto half = [&](auto s_, int fr, int fl, int into) {
      constexpr int s = decltype(s_)::value, NP = s == 0 ? NPR : NPL;
#pragma unroll
      for (int q = 0; q < GROUPS; ++q) {
#pragma unroll
        for (int f = q * READS * 3 / 2 / GROUPS; f < (q + 1) * READS * 3 / 2 / GROUPS; ++f)
          if (f < READS) read(fr, fl, s ^ 1, f);
#pragma unroll
        for (int i = q * NP / GROUPS; i < (q + 1) * NP / GROUPS; ++i)
          issue_piece(s == 0, into, s == 0 ? cr.kb : cl.kb, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (q * 4 + e) % NB, t = (q * 4 + e) / NB;
          mfma(acc[i][t], rf[s][i], lf[s][t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int kb = 0; kb < kbs; ++kb) {
      half(std::integral_constant<int, 0>{}, sr, sl, after(sr, 2));
      advance_r();
      wait_lds();
      wait_vm<NPR + (LST - 2) * NPL>();  // the next K-block is there; what was issued after it stays in flight
      barrier();
      __builtin_amdgcn_sched_barrier(0);
      const int sn = sl + 1 == LST ? 0 : sl + 1;
      half(std::integral_constant<int, 1>{}, after(sr, 1), sn, sl);
      advance_l();
      sr = after(sr, 1);
      sl = sn;
    }
    // the MFMAs' results are there 18 wait states after the last
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) asm volatile("" : "+a"(acc[i][t]));

    const int m0 = mt_cur * BM, n0 = nt_cur * (kPair ? HN : BN);
    const int g = lane >> 4, lm = m0 + wm * (BM / 2) + (lane & 15), lc = n0 + wn * (HN / 2) + 4 * g;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const int64_t m = lm + t * 16;
      if (m < a.m) {
#pragma unroll
        for (int i = 0; i < (kPair ? NB / 2 : NB); ++i) {
          const int at = i < NB / 2 ? i * 16 : HN + (i - NB / 2) * 16;
          const int c = lc + at;
          const v4f r = acc[i][t];
          if constexpr (EPI == kPart) {
            if (c < a.n) *reinterpret_cast<v4f*>(a.outf + ((int64_t)blockIdx.y * a.m + m) * a.pitch + c) = r;
          } else if constexpr (EPI == kOutF32) {
            v4f* o = reinterpret_cast<v4f*>(a.outf + m * a.n + c);
            if (c < a.n) *o = a.accumulate ? *o + r : r;
          } else if (i % 2 == 0) {  // two blocks: 8 columns a lane (n is a multiple of 8)
            const int c16 = n0 + wn * (HN / 2) + at + 16 * (g & 1) + 8 * (g >> 1);
            uint16_t* o = a.out + m * a.out_stride + c16;
            u32x2 x[2], y[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const v4f q = acc[i + k][t];
              float f[4] = {q[0], q[1], q[2], q[3]};
              if constexpr (EPI == kSwiglu) {
                const v4f w = acc[NB / 2 + i + k][t];
                if (a.gu && c + 16 * k < a.n) {
                  float* p = a.gu + m * 2 * (int64_t)a.n + c + 16 * k;
                  *reinterpret_cast<v4f*>(p) = q;
                  *reinterpret_cast<v4f*>(p + a.n) = w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = swiglu(q[e], w[e]);
              } else if constexpr (EPI == kDswiglu) {
                const float* p = a.gu + m * 2 * (int64_t)a.n + min(c + 16 * k, a.n - 4);
                const v4f gate = *reinterpret_cast<const v4f*>(p), up = *reinterpret_cast<const v4f*>(p + a.n);
                float du[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) dswiglu(gate[e], up[e], q[e], f[e], du[e]);
                y[k] = pack4(du);
              }
              x[k] = pack4(f);
            }
            const u32x4 first = join16(x[0], x[1]);
            if (c16 < a.n) *reinterpret_cast<u32x4*>(o) = first;
            if constexpr (EPI == kDswiglu) {
              const u32x4 second = join16(y[0], y[1]);
              if (c16 < a.n) *reinterpret_cast<u32x4*>(o + a.n) = second;
            }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    v = next(v + gridDim.x);
    if (v >= ids) break;
    mt_cur = mt;
    nt_cur = nt;
  }
  wait_vm<0>();  // no load into LDS outlives the workgroup
}

}  // namespace dense
}  // namespace moe
