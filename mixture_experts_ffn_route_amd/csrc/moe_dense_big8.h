// e4m3 products with block scales on tiles of 256 rows of R and BM (256, 128) of L.
//
// Every block's sum P has to leave the MFMA to be multiplied by its own scales:
// acc += sx sw P, four multiply-adds a lane beside each 16 x 16 x 128 MFMA (16 of
// its 32 cycles).  Those need the accumulators in ordinary registers, so eight
// waves share the tile (64 x BM / 2 each, 128 registers at 256), two a SIMD, in two groups
// of four that own half of L's rows each and run one slot apart: a K-block of 128
// is a load slot (the loads of the next K-block, the fragments of R) and an MFMA
// slot (32 MFMAs, L's fragments as they come, the multiply-adds of the MFMA
// before the last), with a barrier behind each, and while one group multiplies
// the other loads.
//
// Two stages of 64 KB, loaded one K-block ahead, or with 128 rows of L, whose
// MFMA slots are half as long, three of 48 KB, loaded two ahead.  Group 0 loads R
// and its rows of L, group 1 its rows; a wave waits for its loads of the next
// K-block at the end of its MFMA slot, and the barrier there publishes them.
//
// M=16384 N=K=7168: 727 to 743 us, 2.27 to 2.32 PFLOP/s.  The card's power bounds it in long runs
// (740 us at first, 840 behind others of its kind at 1.6 GHz, the MFMAs busy 62 %
// of the cycles); what the multiply-adds and LDS reads cost is seen without them:
// 543 and 606 us in place of 895, without the DMA 757.
#pragma once

#include "moe_dense_tile.h"

namespace moe {
namespace dense {

// CUT: K is no multiple of 128.  VEC: eight columns are stored at once (kOut).
// blockIdx.y: the part of K (kPart).
template <int EPI, bool CUT, bool VEC, int BM>
__global__ __launch_bounds__(512, 1) void big8_kernel(Args a) {
  constexpr bool kPair = EPI == kSwigluQ;
  constexpr int BN = 256, HN = BN / 2, NB = 4, GM = BM / 2, TB = GM / 16;  // GM: rows of L per group
  constexpr int STAGES = BM == 256 ? 2 : 3, AHEAD = STAGES - 1, LP = GM / 32;  // LP: pieces of L per wave
  constexpr int LOADS0 = 8 + LP + 1, LOADS1 = LP + 1;                          // loads of a wave per K-block
  constexpr int R_BYTES = BN * kLine, L_BYTES = BM * kLine;
  __shared__ __attribute__((aligned(1024))) uint8_t r_lds[STAGES * R_BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t l_lds[STAGES * L_BYTES];
  __shared__ __attribute__((aligned(16))) float sx_lds[STAGES][BM];
  __shared__ uint32_t top_s[kPair ? 4 * BM : 1];
  typedef __attribute__((address_space(3))) const float lds_f32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 3, grp = wave >> 2;
  const int total = a.m_tiles * a.n_tiles;
  const int kb0 = blockIdx.y * a.kb_per_split, kbs = min(a.kb_per_split, a.kbs - kb0);
  const int blocks = ((kPair ? 2 * a.n : a.n) + 127) / 128;

  // the tile whose loads are being issued
  const uint8_t *rb[2], *lb;
  const float* sxb;
  int rrows[2], lrows;
  auto setup = [&](int mt, int nt) {
    const int m0 = mt * BM, n0 = nt * (kPair ? HN : BN);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int row = kPair ? n0 + h * a.n : n0 + h * HN, left = kPair ? a.n - n0 : a.n - n0 - h * HN;
      if (left <= 0) {  // nothing there: half 0 again, not stored
        row = n0;
        left = a.n - n0;
      }
      rb[h] = a.r + row * a.r_stride;
      rrows[h] = min(left, HN);
    }
    lb = a.l + m0 * a.l_stride;
    lrows = min(a.m - m0, BM);
    sxb = a.ls + (int64_t)m0 * a.kbs;
  };
  // Pieces: wave w of a group takes pieces 4 i + w of 8 rows: of a half of R
  // (16 pieces) i = 0..3, of the group's rows of L i = 0..LP-1.
  const int in_row = 8 * wn + (lane >> 3), in_c = ((lane & 7) ^ swz(in_row & 15)) * 16;
  const int sx_row = GM * grp + wn * 64 % GM;  // 64 scales a wave; the waves past the group's rows load them again
  auto piece = [&](const uint8_t* from, int64_t stride, int row, int rows, int kb, const lds_u8* to) {
    const uint32_t off = __umul24(min(row, rows - 1), (uint32_t)stride) + in_c;
    if constexpr (!CUT)
      dma16(from + (int64_t)kb * kLine, off, to);
    else
      dma16_at(in_c < a.k - kb * kLine ? from + (int64_t)kb * kLine + off : (const uint8_t*)&kZeros, to);
  };
  auto issue = [&](int stage, int kb_local) {
    const int kb = kb0 + kb_local;
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        piece(rb[i >> 2], a.r_stride, 32 * (i & 3) + in_row, rrows[i >> 2], kb,
              (const lds_u8*)r_lds + stage * R_BYTES + (i * 4 + wn) * 1024);
    }
#pragma unroll
    for (int i = 0; i < LP; ++i)
      piece(lb, a.l_stride, GM * grp + 32 * i + in_row, lrows, kb,
            (const lds_u8*)l_lds + stage * L_BYTES + (4 * LP * grp + i * 4 + wn) * 1024);
    dma4(sxb + kb, __umul24(min(sx_row + lane, lrows - 1), (uint32_t)a.kbs) * 4u, (const lds_u8*)&sx_lds[stage][sx_row]);
  };

  // The K-block to load next is kb_in of tile v_in; after the last tile its last
  // K-block is loaded again, into a stage that nothing reads.
  const int ids = (total + 7) / 8 * 8;  // grid is a multiple of 8: a workgroup keeps its XCD
  int mt = 0, nt = 0;
  auto next = [&](int id) {
    while (id < ids && !tile_of(id, a.m_tiles, a.n_tiles, 4, mt, nt)) id += gridDim.x;
    return id;
  };
  int v = next(blockIdx.x);
  if (v >= ids) return;
  int v_in = v, kb_in = 0, mt_cur = mt, nt_cur = nt;
  setup(mt, nt);
  const float *sw0, *sw1;  // the current tile's weight scales
  auto tile_scales = [&]() {
    const int n0 = nt_cur * (kPair ? HN : BN);
    const int n1 = kPair ? n0 + a.n : (a.n - n0 > HN ? n0 + HN : n0);
    sw0 = a.rs + (int64_t)min(n0 / 128, blocks - 1) * a.kbs + kb0;
    sw1 = a.rs + (int64_t)min(n1 / 128, blocks - 1) * a.kbs + kb0;
  };
  tile_scales();
  auto advance = [&]() {
    if (++kb_in < kbs) return;
    if (v_in < ids) v_in = next(v_in + gridDim.x);
    kb_in = v_in < ids ? 0 : kbs - 1;
    if (v_in < ids) setup(mt, nt);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    issue(i, kb_in);
    advance();
  }
  wait_vm<0>();
  __syncthreads();

  const int tl = lane & 15, g = lane >> 4;
  const int lo = chunk_at(tl, 2 * g), hi = chunk_at(tl, 2 * g + 1);
  auto frag = [&](const lds_u8* block) {
    const u32x4 x = lds16(block + lo), y = lds16(block + hi);
    return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };
  int stage = 0;
  while (true) {
    v4f acc[NB][TB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
    if (grp == 1) barrier();  // one slot behind
    for (int kb = 0; kb < kbs; ++kb) {
      // load slot
      issue(stage + AHEAD >= STAGES ? stage + AHEAD - STAGES : stage + AHEAD, kb_in);
      const float w0 = scalar_f32(sw0 + kb), w1 = scalar_f32(sw1 + kb);
      const lds_u8* rt = (const lds_u8*)r_lds + stage * R_BYTES;
      const lds_u8* lt = (const lds_u8*)l_lds + stage * L_BYTES + grp * TB * 2048;
      lds_f32* st = (lds_f32*)&sx_lds[stage][GM * grp + tl];
      v8i rf[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) rf[i] = frag(rt + (i < 2 ? 0 : HN * kLine) + (wn * 2 + (i & 1)) * 2048);
      v8i lf = frag(lt);
      float s = st[0];
      advance();
      wait_lds();
#pragma unroll
      for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(rf[i]));  // read before the slot ends
      barrier();
      __builtin_amdgcn_sched_barrier(0);
      // MFMA slot
      v4f p[4];
      float f0 = 0.f, f1 = 0.f, pf0 = 0.f, pf1 = 0.f;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int tn = t + 1 < TB ? t + 1 : t;
        const v8i ln = frag(lt + tn * 2048);
        const float sn = st[tn * 16];
        pf0 = f0;
        pf1 = f1;
        f0 = s * w0;
        f1 = s * w1;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          p[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(rf[i], lf, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
          // the MFMA before the last
          const int q = (t * NB + i) - 2;
          if (q >= 0) {
            const int qt = q / NB, qi = q % NB;
            const float f = qt == t ? (qi < 2 ? f0 : f1) : (qi < 2 ? pf0 : pf1);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[qi][qt][e] = fmaf(p[qi][e], f, acc[qi][qt][e]);
          }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          if (i < 3) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        lf = ln;
        s = sn;
      }
#pragma unroll
      for (int i = 2; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][TB - 1][e] = fmaf(p[i][e], f1, acc[i][TB - 1][e]);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t) asm volatile("" : "+v"(acc[i][t]));  // issued before the slot ends
      // the next K-block is there; the loads behind it stay in flight
      if (grp == 0)
        wait_vm<LOADS0 * (AHEAD - 1)>();
      else
        wait_vm<LOADS1 * (AHEAD - 1)>();
      wait_lds();
      barrier();
      __builtin_amdgcn_sched_barrier(0);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    if (grp == 0) barrier();  // the groups side by side again

    const int m0 = mt_cur * BM, n0 = nt_cur * (kPair ? HN : BN);
    const int lm = m0 + GM * grp + tl, lc = n0 + wn * 32 + 4 * g;
    if constexpr (kPair) {
      float h[2][TB][4];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint32_t top = 0;  // max |h| as bits: a NaN is larger than every number
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[i][t][e] = swiglu(acc[i][t][e], acc[2 + i][t][e]);
            top = max(top, __float_as_uint(h[i][t][e]) & 0x7fffffffu);
          }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        if (lane < 16) top_s[wn * BM + GM * grp + t * 16 + tl] = top;
      }
      wait_lds();
      barrier();
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const int r = GM * grp + t * 16 + tl;
        const int64_t m = m0 + r;
        const uint32_t top = max(max(top_s[r], top_s[BM + r]), max(top_s[2 * BM + r], top_s[3 * BM + r]));
        const float sc = __uint_as_float(top) / kE4m3Max;
        if (m < a.m) {
          if (wn == 0 && lane < 16) a.hs[m * (a.n / 128) + nt_cur] = sc;
          uint32_t q0 = quant4(h[0][t], sc), q1 = quant4(h[1][t], sc);
          swap_rows(q0, q1);  // 8 columns of one of the two blocks
          *reinterpret_cast<u32x2*>(a.hq + m * a.n + n0 + wn * 32 + 16 * (g & 1) + 8 * (g >> 1)) = u32x2{q0, q1};
        }
      }
      wait_lds();
      barrier();  // top_s is read before the next tile's
    } else {
      if constexpr (EPI == kOut && VEC) {
        const int c16 = n0 + wn * 32 + 16 * (g & 1) + 8 * (g >> 1);  // this lane's 8 columns of a pair of blocks
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const int64_t m = lm + t * 16;  // the lanes that exchange have one row: all or none store
          if (m < a.m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = c16 + h * HN;
              v4f x = acc[2 * h][t], y = acc[2 * h + 1][t];
              if (a.add) {
                u32x2 dx, dy;
                part16(*reinterpret_cast<const u32x4*>(a.add + m * a.add_stride + min(c, a.n - 8)), dx, dy);
                float e[4], f[4];
                unpack4(dx, e);
                unpack4(dy, f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  x[k] += e[k];
                  y[k] += f[k];
                }
              }
              const float p[4] = {x[0], x[1], x[2], x[3]}, q[4] = {y[0], y[1], y[2], y[3]};
              const u32x4 o = join16(pack4(p), pack4(q));
              if (c < a.n) *reinterpret_cast<u32x4*>(a.out + m * a.out_stride + c) = o;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const int64_t m = lm + t * 16;
          if (m < a.m) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int c = lc + (i < 2 ? i * 16 : HN + (i - 2) * 16);
              const v4f r = acc[i][t];
              float f[4] = {r[0], r[1], r[2], r[3]};
              if constexpr (EPI == kPart) {
                if (c < a.pitch) *reinterpret_cast<v4f*>(a.outf + ((int64_t)blockIdx.y * a.m + m) * a.pitch + c) = r;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (c + e < a.n)
                    a.out[m * a.out_stride + c + e] = (uint16_t)f32_to_bf16_rne(
                        a.add ? f[e] + bf16_to_f32(a.add[m * a.add_stride + c + e]) : f[e]);
              }
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    v = next(v + gridDim.x);
    if (v >= ids) break;
    mt_cur = mt;
    nt_cur = nt;
    tile_scales();
  }
  wait_vm<0>();  // no load into LDS outlives the workgroup
}

}  // namespace dense
}  // namespace moe
