// The router: gate product, scores, group-limited top-k and routing weights
// of a batch, in the form the layer stages (topk_idx with -1 for experts of
// other GPUs, topk_w).
//
//   l = x W^T                                  [T, E]
//   score = softmax(l) over E, or sigmoid(l)
//   choice = score + bias (sigmoid), l (softmax: the same order)
//   a group's value: the sum of its two largest choices (sigmoid), its
//   largest (softmax); the top_groups largest groups stay
//   the top_k largest choices of the groups that stay, in descending order
//   w_k = score_k (/ sum over the k) * scale
// Ties go to the lowest group and the lowest expert; a NaN ranks below
// every number.
//
// Two launches:
//  * router_gemm_kernel: FP32 logits on the BF16 MFMA, split over K where a
//    batch has few token tiles.  Experts are the MFMA rows and tokens its
//    columns (one MFMA is 32 experts x 32 tokens x 16).  The weights were laid
//    out at create as MFMA fragments, so a wave loads them straight into
//    registers (1 KB per instruction, L2 hits); the token rows go through LDS,
//    where every wave reads them.
//  * router_select_kernel: sums the K parts in order and selects, 16 lanes
//    per token and four tokens per wave, so that every cross-lane step is a
//    DPP row operation for four tokens at once.
//
// The ids are those of 64-bit arithmetic: where two choices that matter lie
// closer than twice the margin
//   B = kLogitMargin * (|x| max_e|w_e| / sqrt(H) + max_e|l_e|)
// the wave computes these experts' logits again in FP64 (two or three of
// them as a rule) and selects among FP64 choices.  |x| |w| / sqrt(H) is the
// size of a logit whose terms have random signs, and the FP32 error grows with
// it and with the logits themselves.
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include <new>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kGemmThreads = 512;
constexpr int kGemmWaves = 8;
constexpr int kKC = 128;            // K per chunk: one staged piece of the token rows
constexpr int kPieces = kKC / 8;    // 16-byte pieces per row and chunk
constexpr int kTileExperts = 256;   // experts per workgroup at most
constexpr int kTargetGroups = 256;  // workgroups a split over K aims at
constexpr int kMaxGroups = 16;
constexpr int kMaxTopK = 8;
constexpr float kLogitMargin = 0x1p-15f;

struct RouterGemmArgs {
  const uint16_t* x;
  int64_t x_stride;
  const uint8_t* w;  // fragments: [expert blocks of 32][H / 16][64 lanes][16 bytes]
  int32_t tokens, hidden;
  int32_t blocks;    // expert blocks of 32
  int32_t row;       // floats per logit row (padded experts)
  int32_t splits, chunks_per_split;
  float* part;       // [splits][tokens][row]
  float* norm2;      // [splits][tokens]: squared norms of the token rows' parts
};

struct RouterSelectArgs {
  const float* part;
  const float* norm2;
  const float* limits;  // [0] max |w_e|, [1] max |bias|
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* w;  // [E, H] as the caller holds it
  const float* bias;  // null: none
  int32_t tokens, hidden, experts, row, splits;
  int32_t top_k, groups, group_size, top_groups;
  int32_t sigmoid, renormalize;
  float scale;
  int32_t expert_base, local_experts;
  int32_t* idx;
  float* out_w;
  int32_t* ids;  // null: not wanted
};

// Position of 16-byte piece c of token row r in the staged chunk: rows of
// 256 bytes, pieces swizzled so that 16 lanes that read one piece of 16
// consecutive rows touch 16 different bank groups.
__device__ __forceinline__ int piece_at(int r, int c) { return r * kPieces + (c ^ (r & (kPieces - 1))); }

// BT tokens (32, 64 or 128) x WE * EW * 32 experts per workgroup.  Wave
// (we, wk): expert blocks [we * EW, +EW) of the tile, and K steps wk of every
// chunk (8 / WE wave groups share a chunk's eight 16-wide steps).
template <int BT, int WE, int EW>
__global__ __launch_bounds__(kGemmThreads, 1) void router_gemm_kernel(RouterGemmArgs a) {
  constexpr int WK = kGemmWaves / WE;
  constexpr int STEPS = kKC / 16 / WK;              // MFMA steps of a wave per chunk
  constexpr int TB = BT / 32;                       // token blocks
  constexpr int NP = BT * kPieces / kGemmThreads;   // staged pieces per thread
  static_assert(NP >= 1 && STEPS >= 1, "tile shape");
  constexpr int kStage = 2 * BT * kPieces, kRed = WE * EW * 4 * 64;  // 16-byte pieces
  __shared__ __attribute__((aligned(1024))) u32x4 lds[kStage > kRed ? kStage : kRed];
  u32x4* const stage[2] = {lds, lds + BT * kPieces};

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int we = wave % WE, wk = wave / WE;
  const int t0 = blockIdx.x * BT;
  const int eb0 = (int)blockIdx.y * (kTileExperts / 32) + we * EW;
  const int split = blockIdx.z;
  const int c0 = split * a.chunks_per_split;
  const int c1 = min(c0 + a.chunks_per_split, a.hidden / kKC);

  // token pieces of this thread: piece tid % 16 of rows tid / 16 + 32 j
  const int pc = tid & (kPieces - 1), pr = tid / kPieces;
  const uint16_t* xp[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int t = min(t0 + pr + j * (kGemmThreads / kPieces), a.tokens - 1);
    xp[j] = a.x + (int64_t)t * a.x_stride + pc * 8;
  }
  // weight fragments: expert blocks past the last read the last (their
  // results are not stored)
  const uint8_t* wp[EW];
  const int64_t steps_all = a.hidden / 16;
#pragma unroll
  for (int b = 0; b < EW; ++b)
    wp[b] = a.w + ((int64_t)min(eb0 + b, a.blocks - 1) * steps_all + wk * STEPS) * 1024 + lane * 16;

  f32x16 acc[EW][TB];
#pragma unroll
  for (int b = 0; b < EW; ++b)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[b][t][i] = 0.0f;
  float ss[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) ss[j] = 0.0f;

  u32x4 xr[2][NP];
  u32x4 wr[STEPS][EW];
  // Loads past the last chunk read the last again (L2 hits), so that every
  // chunk issues the same loads.
  auto load_x = [&](u32x4 (&r)[NP], int c) {
    const int64_t at = (int64_t)min(c, c1 - 1) * kKC;
#pragma unroll
    for (int j = 0; j < NP; ++j) r[j] = *reinterpret_cast<const u32x4*>(xp[j] + at);
  };
  auto load_w = [&](int s, int c) {
    const int64_t at = ((int64_t)min(c, c1 - 1) * (kKC / 16) + s) * 1024;
#pragma unroll
    for (int b = 0; b < EW; ++b) wr[s][b] = *reinterpret_cast<const u32x4*>(wp[b] + at);
  };
  auto put_x = [&](const u32x4 (&r)[NP], int buf) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      stage[buf][piece_at(pr + j * (kGemmThreads / kPieces), pc)] = r[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2 v = __builtin_bit_cast(bf16x2, r[j][i]);
        ss[j] = __builtin_amdgcn_fdot2_f32_bf16(v, v, ss[j], false);
      }
    }
  };
  auto compute = [&](int buf, int c) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int piece = (wk * STEPS + s) * 2 + (lane >> 5);
      bf16x8 bf[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t)
        bf[t] = __builtin_bit_cast(bf16x8, stage[buf][piece_at(t * 32 + (lane & 31), piece)]);
#pragma unroll
      for (int b = 0; b < EW; ++b)
#pragma unroll
        for (int t = 0; t < TB; ++t)
          acc[b][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wr[s][b]), bf[t], acc[b][t],
                                                              0, 0, 0);
      load_w(s, c + 1);  // this step of the next chunk
    }
  };

  // Chunk c is staged while chunk c - 1 is computed; its rows were loaded two
  // chunks before, its weights one.
  load_x(xr[0], c0);
  load_x(xr[1], c0 + 1);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) load_w(s, c0);
  put_x(xr[0], 0);
  load_x(xr[0], c0 + 2);
  __syncthreads();
  for (int c = c0; c < c1; c += 2) {
    if (c + 1 < c1) put_x(xr[1], 1);
    load_x(xr[1], c + 3);
    compute(0, c);
    __syncthreads();
    if (c + 1 >= c1) break;
    if (c + 2 < c1) put_x(xr[0], 0);
    load_x(xr[0], c + 4);
    compute(1, c + 1);
    __syncthreads();
  }

  // Sum of the wave groups, one 32-token block at a time: groups 1.. leave
  // theirs in LDS in turn, group 0 adds them in order.
  f32x4* const red = reinterpret_cast<f32x4*>(lds) + we * EW * 256 + lane;
  for (int g = 1; g < WK; ++g) {
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      if (wk == g) {
#pragma unroll
        for (int b = 0; b < EW; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            red[(b * 4 + i) * 64] =
                f32x4{acc[b][t][4 * i], acc[b][t][4 * i + 1], acc[b][t][4 * i + 2], acc[b][t][4 * i + 3]};
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int b = 0; b < EW; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = red[(b * 4 + i) * 64];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[b][t][4 * i + k] += v[k];
          }
      }
      __syncthreads();
    }
  }
  // squared norms of the rows' parts: 16 consecutive lanes hold one row
  if (blockIdx.y == 0) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float v = ss[j];
#pragma unroll
      for (int m = 1; m < kPieces; m <<= 1) v += __shfl_xor(v, m, kPieces);
      const int t = t0 + pr + j * (kGemmThreads / kPieces);
      if (pc == 0 && t < a.tokens) a.norm2[(int64_t)split * a.tokens + t] = v;
    }
  }
  if (wk != 0) return;
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int tok = t0 + t * 32 + (lane & 31);
    if (tok >= a.tokens) continue;
    float* row = a.part + ((int64_t)split * a.tokens + tok) * a.row;
#pragma unroll
    for (int b = 0; b < EW; ++b) {
      if (eb0 + b >= a.blocks) continue;
      // MFMA output i of a lane: expert 8 (i / 4) + 4 (lane / 32) + i % 4
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(row + (eb0 + b) * 32 + 8 * i + 4 * (lane >> 5)) =
            f32x4{acc[b][t][4 * i], acc[b][t][4 * i + 1], acc[b][t][4 * i + 2], acc[b][t][4 * i + 3]};
    }
  }
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------

// v of the lane that DPP control CTRL names, within a row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;  // quad_perm, quad_perm, ...

__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  return max(v, dpp<kMirror>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, dpp<kXor1>(v));
  v = min(v, dpp<kXor2>(v));
  v = min(v, dpp<kHalfMirror>(v));
  return min(v, dpp<kMirror>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  return v + dppf<kMirror>(v);
}

// Floats in the order of their values as unsigned integers.  NaN is 1, below
// every number; 0 stands for "not a candidate".
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 counts as +0
  return f != f ? 1u : ((u & 0x80000000u) ? ~u : (u | 0x80000000u));
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return k < 2u ? -INFINITY : __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float sigmoid_fast(float l) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * l));
}

// Order of LDS accesses between the lanes of one wave (whose LDS operations
// complete in order): a fence for the compiler only.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One flagged token, by a whole wave: the choices that lie too close are
// computed again in FP64.  All values are wave-uniform unless they carry a
// lane.
struct Exact {
  double* logit;    // LDS [experts]: FP32 logits, FP64 where recomputed
  double* choice;   // LDS [experts]
  uint32_t* mark;   // LDS [32]: experts to recompute
  const RouterSelectArgs& a;
  int64_t t;
  double margin;    // Bk: bound on a choice's error
  uint32_t kept;    // groups that stay
  int lane;

  __device__ double choice_of(double l, int e) const {
    double c = l;
    if (a.sigmoid) c = 1.0 / (1.0 + exp(-l)) + (a.bias ? (double)a.bias[e] : 0.0);
    return c != c ? -INFINITY : c;
  }
  __device__ bool candidate(int e) const { return a.groups == 1 || ((kept >> (e / a.group_size)) & 1u); }

  // FP64 logits of the marked experts, then no marks.
  __device__ void recompute() {
    wave_fence();
    for (int w = 0; w < (a.experts + 31) / 32; ++w) {
      uint32_t bits = __builtin_amdgcn_readfirstlane(mark[w]);
      while (bits) {
        const int e = w * 32 + __builtin_ctz(bits);
        bits &= bits - 1;
        const uint16_t* x = a.x + t * a.x_stride;
        const uint16_t* wr = a.w + (int64_t)e * a.hidden;
        double s = 0.0;
#pragma unroll 4
        for (int i = lane * 8; i < a.hidden; i += 512) {
          const u32x4 xv = *reinterpret_cast<const u32x4*>(x + i), wv = *reinterpret_cast<const u32x4*>(wr + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s = fma((double)bf16_to_f32(xv[k] & 0xffffu), (double)bf16_to_f32(wv[k] & 0xffffu), s);
            s = fma((double)bf16_to_f32(xv[k] >> 16), (double)bf16_to_f32(wv[k] >> 16), s);
          }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
        if (lane == 0) {
          logit[e] = s;
          choice[e] = choice_of(s, e);
        }
      }
    }
    wave_fence();
    if (lane < 32) mark[lane] = 0u;
    wave_fence();
  }

  // Largest candidate after (c, e) in descending order of choice, lowest
  // expert first; e < 0 when there is none.
  __device__ void next(double& c, int& e) const {
    double best = 0.0;
    int at = 0x7fffffff;
    for (int i = lane; i < a.experts; i += 64) {
      const double v = choice[i];
      if (!candidate(i) || !(e < 0 || v < c || (v == c && i > e))) continue;
      if (at == 0x7fffffff || v > best) {
        best = v;
        at = i;
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double ov = __shfl_xor(best, m, 64);
      const int oe = __shfl_xor(at, m, 64);
      if (oe != 0x7fffffff && (at == 0x7fffffff || ov > best || (ov == best && oe < at))) {
        best = ov;
        at = oe;
      }
    }
    c = best;
    e = __builtin_amdgcn_readfirstlane(at == 0x7fffffff ? -1 : at);
  }

  // Group values (lane g holds group g's) and the groups that stay.  With
  // `mark_close` the members that decide a border closer than the margins
  // are marked; returns whether there is such a border.
  __device__ bool pick_groups(bool mark_close) {
    const int n = a.group_size;
    double k1 = -INFINITY, k2 = -INFINITY;
    if (lane < a.groups)
      for (int i = lane * n; i < lane * n + n; ++i) {
        const double v = choice[i];
        if (v > k1) {
          k2 = k1;
          k1 = v;
        } else if (v > k2) {
          k2 = v;
        }
      }
    const bool two = a.sigmoid && n > 1;
    const double gv = two ? k1 + k2 : k1;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(gv, g, 64);
      rank += (o > gv || (o == gv && g < lane)) ? 1 : 0;
    }
    const bool in = lane < a.groups && rank < a.top_groups;
    kept = (uint32_t)__ballot(in);
    double lo = in ? gv : INFINITY;                           // smallest value that stays
    double hi = (lane < a.groups && !in) ? gv : -INFINITY;    // largest that does not
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      lo = fmin(lo, __shfl_xor(lo, m, 64));
      hi = fmax(hi, __shfl_xor(hi, m, 64));
    }
    const double g4 = 4.0 * margin;
    if (!mark_close || !(lo - hi <= g4)) return false;
    if (lane < a.groups && (fabs(gv - lo) <= g4 || fabs(gv - hi) <= g4)) {
      const double from = (two ? k2 : k1) - 2.0 * margin;
      for (int i = lane * n; i < lane * n + n; ++i)
        if (choice[i] >= from) atomicOr(&mark[i >> 5], 1u << (i & 31));
    }
    return true;
  }

  // The ids of the K largest, ids[k] in lane k.
  __device__ int select() {
    if (lane < 32) mark[lane] = 0u;
    wave_fence();
    if (a.groups > 1 && pick_groups(true)) {
      recompute();
      pick_groups(false);
    }
    // neighbours in the order of the choices that lie closer than the margins
    double c = 0.0, pc = 0.0, border = 0.0;
    int e = -1, pe = -1;
    bool any = false;
    for (int k = 0;; ++k) {
      next(c, e);
      if (e < 0) break;
      if (k > 0 && pc - c <= 2.0 * margin) {
        any = true;
        if (lane == 0) {
          atomicOr(&mark[e >> 5], 1u << (e & 31));
          atomicOr(&mark[pe >> 5], 1u << (pe & 31));
        }
      }
      if (k == a.top_k - 1) border = c;
      if (k >= a.top_k && c < border - 2.0 * margin) break;
      pc = c;
      pe = e;
    }
    if (any) recompute();
    int mine = -1;
    c = 0.0;
    e = -1;
    for (int k = 0; k < a.top_k; ++k) {
      next(c, e);
      if (lane == k) mine = e;
    }
    return mine;
  }
};

// EPL experts per lane: lane q of a token's 16 holds experts [q EPL, +EPL).
template <int EPL>
__global__ __launch_bounds__(256) void router_select_kernel(RouterSelectArgs a) {
  __shared__ double lds_logit[4][16 * EPL];
  __shared__ double lds_choice[4][16 * EPL];
  __shared__ uint32_t lds_mark[4][32];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t tw = ((int64_t)blockIdx.x * 4 + wave) * 4;  // first token of the wave
  if (tw >= a.tokens) return;
  const int64_t t = tw + (lane >> 4);
  const bool live = t < a.tokens;
  const int64_t tt = live ? t : a.tokens - 1;

  float l[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) l[j] = 0.0f;
  float n2 = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float* p = a.part + ((int64_t)s * a.tokens + tt) * a.row + q * EPL;
    if constexpr (EPL >= 4) {
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) l[j + k] += v[k];
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) l[j] += p[j];
    }
    n2 += a.norm2[(int64_t)s * a.tokens + tt];
  }

  // choices as ordered integers, and the margin of a choice
  uint32_t key[EPL];
  float largest = 0.0f;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = q * EPL + j;
    const bool in = e < a.experts;
    float c = l[j];
    if (a.sigmoid) c = sigmoid_fast(l[j]) + (a.bias && in ? a.bias[e] : 0.0f);
    key[j] = in ? ordered(c) : 0u;
    if (in) {
      largest = fmaxf(largest, fabsf(l[j]));
      top = fmaxf(top, l[j]);
    }
  }
  largest = __uint_as_float(row_max(__float_as_uint(largest)));  // not negative
  float margin = kLogitMargin * (sqrtf(n2) * a.limits[0] * rsqrtf((float)a.hidden) + largest);
  // a sigmoid's slope is at most 1/4; evaluating it and adding the bias costs
  // less than 2^-20 of their size
  if (a.sigmoid) margin = 0.25f * margin + 0x1p-20f * (1.0f + a.limits[1]);
  const bool guard = margin < INFINITY;  // not for rows with a NaN or an overflow
  bool close = false;

  if (a.groups > 1) {
    const int n = a.group_size;
    const bool two = a.sigmoid && n > 1;
    float gv = -INFINITY;
    for (int g = 0; g < a.groups; ++g) {
      uint32_t k1 = 0, k2 = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t v = (uint32_t)(q * EPL + j - g * n) < (uint32_t)n ? key[j] : 0u;
        k2 = max(k2, min(k1, v));
        k1 = max(k1, v);
      }
      auto merge = [&](uint32_t o1, uint32_t o2) {
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
      };
      merge(dpp<kXor1>(k1), dpp<kXor1>(k2));
      merge(dpp<kXor2>(k1), dpp<kXor2>(k2));
      merge(dpp<kHalfMirror>(k1), dpp<kHalfMirror>(k2));
      merge(dpp<kMirror>(k1), dpp<kMirror>(k2));
      if (q == g) gv = two ? unordered(k1) + unordered(k2) : unordered(k1);
    }
    // groups ahead of this lane's, by rotating the row
    int rank = 0;
    auto ahead = [&](float o, int lane_from) { rank += (o > gv || (o == gv && lane_from < q)) ? 1 : 0; };
#define MOE_ROT(N) ahead(dppf<0x120 + N>(gv), (q - N) & 15)
    MOE_ROT(1); MOE_ROT(2); MOE_ROT(3); MOE_ROT(4); MOE_ROT(5); MOE_ROT(6); MOE_ROT(7); MOE_ROT(8);
    MOE_ROT(9); MOE_ROT(10); MOE_ROT(11); MOE_ROT(12); MOE_ROT(13); MOE_ROT(14); MOE_ROT(15);
#undef MOE_ROT
    const bool in = q < a.groups && rank < a.top_groups;
    const uint32_t kept = (uint32_t)(__ballot(in) >> (lane & 48)) & 0xffffu;
    const uint32_t lo = row_min(in ? ordered(gv) : 0xffffffffu);
    const uint32_t hi = row_max(q < a.groups && !in ? ordered(gv) : 0u);
    close = hi > 1u && unordered(lo) - unordered(hi) <= 4.0f * margin;
    const uint32_t magic = ((1u << 20) + n - 1) / n;  // e / n for e and n up to 1024
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint32_t g = ((uint32_t)(q * EPL + j) * magic) >> 20;
      if (!((kept >> g) & 1u)) key[j] = 0u;
    }
  }

  // the K largest in order, lane k of the row keeping the k-th, and one more
  // to see whether it lies close
  int id = -1;
  float mine = 0.0f;
  float before = INFINITY;
  for (int k = 0; k <= a.top_k; ++k) {
    uint32_t bk = 0;
    int bj = 0;
    float bl = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
        bl = l[j];
      }
    const uint32_t m = row_max(bk);
    if (m > 1u) {
      const float c = unordered(m);
      close |= before - c <= 2.0f * margin;
      before = c;
    }
    if (k == a.top_k) break;
    const uint32_t e = row_min(bk == m ? (uint32_t)(q * EPL + bj) : 0xffffffffu);
    const float el = __shfl(bl, (lane & 48) + (int)(e / EPL), 64);
    if (q == k) {
      id = (int)e;
      mine = el;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if ((uint32_t)(q * EPL + j) == e) key[j] = 0u;
  }

  // tokens with choices too close to call
  uint64_t todo = __ballot(close && guard && live && q == 0);
  while (todo) {
    const int from = __builtin_ctzll(todo);  // first lane of the token's row
    todo &= todo - 1;
    Exact x{lds_logit[wave], lds_choice[wave], lds_mark[wave], a, tw + (from >> 4), 0.0, 0xffffu, lane};
    x.margin = (double)__shfl(margin, from, 64);
    if ((lane & 48) == from) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) x.logit[q * EPL + j] = (double)l[j];
    }
    wave_fence();
    for (int e = lane; e < a.experts; e += 64) x.choice[e] = x.choice_of(x.logit[e], e);
    wave_fence();
    const int got = __shfl(x.select(), q, 64);  // lane k of the wave holds the k-th
    if ((lane & 48) == from && q < a.top_k) {
      id = got;
      mine = (float)x.logit[got];
    }
    wave_fence();
  }

  // routing weights
  const bool slot = q < a.top_k;
  float w;
  if (a.sigmoid) {
    w = slot ? 1.0f / (1.0f + expf(-mine)) : 0.0f;
  } else if (a.renormalize) {  // the sum over all experts cancels
    const float m = unordered(row_max(slot ? ordered(mine) : 0u));
    w = slot ? expf(mine - m) : 0.0f;
  } else {
    const float m = unordered(row_max(ordered(top)));
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (q * EPL + j < a.experts) z += expf(l[j] - m);
    z = row_sum(z);
    w = slot ? expf(mine - m) / z : 0.0f;
  }
  if (a.renormalize) {
    const float sum = row_sum(w);
    w = sum != 0.0f ? w / sum : 0.0f;
  }
  if (live && slot) {
    const int64_t at = t * a.top_k + q;
    const int here = id - a.expert_base;
    a.idx[at] = here >= 0 && here < a.local_experts ? here : -1;
    a.out_w[at] = w * a.scale;
    if (a.ids) a.ids[at] = id;
  }
}

// ---------------------------------------------------------------------------
// Create: weight fragments and limits
// ---------------------------------------------------------------------------

// One thread per 16-byte piece of the fragments: block eb, step s, lane l
// holds expert 32 eb + l % 32, K elements 16 s + 8 (l / 32) + 0..7; experts
// past the last are zero.
__global__ __launch_bounds__(256) void router_tile_kernel(const uint16_t* w, u32x4* dst, int64_t pieces, int experts,
                                                          int hidden) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= pieces) return;
  const int lane = (int)(c & 63);
  const int64_t step = (c >> 6) % (hidden / 16);
  const int e = (int)((c >> 6) / (hidden / 16)) * 32 + (lane & 31);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (e < experts) v = *reinterpret_cast<const u32x4*>(w + (int64_t)e * hidden + step * 16 + 8 * (lane >> 5));
  dst[c] = v;
}

// limits[0] = max_e |w_e|, limits[1] = max_e |bias_e|; one wave per expert.
// A maximum does not depend on the order of the atomics; as bits, a NaN is
// larger than every number.
__global__ __launch_bounds__(64) void router_limits_kernel(const uint16_t* w, const float* bias, int hidden,
                                                           uint32_t* limits) {
  const int e = blockIdx.x;
  float s = 0.0f;
  for (int i = threadIdx.x; i < hidden; i += 64) {
    const float v = bf16_to_f32(w[(int64_t)e * hidden + i]);
    s = fmaf(v, v, s);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
  if (threadIdx.x == 0) {
    atomicMax(&limits[0], __float_as_uint(sqrtf(s)) & 0x7fffffffu);
    if (bias) atomicMax(&limits[1], __float_as_uint(bias[e]) & 0x7fffffffu);
  }
}

// Token tile and K split of a batch.
struct Plan {
  int bt;
  int splits, chunks_per_split;
};

Plan plan_for(const moe_router_config_t& c, int64_t tokens) {
  Plan p;
  p.bt = tokens <= 1024 ? 32 : (tokens <= 8192 ? 64 : 128);
  const int64_t tiles = (tokens + p.bt - 1) / p.bt * ((c.num_experts + kTileExperts - 1) / kTileExperts);
  const int chunks = c.hidden / kKC;
  int64_t want = kTargetGroups / tiles;
  want = want < 1 ? 1 : (want > chunks ? chunks : want);
  p.chunks_per_split = (int)((chunks + want - 1) / want);
  p.splits = (chunks + p.chunks_per_split - 1) / p.chunks_per_split;
  return p;
}

// Floats per logit row: 16 lanes x a power of two.
int row_of(int experts) {
  int r = 32;
  while (r < experts) r <<= 1;
  return r;
}

struct RouterLayout {
  size_t w, limits, part, norm2, total;
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

RouterLayout router_layout(const moe_router_config_t& c, int64_t max_rows) {
  RouterLayout L;
  // largest splits x tokens of any batch: within a token tile size the split
  // falls as the tokens grow, so the tile count times the split is bounded
  int64_t rows = max_rows;
  const int64_t edges[3] = {1024, 8192, max_rows};
  for (int64_t e : edges) {
    const int64_t t = e < max_rows ? e : max_rows;
    const Plan p = plan_for(c, t);
    const int64_t bound = (int64_t)kTargetGroups * p.bt, all = (int64_t)(c.hidden / kKC) * t;
    const int64_t r = bound < all ? bound : all;
    rows = r > rows ? r : rows;
  }
  L.w = 0;
  L.limits = L.w + align256((size_t)((c.num_experts + 31) / 32) * 32 * c.hidden * 2);
  L.part = L.limits + 256;
  L.norm2 = L.part + align256((size_t)rows * row_of(c.num_experts) * 4);
  L.total = L.norm2 + align256((size_t)rows * 4);
  return L;
}

moe_status_t validate(const moe_router_config_t* c, int32_t max_rows) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
  if (c->hidden <= 0) return fail(MOE_ERR_INVALID_ARG, "hidden (%d) must be positive", c->hidden);
  if (c->hidden % 128 || c->hidden > 16384)
    return fail(MOE_ERR_UNSUPPORTED, "hidden (%d) must be a multiple of 128, at most 16384", c->hidden);
  if (c->num_experts < 1 || c->num_experts > kMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "num_experts %d outside [1, %d]", c->num_experts, kMaxExperts);
  if (c->top_k < 1 || c->top_k > kMaxTopK)
    return fail(MOE_ERR_UNSUPPORTED, "top_k %d outside [1, %d]", c->top_k, kMaxTopK);
  if (c->top_k > c->num_experts)
    return fail(MOE_ERR_INVALID_ARG, "top_k %d exceeds num_experts %d", c->top_k, c->num_experts);
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "unknown score %d", c->score);
  if (c->num_groups < 1 || c->num_groups > kMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "num_groups %d outside [1, %d]", c->num_groups, kMaxGroups);
  if (c->num_experts % c->num_groups)
    return fail(MOE_ERR_INVALID_ARG, "num_experts %d is not a multiple of num_groups %d", c->num_experts, c->num_groups);
  if (c->top_groups < 1 || c->top_groups > c->num_groups)
    return fail(MOE_ERR_INVALID_ARG, "top_groups %d outside [1, %d]", c->top_groups, c->num_groups);
  if (c->num_experts / c->num_groups * c->top_groups < c->top_k)
    return fail(MOE_ERR_INVALID_ARG, "top_groups %d hold fewer than top_k %d experts", c->top_groups, c->top_k);
  if (c->renormalize != 0 && c->renormalize != 1)
    return fail(MOE_ERR_INVALID_ARG, "renormalize must be 0 or 1");
  if (!isfinite(c->scale)) return fail(MOE_ERR_INVALID_ARG, "scale must be finite");
  if (c->expert_base < 0 || c->local_experts < 1 || c->local_experts > c->num_experts ||
      c->expert_base > c->num_experts - c->local_experts)
    return fail(MOE_ERR_INVALID_ARG, "local experts [%d, +%d) outside the %d experts", c->expert_base,
                c->local_experts, c->num_experts);
  if (max_rows < 1) return fail(MOE_ERR_INVALID_ARG, "max_rows %d must be >= 1", max_rows);
  if (max_rows > 1 << 24) return fail(MOE_ERR_UNSUPPORTED, "max_rows %d above 2^24", max_rows);
  return MOE_OK;
}

template <int BT>
void launch_gemm(const RouterGemmArgs& g, dim3 grid, hipStream_t s) {
  const dim3 block(kGemmThreads);
  if (g.blocks > 4)
    hipLaunchKernelGGL((router_gemm_kernel<BT, 4, 2>), grid, block, 0, s, g);
  else if (g.blocks > 2)
    hipLaunchKernelGGL((router_gemm_kernel<BT, 4, 1>), grid, block, 0, s, g);
  else if (g.blocks > 1)
    hipLaunchKernelGGL((router_gemm_kernel<BT, 2, 1>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((router_gemm_kernel<BT, 1, 1>), grid, block, 0, s, g);
}

}  // namespace
}  // namespace moe

struct moe_router {
  moe_router_config_t cfg;
  const uint16_t* w;
  const float* bias;
  uint8_t* ws;
  moe::RouterLayout L;
  int32_t max_rows;
};

namespace {
moe_status_t router_hip_fail(const char* what) {
  return moe::fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(hipGetLastError()));
}
}  // namespace

extern "C" moe_status_t moe_router_workspace_query(const moe_router_config_t* cfg, int32_t max_rows,
                                                   size_t* ws_bytes) {
  moe::clear_error();
  const moe_status_t s = moe::validate(cfg, max_rows);
  if (s != MOE_OK) return s;
  if (!ws_bytes) return moe::fail(MOE_ERR_INVALID_ARG, "ws_bytes is NULL");
  *ws_bytes = moe::router_layout(*cfg, max_rows).total;
  return MOE_OK;
}

extern "C" moe_status_t moe_router_create(const moe_router_config_t* cfg, int32_t max_rows, const void* weight,
                                          const float* bias, void* workspace, size_t ws_bytes, void* stream,
                                          moe_router_t** out) {
  moe::clear_error();
  moe_status_t st = moe::validate(cfg, max_rows);
  if (st != MOE_OK) return st;
  if (!out) return moe::fail(MOE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!weight || ((uintptr_t)weight & 15))
    return moe::fail(MOE_ERR_INVALID_ARG, "weight must be non-NULL and 16-byte aligned");
  if ((uintptr_t)bias & 3) return moe::fail(MOE_ERR_INVALID_ARG, "bias must be 4-byte aligned");
  if (bias && cfg->score != MOE_SCORE_SIGMOID)
    return moe::fail(MOE_ERR_UNSUPPORTED, "a selection bias needs sigmoid scores");
  if (!workspace || ((uintptr_t)workspace & 255))
    return moe::fail(MOE_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  const moe::RouterLayout L = moe::router_layout(*cfg, max_rows);
  if (ws_bytes < L.total)
    return moe::fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes, L.total);
  moe_router* r = new (std::nothrow) moe_router();
  if (!r) return moe::fail(MOE_ERR_INVALID_ARG, "out of host memory");
  r->cfg = *cfg;
  r->w = static_cast<const uint16_t*>(weight);
  r->bias = bias;
  r->ws = static_cast<uint8_t*>(workspace);
  r->L = L;
  r->max_rows = max_rows;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t pieces = (int64_t)((cfg->num_experts + 31) / 32) * (cfg->hidden / 16) * 64;
  uint32_t* limits = reinterpret_cast<uint32_t*>(r->ws + L.limits);
  bool ok = moe::launch_fill_zero(limits, 64, stream) == 0;
  if (ok) {
    hipLaunchKernelGGL(moe::router_tile_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, r->w,
                       reinterpret_cast<moe::u32x4*>(r->ws + L.w), pieces, cfg->num_experts, cfg->hidden);
    hipLaunchKernelGGL(moe::router_limits_kernel, dim3(cfg->num_experts), dim3(64), 0, s, r->w, bias, cfg->hidden,
                       limits);
    ok = hipGetLastError() == hipSuccess;
  }
  if (!ok) {
    delete r;
    return router_hip_fail("router weight launch");
  }
  *out = r;
  return MOE_OK;
}

extern "C" moe_status_t moe_router_forward(moe_router_t* r, const void* x, int64_t x_stride, int32_t num_tokens,
                                           int32_t* topk_idx, float* topk_w, int32_t* ids, void* stream) {
  moe::clear_error();
  if (!r) return moe::fail(MOE_ERR_INVALID_ARG, "router is NULL");
  if (num_tokens < 0) return moe::fail(MOE_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens > r->max_rows)
    return moe::fail(MOE_ERR_CAPACITY, "num_tokens %d exceeds max_rows %d", num_tokens, r->max_rows);
  if (num_tokens == 0) return MOE_OK;
  const moe_router_config_t& c = r->cfg;
  if (!x || !topk_idx || !topk_w) return moe::fail(MOE_ERR_INVALID_ARG, "x, topk_idx and topk_w must be non-NULL");
  if ((uintptr_t)x & 15) return moe::fail(MOE_ERR_INVALID_ARG, "x must be 16-byte aligned");
  if (((uintptr_t)topk_idx | (uintptr_t)topk_w | (uintptr_t)ids) & 3)
    return moe::fail(MOE_ERR_INVALID_ARG, "topk_idx, topk_w and ids must be 4-byte aligned");
  if (num_tokens > 1 && (x_stride < c.hidden || x_stride % 8))
    return moe::fail(MOE_ERR_INVALID_ARG, "x_stride %lld", (long long)x_stride);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe::Plan p = moe::plan_for(c, num_tokens);
  moe::RouterGemmArgs g;
  g.x = static_cast<const uint16_t*>(x);
  g.x_stride = x_stride;
  g.w = r->ws + r->L.w;
  g.tokens = num_tokens;
  g.hidden = c.hidden;
  g.blocks = (c.num_experts + 31) / 32;
  g.row = moe::row_of(c.num_experts);
  g.splits = p.splits;
  g.chunks_per_split = p.chunks_per_split;
  g.part = reinterpret_cast<float*>(r->ws + r->L.part);
  g.norm2 = reinterpret_cast<float*>(r->ws + r->L.norm2);
  const dim3 grid((num_tokens + p.bt - 1) / p.bt, (c.num_experts + moe::kTileExperts - 1) / moe::kTileExperts,
                  p.splits);
  if (p.bt == 32)
    moe::launch_gemm<32>(g, grid, s);
  else if (p.bt == 64)
    moe::launch_gemm<64>(g, grid, s);
  else
    moe::launch_gemm<128>(g, grid, s);
  moe::RouterSelectArgs a;
  a.part = g.part;
  a.norm2 = g.norm2;
  a.limits = reinterpret_cast<const float*>(r->ws + r->L.limits);
  a.x = g.x;
  a.x_stride = x_stride;
  a.w = r->w;
  a.bias = r->bias;
  a.tokens = num_tokens;
  a.hidden = c.hidden;
  a.experts = c.num_experts;
  a.row = g.row;
  a.splits = p.splits;
  a.top_k = c.top_k;
  a.groups = c.top_groups == c.num_groups ? 1 : c.num_groups;  // every group stays
  a.group_size = c.num_experts / c.num_groups;
  a.top_groups = c.top_groups;
  a.sigmoid = c.score == MOE_SCORE_SIGMOID;
  a.renormalize = c.renormalize;
  a.scale = c.scale;
  a.expert_base = c.expert_base;
  a.local_experts = c.local_experts;
  a.idx = topk_idx;
  a.out_w = topk_w;
  a.ids = ids;
  const dim3 sg((num_tokens + 15) / 16), sb(256);
  switch (g.row) {
    case 32: hipLaunchKernelGGL(moe::router_select_kernel<2>, sg, sb, 0, s, a); break;
    case 64: hipLaunchKernelGGL(moe::router_select_kernel<4>, sg, sb, 0, s, a); break;
    case 128: hipLaunchKernelGGL(moe::router_select_kernel<8>, sg, sb, 0, s, a); break;
    case 256: hipLaunchKernelGGL(moe::router_select_kernel<16>, sg, sb, 0, s, a); break;
    case 512: hipLaunchKernelGGL(moe::router_select_kernel<32>, sg, sb, 0, s, a); break;
    default: hipLaunchKernelGGL(moe::router_select_kernel<64>, sg, sb, 0, s, a); break;
  }
  if (hipGetLastError() != hipSuccess) return moe::fail(MOE_ERR_HIP, "router launch failed");
  return MOE_OK;
}

extern "C" moe_status_t moe_router_destroy(moe_router_t* r) {
  moe::clear_error();
  delete r;
  return MOE_OK;
}
