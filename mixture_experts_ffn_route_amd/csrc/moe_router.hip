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
// Its floor is the token rows read once and the product on the MFMA: T=4096
// H=7168 E=256 9 and 11 us, T=32768 68 and 89.  A call takes 10.5 us (T=1), 26
// (512), 47 (4096), 180 (32768), of which the product 5, 9, 23 and 135 (1 and 5
// for sampling its partial sums at the last two) and the 64-bit decisions about
// 10 from T=512 on, 20 at the last: two FP64 logits take a wave 4 us (2 x 7168
// products, converted and added one by one), a token whose groups or experts lie
// close needs two to six of them, and the launch waits for the slowest.  With a
// tenth of the bound below a call would take 44 (4096) and 170 us.
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
//    DPP row operation for four tokens at once.  Smaller batches take 32 or 64
//    lanes, and more than 256 experts too, so that a lane never holds more than
//    16: with 32 and 64 of them it spilled its registers (E=512 H=4096 T=4096 69
//    us against 49, E=1024 T=1 26 against 13).
//
// The ids are those of 64-bit arithmetic: where two choices that matter lie
// closer than the bounds on their FP32 errors (and, of a sigmoid, on what
// evaluating it and adding its own bias may cost), the wave computes these
// experts' logits again in FP64 (two or three of them as a rule) and selects
// among FP64 choices.
//
// The bound on a logit's error follows its sum.  With u = 2^-24, a step of an
// accumulator (one MFMA: C + 16 products, added in two halves) errs by at most
//   kStepError u |partial sum| + kProductError u max|product|
// (measured: 2.0, and 2.9 where all products are lost beside C; 7.0 for a
// large product beside small ones), so the logit by
//   u (kStepError sum_k |p_k| + kProductError |x| V),
//   V = max_e sqrt(sum over the steps of max w_e^2) >= sum_k max|product| / |x|.
// The product samples the partial sums p_k, the largest of each token over the
// experts, every S steps.  Between two samples a partial sum differs from the
// nearer one by the steps between, each at most |x_k| |w_k|; every step stands
// between at most S / 2 partial sums (and the half of its own) and their
// sample, and sum |x_k| |w_k| <= |x| |w|:
//   sum_k |p_k| <= S sum |samples| + (S / 2 + 1 / 2) |x| |w|.
// So rows of large terms that cancel are covered like any other.  For rows and
// gates of random signs, H = 7168, the bound is 1.4e-4 (T=4096, two K parts) to
// 2.1e-4 (one part, 8 accumulators a wave) of a logit's size |x| |w| / sqrt(H).
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include <new>
#include <type_traits>

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
constexpr int kTargetGroups = 256;  // workgroups a split over K aims at
constexpr int kMaxSplits = 8;
constexpr int kMaxGroups = 16;
constexpr int kMaxTopK = 8;
constexpr int kMaxPerLane = 16;     // experts of a lane of the selection
constexpr float kStepError = 3.0f, kProductError = 8.0f;  // in units of 2^-24

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
  float* partial;    // [expert tiles][splits][tokens]: sums of |partial sum| over the steps
};

struct RouterSelectArgs {
  const float* part;
  const float* norm2;
  const float* partial;
  int32_t tiles;        // expert tiles of `partial`
  float steps;          // of all accumulators together
  float slack;          // steps between samples, as above
  const float* limits;  // [0] max |w_e|, [1] V
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* w;  // [E, H] as the caller holds it
  const float* bias;    // [row]: zeros where there is none
  int32_t tokens, hidden, row, splits;
  int32_t top_k, groups, group_size, top_groups;
  int32_t lane_shift, per_lane;  // log2 of the lanes per group; see router_select_kernel
  int32_t sigmoid, renormalize;
  int32_t biased;
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

// Chunks of 128 columns per sample of the partial sums, for so many accumulators
// a wave: a sample looks at all of them.
constexpr int samples_every(int accumulators) { return accumulators >= 8 ? 2 : 1; }

// BT tokens (32, 64 or 128) x WE * EW * 32 experts per workgroup.  Wave
// (we, wk): expert blocks [we * EW, +EW) of the tile, and K steps wk of every
// chunk (8 / WE wave groups share a chunk's eight 16-wide steps).  ONCE: no
// other workgroup reads these token rows, so they are loaded non-temporally
// and leave the L2 to the weights (T=32768, H=7168, E=256: 172 -> 164 us with
// the selection; where a second workgroup reads them, T=4096, 44 -> 48 us).
template <int BT, int WE, int EW, bool ONCE = false>
__global__ __launch_bounds__(kGemmThreads, 1) void router_gemm_kernel(RouterGemmArgs a) {
  constexpr int WK = kGemmWaves / WE;
  constexpr int STEPS = kKC / 16 / WK;              // MFMA steps of a wave per chunk
  constexpr int TB = BT / 32;                       // token blocks
  constexpr int NP = BT * kPieces / kGemmThreads;   // staged pieces per thread
  constexpr int NS = samples_every(EW * TB);        // chunks per sample of the partial sums
  static_assert(NP >= 1 && STEPS >= 1, "tile shape");
  constexpr int kStage = 3 * BT * kPieces, kRed = WE * EW * 4 * 64;  // 16-byte pieces
  __shared__ __attribute__((aligned(1024))) u32x4 lds[kStage > kRed ? kStage : kRed];
  __shared__ uint32_t partial[WK][BT];  // per wave group and token, as bits
  static_assert(WK > 1, "the wave groups' sum has the barriers that partial needs");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int we = wave % WE, wk = wave / WE;
  for (int i = tid; i < WK * BT; i += kGemmThreads) (&partial[0][0])[i] = 0u;
  const int t0 = blockIdx.x * BT;
  const int eb0 = (int)blockIdx.y * (WE * EW) + we * EW;
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
    for (int j = 0; j < NP; ++j) {
      const u32x4* from = reinterpret_cast<const u32x4*>(xp[j] + at);
      r[j] = ONCE ? __builtin_nontemporal_load(from) : *from;
    }
  };
  auto load_w = [&](int s, int c) {
    const int64_t at = ((int64_t)min(c, c1 - 1) * (kKC / 16) + s) * 1024;
#pragma unroll
    for (int b = 0; b < EW; ++b) wr[s][b] = *reinterpret_cast<const u32x4*>(wp[b] + at);
  };
  auto put_x = [&](const u32x4 (&r)[NP], int buf) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      lds[buf * (BT * kPieces) + piece_at(pr + j * (kGemmThreads / kPieces), pc)] = r[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2 v = __builtin_bit_cast(bf16x2, r[j][i]);
        ss[j] = __builtin_amdgcn_fdot2_f32_bf16(v, v, ss[j], false);
      }
    }
  };
  auto load_b = [&](bf16x8 (&r)[TB], int buf, int step) {
    const int piece = (wk * STEPS + step) * 2 + (lane >> 5);
#pragma unroll
    for (int t = 0; t < TB; ++t)
      r[t] = __builtin_bit_cast(bf16x8, lds[buf * (BT * kPieces) + piece_at(t * 32 + (lane & 31), piece)]);
  };
  // Chunk c's rows are put into LDS during chunk c - 2, loaded into registers
  // two chunks before that; its weights are loaded during chunk c - 1.  With
  // three buffers the fragments of a chunk's first step are read during the
  // last step of the chunk before, so no wave stands still after the barrier.
  // The scheduling barriers keep each step's weight loads in their step: left
  // alone, the compiler issues them all at the end of the chunk, right before
  // they are needed.
  bf16x8 bf[2][TB];
  load_x(xr[0], c0);
  load_x(xr[1], c0 + 1);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) load_w(s, c0);
  put_x(xr[0], 0);
  load_x(xr[0], c0 + 2);
  if (c0 + 1 < c1) put_x(xr[1], 1);
  load_x(xr[1], c0 + 3);
  __syncthreads();
  load_b(bf[0], 0, 0);
  int buf = 0;  // of chunk c
  auto chunk = [&](u32x4 (&x)[NP], int c) {
    const int next = buf == 2 ? 0 : buf + 1, after = next == 2 ? 0 : next + 1;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + 1 < STEPS)
        load_b(bf[(s + 1) & 1], buf, s + 1);
      else
        load_b(bf[(s + 1) & 1], next, 0);
#pragma unroll
      for (int b = 0; b < EW; ++b)
#pragma unroll
        for (int t = 0; t < TB; ++t)
          acc[b][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wr[s][b]), bf[s & 1][t],
                                                              acc[b][t], 0, 0, 0);
      load_w(s, c + 1);  // this step of the next chunk
      __builtin_amdgcn_sched_barrier(0);
      if (s == (STEPS > 1 ? STEPS / 2 - 1 : 0)) {
        if (c + 2 < c1) put_x(x, after);
        load_x(x, c + 4);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (STEPS & 1) {  // an odd number of steps leaves the next fragments in the other set
#pragma unroll
      for (int t = 0; t < TB; ++t) bf[0][t] = bf[1][t];
    }
    buf = next;
    __syncthreads();
  };
  // |partial sum| of the token, the largest of this lane's experts; a segment
  // counts with its last one.
  float seen[TB], last[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) seen[t] = 0.0f;
  auto sample = [&]() {
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      float m = 0.0f;  // a NaN does not count, an infinity does
#pragma unroll
      for (int b = 0; b < EW; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(acc[b][t][i]));
      seen[t] += m;
      last[t] = m;
    }
  };
  for (int c = c0; c < c1; c += 2) {
    chunk(xr[0], c);
    if (NS == 1 || c + 1 >= c1) sample();
    if (c + 1 < c1) {
      chunk(xr[1], c + 1);
      sample();
    }
  }
  // The group's, over all lanes and waves of a token; adding the groups and
  // parts are a few steps more.
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    float v = fmaf(seen[t], (float)(STEPS * NS), last[t] * (float)(WK + a.splits));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
    if (lane < 32) atomicMax(&partial[wk][t * 32 + lane], __float_as_uint(v));
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
  if (tid < BT && t0 + tid < a.tokens) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < WK; ++g) v += __uint_as_float(partial[g][tid]);
    a.partial[((int64_t)blockIdx.y * a.splits + split) * a.tokens + t0 + tid] = v;
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
constexpr int kXor1 = 0xb1, kXor2 = 0x4e;              // quad_perm: lane ^ 1, lane ^ 2
constexpr int kHalfMirror = 0x141, kMirror = 0x140;    // lane ^ 7, lane ^ 15
constexpr int kNext = 0x101;                           // row_shl:1, the lane after; 0 in the last

// Over a token's L lanes: a row of 16, two or all four.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  if constexpr (L > 16) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
  if constexpr (L > 32) v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  return ~lanes_max<L>(~v);
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dppf<kXor1>(v);
  v += dppf<kXor2>(v);
  v += dppf<kHalfMirror>(v);
  v += dppf<kMirror>(v);
  if constexpr (L > 16) v += __shfl_xor(v, 16, 64);
  if constexpr (L > 32) v += __shfl_xor(v, 32, 64);
  return v;
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

// A choice known in FP64 is a float and a rest: the difference in units of
// 2^-53 of the float's binade (FP64's own steps there, or halves of them), as
// an ordered integer.  It is below 2^30.  Where the float is subnormal or 0 the
// rest is the FP64 value's upper half, which orders it to 2^-20 of itself.
constexpr uint32_t kNoRest = 0x80000000u;
__device__ __forceinline__ uint32_t rest_of(double c) {
  const float hi = (float)c;
  if (fabsf(hi) < 0x1p-126f) {
    const uint32_t up = (uint32_t)(__double_as_longlong(fabs(c)) >> 32);
    return c < 0.0 ? kNoRest - up : kNoRest + up;
  }
  return kNoRest + (uint32_t)(int)ldexp(c - (double)hi, 53 - ilogbf(hi));
}
__device__ __forceinline__ double with_rest(uint32_t key, uint32_t rest) {
  const float hi = unordered(key);
  const int r = (int)(rest - kNoRest);
  if (r == 0) return (double)hi;
  if (fabsf(hi) < 0x1p-126f) return copysign(__longlong_as_double((int64_t)abs(r) << 32), (double)r);
  return (double)hi + ldexp((double)r, ilogbf(hi) - 53);
}

__device__ __forceinline__ float sigmoid_fast(float l) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * l));
}

// Batcher's odd-even merge sort, N a power of two.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1) {
#pragma unroll
    for (int k = p; k >= 1; k >>= 1) {
#pragma unroll
      for (int i = 0; i + k < N; ++i) {
        // pairs (i, i + k) of this pass
        if (i >= k % p && ((i - k % p) / k) % 2 == 0 && i / (2 * p) == (i + k) / (2 * p)) {
          const uint32_t a = v[i], b = v[i + k];
          v[i] = max(a, b);
          v[i + k] = min(a, b);
        }
      }
    }
  }
}

// Where the experts of a token sit: lane q of its LPT (16, 32 or 64) belongs to
// group q / lanes and holds `per_lane` experts of it from (q % lanes) *
// per_lane on, at most EPL (one group: all lanes).  An expert's slot, q EPL +
// j, rises with its number.
//
// A choice known in FP64 is kept as its value rounded to float32 and the rest:
// key (ordered) then rest.  The rest is 0 for choices known in FP32.
template <int EPL, int LPT, bool SPLIT>
__global__ __launch_bounds__(64) void router_select_kernel(RouterSelectArgs a) {
  constexpr uint32_t kSlots = LPT * EPL;   // a power of two
  constexpr uint32_t kSlotMask = kSlots - 1;
  constexpr int kTokens = 64 / LPT;        // of a wave
  extern __shared__ __attribute__((aligned(16))) float sums[];  // SPLIT: [kTokens][row]
  const int lane = threadIdx.x, q = lane & (LPT - 1), row0 = lane - q;
  const int64_t tw = (int64_t)blockIdx.x * kTokens;  // the wave's first token
  const int64_t t = tw + lane / LPT;
  auto row_max = [](uint32_t v) { return lanes_max<LPT>(v); };
  auto row_min = [](uint32_t v) { return lanes_min<LPT>(v); };
  auto row_sum = [](float v) { return lanes_sum<LPT>(v); };
  const bool live = t < a.tokens;
  const int64_t tt = live ? t : a.tokens - 1;
  // this lane's experts
  const int grp = q >> a.lane_shift, sub = q - (grp << a.lane_shift);
  const int e0 = grp * a.group_size + sub * a.per_lane;
  const int count = grp < a.groups ? max(0, min(a.per_lane, a.group_size - sub * a.per_lane)) : 0;

  // Squared norms of the row's parts and sums of |partial sum|, the largest of
  // the expert tiles (this half row's): asked for first, wanted last.
  const int part = lane & 7, odd = lane >> 3 & 1;
  static_assert(kMaxSplits <= 8, "a lane of eight per part");
  const bool has_part = part < a.splits;
  const int64_t at_part = (int64_t)(has_part ? part : 0) * a.tokens + tt;
  float n2 = a.norm2[at_part];
  float sampled = 0.0f;
  for (int y = 0; y < a.tiles; y += 8) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = a.partial[(int64_t)min(y + 2 * i + odd, a.tiles - 1) * a.splits * a.tokens + at_part];
    sampled = fmaxf(fmaxf(sampled, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
  }

  // Its logits and biases.  Slots past the count read the lane's first
  // expert (the row's first, if it has none).
  float l[EPL], bias[EPL];
  auto load_row = [&](const float* src, float (&v)[EPL]) {
    if (EPL >= 4 && (a.per_lane | a.group_size) % 4 == 0) {  // whole 16-byte pieces
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(src + (j < count ? e0 + j : (count ? e0 : 0)));
#pragma unroll
        for (int k = 0; k < 4 && j + k < EPL; ++k) v[j + k] = p[k];
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = src[j < count ? e0 + j : (count ? e0 : 0)];
    }
  };
  load_row(a.bias, bias);
  const float* row_logits;
  if constexpr (SPLIT) {
    // the K parts of the wave's tokens, summed in order
    const int n4 = (int)min((int64_t)kTokens, a.tokens - tw) * (a.row / 4);
    const f32x4* p = reinterpret_cast<const f32x4*>(a.part + tw * a.row);
    const int64_t step = (int64_t)a.tokens * a.row / 4;
    // up to 32 loads of a lane in flight; pieces past the end repeat the last
    auto sum_parts = [&](auto parts) {
      constexpr int S = decltype(parts)::value, U = 32 / S;
      for (int i0 = lane; i0 - lane < n4; i0 += 64 * U) {
        f32x4 v[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int s = 0; s < S; ++s) v[u][s] = p[min(s, a.splits - 1) * step + min(i0 + 64 * u, n4 - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          f32x4 t = v[u][0];
#pragma unroll
          for (int s = 1; s < S; ++s)
            if (s < a.splits) t += v[u][s];
          if (i0 + 64 * u < n4) reinterpret_cast<f32x4*>(sums)[i0 + 64 * u] = t;
        }
      }
    };
    if (a.splits <= 2)
      sum_parts(std::integral_constant<int, 2>{});
    else if (a.splits <= 4)
      sum_parts(std::integral_constant<int, 4>{});
    else
      sum_parts(std::integral_constant<int, kMaxSplits>{});
    __syncthreads();
    row_logits = sums + (tt - tw) * a.row;
  } else {
    row_logits = a.part + tt * a.row;
  }
  load_row(row_logits, l);
  n2 = 0.5f * lanes_sum<16>(has_part ? n2 : 0.0f);  // both halves of the row hold it
  sampled = fmaxf(sampled, dppf<0x128>(sampled));  // row_ror:8, the other half's tiles
  sampled = 0.5f * lanes_sum<16>(has_part ? sampled : 0.0f);

  auto choice = [&](float logit, float bias) { return a.sigmoid ? sigmoid_fast(logit) + bias : logit; };
  uint32_t key[EPL], rest[EPL];
  auto make_keys = [&]() {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      key[j] = j < count ? ordered(choice(l[j], bias[j])) : 0u;
      rest[j] = kNoRest;
    }
  };
  make_keys();
  float largest = 0.0f;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    largest = fmaxf(largest, j < count && fabsf(l[j]) < INFINITY ? fabsf(l[j]) : 0.0f);
    top = fmaxf(top, j < count ? l[j] : -INFINITY);
  }
  // softmax over all experts, where the K scores' sum does not cancel it
  float all_max = 0.0f, all_sum = 1.0f;
  if (!a.sigmoid && !a.renormalize) {
    all_max = unordered(row_max(ordered(top)));
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < count) z += expf(l[j] - all_max);
    all_sum = row_sum(z);
  }
  largest = __uint_as_float(row_max(__float_as_uint(largest)));  // not negative
  // Rows whose logits FP64 can tell apart where FP32 cannot.  Rows of zeros
  // and rows whose squared norm leaves float32's range go by their FP32 logits
  // as they are: what lies close there is evaluated again in FP64 from these.
  // Without a bias the choices of a row of zeros are all equal, and in order.
  const float xw = sqrtf(n2) * a.limits[0];
  // beside a gate row with an infinity the samples say nothing
  const float partials = sampled < INFINITY ? fmaf(a.slack, xw, sampled) : a.steps * xw;
  const float bound = 1.02f * 0x1p-24f * fmaf(kStepError, partials, kProductError * a.limits[1] * sqrtf(n2));
  const bool guard = live && bound < INFINITY && n2 >= 0x1p-100f;
  const bool decide = live && (guard || a.biased || largest > 0.0f);
  const float logit_margin = guard ? bound : 0.0f;
  // Margin of a choice c.  A sigmoid's slope is s (1 - s), 1/4 at most;
  // evaluating it costs less than 2^-20, adding its bias a rounding of c.  It
  // grows with |c| so slowly that c - margin and c + margin rise with c: what
  // holds for a largest choice holds for those below it, however large their
  // biases are.  Choices that are not finite are exact as they are.
  const float ev = a.sigmoid ? 0x1p-22f : 0.0f, eval = a.sigmoid ? 0x1p-20f : 0.0f;
  const float base = a.sigmoid ? fmaf(0.25f, logit_margin, eval) : logit_margin;
  auto margin_of = [&](float c) { return fmaf(ev, fabsf(c), base); };
  // At a known logit the slope is s (1 - s) there, and within the margin at
  // most exp(logit_margin) times that.
  const float steeper = logit_margin < 1.0f ? fmaf(2.0f, logit_margin, 1.01f) : INFINITY;
  auto slope_margin = [&](float logit) {
    const float s = sigmoid_fast(logit);
    return a.sigmoid ? fmaf(fminf(0.25f, s * (1.0f - s) * steeper), logit_margin, eval) : logit_margin;
  };
  // FP64 logits of two (token row, expert) pairs at a time, in every lane, so
  // that a pair of neighbours costs one trip to memory.
  auto dot2 = [&](int from0, int expert0, int from1, int expert1, double& out0, double& out1) {
    const uint16_t* rows[4] = {a.x + (tw + from0 / LPT) * a.x_stride, a.w + (int64_t)expert0 * a.hidden,
                               a.x + (tw + from1 / LPT) * a.x_stride, a.w + (int64_t)expert1 * a.hidden};
    // Two batches of loads, one on its way while the other is added up.
    constexpr int kBatch = 2;  // pieces of a row per batch: the additions, not the loads, take the time
    double d[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
    u32x4 v[2][4][kBatch];
    auto fetch = [&](u32x4 (&to)[4][kBatch], int base) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = base + k * 512 < a.hidden ? base + k * 512 : 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) to[r][k] = *reinterpret_cast<const u32x4*>(rows[r] + i);
      }
    };
    auto add = [&](const u32x4 (&from)[4][kBatch], int base) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (base + k * 512 >= a.hidden) continue;
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t xv = from[2 * o][k][i], wv = from[2 * o + 1][k][i];
            // a product of two bfloat16 has 16 bits: exact in float32
            d[o][0] += (double)(bf16_to_f32(xv & 0xffffu) * bf16_to_f32(wv & 0xffffu));
            d[o][1] += (double)(__uint_as_float(xv & 0xffff0000u) * __uint_as_float(wv & 0xffff0000u));
          }
      }
    };
    constexpr int kStep = kBatch * 512;
    fetch(v[0], lane * 8);
    for (int base = lane * 8; base - lane * 8 < a.hidden; base += 2 * kStep) {
      fetch(v[1], base + kStep);
      add(v[0], base);
      fetch(v[0], base + 2 * kStep);
      add(v[1], base + kStep);
    }
    out0 = d[0][0] + d[0][1];
    out1 = d[1][0] + d[1][1];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      out0 += __shfl_xor(out0, m, 64);
      out1 += __shfl_xor(out1, m, 64);
    }
  };
  auto choice64 = [&](double logit, int e) -> double {
    return a.sigmoid ? 1.0 / (1.0 + exp(-logit)) + (double)a.bias[e] : logit;
  };

  // Choices of marked slots (bits of the lanes' `need`) in FP64.
  auto recompute = [&](uint64_t need) {
    int from[2], j0[2], e[2];
    // the next marked slot, which loses its mark
    auto next = [&](int k) -> bool {
      const uint64_t lanes = __ballot(need != 0);
      if (!lanes) return false;
      from[k] = __builtin_ctzll(lanes);
      const uint64_t bits = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(need >> 32), from[k]) << 32) |
                            (uint32_t)__builtin_amdgcn_readlane((int)need, from[k]);
      j0[k] = __builtin_ctzll(bits);
      e[k] = __builtin_amdgcn_readlane(e0, from[k]) + j0[k];
      if (lane == from[k]) need &= need - 1;
      return true;
    };
    while (next(0)) {
      if (!next(1)) from[1] = from[0], j0[1] = j0[0], e[1] = e[0];
      double d[2];
      dot2(from[0], e[0], from[1], e[1], d[0], d[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const double c = choice64(d[k], e[k]);
        const uint32_t hi = ordered((float)c), lo = rest_of(c);
        if (lane == from[k]) {
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (j == j0[k]) {
              l[j] = (float)d[k];
              key[j] = hi;
              rest[j] = lo;
            }
        }
      }
    }
  };

  // The same from the FP32 logits, for the marked slots of rows that go by these.
  auto from_logits = [&](uint64_t marked) {
#pragma unroll 1
    for (int j0 = 0; j0 < EPL; ++j0) {
      const bool now = (marked >> j0) & 1u;
      if (!__ballot(now)) continue;
      const int e = now ? e0 + j0 : 0;
      const double c = choice64(row_logits[e], e);
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (now && j == j0) {
          key[j] = ordered((float)c);
          rest[j] = rest_of(c);
        }
    }
  };

  bool in = true;  // whether this lane's group stays
  if (a.groups > 1) {
    const bool two = a.sigmoid && a.group_size > 1;
    // the group's two largest choices, in all its lanes
    uint32_t k1 = 0, k2 = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      k2 = max(k2, min(k1, key[j]));
      k1 = max(k1, key[j]);
    }
    auto merge = [&](uint32_t o1, uint32_t o2) {
      k2 = max(min(k1, o1), max(k2, o2));
      k1 = max(k1, o1);
    };
    if (a.lane_shift > 0) merge(dpp<kXor1>(k1), dpp<kXor1>(k2));
    if (a.lane_shift > 1) merge(dpp<kXor2>(k1), dpp<kXor2>(k2));
    if (a.lane_shift > 2) merge(dpp<kHalfMirror>(k1), dpp<kHalfMirror>(k2));
    if constexpr (LPT > 16) {
      if (a.lane_shift > 3) merge(dpp<kMirror>(k1), dpp<kMirror>(k2));
      if (a.lane_shift > 4) merge(__shfl_xor((int)k1, 16, 64), __shfl_xor((int)k2, 16, 64));
    }
    const float b1 = unordered(k1), b2 = two ? unordered(k2) : 0.0f;
    const float v = (two ? k2 : k1) > 1u ? b1 + b2 : NAN;
    const bool valid = grp < a.groups;
    const uint32_t vk = valid ? ordered(v) : 0u;
    int ahead = 0;
    if constexpr (LPT == 16) {  // lanes of groups ahead of this one, by rotating the row
#define MOE_ROT(N)                                                                  \
  {                                                                                 \
    const uint32_t o = dpp<0x120 + N>(vk);                                          \
    ahead += (o > vk || (o == vk && ((q - N) & 15) >> a.lane_shift < grp)) ? 1 : 0; \
  }
      MOE_ROT(1) MOE_ROT(2) MOE_ROT(3) MOE_ROT(4) MOE_ROT(5) MOE_ROT(6) MOE_ROT(7) MOE_ROT(8)
      MOE_ROT(9) MOE_ROT(10) MOE_ROT(11) MOE_ROT(12) MOE_ROT(13) MOE_ROT(14) MOE_ROT(15)
#undef MOE_ROT
      in = valid && ahead < a.top_groups << a.lane_shift;
    } else {
      for (int g = 0; g < a.groups; ++g) {
        const uint32_t o = (uint32_t)__shfl((int)vk, row0 + (g << a.lane_shift), 64);
        ahead += (o > vk || (o == vk && g < grp)) ? 1 : 0;
      }
      in = valid && ahead < a.top_groups;
    }
    // least that the values that stay can be, most that the others can be
    const float gm = fmaf(ev, fabsf(b1) + fabsf(b2), two ? 2.0f * base : base);
    const bool number = fabsf(v) < INFINITY;
    const float lo = unordered(row_min(in ? ordered(number ? v - gm : v) : 0xffffffffu));
    const float hi = unordered(row_max(valid && !in ? ordered(number ? v + gm : v) : 0u));
    const bool close = decide && fabsf(lo) < INFINITY && fabsf(hi) < INFINITY && lo <= hi;
    if (__ballot(close)) {
      // FP64 for the members that can make the values of groups at the border
      const bool at = close && valid && number && (in ? v - gm <= hi : v + gm >= lo);
      const float least = two ? b2 : b1, from = least - margin_of(least);
      uint64_t need = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (at && key[j] > 1u && unordered(key[j]) + margin_of(unordered(key[j])) >= from) need |= 1ull << j;
      recompute(guard ? need : 0);
      from_logits(guard ? 0 : need);
      double c1 = -INFINITY, c2 = -INFINITY;
      auto put = [&](double c) {
        c2 = fmax(c2, fmin(c1, c));
        c1 = fmax(c1, c);
      };
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        put(key[j] > 1u ? with_rest(key[j], rest[j]) : -INFINITY);
      for (int m = 1; m < 1 << a.lane_shift; m <<= 1) {
        const double o1 = __shfl_xor(c1, m, 64), o2 = __shfl_xor(c2, m, 64);
        put(o1);
        put(o2);
      }
      double gv = two ? c1 + c2 : c1;
      gv = vk > 1u && gv == gv ? gv : -INFINITY;
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl(gv, row0 + (g << a.lane_shift), 64);
        const uint32_t ok = (uint32_t)__shfl((int)vk, row0 + (g << a.lane_shift), 64);
        // -inf is not recomputed, and before NaN
        const bool tie_first = gv == -INFINITY && ok != vk ? ok > vk : g < grp;
        rank += (o > gv || (o == gv && tie_first)) ? 1 : 0;
      }
      in = valid && rank < a.top_groups;
    }
  }

  // The K + 1 largest, by keys whose low bits give way to the slot (the lowest
  // slot the largest): one maximum finds value and expert, lane k of the row
  // keeping the k-th.
  uint32_t pk[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    pk[j] = in && key[j] ? (max(key[j], kSlots) & ~kSlotMask) | (kSlotMask - (uint32_t)(q * EPL + j)) : 0u;
  // Each lane sorts its own first, so that a maximum looks at one key per lane
  // (T=4096: the selection's instructions halve).
  sort_descending<EPL>(pk);
  uint32_t mk = 0;  // lane k of the token's first 16: the k-th packed key
  auto take = [&](int k) -> uint32_t {
    const uint32_t m = row_max(pk[0]);
    const bool hit = pk[0] == m;
#pragma unroll
    for (int j = 0; j + 1 < EPL; ++j) pk[j] = hit ? pk[j + 1] : pk[j];
    pk[EPL - 1] = hit ? 0u : pk[EPL - 1];
    if (q == k) mk = m;
    return m;
  };
  for (int k = 0; k <= a.top_k; ++k) (void)take(k);
  auto expert_of = [&](uint32_t m) -> int {
    const int slot = (int)(kSlotMask - (m & kSlotMask));
    const int qs = slot / EPL, gs = qs >> a.lane_shift;
    return gs * a.group_size + (qs - (gs << a.lane_shift)) * a.per_lane + slot % EPL;
  };
  // largest choice that a packed key can stand for
  auto upper = [&](uint32_t m) { return m >= 2 * kSlots ? unordered(m | kSlotMask) : -INFINITY; };
  int id = mk ? expert_of(mk) : 0;
  float ml = row_logits[id];  // of the lane's entry
  float c = mk ? choice(ml, a.bias[id]) : -INFINITY;
  float mine = ml;
  // Too close: neighbours among the K within the largest of their margins,
  // or the last of them and what follows within its margin and any.
  const uint32_t after = dpp<kNext>(mk);
  const float among = unordered(row_max(q < a.top_k ? ordered(slope_margin(ml)) : 0u));
  const float next = upper(after);
  const bool number = fabsf(c) < INFINITY;
  const bool tight = decide && q < a.top_k && number && fabsf(next) < INFINITY &&
                     c - next <= fmaf(ev, fabsf(c) + fabsf(next), among + (q + 1 < a.top_k ? among : base));
  if (__ballot(tight)) {
    // Some token of the wave has neighbours too close to call.  Its list goes
    // on while choices may belong to the K after all.
    const bool mineclose = ((__ballot(tight) >> row0) & 0xffffu) != 0;
    const float border =
        unordered(row_min(q < a.top_k && number ? ordered(c - fmaf(ev, fabsf(c), among)) : 0xffffffffu));
    int n = a.top_k + 1;
    bool more = true;
    for (; n < 16 && more; ++n) {
      const uint32_t m = take(n);
      more = __ballot(mineclose && upper(m) + margin_of(upper(m)) >= border) != 0;
    }
    if (!more) {
      id = mk ? expert_of(mk) : 0;
      ml = row_logits[id];
      c = mk ? choice(ml, a.bias[id]) : -INFINITY;
      mine = ml;
      // those within the margins of another, in FP64
      bool redo = false;
      const float mm = fabsf(c) < INFINITY ? fmaf(ev, fabsf(c), slope_margin(ml)) : 0.0f;
#define MOE_ROT(N)                                                     \
  {                                                                    \
    const float o = dppf<0x120 + N>(c);                                \
    redo |= fabsf(c - o) <= mm + dppf<0x120 + N>(mm);                  \
  }
      MOE_ROT(1) MOE_ROT(2) MOE_ROT(3) MOE_ROT(4) MOE_ROT(5) MOE_ROT(6) MOE_ROT(7) MOE_ROT(8)
      MOE_ROT(9) MOE_ROT(10) MOE_ROT(11) MOE_ROT(12) MOE_ROT(13) MOE_ROT(14) MOE_ROT(15)
#undef MOE_ROT
      double exact = c == c ? c : -INFINITY;
      if (redo && !guard && mk != 0) exact = choice64(ml, id);
      uint64_t todo = __ballot(redo && guard && mineclose && mk != 0);
      while (todo) {
        const int f0 = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int f1 = todo ? __builtin_ctzll(todo) : f0;
        todo &= todo - 1;  // 0 stays 0
        double d0, d1;
        dot2(f0, __builtin_amdgcn_readlane(id, f0), f1, __builtin_amdgcn_readlane(id, f1), d0, d1);
        if (lane == f0 || lane == f1) {
          const double d = lane == f0 ? d0 : d1;
          exact = choice64(d, id);
          mine = (float)d;
        }
      }
      // their order, ties to the lowest expert (-inf and NaN are in order as
      // they stand); lane k takes the k-th
      if (!mk) exact = -INFINITY;
      int rank = 0;
      for (int i = 0; i < 16; ++i) {
        const double o = __shfl(exact, row0 + i, 64);
        const int oe = __shfl(id, row0 + i, 64);
        const bool there = __shfl((int)(mk != 0), row0 + i, 64) != 0;
        rank += there && (!mk || o > exact || (o == exact && (o == -INFINITY ? i < q : oe < id))) ? 1 : 0;
      }
      int at = row0;
      for (int i = 0; i < 16; ++i)
        if (__shfl(mk ? rank : 16, row0 + i, 64) == q) at = row0 + i;
      const int nid = __shfl(id, at, 64);
      const float nl = __shfl(mine, at, 64);
      if (mineclose) {
        id = nid;
        mine = nl;
      }
    } else {
      // Too many for the list: every choice within the margin of its
      // neighbour, among all experts.  The keys are made again, which keeps
      // their registers free until here.
      load_row(row_logits, l);
      load_row(a.bias, bias);
      make_keys();
      if (!in) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = 0u;
      }
      auto extract = [&](auto exact) -> uint64_t {
        constexpr bool kExact = decltype(exact)::value;
        uint64_t taken = 0, need = 0;
        float before = INFINITY, last = -INFINITY;
        uint32_t ps = 0;
        for (int k = 0;; ++k) {
          uint32_t bk = 0, br = 0, bs = 0;
          float bl = 0.0f;
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const uint32_t kj = (taken >> j) & 1u ? 0u : key[j];
            if (kExact ? (kj > bk || (kj == bk && kj != 0u && rest[j] > br)) : kj > bk) {
              bk = kj;
              br = rest[j];
              bs = (uint32_t)(q * EPL + j);
              bl = l[j];
            }
          }
          const uint32_t m = row_max(bk);
          bool best = bk == m;
          if constexpr (kExact) {
            const uint32_t r = row_max(best ? br : 0u);
            best = best && br == r;
          }
          const uint32_t s = row_min(best ? bs : 0xffffffffu) & kSlotMask;
          const bool own = s / EPL == (uint32_t)q;
          if constexpr (!kExact) {
            const float ck = unordered(m);
            const bool number = fabsf(ck) < INFINITY;
            if (number && guard && before < INFINITY && before - ck <= margin_of(before) + margin_of(ck)) {
              if (own) need |= 1ull << (s % EPL);
              if (ps / EPL == (uint32_t)q) need |= 1ull << (ps % EPL);
            }
            if (k == a.top_k - 1) last = ck;
            const bool reach = last > -INFINITY && ck + margin_of(ck) >= last - margin_of(last);
            if (!__ballot(k < a.top_k || (number && guard && reach))) break;
            before = number ? ck : INFINITY;
            ps = s;
          } else {
            const float el = __shfl(bl, row0 + (int)(s / EPL), 64);
            if (q == k && mineclose) {
              id = expert_of(kSlotMask - s);
              mine = el;
            }
            if (k == a.top_k - 1) break;
          }
          if (own) taken |= 1ull << (s % EPL);
        }
        return need;
      };
      recompute(extract(std::false_type{}));
      uint64_t all = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (mineclose && !guard && fabsf(unordered(key[j])) < INFINITY) all |= 1ull << j;
      from_logits(all);
      extract(std::true_type{});
    }
  }

  // routing weights
  const bool slot = q < a.top_k;
  float w;
  if (a.sigmoid) {
    // exp(-l) overflows below -88: there a score is exp(l), and where the
    // scores' sum cancels, all of them are taken exp(m) times as large, m the
    // largest logit if it is negative.
    const float m = fminf(unordered(row_max(slot ? ordered(mine) : 0u)), 0.0f);
    const bool small = a.renormalize && unordered(row_min(slot ? ordered(mine) : 0xffffffffu)) < -80.0f;
    const float by = small && m > -INFINITY ? m : 0.0f;
    w = small || mine < -80.0f ? expf(fminf(mine, 0.0f) - by) / (1.0f + expf(-fabsf(mine)))
                               : 1.0f / (1.0f + expf(-mine));
    w = slot ? (mine == mine ? w : mine) : 0.0f;
  } else if (a.renormalize) {  // the sum over all experts cancels
    const float m = unordered(row_max(slot ? ordered(mine) : 0u));
    w = slot ? expf(mine - m) : 0.0f;
  } else {
    w = slot ? expf(mine - all_max) / all_sum : 0.0f;
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

// limits[0] = max |w_e| and limits[1] = max of sqrt(sum over 16-column steps
// of max w_e^2), over the experts without an infinite or NaN weight (whose
// logits are neither numbers nor close to any), and the padded copy of the
// biases; one wave per expert slot of a logit row.  A maximum does not depend
// on the order of the atomics.
__global__ __launch_bounds__(64) void router_limits_kernel(const uint16_t* w, const float* bias, int experts,
                                                           int hidden, uint32_t* limits, float* bias_copy) {
  const int e = blockIdx.x;
  if (threadIdx.x == 0) bias_copy[e] = bias && e < experts ? bias[e] : 0.0f;
  if (e >= experts) return;
  float squares = 0.0f, steps = 0.0f;
  bool bad = false;
  for (int i = threadIdx.x * 8; i - (int)threadIdx.x * 8 < hidden; i += 512) {  // two threads a step
    float most = 0.0f;
    if (i < hidden) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = bf16_to_f32(w[(int64_t)e * hidden + i + k]);
        squares = fmaf(v, v, squares);
        most = fmaxf(most, fabsf(v));
        bad |= !(fabsf(v) < INFINITY);
      }
    }
    most = fmaxf(most, __shfl_xor(most, 1, 64));
    if (!(threadIdx.x & 1)) steps = fmaf(most, most, steps);
  }
  if (__ballot(bad)) return;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    squares += __shfl_xor(squares, m, 64);
    steps += __shfl_xor(steps, m, 64);
  }
  if (threadIdx.x == 0) {
    atomicMax(&limits[0], __float_as_uint(sqrtf(squares)));
    atomicMax(&limits[1], __float_as_uint(sqrtf(steps)));
  }
}

// Token tile and K split of a batch.
struct Plan {
  int bt, be;  // tokens and 32-expert blocks per workgroup
  int splits, chunks_per_split;
};

// Few tokens take narrow expert tiles, so that the K split, whose parts the
// selection reads back, stays at most kMaxSplits; many take wide tiles, which
// read the token rows once.  Where the steps lie hardly matters below a
// thousand tokens and much above (H=7168 E=256, us for the whole call with the
// next smaller, this and the next larger tile):
//   tokens: T=512 - / 23.7 / 24.4, 4096 46.3 / 42.4 / 44.0, 16384 121.7 / 98.3 / -
//   experts: T=32 - / 14.1 / 13.1, 256 23.7 / 22.4 / 23.0, 4096 46.0 / 42.4 / -,
//            8192 73.9 / 65.9 / 70.3, 16384 103.1 / 98.3 / -
// Where one block holds all experts the rows are everything that is read, and
// more, smaller workgroups bring them faster (H=2048 E=32: T=1024 11.5 us with
// 32 tokens against 12.8 with 64, T=8192 17.6 against 23.3 with 128, T=32768
// 48.6 with 64 against 52.3; H=7168 E=16 T=32768 64 tokens 99, 32 109, 128
// 102).
Plan plan_for(const moe_router_config_t& c, int64_t tokens) {
  Plan p;
  p.bt = tokens <= 512 ? 32 : (tokens <= 4096 ? 64 : 128);
  const int blocks = (c.num_experts + 31) / 32;
  p.be = tokens <= 32 ? 1 : (tokens <= 256 ? 2 : (tokens <= 8192 ? 4 : 8));
  while (p.be / 2 >= blocks) p.be /= 2;
  if (blocks == 1) p.bt = tokens <= 8192 ? 32 : 64;
  const int64_t tiles = (tokens + p.bt - 1) / p.bt * ((blocks + p.be - 1) / p.be);
  const int chunks = c.hidden / kKC;
  int64_t want = kTargetGroups / tiles;
  want = want < 1 ? 1 : (want > kMaxSplits ? kMaxSplits : want);
  if (want > chunks) want = chunks;
  p.chunks_per_split = (int)((chunks + want - 1) / want);
  p.splits = (chunks + p.chunks_per_split - 1) / p.chunks_per_split;
  return p;
}

// Floats per logit row: whole blocks of 32 experts.
int row_of(int experts) { return (experts + 31) / 32 * 32; }

// Lanes of a token: 16, or as many more as leave a lane 16 experts at most, or
// 4 at least where that makes no more than kSelectWaves waves of the batch (each
// then has fewer tokens' FP64 logits to wait for; H=7168 E=256, us for the whole
// call with 16, 32 and 64 lanes: T=1 11.6 / 10.7 / 10.5, 512 29.7 / 25.4 / 24.9,
// 1024 33.7 / 31.4 / 30.4, 4096 52.2 / 48.1 / 49.0, 8192 76.8 / 78.2 / 82.8; E=32
// T=509 12.2 / 12.5 / 13.0); those of a group, a power of two, and experts per lane.
constexpr int64_t kSelectWaves = 2048;
struct Lanes {
  int groups, of_token, lanes, per_lane;
};
Lanes lanes_for(const moe_router_config_t& c, int64_t tokens) {
  Lanes r;
  r.groups = c.top_groups == c.num_groups ? 1 : c.num_groups;  // every group stays: none to pick
  for (r.of_token = 16;; r.of_token *= 2) {
    r.lanes = r.of_token;
    while (r.lanes * r.groups > r.of_token) r.lanes >>= 1;
    r.per_lane = (c.num_experts / r.groups + r.lanes - 1) / r.lanes;
    const bool more = r.per_lane >= 8 && tokens * r.of_token * 2 <= kSelectWaves * 64;
    if (r.of_token == 64 || (r.per_lane <= kMaxPerLane && !more)) return r;
  }
}

struct RouterLayout {
  size_t w, limits, bias, part, norm2, partial, total;
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

RouterLayout router_layout(const moe_router_config_t& c, int64_t max_rows) {
  RouterLayout L;
  // splits x tokens of any batch: at most kMaxSplits parts, and no more token
  // tiles than kTargetGroups where there are several
  const int64_t split_rows = (int64_t)kTargetGroups * 128;
  int64_t rows = max_rows * kMaxSplits;
  if (rows > split_rows) rows = max_rows > split_rows ? max_rows : split_rows;
  L.w = 0;
  L.limits = L.w + align256((size_t)((c.num_experts + 31) / 32) * 32 * c.hidden * 2);
  L.bias = L.limits + 256;
  L.part = L.bias + align256((size_t)row_of(c.num_experts) * 4);
  L.norm2 = L.part + align256((size_t)rows * row_of(c.num_experts) * 4);
  L.partial = L.norm2 + align256((size_t)rows * 4);
  L.total = L.partial + align256((size_t)rows * (row_of(c.num_experts) / 32) * 4);
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
  const Lanes n = lanes_for(*c, max_rows);
  if (n.per_lane > kMaxPerLane)
    return fail(MOE_ERR_UNSUPPORTED, "groups of %d experts: %d groups take at most %d each",
                c->num_experts / c->num_groups, c->num_groups, kMaxPerLane * n.lanes);
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
void launch_gemm(const RouterGemmArgs& g, int be, dim3 grid, hipStream_t s) {
  const dim3 block(kGemmThreads);
  if constexpr (BT == 128) {  // plan_for takes 8 blocks with 128 tokens only
    if (be == 8 && grid.y == 1) {
      hipLaunchKernelGGL((router_gemm_kernel<BT, 4, 2, true>), grid, block, 0, s, g);
      return;
    }
    if (be == 8) {
      hipLaunchKernelGGL((router_gemm_kernel<BT, 4, 2>), grid, block, 0, s, g);
      return;
    }
  }
  if constexpr (BT < 128) {  // and one block with fewer only
    if (be == 1) {
      hipLaunchKernelGGL((router_gemm_kernel<BT, 1, 1>), grid, block, 0, s, g);
      return;
    }
  }
  if (be == 4)
    hipLaunchKernelGGL((router_gemm_kernel<BT, 4, 1>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((router_gemm_kernel<BT, 2, 1>), grid, block, 0, s, g);
}

template <int EPL, int LPT>
void launch_select(const RouterSelectArgs& a, hipStream_t s) {
  constexpr int kTokens = 64 / LPT;
  const dim3 grid((a.tokens + kTokens - 1) / kTokens), block(64);
  if (a.splits > 1)
    hipLaunchKernelGGL((router_select_kernel<EPL, LPT, true>), grid, block, kTokens * a.row * sizeof(float), s, a);
  else
    hipLaunchKernelGGL((router_select_kernel<EPL, LPT, false>), grid, block, 0, s, a);
}

template <int LPT>
void launch_select_lanes(const RouterSelectArgs& a, hipStream_t s) {
  if (LPT == 16 && a.per_lane <= 2)  // lanes_for leaves the wider ones four at least
    launch_select<2, 16>(a, s);
  else if (a.per_lane <= 4)
    launch_select<4, LPT>(a, s);
  else if (a.per_lane <= 8)
    launch_select<8, LPT>(a, s);
  else
    launch_select<16, LPT>(a, s);
}

}  // namespace
}  // namespace moe

struct moe_router {
  moe_router_config_t cfg;
  const uint16_t* w;
  uint8_t* ws;
  moe::RouterLayout L;
  int32_t max_rows;
  bool biased;
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
  r->ws = static_cast<uint8_t*>(workspace);
  r->L = L;
  r->max_rows = max_rows;
  r->biased = bias != nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t pieces = (int64_t)((cfg->num_experts + 31) / 32) * (cfg->hidden / 16) * 64;
  uint32_t* limits = reinterpret_cast<uint32_t*>(r->ws + L.limits);
  bool ok = moe::launch_fill_zero(limits, 64, stream) == 0;
  if (ok) {
    hipLaunchKernelGGL(moe::router_tile_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, r->w,
                       reinterpret_cast<moe::u32x4*>(r->ws + L.w), pieces, cfg->num_experts, cfg->hidden);
    hipLaunchKernelGGL(moe::router_limits_kernel, dim3(moe::row_of(cfg->num_experts)), dim3(64), 0, s, r->w, bias,
                       cfg->num_experts, cfg->hidden, limits, reinterpret_cast<float*>(r->ws + L.bias));
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
  g.partial = reinterpret_cast<float*>(r->ws + r->L.partial);
  const dim3 grid((num_tokens + p.bt - 1) / p.bt, (g.blocks + p.be - 1) / p.be, p.splits);
  if (p.bt == 32)
    moe::launch_gemm<32>(g, p.be, grid, s);
  else if (p.bt == 64)
    moe::launch_gemm<64>(g, p.be, grid, s);
  else
    moe::launch_gemm<128>(g, p.be, grid, s);
  moe::RouterSelectArgs a;
  a.part = g.part;
  a.norm2 = g.norm2;
  a.partial = g.partial;
  a.tiles = (int32_t)grid.y;
  // as launch_gemm's kernels take them
  const int groups = moe::kGemmWaves / (p.be < 4 ? p.be : 4);
  const int sampled = moe::kKC / 16 / groups * moe::samples_every((p.be == 8 ? 2 : 1) * (p.bt / 32));
  a.steps = (float)(c.hidden / 16 + groups + p.splits);
  a.slack = (float)(sampled / 2) + 0.5f;
  a.limits = reinterpret_cast<const float*>(r->ws + r->L.limits);
  a.x = g.x;
  a.x_stride = x_stride;
  a.w = r->w;
  a.bias = reinterpret_cast<const float*>(r->ws + r->L.bias);
  a.tokens = num_tokens;
  a.hidden = c.hidden;
  a.row = g.row;
  a.splits = p.splits;
  a.top_k = c.top_k;
  const moe::Lanes n = moe::lanes_for(c, num_tokens);
  a.groups = n.groups;
  a.group_size = c.num_experts / n.groups;
  a.lane_shift = 0;
  while (1 << a.lane_shift < n.lanes) ++a.lane_shift;
  a.per_lane = n.per_lane;
  a.top_groups = c.top_groups;
  a.sigmoid = c.score == MOE_SCORE_SIGMOID;
  a.renormalize = c.renormalize;
  a.biased = r->biased;
  a.scale = c.scale;
  a.expert_base = c.expert_base;
  a.local_experts = c.local_experts;
  a.idx = topk_idx;
  a.out_w = topk_w;
  a.ids = ids;
  if (n.of_token == 64)
    moe::launch_select_lanes<64>(a, s);
  else if (n.of_token == 32)
    moe::launch_select_lanes<32>(a, s);
  else
    moe::launch_select_lanes<16>(a, s);
  if (hipGetLastError() != hipSuccess) return moe::fail(MOE_ERR_HIP, "router launch failed");
  return MOE_OK;
}

extern "C" moe_status_t moe_router_destroy(moe_router_t* r) {
  moe::clear_error();
  delete r;
  return MOE_OK;
}
