// The layer for a few tokens (moe_layer_decode): at most 16 of them, two
// launches, on the layer's own weight tiles and with its arithmetic.
//
//   decode_fc1_kernel   x -> e4m3 1x128 (or given so), gate and up rows,
//                       h = silu(g) u, h -> e4m3 1x128
//   decode_fc2_kernel   y = h W2^T, out[t] = bf16(sum_k w[t, k] y_k)
//
// The weights of the chosen experts are nearly the whole traffic (T=1 H=7168
// I=2048 K=8: 352 MB, 52 us at the 6.8 TB/s that a plain read reaches; T=16:
// 1.40 GB, 206 us), so everything is arranged around streaming them once:
//  * The MFMA takes 16 weight rows x 16 tokens, and 16 columns hold every
//    token: no staging, no compaction and no token tiles.  A lane's weight
//    operand of a K-block is 32 bytes of the create-time tiles, loaded straight
//    into registers, 1 KB per instruction.
//  * A workgroup takes few output columns of one expert (FC1) or of all of
//    them (FC2), and its waves split the K-blocks, so that a single token's
//    few experts still make several hundred workgroups.  The waves' sums meet
//    in LDS.
//  * BF16 rows for FP8 weights are quantised by every FC1 workgroup for itself
//    (T=16 H=7168: 229 KB of rows, from L2, each block by eight lanes; 242 us
//    for the call against 223 with e4m3 rows given).
//  * h is quantised per 128 columns.  A workgroup makes whole blocks where the
//    chosen experts have enough of them; the tasks of the others go to several
//    workgroups, which store FP32 columns, and the last to arrive quantises
//    the block.
//  * FC2 adds the experts' rows in FP32 with the routing weights applied to
//    the partial sums, so there are no y rows and no combine.
// The whole call, FP8 weights and e4m3 rows, H=7168 I=2048 K=8 of 32 experts:
// T=1 67 us, 2 108, 4 160, 8 205, 16 223 (5.3 to 6.2 TB/s; FC1 takes two
// thirds); MXFP8 67, 105, 163, 219, 282.  H=2048 I=768 K=6: T=1 18 us, 5 33,
// 16 44, where the two launches' starts and ends, about 10 us, are what is
// left beside the stream.
#include <hip/hip_runtime.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_quant_dev.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = 8;                // waves that stream weights
constexpr int kRing = 4;                 // FC1: finishing waves, and sums between them and the streaming ones
constexpr int kFc1Threads = (kWaves + kRing) * 64;
constexpr int kCols = kDecodeTokens;     // MFMA columns
constexpr int kSlots = kDecodeSlots;
constexpr int kTileBytes = 32 * 1024;    // a 256 x 128 weight tile
constexpr int kFragBytes = 2 * 1024;     // its 16 x 128 fragments

struct Frag {
  u32x4 lo, hi;
};
__device__ __forceinline__ v8i operand(const Frag& f) {
  v8i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = (int)f.lo[i];
    r[4 + i] = (int)f.hi[i];
  }
  return r;
}
// Weights are read once by one workgroup: non-temporal.
__device__ __forceinline__ Frag load_frag_nt(const uint8_t* p) {
  return Frag{__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)),
              __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 1024))};
}
// Eight e4m3 codes as bfloat16, exactly.
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The same for MX codes (e4m3, or e5m2 with E5M2) times the power of two whose
// E8M0 exponent is `e`, held in a float's exponent bits.
template <bool E5M2>
__device__ __forceinline__ bf16x8 widen8_mx(uint32_t lo, uint32_t hi, float e) {
  bf16x2 a, b, c, d;
  if constexpr (E5M2) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)lo, e, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)lo, e, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)hi, e, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)hi, e, true);
  } else {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, e, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, e, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, e, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, e, true);
  }
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One K-block of MX weights (16 rows) and BF16 rows on the BF16 MFMA.  A
// lane's first 16 weight bytes are columns 16 g.. of the block (g = lane / 16)
// and its last 16 columns 64 + 16 g..; x[0], x[1] and x[2], x[3] hold the same
// columns of its token, and e0, e1 are the two halves' exponent words with
// this row block's byte at `shift`.
template <bool E5M2>
__device__ __forceinline__ v4f mfma_mx_bf16(const Frag& w, const u32x4 (&x)[4], uint32_t e0, uint32_t e1, int shift) {
  const float f0 = __uint_as_float((e0 >> shift & 0xffu) << 23), f1 = __uint_as_float((e1 >> shift & 0xffu) << 23);
  v4f p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8_mx<E5M2>(w.lo[2 * i], w.lo[2 * i + 1], f0),
                                                __builtin_bit_cast(bf16x8, x[i]), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8_mx<E5M2>(w.hi[2 * i], w.hi[2 * i + 1], f1),
                                                __builtin_bit_cast(bf16x8, x[2 + i]), p, 0, 0, 0);
  }
  return p;
}
// Lane of the exponent words that covers the first half of this lane's
// columns; the second half's is 32 further.
__device__ __forceinline__ int mx_word(int lane) { return (lane & 15) + 16 * (lane >> 5); }
// BF16 columns of K-block `kb` of a row that go with this lane's weight bytes.
__device__ __forceinline__ void load_bf16_k(u32x4 (&x)[4], const uint16_t* row, int kb, int grp) {
  const u32x4* q = reinterpret_cast<const u32x4*>(row + kb * 128 + grp * 16);
  x[0] = q[0];
  x[1] = q[1];
  x[2] = q[8];
  x[3] = q[9];
}

// acc + p * (sx * sw) for scales of any size: the product's mantissas and
// exponents are applied apart, so that a product of scales beyond float32's
// range neither overflows nor vanishes on the way.
__device__ __forceinline__ v4f add_scaled(v4f acc, const v4f& p, float sx, float sw) {
  const float m = __builtin_amdgcn_frexp_mantf(sx) * __builtin_amdgcn_frexp_mantf(sw);
  const int e = __builtin_amdgcn_frexp_expf(sx) + __builtin_amdgcn_frexp_expf(sw);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += __builtin_amdgcn_ldexpf(p[i] * m, e);
  return acc;
}

// Checked routes of the call in LDS: ids (-1 masked) and weights, with
// moe_stage_inputs' rules.
struct Routes {
  int32_t raw[kSlots];
  int32_t id[kSlots];
  float w[kSlots];
};

// Order of LDS accesses between the lanes of one wave, whose LDS operations
// complete in order: a fence for the compiler.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// By one wave: checks the routes and lists the experts they reach in the
// order of their first routes.  Returns the MOE_DEV_* bits.
__device__ __forceinline__ uint32_t check_routes(const DecodeArgs& a, Routes& r, DecodePlan& plan, int lane) {
  const int n = a.tokens * a.top_k;
  int id[2];
  float w[2];
  uint32_t bits = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = h * 64 + lane;
    id[h] = i < n ? a.topk_idx[i] : -1;
    w[h] = i < n ? a.topk_w[i] : 0.0f;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (id[h] < -1 || id[h] >= a.num_experts) {
      bits |= MOE_DEV_BAD_EXPERT;
      id[h] = -1;
    }
    r.raw[h * 64 + lane] = id[h];
  }
  wave_fence();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = h * 64 + lane;
    if ((a.flags & MOE_FLAG_CHECK_ROUTES) && id[h] >= 0) {
      // the lowest slot of an id stays, whatever its weight
      bool again = false;
      for (int j = i - i % a.top_k; j < i; ++j) again |= r.raw[j] == id[h];
      if (again) {
        bits |= MOE_DEV_DUPLICATE;
        id[h] = -1;
      } else if (!isfinite(w[h])) {
        bits |= MOE_DEV_NONFINITE;
        id[h] = -1;
      }
    }
    r.id[i] = id[h];
    r.w[i] = id[h] >= 0 ? w[h] : 0.0f;
  }
  wave_fence();
  bool first[2] = {id[0] >= 0, id[1] >= 0};
  for (int j = 0; j < n; ++j) {
    const int o = r.id[j];
    if (j < lane && o == id[0]) first[0] = false;
    if (j < 64 + lane && o == id[1]) first[1] = false;
  }
  const uint64_t b0 = __ballot(first[0]), b1 = __ballot(first[1]), below = (1ull << lane) - 1;
  if (first[0]) plan.expert[__popcll(b0 & below)] = id[0];
  if (first[1]) plan.expert[__popcll(b0) + __popcll(b1 & below)] = id[1];
  if (lane == 0) plan.experts = __popcll(b0) + __popcll(b1);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) bits |= __shfl_xor(bits, m, 64);
  return bits;
}

// Per expert and token the route (the lowest, -1 for none) and its weight; a
// repeated id, which only stays without route checks, adds up in the weight.
__device__ __forceinline__ void map_routes(const DecodeArgs& a, const Routes& r, DecodePlan& plan, int i, int threads) {
  for (int j = i; j < plan.experts * kCols; j += threads) {
    const int t = j & 15, e = plan.expert[j >> 4];
    int slot = -1;
    float sum = 0.0f;
    if (t < a.tokens)
      for (int k = 0; k < a.top_k; ++k)
        if (r.id[t * a.top_k + k] == e) {
          if (slot < 0) slot = t * a.top_k + k;
          sum += r.w[t * a.top_k + k];
        }
    plan.row[j] = slot;
    plan.weight[j] = sum;
  }
}

// ---------------------------------------------------------------------------
// FC1
// ---------------------------------------------------------------------------

// Codes and scale of one 128-column block of h: 16 lanes, 8 columns each.
__device__ __forceinline__ void store_block(const DecodeArgs& a, const float h[8], int row, int blk, int lane16) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(h[i]) & 0x7fffffffu);
  const float s = __uint_as_float(row16_max(m)) / kE4m3Max;
  *reinterpret_cast<q_u32x2*>(a.hq + (int64_t)row * a.inter + blk * 128 + lane16 * 8) = quant8(h, s);
  if (lane16 == 0) a.hs[(int64_t)row * (a.inter / 128) + blk] = s;
}

// One workgroup per CU walks over tasks of 16 columns of h of one expert.
// Eight waves stream: wave w takes K-blocks [w kbs / 8, (w + 1) kbs / 8), at
// most NK, of every task; it keeps its part of the token rows, quantised, in
// registers for all tasks, and has one K-block of weights (4 KB) in flight,
// running on into the next task.  More in flight only makes every wait for
// memory longer: a copy of this access pattern without arithmetic reads 6.96
// TB/s with one K-block per wave, 6.52 with two and 6.50 with seven (939 MB),
// and the call takes 67 us against 69 with two (T=1 H=7168 I=2048 K=8).
// Four more waves take turns at finishing tasks: sum of
// the eight parts, SwiGLU, the stores of h, and the quantisation of a
// 128-column block that is complete.  They wait for memory several times a
// task, which a streaming wave could only do by letting its loads run dry.
// The two kinds meet in a ring of kRing sums in LDS with counters, not
// barriers, so no wave waits for the others' memory.
//
// With MX weights (FMT 1 e4m3, 2 e5m2) the rows stay BF16: a K-block's token
// operand (twice the size) is loaded with its weights instead of staying in
// registers, and h is rounded to BF16 column by column, so that its tasks
// need no exchange at all.
template <int NK, int FMT>
__global__ __launch_bounds__(kFc1Threads, 1) void decode_fc1_kernel(DecodeArgs a) {
  __shared__ Routes routes;
  __shared__ DecodePlan plan;
  __shared__ v4f red[kRing][kWaves][2][64];  // [task % kRing][wave][gate, up][lane]
  __shared__ int32_t filled[kRing];           // streaming waves that have put their sums, over all tasks
  __shared__ int32_t emptied[kRing];          // tasks finished
  __shared__ int32_t mapped;                  // finishing waves whose part of the plan stands
  __shared__ float hbuf[2][kCols][128];       // h of a block that one workgroup makes alone, [block parity]
  __shared__ int32_t done[2];                 // its finished sixteenths
  __shared__ float xscale[sizeof(red) / 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int kbs = a.hidden / 128, nb = a.inter / 128;

  const int kb0 = wave * kbs / kWaves, nk = wave < kWaves ? (wave + 1) * kbs / kWaves - kb0 : 0;
  // The streaming waves' token operands (columns past the last token repeat
  // it), while a finishing wave lists the experts.
  v8i xb[NK];
  float sx[NK];
  if (wave == kWaves) {
    if (lane < kRing) filled[lane] = emptied[lane] = 0;
    if (lane < 2) done[lane] = 0;
    if (lane == kRing) mapped = 0;
    const uint32_t bits = check_routes(a, routes, plan, lane);
    if (blockIdx.x == 0 && lane == 0 && a.status) *a.status = bits;
  }
  if constexpr (FMT != 0) {
    // nothing to prepare
  } else if (a.x_scale) {
    if (wave < kWaves && nk > 0) {
      const int64_t t = min(col, a.tokens - 1);
      const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.hidden + (int64_t)kb0 * 128 + grp * 32;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int at = min(k, nk - 1);
        const u32x4* q = reinterpret_cast<const u32x4*>(x + at * 128);
        xb[k] = operand(Frag{q[0], q[1]});
        sx[k] = a.x_scale[t * kbs + kb0 + at];
      }
    }
  } else {
    // BF16 rows: each 128-column block is quantised once, by eight lanes, into
    // the LDS that holds sums later, as many tokens at a time as fit.
    uint8_t* const codes = reinterpret_cast<uint8_t*>(&red[0][0][0][0]);
    const int fit = min(kCols, (int)sizeof(red) / a.hidden);
    for (int t0 = 0; t0 < a.tokens; t0 += fit) {
      const int rows = min(fit, a.tokens - t0);
      for (int g = tid >> 3; g < rows * kbs; g += kFc1Threads / 8) {
        const int t = g / kbs, kb = g - t * kbs, c = kb * 128 + (tid & 7) * 16;
        const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) +
                                                        (int64_t)(t0 + t) * a.hidden + c);
        const u32x4 r[2] = {q[0], q[1]};
        float v[16];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = r[i / 4][i % 4];
          v[2 * i] = bf16_to_f32(w & 0xffffu);
          v[2 * i + 1] = bf16_to_f32(w >> 16);
          m = max(m, max(__float_as_uint(v[2 * i]) & 0x7fffffffu, __float_as_uint(v[2 * i + 1]) & 0x7fffffffu));
        }
        const float scale = __uint_as_float(row8_max(m)) / kE4m3Max;
        const q_u32x2 lo = quant8(v, scale), hi = quant8(v + 8, scale);
        *reinterpret_cast<u32x4*>(codes + t * a.hidden + c) = u32x4{lo[0], lo[1], hi[0], hi[1]};
        if ((tid & 7) == 0) xscale[t * kbs + kb] = scale;
      }
      __syncthreads();
      const int t = min(col, a.tokens - 1) - t0;
      if (nk > 0 && t >= 0 && t < rows) {
        const uint8_t* x = codes + t * a.hidden + kb0 * 128 + grp * 32;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const int at = min(k, nk - 1);
          const u32x4* q = reinterpret_cast<const u32x4*>(x + at * 128);
          xb[k] = operand(Frag{q[0], q[1]});
          sx[k] = xscale[t * kbs + kb0 + at];
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();
  // Tasks.  Whole blocks of 128 columns (eight tasks in a row, whose h never
  // leaves the workgroup) as long as there is one for every workgroup.  The
  // tasks of the blocks that remain are dealt out one by one, unless they are
  // blocks for most workgroups: exchanging h through memory then costs more
  // than the idle ones (208 blocks left for 256 workgroups, T=8 H=7168 I=2048:
  // 222 us dealt out, 212 whole; 128 left, T=1: 68 and 71).
  const int blocks = __builtin_amdgcn_readfirstlane(plan.experts) * nb;
  const int grid = gridDim.x;
  int rounds = FMT == 0 ? blocks / grid : 0;  // of whole blocks
  if (FMT == 0 && (blocks - rounds * grid) * 8 > grid * 5) ++rounds;
  const int whole = 8 * (rounds - (rounds * grid > blocks && (rounds - 1) * grid + (int)blockIdx.x >= blocks ? 1 : 0));
  const int loose = max(blocks - rounds * grid, 0) * 8;
  const int turns = whole + (loose > (int)blockIdx.x ? (loose - (int)blockIdx.x + grid - 1) / grid : 0);
  const auto task_at = [&](int turn, int& n, int& blk, int& sub) {
    int b;
    if (turn < whole) {
      b = (turn >> 3) * grid + (int)blockIdx.x;
      sub = turn & 7;
    } else {
      const int i = (turn - whole) * grid + (int)blockIdx.x;
      b = rounds * grid + (i >> 3);
      sub = i & 7;
    }
    n = b / nb;
    blk = b - n * nb;
  };

  if (wave >= kWaves) {
    // ---- finishing waves: turns wave - kWaves, + kRing, ... ----
    map_routes(a, routes, plan, tid - kThreads, kRing * 64);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (lane == 0) __hip_atomic_fetch_add(&mapped, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    while (__hip_atomic_load(&mapped, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < kRing)
      __builtin_amdgcn_s_sleep(1);
    if (blockIdx.x == 0) {  // FC2 takes the plan from here
      const uint32_t* from = reinterpret_cast<const uint32_t*>(&plan);
      uint32_t* to = reinterpret_cast<uint32_t*>(a.plan);
      for (int i = tid - kThreads; i < (int)(sizeof(DecodePlan) / 4); i += kRing * 64) to[i] = from[i];
    }
    for (int turn = wave - kWaves; turn < turns; turn += kRing) {
      const int buf = turn % kRing, round = turn / kRing;
      while (__hip_atomic_load(&filled[buf], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < kWaves * (round + 1))
        __builtin_amdgcn_s_sleep(1);
      v4f g = red[buf][0][0][lane], u = red[buf][0][1][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        g += red[buf][w][0][lane];
        u += red[buf][w][1][lane];
      }
      if (lane == 0) __hip_atomic_store(&emptied[buf], round + 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
      int n, blk, sub;
      task_at(turn, n, blk, sub);
      // lane l: columns 4 (l / 16) + 0..3 of the tile, token l % 16
      const int slot = plan.row[n * kCols + col];
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = swiglu(g[i], u[i]);
      if constexpr (FMT != 0) {
        if (slot >= 0)
          *reinterpret_cast<q_u32x2*>(a.hb + (int64_t)slot * a.inter + blk * 128 + sub * 16 + grp * 4) =
              q_u32x2{bf16x2_rne(h[0], h[1]), bf16x2_rne(h[2], h[3])};
        continue;
      }
      if (turn < whole) {
        const int par = (turn >> 3) & 1;
        *reinterpret_cast<v4f*>(&hbuf[par][col][sub * 16 + grp * 4]) = v4f{h[0], h[1], h[2], h[3]};
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        int old = 0;
        if (lane == 0) old = __hip_atomic_fetch_add(&done[par], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (__builtin_amdgcn_readfirstlane(old) != 7) continue;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        if (lane == 0) __hip_atomic_store(&done[par], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        // The buffer is free for the block after the next: its first sums can
        // only be put after this wave has emptied a later turn.
        for (int t0 = 0; t0 < a.tokens; t0 += 4) {  // 16 lanes per row, 8 columns each
          const int to = plan.row[n * kCols + t0 + grp];
          if (to < 0) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = hbuf[par][t0 + grp][col * 8 + i];
          store_block(a, v, to, blk, col);
        }
        continue;
      }
      if (slot >= 0) {
        uint64_t* dst = reinterpret_cast<uint64_t*>(a.hf + (int64_t)slot * a.inter + blk * 128 + sub * 16 + grp * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __hip_atomic_store(dst + i, (uint64_t)__float_as_uint(h[2 * i]) | ((uint64_t)__float_as_uint(h[2 * i + 1]) << 32),
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      // The stores are write-through (agent scope) and complete before the
      // arrival; the eighth to arrive at a 128-column block reads it with
      // agent-scope loads, so no cache has to be flushed.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      int old = 0;
      if (lane == 0) {
        int32_t* ctr = a.arrive + n * nb + blk;
        old = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (old == 7) __hip_atomic_store(ctr, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
      }
      if (__builtin_amdgcn_readfirstlane(old) != 7) continue;
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
      for (int t0 = 0; t0 < a.tokens; t0 += 4) {
        const int to = plan.row[n * kCols + t0 + grp];
        if (to < 0) continue;
        const uint64_t* src = reinterpret_cast<const uint64_t*>(a.hf + (int64_t)to * a.inter + blk * 128 + col * 8);
        uint64_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __hip_atomic_load(src + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float((uint32_t)p[i]);
          v[2 * i + 1] = __uint_as_float((uint32_t)(p[i] >> 32));
        }
        store_block(a, v, to, blk, col);
      }
    }
    return;
  }

  // ---- streaming waves ----
  struct Stage {
    Frag g, u;
  };
  Stage st;
  // weights of a turn's column tile; a turn past the last repeats the last
  auto base_of = [&](int turn) -> const uint8_t* {
    int n, blk, sub;
    task_at(min(turn, turns - 1), n, blk, sub);
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[n]);
    return a.w13 + (((int64_t)e * nb + blk) * kbs + kb0) * kTileBytes + sub * kFragBytes + lane * 16;
  };
  // weight scales of the wave's K-blocks: gate in lanes 0.., up in lanes 32..
  auto scales_of = [&](int turn) -> float {
    int n, blk, sub;
    task_at(min(turn, turns - 1), n, blk, sub);
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[n]);
    const int j = min(lane & 31, nk - 1);
    return a.w13_scale[((int64_t)e * 2 * nb + (lane < 32 ? blk : nb + blk)) * kbs + kb0 + j];
  };
  auto load = [&](Stage& s, const uint8_t* base, int k) {
    const uint8_t* p = base + (int64_t)k * kTileBytes;
    s.g = load_frag_nt(p);
    s.u = load_frag_nt(p + 8 * kFragBytes);
  };
  auto put = [&](int turn, const v4f& accg, const v4f& accu) {
    const int buf = turn % kRing, round = turn / kRing;
    while (__hip_atomic_load(&emptied[buf], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < round)
      __builtin_amdgcn_s_sleep(1);
    red[buf][wave][0][lane] = accg;
    red[buf][wave][1][lane] = accu;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (lane == 0) __hip_atomic_fetch_add(&filled[buf], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  };
  if (turns == 0) return;

  if constexpr (FMT != 0) {
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)min(col, a.tokens - 1) * a.hidden;
    struct MxStage {
      Frag g, u;
      u32x4 x[4];
      uint32_t eg[2], eu[2];
    };
    MxStage st;
    int at_turn = 0, at_k = 0;  // next to load
    int shift_next = 0;
    auto load_mx = [&]() {
      int n, blk, sub;
      task_at(at_turn, n, blk, sub);
      const int e = __builtin_amdgcn_readfirstlane(plan.expert[n]);
      const int64_t tile = ((int64_t)e * nb + blk) * kbs + kb0 + at_k;
      const uint8_t* p = a.w13 + tile * kTileBytes + sub * kFragBytes + lane * 16;
      st.g = load_frag_nt(p);
      st.u = load_frag_nt(p + 8 * kFragBytes);
      const uint32_t* w = a.w13_exp + tile * 256 + (sub >> 2) * 64 + mx_word(lane);
      st.eg[0] = w[0];
      st.eg[1] = w[32];
      st.eu[0] = w[128];
      st.eu[1] = w[160];
      load_bf16_k(st.x, x, kb0 + at_k, grp);
      shift_next = 8 * (sub & 3);
      if (++at_k == nk) {
        at_k = 0;
        ++at_turn;
      }
    };
    if (nk > 0) load_mx();
    for (int turn = 0; turn < turns; ++turn) {
      v4f accg = {0.0f, 0.0f, 0.0f, 0.0f}, accu = accg;
      for (int k = 0; k < nk; ++k) {
        const MxStage now = st;
        const int shift = shift_next;
        if (at_turn < turns) load_mx();
        accg += mfma_mx_bf16<FMT == 2>(now.g, now.x, now.eg[0], now.eg[1], shift);
        accu += mfma_mx_bf16<FMT == 2>(now.u, now.x, now.eu[0], now.eu[1], shift);
      }
      put(turn, accg, accu);
    }
    return;
  }
  const uint8_t* base = nullptr;
  float wsc = 0.0f;
  if (nk > 0) {
    base = base_of(0);
    wsc = scales_of(0);
    load(st, base, 0);
  }
  for (int turn = 0; turn < turns; ++turn) {
    v4f accg = {0.0f, 0.0f, 0.0f, 0.0f}, accu = accg;
    if (nk > 0) {
      const uint8_t* next = base_of(turn + 1);
      const float wsc_next = scales_of(turn + 1);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        if (k >= nk) continue;
        const float sg = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsc), k));
        const float su = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsc), 32 + k));
        const v8i wg = operand(st.g), wu = operand(st.u);
        if (k + 1 < nk)
          load(st, base, k + 1);
        else
          load(st, next, 0);
        // FC1 multiplies on the BF16 MFMA, whose sums of exact products keep
        // float32; the FP8 one loses about 2^-11 of the largest product,
        // which moves codes of h across ties (error of the output against 64
        // bits 1.9e-3 to 2.6e-3, here 1.7e-3, its bfloat16 rounding).  The
        // x codes stay narrow: the empty statement keeps the compiler from
        // widening them once for all tasks, for which registers are lacking.
        v4f pg = {0.0f, 0.0f, 0.0f, 0.0f}, pu = pg;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int x0 = xb[k][2 * i], x1 = xb[k][2 * i + 1];
          asm volatile("" : "+v"(x0), "+v"(x1));
          const bf16x8 x = widen8(x0, x1);
          pg = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(wg[2 * i], wg[2 * i + 1]), x, pg, 0, 0, 0);
          pu = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(wu[2 * i], wu[2 * i + 1]), x, pu, 0, 0, 0);
        }
        accg = add_scaled(accg, pg, sx[k], sg);
        accu = add_scaled(accu, pu, sx[k], su);
      }
      base = next;
      wsc = wsc_next;
    }
    put(turn, accg, accu);
  }
}

// ---------------------------------------------------------------------------
// FC2 and the combine
// ---------------------------------------------------------------------------

// Workgroup `tile`: 16 F columns of the output, all tokens.  Wave w takes
// every W-th (expert, K-block) pair of the call, so that the waves read
// neighbouring weight tiles (T=16 H=7168: 230 us for the call against 234 with
// a contiguous share each).
template <int F, int D, int W, int FMT>
__global__ __launch_bounds__(W * 64) void decode_fc2_kernel(DecodeArgs a) {
  __shared__ DecodePlan plan;
  __shared__ v4f red[W][F][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(a.plan);
    uint32_t* to = reinterpret_cast<uint32_t*>(&plan);
    for (int i = tid; i < (int)(sizeof(DecodePlan) / 4); i += W * 64) to[i] = from[i];
  }
  __syncthreads();
  const int ne = __builtin_amdgcn_readfirstlane(plan.experts);
  const int col = lane & 15, grp = lane >> 4;
  const int nb = a.inter / 128, n_tiles = (a.hidden + 255) / 256;
  const int tile = blockIdx.x;
  const int nt = tile * F / 16, rb = tile * F % 16;  // weight tile of 256 rows, its first fragment
  const int pairs = ne * nb;

  struct Stage {
    Frag w[F];
    u32x4 h[FMT == 0 ? 2 : 4];
    uint32_t e[2];                    // MX: exponent words
    float sh, sw, rw;                 // e4m3: scales; the routing weight
    bool there;                       // whether the column's token has a route to the expert
  };
  Stage st[D];
  int ln = wave / nb, lk = wave - ln * nb;  // pair of the next load
  auto load = [&](Stage& s) {
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[ln]);
    const int r = plan.row[ln * kCols + col];
    const int64_t t = ((int64_t)e * n_tiles + nt) * nb + lk;
    const uint8_t* p = a.w2 + t * kTileBytes + rb * kFragBytes + lane * 16;
#pragma unroll
    for (int f = 0; f < F; ++f) s.w[f] = load_frag_nt(p + f * kFragBytes);
    const int64_t hr = r >= 0 ? r : 0;  // some row; the column does not count
    if constexpr (FMT == 0) {
      const u32x4* q = reinterpret_cast<const u32x4*>(a.hq + hr * a.inter + lk * 128 + grp * 32);
      s.h[0] = q[0];
      s.h[1] = q[1];
      s.sh = a.hs[hr * nb + lk];
      s.sw = a.w2_scale[((int64_t)e * (a.hidden / 128) + tile * F / 8) * nb + lk];
    } else {
      load_bf16_k(s.h, a.hb + hr * a.inter, lk, grp);
      const uint32_t* w = a.w2_exp + t * 256 + (rb >> 2) * 64 + mx_word(lane);  // F blocks within one word
#pragma unroll
      for (int i = 0; i < 2; ++i) s.e[i] = w[32 * i];
    }
    s.rw = plan.weight[ln * kCols + col];
    s.there = r >= 0;
    for (lk += W; lk >= nb; lk -= nb) ++ln;
  };
  v4f acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](Stage& s) {
    bf16x8 h[4];  // e4m3: widened
    if constexpr (FMT == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = widen8(s.h[i / 2][i % 2 * 2], s.h[i / 2][i % 2 * 2 + 1]);
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
      v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (FMT == 0) {
        // on the BF16 MFMA, as FC1 (the call takes as long: T=1 66.8 us against
        // 66.3 on the FP8 one, T=8 204.9 against 204.0)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32x4& w = i < 2 ? s.w[f].lo : s.w[f].hi;
          y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w[i % 2 * 2], w[i % 2 * 2 + 1]), h[i], y, 0, 0, 0);
        }
        y = add_scaled(v4f{0.0f, 0.0f, 0.0f, 0.0f}, y, s.sh, s.sw);
      } else
        y = mfma_mx_bf16<FMT == 2>(s.w[f], s.h, s.e[0], s.e[1], 8 * ((rb + f) & 3));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = s.there ? fmaf(s.rw, y[i], acc[f][i]) : acc[f][i];
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + d * W < pairs) load(st[d]);
  for (int p = wave; p < pairs; p += D * W) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (p + d * W >= pairs) break;
      compute(st[d]);
      if (p + (d + D) * W < pairs) load(st[d]);
    }
  }
#pragma unroll
  for (int f = 0; f < F; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  // output pairs of columns: values 2 i, 2 i + 1 of MFMA lane l
  for (int v = tid; v < F * 128; v += W * 64) {
    const int f = v >> 7, l = (v >> 1) & 63, i = (v & 1) * 2;
    const int t = l & 15;
    if (t >= a.tokens) continue;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s0 += red[w][f][l][i];
      s1 += red[w][f][l][i + 1];
    }
    *reinterpret_cast<uint32_t*>(a.out + (int64_t)t * a.hidden + (tile * F + f) * 16 + 4 * (l >> 4) + i) =
        bf16x2_rne(s0, s1);
  }
}

template <int NK, int FMT>
void launch_fc1(const DecodeArgs& a, hipStream_t s) {
  // a task at least per workgroup, at most one workgroup per CU
  const int64_t tasks = (int64_t)(a.tokens * a.top_k) * (a.inter / 16);
  const unsigned grid = (unsigned)(tasks < a.grid ? tasks : a.grid);
  hipLaunchKernelGGL((decode_fc1_kernel<NK, FMT>), dim3(grid), dim3(kFc1Threads), 0, s, a);
}

template <int FMT>
void launch_fc2(const DecodeArgs& a, hipStream_t s) {
  const int tiles = a.hidden / 16;
  // Two tiles per workgroup where that still is a workgroup for three of four
  // CUs (the token operand of a K-block then serves twice the weights: H=7168
  // T=8 202 us against 209); else one, with sixteen waves where the tiles do
  // not fill the CUs (H=2048 T=5 I=768: 29 us against 37 with eight).
  if (tiles * 2 > a.grid * 3)
    hipLaunchKernelGGL((decode_fc2_kernel<2, 2, 8, FMT>), dim3(tiles / 2), dim3(512), 0, s, a);
  else if (tiles > a.grid)
    hipLaunchKernelGGL((decode_fc2_kernel<1, 2, 8, FMT>), dim3(tiles), dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((decode_fc2_kernel<1, 2, 16, FMT>), dim3(tiles), dim3(1024), 0, s, a);
}

}  // namespace

int launch_decode(const DecodeArgs& a, int weight_format, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (weight_format == MOE_WEIGHT_MXFP8_E4M3) {
    launch_fc1<1, 1>(a, s);
    launch_fc2<1>(a, s);
  } else if (weight_format == MOE_WEIGHT_MXFP8_E5M2) {
    launch_fc1<1, 2>(a, s);
    launch_fc2<2>(a, s);
  } else {
    const int per_wave = (a.hidden / 128 + kWaves - 1) / kWaves;  // K-blocks of FC1
    if (per_wave <= 2)
      launch_fc1<2, 0>(a, s);
    else if (per_wave <= 4)
      launch_fc1<4, 0>(a, s);
    else if (per_wave <= 7)
      launch_fc1<7, 0>(a, s);
    else if (per_wave <= 10)
      launch_fc1<10, 0>(a, s);
    else
      launch_fc1<16, 0>(a, s);
    launch_fc2<0>(a, s);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
