// The layer for a few tokens (moe_layer_decode): at most 16 of them, two
// launches, on the layer's own weight tiles and with its arithmetic.
//
//   decode_fc1_kernel   x -> e4m3 1x128 (or given so), gate and up rows,
//                       h = silu(g) u, h -> e4m3 1x128
//   decode_fc2_kernel   y = h W2^T, out[t] = bf16(sum_k w[t, k] y_k)
//
// The weights of the chosen experts are the whole traffic, so everything is
// arranged around streaming them once:
//  * The MFMA takes 16 weight rows x 16 tokens x 128, and 16 columns hold
//    every token: no staging, no compaction and no token tiles.  A lane's
//    weight operand is 32 bytes of the create-time tiles, loaded straight into
//    registers, 1 KB per instruction.
//  * A workgroup takes few output columns of one expert (FC1) or of all of
//    them (FC2), and its eight waves split the K-blocks, so that a single
//    token's few experts still make several hundred workgroups.  The waves'
//    sums meet in LDS at the end.
//  * A token's operand for a K-block is 32 of its columns per lane, which the
//    lane loads and (for BF16 input) quantises itself; the block maximum takes
//    two lane swaps.
//  * h is quantised per 128 columns, which several workgroups make: each
//    stores its FP32 columns and the last to arrive quantises the block.
//  * FC2 adds the experts' rows in FP32 with the routing weights applied to
//    the partial sums, so there are no y rows and no combine.
#include <hip/hip_runtime.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_quant_dev.h"

namespace moe {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int kCols = 16;                // tokens at most: MFMA columns
constexpr int kSlots = kCols * 8;        // routes at most
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
__device__ __forceinline__ v4f mfma_e4m3(const Frag& a, const v8i& b) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), b, zero, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
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

// Maximum over the four lanes that share a token (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ uint32_t col_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// The routes of the call, staged by every workgroup for itself: checked ids
// (-1 masked) and weights in LDS, with moe_stage_inputs' rules.
struct Routes {
  int32_t id[kSlots];
  float w[kSlots];
  uint32_t status;
};
__device__ __forceinline__ void stage_routes(const DecodeArgs& a, Routes& r, int32_t* raw) {
  const int n = a.tokens * a.top_k, i = threadIdx.x;
  int id = -1;
  float w = 0.0f;
  if (i < n) {
    id = a.topk_idx[i];
    w = a.topk_w[i];
  }
  if (i == 0) r.status = 0u;
  uint32_t bits = 0;
  if (id < -1 || id >= a.num_experts) {
    bits = MOE_DEV_BAD_EXPERT;
    id = -1;
  }
  if (i < kSlots) raw[i] = id;
  __syncthreads();
  if (i < kSlots) {
    if ((a.flags & MOE_FLAG_CHECK_ROUTES) && id >= 0) {
      // the lowest slot of an id stays, whatever its weight
      const int first = i - i % a.top_k;
      bool again = false;
      for (int j = first; j < i; ++j) again |= raw[j] == id;
      if (again) {
        bits |= MOE_DEV_DUPLICATE;
        id = -1;
      } else if (!isfinite(w)) {
        bits |= MOE_DEV_NONFINITE;
        id = -1;
      }
    }
    r.id[i] = id;
    r.w[i] = id >= 0 ? w : 0.0f;
    if (bits) atomicOr(&r.status, bits);
  }
  __syncthreads();
}

// Slot of expert e's first route, from the ballots over a wave's two halves
// of the slots.
__device__ __forceinline__ int first_slot(const Routes& r, int e, int lane) {
  const uint64_t lo = __ballot(r.id[lane] == e), hi = __ballot(r.id[64 + lane] == e);
  return lo ? __builtin_ctzll(lo) : (hi ? 64 + __builtin_ctzll(hi) : kSlots);
}

// ---------------------------------------------------------------------------
// FC1
// ---------------------------------------------------------------------------

// Workgroup (tile, slot): 16 F columns of h of the expert of route `slot`, if
// that is its first route.  Wave w takes K-blocks [w kbs / 8, (w + 1) kbs / 8).
template <int F, bool BF16, int D>
__global__ __launch_bounds__(kThreads) void decode_fc1_kernel(DecodeArgs a) {
  __shared__ Routes routes;
  __shared__ int32_t raw[kSlots];
  __shared__ v4f red[kWaves][2 * F][64];
  __shared__ int32_t col_slot[kCols];  // route of each column's token, -1 past the last
  __shared__ int32_t last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, tile = blockIdx.x;
  stage_routes(a, routes, raw);
  if (a.status && slot == 0 && tile == 0 && tid == 0) *a.status = routes.status;
  const int e = __builtin_amdgcn_readfirstlane(routes.id[slot]);
  if (e < 0 || first_slot(routes, e, lane) != slot) return;

  // the expert's tokens, in order, one per column
  if (tid < kCols) col_slot[tid] = -1;
  __syncthreads();
  if (wave == 0) {
    int mine = -1;
    if (lane < a.tokens)
      for (int k = a.top_k - 1; k >= 0; --k)
        if (routes.id[lane * a.top_k + k] == e) mine = lane * a.top_k + k;
    const uint64_t has = __ballot(mine >= 0);
    if (mine >= 0) col_slot[__popcll(has & ((1ull << lane) - 1))] = mine;
  }
  __syncthreads();
  const int col = lane & 15, grp = lane >> 4;
  const int my_slot = col_slot[col] >= 0 ? col_slot[col] : slot;  // spare columns repeat the first
  const int64_t t = my_slot / a.top_k;

  const int kbs = a.hidden / 128;
  const int kb0 = wave * kbs / kWaves, kb1 = (wave + 1) * kbs / kWaves;
  constexpr int kPer128 = 8 / F;  // tiles per 128 columns
  const int blk = tile / kPer128, sub = tile % kPer128;
  const uint8_t* wbase =
      a.w13 + ((int64_t)e * (a.inter / 128) + blk) * kbs * (int64_t)kTileBytes + sub * F * kFragBytes + lane * 16;
  const uint8_t* x8 = static_cast<const uint8_t*>(a.x) + t * a.hidden + grp * 32;
  const uint16_t* x16 = static_cast<const uint16_t*>(a.x) + t * a.hidden + grp * 32;
  // the wave's weight scales: gate in lanes 0.., up in lanes 32..
  const int nb = a.inter / 128;
  float wsc = 0.0f;
  {
    const int j = kb0 + (lane & 31);
    if (j < kb1) wsc = a.w13_scale[((int64_t)e * 2 * nb + (lane < 32 ? blk : nb + blk)) * kbs + j];
  }

  struct Stage {
    Frag g[F], u[F];
    u32x4 x[BF16 ? 4 : 2];
    float sx;
  };
  Stage st[D];
  auto load = [&](Stage& s, int kb) {
    const uint8_t* p = wbase + (int64_t)kb * kTileBytes;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      s.g[f] = load_frag_nt(p + f * kFragBytes);
      s.u[f] = load_frag_nt(p + (8 + f) * kFragBytes);
    }
    if constexpr (BF16) {
      const u32x4* q = reinterpret_cast<const u32x4*>(x16 + kb * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) s.x[i] = q[i];
    } else {
      const u32x4* q = reinterpret_cast<const u32x4*>(x8 + kb * 128);
      s.x[0] = q[0];
      s.x[1] = q[1];
      s.sx = a.x_scale[t * kbs + kb];
    }
  };
  v4f accg[F], accu[F];
#pragma unroll
  for (int f = 0; f < F; ++f) accg[f] = accu[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](Stage& s, int kb) {
    v8i b;
    float sx;
    if constexpr (BF16) {
      float v[32];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t w = s.x[i / 4][i % 4];
        v[2 * i] = bf16_to_f32(w & 0xffffu);
        v[2 * i + 1] = bf16_to_f32(w >> 16);
        m = max(m, max(__float_as_uint(v[2 * i]) & 0x7fffffffu, __float_as_uint(v[2 * i + 1]) & 0x7fffffffu));
      }
      sx = __uint_as_float(col_max(m)) / kE4m3Max;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const q_u32x2 c = quant8(v + 8 * i, sx);
        b[2 * i] = (int)c[0];
        b[2 * i + 1] = (int)c[1];
      }
    } else {
      b = operand(Frag{s.x[0], s.x[1]});
      sx = s.sx;
    }
    const int j = kb - kb0;
    const float sg = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsc), j));
    const float su = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsc), 32 + j));
#pragma unroll
    for (int f = 0; f < F; ++f) {
      accg[f] = add_scaled(accg[f], mfma_e4m3(s.g[f], b), sx, sg);
      accu[f] = add_scaled(accu[f], mfma_e4m3(s.u[f], b), sx, su);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (kb0 + d < kb1) load(st[d], kb0 + d);
  for (int kb = kb0; kb < kb1; kb += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (kb + d >= kb1) break;
      compute(st[d], kb + d);
      if (kb + d + D < kb1) load(st[d], kb + d + D);
    }
  }
#pragma unroll
  for (int f = 0; f < F; ++f) {
    red[wave][f][lane] = accg[f];
    red[wave][F + f][lane] = accu[f];
  }
  __syncthreads();

  // h of the tile: value i of MFMA lane l is column 16 f + 4 (l / 16) + i of
  // token column l % 16
  const int c128 = blk * 128;
  for (int v = tid; v < F * 256; v += kThreads) {
    const int f = v >> 8, l = (v >> 2) & 63, i = v & 3;
    const int to = col_slot[l & 15];
    if (to < 0) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      g += red[w][f][l][i];
      u += red[w][F + f][l][i];
    }
    __hip_atomic_store(a.hf + (int64_t)to * a.inter + c128 + (sub * F + f) * 16 + 4 * (l >> 4) + i, swiglu(g, u),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // The stores are write-through (agent scope) and complete before the
  // arrival; the workgroup that arrives last reads the whole block with
  // agent-scope loads, so no cache has to be flushed.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  int32_t* ctr = a.arrive + (int64_t)slot * nb + blk;
  if (tid == 0) {
    last = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == kPer128 - 1;
    if (last) __hip_atomic_store(ctr, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
  }
  __syncthreads();
  if (!last) return;
  const int to = (tid >> 4) < kCols ? col_slot[tid >> 4] : -1;
  if (to < 0) return;  // whole groups of 16 lanes
  const int c = c128 + (tid & 15) * 8;
  float h[8];
  uint32_t m = 0;
  const uint64_t* src = reinterpret_cast<const uint64_t*>(a.hf + (int64_t)to * a.inter + c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t p = __hip_atomic_load(src + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    h[2 * i] = __uint_as_float((uint32_t)p);
    h[2 * i + 1] = __uint_as_float((uint32_t)(p >> 32));
    m = max(m, max((uint32_t)p & 0x7fffffffu, (uint32_t)(p >> 32) & 0x7fffffffu));
  }
  const float s = __uint_as_float(row16_max(m)) / kE4m3Max;
  *reinterpret_cast<q_u32x2*>(a.hq + (int64_t)to * a.inter + c) = quant8(h, s);
  if ((tid & 15) == 0) a.hs[(int64_t)to * nb + blk] = s;
}

// ---------------------------------------------------------------------------
// FC2 and the combine
// ---------------------------------------------------------------------------

// Workgroup `tile`: 16 F columns of the output, all tokens.  The (expert,
// K-block) pairs of the call are split evenly over the waves in order.
template <int F, int D>
__global__ __launch_bounds__(kThreads) void decode_fc2_kernel(DecodeArgs a) {
  __shared__ Routes routes;
  __shared__ int32_t raw[kSlots];
  __shared__ int32_t expert[kSlots];          // the call's experts, by first route
  __shared__ int16_t row[kSlots][kCols];      // route of (expert, token), -1 none
  __shared__ int32_t n_experts;
  __shared__ v4f red[kWaves][F][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  stage_routes(a, routes, raw);
  const int n = a.tokens * a.top_k;
  if (wave == 0) {
    // first routes of the lane's two slots
    bool f0 = routes.id[lane] >= 0, f1 = routes.id[64 + lane] >= 0;
    for (int j = 0; j < n; ++j) {
      const int o = routes.id[j];
      if (j < lane && o == routes.id[lane]) f0 = false;
      if (j < 64 + lane && o == routes.id[64 + lane]) f1 = false;
    }
    const uint64_t b0 = __ballot(f0), b1 = __ballot(f1), below = (1ull << lane) - 1;
    if (f0) expert[__popcll(b0 & below)] = routes.id[lane];
    if (f1) expert[__popcll(b0) + __popcll(b1 & below)] = routes.id[64 + lane];
    if (lane == 0) n_experts = __popcll(b0) + __popcll(b1);
  }
  __syncthreads();
  const int ne = __builtin_amdgcn_readfirstlane(n_experts);
  for (int i = tid; i < ne * kCols; i += kThreads) {
    const int t = i & 15, e = expert[i >> 4];
    int r = -1;
    if (t < a.tokens)
      for (int k = a.top_k - 1; k >= 0; --k)
        if (routes.id[t * a.top_k + k] == e) r = t * a.top_k + k;
    row[i >> 4][t] = (int16_t)r;
  }
  __syncthreads();

  const int col = lane & 15, grp = lane >> 4;
  const int nb = a.inter / 128, n_tiles = (a.hidden + 255) / 256;
  const int tile = blockIdx.x;
  const int nt = tile * F / 16, rb = tile * F % 16;  // weight tile of 256 rows, its first fragment
  const int pairs = ne * nb;
  const int p0 = wave * pairs / kWaves, p1 = (wave + 1) * pairs / kWaves;

  struct Stage {
    Frag w[F];
    u32x4 h[2];
    float sh, sw, rw;
  };
  Stage st[D];
  int ln = p0 / nb, lk = p0 - ln * nb;  // pair of the next load
  auto load = [&](Stage& s) {
    const int e = __builtin_amdgcn_readfirstlane(expert[ln]);
    const int r = row[ln][col];
    const uint8_t* p =
        a.w2 + (((int64_t)e * n_tiles + nt) * nb + lk) * (int64_t)kTileBytes + rb * kFragBytes + lane * 16;
#pragma unroll
    for (int f = 0; f < F; ++f) s.w[f] = load_frag_nt(p + f * kFragBytes);
    const int64_t hr = r >= 0 ? r : 0;
    const u32x4* q = reinterpret_cast<const u32x4*>(a.hq + hr * a.inter + lk * 128 + grp * 32);
    s.h[0] = q[0];
    s.h[1] = q[1];
    s.sh = a.hs[hr * nb + lk];
    s.sw = a.w2_scale[((int64_t)e * (a.hidden / 128) + tile * F / 8) * nb + lk];
    // the weights of a repeated id add up (only without route checks)
    float rw = 0.0f;
    if (r >= 0) {
      rw = routes.w[r];
      for (int k = r + 1; k < (r / a.top_k + 1) * a.top_k; ++k)
        if (routes.id[k] == e) rw += routes.w[k];
    }
    s.rw = r >= 0 ? rw : 0.0f;
    if (r < 0) s.sh = -1.0f;  // a scale is not negative: the column has no such route
    if (++lk == nb) {
      lk = 0;
      ++ln;
    }
  };
  v4f acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](Stage& s) {
    const v8i b = operand(Frag{s.h[0], s.h[1]});
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const v4f y = add_scaled(v4f{0.0f, 0.0f, 0.0f, 0.0f}, mfma_e4m3(s.w[f], b), s.sh, s.sw);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[f][i] = s.sh < 0.0f ? acc[f][i] : fmaf(s.rw, y[i], acc[f][i]);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (p0 + d < p1) load(st[d]);
  for (int p = p0; p < p1; p += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (p + d >= p1) break;
      compute(st[d]);
      if (p + d + D < p1) load(st[d]);
    }
  }
#pragma unroll
  for (int f = 0; f < F; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  // output pairs of columns: values 2 i, 2 i + 1 of MFMA lane l
  for (int v = tid; v < F * 128; v += kThreads) {
    const int f = v >> 7, l = (v >> 1) & 63, i = (v & 1) * 2;
    const int t = l & 15;
    if (t >= a.tokens) continue;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      s0 += red[w][f][l][i];
      s1 += red[w][f][l][i + 1];
    }
    *reinterpret_cast<uint32_t*>(a.out + (int64_t)t * a.hidden + (tile * F + f) * 16 + 4 * (l >> 4) + i) =
        bf16x2_rne(s0, s1);
  }
}

}  // namespace

int launch_decode(const DecodeArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  constexpr int F1 = 2, F2 = 1;
  const dim3 g1(a.inter / (16 * F1), a.tokens * a.top_k), g2(a.hidden / (16 * F2)), block(kThreads);
  if (a.x_scale)
    hipLaunchKernelGGL((decode_fc1_kernel<F1, false, 3>), g1, block, 0, s, a);
  else
    hipLaunchKernelGGL((decode_fc1_kernel<F1, true, 2>), g1, block, 0, s, a);
  hipLaunchKernelGGL((decode_fc2_kernel<F2, 4>), g2, block, 0, s, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace moe
