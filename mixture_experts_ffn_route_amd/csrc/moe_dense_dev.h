// Device helpers of the dense products (moe_linear.hip, moe_ffn.hip): LDS-DMA,
// the LDS layouts of operand tiles, and tile order.
//
// A product is out[m, n] = sum_k L[m, k] R[n, k].  R is the MFMA's row operand
// and L its column operand, so a lane's four results are four consecutive n of
// one m.  An operand tile is ROWS rows (of m or n) by one K-block of 128 bytes
// (128 e4m3 codes, 64 bfloat16 values), and lies in memory in one of two ways:
//
// K inside (kKin): a row's K-block is 128 consecutive bytes.  In LDS chunk c (16
// bytes) of row r sits at position 8 r + (c ^ swz(r)) of 16 bytes: one DMA
// instruction fetches 8 whole lines.  Lane l reads row l % 16, chunk 2 (l / 16) + s
// for the halves s of the K-block: a 16-byte read is served in groups of lanes
// like 0-3, 12-15, 20-23, 24-27, which then meet distinct banks (with chunk
// 4 s + l / 16 they do not: 4 cycles more a read of 8).
//
// K outside (kKout, bfloat16): rows are consecutive in memory, one line of
// memory a k.  LDS-transposing reads (ds_read_b64_tr_b16) turn it: 16 lanes
// that read a 4 (k) x 16 (rows) block get a row's 4 values each.  Lane l of the
// MFMA holds k = 16 (l / 16) + 8 s + [0, 8) of row l % 16, as above, so one block
// is k = 16 g + 8 s + 4 h + [0, 4), and the reads h of the four lane groups g
// together take 512 bytes.  DMA instruction (s, q, h, j) fetches the 8 lines
// g = 2 j, 2 j + 1 of rows [64 q, 64 q + 64) and lays them down so that each of
// its 4 blocks of 16 rows has 256 consecutive bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_quant_dev.h"

namespace moe {
namespace dense {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kLine = 128;  // bytes of a K-block in one row

// LDS-DMA: lane l's 16 bytes land at lds_base + 16 l.  Inline asm, so that the
// compiler's own waits never drain a ring; the kernels wait on vmcnt
// themselves, and the "memory" clobber keeps LDS accesses in program order.
__device__ __forceinline__ uint32_t lds_addr(const lds_u8* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}
__device__ __forceinline__ const void* uniform_ptr(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const void*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}
// from a wave-uniform base and a per-lane byte offset
__device__ __forceinline__ void dma16(const void* base, uint32_t off, const lds_u8* to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(uniform_ptr(base)), "s"(lds_addr(to)) : "memory", "m0");
}
// the same of lines that are read once
__device__ __forceinline__ void dma16_nt(const void* base, uint32_t off, const lds_u8* to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
               :: "v"(off), "s"(uniform_ptr(base)), "s"(lds_addr(to)) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, const lds_u8* to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(uniform_ptr(base)), "s"(lds_addr(to)) : "memory", "m0");
}
// from a per-lane address
__device__ __forceinline__ void dma16_at(const void* src, const lds_u8* to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(src), "s"(lds_addr(to)) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

// A float at a wave-uniform address that no wave writes, through the scalar cache
// (and so not counted among the loads in flight).
__device__ __forceinline__ float scalar_f32(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)uniform_ptr(p);
}

// 16 bytes of zeros that lanes past the end of K read instead
__device__ const u32x4 kZeros = {0, 0, 0, 0};

// how an operand lies in memory
enum { kKin = 0, kKout = 1 };

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// One operand of a tile: `rows` valid rows from `base` on (the tile's first
// row), `stride` bytes between memory lines (rows for kKin, k for kKout).
struct Operand {
  const uint8_t* base;
  int64_t stride;
  int rows;
};

// Piece p (1 KB, one DMA instruction) of K-block kb of a tile of ROWS rows,
// into the tile at `lds`.  k_valid: values (kKout: lines; kKin: bytes) of this
// K-block that exist; the others become zeros.  Rows past the last valid one
// repeat it (their results are not stored).
template <int LAYOUT>
__device__ __forceinline__ uint32_t piece_offset(const Operand& o, int p, int lane) {
  if constexpr (LAYOUT == kKin) {
    const int v = p * 64 + lane, r = v >> 3, c = (v & 7) ^ swz(r & 15);
    return (uint32_t)min(r, o.rows - 1) * (uint32_t)o.stride + (uint32_t)c * 16u;
  } else {
    const int j = p & 1, h = (p >> 1) & 1, s = (p >> 2) & 1, q = p >> 3;
    const int b = lane >> 4, g = 2 * j + ((lane >> 3) & 1), r = (lane >> 1) & 3, c = lane & 1;
    const int k = 16 * g + 8 * s + 4 * h + r, n = 64 * q + 16 * b + 8 * c;
    return (uint32_t)k * (uint32_t)o.stride + (uint32_t)min(n, o.rows - 8) * 2u;
  }
}
// Whether this lane's 16 bytes of piece p lie within k_valid.
template <int LAYOUT>
__device__ __forceinline__ bool piece_valid(int p, int lane, int k_valid) {
  if constexpr (LAYOUT == kKin) {
    const int v = p * 64 + lane, r = v >> 3, c = (v & 7) ^ swz(r & 15);
    return c * 16 < k_valid;
  } else {
    const int j = p & 1, h = (p >> 1) & 1, s = (p >> 2) & 1;
    const int g = 2 * j + ((lane >> 3) & 1), r = (lane >> 1) & 3;
    return 16 * g + 8 * s + 4 * h + r < k_valid;
  }
}

// Byte offset in a tile of the 16 bytes of chunk c of row r (kKin).
__device__ __forceinline__ int chunk_at(int r, int c) { return 16 * (8 * r + (c ^ swz(r & 15))); }

__device__ __forceinline__ u32x4 lds16(const lds_u8* p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(p);
}

// Fragment of 16 rows [16 b, 16 b + 16) of a bfloat16 tile, k = 16 (l / 16) + 8 s + [0, 8).
template <int LAYOUT>
__device__ __forceinline__ v8bf frag_bf16(const lds_u8* tile, int b, int s, int lane) {
  if constexpr (LAYOUT == kKin) {
    return __builtin_bit_cast(v8bf, lds16(tile + b * 2048 + chunk_at(lane & 15, 2 * (lane >> 4) + s)));
  } else {
    typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
    const lds_u8* p = tile + (b >> 2) * 8192 + s * 4096 + (b & 3) * 256 + (lane >> 5) * 1024 + ((lane >> 4) & 1) * 128 +
                      (lane & 15) * 8;
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 2048));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// Fragment of 16 rows of an e4m3 tile: lane l holds k = 32 (l / 16) + [0, 32) of row l % 16.
__device__ __forceinline__ v8i frag_fp8(const lds_u8* tile, int b, int lane) {
  const u32x4 lo = lds16(tile + b * 2048 + chunk_at(lane & 15, 2 * (lane >> 4)));
  const u32x4 hi = lds16(tile + b * 2048 + chunk_at(lane & 15, 2 * (lane >> 4) + 1));
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Tile of workgroup `id`: workgroup i runs on XCD i % 8, and each XCD takes one
// contiguous range of the tiles, `deep` row tiles at a time, so that the
// workgroups on its L2 share rows and weights.  Returns false past the end.
__device__ __forceinline__ bool tile_of(int id, int m_tiles, int n_tiles, int deep, int& mt, int& nt) {
  const int total = m_tiles * n_tiles, per = (total + 7) / 8;
  const int v = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || v >= total) return false;
  const int group = v / (deep * n_tiles), rem = v - group * deep * n_tiles;
  const int m0 = group * deep, gm = min(deep, m_tiles - m0);
  mt = m0 + rem % gm;
  nt = rem / gm;
  return true;
}
inline int tile_grid(int64_t tiles) { return (int)((tiles + 7) / 8 * 8); }

// e4m3 codes of 4 values of a block with scale s, code i in byte i: quotients
// from a reciprocal and one correction step, below 2^-90, where a remainder
// could underflow, from a division; a block whose scale is zero or not finite
// has codes zero or NaN.
__device__ __forceinline__ uint32_t quant4(const float v[4], float s) {
  if (s == 0.0f || !isfinite(s)) return codes_without_scale(s)[0];
  const float inv = 1.0f / s;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q0 = v[i] * inv;
    q[i] = s >= 0x1p-90f ? copysignf(fmaf(fmaf(-q0, s, v[i]), inv, q0), v[i]) : v[i] / s;
  }
  return (uint32_t)cvt2_e4m3(q[2], q[3], cvt2_e4m3(q[0], q[1], 0, false), true);
}

// derivative factors of silu(g) u: of u and of g
__device__ __forceinline__ void dswiglu(float g, float u, float dh, float& dg, float& du) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.44269504f));
  du = dh * (g * s);
  dg = dh * u * (s * (1.0f + g * (1.0f - s)));
}

}  // namespace dense
}  // namespace moe
