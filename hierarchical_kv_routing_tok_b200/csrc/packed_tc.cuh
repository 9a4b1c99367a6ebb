// What the tensor-core kernels of packed attention share.
//
// A query tile has 128 rows = pk query heads of one KV head x 128 / pk tokens (row r: token r / pk, head
// r % pk), so that short sequences and the causal diagonal waste few rows and each K/V tile serves pk
// heads.  pk is the largest power of two, up to 8, that divides the query heads per KV head.  Eleven sequences of 1 to 8192
// tokens, 32/8 heads: forward 719 us with 4, 774 with 1; one of 16K: 1819 and 1841; backward, twelve short sequences, 32/4
// heads: 133 us with 8, 154 with 1.
#pragma once

#include <cuda.h>

#include "packed_common.cuh"
#include "tc_common.cuh"

namespace hga {
namespace packed {

constexpr int kBN = 128;                          // keys per tile
constexpr uint32_t kHalfBytes = 128 * 128;        // one 64-dim half of a 128-row bf16 tile
constexpr uint32_t kTileBytes = 2 * kHalfBytes;
constexpr float kLog2eF = 1.4426950408889634f;

inline int packed_heads(int G) { return G % 8 == 0 ? 8 : G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1; }

// bf16 map of a [total, H, 128] tensor with element strides; boxes of {64 dims, heads, tokens}, 128-byte
// swizzle (a box lands as tokens x heads rows of 128 bytes).  Coordinates: (dim, head, token).
bool make_map_packed(CUtensorMap* m, const void* base, int H, int64_t total, Strided s, int heads, int tokens);

// Work unit u of a list of query tiles: units = head units of a tile, side by side, tiles heaviest first.
// CTA c of G takes the units c, 2G-1-c, 2G+c, ... : a snake over the list, which deals out the long ones
// evenly.
__device__ __forceinline__ int64_t unit_of_cta(int k, int c, int G) {
  const int64_t round = k >> 1;
  return (k & 1) ? (2 * round + 2) * G - 1 - c : 2 * round * G + c;
}

// 64 bytes of a row as bf16: whole 32-byte sectors when the tensor is 32-byte aligned.
__device__ __forceinline__ void store32(__nv_bfloat16* dst, const uint32_t (&pk)[16], bool v8) {
  if (v8) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * y), "r"(pk[8 * y]),
                   "r"(pk[8 * y + 1]), "r"(pk[8 * y + 2]), "r"(pk[8 * y + 3]), "r"(pk[8 * y + 4]), "r"(pk[8 * y + 5]),
                   "r"(pk[8 * y + 6]), "r"(pk[8 * y + 7])
                   : "memory");
  } else {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int y = 0; y < 4; ++y) d4[y] = make_uint4(pk[4 * y], pk[4 * y + 1], pk[4 * y + 2], pk[4 * y + 3]);
  }
}

// tc::mbar_wait_w with one suspending try in front: what a wait costs when its phase is complete stands between a
// tensor-core kernel's products.  (Limits below kPollLimitNs poll, so that they expire.)
__device__ __forceinline__ bool wait_w(uint32_t bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns) {
  if (limit_ns >= tc::kPollLimitNs && __all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  return tc::mbar_wait_w(bar, parity, abort, status, limit_ns);
}

// ---- pairs of floats: one instruction for two multiply-adds
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A bf16 tile (n_rows rows, two 64-dim halves of half_bytes) in shared memory made safe for a product in which some of
// its rows meet zeros: rows at or past `rows` become zeros.  Called by a warp.
__device__ __forceinline__ void zero_rows(uint32_t tile, int n_rows, uint32_t half_bytes, int rows) {
  const int lane = threadIdx.x & 31;
  for (int h = 0; h < 2; ++h)
    for (int x = max(rows, 0) * 8 + lane; x < n_rows * 8; x += 32)      // 16-byte pieces
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + h * half_bytes + x * 16), "r"(0) : "memory");
  tc::fence_proxy_async_smem();
}
// Marks (0x8000, 0x80000000) the halves of a bf16 pair that are not finite: exponent bits all ones.
__device__ __forceinline__ uint32_t not_finite_mask(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// The values of a tile of `pieces` 16-byte pieces (a multiple of 256) that are not finite become zeros.  Called by a warp;
// returns (warp-uniform) whether there are any.  Eight pieces in flight per lane and no branch while all is finite.
__device__ __forceinline__ bool zero_not_finite(uint32_t tile, int pieces) {
  const int lane = threadIdx.x & 31;
  uint32_t found = 0;
#pragma unroll 1
  for (int b = 0; b < pieces; b += 256) {
    uint32_t w[8][4], any = 0;
#pragma unroll
    for (int y = 0; y < 8; ++y)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[y][0]), "=r"(w[y][1]), "=r"(w[y][2]), "=r"(w[y][3])
                   : "r"(tile + (b + 32 * y + lane) * 16));
#pragma unroll
    for (int y = 0; y < 8; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= not_finite_mask(w[y][e]);
    if (any) {
      found = 1;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t m = not_finite_mask(w[y][e]);
          if (m & 0x8000u) w[y][e] &= 0xffff0000u;
          if (m & 0x80000000u) w[y][e] &= 0x0000ffffu;
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + (b + 32 * y + lane) * 16), "r"(w[y][0]),
                     "r"(w[y][1]), "r"(w[y][2]), "r"(w[y][3]) : "memory");
      }
    }
  }
  tc::fence_proxy_async_smem();
  return __any_sync(0xffffffffu, found != 0);
}

}  // namespace packed
}  // namespace hga
