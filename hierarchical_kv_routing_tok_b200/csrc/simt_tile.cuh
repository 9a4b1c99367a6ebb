// Tiles of the CUDA-core attention kernels (float32 arithmetic): 64-row tiles of 128 dims in shared
// memory, and their products with a 4 x 4 or 4 x 8 block of results per thread of 256.
#pragma once

#include "common.cuh"

namespace hga {
namespace simt {

constexpr int BM = 64;            // query rows per CTA
constexpr int BN = 64;            // keys per tile
constexpr int LD = kD + 4;        // padded row stride of [64][128] tiles (floats)
constexpr int LP = BN + 4;        // padded row stride of [64][64] tiles
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Load a [64][128] tile of rows given by row_ptr(r) (nullptr = zero row) into smem, scaled.
template <typename T, typename RowPtr>
__device__ __forceinline__ void load_tile(float* dst, RowPtr row_ptr, float mul) {
  constexpr int N = Vec16<T>::N;
  constexpr int LPR = kD / N;                    // threads per row
  constexpr int RPI = kThreads / LPR;            // rows per iteration
  const int col = (threadIdx.x % LPR) * N;
  for (int r = threadIdx.x / LPR; r < BN; r += RPI) {
    const T* src = row_ptr(r);
    float v[N];
    if (src) {
      Vec16<T>::load(src + col, v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < N; e += 4)
      store4(dst + r * LD + col + e, make_float4(v[e] * mul, v[e + 1] * mul, v[e + 2] * mul, v[e + 3] * mul));
  }
}

// acc[i][j] += A[4ty+i] . B[tx+16j] over 128 dims (A, B: [64][LD] smem tiles).
__device__ __forceinline__ void mm_rows_cols(const float* A, const float* Bt, float acc[4][4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
  for (int d = 0; d < kD; d += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(Bt + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
  }
}

// out[i][0..7] += sum_k P[4ty+i][k] * V[k][cols], cols = 4tx..4tx+3, 64+4tx..64+4tx+3.
__device__ __forceinline__ void mm_p_v(const float* P, const float* V, float out[4][8]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
  for (int k = 0; k < BN; ++k) {
    const float4 v0 = *reinterpret_cast<const float4*>(V + k * LD + 4 * tx);
    const float4 v1 = *reinterpret_cast<const float4*>(V + k * LD + 64 + 4 * tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = P[(4 * ty + i) * LP + k];
      out[i][0] += p * v0.x; out[i][1] += p * v0.y; out[i][2] += p * v0.z; out[i][3] += p * v0.w;
      out[i][4] += p * v1.x; out[i][5] += p * v1.y; out[i][6] += p * v1.z; out[i][7] += p * v1.w;
    }
  }
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace simt
}  // namespace hga
