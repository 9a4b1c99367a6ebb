// What the packed attention kernels share: the problem as the kernels see it.
#pragma once

#include "packed_plan.cuh"

namespace hga {
namespace packed {

// A [total, H, 128] tensor with element strides.
struct Strided {
  int64_t t, h;
};

struct Problem {
  int Hq, Hkv, G, n_seqs;
  int64_t total;
  Strided q, k, v;       // o, d_o, dq, dk, dv are contiguous
  float scale;
  int fill_tail;
  int* status;
  uint64_t wait_ns;
};

int f32_tile(int64_t total, int n_seqs, int units);   // tokens per tile of the float32 kernels
constexpr int kKeyTile = 128;  // keys per CTA of the bf16 dK, dV kernel
constexpr int kLeastTile = 16; // no kernel's tiles are shorter
int fwd_tile(int G);           // tokens per unit of the bf16 forward
int dq_tile(int G);            // tokens per unit of the bf16 dQ

int head_units(int Hkv, int G); // units of a tile of the bf16 forward and dQ

cudaError_t launch_fwd_f32(const void* q, const void* k, const void* v, void* o, float* lse, const Work& work,
                           const Problem& p, cudaStream_t st);
cudaError_t launch_bwd_f32(const void* q, const void* k, const void* v, const void* o, const float* lse,
                           const void* d_o, float* delta, void* dq, void* dk, void* dv, const Work& by_query,
                           const Work& by_key, const Problem& p, cudaStream_t st);
cudaError_t launch_fwd_tc(const void* q, const void* k, const void* v, void* o, void* o_lo, float* lse,
                          const Work& work, const Problem& p, cudaStream_t st);
cudaError_t launch_bwd_tc(const void* q, const void* k, const void* v, const void* o, const void* o_lo,
                          const float* lse, const void* d_o, float* stats, void* dq, void* dk, void* dv,
                          const Work& by_query, const Work& by_key, const Problem& p, cudaStream_t st);

// Rows of no sequence: zeros in a [total, H, 128] output, -inf in lse [H, total].  Called by every
// thread of a grid of kernels that share the work by (worker, workers).
template <typename T>
__device__ __forceinline__ void fill_tail_rows(T* x, int H, int64_t end, int64_t total, int64_t worker,
                                               int64_t workers) {
  const int64_t n = (total - end) * H * (kD * (int64_t)sizeof(T) / 16);
  uint4* p = reinterpret_cast<uint4*>(x + end * H * kD);
  for (int64_t i = worker; i < n; i += workers) p[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void fill_tail_lse(float* lse, int H, int64_t end, int64_t total, int64_t worker,
                                              int64_t workers) {
  const int64_t rows = total - end, n = rows * H;
  for (int64_t i = worker; i < n; i += workers) lse[(i / rows) * total + end + i % rows] = -INFINITY;
}

}  // namespace packed
}  // namespace hga
