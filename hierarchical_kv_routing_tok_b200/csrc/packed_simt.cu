// Causal attention over packed sequences on the CUDA cores, forward and backward, in float32
// arithmetic: the float32 path, and the path of any type when the CUDA cores are asked for.
//
//   o_t = sum_{u<=t} p_tu v_u,  p_tu = exp(scale q_t.k_u - lse_t)
//   dp_tu = do_t . v_u,  delta_t = do_t . o_t,  ds_tu = p_tu (dp_tu - delta_t)
//   dq_t = scale sum_u ds_tu k_u,  dk_u = scale sum_t ds_tu q_t,  dv_u = sum_t p_tu do_t
//
// One CTA per (64-token tile of a sequence, head); the tiles come from the plan kernel, heaviest
// first.  A tile walks the other side in 64-token tiles staged in shared memory, each thread holding
// a 4 x 4 block of the 64 x 64 products and a 4 x 8 block of the 64 x 128 ones.  Rows outside the
// sequence are read as zeros.  Every output element has one owner: no atomics.
// Bound by the FMA pipe and the shared-memory reads that feed it (about one 16-byte read per eight
// FMAs).
#include <math.h>

#include "packed_common.cuh"
#include "simt_tile.cuh"

namespace hga {
namespace packed {

using namespace simt;

// out[i][0..7] += sum_{k <= lim[i]} P[4ty+i][k] V[k][cols]: keys past a row's limit are left out whatever
// they hold (0 * NaN is not 0).
__device__ __forceinline__ void mm_p_v_limit(const float* P, const float* V, float out[4][8], const int lim[4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
  for (int k = 0; k < BN; ++k) {
    const float4 v0 = *reinterpret_cast<const float4*>(V + k * LD + 4 * tx);
    const float4 v1 = *reinterpret_cast<const float4*>(V + k * LD + 64 + 4 * tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k <= lim[i]) {
        const float p = P[(4 * ty + i) * LP + k];
        out[i][0] += p * v0.x; out[i][1] += p * v0.y; out[i][2] += p * v0.z; out[i][3] += p * v0.w;
        out[i][4] += p * v1.x; out[i][5] += p * v1.y; out[i][6] += p * v1.z; out[i][7] += p * v1.w;
      }
    }
  }
}

// Row t of head h of a strided tensor; nullptr outside the sequence.
template <typename T>
__device__ __forceinline__ const T* row_of(const T* x, Strided s, const Tile& w, int64_t t, int h) {
  return t < w.len ? x + (w.start + t) * s.t + h * s.h : nullptr;
}

template <typename T>
__device__ __forceinline__ void store_row(T* dst, const float v[8], float mul) {
  const int tx = threadIdx.x % 16;
  store4(dst + 4 * tx, make_float4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul));
  store4(dst + 64 + 4 * tx, make_float4(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul));
}

// ------------------------------------------------------------------------------------ forward
template <typename T>
__global__ void __launch_bounds__(kThreads) packed_fwd_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                              const T* __restrict__ v, T* __restrict__ o,
                                                              float* __restrict__ lse, const Header* hdr,
                                                              const Tile* list, const Problem p) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + BM * LD;
  float* Vs = Ks + BN * LD;
  float* Ps = Vs + BN * LD;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_trigger();
  pdl_wait();
  if (p.fill_tail) {
    const int64_t worker = (int64_t)blockIdx.x * kThreads + threadIdx.x, workers = (int64_t)gridDim.x * kThreads;
    fill_tail_rows(o, p.Hq, hdr->end, p.total, worker, workers);
    fill_tail_lse(lse, p.Hq, hdr->end, p.total, worker, workers);
  }
  const int h = blockIdx.x % p.Hq, kh = h / p.G;
  if ((int)(blockIdx.x / p.Hq) >= hdr->n_tiles[0]) return;
  const Tile w = list[blockIdx.x / p.Hq];
  load_tile<T>(Qs, [&](int r) { return row_of(q, p.q, w, (int64_t)w.t0 + r, h); }, p.scale * kLog2e);

  float m[4], l[4], acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY; l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
  }
  const int64_t n_keys = min((int64_t)w.t0 + BM, (int64_t)w.len);
  for (int64_t k0 = 0; k0 < n_keys; k0 += BN) {
    __syncthreads();
    load_tile<T>(Ks, [&](int r) { return row_of(k, p.k, w, k0 + r, kh); }, 1.f);
    load_tile<T>(Vs, [&](int r) { return row_of(v, p.v, w, k0 + r, kh); }, 1.f);
    __syncthreads();
    float s[4][4] = {};
    mm_rows_cols(Qs, Ks, s);
    int lim[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lim[i] = (int)min((int64_t)w.t0 + 4 * ty + i - k0, (int64_t)BN);   // last key of the tile that the row sees
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (tx + 16 * j > lim[i]) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = half_warp_max(mx);
      const float mnew = fmaxf(m[i], mx);
      const float ref = (mnew == -INFINITY) ? 0.f : mnew;
      const float alpha = exp2f(m[i] - ref);           // 0 when m = -inf
      float rs = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - ref);
        Ps[(4 * ty + i) * LP + tx + 16 * j] = e;
        rs += e;
      }
      l[i] = l[i] * alpha + half_warp_sum(rs);
      m[i] = mnew;
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[i][c] *= alpha;
    }
    __syncthreads();
    if (k0 + BN <= w.t0) mm_p_v(Ps, Vs, acc);
    else mm_p_v_limit(Ps, Vs, acc, lim);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = (int64_t)w.t0 + 4 * ty + i;
    if (t >= w.len) continue;
    const int64_t row = w.start + t;
    store_row(o + (row * p.Hq + h) * kD, acc[i], 1.f / l[i]);
    if (tx == 0) lse[h * p.total + row] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------------------------ backward: dq
// Forms delta of its rows and leaves it in `delta` [Hq, total] for the dk, dv kernel.
template <typename T>
__global__ void __launch_bounds__(kThreads) packed_dq_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                             const T* __restrict__ v, const T* __restrict__ o,
                                                             const float* __restrict__ lse, const T* __restrict__ d_o,
                                                             float* __restrict__ delta, T* __restrict__ dq,
                                                             const Header* hdr, const Tile* list, const Problem p) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Gs = Qs + BM * LD;
  float* Ks = Gs + BM * LD;
  float* Vs = Ks + BN * LD;
  float* Ds = Vs + BN * LD;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_trigger();
  pdl_wait();
  if (p.fill_tail)
    fill_tail_rows(dq, p.Hq, hdr->end, p.total, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                   (int64_t)gridDim.x * kThreads);
  const int h = blockIdx.x % p.Hq, kh = h / p.G;
  if ((int)(blockIdx.x / p.Hq) >= hdr->n_tiles[0]) return;
  const Tile w = list[blockIdx.x / p.Hq];
  const Strided so{(int64_t)p.Hq * kD, kD};
  // O first where K will be: only delta needs it
  load_tile<T>(Qs, [&](int r) { return row_of(q, p.q, w, (int64_t)w.t0 + r, h); }, p.scale * kLog2e);
  load_tile<T>(Gs, [&](int r) { return row_of(d_o, so, w, (int64_t)w.t0 + r, h); }, 1.f);
  load_tile<T>(Ks, [&](int r) { return row_of(o, so, w, (int64_t)w.t0 + r, h); }, 1.f);
  __syncthreads();
  float dl[4], ls[4], acc[4][8] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) x += Gs[r * LD + tx + 16 * c] * Ks[r * LD + tx + 16 * c];
    dl[i] = half_warp_sum(x);
    const int64_t t = (int64_t)w.t0 + r, row = w.start + t;
    ls[i] = 0.f;
    if (t < w.len) {
      ls[i] = lse[h * p.total + row] * kLog2e;
      if (tx == 0) delta[h * p.total + row] = dl[i];
    }
  }
  const int64_t n_keys = min((int64_t)w.t0 + BM, (int64_t)w.len);
  for (int64_t k0 = 0; k0 < n_keys; k0 += BN) {
    __syncthreads();
    load_tile<T>(Ks, [&](int r) { return row_of(k, p.k, w, k0 + r, kh); }, 1.f);
    load_tile<T>(Vs, [&](int r) { return row_of(v, p.v, w, k0 + r, kh); }, 1.f);
    __syncthreads();
    float s[4][4] = {}, dp[4][4] = {};
    mm_rows_cols(Qs, Ks, s);
    mm_rows_cols(Gs, Vs, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = (int64_t)w.t0 + 4 * ty + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool seen = k0 + tx + 16 * j <= t && t < w.len;
        Ds[(4 * ty + i) * LP + tx + 16 * j] = seen ? exp2f(s[i][j] - ls[i]) * (dp[i][j] - dl[i]) : 0.f;
      }
    }
    __syncthreads();
    mm_p_v(Ds, Ks, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = (int64_t)w.t0 + 4 * ty + i;
    if (t < w.len) store_row(dq + ((w.start + t) * p.Hq + h) * kD, acc[i], p.scale);
  }
}

// ------------------------------------------------------------------------------------ backward: dk, dv
// One CTA per (64-key tile, KV head); the query heads of the KV head are summed in registers.
template <typename T>
__global__ void __launch_bounds__(kThreads) packed_dkdv_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                               const T* __restrict__ v,
                                                               const float* __restrict__ lse,
                                                               const T* __restrict__ d_o,
                                                               const float* __restrict__ delta, T* __restrict__ dk,
                                                               T* __restrict__ dv, const Header* hdr,
                                                               const Tile* list, const Problem p) {
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + BN * LD;
  float* Qs = Vs + BN * LD;
  float* Gs = Qs + BM * LD;
  float* Ps = Gs + BM * LD;
  float* Ds = Ps + BN * LP;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_trigger();
  pdl_wait();
  if (p.fill_tail) {
    const int64_t worker = (int64_t)blockIdx.x * kThreads + threadIdx.x, workers = (int64_t)gridDim.x * kThreads;
    fill_tail_rows(dk, p.Hkv, hdr->end, p.total, worker, workers);
    fill_tail_rows(dv, p.Hkv, hdr->end, p.total, worker, workers);
  }
  const int kh = blockIdx.x % p.Hkv;
  if ((int)(blockIdx.x / p.Hkv) >= hdr->n_tiles[1]) return;
  const Tile w = list[blockIdx.x / p.Hkv];
  const Strided so{(int64_t)p.Hq * kD, kD};
  load_tile<T>(Ks, [&](int r) { return row_of(k, p.k, w, (int64_t)w.t0 + r, kh); }, 1.f);
  load_tile<T>(Vs, [&](int r) { return row_of(v, p.v, w, (int64_t)w.t0 + r, kh); }, 1.f);
  float gk[4][8] = {}, gv[4][8] = {};
  const float c2 = p.scale * kLog2e;
  for (int g = 0; g < p.G; ++g) {
    const int h = kh * p.G + g;
    const float* lse_h = lse + h * p.total + w.start;
    const float* delta_h = delta + h * p.total + w.start;
    for (int64_t t0 = w.t0; t0 < w.len; t0 += BM) {
      __syncthreads();
      load_tile<T>(Qs, [&](int r) { return row_of(q, p.q, w, t0 + r, h); }, 1.f);
      load_tile<T>(Gs, [&](int r) { return row_of(d_o, so, w, t0 + r, h); }, 1.f);
      __syncthreads();
      float s[4][4] = {}, dp[4][4] = {};       // rows: keys, columns: queries
      mm_rows_cols(Ks, Qs, s);
      mm_rows_cols(Vs, Gs, dp);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + tx + 16 * j;
        const bool in = t < w.len;
        const float ls = in ? lse_h[t] * kLog2e : 0.f, dl = in ? delta_h[t] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool seen = in && (int64_t)w.t0 + 4 * ty + i <= t;
          const float e = seen ? exp2f(s[i][j] * c2 - ls) : 0.f;
          Ps[(4 * ty + i) * LP + tx + 16 * j] = e;
          Ds[(4 * ty + i) * LP + tx + 16 * j] = seen ? e * (dp[i][j] - dl) : 0.f;
        }
      }
      __syncthreads();
      mm_p_v(Ps, Gs, gv);
      mm_p_v(Ds, Qs, gk);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t u = (int64_t)w.t0 + 4 * ty + i;
    if (u >= w.len) continue;
    store_row(dk + ((w.start + u) * p.Hkv + kh) * kD, gk[i], p.scale);
    store_row(dv + ((w.start + u) * p.Hkv + kh) * kD, gv[i], 1.f);
  }
}

// ------------------------------------------------------------------------------------ host side
namespace {
constexpr size_t kTileBytes = (size_t)BM * LD * sizeof(float), kProdBytes = (size_t)BM * LP * sizeof(float);

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t grid, size_t smem, cudaStream_t st, A... args) {
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)(grid < 1 ? 1 : grid)), dim3(kThreads), smem, st, 1, args...);
}

template <typename T>
cudaError_t fwd(const void* q, const void* k, const void* v, void* o, float* lse, const Header* hdr, const Tile* list,
                const Problem& p, cudaStream_t st) {
  return launch(packed_fwd_kernel<T>, list_capacity(p.total, p.n_seqs, kSimtTile) * p.Hq, 3 * kTileBytes + kProdBytes,
                st, (const T*)q, (const T*)k, (const T*)v, (T*)o, lse, hdr, list, p);
}
template <typename T>
cudaError_t bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* d_o,
                float* delta, void* dq, void* dk, void* dv, const Header* hdr, const Tile* by_query,
                const Tile* by_key, const Problem& p, cudaStream_t st) {
  const int64_t n = list_capacity(p.total, p.n_seqs, kSimtTile);
  cudaError_t e = launch(packed_dq_kernel<T>, n * p.Hq, 4 * kTileBytes + kProdBytes, st, (const T*)q, (const T*)k,
                         (const T*)v, (const T*)o, lse, (const T*)d_o, delta, (T*)dq, hdr, by_query, p);
  if (e != cudaSuccess) return e;
  return launch(packed_dkdv_kernel<T>, n * p.Hkv, 4 * kTileBytes + 2 * kProdBytes, st, (const T*)q, (const T*)k,
                (const T*)v, lse, (const T*)d_o, (const float*)delta, (T*)dk, (T*)dv, hdr, by_key, p);
}
}  // namespace

cudaError_t launch_fwd_simt(bool bf16, const void* q, const void* k, const void* v, void* o, float* lse,
                            const Header* hdr, const Tile* list, const Problem& p, cudaStream_t st) {
  return (bf16 ? fwd<__nv_bfloat16> : fwd<float>)(q, k, v, o, lse, hdr, list, p, st);
}
cudaError_t launch_bwd_simt(bool bf16, const void* q, const void* k, const void* v, const void* o, const float* lse,
                            const void* d_o, float* delta, void* dq, void* dk, void* dv, const Header* hdr,
                            const Tile* by_query, const Tile* by_key, const Problem& p, cudaStream_t st) {
  return (bf16 ? bwd<__nv_bfloat16> : bwd<float>)(q, k, v, o, lse, d_o, delta, dq, dk, dv, hdr, by_query, by_key, p,
                                                  st);
}

}  // namespace packed
}  // namespace hga
