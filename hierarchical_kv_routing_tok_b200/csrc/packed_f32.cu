// Causal attention over packed sequences for float32 tensors, forward and backward.
//
//   o_t = sum_{u<=t} p_tu v_u,  p_tu = exp(scale q_t.k_u - lse_t)
//   dp_tu = do_t . v_u,  delta_t = do_t . o_t,  ds_tu = p_tu (dp_tu - delta_t)
//   dq_t = scale sum_u ds_tu k_u,  dk_u = scale sum_t ds_tu q_t,  dv_u = sum_t p_tu do_t
//
// Products on the tensor cores with float32 accuracy: each operand is split into x = hi + lo, two tf32 numbers
// (11 + 11 significant bits), and x y = hi hi' + hi lo' + lo hi' accumulates in float32.  What is left out, lo lo'
// and the last bits of lo, is below 2^-21 of |x y|, less than the float32 accumulation's own rounding over 128 terms.
// Three m16n8k8 products run at 90 TFLOP/s (271 measured for one, against 67 for the FMA pipe), and a fragment
// serves several products, where the FMA pipe would wait for shared memory.
//
// One CTA per (row tile, head): eight warps of 16 rows each, in RW row positions and 8 / RW groups that share out the
// columns of every 64-column tile and meet at the end.  RW = 4 (64 rows, two groups of 32 columns), or 2 (32 rows, four
// groups of 16) while that leaves SMs without work: the longest row
// tile then takes half as long.  Column tiles arrive by 16-byte asynchronous copies, double-buffered; rows outside the
// sequence arrive as zeros.  The rows are queries (forward, dq) or keys (dk, dv).  Every output element has one owner: no
// atomics.  Bound by the tensor pipe (with the splits into tf32 pairs beside it), or, for few tiles, by the longest row
// tile.  4096 tokens, 32/8 heads: forward 50 TFLOP/s (2.75 ms), backward 38 (8.99 ms) of the formulas' products.
#include <math.h>

#include "packed_common.cuh"
#include "tc_common.cuh"

namespace hga {
namespace packed {

namespace {

constexpr int kCols = 64;                  // columns of a tile
constexpr int LD = kD + 4;                 // row stride of a tile in shared memory: no bank conflicts
constexpr int kTileFloats = 64 * LD;
constexpr int kThreads = 256;
constexpr float kLog2eF = 1.4426950408889634f;

// x = hi + lo: hi rounded to tf32 (10 explicit mantissa bits), lo the rest, cut to tf32.  A number that would round to
// infinity gets tf32's largest (an infinite one too: its lo is infinite).  Rounding by an addition and a mask, without that:
// 3 % slower.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four 8 x 4 float matrices: lane l addresses row l mod 8 of matrix l / 8 and receives element (l / 4, l mod 4) of each.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const float* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(tc::smem_u32(p)) : "memory");
}

// The tensor cores cut their sums (round towards zero): a product's chain is kept to 32 inner terms and added to its
// total on the FMA pipe, which rounds to nearest.  (One chain over everything was six times further off: 3.5e-6.)
template <int N>
__device__ __forceinline__ void add(float (&c)[N][4], const float (&x)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] += x[n][e];
}

// c[n][..] = A[16 rows] . B[8 N columns]^T over 128 dims (n: eight columns each).  kSplit: A is already split, its low parts at
// A_lo (backward of the tiny layer below: 137 -> 133 us; 16 warps in place of eight, for more in flight, 150).
template <bool kSplit, int N>
__device__ __forceinline__ void mul_abt(float (&c)[N][4], const float* A, const float* A_lo, const float* B) {
  const int lane = threadIdx.x & 31;
  const float* pa = A + ((lane & 7) + ((lane >> 3) & 1) * 8) * LD + (lane >> 4) * 4;
  const float* pl = A_lo + (pa - A);
  const float* pb = B + ((lane & 7) + (lane >> 4) * 8) * LD + ((lane >> 3) & 1) * 4;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < kD / 8; k0 += 4) {
    float x[N][4] = {};
#pragma unroll
    for (int ks = k0; ks < k0 + 4; ++ks) {
      uint32_t a[4], ah[4], al[4], b[N / 2][4], bh[N / 2][4], bl[N / 2][4];
      if (kSplit) {
        ldsm4(ah, pa + 8 * ks);
        ldsm4(al, pl + 8 * ks);
      } else {
        ldsm4(a, pa + 8 * ks);
      }
#pragma unroll
      for (int y = 0; y < N / 2; ++y) ldsm4(b[y], pb + 16 * y * LD + 8 * ks);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!kSplit) split(__uint_as_float(a[e]), ah[e], al[e]);
#pragma unroll
        for (int y = 0; y < N / 2; ++y) split(__uint_as_float(b[y][e]), bh[y][e], bl[y][e]);
      }
#pragma unroll
      for (int n = 0; n < N; ++n) mma_tf32(x[n], ah, bl[n >> 1][2 * (n & 1)], bl[n >> 1][2 * (n & 1) + 1]);
#pragma unroll
      for (int n = 0; n < N; ++n) mma_tf32(x[n], al, bh[n >> 1][2 * (n & 1)], bh[n >> 1][2 * (n & 1) + 1]);
#pragma unroll
      for (int n = 0; n < N; ++n) mma_tf32(x[n], ah, bh[n >> 1][2 * (n & 1)], bh[n >> 1][2 * (n & 1) + 1]);
    }
    add(c, x);
  }
}

// acc[n][..] += P[16 rows][8 N columns] . B[8 N columns][128 dims].  P is a result fragment of mul_abt: its column
// pair (2t, 2t + 1) of eight serves as the product's inner indexes t, t + 4, with the rows of B taken to match.
// kFinite: values of B that are not finite count as 0 and set *found (0 * inf would not be 0).
template <bool kFinite, int N>
__device__ __forceinline__ void mul_pb(float (&acc)[16][4], const float (&P)[N][4], const float* B, bool* found) {
  const int lane = threadIdx.x & 31;
  const float* pb = B + 2 * (lane & 3) * LD + (lane >> 2);
  uint32_t ah[N][4], al[N][4];
#pragma unroll
  for (int kb = 0; kb < N; ++kb) {
    split(P[kb][0], ah[kb][0], al[kb][0]);
    split(P[kb][2], ah[kb][1], al[kb][1]);
    split(P[kb][1], ah[kb][2], al[kb][2]);
    split(P[kb][3], ah[kb][3], al[kb][3]);
  }
#pragma unroll
  for (int n0 = 0; n0 < 16; n0 += 4) {
    float x[4][4] = {};
#pragma unroll
    for (int kb = 0; kb < N; ++kb) {
      uint32_t bh[4][2], bl[4][2];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float z = pb[(8 * kb + y) * LD + 8 * (n0 + n)];
          if (kFinite && !(fabsf(z) < INFINITY)) {
            z = 0.f;
            *found = true;
          }
          split(z, bh[n][y], bl[n][y]);
        }
#pragma unroll
      for (int n = 0; n < 4; ++n) mma_tf32(x[n], ah[kb], bl[n][0], bl[n][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma_tf32(x[n], al[kb], bh[n][0], bh[n][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma_tf32(x[n], ah[kb], bh[n][0], bh[n][1]);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n0 + n][e] += x[n][e];
  }
}

// Rows t0 .. t0 + R - 1 of head h of a strided tensor into a tile; zeros outside [0, len).
template <int R>
__device__ __forceinline__ void load_tile_async(float* dst, const float* x, Strided s, const Tile& w, int64_t t0, int h) {
#pragma unroll
  for (int i = 0; i < R * (kD / 4) / kThreads; ++i) {
    const int y = i * kThreads + (int)threadIdx.x, r = y / (kD / 4), c = 4 * (y % (kD / 4));
    const int64_t t = t0 + r;
    const bool in = t < w.len;
    const float* src = x + (w.start + (in ? t : 0)) * s.t + h * s.h + c;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + r * LD + c)), "l"(src),
                 "r"(in ? 16u : 0u)
                 : "memory");
  }
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A warp's 16 x 128 result fragments to and from a tile.
__device__ __forceinline__ void put_rows(float* tile, int row0, const float (&acc)[16][4], float f0, float f1) {
  const int lane = threadIdx.x & 31;
  float* p = tile + (row0 + (lane >> 2)) * LD + 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    *reinterpret_cast<float2*>(p + 8 * n) = make_float2(acc[n][0] * f0, acc[n][1] * f0);
    *reinterpret_cast<float2*>(p + 8 * LD + 8 * n) = make_float2(acc[n][2] * f1, acc[n][3] * f1);
  }
}
__device__ __forceinline__ void add_rows(float* tile, int row0, const float (&acc)[16][4], float f0, float f1) {
  const int lane = threadIdx.x & 31;
  float* p = tile + (row0 + (lane >> 2)) * LD + 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    float2* x = reinterpret_cast<float2*>(p + 8 * n);
    float2* y = reinterpret_cast<float2*>(p + 8 * LD + 8 * n);
    *x = make_float2(x->x + acc[n][0] * f0, x->y + acc[n][1] * f0);
    *y = make_float2(y->x + acc[n][2] * f1, y->y + acc[n][3] * f1);
  }
}
// Rows [r0, r1) of a finished tile, scaled, to rows t0 + r of head h of a contiguous output.
__device__ __forceinline__ void store_tile(float* out, const float* tile, int r0, int r1, const Tile& w, int H, int h,
                                           float mul) {
  for (int y = threadIdx.x + r0 * (kD / 4); y < r1 * (kD / 4); y += kThreads) {
    const int r = y / (kD / 4), c = 4 * (y % (kD / 4));
    const int64_t t = (int64_t)w.t0 + r;
    if (t >= w.len) continue;
    float4 v = *reinterpret_cast<const float4*>(tile + r * LD + c);
    v.x *= mul; v.y *= mul; v.z *= mul; v.w *= mul;
    *reinterpret_cast<float4*>(out + ((w.start + t) * H + h) * kD + c) = v;
  }
}

// A tile of R rows split in place: high parts stay, low parts to `lo`.
template <int R>
__device__ __forceinline__ void split_tile(float* x, float* lo) {
#pragma unroll
  for (int i = 0; i < R * (kD / 4) / kThreads; ++i) {
    const int y = i * kThreads + (int)threadIdx.x, at = y / (kD / 4) * LD + 4 * (y % (kD / 4));
    uint4 h, l;
    const float4 v = *reinterpret_cast<const float4*>(x + at);
    split(v.x, h.x, l.x);
    split(v.y, h.y, l.y);
    split(v.z, h.z, l.z);
    split(v.w, h.w, l.w);
    *reinterpret_cast<uint4*>(x + at) = h;
    *reinterpret_cast<uint4*>(lo + at) = l;
  }
}

// The column groups' sums of a row tile meet in `tile`, in the order of the groups.  Called by all threads; ends with a
// barrier.
template <int RW>
__device__ __forceinline__ void meet(float* tile, int grp, int row0, const float (&acc)[16][4], float f0, float f1) {
#pragma unroll
  for (int x = 0; x < 8 / RW; ++x) {
    if (grp == x) {
      if (x == 0) put_rows(tile, row0, acc, f0, f1);
      else add_rows(tile, row0, acc, f0, f1);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------ forward
template <int RW, bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_f32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                          float* __restrict__ o, float* __restrict__ lse, const Work work, const Problem p) {
  extern __shared__ __align__(16) float f32_smem[];
  float* Qs = f32_smem;
  float* Ks = Qs + kTileFloats;            // two stages each
  float* Vs = Ks + 2 * kTileFloats;
  constexpr bool kSplit = RW == 2;         // (64 rows leave no room for the low parts)
  float* Ql = Qs + 32 * LD;                // (the room of 64 rows holds 32 and their low parts)
  __shared__ float s_m[8 / RW][16 * RW], s_l[8 / RW][16 * RW];
  __shared__ int s_found;
  constexpr int kRows = 16 * RW, kGroup = 8 * RW, NC = RW;    // rows of the tile; columns, and their eights, of a group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp / RW, row0 = 16 * (warp % RW);
  const int g = lane >> 2, tq = lane & 3;
  pdl_trigger();
  pdl_wait();
  __shared__ Own own;
  if (kOwn) {
    if (warp == 0) own_tile(work, blockIdx.x / p.Hq, &own);
    __syncthreads();
  }
  if (p.fill_tail) {
    const int64_t worker = (int64_t)blockIdx.x * kThreads + threadIdx.x, workers = (int64_t)gridDim.x * kThreads;
    const int64_t end = end_of<kOwn>(work, own);
    fill_tail_rows(o, p.Hq, end, p.total, worker, workers);
    fill_tail_lse(lse, p.Hq, end, p.total, worker, workers);
  }
  const int h = blockIdx.x % p.Hq, kh = h / p.G;
  if (blockIdx.x >= units_of<kOwn>(work, own, p.Hq)) return;
  const int4 w4 = tile_of<kOwn>(work, own, blockIdx.x / p.Hq);
  const Tile w{w4.x, w4.y, w4.z, 0};
  const int n_tiles = (int)((min((int64_t)w.t0 + kRows, (int64_t)w.len) - 1) / kCols) + 1;
  if (threadIdx.x == 0) s_found = 0;
  load_tile_async<kRows>(Qs, q, p.q, w, w.t0, h);
  load_tile_async<kCols>(Ks, k, p.k, w, 0, kh);
  load_tile_async<kCols>(Vs, v, p.v, w, 0, kh);
  async_commit();

  const float c2 = p.scale * kLog2eF;
  float acc[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  bool found = false;
  for (int j = 0; j < n_tiles; ++j) {
    if (j + 1 < n_tiles) {
      load_tile_async<kCols>(Ks + ((j + 1) & 1) * kTileFloats, k, p.k, w, (int64_t)(j + 1) * kCols, kh);
      load_tile_async<kCols>(Vs + ((j + 1) & 1) * kTileFloats, v, p.v, w, (int64_t)(j + 1) * kCols, kh);
    }
    async_commit();
    async_wait<1>();
    __syncthreads();
    if (kSplit && j == 0) {
      split_tile<kRows>(Qs, Ql);
      __syncthreads();
    }
    const int col0 = j * kCols + kGroup * grp;             // this group's first key
    const int last = w.t0 + row0 + 15 - col0;          // last of them that the warp's last row attends
    if (last >= 0) {
      float s[NC][4];
      mul_abt<kSplit>(s, Qs + row0 * LD, Ql + row0 * LD, Ks + (j & 1) * kTileFloats + kGroup * grp * LD);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int lim = w.t0 + row0 + g + 8 * x - col0; // last key that row g + 8x attends
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& y = s[n][2 * x + e];
            y = 8 * n + 2 * tq + e <= lim ? y * c2 : -INFINITY;
            mx = fmaxf(mx, y);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mnew = fmaxf(m[x], mx), ref = mnew == -INFINITY ? 0.f : mnew;
        const float alpha = exp2f(m[x] - ref);          // 0 when m = -inf
        float rs = 0.f;
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& y = s[n][2 * x + e];
            y = exp2f(y - ref);
            rs += y;
          }
        l[x] = l[x] * alpha + rs;                       // of this thread's columns
        m[x] = mnew;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          acc[n][2 * x] *= alpha;
          acc[n][2 * x + 1] *= alpha;
        }
      }
      mul_pb<true>(acc, s, Vs + (j & 1) * kTileFloats + kGroup * grp * LD, &found);
    }
    __syncthreads();                                    // the stage is free
  }
  // ---- the groups' statistics and outputs meet in the K area
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if (tq == 0) {
      s_m[grp][row0 + g + 8 * x] = m[x];
      s_l[grp][row0 + g + 8 * x] = l[x];
    }
  }
  if (found) s_found = 1;
  __syncthreads();
  float f[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = row0 + g + 8 * x;
    float mt = s_m[0][r];
#pragma unroll
    for (int y = 1; y < 8 / RW; ++y) mt = fmaxf(mt, s_m[y][r]);
    // (every row attends the first key of its sequence, so group 0 has a maximum; a group without keys has sum 0)
    float lt = 0.f;
#pragma unroll
    for (int y = 0; y < 8 / RW; ++y) lt += s_l[y][r] == 0.f ? 0.f : s_l[y][r] * exp2f(s_m[y][r] - mt);
    f[x] = m[x] == -INFINITY ? 0.f : exp2f(m[x] - mt) / lt;
    const int64_t t = (int64_t)w.t0 + r;
    if (grp == 0 && tq == 0 && t < w.len)
      lse[h * p.total + w.start + t] = (mt + log2f(lt)) * 0.6931471805599453f;
  }
  meet<RW>(Ks, grp, row0, acc, f[0], f[1]);
  if (s_found) {
    // values that counted as 0 in the products: each adds itself to the rows that attend it
    for (int y = threadIdx.x; y < kRows * kD; y += kThreads) {
      const int r = y / kD, c = y % kD;
      const int64_t t = (int64_t)w.t0 + r;
      if (t >= w.len) continue;
      float x = Ks[r * LD + c];
      for (int64_t u = 0; u <= t; ++u) {
        const float z = v[(w.start + u) * p.v.t + kh * p.v.h + c];
        if (!(fabsf(z) < INFINITY)) x += z;
      }
      Ks[r * LD + c] = x;
    }
    __syncthreads();
  }
  store_tile(o, Ks, 0, kRows, w, p.Hq, h, 1.f);
}

// ------------------------------------------------------------------------------------ backward: dq
// Forms delta of its rows and leaves it in `delta` [Hq, total] for the dk, dv kernel.
template <int RW, bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_f32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                         const float* __restrict__ o, const float* __restrict__ lse, const float* __restrict__ d_o,
                         float* __restrict__ delta, float* __restrict__ dq, const Work work, const Problem p) {
  extern __shared__ __align__(16) float f32_smem[];
  float* Qs = f32_smem;
  float* Gs = Qs + kTileFloats;
  float* Ks = Gs + kTileFloats;            // two stages each
  float* Vs = Ks + 2 * kTileFloats;
  constexpr bool kSplit = RW == 2;         // (64 rows leave no room for the low parts)
  float *Ql = Qs + 32 * LD, *Gl = Gs + 32 * LD;      // (the room of 64 rows holds 32 and their low parts)
  __shared__ float s_lse[16 * RW], s_delta[16 * RW];
  constexpr int kRows = 16 * RW, kGroup = 8 * RW, NC = RW;    // rows of the tile; columns, and their eights, of a group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp / RW, row0 = 16 * (warp % RW);
  const int g = lane >> 2, tq = lane & 3;
  pdl_trigger();
  pdl_wait();
  __shared__ Own own;
  if (kOwn) {
    if (warp == 0) own_tile(work, blockIdx.x / p.Hq, &own);
    __syncthreads();
  }
  if (p.fill_tail)
    fill_tail_rows(dq, p.Hq, end_of<kOwn>(work, own), p.total, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                   (int64_t)gridDim.x * kThreads);
  const int h = blockIdx.x % p.Hq, kh = h / p.G;
  if (blockIdx.x >= units_of<kOwn>(work, own, p.Hq)) return;
  const int4 w4 = tile_of<kOwn>(work, own, blockIdx.x / p.Hq);
  const Tile w{w4.x, w4.y, w4.z, 0};
  const Strided so{(int64_t)p.Hq * kD, kD};
  const int n_tiles = (int)((min((int64_t)w.t0 + kRows, (int64_t)w.len) - 1) / kCols) + 1;
  load_tile_async<kRows>(Qs, q, p.q, w, w.t0, h);
  load_tile_async<kRows>(Gs, d_o, so, w, w.t0, h);
  load_tile_async<kCols>(Ks, k, p.k, w, 0, kh);
  load_tile_async<kCols>(Vs, v, p.v, w, 0, kh);
  async_commit();
  // delta and lse of the tile's rows: shared out to the warps
  for (int r = kRows / 8 * warp; r < kRows / 8 * (warp + 1); ++r) {
    const int64_t t = (int64_t)w.t0 + r, row = w.start + t;
    float x = 0.f, y = 0.f;
    if (t < w.len) {
      const float4 a = load4(o + (row * p.Hq + h) * kD + 4 * lane), b = load4(d_o + (row * p.Hq + h) * kD + 4 * lane);
      x = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
      y = lse[h * p.total + row] * kLog2eF;
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    if (lane == 0) {
      s_delta[r] = x;
      s_lse[r] = y;
      if (t < w.len) delta[h * p.total + row] = x;
    }
  }
  const float c2 = p.scale * kLog2eF;
  float acc[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  for (int j = 0; j < n_tiles; ++j) {
    if (j + 1 < n_tiles) {
      load_tile_async<kCols>(Ks + ((j + 1) & 1) * kTileFloats, k, p.k, w, (int64_t)(j + 1) * kCols, kh);
      load_tile_async<kCols>(Vs + ((j + 1) & 1) * kTileFloats, v, p.v, w, (int64_t)(j + 1) * kCols, kh);
    }
    async_commit();
    async_wait<1>();
    __syncthreads();
    if (kSplit && j == 0) {
      split_tile<kRows>(Qs, Ql);
      split_tile<kRows>(Gs, Gl);
      __syncthreads();
    }
    const int col0 = j * kCols + kGroup * grp;
    if (w.t0 + row0 + 15 - col0 >= 0) {
      const float* kt = Ks + (j & 1) * kTileFloats + kGroup * grp * LD;
      const float* vt = Vs + (j & 1) * kTileFloats + kGroup * grp * LD;
      float s[NC][4], dp[NC][4];
      mul_abt<kSplit>(s, Qs + row0 * LD, Ql + row0 * LD, kt);
      mul_abt<kSplit>(dp, Gs + row0 * LD, Gl + row0 * LD, vt);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = row0 + g + 8 * x;
        // last key that the row attends; a sequence's first token attends one key, whose ds is 0 (dp - delta would be the
        // rounding of two sums of the same terms)
        const int lim = w.t0 + r < w.len && w.t0 + r > 0 ? w.t0 + r - col0 : -1;
        const float ls = s_lse[r], dl = s_delta[r];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& y = s[n][2 * x + e];
            y = 8 * n + 2 * tq + e <= lim ? exp2f(y * c2 - ls) * (dp[n][2 * x + e] - dl) : 0.f;
          }
      }
      mul_pb<false>(acc, s, kt, nullptr);
    }
    __syncthreads();
  }
  meet<RW>(Ks, grp, row0, acc, 1.f, 1.f);
  store_tile(dq, Ks, 0, kRows, w, p.Hq, h, p.scale);
}

// ------------------------------------------------------------------------------------ backward: dk, dv
// The rows are keys, the columns the queries of the KV head's query heads, one head after another.  When there are
// fewer (tile, KV head) units than SMs, the heads are split over a cluster of cs CTAs; their sums meet through
// distributed shared memory, each CTA adding and storing its share of the rows in the order of the ranks.
template <int RW, bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkdv_f32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                           const float* __restrict__ lse, const float* __restrict__ d_o,
                           const float* __restrict__ delta, float* __restrict__ dk, float* __restrict__ dv,
                           const Work work, const Problem p, int cs) {
  extern __shared__ __align__(16) float f32_smem[];
  float* Ks = f32_smem;
  float* Vs = Ks + kTileFloats;
  float* Qs = Vs + kTileFloats;            // two stages each
  float* Gs = Qs + 2 * kTileFloats;
  constexpr bool kSplit = RW == 2;         // (64 rows leave no room for the low parts)
  float *Kl = Ks + 32 * LD, *Vl = Vs + 32 * LD;      // (the room of 64 rows holds 32 and their low parts)
  __shared__ float s_lse[2][kCols], s_delta[2][kCols];
  constexpr int kRows = 16 * RW, kGroup = 8 * RW, NC = RW;    // rows of the tile; columns, and their eights, of a group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp / RW, row0 = 16 * (warp % RW);
  const int g = lane >> 2, tq = lane & 3;
  pdl_trigger();
  pdl_wait();
  const int rank = blockIdx.x % cs, unit = blockIdx.x / cs;
  __shared__ Own own;
  if (kOwn) {
    if (warp == 0) own_tile(work, unit / p.Hkv, &own);
    __syncthreads();
  }
  if (p.fill_tail) {
    const int64_t worker = (int64_t)blockIdx.x * kThreads + threadIdx.x, workers = (int64_t)gridDim.x * kThreads;
    const int64_t end = end_of<kOwn>(work, own);
    fill_tail_rows(dk, p.Hkv, end, p.total, worker, workers);
    fill_tail_rows(dv, p.Hkv, end, p.total, worker, workers);
  }
  const int kh = unit % p.Hkv;
  if (unit >= units_of<kOwn>(work, own, p.Hkv)) return;        // the whole cluster
  const int4 w4 = tile_of<kOwn>(work, own, unit / p.Hkv);
  const Tile w{w4.x, w4.y, w4.z, 0};
  const Strided so{(int64_t)p.Hq * kD, kD};
  const int hpc = p.G / cs, h0 = kh * p.G + rank * hpc;
  const int per_head = (w.len - w.t0 + kCols - 1) / kCols;      // query tiles from the key tile on
  const int n_tiles = hpc * per_head;
  // tile j's queries and their statistics into stage j mod 2
  auto load_step = [&](int j) {
    const int h = h0 + j / per_head;
    const int64_t t0 = w.t0 + (int64_t)(j % per_head) * kCols;
    load_tile_async<kCols>(Qs + (j & 1) * kTileFloats, q, p.q, w, t0, h);
    load_tile_async<kCols>(Gs + (j & 1) * kTileFloats, d_o, so, w, t0, h);
    if (threadIdx.x < 2 * kCols) {
      const int c = threadIdx.x & (kCols - 1);
      const bool in = t0 + c < w.len;
      const int64_t at = h * p.total + w.start + (in ? t0 + c : 0);
      const bool second = threadIdx.x >= kCols;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                       tc::smem_u32(second ? &s_delta[j & 1][c] : &s_lse[j & 1][c])),
                   "l"((second ? delta : lse) + at), "r"(in ? 4u : 0u)
                   : "memory");
    }
  };
  load_tile_async<kRows>(Ks, k, p.k, w, w.t0, kh);
  load_tile_async<kRows>(Vs, v, p.v, w, w.t0, kh);
  load_step(0);
  async_commit();
  const float c2 = p.scale * kLog2eF;
  float gk[16][4], gv[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) gk[n][e] = gv[n][e] = 0.f;
  for (int j = 0; j < n_tiles; ++j) {
    if (j + 1 < n_tiles) load_step(j + 1);
    async_commit();
    async_wait<1>();
    __syncthreads();
    if (kSplit && j == 0) {
      split_tile<kRows>(Ks, Kl);
      split_tile<kRows>(Vs, Vl);
      __syncthreads();
    }
    const int col0 = w.t0 + j % per_head * kCols + kGroup * grp;      // this group's first query
    if (col0 + kGroup - 1 >= w.t0 + row0 && col0 < w.len) {
      const float* qt = Qs + (j & 1) * kTileFloats + kGroup * grp * LD;
      const float* gt = Gs + (j & 1) * kTileFloats + kGroup * grp * LD;
      float s[NC][4], dp[NC][4];
      mul_abt<kSplit>(s, Ks + row0 * LD, Kl + row0 * LD, qt);
      mul_abt<kSplit>(dp, Vs + row0 * LD, Vl + row0 * LD, gt);
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 8 * n + 2 * tq + e, t = col0 + c;
          const float ls = s_lse[j & 1][kGroup * grp + c] * kLog2eF, dl = s_delta[j & 1][kGroup * grp + c];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool seen = t >= w.t0 + row0 + g + 8 * x && t < w.len;
            const float y = seen ? exp2f(s[n][2 * x + e] * c2 - ls) : 0.f;
            s[n][2 * x + e] = y;
            dp[n][2 * x + e] = seen && t > 0 ? y * (dp[n][2 * x + e] - dl) : 0.f;   // (token 0: one key, ds = 0)
          }
        }
      mul_pb<false>(gv, s, gt, nullptr);
      mul_pb<false>(gk, dp, qt, nullptr);
    }
    __syncthreads();
  }
  // ---- the groups meet (dK in the first Q stage, dV in the second), then the cluster's CTAs
  float* tk = Qs;
  float* tv = Qs + kTileFloats;
  meet<RW>(tk, grp, row0, gk, 1.f, 1.f);
  meet<RW>(tv, grp, row0, gv, 1.f, 1.f);
  if (cs == 1) {
    store_tile(dk, tk, 0, kRows, w, p.Hkv, kh, p.scale);
    store_tile(dv, tv, 0, kRows, w, p.Hkv, kh, 1.f);
    return;
  }
  tc::cluster_sync();
  const int r0 = kRows * rank / cs, r1 = kRows * (rank + 1) / cs;
  for (int y = threadIdx.x + r0 * (kD / 4); y < r1 * (kD / 4); y += kThreads) {
    const int r = y / (kD / 4), c = 4 * (y % (kD / 4));
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int x = 0; x < cs; ++x) {
      float4 u[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32((z ? tv : tk) + r * LD + c)), "r"(x));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u[z].x), "=f"(u[z].y), "=f"(u[z].z), "=f"(u[z].w) : "r"(at) : "memory");
      }
      a.x += u[0].x; a.y += u[0].y; a.z += u[0].z; a.w += u[0].w;
      b.x += u[1].x; b.y += u[1].y; b.z += u[1].z; b.w += u[1].w;
    }
    const int64_t t = (int64_t)w.t0 + r;
    if (t >= w.len) continue;
    const int64_t at = ((w.start + t) * p.Hkv + kh) * kD + c;
    *reinterpret_cast<float4*>(dk + at) = make_float4(a.x * p.scale, a.y * p.scale, a.z * p.scale, a.w * p.scale);
    *reinterpret_cast<float4*>(dv + at) = b;
  }
  tc::cluster_sync();                                   // no CTA leaves while its sums are being read
}

// ------------------------------------------------------------------------------------ host side
template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t grid, size_t smem, unsigned cluster, cudaStream_t st, A... args) {
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), smem, st, cluster, args...);
}
constexpr size_t kTileBytesF = kTileFloats * sizeof(float);

}  // namespace

// Whether 64-row tiles leave SMs without work (units: heads of one tile): then tiles of 32.  Forward + backward, 975 tokens
// in five sequences, 4/1 heads: 72 + 219 us with 64 rows, 41 + 126 with 32; 4096 tokens, 32/8 heads: 2746 + 8985 us against
// 3247 + 9885 (each tile's keys serve half as many rows).
int f32_tile(int64_t total, int n_seqs, int units) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return list_capacity(total, n_seqs, 64) * units < sms ? 32 : 64;
}

cudaError_t launch_fwd_f32(const void* q, const void* k, const void* v, void* o, float* lse, const Work& work,
                           const Problem& p, cudaStream_t st) {
  const int tile = f32_tile(p.total, p.n_seqs, p.Hq);
  const int64_t n = list_capacity(p.total, p.n_seqs, tile) * p.Hq;
  auto kernel = tile == 64 ? packed_fwd_f32_kernel<4, false>
                : work.cu  ? packed_fwd_f32_kernel<2, true>
                           : packed_fwd_f32_kernel<2, false>;
  return launch(kernel, n < 1 ? 1 : n, 5 * kTileBytesF, 1, st,
                (const float*)q, (const float*)k, (const float*)v, (float*)o, lse, work, p);
}

cudaError_t launch_bwd_f32(const void* q, const void* k, const void* v, const void* o, const float* lse,
                           const void* d_o, float* delta, void* dq, void* dk, void* dv, const Work& by_query,
                           const Work& by_key, const Problem& p, cudaStream_t st) {
  // (both lists by the query heads: a cluster may share out the heads of a key tile)
  const int tile = f32_tile(p.total, p.n_seqs, p.Hq);
  const int64_t tiles = list_capacity(p.total, p.n_seqs, tile);
  const int64_t nq = tiles * p.Hq, nk = tiles * p.Hkv;
  auto dq_kernel = tile == 64    ? packed_dq_f32_kernel<4, false>
                   : by_query.cu ? packed_dq_f32_kernel<2, true>
                                 : packed_dq_f32_kernel<2, false>;
  auto dkdv_kernel = tile == 64  ? packed_dkdv_f32_kernel<4, false>
                     : by_key.cu ? packed_dkdv_f32_kernel<2, true>
                                 : packed_dkdv_f32_kernel<2, false>;
  cudaError_t e = launch(dq_kernel, nq < 1 ? 1 : nq, 6 * kTileBytesF,
                         1, st, (const float*)q, (const float*)k, (const float*)v, (const float*)o, lse,
                         (const float*)d_o, delta, (float*)dq, by_query, p);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // The largest split of the heads into a portable cluster, while there are fewer key tiles than SMs.  Whole backward pass with
  // one CTA per key tile and with the split: the tiny batch above 322 and 126 us (4/1 heads: four CTAs), 300 tokens 8/1 heads
  // 278 and 65 (eight), 1000 tokens 6/1 heads 682 and 186 (six), 512 tokens 32/8 heads 448 and 201 (four).
  int cs = 1;
  if (nk < sms)
    for (int c = 2; c <= 8; ++c)
      if (p.G % c == 0) cs = c;
  return launch(dkdv_kernel, (nk < 1 ? 1 : nk) * cs,
                6 * kTileBytesF, (unsigned)cs, st, (const float*)q, (const float*)k, (const float*)v, lse,
                (const float*)d_o, (const float*)delta, (float*)dk, (float*)dv, by_key, p, cs);
}

}  // namespace packed
}  // namespace hga
