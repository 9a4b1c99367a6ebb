// Causal attention over packed sequences, backward, on the tensor cores (tcgen05, bf16).
//
//   P = exp(scale Q K^T - lse), dP = dO V^T, delta = rowsum(dO o O), dS = P o (dP - delta),
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO   (dK, dV summed over a KV head's query heads)
//
// Two kernels, each owning its outputs (no atomics on sums): dQ over query tiles, which also forms delta, then
// dK/dV over key tiles.  Both recompute P, so the pair does seven products where five would do.  Bound by the
// tensor pipe and the element-wise work between the products (exp, two fused multiply-adds, two packings per
// score): 16,373 tokens in eleven sequences, 32/8 heads, 2.18 ms over ten passes,
// 805 TFLOP/s of the formulas' products (a long run is at the power limit); tensor pipe active for 60 % of the cycles.
//
// Rows outside a sequence are in its last tiles (they belong to its neighbours): they are masked where they
// are rows or columns of S, and zeroed in shared memory where they are summed over (a masked 0 times a value
// that is not finite would not be 0).
//
// P and dS are rounded to bf16 for their second products, the operand type that takes K, Q and dO as they are: each adds
// about as much as the rounding of the result (dv: 2.3e-3 of the norm, 1.7e-3 from rounding the exact one).
// In dQ and dK, whose norms lie most in a sequence's first tokens, the diagonal takes what the rounding left of dS as a
// further operand.  dQ: 2.5e-3 -> 2.05e-3, for 2130 -> 2150 us of the packed 16K batch (every tile: 1.8e-3 and 2370).  dK:
// 2.4e-3 -> 2.0e-3, sequences of one tile 2.4e-3 -> 1.75e-3, for 2165 -> 2177 us (twelve short sequences, 32/4 heads: 127 -> 133;
// one of 3000, 4/1: 158 -> 147, which is the split of the loop).
#include <cuda_bf16.h>

#include "packed_tc.cuh"

namespace hga {
namespace packed {

using namespace tc;

namespace {

struct BwdParams {
  int Hq, Hkv, G, pk;
  int64_t total;
  float c2, scale;                         // scale * log2(e), scale
  const __nv_bfloat16* o;
  const __nv_bfloat16* o_lo;               // or nullptr
  const float* lse;                        // [Hq, total]
  float* stats;                            // [2][Hq, total]: -lse log2(e), -delta; written by dQ for dK, dV
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  Work work;
  int fill_tail;
  int* status;
  uint64_t wait_ns;
};

// ======================================================================================== dQ
namespace dq {

constexpr int KS = 3;                      // K stages (a K tile lives until its dQ products are done)
constexpr int VS = 2;                      // V stages (a V tile lives until its dP products are done)
constexpr int kEW = 16;                    // element-wise warps, four per 32 key columns
constexpr int kThreads = 128 + 32 * kEW;

struct Smem {
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kDO = kQ + kTileBytes;
  static constexpr uint32_t kK = kDO + kTileBytes;
  static constexpr uint32_t kV = kK + KS * kTileBytes;
  static constexpr uint32_t kBar = kV + VS * kTileBytes;
  // qdo_full, kv_full[KS], k_empty[KS], v_empty[VS], s_full[2], dp_full, dp_free, ds_full[2], dq_ready,
  // mma_done, qdo_empty, delta_bar, qdo_issued, k_clean[KS]
  static constexpr int kNumBars = 1 + 2 * KS + VS + 11 + KS;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;
  static constexpr uint32_t kOwn = (kMisc + 16 + 15) & ~15u;
  static constexpr uint32_t kBytes = kOwn + sizeof(Own);
};
static_assert(Smem::kBytes + 1024 <= 227 * 1024, "shared memory");

struct Unit {
  int start, len, t0, h0, kh, T;
};
template <bool kOwn>
__device__ __forceinline__ bool load_unit(const BwdParams& p, const Own& own, int64_t n_units, int k, Unit* x) {
  const int64_t u = unit_of_cta(k, blockIdx.x, gridDim.x);
  if (u >= n_units) return false;
  const int per = p.G / p.pk, hus = p.Hkv * per;
  const int4 w = tile_of<kOwn>(p.work, own, u / hus);
  const int hu = (int)(u % hus);
  x->start = w.x;
  x->len = w.y;
  x->t0 = w.z;
  x->kh = hu / per;
  x->h0 = x->kh * p.G + (hu % per) * p.pk;
  x->T = (int)((min((int64_t)w.z + 128 / p.pk, (int64_t)w.y) - 1) / kBN) + 1;
  return true;
}

// Persistent, one CTA per SM; a unit is one query tile of 128 rows (packed_tc.cuh) against its key tiles of 128.
// TMEM: S in two buffers (columns 0 and 128), dP (256), dQ (384).  Per tile J the MMA warp issues S(J+1) into
// the other S buffer, dP(J+1) once the element-wise warps hold dP(J), and dQ += dS(J) K(J) once they have written
// dS(J) as bf16 over S(J).  A running tile count J carries rings and barrier phases across units; the next unit's
// Q/dO are loaded as soon as the last S and dP products of the current unit have read them.
// Warps: 0 K, 3 V, 2 Q/dO and the cleaning of the unit's last K tile, 1 products, 4..19 element-wise (thread =
// row, four warpgroups of 32 key columns).
template <bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const BwdParams p) {
  using L = Smem;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) { return sbase + L::kBar + 8u * (uint32_t)i; };
  const uint32_t qdo_full = BAR(0);
  auto kv_full = [&](int s) { return BAR(1 + s); };          // K(J) and V(J) of tile J, slot J mod KS
  auto k_empty = [&](int s) { return BAR(1 + KS + s); };
  auto v_empty = [&](int s) { return BAR(1 + 2 * KS + s); };
  // S, dS of tile J live in S buffer J mod 2: barriers per buffer (phase J / 2), so that S(J+1), issued before
  // the element-wise warps are done with tile J, never runs a phase ahead
  auto s_full = [&](int b) { return BAR(1 + 2 * KS + VS + b); };
  const uint32_t dp_full = BAR(3 + 2 * KS + VS);
  const uint32_t dp_free = BAR(4 + 2 * KS + VS);
  auto ds_full = [&](int b) { return BAR(5 + 2 * KS + VS + b); };
  const uint32_t dq_ready = BAR(7 + 2 * KS + VS);
  const uint32_t mma_done = BAR(8 + 2 * KS + VS);
  const uint32_t qdo_empty = BAR(9 + 2 * KS + VS);           // the unit's Q/dO fully read
  const uint32_t delta_bar = BAR(10 + 2 * KS + VS);          // delta partial sums in TMEM
  const uint32_t qdo_issued = BAR(11 + 2 * KS + VS);         // a unit's Q/dO loads are issued
  auto k_clean = [&](int s) { return BAR(12 + 2 * KS + VS + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(qdo_full, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(kv_full(s), 2);             // the K and the V producer
      mbar_init(k_empty(s), 2);             // the products' commit, and the cleaning warp, which waits for every tile
      mbar_init(k_clean(s), 1);
    }
    for (int s = 0; s < VS; ++s) mbar_init(v_empty(s), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(ds_full(b), kEW);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_free, kEW);
    mbar_init(dq_ready, 1);
    mbar_init(mma_done, 1);
    mbar_init(qdo_empty, 1 + kEW);          // the MMA warp's commit and every element-wise warp
    mbar_init(delta_bar, kEW);
    mbar_init(qdo_issued, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  const int per_tile = p.Hkv * (p.G / p.pk);
  Own& own = *reinterpret_cast<Own*>(smem + L::kOwn);
  if (kOwn && warp == 2) {
    pdl_wait();
    own_tile(p.work, blockIdx.x / per_tile, &own);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();                               // the work list comes from the kernel before
  const int64_t n_units = units_of<kOwn>(p.work, own, per_tile);
  Unit x;

  if (warp == 0 || warp == 3) {
    // ======================= TMA producers of K(J) (warp 0) and V(J) (warp 3); both arrive on kv_full of the
    // tile.  A unit's first tiles are issued only after its Q/dO loads, which are needed first.
    if (lane == 0) {
      const bool is_v = warp == 3;
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      int64_t J = 0;
      bool ok = true;
      for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
        if (!(ok = mbar_wait(qdo_issued, k & 1, abort_flag, p.status, p.wait_ns))) break;
        for (int j = 0; j < x.T; ++j, ++J) {
          const int ks = (int)(J % KS), vs = (int)(J % VS);
          ok = is_v ? mbar_wait(v_empty(vs), (uint32_t)((J / VS) & 1) ^ 1, abort_flag, p.status, p.wait_ns)
                    : mbar_wait(k_empty(ks), (uint32_t)((J / KS) & 1) ^ 1, abort_flag, p.status, p.wait_ns);
          if (!ok) break;
          mbar_arrive_expect_tx(kv_full(ks), kTileBytes);
          const uint32_t dst = is_v ? sbase + L::kV + vs * kTileBytes : sbase + L::kK + ks * kTileBytes;
          tma_load_3d(dst, map, 0, x.kh, x.start + j * kBN, kv_full(ks));
          tma_load_3d(dst + kHalfBytes, map, 64, x.kh, x.start + j * kBN, kv_full(ks));
        }
      }
      // every load this warp issued has landed (its tile's barrier completed) before the CTA exits
      for (int64_t j = J > KS ? J - KS : 0; j < J; ++j)
        drain_wait(kv_full((int)(j % KS)), (uint32_t)((j / KS) & 1), p.status);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ======================= each unit's Q and dO (once the previous unit's last S, dP products and delta reads
    // are done with them), then the rows past the sequence in the unit's last K tile
    int loads = 0;
    int64_t J = 0;
    bool ok = true;
    for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
      if (k > 0) ok = wait_w(qdo_empty, (k - 1) & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(qdo_full, 2 * kTileBytes);
        for (int h = 0; h < 2; ++h) {
          tma_load_3d(sbase + L::kQ + h * kHalfBytes, &tm_q, 64 * h, x.h0, x.start + x.t0, qdo_full);
          tma_load_3d(sbase + L::kDO + h * kHalfBytes, &tm_do, 64 * h, x.h0, x.start + x.t0, qdo_full);
        }
        mbar_arrive(qdo_issued);
      }
      __syncwarp();
      ++loads;
      for (int j = 0; j < x.T; ++j, ++J) {                   // (every tile is waited for, and its stage is free only
        const int s = (int)(J % KS);                         // behind this warp: a parity names the current phase and
        ok = wait_w(kv_full(s), (uint32_t)((J / KS) & 1), abort_flag, p.status, p.wait_ns);      // the one before)
        if (!ok) break;
        if (x.len - j * kBN < kBN) {
          zero_rows(sbase + L::kK + s * kTileBytes, kBN, kHalfBytes, x.len - j * kBN);
          __syncwarp();
          if (lane == 0) mbar_arrive(k_clean(s));
        }
        if (lane == 0) mbar_arrive(k_empty(s));
      }
    }
    if (lane == 0 && loads) drain_wait(qdo_full, (loads - 1) & 1, p.status);
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issuer: the whole warp runs the loop, one elected lane issues
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kBN, false);
    constexpr uint32_t idesc_dq = idesc_bf16_f32(128, kD, true);
    uint64_t qa[8], da[8];
    kmajor_descs(qa, sbase + L::kQ, kHalfBytes, 1024);
    kmajor_descs(da, sbase + L::kDO, kHalfBytes, 1024);
    const uint64_t k0 = smem_desc_sw128(sbase + L::kK, 16, 1024), v0 = smem_desc_sw128(sbase + L::kV, 16, 1024);
    const uint64_t kmn0 = smem_desc_sw128(sbase + L::kK, kHalfBytes, 1024);
    auto issue_s = [&](int64_t J) {         // S(J) = Q K(J)^T
      tc_fence_after();
      uint64_t bb[8];
      kmajor_from_base(bb, k0 + (uint64_t)((int)(J % KS) * (kTileBytes >> 4)), kHalfBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ss_w(tmem + (uint32_t)(J & 1) * 128, qa[ks], bb[ks], idesc_s, ks > 0);
      mma_commit_w(s_full((int)(J & 1)));
    };
    auto issue_dp = [&](int64_t J) {        // dP(J) = dO V(J)^T
      tc_fence_after();
      uint64_t bb[8];
      kmajor_from_base(bb, v0 + (uint64_t)((int)(J % VS) * (kTileBytes >> 4)), kHalfBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ss_w(tmem + 256, da[ks], bb[ks], idesc_s, ks > 0);
      mma_commit_w(dp_full);
      mma_commit_w(v_empty((int)(J % VS)));
    };
    // dQ (+)= dS(J) K(J); dS of keys 32w..32w+31 sits in columns 32w..32w+15 of S buffer J mod 2, the low parts of a unit's
    // last tile in 32w+16..32w+31
    auto issue_dq = [&](int64_t J, bool first, bool last) {
      uint64_t bb[8];
      mnmajor_from_base<8>(bb, kmn0 + (uint64_t)((int)(J % KS) * (kTileBytes >> 4)), (2 * 1024u) >> 4);
      const uint32_t sb = tmem + (uint32_t)(J & 1) * 128;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_ts_w(tmem + 384, sb + (ks >> 1) * 32 + (ks & 1) * 8, bb[ks], idesc_dq, !(first && ks == 0));
      if (!last) return;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ts_w(tmem + 384, sb + 16 + (ks >> 1) * 32 + (ks & 1) * 8, bb[ks], idesc_dq, true);
    };
    bool ok = true;
    int64_t J = 0;
    uint32_t clean_phase = 0;               // bit s: parity of the next cleaned tile in K stage s
    bool have = load_unit<kOwn>(p, own, n_units, 0, &x);
    if (have) {
      ok = wait_w(qdo_full, 0, abort_flag, p.status, p.wait_ns) &&
           wait_w(kv_full(0), 0, abort_flag, p.status, p.wait_ns);
      if (ok) {
        issue_s(0);
        issue_dp(0);
        if (x.T == 1) mma_commit_w(qdo_empty);
      }
    }
    for (int k = 0; ok && have; ++k) {
      Unit xn = x;
      const bool has_next = load_unit<kOwn>(p, own, n_units, k + 1, &xn);
      for (int j = 0; j < x.T; ++j, ++J) {
        const bool last = j + 1 == x.T;
        const bool next = !last || has_next;
        const int jn = last ? 0 : j + 1;    // the next tile's index in its unit
        const int Tn = last ? xn.T : x.T;
        auto finish_tile = [&]() {          // dQ (+)= dS(J) K(J), then K(J) is free
          const int s = (int)(J % KS);
          ok = wait_w(ds_full((int)(J & 1)), (uint32_t)((J >> 1) & 1), abort_flag, p.status, p.wait_ns);
          if (ok && x.len - j * kBN < kBN) {
            ok = wait_w(k_clean(s), (clean_phase >> s) & 1u, abort_flag, p.status, p.wait_ns);
            clean_phase ^= 1u << s;
          }
          if (!ok) return;
          tc_fence_after();
          issue_dq(J, j == 0, last);
          mma_commit_w(k_empty(s));
        };
        // at a unit's last tile its dQ comes first, so that the epilogue does not wait for the next unit's loads
        if (last) {
          finish_tile();
          if (!ok) break;
          mma_commit_w(dq_ready);
        }
        if (next) {
          if (last) ok = wait_w(qdo_full, (k + 1) & 1, abort_flag, p.status, p.wait_ns);
          if (ok)
            ok = wait_w(kv_full((int)((J + 1) % KS)), (uint32_t)(((J + 1) / KS) & 1), abort_flag, p.status, p.wait_ns);
          if (!ok) break;
          issue_s(J + 1);
        }
        ok = wait_w(dp_free, (uint32_t)(J & 1), abort_flag, p.status, p.wait_ns);
        if (!ok) break;
        if (next) {
          issue_dp(J + 1);
          if (jn + 1 == Tn) mma_commit_w(qdo_empty);
        }
        if (!last) {
          finish_tile();
          if (!ok) break;
        }
      }
      if (!ok) break;
      have = has_next;
      x = xn;
    }
    mma_commit_w(mma_done);
    drain_wait(mma_done, 0, p.status);
  } else {
    // ======================= element-wise: dS = P o (dP - delta), P = exp2(S c2 - lse log2 e)
    if (p.fill_tail)
      fill_tail_rows(p.dq, p.Hq, end_of<kOwn>(p.work, own), p.total, (int64_t)blockIdx.x * 512 + (threadIdx.x - 128),
                     (int64_t)gridDim.x * 512);
    const int w = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int c0 = 32 * w;                  // this warpgroup's key columns
    const bool v8 = (reinterpret_cast<uintptr_t>(p.dq) & 31u) == 0;
    bool ok = true;
    int64_t J = 0;
    for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
      const int head = x.h0 + r % p.pk;
      const int t_pos = x.t0 + r / p.pk;
      const bool in = t_pos < x.len;
      const int64_t row = (int64_t)x.start + t_pos;
      const float nlse2 = in ? -p.lse[head * p.total + row] * kLog2eF : 0.f;
      // delta = sum_d dO o O of this row.  Warpgroup w takes columns 32w .. 32w+31: O from global memory (issued
      // before the wait for the Q/dO tile), dO from the swizzled tile (row r: 8-row atom r/8, 16-byte chunk c of a
      // 64-column half at position c ^ (r mod 8)).  The four partial sums meet in TMEM column 384 + 32w (the first
      // of this warpgroup's dQ, read out for the previous unit, not rewritten before this unit's first dS K
      // product) and every thread adds them in order.
      uint4 ov[4];
      const int64_t at = (row * p.Hq + head) * kD + c0;
#pragma unroll
      for (int c = 0; c < 4; ++c) ov[c] = in ? reinterpret_cast<const uint4*>(p.o + at)[c] : make_uint4(0, 0, 0, 0);
      ok = wait_w(qdo_full, k & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      float part;
      {
        float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int chunk = 4 * w + c;
          const uint32_t off = (uint32_t)(chunk >> 3) * kHalfBytes + (uint32_t)(r >> 3) * 1024u +
                               (uint32_t)(r & 7) * 128u + ((uint32_t)((chunk & 7) ^ (r & 7)) << 4);
          const uint4 dv4 = *reinterpret_cast<const uint4*>(smem + L::kDO + off);
          const uint32_t a[4] = {ov[c].x, ov[c].y, ov[c].z, ov[c].w}, d4[4] = {dv4.x, dv4.y, dv4.z, dv4.w};
          const uint4 lo = in && p.o_lo ? reinterpret_cast<const uint4*>(p.o_lo + at)[c] : make_uint4(0, 0, 0, 0);
          const uint32_t b[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc0 = fmaf(__uint_as_float(a[e] << 16) + __uint_as_float(b[e] << 16), __uint_as_float(d4[e] << 16), acc0);
            acc1 = fmaf(__uint_as_float(a[e] & 0xffff0000u) + __uint_as_float(b[e] & 0xffff0000u),
                        __uint_as_float(d4[e] & 0xffff0000u), acc1);
          }
        }
        part = acc0 + acc1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qdo_empty);                 // this warp is done with dO
      tmem_st1(tmem + lane_off + 384 + c0, __float_as_uint(part));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(delta_bar);
      ok = wait_w(delta_bar, k & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      float dl;
      {
        uint32_t pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                       : "=r"(pv[i])
                       : "r"(tmem + lane_off + 384 + 32 * i));
        tmem_wait_ld();
        dl = ((__uint_as_float(pv[0]) + __uint_as_float(pv[1])) + __uint_as_float(pv[2])) + __uint_as_float(pv[3]);
      }
      if (w == 0 && in) {
        p.stats[head * p.total + row] = nlse2;
        p.stats[(p.Hq + head) * p.total + row] = -dl;
      }
      const uint64_t c2 = pair(p.c2, p.c2), nl2 = pair(nlse2, nlse2), nd2 = pair(-dl, -dl);
      for (int j = 0; j < x.T; ++j, ++J) {
        // P of this warpgroup's 32 keys while dP is still in the tensor pipe; then dP, which frees its columns
        ok = wait_w(s_full((int)(J & 1)), (uint32_t)((J >> 1) & 1), abort_flag, p.status, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + (uint32_t)(J & 1) * 128 + c0;
        // of this warpgroup's keys, those that the row attends (none for a row outside the sequence, nor for a sequence's
        // first token: it attends one key, whose dS is 0, where dP - delta would be the rounding of two sums)
        const int nvalid = in && t_pos > 0 ? t_pos - j * kBN + 1 - c0 : 0;
        uint64_t pr[16];
        {
          uint32_t sv[32];
          tmem_ld32(tS, sv);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            unpair(fma2(pair(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nl2), p0, p1);
            pr[e >> 1] = pair(ex2(p0), ex2(p1));
          }
        }
        ok = wait_w(dp_full, (uint32_t)(J & 1), abort_flag, p.status, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t dv[32], pk[16];
        tmem_ld32(tmem + lane_off + 256 + c0, dv);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_free);
        if (j + 1 == x.T) {                 // the diagonal (no other tile has keys that a row does not attend)
          uint32_t lo[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float d0, d1;
            unpair(mul2(pr[e >> 1], add2(pair(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])), nd2)), d0, d1);
            d0 = e < nvalid ? d0 : 0.f;
            d1 = e + 1 < nvalid ? d1 : 0.f;
            pk[e >> 1] = pack_bf16(d0, d1);
            lo[e >> 1] = pack_bf16(d0 - __uint_as_float(pk[e >> 1] << 16), d1 - __uint_as_float(pk[e >> 1] & 0xffff0000u));
          }
          tmem_st16(tS + 16, lo);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float d0, d1;
            unpair(mul2(pr[e >> 1], add2(pair(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])), nd2)), d0, d1);
            pk[e >> 1] = pack_bf16(d0, d1);
          }
        }
        // packed bf16 dS stays inside this warpgroup's own (already read) column range
        tmem_st16(tS, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full((int)(J & 1)));
      }
      if (ok) ok = wait_w(dq_ready, k & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[32], pk[16];
      tmem_ld32(tmem + lane_off + 384 + c0, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; e += 2)
        pk[e >> 1] = pack_bf16(__uint_as_float(v[e]) * p.scale, __uint_as_float(v[e + 1]) * p.scale);
      if (in) store32(p.dq + (row * p.Hq + head) * kD + c0, pk, v8);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace dq

// ======================================================================================== dK, dV
namespace dkdv {

constexpr int BM = 128;                     // keys per CTA (the M dimension)
constexpr int BQ = 64;                      // query rows per step: pk heads x 64 / pk tokens
constexpr int NS = 4;                       // Q / dO / statistics stages
constexpr uint32_t kQTile = BQ * 256, kQHalf = BQ * 128;
constexpr uint32_t kStatBytes = 2 * BQ * 4; // -lse log2(e) [64], -delta [64]
constexpr int kThreads = 640;

struct Smem {
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + kTileBytes;
  static constexpr uint32_t kQ = kV + kTileBytes;
  static constexpr uint32_t kDO = kQ + NS * kQTile;
  static constexpr uint32_t kStat = kDO + NS * kQTile;
  static constexpr uint32_t kBar = kStat + NS * kStatBytes;
  // kv_full, q_full[NS], q_empty[NS], q_clean[NS], sd_full[2], pd_full[2], done, mma_done, stat_full[NS]
  static constexpr int kNumBars = 1 + 4 * NS + 4 + 2;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;
  static constexpr uint32_t kOwn = (kMisc + 16 + 15) & ~15u;
  static constexpr uint32_t kBytes = kOwn + sizeof(Own);
};
static_assert(Smem::kBytes + 1024 <= 227 * 1024, "shared memory");

// One CTA per (128-key tile, KV head): S^T = K Q^T and dP^T = V dO^T per step of 64 query rows (double-buffered in
// TMEM), P^T and dS^T as bf16 back into TMEM, dV += P^T dO and dK += dS^T Q.  All of the KV head's query heads
// accumulate into the same TMEM dK, dV.  Warps: 0 loads Q and dO, 2 their lse and delta, 3 zeroes the rows past the
// sequence in a head's last step, 1 products, 4..19 element-wise (thread = key row; warpgroups split the steps by
// parity and the 64 query columns in two).
// With cs = 2 a cluster of two CTAs takes the steps of a unit in turn; each then has half of the key rows to store, and
// adds what the other, through its shared memory, has summed for them (two terms: the order does not matter).
template <bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const BwdParams p, const int cs) {
  using L = Smem;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) { return sbase + L::kBar + 8u * (uint32_t)i; };
  const uint32_t kv_full = BAR(0);
  auto q_full = [&](int s) { return BAR(1 + s); };
  auto q_empty = [&](int s) { return BAR(1 + NS + s); };
  auto q_clean = [&](int s) { return BAR(1 + 2 * NS + s); };
  auto sd_full = [&](int b) { return BAR(1 + 3 * NS + b); };
  auto pd_full = [&](int b) { return BAR(3 + 3 * NS + b); };
  const uint32_t done = BAR(5 + 3 * NS), mma_done = BAR(6 + 3 * NS);
  auto stat_full = [&](int s) { return BAR(7 + 3 * NS + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();                               // the work list, lse and delta come from the kernels before
  const int rank = (int)(blockIdx.x % cs), unit = (int)(blockIdx.x / cs);
  Own& own = *reinterpret_cast<Own*>(smem + L::kOwn);
  if (kOwn) {
    if (warp == 2) own_tile(p.work, unit / p.Hkv, &own);
    __syncthreads();
  }
  if (p.fill_tail) {
    const int64_t worker = (int64_t)blockIdx.x * kThreads + threadIdx.x, workers = (int64_t)gridDim.x * kThreads;
    const int64_t end = end_of<kOwn>(p.work, own);
    fill_tail_rows(p.dk, p.Hkv, end, p.total, worker, workers);
    fill_tail_rows(p.dv, p.Hkv, end, p.total, worker, workers);
  }
  if (unit >= units_of<kOwn>(p.work, own, p.Hkv)) return;     // (the whole cluster)
  const int4 wk = tile_of<kOwn>(p.work, own, unit / p.Hkv);
  const int start = wk.x, len = wk.y, t0 = wk.z;
  const int kh = unit % p.Hkv;
  const int tq = BQ / p.pk;                 // tokens per step
  const int per = p.G / p.pk;               // passes over the queries, pk heads each
  const int Tq = (len - t0 + tq - 1) / tq;  // steps per pass
  const int NA = per * Tq;                  // steps of the unit; this CTA's are rank, rank + cs, ...
  const int NJ = (NA - rank + cs - 1) / cs;
  // this CTA's step j: pass and step within the pass
  auto pass_of = [&](int j) { return (j * cs + rank) / Tq; };
  auto step_of = [&](int j) { return (j * cs + rank) % Tq; };
  const bool ragged = (len - t0) % tq != 0; // a pass's last step holds rows past the sequence
  const int diag_steps = (BM + tq - 1) / tq;                // a pass's steps that overlap the key tile

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(stat_full(s), 32);          // the 32 lanes' copies of lse and delta
      mbar_init(q_empty(s), ragged ? 2 : 1);      // the products' commit, and warp 3 where it waits for every step
      mbar_init(q_clean(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sd_full(b), 1);
      mbar_init(pd_full(b), 8);
    }
    mbar_init(done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) pdl_trigger();      // (behind the allocation: no kernel behind this one can hold TMEM that it waits for)
  bool ew_ok = false;                       // an element-wise warp whose accumulators are complete

  if (warp == 0) {
    // ======================= TMA producer
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * kTileBytes);
      for (int h = 0; h < 2; ++h) {
        tma_load_3d(sbase + L::kK + h * kHalfBytes, &tm_k, 64 * h, kh, start + t0, kv_full);
        tma_load_3d(sbase + L::kV + h * kHalfBytes, &tm_v, 64 * h, kh, start + t0, kv_full);
      }
      int issued = 0;
      for (int j = 0; j < NJ; ++j) {
        const int s = j % NS, g = pass_of(j), i = step_of(j);
        if (!mbar_wait(q_empty(s), ((j / NS) & 1) ^ 1, abort_flag, p.status, p.wait_ns)) break;
        mbar_arrive_expect_tx(q_full(s), 2 * kQTile);
        const int h0 = kh * p.G + g * p.pk, tok = start + t0 + i * tq;
        for (int h = 0; h < 2; ++h) {
          tma_load_3d(sbase + L::kQ + s * kQTile + h * kQHalf, &tm_q, 64 * h, h0, tok, q_full(s));
          tma_load_3d(sbase + L::kDO + s * kQTile + h * kQHalf, &tm_do, 64 * h, h0, tok, q_full(s));
        }
        ++issued;
      }
      drain_wait(kv_full, 0, p.status);
      for (int j = issued > NS ? issued - NS : 0; j < issued; ++j) drain_wait(q_full(j % NS), (j / NS) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ======================= lse and delta of each step's rows: 4-byte asynchronous copies (a row's place depends on
    // its head and token), zeros past the sequence
    bool ok = true;
    for (int j = 0; j < NJ; ++j) {
      const int s = j % NS, g = pass_of(j), i = step_of(j);
      ok = ok && wait_w(q_empty(s), ((j / NS) & 1) ^ 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = lane + 32 * y;
        const int t = t0 + i * tq + r / p.pk;
        const int64_t at = (int64_t)(kh * p.G + g * p.pk + r % p.pk) * p.total + start + (t < len ? t : t0);
        const uint32_t dst = sbase + L::kStat + s * kStatBytes + r * 4, n = t < len ? 4u : 0u;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(p.stats + at), "r"(n) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + BQ * 4), "l"(p.stats + p.Hq * p.total + at),
                     "r"(n) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(stat_full(s)) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 3) {
    // ======================= zeroes the rows past the sequence in each pass's last step
    bool ok = ragged;
    for (int j = 0; ok && j < NJ; ++j) {
      const int s = j % NS;
      ok = wait_w(q_full(s), (j / NS) & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      if (step_of(j) == Tq - 1) {
        const int rows = (len - t0 - (Tq - 1) * tq) * p.pk;
        zero_rows(sbase + L::kQ + s * kQTile, BQ, kQHalf, rows);
        zero_rows(sbase + L::kDO + s * kQTile, BQ, kQHalf, rows);
        __syncwarp();
        if (lane == 0) mbar_arrive(q_clean(s));
      }
      if (lane == 0) mbar_arrive(q_empty(s));            // (a parity names only the current phase and the one before)
    }
  } else if (warp == 1) {
    // ======================= MMA issuer: the whole warp runs the loop, one elected lane issues
    constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BQ, false);
    constexpr uint32_t idesc_g = idesc_bf16_f32(BM, kD, true);
    uint64_t kd[8], vd[8];
    kmajor_descs(kd, sbase + L::kK, kHalfBytes, 1024);
    kmajor_descs(vd, sbase + L::kV, kHalfBytes, 1024);
    const uint64_t q0 = smem_desc_sw128(sbase + L::kQ, 16, 1024), do0 = smem_desc_sw128(sbase + L::kDO, 16, 1024);
    const uint64_t qmn0 = smem_desc_sw128(sbase + L::kQ, kQHalf, 1024);
    const uint64_t domn0 = smem_desc_sw128(sbase + L::kDO, kQHalf, 1024);
    auto issue_sd = [&](int j, int b) {
      const uint64_t soff = (uint64_t)((j % NS) * (kQTile >> 4));
      uint64_t bb[8];
      kmajor_from_base(bb, q0 + soff, kQHalf >> 4);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ss_w(tmem + b * 128, kd[ks], bb[ks], idesc_s, ks > 0);
      kmajor_from_base(bb, do0 + soff, kQHalf >> 4);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma_ss_w(tmem + b * 128 + 64, vd[ks], bb[ks], idesc_s, ks > 0);
      mma_commit_w(sd_full(b));
    };
    // dV += P^T dO, dK += dS^T Q; P^T / dS^T of queries 32h..32h+31 sit in columns 32h..32h+15 of their region
    auto issue_grad = [&](int j, int b) {
      const uint64_t soff = (uint64_t)((j % NS) * (kQTile >> 4));
      uint64_t b1[4], b2[4];
      mnmajor_from_base<4>(b1, domn0 + soff, 2048u >> 4);
      mnmajor_from_base<4>(b2, qmn0 + soff, 2048u >> 4);
#pragma unroll
      for (int ks = 0; ks < BQ / 16; ++ks) {
        const uint32_t acol = (ks >> 1) * 32 + (ks & 1) * 8;
        mma_ts_w(tmem + 256, tmem + b * 128 + acol, b1[ks], idesc_g, (j > 0 || ks > 0));
        mma_ts_w(tmem + 384, tmem + b * 128 + 64 + acol, b2[ks], idesc_g, (j > 0 || ks > 0));
      }
    };
    // dK += (what rounding took from dS)^T Q, in columns 32h+16..32h+31 of the dS^T region
    auto issue_low = [&](int j, int b) {
      uint64_t b2[4];
      mnmajor_from_base<4>(b2, qmn0 + (uint64_t)((j % NS) * (kQTile >> 4)), 2048u >> 4);
#pragma unroll
      for (int ks = 0; ks < BQ / 16; ++ks)
        mma_ts_w(tmem + 384, tmem + b * 128 + 80 + (ks >> 1) * 32 + (ks & 1) * 8, b2[ks], idesc_g, true);
    };
    uint32_t clean_phase = 0;               // bit s: parity of the next cleaned step in stage s
    auto step_ready = [&](int j) {
      const int s = j % NS;
      bool ok = wait_w(q_full(s), (j / NS) & 1, abort_flag, p.status, p.wait_ns);
      if (ok && ragged && step_of(j) == Tq - 1) {
        ok = wait_w(q_clean(s), (clean_phase >> s) & 1u, abort_flag, p.status, p.wait_ns);
        clean_phase ^= 1u << s;
      }
      tc_fence_after();
      return ok;
    };
    bool ok = wait_w(kv_full, 0, abort_flag, p.status, p.wait_ns);
    for (int j = 0; ok && j < 2 && j < NJ; ++j) {
      ok = step_ready(j);
      if (ok) issue_sd(j, j & 1);
    }
    auto step = [&](int j, bool low) {
      const int b = j & 1;
      ok = wait_w(pd_full(b), (j >> 1) & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) return;
      tc_fence_after();
      issue_grad(j, b);
      if (low) issue_low(j, b);
      mma_commit_w(q_empty(j % NS));
      if (j + 2 < NJ) {
        ok = step_ready(j + 2);
        if (ok) issue_sd(j + 2, b);
      }
    };
    // each pass begins with its steps on the diagonal (loops of their own: a condition in one loop cost 5 %)
    for (int j = 0; ok && j < NJ;) {
      const int i = step_of(j);
      const int d1 = min(NJ, j + (max(min(diag_steps, Tq) - i, 0) + cs - 1) / cs);
      for (; ok && j < d1; ++j) step(j, true);
      const int i2 = step_of(j);
      const int e1 = i2 < diag_steps ? j : min(NJ, j + (Tq - i2 + cs - 1) / cs);
      for (; ok && j < e1; ++j) step(j, false);
    }
    if (ok) mma_commit_w(done);
    mma_commit_w(mma_done);
    drain_wait(mma_done, 0, p.status);
  } else if (warp >= 4) {
    // ======================= element-wise: P^T, dS^T.  Warpgroup w4 takes the steps j = w4 mod 2 and the 32 query
    // columns 32 (w4 / 2) .. of each (thread = TMEM lane = key row).
    const int w4 = (warp - 4) >> 2;
    const int b = w4 & 1, hc = w4 >> 1;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;      // key row within the tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + b * 128;
    const uint32_t tP = tS + 64;
    const float* stat_base = reinterpret_cast<const float*>(smem + L::kStat);
    const uint64_t c2 = pair(p.c2, p.c2);
    bool ok = true;
    int i = step_of(b);
    for (int j = b; j < NJ; j += 2) {
      const int s = j % NS;
      ok = wait_w(stat_full(s), (j / NS) & 1, abort_flag, p.status, p.wait_ns) &&
           wait_w(sd_full(b), (j >> 1) & 1, abort_flag, p.status, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const float* nlse = stat_base + s * (kStatBytes / 4) + 32 * hc;
      const float* ndelta = nlse + BQ;
      // one TMEM round trip per step: both loads in flight, one wait, compute, both stores
      uint32_t sv[32], dv[32], pp[16], pd[16];
      tmem_ld32(tS + 32 * hc, sv);
      tmem_ld32(tP + 32 * hc, dv);
      tmem_wait_ld();
      // query column c of this step is token i tq + c / pk of the tile's own tokens: columns before `from` are not
      // attended by it
      const int from = i < diag_steps ? (r - i * tq) * p.pk - 32 * hc : 0;
      const int dfrom = t0 == 0 && i == 0 ? max(from, p.pk - 32 * hc) : from;      // (token 0: one key, dS = 0)
      auto pairs = [&](bool masked) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t nl = *reinterpret_cast<const uint64_t*>(nlse + e), nd = *reinterpret_cast<const uint64_t*>(ndelta + e);
          float p0, p1, d0, d1;
          unpair(fma2(pair(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nl), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          unpair(mul2(pair(p0, p1), add2(pair(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])), nd)), d0, d1);
          if (masked) {
            p0 = e >= from ? p0 : 0.f;
            d0 = e >= dfrom ? d0 : 0.f;
            p1 = e + 1 >= from ? p1 : 0.f;
            d1 = e + 1 >= dfrom ? d1 : 0.f;
          }
          pp[e >> 1] = pack_bf16(p0, p1);
          pd[e >> 1] = pack_bf16(d0, d1);
          if (masked)                       // (of the dP registers behind e, none is needed any more)
            dv[e >> 1] = pack_bf16(d0 - __uint_as_float(pd[e >> 1] << 16), d1 - __uint_as_float(pd[e >> 1] & 0xffff0000u));
        }
      };
      if (i < diag_steps) {
        pairs(true);
        tmem_st16(tP + 32 * hc + 16, reinterpret_cast<const uint32_t(&)[16]>(dv));
      } else {
        pairs(false);
      }
      // packed bf16 stays inside this warpgroup's own (already read) column range
      tmem_st16(tS + 32 * hc, pp);
      tmem_st16(tP + 32 * hc, pd);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pd_full(b));
      i += 2 * cs;
      while (i >= Tq) i -= Tq;
    }
    // (a CTA without steps, the second of a cluster that has one step, has nothing in its accumulators)
    if (ok) ok = wait_w(done, 0, abort_flag, p.status, p.wait_ns);
    ew_ok = ok;
  }
  // ---- epilogue: warpgroups 0, 1 own dV columns 0-63 / 64-127, warpgroups 2, 3 the same of dK
  const int w4 = (warp - 4) >> 2;
  const int er = (warp & 3) * 32 + lane;    // key row of an element-wise thread
  const uint32_t tacc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (w4 >= 2 ? 384 : 256) + 64 * (w4 & 1);
  const bool mine = cs == 1 || (er >> 6) == rank;        // (whole warps)
  auto piece = [&](int c) {                 // of the exchange: 16-byte piece c of a warpgroup's 64 columns
    return sbase + L::kQ + (uint32_t)(((w4 * 16 + c) * 64 + (er & 63)) * 16);
  };
  if (cs == 2) {
    if (warp >= 4 && !mine && ew_ok) {
      tc_fence_after();
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t v[32];
        tmem_ld32(tacc + 32 * y, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece(8 * y + c)), "r"(NJ ? v[4 * c] : 0u),
                       "r"(NJ ? v[4 * c + 1] : 0u), "r"(NJ ? v[4 * c + 2] : 0u), "r"(NJ ? v[4 * c + 3] : 0u)
                       : "memory");
      }
    }
    __syncwarp();
    cluster_sync();                         // (every thread of both CTAs, on the error path too)
  }
  if (warp >= 4 && mine && ew_ok) {
    tc_fence_after();
    const bool is_dk = w4 >= 2;
    const float mul = is_dk ? p.scale : 1.f;
    __nv_bfloat16* base = is_dk ? p.dk : p.dv;
    const bool v8 = (reinterpret_cast<uintptr_t>(base) & 31u) == 0;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t v[32], pk[16];
      tmem_ld32(tacc + 32 * y, v);
      tmem_wait_ld();
      if (cs == 2) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t at;
          float u[4];
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(piece(8 * y + c)), "r"(rank ^ 1));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3]) : "r"(at) : "memory");
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[4 * c + e] = __float_as_uint((NJ ? __uint_as_float(v[4 * c + e]) : 0.f) + u[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 32; e += 2)
        pk[e >> 1] = pack_bf16(__uint_as_float(v[e]) * mul, __uint_as_float(v[e + 1]) * mul);
      if (t0 + er < len)
        store32(base + (((int64_t)start + t0 + er) * p.Hkv + kh) * kD + 64 * (w4 & 1) + 32 * y, pk, v8);
    }
  }
  tc_fence_before();
  __syncwarp();
  if (cs == 2) cluster_sync();              // no CTA leaves while the other reads its sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace dkdv
}  // namespace

int dq_tile(int G) { return 128 / packed_heads(G); }

cudaError_t launch_bwd_tc(const void* q, const void* k, const void* v, const void* o, const void* o_lo,
                          const float* lse, const void* d_o, float* stats, void* dq, void* dk, void* dv,
                          const Work& by_query, const Work& by_key, const Problem& p, cudaStream_t st) {
  const int pk = packed_heads(p.G);
  size_t smem = dq::Smem::kBytes + 1024;
  auto dq_kernel = by_query.cu ? dq::packed_dq_tc_kernel<true> : dq::packed_dq_tc_kernel<false>;
  cudaError_t e = set_smem(dq_kernel, smem);
  if (e != cudaSuccess) return e;
  const Strided so{(int64_t)p.Hq * kD, kD};
  CUtensorMap mq, mdo, mk, mv, mq64, mdo64;
  if (!make_map_packed(&mq, q, p.Hq, p.total, p.q, pk, 128 / pk) ||
      !make_map_packed(&mdo, d_o, p.Hq, p.total, so, pk, 128 / pk) ||
      !make_map_packed(&mq64, q, p.Hq, p.total, p.q, pk, 64 / pk) ||
      !make_map_packed(&mdo64, d_o, p.Hq, p.total, so, pk, 64 / pk) ||
      !make_map_packed(&mk, k, p.Hkv, p.total, p.k, 1, kBN) || !make_map_packed(&mv, v, p.Hkv, p.total, p.v, 1, kBN))
    return cudaErrorInvalidValue;
  BwdParams a{p.Hq, p.Hkv, p.G, pk, p.total, p.scale * kLog2eF, p.scale, static_cast<const __nv_bfloat16*>(o),
              static_cast<const __nv_bfloat16*>(o_lo), lse, stats,
              static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv),
              by_query, p.fill_tail, p.status, p.wait_ns};
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t units = list_capacity(p.total, p.n_seqs, dq_tile(p.G)) * p.Hkv * (p.G / pk);
  e = launch_dependent(dq_kernel, dim3((unsigned)(units < 1 ? 1 : units < sms ? units : sms)),
                       dim3(dq::kThreads), smem, st, 1, mq, mdo, mk, mv, a);
  if (e != cudaSuccess) return e;
  a.work = by_key;
  smem = dkdv::Smem::kBytes + 1024;
  auto dkdv_kernel = by_key.cu ? dkdv::packed_dkdv_tc_kernel<true> : dkdv::packed_dkdv_tc_kernel<false>;
  e = set_smem(dkdv_kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = list_capacity(p.total, p.n_seqs, kKeyTile) * p.Hkv;
  // Two CTAs per unit while there are fewer units than SMs.  Whole backward pass, 32/8 heads: 1024 tokens (64 units) 103 us
  // with one, 73 with two; 2048 (128) 240 and 170; 4096 (256) 456 and 474; 8/8 heads, 4096 (256) 128 and 156.
  const int cs = tiles < sms ? 2 : 1;
  return launch_dependent(dkdv_kernel, dim3((unsigned)((tiles < 1 ? 1 : tiles) * cs)), dim3(dkdv::kThreads),
                          smem, st, (unsigned)cs, mq64, mdo64, mk, mv, a, cs);
}

}  // namespace packed
}  // namespace hga
