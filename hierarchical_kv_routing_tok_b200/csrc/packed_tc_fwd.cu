// Causal attention over packed sequences, forward, on the tensor cores (tcgen05, bf16).
//
//   o_t = sum_{u<=t} softmax_u(scale q_t.k_u) v_u,   lse_t = log sum_{u<=t} exp(scale q_t.k_u)
// with the online softmax: running maximum m and sum l per row, o rescaled when m grows by more than 2^8.
//
// Bound by the tensor pipe (two 128 x 128 x 128 products per tile) and, about as much, by the exponentials
// (16 per clock and SM): one sequence of 16K tokens, 32/8 heads, 1.81 ms over ten passes, 1210 TFLOP/s of
// the formula's products (in a long run, at the power limit, 2.11 ms and 1040); tensor pipe active for 55 % of the cycles.  A unit is two query tiles of 128 rows (packed_tc.cuh) that share their K/V tiles of
// 128 keys.  One CTA per SM walks the units of the work list, heaviest first; barriers and rings count tiles
// across units, so the next unit's loads and first products run under the epilogue of the current one.
// Warps: 16 loads (TMA; a ring of two items, V(j) with K(j+1), so that the issuing warp waits once for both), 17 issues the
// products, 0-7 and 8-15 are the softmax of the two tiles (thread = half a row), 18 checks the V tiles that masked rows meet: on
// the causal diagonal p = 0 meets values that the row does not attend, and 0 * inf is not 0.  Values there that are not
// finite become 0 before the product, and the epilogue adds them to the rows that do attend them.
// P is rounded to bf16, the type of V, for its product: o is 2.0e-3 of the norm from exact (16K: 2.2e-3), of which rounding
// o takes 1.6e-3.  (What the rounding took as a further operand on the diagonal, as in the backward: 1.8e-3 (1.9e-3), but 37
// tokens 11.7 -> 12.6 us, 2048 tokens 53 -> 57, the packed batch 668 -> 685, 16K 1843 -> 1855 with a loop of its own, and 1970
// at 16K without: the softmax warps have no registers to spare.)
// TMEM: S_0 S_1 O_0 O_1 (128 columns each); P_i as bf16 over the first half of S_i.  Issue order S_0 S_1 |
// PV_0 S_0' PV_1 S_1' | ...: S_i(j+1) complete implies PV_i(j) complete, so no barrier guards the rescale.
// (Measured slower: S in two buffers of 64 keys, 2406 against 1903 us at 16K, whose products of 64 columns wait for shared
// memory, 48 cycles in place of 32; a part of the exponentials by a polynomial on the FMA pipe, 2160 -> 2550 us.)
#include <cuda_bf16.h>

#include "packed_tc.cuh"

namespace hga {
namespace packed {

using namespace tc;

namespace {

constexpr float kRescaleThreshold = 8.f;   // log2 units
constexpr int NS = 2;                      // ring items
constexpr int kSoftmax = 512;              // threads of the 16 softmax warps
constexpr int kMmaWarp = 17;
constexpr int kThreads = kSoftmax + 96;

struct FwdParams {
  int Hq, Hkv, G, pk, pk_shift, tp;        // pk = 1 << pk_shift; tp: tokens per query tile, 128 / pk
  int hu;                                  // head units: Hkv * G / pk
  int64_t total;
  float scale_log2;
  const __nv_bfloat16* v;                  // for the values that are not finite
  Strided vs;
  __nv_bfloat16* o;
  __nv_bfloat16* o_lo;                     // what rounding took from o, or nullptr
  float* lse;
  Work work;
  int fill_tail;
  int* status;
  uint64_t wait_ns;
};

struct FwdSmem {
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kTileBytes;
  static constexpr uint32_t kV = kK + NS * kTileBytes;
  static constexpr uint32_t kO = kV + NS * kTileBytes;          // 2 KB per softmax warp: 32 rows x 32 dims of o
  static constexpr uint32_t kBar = kO + 16 * 2048;
  // q_full, q_empty, full[NS], empty[NS], v_clean[NS], s_full[2], p_full[2], o_full[2], mma_done, flag_free[2][4]
  static constexpr int kNumBars = 2 + 3 * NS + 6 + 1 + 8;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;        // TMEM address, abort, flags of 2 x 4 units
  static constexpr uint32_t kNeed = kMisc + 48;                 // [tile parity][pair of warps][half]
  static constexpr uint32_t kOwn = (kNeed + 2 * 8 * 2 * 4 + 15) & ~15u;
  static constexpr uint32_t kBytes = kOwn + sizeof(Own);
};
static_assert(FwdSmem::kBytes + 1024 <= 227 * 1024, "shared memory");

struct Unit {
  int start, len, t0, h0, kh;
  int T[2], Tmax;                          // key tiles of the two query tiles
};

template <bool kOwn>
__device__ __forceinline__ bool load_unit(const FwdParams& p, const Own& own, int64_t n_units, int k, Unit* x) {
  const int64_t u = unit_of_cta(k, blockIdx.x, gridDim.x);
  if (u >= n_units) return false;
  const int4 w = tile_of<kOwn>(p.work, own, u / p.hu);
  const int hu = (int)(u % p.hu), per = p.G / p.pk;
  x->start = w.x;
  x->len = w.y;
  x->t0 = w.z;
  x->kh = hu / per;
  x->h0 = x->kh * p.G + (hu % per) * p.pk;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t first = (int64_t)w.z + i * p.tp;
    x->T[i] = first < w.y ? (int)((min(first + p.tp, (int64_t)w.y) - 1) / kBN) + 1 : 0;
  }
  x->Tmax = max(x->T[0], x->T[1]);
  return true;
}

// A softmax warp's output: its 32 rows of 64 dims (two passes of 32) of the unnormalised O at tO.
struct OutArgs {
  int start, len, t0, kh, h0;
  int tok0, row0;              // first token of the query tile after t0; the warp's first row in it
  int dim0, t_pos;             // first dim; this lane's token
  uint32_t tO, stage;
  float inv;
  bool fix;
};
__device__ __noinline__ void write_output(const FwdParams& p, const OutArgs w) {
  const int lane = threadIdx.x & 31;
  const bool store = w.t_pos < w.len;
  // O / l as bf16, 32 dims at a time through this warp's 2 KB (16-byte pieces at position c ^ (row / 2 mod 4): no bank
  // conflicts), so that the stores to global memory are whole 64-byte runs
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    const int d0 = w.dim0 + 32 * cc;
    uint32_t v[32];
    tmem_ld32(w.tO + cc * 32, v);
    tmem_wait_ld();
    if (w.fix && store) {
      // values of the diagonal tiles that were set to 0 for the product: each adds itself
      for (int u = w.t0 / kBN * kBN; u <= w.t_pos; ++u) {
        const __nv_bfloat16* vr = p.v + ((int64_t)w.start + u) * p.vs.t + w.kh * p.vs.h + d0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float y = __bfloat162float(vr[e]);
          if (!isfinite(y)) v[e] = __float_as_uint(__uint_as_float(v[e]) + y);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * w.inv);
    // o, then what its rounding took
#pragma unroll 1
    for (int part = 0; part < (p.o_lo ? 2 : 1); ++part) {
      __nv_bfloat16* out = part ? p.o_lo : p.o;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int z = 8 * y + 2 * e;
          w4[e] = pack_bf16(__uint_as_float(v[z]), __uint_as_float(v[z + 1]));
          v[z] = __float_as_uint(__uint_as_float(v[z]) - __uint_as_float(w4[e] << 16));
          v[z + 1] = __float_as_uint(__uint_as_float(v[z + 1]) - __uint_as_float(w4[e] & 0xffff0000u));
        }
        const uint32_t a = w.stage + lane * 64u + (uint32_t)((y ^ ((lane >> 1) & 3)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w4[0]), "r"(w4[1]), "r"(w4[2]), "r"(w4[3]) : "memory");
      }
      __syncwarp();
      const int c = lane & 3;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int rr = 8 * y + (lane >> 2), rt = w.row0 + rr;      // row of the warp, of the tile
        const int t = w.t0 + w.tok0 + (rt >> p.pk_shift);
        uint32_t w4[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w4[0]), "=r"(w4[1]), "=r"(w4[2]), "=r"(w4[3])
                     : "r"(w.stage + rr * 64u + (uint32_t)((c ^ ((rr >> 1) & 3)) << 4)));
        if (t < w.len)
          *reinterpret_cast<uint4*>(out + (((int64_t)w.start + t) * p.Hq + w.h0 + (rt & (p.pk - 1))) * kD + d0 + 8 * c) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
      __syncwarp();
    }
  }
}

template <bool kOwn>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
  using L = FwdSmem;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) { return sbase + L::kBar + 8u * (uint32_t)i; };
  const uint32_t q_full = BAR(0), q_empty = BAR(1);
  auto full = [&](int s) { return BAR(2 + s); };
  auto empty = [&](int s) { return BAR(2 + NS + s); };
  auto v_clean = [&](int s) { return BAR(2 + 2 * NS + s); };
  auto s_full = [&](int i) { return BAR(2 + 3 * NS + i); };
  auto p_full = [&](int i) { return BAR(4 + 3 * NS + i); };
  auto o_full = [&](int i) { return BAR(6 + 3 * NS + i); };
  const uint32_t mma_done = BAR(8 + 3 * NS);
  auto flag_free = [&](int i, int n) { return BAR(9 + 3 * NS + 4 * i + (n & 3)); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  // whether the diagonal tiles hold values that are not finite: of query tile i's n-th output (units without that tile do
  // not count) in slot 4 i + n mod 4, free when the tile's eight softmax warps have read what output n - 4 left there
  volatile int* not_finite = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 2);               // the products' commit, and the checking warp, which waits for every item
      mbar_init(v_clean(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 8);
      mbar_init(o_full(i), 1);
    }
    mbar_init(mma_done, 1);
    for (int n = 0; n < 8; ++n) mbar_init(flag_free(n >> 2, n), 8);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  Own& own = *reinterpret_cast<Own*>(smem + L::kOwn);
  if (kOwn && warp == 16) {
    pdl_wait();
    own_tile(p.work, blockIdx.x / p.hu, &own);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();                              // the work list comes from the kernel before
  const int64_t n_units = units_of<kOwn>(p.work, own, p.hu);
  Unit x;

  if (warp == 16) {
    // ======================= TMA producer: per unit Q, then the items K(0) | V(0) K(1) | ... | V(T-1)
    if (lane == 0) {
      int64_t J = 0;
      bool ok = true;
      int loads = 0;
      for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
        if (k > 0 && !(ok = mbar_wait(q_empty, (k - 1) & 1, abort_flag, p.status, p.wait_ns))) break;
        mbar_arrive_expect_tx(q_full, 2 * kTileBytes);
        for (int i = 0; i < 2; ++i)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sbase + L::kQ + i * kTileBytes + h * kHalfBytes, &tm_q, 64 * h, x.h0, x.start + x.t0 + i * p.tp,
                        q_full);
        ++loads;
        for (int j = -1; j < x.Tmax; ++j, ++J) {
          const int s = (int)(J % NS);
          if (!(ok = mbar_wait(empty(s), (uint32_t)((J / NS) & 1) ^ 1, abort_flag, p.status, p.wait_ns))) break;
          const bool has_v = j >= 0, has_k = j + 1 < x.Tmax;
          mbar_arrive_expect_tx(full(s), has_v && has_k ? 2 * kTileBytes : kTileBytes);
          if (has_v)
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sbase + L::kV + s * kTileBytes + h * kHalfBytes, &tm_v, 64 * h, x.kh, x.start + j * kBN, full(s));
          if (has_k)
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sbase + L::kK + s * kTileBytes + h * kHalfBytes, &tm_k, 64 * h, x.kh, x.start + (j + 1) * kBN, full(s));
        }
      }
      // every load of this warp has landed before the CTA may exit
      for (int64_t j = J > NS ? J - NS : 0; j < J; ++j)
        drain_wait(full((int)(j % NS)), (uint32_t)((j / NS) & 1), p.status);
      if (loads) drain_wait(q_full, (loads - 1) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == 18) {
    // ======================= check of the V tiles at or behind the unit's first token
    int64_t J = 0;
    int n1 = 0;                                         // second query tiles so far (every unit has a first)
    bool ok = true;
    for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
      const int jd = x.t0 / kBN;
      bool any = false;
      const bool two = x.T[1] > 0;
      ok = mbar_wait_w(flag_free(0, k), (uint32_t)((k >> 2) & 1) ^ 1, abort_flag, p.status, p.wait_ns) &&
           (!two || mbar_wait_w(flag_free(1, n1), (uint32_t)((n1 >> 2) & 1) ^ 1, abort_flag, p.status, p.wait_ns));
      if (!ok) break;
      for (int j = -1; j < x.Tmax; ++j, ++J) {          // (every item is waited for, and its slot is free only behind
        const int s = (int)(J % NS);                    // this warp: a parity names the current phase and the one before)
        ok = mbar_wait_w(full(s), (uint32_t)((J / NS) & 1), abort_flag, p.status, p.wait_ns);
        if (!ok) break;
        if (j >= jd) {
          const uint32_t tile = sbase + L::kV + s * kTileBytes;
          if (x.len - j * kBN < kBN) {
            zero_rows(tile, kBN, kHalfBytes, x.len - j * kBN);
            __syncwarp();
          }
          any |= zero_not_finite(tile, kBN * 16);
          if (lane == 0) {                              // (the first query tile may end before the second)
            not_finite[k & 3] = any;
            if (two) not_finite[4 + (n1 & 3)] = any;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(v_clean(s));
        }
        if (lane == 0) mbar_arrive(empty(s));
      }
      n1 += two;
    }
  } else if (warp == kMmaWarp) {
    // ======================= MMA issuer: the whole warp runs the loop, one elected lane issues.  Per tile it waits for the
    // item, P_0 and P_1, and commits S_0, S_1 and the item: each wait costs the tensor pipe about 100 cycles.
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kBN, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, kD, true);
    uint64_t qd[2][8], kd[8], vd[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) kmajor_descs(qd[i], sbase + L::kQ + i * kTileBytes, kHalfBytes, 1024);
    const uint64_t k0 = smem_desc_sw128(sbase + L::kK, 16, 1024), v0 = smem_desc_sw128(sbase + L::kV, kHalfBytes, 1024);
    int64_t J = 0;
    int np[2] = {0, 0};                    // P tiles taken of each query tile
    uint32_t clean_phase = 0;              // bit s: parity of the next checked item in slot s
    bool ok = true;
    for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
      ok = wait_w(q_full, k & 1, abort_flag, p.status, p.wait_ns);
      const int jd = x.t0 / kBN;
      for (int j = -1; ok && j < x.Tmax; ++j, ++J) {
        const int s = (int)(J % NS);
        if (j >= jd) {
          ok = wait_w(v_clean(s), (clean_phase >> s) & 1u, abort_flag, p.status, p.wait_ns);
          clean_phase ^= 1u << s;
        } else {
          ok = wait_w(full(s), (uint32_t)((J / NS) & 1), abort_flag, p.status, p.wait_ns);
        }
        if (!ok) break;
        tc_fence_after();
        const uint64_t soff = (uint64_t)(s * (kTileBytes >> 4));
        kmajor_from_base(kd, k0 + soff, kHalfBytes >> 4);
        mnmajor_from_base<8>(vd, v0 + soff, (2 * 1024u) >> 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j >= x.T[i]) continue;
          if (j >= 0) {
            ok = wait_w(p_full(i), np[i] & 1, abort_flag, p.status, p.wait_ns);
            if (!ok) break;
            ++np[i];
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ts_w(tmem + 256 + i * 128, tmem + i * 128 + (ks >> 2) * 64 + (ks & 3) * 8, vd[ks], idesc_pv, (j > 0 || ks > 0));
          }
          if (j + 1 < x.T[i]) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) mma_ss_w(tmem + i * 128, qd[i][ks], kd[ks], idesc_qk, ks > 0);
            mma_commit_w(s_full(i));
          } else if (j >= 0) {
            mma_commit_w(o_full(i));       // the last product of this query tile
          }
        }
        if (!ok) break;
        mma_commit_w(empty(s));
        if (j + 2 == x.Tmax) mma_commit_w(q_empty);          // the unit's last S products are issued
      }
    }
    mma_commit_w(mma_done);
    drain_wait(mma_done, 0, p.status);
  } else {
    // ======================= softmax and epilogue: two warpgroups per query tile, 64 keys of each tile (and 64 dims of the
    // output) each.  The two warps of a row (a pair) keep the same maximum m; each has the sum of its keys.
    const int st = threadIdx.x;
    if (p.fill_tail) {
      const int64_t worker = (int64_t)blockIdx.x * kSoftmax + st, workers = (int64_t)gridDim.x * kSoftmax;
      const int64_t end = end_of<kOwn>(p.work, own);
      fill_tail_rows(p.o, p.Hq, end, p.total, worker, workers);
      if (p.o_lo) fill_tail_rows(p.o_lo, p.Hq, end, p.total, worker, workers);
      fill_tail_lse(p.lse, p.Hq, end, p.total, worker, workers);
    }
    const int i = st >> 8, half = (st >> 7) & 1;
    const int quarter = warp & 3, pair_id = 4 * i + quarter;
    const int r = quarter * 32 + lane;                  // row of the query tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + i * 128 + 64 * half;
    const uint32_t tO = tmem + lane_off + 256 + i * 128 + 64 * half;
    const uint32_t s_need = sbase + L::kNeed + 8 * pair_id;             // + 64 * parity + 4 * half
    // a row's maximum or sum for the other warp: in the writer's part of the output staging
    const uint32_t s_row = sbase + L::kO + (8 * i + quarter) * 2048 + 4 * lane;      // + 8192 * half
    auto put = [](uint32_t a, uint32_t y) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(y) : "memory"); };
    auto get = [](uint32_t a) {
      uint32_t y;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(a) : "memory");
      return y;
    };
    auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + pair_id) : "memory"); };
    int ns = 0, no = 0;                                 // S tiles, outputs taken
    bool ok = true;
    for (int k = 0; ok && load_unit<kOwn>(p, own, n_units, k, &x); ++k) {
      const int T = x.T[i];
      if (T == 0) continue;
      const int t_pos = x.t0 + i * p.tp + (r >> p.pk_shift);    // (rows past the sequence compute, and store nothing)
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < T; ++j, ++ns) {
        ok = wait_w(s_full(i), ns & 1, abort_flag, p.status, p.wait_ns);
        tc_fence_after();
        const int nvalid = t_pos - j * kBN + 1 - 64 * half;     // of this warp's keys, those that the row attends
        uint32_t v[32], v2[32];
        tmem_ld32(tS, v);
        tmem_ld32(tS + 32, v2);
        tmem_wait_ld();
        const bool masked = __any_sync(0xffffffffu, nvalid < 64);
        auto mask = [&](uint32_t(&y)[32], int n) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= n) y[e] = __float_as_uint(-INFINITY);
        };
        if (masked) {
          mask(v, nvalid);
          mask(v2, nvalid - 32);
        }
        float mx[2] = {-INFINITY, -INFINITY};   // of the raw products (the scale is positive)
#pragma unroll
        for (int e = 0; e < 32; e += 4)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            mx[y] = max3(mx[y], __uint_as_float(v[e + 2 * y]), __uint_as_float(v[e + 2 * y + 1]));
            mx[y] = max3(mx[y], __uint_as_float(v2[e + 2 * y]), __uint_as_float(v2[e + 2 * y + 1]));
          }
        float mt = fmaxf(mx[0], mx[1]) * p.scale_log2;
        // The reference moves only when the maximum grows by more than 2^8: rarely.  Each warp tells the other whether its
        // keys ask for it, and does the first 32 keys with the standing reference meanwhile.
        auto asks = [&](float y) { return y > m + kRescaleThreshold || (m == -INFINITY && y > -INFINITY); };
        const bool any = __any_sync(0xffffffffu, asks(mt));
        if (lane == 0) put(s_need + 64 * (j & 1) + 4 * half, ok ? any : 2);      // (2: a wait expired; both warps leave here)
        const uint64_t c2 = pair(p.scale_log2, p.scale_log2);
        uint64_t rs = 0ull;
        uint32_t pk[16];
        auto probs = [&](const uint32_t(&y)[32]) {      // of 32 keys: their sum in float32, and as bf16 (the operand type)
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t mr2 = pair(-ref, -ref);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            unpair(fma2(pair(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), c2, mr2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            rs = add2(rs, pair(p0, p1));
            pk[e >> 1] = pack_bf16(p0, p1);
          }
        };
        probs(v);
        pair_sync();
        const int other = (int)get(s_need + 64 * (j & 1) + 4 * (half ^ 1));
        ok = ok && other != 2;
        if (!ok) break;
        if (any || other) {
          put(s_row + 8192 * half, __float_as_uint(mt));
          pair_sync();
          mt = fmaxf(mt, __uint_as_float(get(s_row + 8192 * (half ^ 1))));
          pair_sync();                                  // both have read
          const bool move = asks(mt);
          const float mnew = move ? mt : m, alpha = move ? ex2(m - mnew) : 1.f;      // m = -inf -> 0
          if (j > 0) {
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {            // (S(j) complete implies that the product before it is in O)
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + cc * 32, o);
            }
          }
          l *= alpha;
          m = mnew;
          rs = 0ull;
          tmem_ld32(tS, v);                             // (not kept in registers for this)
          tmem_wait_ld();
          if (masked) mask(v, nvalid);
          probs(v);
        }
        // P stays within this warp's own (already read) columns
        tmem_st16(tS, pk);
        probs(v2);
        tmem_st16(tS + 16, pk);
        float r0, r1;
        unpair(rs, r0, r1);
        l += r0 + r1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i));
      }
      if (!ok) break;
      ok = wait_w(o_full(i), no & 1, abort_flag, p.status, p.wait_ns);
      if (lane == 0) put(s_need + 64 * (T & 1) + 4 * half, ok ? 0 : 2);
      put(s_row + 8192 * half, __float_as_uint(l));
      pair_sync();
      l += __uint_as_float(get(s_row + 8192 * (half ^ 1)));       // the row's sum (of two terms: the same in both warps)
      ok = ok && get(s_need + 64 * (T & 1) + 4 * (half ^ 1)) != 2;
      pair_sync();
      if (!ok) break;
      tc_fence_after();
      const bool fix = not_finite[4 * i + (no & 3)] != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(flag_free(i, no));
      ++no;
      write_output(p, OutArgs{x.start, x.len, x.t0, x.kh, x.h0, i * p.tp, quarter * 32, 64 * half, t_pos, tO,
                              sbase + L::kO + (uint32_t)(st >> 5) * 2048u, 1.f / l, fix});
      if (t_pos < x.len && half == 0)
        p.lse[(x.h0 + (r & (p.pk - 1))) * p.total + (int64_t)x.start + t_pos] = (m + __log2f(l)) * 0.6931471805599453f;
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

// ------------------------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool make_map_packed(CUtensorMap* m, const void* base, int H, int64_t total, Strided s, int heads, int tokens) {
  static EncodeTiledFn enc = nullptr;      // resolved once; the driver symbol never changes
  if (!enc) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)H, (cuuint64_t)total};
  cuuint64_t strides[2] = {(cuuint64_t)s.h * 2, (cuuint64_t)s.t * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int fwd_tile(int G) { return 256 / packed_heads(G); }
int head_units(int Hkv, int G) { return Hkv * (G / packed_heads(G)); }

cudaError_t launch_fwd_tc(const void* q, const void* k, const void* v, void* o, void* o_lo, float* lse,
                          const Work& work, const Problem& p, cudaStream_t st) {
  const int pk = packed_heads(p.G);
  const size_t smem = FwdSmem::kBytes + 1024;
  auto kernel = work.cu ? packed_fwd_tc_kernel<true> : packed_fwd_tc_kernel<false>;
  cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!make_map_packed(&mq, q, p.Hq, p.total, p.q, pk, 128 / pk) || !make_map_packed(&mk, k, p.Hkv, p.total, p.k, 1, kBN) ||
      !make_map_packed(&mv, v, p.Hkv, p.total, p.v, 1, kBN))
    return cudaErrorInvalidValue;
  FwdParams a{p.Hq, p.Hkv, p.G, pk, pk == 8 ? 3 : pk == 4 ? 2 : pk - 1, 128 / pk, p.Hkv * (p.G / pk), p.total, p.scale * kLog2eF,
              static_cast<const __nv_bfloat16*>(v), p.v, static_cast<__nv_bfloat16*>(o), static_cast<__nv_bfloat16*>(o_lo), lse,
              work, p.fill_tail, p.status, p.wait_ns};
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t units = list_capacity(p.total, p.n_seqs, fwd_tile(p.G)) * a.hu;
  return launch_dependent(kernel, dim3((unsigned)(units < 1 ? 1 : units < sms ? units : sms)),
                          dim3(kThreads), smem, st, 1, mq, mk, mv, a);
}

}  // namespace packed
}  // namespace hga
