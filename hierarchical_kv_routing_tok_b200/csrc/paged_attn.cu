// Attention of one new token per sequence over a paged K/V cache.
//
//   o = sum_u softmax_u(scale q.k_u) v_u over the cached tokens u < seq_len of the query's sequence
//
// Bound by reading the cache once: 4 Hq/Hkv flops per element read.  The work is the list of token tiles of all (query, KV
// head) pairs in order, each pair counting kPairCost tiles more for what its start and end cost; CTA c of N takes the
// share [cW/N, (c+1)W/N) of the list, so every SM has the same work whatever the lengths are.  A pair whose tiles fall to
// several CTAs is joined: each CTA leaves its running maximum, sum and unnormalised output in the workspace, and the CTA
// that finishes last (a counter) adds the parts in the order of their tiles, so the result does not depend on which one that
// is.  Each CTA has at most two such parts, its first and its last.
//
// A producer warp brings a tile's pages with TMA (one box per page) into a ring of three 32 KB stages, two CTAs per SM; four
// warps take a quarter of each tile's tokens, with softmax statistics of their own that meet at the end of the pair.  The
// queries of a KV head are the rows of a pair (up to 16: more query heads are further pairs).
//   bf16: 64 tokens per tile, m16n8k16 products with the queries as rows.  Few rows cannot fill a tcgen05 tile, and the
//         memory is the limit by far.
//         P enters its product as the sum of two bf16 numbers, so that nothing but the output is rounded (error of o at 131K
//         2.25e-3 -> 1.66e-3 of the norm): with up to eight rows the low parts are the tile's empty upper half (no time:
//         170.4 us with and without); with more they take products of their own (32/2 heads, 2 x 131K: 64.7 -> 65.3 us).
//         48 ragged sequences, 32/8 heads: 70 us, 5.7 TB/s; two of 131K: 169 us, 6.3 TB/s; one of 513: 9.3 us, latency.
//   float32: 32 tokens per tile, float32 FMAs: a lane holds four dims; the dot products of eight tokens and four rows
//         are summed over the lanes together, in 31 shuffles that leave one sum on each lane.  The same 48: 125 us, 6.4 TB/s.
#include <cuda.h>
#include <math.h>

#include "pages.cuh"
#include "tc_common.cuh"

namespace hga {
namespace pages {

using namespace tc;

namespace {

constexpr int kRows = 16;              // most query rows of a pair
constexpr int kConsumers = 128;        // threads of the four computing warps
constexpr int kThreads = kConsumers + 32;
constexpr int kStages = 3;
constexpr uint32_t kTileBytes = 16384; // of K, and of V
constexpr int kWindow = 32;            // queries whose row and length are kept in shared memory
// What a pair's start and end cost, in tiles: us with 0, 1, 3 and 6.
//                              bf16                          float32
//   48 ragged, 8/8 heads       74.5  70.4  69.0  68.7        130.6  123.7  123.9  125.2
//   48 ragged, 32/8            79.9  74.3  69.8  69.9        132.7  125.6  125.9  125.2
//   48 ragged, 16/1            26.6  25.4  23.2  23.4        117.2  107.1  107.9  114.3
//   64 of 200 to 600, 32/8     32.5  31.4  30.6  30.8         46.8   45.4   46.0   47.2
//   64 of 200 to 600, 32/2     18.6  18.3  16.0  16.5         70.8   70.7   76.2   84.3
// Equal lengths: any.  One number for both: float32 would gain up to 8 % from 1 with wide groups, nothing with others.
constexpr int kPairCost = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kErrArg = -1;

template <typename T> constexpr int kTileOf = (int)(kTileBytes / (kD * sizeof(T)));   // tokens per tile: 64 or 32

struct Part {                          // in the workspace, two per CTA
  float o[kRows * kD];
  float m[kRows], l[kRows];            // maximum in units of log2, sum
};

struct Args {
  const int32_t* rows;
  const int32_t* table;
  const int32_t* seq_len;
  const void* q;
  void* o;
  float* lse;
  Part* parts;
  int* counters;                       // one per CTA, zero between calls
  int* status;
  int64_t q_stride_n;
  int n, Hq, Hkv, G, subs;             // subs: pairs per KV head (16 query rows each)
  int page, max_seqs, max_pages, n_pages;
  float c2;                            // scale * log2(e)
  uint64_t wait_ns;
};

struct Range {
  int64_t begin, end, first;           // this CTA's share of the list; where the query at `begin` starts
  int64_t total;
  int n_cta, query;
};

struct Smem {
  unsigned char kv[kStages][2][kTileBytes];          // 1 KB aligned (128-byte swizzle)
  float merge[4][8][kD];                             // the four warps' outputs, eight rows at a time
  float m[4][kRows], l[4][kRows];
  uint64_t full[kStages], empty[kStages];
  Range range;
  int win_row[kWindow], win_len[kWindow];            // of the queries from range.query on
  int64_t sums[kThreads / 32];
  uint32_t valid[kStages];                           // pages of the tile that were loaded, one bit each
  int abort, flag;
};
static_assert(2 * (sizeof(Smem) + 1024) <= 228 * 1024, "two CTAs per SM");

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Tokens of query i, and its row (0 tokens for a bad row or length: recorded).
__device__ __forceinline__ int tokens_of(const Args& a, int i, int* row) {
  const int r = a.rows[i];
  int L = r >= 0 && r < a.max_seqs ? a.seq_len[r] : -1;
  if (L < 0 || (int64_t)L > (int64_t)a.max_pages * a.page) {
    set_status(a.status, kErrArg);
    L = 0;
  }
  *row = r;
  return L;
}
template <typename T>
__device__ __forceinline__ int64_t units_of(int L) {   // of one pair
  return L ? (L + kTileOf<T> - 1) / kTileOf<T> + kPairCost : 0;
}
__device__ __forceinline__ int64_t cta_of(int64_t w, int64_t total, int64_t n) { return ((w + 1) * n - 1) / total; }

// Finds this CTA's share.  Called by all threads.
template <typename T>
__device__ __forceinline__ void find_range(const Args& a, Smem& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
  const int pairs = a.Hkv * a.subs;
  int64_t mine = 0;
  int L = 0, row = 0;                                  // of the last of this thread's queries
  for (int i = i0; i < i1; ++i) {
    L = tokens_of(a, i, &row);
    mine += units_of<T>(L) * pairs;
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s.sums[warp] = x;
  __syncthreads();
  int64_t base = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += s.sums[w];
    total += s.sums[w];
  }
  const int64_t n_cta = min((int64_t)gridDim.x, total);
  const int64_t begin = blockIdx.x < n_cta ? blockIdx.x * total / n_cta : 0;
  const int64_t end = blockIdx.x < n_cta ? (blockIdx.x + 1) * total / n_cta : 0;
  if (tid == 0) {
    s.range.total = total;
    s.range.n_cta = (int)n_cta;
    s.range.begin = begin;
    s.range.end = end;
    s.range.query = 0;
    s.range.first = 0;
  }
  __syncthreads();
  if (begin < end && begin >= base && begin < base + mine) {
    int64_t at = base;
    for (int i = i0; i < i1; ++i) {
      int r;
      const int64_t t = units_of<T>(per == 1 ? L : tokens_of(a, i, &r)) * pairs;
      if (begin < at + t) {
        s.range.query = i;
        s.range.first = at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  const int q0 = s.range.query;
  if (per == 1) {
    if (tid >= q0 && tid < q0 + kWindow && tid < a.n) {
      s.win_row[tid - q0] = row;
      s.win_len[tid - q0] = L;
    }
  } else if (tid < kWindow && q0 + tid < a.n) {
    s.win_len[tid] = tokens_of(a, q0 + tid, &row);
    s.win_row[tid] = row;
  }
  __syncthreads();
}

// Tiles [t0, t1) of pair `pair` (of nt tiles) of query i.
struct Segment {
  int i, row, L, nt, kh, h0, n_rows;   // KV head, first query head, query heads of the pair
  int t0, t1;
  int64_t tile0;                       // list position of the pair's first tile
};
// The walk over this CTA's segments; each warp walks by itself.
struct Walk {
  int64_t w, end, first;
  int i;
};
template <typename T>
__device__ __forceinline__ bool next_segment(const Args& a, const Smem& s, Walk& k, Segment* g) {
  const int pairs = a.Hkv * a.subs;
  while (k.w < k.end) {
    int64_t u;
    for (;;) {
      const int x = k.i - s.range.query;
      if (x < kWindow) {
        g->L = s.win_len[x];
        g->row = s.win_row[x];
      } else {
        g->L = tokens_of(a, k.i, &g->row);
      }
      u = units_of<T>(g->L);
      if (k.w < k.first + u * pairs) break;
      k.first += u * pairs;
      ++k.i;
    }
    g->i = k.i;
    g->nt = (int)(u - kPairCost);
    const int64_t x = k.w - k.first, pair = x / u, y = x - pair * u;
    const int64_t take = min(u - y, k.end - k.w);
    g->kh = (int)(a.subs == 1 ? pair : pair / a.subs);
    const int sub = (int)(pair - (int64_t)g->kh * a.subs);
    g->h0 = g->kh * a.G + sub * kRows;
    g->n_rows = min(kRows, a.G - sub * kRows);
    g->t0 = (int)max(y - kPairCost, (int64_t)0);
    g->t1 = (int)max(y + take - kPairCost, (int64_t)0);
    g->tile0 = k.first + pair * u + kPairCost;
    k.w += take;
    if (g->t1 > g->t0) return true;
  }
  return false;
}

// One row's final 4 dims and, once, its lse.
template <typename T>
__device__ __forceinline__ void emit(const Args& a, const Segment& g, int r, int c4, float4 v, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;          // (0: every token was left out)
  v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
  const int64_t row = (int64_t)g.i * a.Hq + g.h0 + r;
  store4(static_cast<T*>(a.o) + row * kD + 4 * c4, v);
  if (c4 == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

// After a CTA's part of a split pair is in the workspace: the last CTA to get here adds the parts up, in order.  Called by the
// 128 consumer threads; a warp has the rows w, w + 4, ...  (One part after another took up to 33000 cycles under load.)
template <typename T>
__device__ __forceinline__ void join(const Args& a, const Segment& g, Smem& s) {
  const int64_t c0 = cta_of(g.tile0, s.range.total, s.range.n_cta), c1 = cta_of(g.tile0 + g.nt - 1, s.range.total, s.range.n_cta);
  const int n = (int)(c1 - c0 + 1);
  __threadfence();
  consumer_sync();
  if (threadIdx.x == 0) {
    const int before = atomicAdd(&a.counters[c0], 1);
    s.flag = before == n - 1;
    if (before == n - 1) a.counters[c0] = 0;
  }
  consumer_sync();
  if (!s.flag) return;
  __threadfence();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto part = [&](int p) -> const Part* { return a.parts + (p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)); };
  float m[4], l[4];
  float4 acc[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    m[y] = -INFINITY;
    l[y] = 0.f;
    acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int p0 = 0; p0 < n; p0 += 32) {                 // 32 parts: a lane has the statistics of one
    float f[4], lp[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const bool in = p0 + lane < n && warp + 4 * y < g.n_rows;
      f[y] = in ? __ldcg(&part(p0 + lane)->m[warp + 4 * y]) : -INFINITY;
      lp[y] = in ? __ldcg(&part(p0 + lane)->l[warp + 4 * y]) : 0.f;
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float mn = f[y];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mn = fmaxf(mn, m[y]);
      const float ref = mn == -INFINITY ? 0.f : mn, old = exp2f(m[y] - ref);
      m[y] = mn;
      f[y] = exp2f(f[y] - ref);
      float x = f[y] * lp[y];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      l[y] = l[y] * old + x;
      acc[y].x *= old; acc[y].y *= old; acc[y].z *= old; acc[y].w *= old;
    }
    const int np = min(32, n - p0);
    for (int p = 0; p < np; p += 4) {
      float4 v[4][4];                                  // four parts of up to four rows in flight
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          v[z][y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p + z < np && warp + 4 * y < g.n_rows)
            v[z][y] = __ldcg(reinterpret_cast<const float4*>(part(p0 + p + z)->o + (warp + 4 * y) * kD) + lane);
        }
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float e = __shfl_sync(0xffffffffu, f[y], p + z);       // (0 past the last part)
          acc[y].x += e * v[z][y].x; acc[y].y += e * v[z][y].y; acc[y].z += e * v[z][y].z; acc[y].w += e * v[z][y].w;
        }
    }
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
    if (warp + 4 * y < g.n_rows) emit<T>(a, g, warp + 4 * y, lane, acc[y], m[y], l[y]);
}

// Eight rows (8 x ..) of the four warps' outputs in s.merge, their statistics in s.m, s.l: summed, and stored as the result
// or as this CTA's part.  kSwap: columns are permuted by row (4 c ^ 8 (row mod 4)).
template <typename T, bool kSwap>
__device__ __forceinline__ void sum_warps(const Args& a, const Segment& g, const Smem& s, int x, bool whole, Part* part) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int rr = ((int)threadIdx.x >> 5) + 4 * y, c4 = threadIdx.x & 31, row = rr + 8 * x;
    if (row >= g.n_rows) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) mm = fmaxf(mm, s.m[k][row]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float ll = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = ex2(s.m[k][row] - ref);
      const float4 u = *reinterpret_cast<const float4*>(&s.merge[k][rr][kSwap ? (4 * c4) ^ ((rr & 3) << 3) : 4 * c4]);
      v.x += f * u.x; v.y += f * u.y; v.z += f * u.z; v.w += f * u.w;
      ll += f * s.l[k][row];
    }
    if (whole) {
      emit<T>(a, g, row, c4, v, mm, ll);
    } else {
      __stcg(reinterpret_cast<float4*>(part->o + row * kD) + c4, v);
      if (c4 == 0) {
        __stcg(&part->m[row], mm);
        __stcg(&part->l[row], ll);
      }
    }
  }
}

// p = first part (cut to bf16) + rest.  The rest is never 0 nor negative (2^-126 is far below any sum's rounding): both products
// with an infinite v then have its sign, where 0 or a change of sign would make their sum NaN.
__device__ __forceinline__ uint32_t first_parts(float p0, float p1) {
  return __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
}
__device__ __forceinline__ float rest(float p) {
  return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xffff0000u), 1.17549435e-38f);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t row, int32_t head, int32_t page,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int32_t row, int32_t head,
                                            int32_t page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// What both kernels begin with: barriers, this CTA's share, and whether there is any.
template <typename T>
__device__ __forceinline__ bool begin(const Args& a, Smem& s) {
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 4);
    }
    s.abort = 0;
    mbar_fence_init();
  }
  pdl_wait();
  find_range<T>(a, s);                                 // (its barriers also publish the mbarriers)
  return s.range.begin < s.range.end;
}

// Queries without tokens: zeros and -inf, spread over the CTAs.  Called by the producer warp, when its loads are issued.
template <typename T>
__device__ __forceinline__ void write_empty(const Args& a) {
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    int row;
    if (tokens_of(a, i, &row) != 0) continue;
    for (int h = 0; h < a.Hq; ++h) {
      store4(static_cast<T*>(a.o) + ((int64_t)i * a.Hq + h) * kD + 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f));
      if (lane == 0) a.lse[(int64_t)i * a.Hq + h] = -INFINITY;
    }
  }
}

// The producer warp: the tiles of this CTA's segments, one after another.
template <typename T>
__device__ __forceinline__ void produce(const Args& a, Smem& s, const CUtensorMap& tm_k, const CUtensorMap& tm_v) {
  constexpr int kTile = kTileOf<T>;
  const int lane = threadIdx.x & 31;
  auto full = [&](int i) { return smem_u32(&s.full[i]); };
  volatile int* abort_flag = &s.abort;
  const int R = min(a.page, kTile);                    // tokens per box
  const int boxes = kTile / R;                         // boxes of a tile
  const uint32_t kv0 = smem_u32(&s.kv[0][0][0]);
  Walk walk{s.range.begin, s.range.end, s.range.first, s.range.query};
  Segment g;
  int64_t J = 0;
  bool ok = true;
  while (ok && next_segment<T>(a, s, walk, &g)) {
    const int32_t* ids = a.table + (int64_t)g.row * a.max_pages;
    // box b of the sequence: tokens b R ..; lane l holds the pages of 32 boxes at a time
    const int b_end = min(g.t1 * boxes, (g.L + R - 1) / R);
    int b0 = g.t0 * boxes;
    auto page_of = [&](int b) { return b < b_end ? ids[(int64_t)b * R / a.page] : -1; };
    int32_t cur = page_of(b0 + lane), nxt = page_of(b0 + 32 + lane);
    for (int t = g.t0; t < g.t1; ++t, ++J) {
      const int st = (int)(J % kStages);
      if (t * boxes >= b0 + 32) {
        b0 += 32;
        cur = nxt;
        nxt = page_of(b0 + 32 + lane);
      }
      const int b = t * boxes + lane;                  // this lane's box of the tile
      const int32_t id = __shfl_sync(0xffffffffu, cur, (t * boxes - b0 + lane) & 31);
      const bool have = lane < boxes && b < b_end, good = have && id >= 0 && id < a.n_pages;
      if (have && !good) set_status(a.status, kErrArg);
      const uint32_t mask = __ballot_sync(0xffffffffu, good);
      int go = 1;
      if (lane == 0) {
        go = mbar_wait(smem_u32(&s.empty[st]), (uint32_t)((J / kStages) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
        if (go) {
          s.valid[st] = mask;
          mbar_arrive_expect_tx(full(st), (uint32_t)__popc(mask) * R * kD * sizeof(T) * 2);
        }
      }
      ok = __shfl_sync(0xffffffffu, go, 0) != 0;
      if (!ok) break;
      if (good) {
        const uint32_t dst = kv0 + st * 2 * kTileBytes + lane * R * (kD * (uint32_t)sizeof(T));
        const int row = (int)((int64_t)b * R % a.page);
        if (sizeof(T) == 2) {
          tma_load_5d(dst, &tm_k, row, g.kh, id, full(st));
          tma_load_5d(dst + kTileBytes, &tm_v, row, g.kh, id, full(st));
        } else {
          tma_load_4d(dst, &tm_k, row, g.kh, id, full(st));
          tma_load_4d(dst + kTileBytes, &tm_v, row, g.kh, id, full(st));
        }
      }
      __syncwarp();
    }
  }
  write_empty<T>(a);
  // its loads have landed before the CTA may exit
  if (lane == 0)
    for (int64_t j = J > kStages ? J - kStages : 0; j < J; ++j)
      drain_wait(full((int)(j % kStages)), (uint32_t)((j / kStages) & 1), a.status);
}

// ------------------------------------------------------------------------------------ bf16, tensor cores
// RH: 1 when a pair has at most 8 query rows (the upper half of the m16 tile is free for the low parts of P), else 2.  One
// sequence of 513 tokens, 32/8 heads: 9.3 us with 1, 9.6 with 2; eight of 1000: 14.8 and 15.4; long ones the same.
template <int RH>
__global__ void __launch_bounds__(kThreads, 2)
    paged_bf16_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
  typedef __nv_bfloat16 T;
  constexpr int kTile = kTileOf<T>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = &s.abort;
  const bool work = begin<T>(a, s);
  if (warp == 4) produce<T>(a, s, tm_k, tm_v);
  if (warp == 4 || !work) return;
  // ======================= the four computing warps: keys 16 warp .. + 15 of each tile
  const int R = min(a.page, kTile);
  const int fg = lane >> 2, tq = lane & 3;             // fragment row and column pair
  const int key0 = 16 * warp;
  Walk walk{s.range.begin, s.range.end, s.range.first, s.range.query};
  Segment g;
  int64_t J = 0;
  bool alive = true;                                   // no wait has expired
  while (next_segment<T>(a, s, walk, &g)) {
    // queries: rows fg and fg + 8, dims 16 ks + 2 tq + {0, 1} and + 8
    uint32_t qf[8][4];
    {
      const T* qb = static_cast<const T*>(a.q) + g.i * a.q_stride_n + (int64_t)g.h0 * kD + 2 * tq;
      const bool in0 = fg < g.n_rows, in1 = RH == 2 && fg + 8 < g.n_rows;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const T *p0 = qb + fg * kD + 16 * ks, *p1 = p0 + 8 * kD;
        qf[ks][0] = in0 ? *reinterpret_cast<const uint32_t*>(p0) : 0u;
        qf[ks][2] = in0 ? *reinterpret_cast<const uint32_t*>(p0 + 8) : 0u;
        qf[ks][1] = in1 ? *reinterpret_cast<const uint32_t*>(p1) : 0u;
        qf[ks][3] = in1 ? *reinterpret_cast<const uint32_t*>(p1 + 8) : 0u;
      }
    }
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[RH], l[RH];
#pragma unroll
    for (int x = 0; x < RH; ++x) { m[x] = -INFINITY; l[x] = 0.f; }

    for (int t = g.t0; t < g.t1; ++t, ++J) {
      const int st = (int)(J % kStages);
      alive = alive && mbar_wait_w(smem_u32(&s.full[st]), (uint32_t)((J / kStages) & 1), abort_flag, a.status, a.wait_ns);
      const int nvalid = min(kTile, g.L - t * kTile) - key0;       // of this warp's 16 keys
      if (alive && nvalid > 0 && (s.valid[st] >> (key0 / R) & 1u)) {
        // key x of this warp: row (key0 + x) % R of its box
        const uint32_t kbase = smem_u32(&s.kv[st][0][0]) + (key0 / R) * R * (kD * 2), vbase = kbase + kTileBytes;
        const int r0 = key0 % R;
        if (nvalid < 16) {
          // keys past the end: whatever the page holds there must not meet p = 0
          for (int x = nvalid * 16 + lane; x < 16 * 16; x += 32) {
            const int r = r0 + (x >> 4), ch = x & 15;
            const uint32_t ad = vbase + (ch >> 3) * R * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ad), "r"(0) : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        float c[2][4] = {};
        {
          // matrices of one ldmatrix: keys 0-7 dims 0-7, keys 0-7 dims 8-15, keys 8-15 dims 0-7, 8-15
          const int r = r0 + (lane & 7) + ((lane >> 4) << 3);
          const uint32_t rb = kbase + r * 128;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const int ch = 2 * (ks & 3) + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm4(b, rb + (ks >> 2) * R * 128 + ((ch ^ (r & 7)) << 4));
            mma16816(c[0], qf[ks], b[0], b[1]);
            mma16816(c[1], qf[ks], b[2], b[3]);
          }
        }
        if (nvalid < 16) {
#pragma unroll
          for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * n8 + 2 * tq + (e & 1) >= nvalid) c[n8][e] = -INFINITY;
        }
        uint32_t pf[4], pl[4];                         // P: its first parts, its low parts
        float alpha[2] = {1.f, 1.f};
        bool moved = false;
#pragma unroll
        for (int x = 0; x < RH; ++x) {
          float mx = fmaxf(fmaxf(c[0][2 * x], c[0][2 * x + 1]), fmaxf(c[1][2 * x], c[1][2 * x + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * a.c2;
          const float mnew = fmaxf(m[x], mx);
          const float ref = mnew == -INFINITY ? 0.f : mnew;
          moved |= mnew != m[x];
          alpha[x] = ex2(m[x] - ref);
          m[x] = mnew;
          const float p0 = ex2(fmaf(c[0][2 * x], a.c2, -ref)), p1 = ex2(fmaf(c[0][2 * x + 1], a.c2, -ref));
          const float p2 = ex2(fmaf(c[1][2 * x], a.c2, -ref)), p3 = ex2(fmaf(c[1][2 * x + 1], a.c2, -ref));
          l[x] = l[x] * alpha[x] + ((p0 + p1) + (p2 + p3));        // of this thread's columns
          pf[x] = first_parts(p0, p1);
          pf[2 + x] = first_parts(p2, p3);
          pl[x] = pack_bf16(rest(p0), rest(p1));
          pl[2 + x] = pack_bf16(rest(p2), rest(p3));
        }
        if (RH == 1) {                                 // the low parts take the empty upper half of the tile
          pf[1] = pl[0];
          pf[3] = pl[2];
          alpha[1] = alpha[0];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i][0] *= alpha[0]; o[i][1] *= alpha[0];
            o[i][2] *= alpha[1]; o[i][3] *= alpha[1];
          }
        }
        {
          // matrices: keys 0-7 dims 0-7, keys 8-15 dims 0-7, keys 0-7 dims 8-15, keys 8-15 dims 8-15
          const int r = r0 + (lane & 15);
          const uint32_t rb = vbase + r * 128;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const int ch = 2 * (d & 3) + (lane >> 4);
            uint32_t b[4];
            ldsm4t(b, rb + (d >> 2) * R * 128 + ((ch ^ (r & 7)) << 4));
            mma16816(o[2 * d], pf, b[0], b[1]);
            mma16816(o[2 * d + 1], pf, b[2], b[3]);
            if (RH == 2) {
              mma16816(o[2 * d], pl, b[0], b[1]);
              mma16816(o[2 * d + 1], pl, b[2], b[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[st]));
    }

    // ---- the four warps' statistics and outputs meet
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    Part* part = a.parts + 2 * (int64_t)blockIdx.x + (g.t0 == 0 ? 1 : 0);
    consumer_sync();                                   // the last pair's sums have been read
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (tq == 0) {
        s.m[warp][fg + 8 * x] = m[x];
        s.l[warp][fg + 8 * x] = l[x];
      }
    }
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      if (x) consumer_sync();                          // the first eight rows have been read
#pragma unroll
      for (int i = 0; i < 16; ++i)                     // (columns permuted by row: no bank conflicts)
        *reinterpret_cast<float2*>(&s.merge[warp][fg][(8 * i + 2 * tq) ^ ((fg & 3) << 3)]) =
            RH == 1 ? make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]) : make_float2(o[i][2 * x], o[i][2 * x + 1]);
      consumer_sync();
      sum_warps<T, true>(a, g, s, x, whole, part);
    }
    if (!whole) join<T>(a, g, s);
  }
}

// ------------------------------------------------------------------------------------ float32
// Sums v[0 .. 31] over the lanes: lane l gets the sum of v[l].
__device__ __forceinline__ float lane_sums(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  return v[0];
}

// NB: blocks of four query rows (1, 2 or 4 for pairs of at most 4, 8 or 16).  48 sequences, 32/8 heads: 126 us with 1, 217 with 4.
template <int NB>
__global__ void __launch_bounds__(kThreads, 2)
    paged_f32_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
  typedef float T;
  constexpr int kTile = kTileOf<T>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = &s.abort;
  const bool work = begin<T>(a, s);
  if (warp == 4) produce<T>(a, s, tm_k, tm_v);
  if (warp == 4 || !work) return;
  // ======================= the four computing warps: keys 8 warp .. + 7 of each tile; a lane has dims 4 lane .. + 3
  const int R = min(a.page, kTile);
  const int key0 = 8 * warp;
  Walk walk{s.range.begin, s.range.end, s.range.first, s.range.query};
  Segment g;
  int64_t J = 0;
  bool alive = true;                                   // no wait has expired
  while (next_segment<T>(a, s, walk, &g)) {
    float4 q[4 * NB], o[4 * NB];
#pragma unroll
    for (int r = 0; r < 4 * NB; ++r) {
      q[r] = o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < g.n_rows) {
        q[r] = load4(static_cast<const T*>(a.q) + g.i * a.q_stride_n + (int64_t)(g.h0 + r) * kD + 4 * lane);
        q[r].x *= a.c2; q[r].y *= a.c2; q[r].z *= a.c2; q[r].w *= a.c2;
      }
    }
    // lane l has the score of key l / 4, row l % 4 of a block; m, l of that row, the same in its eight lanes
    float m[NB], l[NB];
#pragma unroll
    for (int x = 0; x < NB; ++x) { m[x] = -INFINITY; l[x] = 0.f; }
    for (int t = g.t0; t < g.t1; ++t, ++J) {
      const int st = (int)(J % kStages);
      alive = alive && mbar_wait_w(smem_u32(&s.full[st]), (uint32_t)((J / kStages) & 1), abort_flag, a.status, a.wait_ns);
      const int nvalid = min(kTile, g.L - t * kTile) - key0;       // of this warp's 8 keys
      if (alive && nvalid > 0 && (s.valid[st] >> (key0 / R) & 1u)) {
        const float4* kt = reinterpret_cast<const float4*>(&s.kv[st][0][0]) + key0 * (kD / 4) + lane;
        const float4* vt = reinterpret_cast<const float4*>(&s.kv[st][1][0]) + key0 * (kD / 4) + lane;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          if (4 * x >= g.n_rows) break;
          float d[32];
#pragma unroll
          for (int key = 0; key < 8; ++key) {
            const float4 k = kt[key * (kD / 4)];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float4 y = q[4 * x + r];
              d[4 * key + r] = k.x * y.x + k.y * y.y + k.z * y.z + k.w * y.w;
            }
          }
          float sc = lane_sums(d);
          if ((lane >> 2) >= nvalid) sc = -INFINITY;
          float mx = sc;
#pragma unroll
          for (int h = 4; h < 32; h <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
          const float mnew = fmaxf(m[x], mx), ref = mnew == -INFINITY ? 0.f : mnew;
          const float alpha = exp2f(m[x] - ref), p = exp2f(sc - ref);
          m[x] = mnew;
          l[x] = l[x] * alpha + p;                     // of this lane's key
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float al = __shfl_sync(0xffffffffu, alpha, r);
              float4& y = o[4 * x + r];
              y.x *= al; y.y *= al; y.z *= al; y.w *= al;
            }
          }
#pragma unroll
          for (int key = 0; key < 8; ++key) {
            if (key >= nvalid) break;                  // (whatever the page holds there)
            const float4 v = vt[key * (kD / 4)];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float pr = __shfl_sync(0xffffffffu, p, 4 * key + r);
              float4& y = o[4 * x + r];
              y.x += pr * v.x; y.y += pr * v.y; y.z += pr * v.z; y.w += pr * v.w;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[st]));
    }
    // ---- the four warps' statistics and outputs meet
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    Part* part = a.parts + 2 * (int64_t)blockIdx.x + (g.t0 == 0 ? 1 : 0);
    consumer_sync();                                   // the last pair's sums have been read
#pragma unroll
    for (int x = 0; x < NB; ++x) {
#pragma unroll
      for (int h = 4; h < 32; h <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], h);
      if (lane < 4) {
        s.m[warp][4 * x + lane] = m[x];
        s.l[warp][4 * x + lane] = l[x];
      }
    }
#pragma unroll
    for (int x = 0; x < (NB + 1) / 2; ++x) {
      if (8 * x >= g.n_rows) break;
      if (x) consumer_sync();                          // the first eight rows have been read
#pragma unroll
      for (int r = 0; r < (NB == 1 ? 4 : 8); ++r) store4(&s.merge[warp][r][4 * lane], o[8 * x + r]);
      consumer_sync();
      sum_warps<T, false>(a, g, s, x, whole, part);
    }
    if (!whole) join<T>(a, g, s);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A layer's pool; a box is one page's tokens (at most a tile's) of one head.  bf16: {64 dims, tokens, 2 halves, KV heads,
// pages}, the two 64-dim halves one after the other, 128-byte swizzle.  float32: {128 dims, tokens, KV heads, pages}.
bool make_pool_map(CUtensorMap* m, const void* base, const Cache& c) {
  static EncodeTiledFn enc = nullptr;    // resolved once; the driver symbol never changes
  if (!enc) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  const bool bf16 = c.elem == 2;
  const cuuint64_t row = (cuuint64_t)kD * c.elem, page = row * c.page;
  const cuuint32_t tile = bf16 ? kTileOf<__nv_bfloat16> : kTileOf<float>, R = c.page < (int)tile ? c.page : tile;
  const cuuint64_t dims5[5] = {64, (cuuint64_t)c.page, 2, (cuuint64_t)c.Hkv, (cuuint64_t)c.n_pages};
  const cuuint64_t strides5[4] = {row, 128, page, (cuuint64_t)c.page_bytes};
  const cuuint32_t box5[5] = {64, R, 2, 1, 1};
  const cuuint64_t dims4[4] = {kD, (cuuint64_t)c.page, (cuuint64_t)c.Hkv, (cuuint64_t)c.n_pages};
  const cuuint64_t strides4[3] = {row, page, (cuuint64_t)c.page_bytes};
  const cuuint32_t box4[4] = {kD, R, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, bf16 ? 5 : 4,
             const_cast<void*>(base), bf16 ? dims5 : dims4, bf16 ? strides5 : strides4, bf16 ? box5 : box4, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxCtas = 2 * 256;      // CTAs the workspace has room for (two per SM)
constexpr size_t kCounterBytes = kMaxCtas * sizeof(int);

}  // namespace

size_t paged_attn_scratch_bytes() { return kCounterBytes + 2 * (size_t)kMaxCtas * sizeof(Part); }

cudaError_t launch_paged_attn(bool bf16, const Cache& c, int layer, int n, int Hq, float scale,
                              const int32_t* rows, const void* q, int64_t q_stride_n, const void* k_pool,
                              const void* v_pool, void* o, float* lse, void* scratch, uint64_t wait_ns,
                              cudaStream_t st) {
  Args a{};
  a.rows = rows;
  a.table = c.table;
  a.seq_len = c.seq_len;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.counters = static_cast<int*>(scratch);
  a.parts = reinterpret_cast<Part*>(static_cast<char*>(scratch) + kCounterBytes);
  a.status = c.status;
  a.q_stride_n = q_stride_n;
  a.n = n;
  a.Hq = Hq;
  a.Hkv = c.Hkv;
  a.G = Hq / c.Hkv;
  a.subs = (a.G + kRows - 1) / kRows;
  a.page = c.page;
  a.max_seqs = c.max_seqs;
  a.max_pages = c.max_pages;
  a.n_pages = c.n_pages;
  a.c2 = scale * kLog2e;
  a.wait_ns = wait_ns;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  auto kernel = bf16       ? (a.G <= 8 ? paged_bf16_kernel<1> : paged_bf16_kernel<2>)
                : a.G <= 4 ? paged_f32_kernel<1>
                : a.G <= 8 ? paged_f32_kernel<2>
                           : paged_f32_kernel<4>;
  e = set_smem(kernel, sizeof(Smem));
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, static_cast<const char*>(k_pool) + layer * c.layer_bytes, c) ||
      !make_pool_map(&mv, static_cast<const char*>(v_pool) + layer * c.layer_bytes, c))
    return cudaErrorInvalidValue;
  // two CTAs per SM, and no more than there can be units of work
  const int64_t tile = bf16 ? kTileOf<__nv_bfloat16> : kTileOf<float>;
  const int64_t units = (int64_t)n * c.Hkv * a.subs * (((int64_t)c.max_pages * c.page + tile - 1) / tile + kPairCost);
  int64_t grid = 2LL * sms;
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (grid > units) grid = units;
  return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), sizeof(Smem), st, 1, mk, mv, a);
}

}  // namespace pages
}  // namespace hga
