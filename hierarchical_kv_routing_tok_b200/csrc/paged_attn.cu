// Attention of one new token per sequence over a paged K/V cache.
//
//   o = sum_u softmax_u(scale q.k_u) v_u over the cached tokens u < seq_len of the query's sequence
//
// Bound by reading the cache once: 4 Hq/Hkv flops per element read.  The work is the list of 64-token
// tiles of all (query, KV head) pairs in order; CTA c of N takes the tiles [cW/N, (c+1)W/N), so every
// SM reads the same number of bytes whatever the lengths are.  A pair whose tiles fall to several CTAs
// is joined: each CTA leaves its running maximum, sum and unnormalised output in the workspace, and
// the CTA that finishes last (a counter) adds the parts in the order of their tiles, so the result
// does not depend on which one that is.  Each CTA has at most two such parts, its first and its last.
//
// bf16: the queries of a KV head are the rows of an m16n8k16 product (up to 16 rows: more query heads
// are further pairs).  A producer warp brings a tile's pages with TMA (one box of {64 dims, rows, 2
// halves} per page, 128-byte swizzle) into a ring; four warps take 16 keys of each tile, with softmax
// statistics of their own that meet at the end of the pair.  Few rows cannot fill a tcgen05 tile, and
// the memory is the limit by far.  float32: CUDA cores.
#include <cuda.h>
#include <math.h>

#include "pages.cuh"
#include "tc_common.cuh"

namespace hga {
namespace pages {

using namespace tc;

namespace {

constexpr int kTile = 64;              // tokens per tile
constexpr int kRows = 16;              // most query rows of a pair
constexpr int kConsumers = 128;        // threads of the four computing warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kErrArg = -1;

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
  int page, max_seqs, max_pages, n_pages, layer;
  int64_t page_elems;                  // elements between pages of the layer
  const void* k_pool;                  // of the layer
  const void* v_pool;
  float c2;                            // scale * log2(e)
  uint64_t wait_ns;
};

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Tokens of query i (0 for a bad row or length: recorded).
__device__ __forceinline__ int tokens_of(const Args& a, int i) {
  const int r = a.rows[i];
  int L = r >= 0 && r < a.max_seqs ? a.seq_len[r] : -1;
  if (L < 0 || (int64_t)L > (int64_t)a.max_pages * a.page) {
    set_status(a.status, kErrArg);
    L = 0;
  }
  return L;
}

struct Range {
  int64_t total, begin, end, first;    // tiles of all, of this CTA; first tile of the query at `begin`
  int n_cta, query;
};

__device__ __forceinline__ int64_t cta_of(int64_t w, int64_t total, int64_t n) { return ((w + 1) * n - 1) / total; }

// Finds this CTA's range.  Every thread of the block calls it (kThreads of them).
template <int kThreads>
__device__ __forceinline__ void find_range(const Args& a, Range* out, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
  const int pairs = a.Hkv * a.subs;
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += (int64_t)((tokens_of(a, i) + kTile - 1) / kTile) * pairs;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int64_t base = x - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += sums[w];
    total += sums[w];
  }
  const int64_t n_cta = min((int64_t)gridDim.x, total);
  if (tid == 0) {
    out->total = total;
    out->n_cta = (int)n_cta;
    out->begin = out->end = 0;
    if (blockIdx.x < n_cta) {
      out->begin = blockIdx.x * total / n_cta;
      out->end = (blockIdx.x + 1) * total / n_cta;
    }
  }
  if (blockIdx.x < n_cta) {
    const int64_t begin = blockIdx.x * total / n_cta;
    if (begin >= base && begin < base + mine) {
      int64_t at = base;
      for (int i = i0; i < i1; ++i) {
        const int64_t t = (int64_t)((tokens_of(a, i) + kTile - 1) / kTile) * pairs;
        if (begin < at + t) {
          out->query = i;
          out->first = at;
          break;
        }
        at += t;
      }
    }
  }
  __syncthreads();
}

// One segment: tiles [t0, t1) of pair `pair` (of nt tiles each) of query i, whose tiles start at
// list position `first`.
struct Segment {
  int i, row, L, nt, pair, t0, t1;
  int64_t pair_first;                  // list position of the pair's first tile
};
// The segment at list position w; *i, *first move on to its query.
__device__ __forceinline__ Segment segment_at(const Args& a, const Range& r, int64_t w, int* i, int64_t* first) {
  const int pairs = a.Hkv * a.subs;
  Segment s;
  for (;;) {
    s.L = tokens_of(a, *i);
    s.nt = (s.L + kTile - 1) / kTile;
    const int64_t t = (int64_t)s.nt * pairs;
    if (w < *first + t) break;
    *first += t;
    ++*i;
  }
  s.i = *i;
  s.row = a.rows[s.i];
  const int64_t x = w - *first;
  s.pair = (int)(x / s.nt);
  s.t0 = (int)(x - (int64_t)s.pair * s.nt);
  s.t1 = (int)min((int64_t)s.nt, s.t0 + (r.end - w));
  s.pair_first = *first + (int64_t)s.pair * s.nt;
  return s;
}

// Query head of row r of a pair, or -1.
__device__ __forceinline__ int head_of(const Args& a, int pair, int r) {
  const int kh = pair / a.subs, x = (pair - kh * a.subs) * kRows + r;
  return x < a.G ? kh * a.G + x : -1;
}

// One row's final 4 dims and, once, its lse.
template <typename T>
__device__ __forceinline__ void emit(const Args& a, const Segment& s, int r, int c4, float4 v, float m, float l) {
  const int h = head_of(a, s.pair, r);
  if (h < 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;          // (0: every token was left out)
  v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
  store4(static_cast<T*>(a.o) + ((int64_t)s.i * a.Hq + h) * kD + 4 * c4, v);
  if (c4 == 0) a.lse[(int64_t)s.i * a.Hq + h] = (m + log2f(l)) * 0.6931471805599453f;
}

// After a CTA's part of a split pair is in the workspace: the last CTA to get here adds the parts up.
// `flag`: an int in shared memory.  Called by the 128 consumer threads.
template <typename T>
__device__ __forceinline__ void join(const Args& a, const Segment& s, const Range& r, int* flag) {
  const int64_t c0 = cta_of(s.pair_first, r.total, r.n_cta), c1 = cta_of(s.pair_first + s.nt - 1, r.total, r.n_cta);
  const int n = (int)(c1 - c0 + 1);
  __threadfence();
  consumer_sync();
  if (threadIdx.x == 0) {
    const int before = atomicAdd(&a.counters[c0], 1);
    *flag = before == n - 1;
    if (before == n - 1) a.counters[c0] = 0;
  }
  consumer_sync();
  if (!*flag) return;
  __threadfence();
  const int lane = threadIdx.x & 31;
  auto part = [&](int p) -> const Part* { return a.parts + (p == 0 ? 2 * c0 + 1 : 2 * (c0 + p)); };
  for (int row = threadIdx.x >> 5; row < kRows; row += kConsumers / 32) {
    if (head_of(a, s.pair, row) < 0) continue;
    float m = -INFINITY;
    for (int p = lane; p < n; p += 32) m = fmaxf(m, __ldcg(&part(p)->m[row]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const Part* x = part(p);
      const float f = exp2f(__ldcg(&x->m[row]) - ref);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(x->o + row * kD) + lane);
      l += f * __ldcg(&x->l[row]);
      acc.x += f * v.x; acc.y += f * v.y; acc.z += f * v.z; acc.w += f * v.w;
    }
    emit<T>(a, s, row, lane, acc, m, l);
  }
}

// Queries without tokens: zeros and -inf.  Spread over the CTAs.
template <typename T>
__device__ __forceinline__ void emit_empty(const Args& a, int threads) {
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    if (tokens_of(a, i) != 0) continue;
    for (int x = threadIdx.x; x < a.Hq * (kD / 4); x += threads)
      store4(static_cast<T*>(a.o) + (int64_t)i * a.Hq * kD + 4 * x, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = threadIdx.x; h < a.Hq; h += threads) a.lse[(int64_t)i * a.Hq + h] = -INFINITY;
  }
}

// ------------------------------------------------------------------------------------ bf16, tensor cores
constexpr int kStages = 3;
constexpr uint32_t kTileBytes = kTile * kD * 2;      // 16 KB of K, 16 KB of V
constexpr int kMmaThreads = kConsumers + 32;

struct MmaSmem {
  unsigned char kv[kStages][2][kTileBytes];          // 1 KB aligned (128-byte swizzle)
  float merge[4][8][kD];                             // the four warps' outputs, eight rows at a time
  float m[4][kRows], l[4][kRows];
  uint64_t full[kStages], empty[kStages];
  int64_t sums[kMmaThreads / 32];
  Range range;
  uint32_t valid[kStages];                           // pages of the tile that were loaded, one bit each
  int abort, flag;
};
static_assert(2 * (sizeof(MmaSmem) + 1024) <= 228 * 1024, "two CTAs per SM");

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
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int32_t row, int32_t head,
                                            int32_t page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// RH: 1 when a pair has at most 8 query rows (the upper half of the m16 tile is empty), else 2.
template <int RH>
__global__ void __launch_bounds__(kMmaThreads, 2)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  MmaSmem& s = *reinterpret_cast<MmaSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto full = [&](int i) { return smem_u32(&s.full[i]); };
  auto empty = [&](int i) { return smem_u32(&s.empty[i]); };
  volatile int* abort_flag = &s.abort;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 4);
    }
    s.abort = 0;
    mbar_fence_init();
  }
  pdl_wait();
  find_range<kMmaThreads>(a, &s.range, s.sums);        // (its barriers also publish the mbarriers)
  emit_empty<__nv_bfloat16>(a, kMmaThreads);
  const Range rg = s.range;
  if (rg.begin == rg.end) return;

  const int R = min(a.page, kTile);                    // tokens per box
  const int boxes = kTile / R;                         // boxes of a tile
  int qi = rg.query;
  int64_t first = rg.first;
  if (warp == 4) {
    // ======================= producer: the tiles of this CTA's segments, one after another
    const uint64_t kv0 = smem_u32(&s.kv[0][0][0]);
    int64_t J = 0;
    bool ok = true;
    for (int64_t w = rg.begin; ok && w < rg.end;) {
      const Segment sg = segment_at(a, rg, w, &qi, &first);
      w += sg.t1 - sg.t0;
      const int32_t* ids = a.table + (int64_t)sg.row * a.max_pages;
      const int kh = sg.pair / a.subs;
      // box b of the segment: tokens (t0 * boxes + b) * R ..; lane l holds the pages of 32 boxes at a time
      const int b_end = min(sg.t1 * boxes, (sg.L + R - 1) / R);
      int b0 = sg.t0 * boxes;
      auto page_of = [&](int b) { return b < b_end ? ids[(int64_t)b * R / a.page] : -1; };
      int32_t cur = page_of(b0 + lane), nxt = page_of(b0 + 32 + lane);
      for (int t = sg.t0; t < sg.t1; ++t, ++J) {
        const int st = (int)(J % kStages);
        if (t * boxes >= b0 + 32) {
          b0 += 32;
          cur = nxt;
          nxt = page_of(b0 + 32 + lane);
        }
        const int b = t * boxes + lane;                // this lane's box of the tile
        const int32_t id = __shfl_sync(0xffffffffu, cur, (t * boxes - b0 + lane) & 31);
        const bool have = lane < boxes && b < b_end, good = have && id >= 0 && id < a.n_pages;
        if (have && !good) set_status(a.status, kErrArg);
        const uint32_t mask = __ballot_sync(0xffffffffu, good);
        int go = 1;
        if (lane == 0) {
          go = mbar_wait(empty(st), (uint32_t)((J / kStages) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
          if (go) {
            s.valid[st] = mask;
            mbar_arrive_expect_tx(full(st), (uint32_t)__popc(mask) * R * kD * 2 * 2);
          }
        }
        ok = __shfl_sync(0xffffffffu, go, 0) != 0;
        if (!ok) break;
        if (good) {
          const uint32_t dst = (uint32_t)kv0 + st * 2 * kTileBytes + lane * R * (kD * 2);
          const int row = (int)((int64_t)b * R % a.page);
          tma_load_5d(dst, &tm_k, row, kh, id, full(st));
          tma_load_5d(dst + kTileBytes, &tm_v, row, kh, id, full(st));
        }
        __syncwarp();
      }
    }
    // its loads have landed before the CTA may exit
    if (lane == 0)
      for (int64_t j = J > kStages ? J - kStages : 0; j < J; ++j)
        drain_wait(full((int)(j % kStages)), (uint32_t)((j / kStages) & 1), a.status);
    return;
  }

  // ======================= the four computing warps: keys 16 warp .. + 15 of each tile
  const int g = lane >> 2, tq = lane & 3;              // fragment row and column pair
  const int key0 = 16 * warp;
  int64_t J = 0;
  bool alive = true;                                   // no wait has expired
  for (int64_t w = rg.begin; w < rg.end;) {
    const Segment sg = segment_at(a, rg, w, &qi, &first);
    w += sg.t1 - sg.t0;
    // queries: rows g and g + 8, dims 16 ks + 2 tq + {0, 1} and + 8
    uint32_t qf[8][4];
    {
      const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + sg.i * a.q_stride_n + 2 * tq;
      const int h0 = head_of(a, sg.pair, g), h1 = RH == 2 ? head_of(a, sg.pair, g + 8) : -1;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const __nv_bfloat16 *p0 = qb + (int64_t)h0 * kD + 16 * ks, *p1 = qb + (int64_t)h1 * kD + 16 * ks;
        qf[ks][0] = h0 >= 0 ? *reinterpret_cast<const uint32_t*>(p0) : 0u;
        qf[ks][2] = h0 >= 0 ? *reinterpret_cast<const uint32_t*>(p0 + 8) : 0u;
        qf[ks][1] = h1 >= 0 ? *reinterpret_cast<const uint32_t*>(p1) : 0u;
        qf[ks][3] = h1 >= 0 ? *reinterpret_cast<const uint32_t*>(p1 + 8) : 0u;
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

    for (int t = sg.t0; t < sg.t1; ++t, ++J) {
      const int st = (int)(J % kStages);
      alive = alive && mbar_wait_w(full(st), (uint32_t)((J / kStages) & 1), abort_flag, a.status, a.wait_ns);
      const int nvalid = min(kTile, sg.L - t * kTile) - key0;      // of this warp's 16 keys
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
        uint32_t pf[4] = {0u, 0u, 0u, 0u};
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
          pf[x] = pack_bf16(p0, p1);
          pf[2 + x] = pack_bf16(p2, p3);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i][0] *= alpha[0]; o[i][1] *= alpha[0];
            if (RH == 2) { o[i][2] *= alpha[1]; o[i][3] *= alpha[1]; }
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
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }

    // ---- the four warps' statistics and outputs meet
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (tq == 0) {
        s.m[warp][g + 8 * x] = m[x];
        s.l[warp][g + 8 * x] = l[x];
      }
    }
    const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
    Part* part = a.parts + 2 * (int64_t)blockIdx.x + (sg.t0 == 0 ? 1 : 0);
    consumer_sync();
#pragma unroll
    for (int x = 0; x < RH; ++x) {
      const int row = g + 8 * x;
      const float mt = fmaxf(fmaxf(s.m[0][row], s.m[1][row]), fmaxf(s.m[2][row], s.m[3][row]));
      const float f = mt == -INFINITY ? 0.f : ex2(m[x] - mt);
      if (x) consumer_sync();                          // the first eight rows have been read
#pragma unroll
      for (int i = 0; i < 16; ++i)                     // (columns permuted by row: no bank conflicts)
        *reinterpret_cast<float2*>(&s.merge[warp][g][(8 * i + 2 * tq) ^ ((g & 3) << 3)]) =
            make_float2(o[i][2 * x] * f, o[i][2 * x + 1] * f);
      consumer_sync();
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int z = tid + 128 * y, rr = z >> 5, c4 = z & 31, rw = rr + 8 * x;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) mm = fmaxf(mm, s.m[k][rw]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 u = *reinterpret_cast<const float4*>(&s.merge[k][rr][(4 * c4) ^ ((rr & 3) << 3)]);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
          ll += mm == -INFINITY ? 0.f : s.l[k][rw] * ex2(s.m[k][rw] - mm);
        }
        if (whole) {
          emit<__nv_bfloat16>(a, sg, rw, c4, v, mm, ll);
        } else {
          __stcg(reinterpret_cast<float4*>(part->o + rw * kD) + c4, v);
          if (c4 == 0) {
            __stcg(&part->m[rw], mm);
            __stcg(&part->l[rw], ll);
          }
        }
      }
    }
    if (!whole) join<__nv_bfloat16>(a, sg, rg, &s.flag);
    consumer_sync();                                   // s.m, s.l, s.flag are free again
  }
}

// ------------------------------------------------------------------------------------ CUDA cores
struct SimtSmem {
  float k[kTile][kD + 4];
  float v[kTile][kD];
  float q[kRows][kD];
  float p[kRows][kTile];
  float m[kRows], l[kRows], alpha[kRows];
  int64_t sums[kConsumers / 32];
  Range range;
  int flag;
};

template <typename T>
__global__ void __launch_bounds__(kConsumers) paged_simt_kernel(const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SimtSmem& s = *reinterpret_cast<SimtSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int N = Vec16<T>::N, LPR = kD / N;
  pdl_trigger();
  pdl_wait();
  find_range<kConsumers>(a, &s.range, s.sums);
  emit_empty<T>(a, kConsumers);
  const Range rg = s.range;
  int qi = rg.query;
  int64_t first = rg.first;
  for (int64_t w = rg.begin; w < rg.end;) {
    const Segment sg = segment_at(a, rg, w, &qi, &first);
    w += sg.t1 - sg.t0;
    const int kh = sg.pair / a.subs;
    const int n_rows = min(kRows, a.G - (sg.pair - kh * a.subs) * kRows);
    __syncthreads();
    for (int x = tid; x < kRows * (kD / 4); x += kConsumers) {
      const int r = x / (kD / 4), c = x % (kD / 4), h = head_of(a, sg.pair, r);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (h >= 0) v = load4(static_cast<const T*>(a.q) + sg.i * a.q_stride_n + (int64_t)h * kD + 4 * c);
      v.x *= a.c2; v.y *= a.c2; v.z *= a.c2; v.w *= a.c2;
      store4(&s.q[r][4 * c], v);
    }
    if (tid < kRows) { s.m[tid] = -INFINITY; s.l[tid] = 0.f; }
    float acc[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) acc[r] = 0.f;
    for (int t = sg.t0; t < sg.t1; ++t) {
      const int nv = min(kTile, sg.L - t * kTile);
      __syncthreads();
      for (int x = tid; x < kTile * LPR; x += kConsumers) {
        const int key = x / LPR, c = (x % LPR) * N;
        const int64_t pos = (int64_t)t * kTile + key;
        float kf[N], vf[N];
#pragma unroll
        for (int e = 0; e < N; ++e) kf[e] = vf[e] = 0.f;
        if (key < nv) {
          const int id = a.table[(int64_t)sg.row * a.max_pages + pos / a.page];
          if (id >= 0 && id < a.n_pages) {
            const int64_t off = id * a.page_elems + ((int64_t)kh * a.page + pos % a.page) * kD + c;
            Vec16<T>::load(static_cast<const T*>(a.k_pool) + off, kf);
            Vec16<T>::load(static_cast<const T*>(a.v_pool) + off, vf);
          } else {
            set_status(a.status, kErrArg);
            kf[0] = NAN;                               // marks the token as left out
          }
        }
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          store4(&s.k[key][c + e], make_float4(kf[e], kf[e + 1], kf[e + 2], kf[e + 3]));
          store4(&s.v[key][c + e], make_float4(vf[e], vf[e + 1], vf[e + 2], vf[e + 3]));
        }
      }
      __syncthreads();
      {
        // scores: thread = key, half of the rows
        const int key = tid & 63, r0 = (tid >> 6) * 8;
        const int id = key < nv ? a.table[(int64_t)sg.row * a.max_pages + ((int64_t)t * kTile + key) / a.page] : -1;
        const bool in = id >= 0 && id < a.n_pages;
        float d[8] = {};
        if (r0 < n_rows)
          for (int c = 0; c < kD; c += 4) {
            const float4 kv = *reinterpret_cast<const float4*>(&s.k[key][c]);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const float4 qv = *reinterpret_cast<const float4*>(&s.q[r0 + r][c]);
              d[r] += kv.x * qv.x + kv.y * qv.y + kv.z * qv.z + kv.w * qv.w;
            }
          }
#pragma unroll
        for (int r = 0; r < 8; ++r) s.p[r0 + r][key] = in ? d[r] : -INFINITY;
      }
      __syncthreads();
      for (int r = warp; r < n_rows; r += 4) {
        const float x0 = s.p[r][lane], x1 = s.p[r][lane + 32];
        float mx = fmaxf(x0, x1);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mo = s.m[r], mnew = fmaxf(mo, mx), ref = mnew == -INFINITY ? 0.f : mnew;
        const float p0 = exp2f(x0 - ref), p1 = exp2f(x1 - ref);
        float sum = p0 + p1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s.p[r][lane] = p0;
        s.p[r][lane + 32] = p1;
        __syncwarp();
        if (lane == 0) {
          const float al = exp2f(mo - ref);
          s.alpha[r] = al;
          s.m[r] = mnew;
          s.l[r] = s.l[r] * al + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (r < n_rows) acc[r] *= s.alpha[r];
      for (int key = 0; key < nv; key += 4) {          // (keys past nv: p = 0, v = 0)
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s.v[key + e][tid];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < n_rows) {
            const float4 p = *reinterpret_cast<const float4*>(&s.p[r][key]);
            acc[r] += p.x * v[0] + p.y * v[1] + p.z * v[2] + p.w * v[3];
          }
      }
    }
    // outputs through the K area, four dims per thread
    __syncthreads();
    const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
    Part* part = a.parts + 2 * (int64_t)blockIdx.x + (sg.t0 == 0 ? 1 : 0);
    float* buf = &s.v[0][0];
#pragma unroll
    for (int r = 0; r < kRows; ++r) buf[r * kD + tid] = acc[r];
    __syncthreads();
    for (int r = warp; r < n_rows; r += 4) {
      const float4 v = *reinterpret_cast<const float4*>(&buf[r * kD + 4 * lane]);
      if (whole) {
        emit<T>(a, sg, r, lane, v, s.m[r], s.l[r]);
      } else {
        __stcg(reinterpret_cast<float4*>(part->o + r * kD) + lane, v);
        if (lane == 0) {
          __stcg(&part->m[r], s.m[r]);
          __stcg(&part->l[r], s.l[r]);
        }
      }
    }
    if (!whole) join<T>(a, sg, rg, &s.flag);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A layer's pool as {64 dims, page tokens, 2 halves, KV heads, pages}; a box is one page's (at most 64)
// tokens of one head, its two 64-dim halves one after the other.
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
  const cuuint64_t row = kD * 2;
  cuuint64_t dims[5] = {64, (cuuint64_t)c.page, 2, (cuuint64_t)c.Hkv, (cuuint64_t)c.n_pages};
  cuuint64_t strides[4] = {row, 128, row * c.page, (cuuint64_t)c.page_bytes};
  cuuint32_t box[5] = {64, (cuuint32_t)(c.page < kTile ? c.page : kTile), 2, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  a.page_elems = c.page_bytes / c.elem;
  a.k_pool = static_cast<const char*>(k_pool) + layer * c.layer_bytes;
  a.v_pool = static_cast<const char*>(v_pool) + layer * c.layer_bytes;
  a.c2 = scale * kLog2e;
  a.wait_ns = wait_ns;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles there can be
  const int64_t tiles = (int64_t)n * c.Hkv * a.subs * (((int64_t)c.max_pages * c.page + kTile - 1) / kTile);
  auto grid_of = [&](int per_sm) {
    int64_t g = (int64_t)sms * per_sm;
    if (g > kMaxCtas) g = kMaxCtas;
    return dim3((unsigned)(g < tiles ? g : tiles));
  };
  if (bf16) {
    CUtensorMap mk, mv;
    if (!make_pool_map(&mk, a.k_pool, c) || !make_pool_map(&mv, a.v_pool, c)) return cudaErrorInvalidValue;
    auto kernel = a.G <= 8 ? paged_mma_kernel<1> : paged_mma_kernel<2>;
    const size_t smem = sizeof(MmaSmem);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, grid_of(2), dim3(kMmaThreads), smem, st, 1, mk, mv, a);
  }
  auto kernel = paged_simt_kernel<float>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SimtSmem));
  if (e != cudaSuccess) return e;
  static_assert(2 * (sizeof(SimtSmem) + 1024) <= 228 * 1024, "two CTAs per SM");
  return launch_dependent(kernel, grid_of(2), dim3(kConsumers), sizeof(SimtSmem), st, 1, a);
}

}  // namespace pages
}  // namespace hga
