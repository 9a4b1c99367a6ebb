// Page moves of a paged K/V cache: reserve and write new tokens, fork, free, compact, copy.
//
// The integers (page table, lengths, reference counts) are changed by one CTA per call, which first
// checks the whole list and then changes all or nothing; the K/V bytes move in a grid-wide kernel
// behind it that reads the list of page pairs it left in the workspace (dependent launch: the second
// kernel is resident before the first has finished).  The single CTA is bound by the latency of a few
// dependent passes over lists that sit in L2; the moves by HBM: compacting a half-used pool of 4096
// pages of 64 tokens in two layers takes 174 us, 6.2 TB/s.
#include "pages.cuh"

namespace hga {
namespace pages {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kErrArg = -1, kErrPages = -8;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Inclusive prefix sum over the CTA (1024 threads), and the total.  `sums` holds 33 ints.
__device__ __forceinline__ int block_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // the previous scan's sums have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sums[lane] = w;
  }
  __syncthreads();
  *total = sums[31];
  return x + (warp ? sums[warp - 1] : 0);
}

// The ids in [begin, end) for which want(ref) holds, in ascending order, into out[0 .. limit): stops
// after the step that has found `limit`.  Returns how many were written.
template <typename Want>
__device__ __forceinline__ int collect(const int32_t* ref, int begin, int end, int limit, int32_t* out, int* sums,
                                       Want want) {
  int found = 0;
  for (int base = begin; base < end && found < limit; base += 4 * kPlanThreads) {
    const int i0 = base + 4 * (int)threadIdx.x;
    int hit[4], n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hit[e] = i0 + e < end && want(ref[i0 + e]);
      n += hit[e];
    }
    int total;
    int at = found + block_scan(n, sums, &total) - n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (hit[e]) {
        if (at < limit) out[at] = i0 + e;
        ++at;
      }
    found += total;
  }
  return min(found, limit);
}

struct PlanSmem {
  uint32_t seen[kMaxSeqs / 32];          // sequence rows already in the list
  int32_t off[kMaxSeqs];                 // first of each entry's pages among the free ones
  int sums[33];
  int bad;
};

__device__ __forceinline__ void plan_init(PlanSmem& s) {
  for (int i = threadIdx.x; i < kMaxSeqs / 32; i += kPlanThreads) s.seen[i] = 0;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
}
// Marks row r; false when it is outside the cache or already marked.
__device__ __forceinline__ bool mark_row(PlanSmem& s, const Cache& c, int r) {
  if (r < 0 || r >= c.max_seqs) return false;
  return !(atomicOr(&s.seen[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u);
}
// The valid length of row r, or -1.
__device__ __forceinline__ int length_of(const Cache& c, int r) {
  if (r < 0 || r >= c.max_seqs) return -1;
  const int L = c.seq_len[r];
  return L < 0 || (int64_t)L > (int64_t)c.max_pages * c.page ? -1 : L;
}

// ------------------------------------------------------------------------------------ reserve
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const Cache c, const Scratch sc, int n,
                                                               const int32_t* rows, const int32_t* add,
                                                               int32_t* pos) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PlanSmem& s = *reinterpret_cast<PlanSmem*>(smem_raw);
  pdl_trigger();
  plan_init(s);
  pdl_wait();
  // the pages each entry needs, in order
  int need = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    int x = 0;
    if (i < n) {
      const int r = rows[i], a = add[i], L = length_of(c, r);
      if (!mark_row(s, c, r) || L < 0 || a < 0 || (int64_t)L + a > (int64_t)c.max_pages * c.page) s.bad = 1;
      else x = ceil_div(L + a, c.page) - ceil_div(L, c.page);
      // an entry beyond the pool cannot be met, and must not overflow the sum
      x = min(x, c.n_pages + 1);
    }
    int total;
    const int inc = block_scan(x, s.sums, &total);
    if (i < n) s.off[i] = need + inc - x;
    need = (int)min((int64_t)need + total, (int64_t)1 << 30);      // (more than any pool has; a step adds up to 2^30 + 1024)
  }
  __syncthreads();
  int err = s.bad ? kErrArg : need > c.n_pages ? kErrPages : 0;
  if (!err && collect(c.ref, 0, c.n_pages, need, sc.dst, s.sums, [](int x) { return x == 0; }) < need) err = kErrPages;
  __syncthreads();                       // the free pages found are visible to the CTA
  if (err) {
    for (int i = threadIdx.x; i < n; i += kPlanThreads) pos[i] = -1;
    if (threadIdx.x == 0) set_status(c.status, err);
    return;
  }
  // a warp per entry deals out its pages
  for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
    const int r = rows[i], L = c.seq_len[r], end = L + add[i];
    const int c0 = ceil_div(L, c.page), k = ceil_div(end, c.page) - c0;
    for (int j = threadIdx.x & 31; j < k; j += 32) {
      const int id = sc.dst[s.off[i] + j];
      c.table[(int64_t)r * c.max_pages + c0 + j] = id;
      c.ref[id] = 1;
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      pos[i] = L;
      c.seq_len[r] = end;
    }
  }
}

// ------------------------------------------------------------------------------------ write
constexpr int kWriteThreads = 256;
constexpr int kWriteTokens = 16;         // most tokens per CTA

struct WriteArgs {
  const int32_t* rows;
  const int32_t* pos;
  const int32_t* cu_new;
  const char* k_new;
  const char* v_new;
  char* k_pool;                          // of the layer
  char* v_pool;
  int64_t total, k_t, k_h, v_t, v_h;     // strides in bytes
  int n, tokens;
};

// A CTA takes `tokens` new tokens: one thread of each finds where it goes, then all move 16-byte pieces.
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const Cache c, const WriteArgs a) {
  __shared__ int64_t dst[kWriteTokens];  // byte offset of the token's row of KV head 0; -1: left out
  pdl_trigger();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  if (threadIdx.x < a.tokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t to = -1;
    if (t < a.total && a.cu_new[0] <= t && t < a.cu_new[a.n]) {
      int lo = 0, hi = a.n - 1;          // the last entry with cu_new[entry] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_new[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int r = a.rows[lo], first = a.pos[lo];
      if (first >= 0) {
        const int64_t p = first + (t - a.cu_new[lo]);
        const int L = length_of(c, r);
        int id = -1;
        if (p < L) id = c.table[(int64_t)r * c.max_pages + p / c.page];
        if (id >= 0 && id < c.n_pages) to = id * c.page_bytes + (p % c.page) * (int64_t)(kD * c.elem);
        else set_status(c.status, kErrArg);
      }
    }
    dst[threadIdx.x] = to;
  }
  // rows that the list promises and no thread finds (it decreases, or ends past the rows there are) are recorded by one CTA
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.n; i += kWriteThreads)
      if (a.cu_new[i] < (i ? a.cu_new[i - 1] : 0) || a.cu_new[i] > a.total) set_status(c.status, kErrArg);
  __syncthreads();
  const int vecs = kD * c.elem / 16;     // 16-byte pieces of a row
  const int per_token = c.Hkv * vecs;
  const int64_t head_bytes = (int64_t)c.page * kD * c.elem;
  const int m = a.tokens * per_token;
  for (int i = threadIdx.x; i < m; i += kWriteThreads) {
    const int tok = i / per_token, x = i - tok * per_token, h = x / vecs, e = x - h * vecs;
    const int64_t to = dst[tok];
    if (to < 0) continue;
    const int64_t off = to + h * head_bytes + e * 16, t = t0 + tok;
    const uint4 k = *reinterpret_cast<const uint4*>(a.k_new + t * a.k_t + h * a.k_h + e * 16);
    const uint4 v = *reinterpret_cast<const uint4*>(a.v_new + t * a.v_t + h * a.v_h + e * 16);
    *reinterpret_cast<uint4*>(a.k_pool + off) = k;
    *reinterpret_cast<uint4*>(a.v_pool + off) = v;
  }
}

// ------------------------------------------------------------------------------------ moving pages
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;
constexpr int64_t kMoveChunk = (int64_t)kMoveThreads * kMoveUnroll * 16;   // 32 KB: a CTA's piece

// Copies the pages of the list (counts[0] pairs) in every layer of both pools; with `remap`, the page
// tables follow the compaction's map.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Cache c, const Scratch sc, char* k_pool,
                                                            char* v_pool, int remap) {
  pdl_trigger();
  pdl_wait();
  const int n = sc.counts[0];
  if (n == 0) return;
  const int chunks = (int)((c.page_data + kMoveChunk - 1) / kMoveChunk);
  const int64_t items = (int64_t)n * c.n_layers * 2 * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    int64_t x = it;
    const int ch = (int)(x % chunks);
    x /= chunks;
    char* pool = (x & 1) ? v_pool : k_pool;
    x >>= 1;
    const int layer = (int)(x % c.n_layers), pair = (int)(x / c.n_layers);
    char* base = pool + layer * c.layer_bytes + ch * kMoveChunk;
    const char* from = base + sc.src[pair] * c.page_bytes;
    char* to = base + sc.dst[pair] * c.page_bytes;
    const int64_t left = c.page_data - ch * kMoveChunk;
    uint4 v[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int64_t o = ((int64_t)i * kMoveThreads + threadIdx.x) * 16;
      if (o < left) v[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
    }
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int64_t o = ((int64_t)i * kMoveThreads + threadIdx.x) * 16;
      if (o < left) __stcs(reinterpret_cast<uint4*>(to + o), v[i]);
    }
  }
  if (remap) {
    const int n_used = sc.counts[1];
    const int64_t cells = (int64_t)c.max_seqs * c.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < cells; i += (int64_t)gridDim.x * kMoveThreads) {
      const int r = (int)(i / c.max_pages), col = (int)(i - (int64_t)r * c.max_pages);
      const int L = length_of(c, r);
      if (L < 0) {
        if (col == 0) set_status(c.status, kErrArg);
        continue;
      }
      if (col >= ceil_div(L, c.page)) continue;
      const int id = c.table[i];
      if (id < 0 || id >= c.n_pages) set_status(c.status, kErrArg);
      else if (id >= n_used && sc.to[id] >= 0) c.table[i] = sc.to[id];
    }
  }
}

// ------------------------------------------------------------------------------------ fork
__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const Cache c, const Scratch sc, int n, const int32_t* src,
                                                            const int32_t* dst) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PlanSmem& s = *reinterpret_cast<PlanSmem*>(smem_raw);
  pdl_trigger();
  plan_init(s);
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (!mark_row(s, c, dst[i]) || c.seq_len[dst[i]] != 0) s.bad = 1;
  __syncthreads();
  int need = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    int x = 0;
    if (i < n) {
      const int r = src[i], L = length_of(c, r);
      if (L < 0 || (s.seen[r >> 5] >> (r & 31) & 1u)) s.bad = 1;
      else x = L % c.page != 0;
    }
    int total;
    const int inc = block_scan(x, s.sums, &total);
    if (i < n) s.off[i] = need + inc - x;
    need += total;
  }
  // every page of a source must be a page of the pool
  for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
    const int r = src[i], L = length_of(c, r);
    const int k = L < 0 ? 0 : ceil_div(L, c.page);
    for (int j = threadIdx.x & 31; j < k; j += 32) {
      const int id = c.table[(int64_t)r * c.max_pages + j];
      if (id < 0 || id >= c.n_pages) s.bad = 1;
    }
  }
  __syncthreads();
  int err = s.bad ? kErrArg : need > c.n_pages ? kErrPages : 0;
  if (!err && collect(c.ref, 0, c.n_pages, need, sc.dst, s.sums, [](int x) { return x == 0; }) < need) err = kErrPages;
  __syncthreads();
  if (threadIdx.x == 0) sc.counts[0] = err ? 0 : need;
  if (err) {
    if (threadIdx.x == 0) set_status(c.status, err);
    return;
  }
  for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
    const int rs = src[i], rd = dst[i], L = c.seq_len[rs], full = L / c.page;
    const int32_t* from = c.table + (int64_t)rs * c.max_pages;
    int32_t* to = c.table + (int64_t)rd * c.max_pages;
    for (int j = threadIdx.x & 31; j < full; j += 32) {
      const int id = from[j];
      to[j] = id;
      atomicAdd(&c.ref[id], 1);
    }
    if ((threadIdx.x & 31) == 0) {
      if (L % c.page) {
        const int id = sc.dst[s.off[i]];
        to[full] = id;
        c.ref[id] = 1;
        sc.src[s.off[i]] = from[full];
      }
      c.seq_len[rd] = L;
    }
  }
}

// ------------------------------------------------------------------------------------ free
__global__ void __launch_bounds__(kPlanThreads) free_kernel(const Cache c, int n, const int32_t* rows) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PlanSmem& s = *reinterpret_cast<PlanSmem*>(smem_raw);
  pdl_trigger();
  plan_init(s);
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (!mark_row(s, c, rows[i]) || length_of(c, rows[i]) < 0) s.bad = 1;
  __syncthreads();
  if (!s.bad) {
    for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
      const int r = rows[i], k = ceil_div(c.seq_len[r], c.page);
      for (int j = threadIdx.x & 31; j < k; j += 32) {
        const int id = c.table[(int64_t)r * c.max_pages + j];
        if (id < 0 || id >= c.n_pages) s.bad = 1;
      }
    }
  }
  __syncthreads();
  if (s.bad) {
    if (threadIdx.x == 0) set_status(c.status, kErrArg);
    return;
  }
  for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
    const int r = rows[i], k = ceil_div(c.seq_len[r], c.page);
    for (int j = threadIdx.x & 31; j < k; j += 32)
      atomicSub(&c.ref[c.table[(int64_t)r * c.max_pages + j]], 1);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) c.seq_len[r] = 0;
  }
}

// ------------------------------------------------------------------------------------ compact
__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const Cache c, const Scratch sc, int32_t* n_used_out) {
  __shared__ int sums[33];
  pdl_trigger();
  pdl_wait();
  int n_used = 0;
  for (int base = 0; base < c.n_pages; base += 4 * kPlanThreads) {
    int x = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = base + 4 * (int)threadIdx.x + e;
      if (i < c.n_pages) x += c.ref[i] > 0;
    }
    int total;
    block_scan(x, sums, &total);
    n_used += total;
  }
  const int holes = collect(c.ref, 0, n_used, n_used, sc.dst, sums, [](int x) { return x <= 0; });
  const int movers = collect(c.ref, n_used, c.n_pages, holes, sc.src, sums, [](int x) { return x > 0; });
  for (int i = n_used + threadIdx.x; i < c.n_pages; i += kPlanThreads) sc.to[i] = -1;
  __syncthreads();                       // as many movers as holes: both are the used pages at or past n_used
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) {
    const int from = sc.src[i], to = sc.dst[i];
    sc.to[from] = to;
    c.ref[to] = c.ref[from];
    c.ref[from] = 0;
  }
  if (threadIdx.x == 0) {
    sc.counts[0] = movers;
    sc.counts[1] = n_used;
    *n_used_out = n_used;
  }
}

// ------------------------------------------------------------------------------------ copy
__global__ void __launch_bounds__(kPlanThreads) copy_list_kernel(const Cache c, const Scratch sc, int n,
                                                                 const int32_t* src, const int32_t* dst) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint32_t* seen = reinterpret_cast<uint32_t*>(smem_raw);      // one bit per page: destinations
  __shared__ int bad;
  pdl_trigger();
  for (int i = threadIdx.x; i < (c.n_pages + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  pdl_wait();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int d = dst[i];
    if (d < 0 || d >= c.n_pages || (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u)) bad = 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int x = src[i];
    if (x < 0 || x >= c.n_pages || (seen[x >> 5] >> (x & 31) & 1u)) bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    sc.counts[0] = bad ? 0 : n;
    if (bad) set_status(c.status, kErrArg);
  }
  if (bad) return;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    sc.src[i] = src[i];
    sc.dst[i] = dst[i];
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// The moves of at most `pairs` page pairs: no more CTAs than pieces of work.
cudaError_t launch_move(const Cache& c, const Scratch& s, int64_t pairs, void* k_pool, void* v_pool, bool remap,
                        cudaStream_t st) {
  const int64_t chunks = (c.page_data + kMoveChunk - 1) / kMoveChunk;
  const int64_t items = pairs * c.n_layers * 2 * chunks, most = 8LL * sm_count();
  const int64_t grid = items < 1 ? 1 : items < most ? items : most;
  return launch_dependent(move_kernel, dim3((unsigned)grid), dim3(kMoveThreads), 0, st, 1, c, s,
                          static_cast<char*>(k_pool), static_cast<char*>(v_pool), remap ? 1 : 0);
}

// One CTA with `smem` bytes, which no call has more than `most` of.  The attribute belongs to the process, not to the call: what
// threads set at the same time must be one value.  (47 KB: what a kernel may have without it, less its static variables.)
template <typename K, typename... A>
cudaError_t launch_one(K kernel, size_t smem, size_t most, cudaStream_t st, A... args) {
  if (smem > 47 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, dim3(1), dim3(kPlanThreads), smem, st, 1, args...);
}

}  // namespace

cudaError_t launch_reserve(const Cache& c, const Scratch& s, int n, const int32_t* rows, const int32_t* add,
                           int32_t* pos, cudaStream_t st) {
  return launch_one(reserve_kernel, sizeof(PlanSmem), sizeof(PlanSmem), st, c, s, n, rows, add, pos);
}

cudaError_t launch_write(const Cache& c, int layer, int n, const int32_t* rows, const int32_t* pos,
                         const int32_t* cu_new, int64_t total, const void* k_new, int64_t k_t, int64_t k_h,
                         const void* v_new, int64_t v_t, int64_t v_h, void* k_pool, void* v_pool, cudaStream_t st) {
  // few tokens: one each, so that they spread over the SMs; many: as many as give four CTAs per SM, up to 16.  64 tokens
  // (with reserve): 9.4 us with one, 12.5 with 16; 16K tokens: 36.4 and 28.6
  int64_t tokens = total / (4LL * sm_count());
  tokens = tokens < 1 ? 1 : tokens > kWriteTokens ? kWriteTokens : tokens;
  WriteArgs a{rows, pos, cu_new, static_cast<const char*>(k_new), static_cast<const char*>(v_new),
              static_cast<char*>(k_pool) + layer * c.layer_bytes, static_cast<char*>(v_pool) + layer * c.layer_bytes,
              total, k_t * c.elem, k_h * c.elem, v_t * c.elem, v_h * c.elem, n, (int)tokens};
  const int64_t grid = (total + tokens - 1) / tokens;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(write_kernel, dim3((unsigned)grid), dim3(kWriteThreads), 0, st, 1, c, a);
}

cudaError_t launch_fork(const Cache& c, const Scratch& s, int n, const int32_t* src, const int32_t* dst, void* k_pool,
                        void* v_pool, cudaStream_t st) {
  cudaError_t e = launch_one(fork_kernel, sizeof(PlanSmem), sizeof(PlanSmem), st, c, s, n, src, dst);
  return e != cudaSuccess ? e : launch_move(c, s, n, k_pool, v_pool, false, st);
}

cudaError_t launch_free(const Cache& c, int n, const int32_t* rows, cudaStream_t st) {
  return launch_one(free_kernel, sizeof(PlanSmem), sizeof(PlanSmem), st, c, n, rows);
}

cudaError_t launch_compact(const Cache& c, const Scratch& s, void* k_pool, void* v_pool, int32_t* n_used,
                           cudaStream_t st) {
  cudaError_t e = launch_dependent(compact_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1, c, s, n_used);
  return e != cudaSuccess ? e : launch_move(c, s, c.n_pages / 2, k_pool, v_pool, true, st);
}

cudaError_t launch_copy(const Cache& c, const Scratch& s, int n, const int32_t* src, const int32_t* dst, void* k_pool,
                        void* v_pool, cudaStream_t st) {
  cudaError_t e = launch_one(copy_list_kernel, (size_t)((c.n_pages + 31) / 32) * 4, kMaxPages / 8, st, c, s, n, src, dst);
  return e != cudaSuccess ? e : launch_move(c, s, n, k_pool, v_pool, false, st);
}

}  // namespace pages
}  // namespace hga
