// The work lists of a packed batch: cu_seqlens -> the tiles of all sequences, heaviest first.
//
// One CTA per list.  A tile slot i belongs to the sequence s with cu[s] / tile + s <= i < cu[s+1] /
// tile + s + 1 (those ranges hold at least ceil(len / tile) slots each and need no prefix sum), found
// by bisection.  The tiles are placed by a counting sort on their work, so that the kernels behind,
// which deal the list out to the SMs in order, start the long tiles first and end with the short ones.
// The order of tiles of equal work is left to the atomics: no result depends on it.  Few tiles of few sequences need no
// list (own_tile).
// Latency-bound (a few dependent shared-memory passes): 2.5 us.
#include "packed_plan.cuh"

namespace hga {
namespace packed {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;        // work classes
constexpr int kCuSmem = 4096;      // sequence bounds kept in shared memory

struct Args {
  const int32_t* cu;
  int n_seqs;
  int64_t total;
  ListSpec lists[2];
  Header* hdr;
  int* status;
  int clear_status;
  int shift;                       // work class = 128-token units >> shift
};

__global__ void __launch_bounds__(kThreads) plan_kernel(const Args a) {
  __shared__ int32_t s_cu[kCuSmem];
  __shared__ int32_t hist[kBins];
  __shared__ int32_t warp_sum[32];
  __shared__ int bad_flag;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const ListSpec L = a.lists[blockIdx.x];
  // a dependent launch: what it writes may still be read by the kernel before it in the stream
  pdl_wait();
  if (a.clear_status && blockIdx.x == 0 && tid == 0) *a.status = 0;
  if (tid == 0) bad_flag = 0;
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i <= a.n_seqs; i += kThreads) {
    const int32_t c = a.cu[i];
    if (i < kCuSmem) s_cu[i] = c;
    if (i == 0) bad |= c != 0;
    else bad |= c < a.cu[i - 1];
    if (i == a.n_seqs) bad |= c < 0 || (int64_t)c > a.total;
  }
  if (bad) bad_flag = 1;
  __syncthreads();
  if (bad_flag) {
    if (tid == 0) {
      a.hdr->n_tiles[blockIdx.x] = 0;
      if (blockIdx.x == 0) {
        a.hdr->end = 0;
        set_status(a.status, -1);
      }
    }
    return;
  }
  const int32_t* cu = a.n_seqs < kCuSmem ? s_cu : a.cu;
  const int64_t end = cu[a.n_seqs];
  const int64_t n_slots = end / L.tile + a.n_seqs;
  // the tile of slot i, if it has one
  auto tile_at = [&](int64_t i, Tile* t) {
    int lo = 0, hi = a.n_seqs - 1;              // the last s with cu[s] / tile + s <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)(cu[mid] / L.tile) + mid <= i) lo = mid;
      else hi = mid - 1;
    }
    t->start = cu[lo];
    t->len = cu[lo + 1] - cu[lo];
    const int64_t t0 = (i - ((int64_t)(cu[lo] / L.tile) + lo)) * L.tile;
    t->t0 = (int32_t)t0;
    t->pad = 0;
    return t0 < t->len;
  };
  auto bin_of = [&](const Tile& t) {            // class 0 is the heaviest
    const int64_t seen = L.by_key ? (int64_t)t.len - t.t0 : min((int64_t)t.t0 + L.tile, (int64_t)t.len);
    return kBins - 1 - (int)min(((seen - 1) / 128) >> a.shift, (int64_t)(kBins - 1));
  };
  for (int64_t i = tid; i < n_slots; i += kThreads) {
    Tile t;
    if (tile_at(i, &t)) atomicAdd(&hist[bin_of(t)], 1);
  }
  __syncthreads();
  // exclusive prefix sum of the classes: two per thread
  const int h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
  int x = h0 + h1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  const int base = (warp ? warp_sum[warp - 1] : 0) + x - (h0 + h1);
  hist[2 * tid] = base;
  hist[2 * tid + 1] = base + h0;
  if (tid == kThreads - 1) {
    a.hdr->n_tiles[blockIdx.x] = base + h0 + h1;
    if (blockIdx.x == 0) a.hdr->end = (int32_t)end;
  }
  __syncthreads();
  for (int64_t i = tid; i < n_slots; i += kThreads) {
    Tile t;
    if (tile_at(i, &t)) *reinterpret_cast<int4*>(&L.list[atomicAdd(&hist[bin_of(t)], 1)]) =
        make_int4(t.start, t.len, t.t0, 0);
  }
}
static_assert(kBins == 2 * kThreads, "the prefix sum takes two classes per thread");

}  // namespace

cudaError_t launch_plan(const int32_t* cu, int n_seqs, int64_t total, int n_lists, const ListSpec* lists, Header* hdr,
                        int* status, bool clear_status, cudaStream_t st) {
  Args a{};
  a.cu = cu;
  a.n_seqs = n_seqs;
  a.total = total;
  for (int i = 0; i < n_lists; ++i) a.lists[i] = lists[i];
  a.hdr = hdr;
  a.status = status;
  a.clear_status = clear_status;
  a.shift = 0;
  while (((total / 128) >> a.shift) >= kBins) ++a.shift;
  return launch_dependent(plan_kernel, dim3((unsigned)n_lists), dim3(kThreads), 0, st, 1, a);
}

}  // namespace packed
}  // namespace hga
