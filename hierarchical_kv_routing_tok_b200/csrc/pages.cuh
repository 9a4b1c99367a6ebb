// A paged K/V cache as its kernels see it, and the scratch its calls keep in the workspace.
#pragma once

#include "common.cuh"

namespace hga {
namespace pages {

constexpr int kMaxSeqs = 8192;         // sequence rows (one bit and one int32 each in shared memory)
constexpr int kMaxPages = 1 << 20;     // pages (one bit each in shared memory)

struct Cache {
  int n_layers, n_pages, page, Hkv, max_seqs, max_pages;
  int elem;                            // bytes per element
  int64_t layer_bytes, page_bytes;     // strides of the pools
  int64_t page_data;                   // bytes of one page of one layer
  int32_t* table;
  int32_t* seq_len;
  int32_t* ref;
  int* status;
};

// Scratch: counts (n_copy), then the page pairs to copy and the free pages found, then the new page of
// each page of the pool (compaction).
struct Scratch {
  int32_t* counts;                     // [64]
  int32_t* src;                        // [n_pages]
  int32_t* dst;                        // [n_pages]
  int32_t* to;                         // [n_pages]
};

cudaError_t launch_reserve(const Cache& c, const Scratch& s, int n, const int32_t* rows, const int32_t* add,
                           int32_t* pos, cudaStream_t st);
cudaError_t launch_write(const Cache& c, int layer, int n, const int32_t* rows, const int32_t* pos,
                         const int32_t* cu_new, int64_t total, const void* k_new, int64_t k_t, int64_t k_h,
                         const void* v_new, int64_t v_t, int64_t v_h, void* k_pool, void* v_pool, cudaStream_t st);
cudaError_t launch_fork(const Cache& c, const Scratch& s, int n, const int32_t* src, const int32_t* dst, void* k_pool,
                        void* v_pool, cudaStream_t st);
cudaError_t launch_free(const Cache& c, int n, const int32_t* rows, cudaStream_t st);
cudaError_t launch_compact(const Cache& c, const Scratch& s, void* k_pool, void* v_pool, int32_t* n_used,
                           cudaStream_t st);
cudaError_t launch_copy(const Cache& c, const Scratch& s, int n, const int32_t* src, const int32_t* dst, void* k_pool,
                        void* v_pool, cudaStream_t st);

size_t paged_attn_scratch_bytes();
cudaError_t launch_paged_attn(bool bf16, const Cache& c, int layer, int n, int Hq, float scale,
                              const int32_t* rows, const void* q, int64_t q_stride_n, const void* k_pool,
                              const void* v_pool, void* o, float* lse, void* scratch, uint64_t wait_ns,
                              cudaStream_t st);

}  // namespace pages
}  // namespace hga
