// C ABI of the dense readout (contract in include/hga.h): causal attention over packed prompts, the
// paged K/V cache and the attention over it.  Validates every argument on the host, then enqueues the
// kernels on the caller's stream.  No allocation, no synchronisation.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "hga.h"
#include "packed_common.cuh"
#include "pages.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_ptrs(std::initializer_list<const void*> ps, uintptr_t align) {
  for (const void* p : ps)
    if (!p) return HGA_ERR_ARG;
  for (const void* p : ps)
    if (!aligned(p, align)) return HGA_ERR_ALIGN;
  return HGA_OK;
}
int check_workspace(const void* ws) {
  if (!ws) return HGA_ERR_WORKSPACE;
  return aligned(ws, 16) ? HGA_OK : HGA_ERR_ALIGN;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? HGA_OK : HGA_ERR_CUDA; }

uint64_t wait_limit(int64_t ns) { return ns > 0 ? (uint64_t)ns : 2000000000ull; }
int elem_bytes(int dtype) { return dtype == HGA_BF16 ? 2 : 4; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
bool bad_scale(float s) { return !(s >= 0.f) || isinf(s * 1.4426950408889634f); }      // (the kernels take scale * log2(e))
float eff_scale(float s) { return s > 0.f ? s : 1.0f / sqrtf((float)hga::kD); }

// A stride of an outer dimension: 0 stands for the contiguous one; else whole 16-byte pieces, at
// least a row (a dimension of one element may have any).
int check_stride(int64_t s, int dtype) {
  if (s == 0) return HGA_OK;
  if (s < hga::kD || s > (int64_t)1 << 37) return HGA_ERR_ARG;
  return s * elem_bytes(dtype) % 16 == 0 ? HGA_OK : HGA_ERR_ALIGN;
}
hga::packed::Strided strided(int64_t t, int64_t h, int H) {
  return {t ? t : (int64_t)H * hga::kD, h ? h : (int64_t)hga::kD};
}

// ---------------------------------------------------------------- packed prompts
int check_packed(const hga_packed_config_t* c) {
  if (!c) return HGA_ERR_ARG;
  if (c->Hq < 1 || c->Hkv < 1 || c->Hq % c->Hkv != 0 || c->n_seqs < 0 || c->total < 0) return HGA_ERR_ARG;
  if (c->dtype != HGA_F32 && c->dtype != HGA_BF16) return HGA_ERR_ARG;
  if (c->D != hga::kD) return HGA_ERR_UNSUPPORTED;
  if (c->flags & ~(HGA_PACKED_FILL_TAIL | HGA_PACKED_CLEAR_STATUS)) return HGA_ERR_ARG;
  if (c->reserved != 0) return HGA_ERR_ARG;
  for (int64_t s : {c->q_stride_t, c->q_stride_h, c->k_stride_t, c->k_stride_h, c->v_stride_t, c->v_stride_h}) {
    const int rc = check_stride(s, c->dtype);
    if (rc) return rc;
  }
  if (bad_scale(c->softmax_scale) || c->wait_limit_ns < 0) return HGA_ERR_ARG;
  // rows are 32-bit tensor-map coordinates, a tile may look past the last one; a CTA per (tile, head)
  if (c->total > (int64_t)INT32_MAX - 256 || c->n_seqs > 1 << 24) return HGA_ERR_UNSUPPORTED;
  if (c->Hq > 4096 || (c->total / hga::packed::kLeastTile + c->n_seqs) * c->Hq > INT32_MAX) return HGA_ERR_UNSUPPORTED;
  return HGA_OK;
}

hga::packed::Problem packed_problem(const hga_packed_config_t* c, void* ws) {
  hga::packed::Problem p{};
  p.Hq = c->Hq;
  p.Hkv = c->Hkv;
  p.G = c->Hq / c->Hkv;
  p.n_seqs = c->n_seqs;
  p.total = c->total;
  p.q = strided(c->q_stride_t, c->q_stride_h, c->Hq);
  p.k = strided(c->k_stride_t, c->k_stride_h, c->Hkv);
  p.v = strided(c->v_stride_t, c->v_stride_h, c->Hkv);
  p.scale = eff_scale(c->softmax_scale);
  p.fill_tail = (c->flags & HGA_PACKED_FILL_TAIL) != 0;
  p.status = static_cast<int*>(ws);
  p.wait_ns = wait_limit(c->wait_limit_ns);
  return p;
}

// Workspace: [status word | header | two work lists | two float32 per row: lse and delta as the dK, dV kernel takes them].
size_t list_bytes(const hga_packed_config_t* c) {
  return round256((size_t)(hga::packed::list_capacity(c->total, c->n_seqs, hga::packed::kLeastTile) + 1) *
                  sizeof(hga::packed::Tile));
}
struct PackedWorkspace {
  hga::packed::Header* hdr;
  hga::packed::Tile* lists[2];
  float* stats;
};
PackedWorkspace packed_workspace(const hga_packed_config_t* c, void* ws) {
  char* p = static_cast<char*>(ws) + hga::kStatusBytes;
  PackedWorkspace w;
  w.hdr = reinterpret_cast<hga::packed::Header*>(p);
  p += sizeof(hga::packed::Header);
  for (int i = 0; i < 2; ++i, p += list_bytes(c)) w.lists[i] = reinterpret_cast<hga::packed::Tile*>(p);
  w.stats = reinterpret_cast<float*>(p);
  return w;
}
size_t packed_bytes(const hga_packed_config_t* c) {
  return hga::kStatusBytes + sizeof(hga::packed::Header) + 2 * list_bytes(c) +
         round256(2 * (size_t)c->Hq * c->total * sizeof(float));
}

// The kernels' work: lists of the plan kernel or, where there are fewer units (tiles of the first list times its head
// units) than SMs, so that none waits for another, nothing: the kernels find their tiles themselves.  37 tokens: 8.5 us
// on the GPU with the plan kernel, 6.0 without, and 9.1 and 3.9 us for the call.
cudaError_t plan_work(const hga_packed_config_t* c, const hga::packed::Problem& p, const int32_t* cu,
                      hga::packed::Header* hdr, int n_lists, const hga::packed::ListSpec* lists, hga::packed::Work* out,
                      cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int per = c->dtype == HGA_BF16 ? hga::packed::head_units(p.Hkv, p.G) : p.Hq;
  const bool clear = (c->flags & HGA_PACKED_CLEAR_STATUS) != 0;
  const bool own = c->total > 0 && c->n_seqs <= hga::packed::kOwnSeqs &&
                   hga::packed::list_capacity(c->total, c->n_seqs, lists[0].tile) * per < sms;
  for (int i = 0; i < n_lists; ++i)
    out[i] = {hdr, lists[i].list, i, own ? cu : nullptr, c->n_seqs, lists[i].tile, clear && i == 0, c->total, p.status};
  if (own) return cudaSuccess;
  return hga::packed::launch_plan(cu, c->n_seqs, c->total, n_lists, lists, hdr, p.status, clear, st);
}

// ---------------------------------------------------------------- pages
int check_pages(const hga_pages_config_t* c) {
  if (!c) return HGA_ERR_ARG;
  if (c->n_layers < 1 || c->n_pages < 1 || c->Hkv < 1 || c->max_seqs < 1 || c->max_pages < 1) return HGA_ERR_ARG;
  if (c->dtype != HGA_F32 && c->dtype != HGA_BF16) return HGA_ERR_ARG;
  if (c->D != hga::kD) return HGA_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return HGA_ERR_UNSUPPORTED;
  if (c->max_seqs > hga::pages::kMaxSeqs || c->n_pages > hga::pages::kMaxPages) return HGA_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page > INT32_MAX - 1024 || c->Hkv > 4096 || c->n_layers > 4096)
    return HGA_ERR_UNSUPPORTED;
  const int64_t least = (int64_t)c->Hkv * c->page * c->D;
  if (c->page_stride != 0 && (c->page_stride < least || c->page_stride > (int64_t)1 << 37)) return HGA_ERR_ARG;
  if (c->layer_stride < 0 || c->layer_stride > (int64_t)1 << 46) return HGA_ERR_ARG;
  if (c->layer_stride != 0 && c->n_layers > 1) {
    // layers either one after another, or side by side within a page's stride
    const int64_t ps = c->page_stride ? c->page_stride : least;
    const bool outside = c->layer_stride >= (c->n_pages - 1) * ps + least;
    const bool inside = c->layer_stride >= least && (c->n_layers - 1) * c->layer_stride + least <= ps;
    if (!outside && !inside) return HGA_ERR_ARG;
  }
  for (int64_t s : {c->page_stride, c->layer_stride})
    if (s * elem_bytes(c->dtype) % 16 != 0) return HGA_ERR_ALIGN;
  if (c->wait_limit_ns < 0) return HGA_ERR_ARG;
  return HGA_OK;
}

hga::pages::Cache cache_of(const hga_pages_config_t* c, const int32_t* table, const int32_t* seq_len,
                           const int32_t* ref, void* ws) {
  hga::pages::Cache k{};
  k.n_layers = c->n_layers;
  k.n_pages = c->n_pages;
  k.page = c->page;
  k.Hkv = c->Hkv;
  k.max_seqs = c->max_seqs;
  k.max_pages = c->max_pages;
  k.elem = elem_bytes(c->dtype);
  k.page_data = (int64_t)c->Hkv * c->page * c->D * k.elem;
  k.page_bytes = c->page_stride ? c->page_stride * k.elem : k.page_data;
  k.layer_bytes = c->layer_stride ? c->layer_stride * k.elem : k.page_bytes * c->n_pages;
  k.table = const_cast<int32_t*>(table);
  k.seq_len = const_cast<int32_t*>(seq_len);
  k.ref = const_cast<int32_t*>(ref);
  k.status = static_cast<int*>(ws);
  return k;
}

// Workspace: [status word | counts | page lists (3 x n_pages) | attention: counters and parts].
size_t page_list_bytes(const hga_pages_config_t* c) { return round256((size_t)c->n_pages * sizeof(int32_t)); }
hga::pages::Scratch scratch_of(const hga_pages_config_t* c, void* ws) {
  char* p = static_cast<char*>(ws) + hga::kStatusBytes;
  hga::pages::Scratch s;
  s.counts = reinterpret_cast<int32_t*>(p);
  p += 256;
  s.src = reinterpret_cast<int32_t*>(p);
  s.dst = reinterpret_cast<int32_t*>(p + page_list_bytes(c));
  s.to = reinterpret_cast<int32_t*>(p + 2 * page_list_bytes(c));
  return s;
}
void* attn_scratch_of(const hga_pages_config_t* c, void* ws) {
  return static_cast<char*>(ws) + hga::kStatusBytes + 256 + 3 * page_list_bytes(c);
}
int check_entries(int32_t n) { return n < 0 ? HGA_ERR_ARG : n > hga::pages::kMaxSeqs ? HGA_ERR_UNSUPPORTED : HGA_OK; }

}  // namespace

extern "C" {

int hga_packed_workspace_size(const hga_packed_config_t* cfg, size_t* bytes_out) {
  int rc = check_packed(cfg);
  if (rc) return rc;
  if (!bytes_out) return HGA_ERR_ARG;
  *bytes_out = packed_bytes(cfg);
  return HGA_OK;
}

int hga_packed_attn_fwd(const hga_packed_config_t* cfg, const void* q, const void* k, const void* v,
                        const int32_t* cu_seqlens, void* o, void* o_lo, float* lse, void* workspace, void* stream) {
  int rc = check_packed(cfg);
  if (rc) return rc;
  if (cfg->total > 0 && (rc = check_ptrs({q, k, v, o, lse}, 16))) return rc;
  if (!aligned(o_lo, 16)) return HGA_ERR_ALIGN;
  if ((rc = check_ptrs({cu_seqlens}, 4))) return rc;
  if ((rc = check_workspace(workspace))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const hga::packed::Problem p = packed_problem(cfg, workspace);
  const PackedWorkspace w = packed_workspace(cfg, workspace);
  const bool bf16 = cfg->dtype == HGA_BF16;
  const int f32_tile = hga::packed::f32_tile(p.total, p.n_seqs, p.Hq);
  const hga::packed::ListSpec list{bf16 ? hga::packed::fwd_tile(p.G) : f32_tile, 0, w.lists[0]};
  hga::packed::Work work;
  cudaError_t e = plan_work(cfg, p, cu_seqlens, w.hdr, 1, &list, &work, st);
  if (e != cudaSuccess || cfg->total == 0) return from_cuda(e);
  if (bf16) return from_cuda(hga::packed::launch_fwd_tc(q, k, v, o, o_lo, lse, work, p, st));
  return from_cuda(hga::packed::launch_fwd_f32(q, k, v, o, lse, work, p, st));
}

int hga_packed_attn_bwd(const hga_packed_config_t* cfg, const void* q, const void* k, const void* v,
                        const int32_t* cu_seqlens, const void* o, const void* o_lo, const float* lse, const void* d_o,
                        void* dq, void* dk, void* dv, void* workspace, void* stream) {
  int rc = check_packed(cfg);
  if (rc) return rc;
  if (cfg->total > 0 && (rc = check_ptrs({q, k, v, o, lse, d_o, dq, dk, dv}, 16))) return rc;
  if (!aligned(o_lo, 16)) return HGA_ERR_ALIGN;
  if ((rc = check_ptrs({cu_seqlens}, 4))) return rc;
  if ((rc = check_workspace(workspace))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const hga::packed::Problem p = packed_problem(cfg, workspace);
  const PackedWorkspace w = packed_workspace(cfg, workspace);
  const bool bf16 = cfg->dtype == HGA_BF16;
  const int f32_tile = hga::packed::f32_tile(p.total, p.n_seqs, p.Hq);
  const hga::packed::ListSpec lists[2] = {
      {bf16 ? hga::packed::dq_tile(p.G) : f32_tile, 0, w.lists[0]},
      {bf16 ? hga::packed::kKeyTile : f32_tile, 1, w.lists[1]}};
  hga::packed::Work work[2];
  cudaError_t e = plan_work(cfg, p, cu_seqlens, w.hdr, 2, lists, work, st);
  if (e != cudaSuccess || cfg->total == 0) return from_cuda(e);
  if (bf16)
    return from_cuda(
        hga::packed::launch_bwd_tc(q, k, v, o, o_lo, lse, d_o, w.stats, dq, dk, dv, work[0], work[1], p, st));
  return from_cuda(hga::packed::launch_bwd_f32(q, k, v, o, lse, d_o, w.stats, dq, dk, dv, work[0], work[1], p, st));
}

int hga_pages_workspace_size(const hga_pages_config_t* cfg, size_t* bytes_out) {
  int rc = check_pages(cfg);
  if (rc) return rc;
  if (!bytes_out) return HGA_ERR_ARG;
  *bytes_out = hga::kStatusBytes + 256 + 3 * page_list_bytes(cfg) + hga::pages::paged_attn_scratch_bytes();
  return HGA_OK;
}

int hga_pages_reserve(const hga_pages_config_t* cfg, int32_t n, const int32_t* rows, const int32_t* add, int32_t* pos,
                      int32_t* table, int32_t* seq_len, int32_t* ref, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (n > 0 && (rc = check_ptrs({rows, add, pos}, 4))) return rc;
  if ((rc = check_ptrs({table, seq_len, ref}, 4)) || (rc = check_workspace(workspace))) return rc;
  if (n == 0) return HGA_OK;
  return from_cuda(hga::pages::launch_reserve(cache_of(cfg, table, seq_len, ref, workspace),
                                              scratch_of(cfg, workspace), n, rows, add, pos,
                                              static_cast<cudaStream_t>(stream)));
}

int hga_pages_write(const hga_pages_config_t* cfg, int32_t layer, int32_t n, const int32_t* rows, const int32_t* pos,
                    const int32_t* cu_new, int64_t total, const void* k_new, int64_t k_stride_t, int64_t k_stride_h,
                    const void* v_new, int64_t v_stride_t, int64_t v_stride_h, const int32_t* table,
                    const int32_t* seq_len, void* k_pool, void* v_pool, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (layer < 0 || layer >= cfg->n_layers || total < 0) return HGA_ERR_ARG;
  if (total > INT32_MAX) return HGA_ERR_UNSUPPORTED;
  for (int64_t s : {k_stride_t, k_stride_h, v_stride_t, v_stride_h})
    if ((rc = check_stride(s, cfg->dtype))) return rc;
  if (n > 0 && (rc = check_ptrs({rows, pos}, 4))) return rc;
  if (total > 0 && (rc = check_ptrs({k_new, v_new}, 16))) return rc;
  if ((rc = check_ptrs({cu_new, table, seq_len}, 4)) || (rc = check_ptrs({k_pool, v_pool}, 16)) ||
      (rc = check_workspace(workspace)))
    return rc;
  if (n == 0 || total == 0) return HGA_OK;
  const hga::packed::Strided ks = strided(k_stride_t, k_stride_h, cfg->Hkv), vs = strided(v_stride_t, v_stride_h, cfg->Hkv);
  return from_cuda(hga::pages::launch_write(cache_of(cfg, table, seq_len, nullptr, workspace), layer, n, rows, pos,
                                            cu_new, total, k_new, ks.t, ks.h, v_new, vs.t, vs.h, k_pool, v_pool,
                                            static_cast<cudaStream_t>(stream)));
}

int hga_paged_attn(const hga_pages_config_t* cfg, int32_t layer, int32_t n, int32_t Hq, float softmax_scale,
                   const int32_t* rows, const void* q, int64_t q_stride_n, const int32_t* table,
                   const int32_t* seq_len, const void* k_pool, const void* v_pool, void* o, float* lse,
                   void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (layer < 0 || layer >= cfg->n_layers || Hq < 1 || Hq % cfg->Hkv != 0 || bad_scale(softmax_scale))
    return HGA_ERR_ARG;
  if (Hq / cfg->Hkv > 128) return HGA_ERR_UNSUPPORTED;
  if (q_stride_n != 0 && q_stride_n < (int64_t)Hq * hga::kD) return HGA_ERR_ARG;
  if (q_stride_n > (int64_t)1 << 37) return HGA_ERR_ARG;
  if (q_stride_n * elem_bytes(cfg->dtype) % 16 != 0) return HGA_ERR_ALIGN;
  if (n > 0 && ((rc = check_ptrs({rows, lse}, 4)) || (rc = check_ptrs({q, o}, 16)))) return rc;
  if ((rc = check_ptrs({table, seq_len}, 4)) || (rc = check_ptrs({k_pool, v_pool}, 16)) ||
      (rc = check_workspace(workspace)))
    return rc;
  if (n == 0) return HGA_OK;
  return from_cuda(hga::pages::launch_paged_attn(
      cfg->dtype == HGA_BF16, cache_of(cfg, table, seq_len, nullptr, workspace), layer, n, Hq,
      eff_scale(softmax_scale), rows, q, q_stride_n ? q_stride_n : (int64_t)Hq * hga::kD, k_pool, v_pool, o, lse,
      attn_scratch_of(cfg, workspace), wait_limit(cfg->wait_limit_ns), static_cast<cudaStream_t>(stream)));
}

int hga_pages_fork(const hga_pages_config_t* cfg, int32_t n, const int32_t* src, const int32_t* dst, int32_t* table,
                   int32_t* seq_len, int32_t* ref, void* k_pool, void* v_pool, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (n > 0 && (rc = check_ptrs({src, dst}, 4))) return rc;
  if ((rc = check_ptrs({table, seq_len, ref}, 4)) || (rc = check_ptrs({k_pool, v_pool}, 16)) ||
      (rc = check_workspace(workspace)))
    return rc;
  if (n == 0) return HGA_OK;
  return from_cuda(hga::pages::launch_fork(cache_of(cfg, table, seq_len, ref, workspace), scratch_of(cfg, workspace),
                                           n, src, dst, k_pool, v_pool, static_cast<cudaStream_t>(stream)));
}

int hga_pages_free(const hga_pages_config_t* cfg, int32_t n, const int32_t* rows, const int32_t* table,
                   int32_t* seq_len, int32_t* ref, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (n > 0 && (rc = check_ptrs({rows}, 4))) return rc;
  if ((rc = check_ptrs({table, seq_len, ref}, 4)) || (rc = check_workspace(workspace))) return rc;
  if (n == 0) return HGA_OK;
  return from_cuda(hga::pages::launch_free(cache_of(cfg, table, seq_len, ref, workspace), n, rows,
                                           static_cast<cudaStream_t>(stream)));
}

int hga_pages_compact(const hga_pages_config_t* cfg, int32_t* table, const int32_t* seq_len, int32_t* ref,
                      void* k_pool, void* v_pool, int32_t* n_used, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc) return rc;
  if ((rc = check_ptrs({table, seq_len, ref, n_used}, 4)) || (rc = check_ptrs({k_pool, v_pool}, 16)) ||
      (rc = check_workspace(workspace)))
    return rc;
  return from_cuda(hga::pages::launch_compact(cache_of(cfg, table, seq_len, ref, workspace),
                                              scratch_of(cfg, workspace), k_pool, v_pool, n_used,
                                              static_cast<cudaStream_t>(stream)));
}

int hga_pages_copy(const hga_pages_config_t* cfg, int32_t n, const int32_t* src, const int32_t* dst, void* k_pool,
                   void* v_pool, void* workspace, void* stream) {
  int rc = check_pages(cfg);
  if (rc || (rc = check_entries(n))) return rc;
  if (n > 0 && (rc = check_ptrs({src, dst}, 4))) return rc;
  if ((rc = check_ptrs({k_pool, v_pool}, 16)) || (rc = check_workspace(workspace))) return rc;
  if (n == 0) return HGA_OK;
  return from_cuda(hga::pages::launch_copy(cache_of(cfg, nullptr, nullptr, nullptr, workspace),
                                           scratch_of(cfg, workspace), n, src, dst, k_pool, v_pool,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
