// Work lists of the packed (variable-length) attention kernels.
#pragma once

#include "common.cuh"

namespace hga {
namespace packed {

// One tile of a sequence: its rows are start + t0 .. of the packed tensors.
struct Tile {
  int32_t start, len;   // the sequence's first row and its length
  int32_t t0;           // the tile's first token within the sequence
  int32_t pad;
};

// Filled by the plan kernel, read by the kernels behind it in the stream.
struct Header {
  int32_t n_tiles[2];   // entries of the two lists
  int32_t end;          // first row of no sequence (0 when cu_seqlens is not valid)
  int32_t pad[61];
};
static_assert(sizeof(Header) == 256, "the workspace layout counts 256 bytes");

// Entries a list of `tile`-token tiles may need: every sequence ends with at most one partial tile.
inline int64_t list_capacity(int64_t total, int n_seqs, int tile) { return total / tile + n_seqs; }

struct ListSpec {
  int tile;             // tokens per tile
  int by_key;           // 0: a query tile (work: the keys up to its end); 1: a key tile (work: the
                        // queries from its start on)
  Tile* list;
};

// The tiles of one list as a kernel gets them: from the plan kernel's list or, for few tiles, from cu_seqlens itself.
struct Work {
  const Header* hdr;
  const Tile* list;
  int which;            // of the header's two lists
  const int32_t* cu;    // not nullptr: no plan kernel ran; each CTA finds the tile of its slot (own_tile)
  int n_seqs, tile, clear_status;
  int64_t total;
  int* status;
};

// Sequences whose bounds fit the lanes of a warp.
constexpr int kOwnSeqs = 31;

// A CTA's only tile, in its shared memory.
struct alignas(16) Own {
  Tile tile;
  int has, end;         // whether there is one; first row of no sequence
};

// The tile of slot i of the list (as in the plan kernel; slots without a tile stay), which is all that a kernel with a
// CTA per unit needs: the order of the list matters only when some CTAs wait for others.  Called by one warp.
__device__ __forceinline__ void own_tile(const Work& w, int slot, Own* own) {
  const int lane = threadIdx.x & 31;
  const int32_t c = w.cu[min(lane, w.n_seqs)], up = __shfl_up_sync(0xffffffffu, c, 1);
  const bool bad = __any_sync(0xffffffffu, lane == 0 ? c != 0 : c < up || (lane == 31 && c > w.total));
  if (blockIdx.x == 0 && lane == 0) {
    if (w.clear_status) *w.status = 0;
    if (bad) set_status(w.status, -1);
  }
  const int32_t end = __shfl_sync(0xffffffffu, c, 31);
  const uint32_t before = __ballot_sync(0xffffffffu, lane < w.n_seqs && c / w.tile + lane <= slot);
  const int s = before ? 31 - __clz(before) : 0;
  const int32_t start = __shfl_sync(0xffffffffu, c, s), next = __shfl_sync(0xffffffffu, c, s + 1);
  const int64_t t0 = (int64_t)(slot - (start / w.tile + s)) * w.tile;
  if (lane == 0) {
    own->tile = Tile{start, next - start, (int32_t)t0, 0};
    own->has = !bad && before && t0 < next - start;
    own->end = bad ? 0 : end;
  }
}

// The same for kernels of both kinds.
template <bool kOwn>
__device__ __forceinline__ int4 tile_of(const Work& w, const Own& own, int64_t i) {
  return kOwn ? *reinterpret_cast<const int4*>(&own.tile) : __ldg(reinterpret_cast<const int4*>(w.list) + i);
}
// Work units, of `per` a tile: unit blockIdx.x is this CTA's first (own: and only) one.
template <bool kOwn>
__device__ __forceinline__ int64_t units_of(const Work& w, const Own& own, int per) {
  return kOwn ? (own.has ? gridDim.x : 0) : (int64_t)w.hdr->n_tiles[w.which] * per;
}
template <bool kOwn>
__device__ __forceinline__ int64_t end_of(const Work& w, const Own& own) { return kOwn ? own.end : w.hdr->end; }

cudaError_t launch_plan(const int32_t* cu, int n_seqs, int64_t total, int n_lists, const ListSpec* lists, Header* hdr,
                        int* status, bool clear_status, cudaStream_t st);

}  // namespace packed
}  // namespace hga
