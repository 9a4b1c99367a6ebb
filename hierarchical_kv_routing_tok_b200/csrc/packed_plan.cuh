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

cudaError_t launch_plan(const int32_t* cu, int n_seqs, int64_t total, int n_lists, const ListSpec* lists, Header* hdr,
                        int* status, bool clear_status, cudaStream_t st);

}  // namespace packed
}  // namespace hga
