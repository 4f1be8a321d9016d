// The 16-bit paged cache and what its kernels share: slots, positions, trees.
//
// K and V are bf16 or f16 [pages, P, Hkv, D] with byte strides of page, token
// and head (heads before tokens, or K and V in one tensor, are other strides).
// Slot p of request b is row p % P of page table[b, p / P]; P is a power of two
// from 16 to 128. New row n of request b has slot base_b + n. Its position, by
// which keys and queries are rotated and distances counted, is base_b + depth:
// the row's depth in the request's tree, or n in a chain.
#pragma once

#include "q8_common.cuh"

namespace sv {

struct PagedView {
  uint8_t* x[2];              // k, v
  int64_t sp[2], st[2], sh[2];   // bytes: page, token, head
  const int32_t* table;       // [B, max_pages]
  int32_t num_pages, Hkv, page_shift, max_pages;
};

// Page id of logical page lp of request b, or -1 if there is none.
__device__ __forceinline__ int paged_page(const PagedView& c, int b, int lp) {
  if (lp < 0 || lp >= c.max_pages) return -1;
  const int p = c.table[static_cast<int64_t>(b) * c.max_pages + lp];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// A node's parent in a tree whose nodes follow their parents: -1 ends a path,
// and so does what is no earlier node, however far out of range (what is kept
// of the parents in 16 bits is this, never what was given).
__device__ __forceinline__ int tree_up(const int32_t* parents, int n) {
  const int p = parents[n];
  return p >= 0 && p < n ? p : -1;
}
__device__ __forceinline__ int tree_depth(const int32_t* parents, int n) {
  int d = 0;
  for (int m = tree_up(parents, n); m >= 0; m = tree_up(parents, m)) ++d;
  return d;
}
__device__ __forceinline__ bool bad_parent(int p, int n) { return n == 0 ? p != -1 : p < 0 || p >= n; }

}  // namespace sv
