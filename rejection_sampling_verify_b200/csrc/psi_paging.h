// psi_paging.h - index arithmetic of the paged key-value cache and of a
// block's tree, shared by the cache kernels.  Plain functions that compile
// for the host too, so that every index a kernel forms can be checked on the
// CPU (tests/test_paging_cpu.py).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PSI_HD __host__ __device__ __forceinline__
#else
#define PSI_HD inline
#endif

namespace psi {

// One layer's pages.  Offsets are in elements and pass 32 bits in a large pool.
struct Paging {
  const int32_t *table;  // [N][max_pages]
  const int32_t *lens;   // [N]
  int32_t max_pages;
  int32_t num_pages;
  int32_t page_size;
  int64_t page_stride, slot_stride, head_stride;
};

// Positions that a sequence's table row can hold.
PSI_HD int64_t table_capacity(const Paging &g) { return (int64_t)g.max_pages * g.page_size; }

// Page of position t of the sequence whose table row is `row`; -1 where the
// position has no page of the pool.
PSI_HD int32_t page_of(const Paging &g, const int32_t *row, int64_t t) {
  if (t < 0 || t >= table_capacity(g)) return -1;
  const int32_t p = row[(int32_t)(t / g.page_size)];
  return (p >= 0 && p < g.num_pages) ? p : -1;
}

// Element offset of head 0 at position t, or -1.
PSI_HD int64_t slot_offset(const Paging &g, const int32_t *row, int64_t t) {
  const int32_t p = page_of(g, row, t);
  if (p < 0) return -1;
  return (int64_t)p * g.page_stride + (t % g.page_size) * g.slot_stride;
}

// Depth of a block's row (root 0), -1 when its chain of parents holds an
// invalid index.  parents: the sequence's R - 1 entries, or nullptr for a
// chain.  Every valid step goes to a lower row, so the walk ends.
PSI_HD int32_t row_depth(const int32_t *parents, int32_t r) {
  if (!parents) return r;
  int32_t depth = 0;
  while (r > 0) {
    const int32_t p = parents[r - 1];
    if (p < -1 || p >= r - 1) return -1;
    r = p + 1;
    ++depth;
  }
  return depth;
}

// The rows that row r sees (itself and its path to the root) as bits, word
// by word; false (and no bits) when the chain is invalid.
constexpr int kBlockWords = 8;  // PSI_MAX_BLOCK_ROWS / 32
PSI_HD bool row_sees(const int32_t *parents, int32_t r, uint32_t bits[kBlockWords]) {
  for (int w = 0; w < kBlockWords; ++w) {
    const int32_t n = r + 1 - 32 * w;  // rows 0..r of this word
    bits[w] = (parents || n <= 0) ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
  }
  if (!parents) return true;
  if (row_depth(parents, r) < 0) return false;
  for (;;) {
    bits[r >> 5] |= 1u << (r & 31);
    if (r == 0) return true;
    r = parents[r - 1] + 1;
  }
}

// Nodes of an accepted path that can be kept: the leading entries that ascend
// within [0, M).  With `step` over 1 only entries first, first + step, ... are
// looked at; the minimum over first = 0..step - 1 is the answer.
PSI_HD int32_t path_prefix(const int32_t *nodes, int32_t len, int32_t M, int32_t first = 0,
                           int32_t step = 1) {
  const int32_t n = len < 0 ? 0 : len > M ? M : len;
  for (int32_t j = first; j < n; j += step)
    if (nodes[j] <= (j ? nodes[j - 1] : -1) || nodes[j] >= M) return j;
  return n;
}

// How a sequence's positions are dealt to the CTAs of its rows: `units`
// ranges of `per` positions (a multiple of the tile), alike but for a shorter
// last one and never empty; at most `splits` of them, and no more than ranges
// of `least` tiles would make.
struct Ranges {
  int32_t units, per;
};
PSI_HD Ranges deal(int32_t total, int32_t tile, int32_t splits, int32_t least) {
  const int32_t tiles = (total - 1) / tile + 1;
  int32_t per = (tiles - 1) / splits + 1;
  if (per < least) per = least;
  Ranges r;
  r.units = (tiles - 1) / per + 1;
  r.per = ((tiles - 1) / r.units + 1) * tile;  // evenly
  return r;
}

// Pages for `slots` positions.
PSI_HD int64_t pages_for(int64_t slots, int32_t page_size) {
  return slots <= 0 ? 0 : (slots + page_size - 1) / page_size;
}

}  // namespace psi
