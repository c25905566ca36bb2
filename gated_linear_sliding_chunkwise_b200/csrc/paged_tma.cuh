// Page loads of the paged attention kernels that stage keys and values by
// TMA, and their bounded waits.
#pragma once

#include "paged.cuh"
#include "tc_common.cuh"
#include "tc_host.h"

namespace lz {
namespace paged {

// The pool of one layer as rows of d elements, (page, head, slot) outermost to
// innermost; a box is 64 columns x min(page, 64) rows of one page.
inline bool make_pool_map(CUtensorMap *map, const void *pool, const PagedArgs &a) {
  return tc::make_map_bf16_3d(map, pool, a.d, (uint64_t)a.num_pages * a.Hkv * a.page, 1, a.page < 64 ? a.page : 64);
}

// Waits that give up: the first one that does records the timeout and makes
// the CTA's later ones return at once, so that every role keeps its control
// flow (and its barriers) to the end.
struct Waits {
  volatile uint32_t *dead;   // shared memory, 0 at the start
  uint32_t *status;
  LZ_DEV bool operator()(uint64_t *bar, uint32_t parity) const {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
    if (tc::mbar_wait(bar, parity, status, ST_TIMEOUT)) return true;
    *dead = 1;
    return false;
  }
};

// Key range that some token of the piece sees: [0, sinks) and [low, end).
struct Range {
  int low, end, sinks;
  LZ_DEV Range(const PagedArgs &a, const Piece &p) {
    const int base = p.q.s - p.q.n;
    end = max(base + p.i1, 0);
    low = a.window > 0 ? max(base + p.i0 - a.window + 1, 0) : 0;
    sinks = a.window > 0 ? a.sinks : 0;
  }
  LZ_DEV bool any(int j) const { return j < end && (j >= low || j < sinks); }
  // whether any key of [j, j + n) is seen
  LZ_DEV bool some(int j, int n) const { return j < end && (j + n > low || j < sinks); }
  // whether every key of [j, j + n) is seen by some token
  LZ_DEV bool whole(int j, int n) const { return j + n <= end && (j >= low || j + n <= sinks); }
};

// Row of the pool's map where the box of tokens [j, j + box) begins.  Boxes
// without a key that is seen, and pages outside the pool, lie past the map's
// end: they read as zeros.
LZ_DEV int box_row(const PagedArgs &a, uint32_t *status, const Piece &p, const Range &r, int j, int box) {
  const int none = a.num_pages * a.Hkv * a.page;
  if (!r.some(j, box)) return none;
  const int id = page_id(a, status, p.q.row, j >> a.shift);
  return id < 0 ? none : ((id * a.Hkv + p.h) << a.shift) + (j & (a.page - 1));
}

}  // namespace paged
}  // namespace lz
