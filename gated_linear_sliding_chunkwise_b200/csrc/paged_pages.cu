// The paged cache's bookkeeping: pages handed out, given back, shared and
// closed up, on the device.
//
// A call's bookkeeping is one launch of N 1024-thread CTAs whose phases depend
// on one another: N = 8 CTAs of a cluster with cluster barriers between them,
// or one CTA for short lists and small pools, where the barriers cost more
// than the other CTAs' help (the rule is at launch_book).  The pool's counts
// are read once, coalesced, into a bit per page in shared memory (CTA c keeps
// the c-th part of the pool); ranks among the free pages are population counts
// and a block scan over those words.  It is bound by that chain of latencies,
// not by bytes: loops over a row's pages keep kAhead loads under way per lane.
// Page contents move in a second launch over the whole GPU, which reads the
// list of copies that the first one made: bound by HBM.
#include "paged.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kMost = 8, kThreads = 1024, kWarps = kThreads / 32;   // kMost: CTAs of a cluster
constexpr uint32_t ST_PAGES = 8u;
constexpr int kAhead = 8;   // entries of a row under way per lane

template <int N> LZ_DEV int cluster_rank() {
  if (N == 1) return 0;
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return (int)r;
}
// All threads of the call; global writes before it are visible after it.
template <int N> LZ_DEV void book_sync() {
  if (N == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
LZ_DEV void report(const PagesArgs &a, uint32_t bit) { atomicOr(a.status, bit); }
// Whether the list was refused.  Asked after the barrier behind its checks:
// only ST_INDEX is settled there.  ST_PAGES is recorded later, by one thread
// and with no barrier behind it, while threads of other CTAs may still ask
// here: they must not see it, or a CTA would go on without some of its warps.
// (Each CTA compares the sums for itself, so all agree without the bit.)
LZ_DEV bool list_refused(const PagesArgs &a) { return *reinterpret_cast<volatile uint32_t *>(a.status) & ST_INDEX; }

// Exclusive prefix of v over the block's threads, and the block's sum.
LZ_DEV int block_scan(int v, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // the last scan's reads of sums
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int w = sums[lane];                    // kWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  return x - v + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// The pages of CTA c: [lo, hi), lo a multiple of 128.
struct Segment {
  int lo, hi, words;
};
template <int N> LZ_DEV Segment segment_of(const PagesArgs &a, int c) {
  const int per = ((a.num_pages + N * 128 - 1) / (N * 128)) * 128;
  Segment g;
  g.lo = min(c * per, a.num_pages);
  g.hi = min(g.lo + per, a.num_pages);
  g.words = (g.hi - g.lo + 31) / 32;
  return g;
}

// One bit per page of the segment: refs > 0.  Bits past the pool are 1 (never
// free); `live` masks them out where live pages are counted.
LZ_DEV void read_live(const PagesArgs &a, const Segment &g, uint32_t *bits) {
  const int lane = threadIdx.x & 31;
  for (int p0 = g.lo + (threadIdx.x >> 5) * 128; p0 < g.hi; p0 += kWarps * 128) {
    const int p = p0 + lane * 4;
    int4 r = make_int4(1, 1, 1, 1);
    if (p + 3 < g.hi) {
      r = *reinterpret_cast<const int4 *>(a.refs + p);
    } else {
      if (p < g.hi) r.x = a.refs[p];
      if (p + 1 < g.hi) r.y = a.refs[p + 1];
      if (p + 2 < g.hi) r.z = a.refs[p + 2];
    }
    uint32_t w = (r.x != 0) | (r.y != 0) << 1 | (r.z != 0) << 2 | (r.w != 0) << 3;
    w <<= 4 * (lane & 7);
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if ((lane & 7) == 0 && p < g.hi) bits[(p - g.lo) / 32] = w;
  }
  __syncthreads();
}

// Number of set bits of f(word index) over the segment, block-wide.
template <typename F> LZ_DEV int count_bits(const Segment &g, int *sums, F f) {
  int n = 0, total;
  for (int w = threadIdx.x; w < g.words; w += kThreads) n += __popc(f(w));
  block_scan(n, sums, total);
  return total;
}
// Calls put(rank, page) for the set bits of f, ranks from `rank` on, as long
// as the rank is below `most`.  The ranks of the words come from a block scan;
// then a warp takes a word and a lane a bit, so that what put writes by rank is
// written coalesced (a thread per word took 8 us for 48 K pages, this 2).
template <typename F, typename G>
LZ_DEV void each_bit(const Segment &g, int *sums, int *first, int rank, int most, F f, G put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w0 = 0; w0 < g.words && rank < most; w0 += kThreads) {
    const int w = w0 + threadIdx.x;
    int total;
    const int before = block_scan(w < g.words ? __popc(f(w)) : 0, sums, total);
    first[threadIdx.x] = rank + before;
    __syncthreads();
    for (int y = warp; y < kThreads && w0 + y < g.words; y += kWarps) {
      const uint32_t x = f(w0 + y);
      const int r = first[y] + __popc(x & ((1u << lane) - 1u));
      if ((x >> lane & 1u) && r < most) put(r, g.lo + (w0 + y) * 32 + lane);
    }
    rank += total;
    __syncthreads();                     // first is written anew
  }
}

LZ_DEV bool row_ok(const PagesArgs &a, int r) { return r >= 0 && r < a.rows; }
LZ_DEV bool len_ok(const PagesArgs &a, int n) { return n >= 0 && n <= (long long)a.max_pages * a.page; }
LZ_DEV int pages_of(const PagesArgs &a, int n) { return (int)(((long long)n + a.page - 1) / a.page); }

// Marks row r as listed; false when it was listed before.
LZ_DEV bool first_mark(const PagesArgs &a, int r) { return atomicExch(a.mark + r, 1) == 0; }
template <int N> LZ_DEV void clear_marks(const PagesArgs &a, int c) {
  for (int i = c * kThreads + threadIdx.x; i < a.rows; i += N * kThreads) a.mark[i] = 0;
  if (c == 0 && threadIdx.x == 0) *a.status = 0;
}
// The entries of a row's pages are live pages of the pool; one warp.
LZ_DEV bool entries_ok(const PagesArgs &a, const int *entries, int held) {
  bool ok = true;
  for (int j0 = threadIdx.x & 31; j0 < held; j0 += 32 * kAhead) {
    int p[kAhead], r[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) p[i] = j0 + 32 * i < held ? entries[j0 + 32 * i] : entries[j0];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) r[i] = p[i] >= 0 && p[i] < a.num_pages ? a.refs[p[i]] : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ok = ok && r[i] > 0;
  }
  return __all_sync(0xffffffffu, ok);
}

// Offsets of the list's needs (exclusive prefix) and their sum.  Every CTA
// finds them for itself and writes the same values: one barrier of the call
// less than with one CTA for all.  A sum past 2^31 cannot be: it is at most
// n * max_pages, which is kept below 2^31.
LZ_DEV int scan_needs(const PagesArgs &a, int *sums) {
  int base = 0;
  for (int i0 = 0; i0 < a.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int total;
    const int off = block_scan(i < a.n ? a.need[i] : 0, sums, total);
    if (i < a.n) a.offset[i] = base + off;
    base += total;
  }
  __syncthreads();
  return base;
}

// Free pages before this CTA's segment and in the whole pool.
template <int N> LZ_DEV void free_before(const PagesArgs &a, int c, int &before, int &all) {
  before = all = 0;
  for (int x = 0; x < N; ++x) {
    const int n = reinterpret_cast<volatile int *>(a.count)[x];
    if (x < c) before += n;
    all += n;
  }
}

template <int N> __global__ void __launch_bounds__(kThreads, 1) pages_reserve_kernel(PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], first[kThreads];
  const int c = cluster_rank<N>(), tid = threadIdx.x, lane = tid & 31;
  const Segment g = segment_of<N>(a, c);
  clear_marks<N>(a, c);
  read_live(a, g, bits);
  const auto free_word = [&](int w) { return ~bits[w]; };
  const int mine = count_bits(g, sums, free_word);
  if (tid == 0) a.count[c] = mine;
  book_sync<N>();
  for (int i = c * kThreads + tid; i < a.n; i += N * kThreads) {
    const int r = a.row[i], grow = a.grow[i];
    int need = 0;
    bool ok = row_ok(a, r) && grow >= 0;
    if (ok) {
      const int old = a.lens[r];
      ok = len_ok(a, old) && (long long)old + grow <= (long long)a.max_pages * a.page && first_mark(a, r);
      if (ok) need = pages_of(a, old + grow) - pages_of(a, old);
    }
    if (!ok) report(a, ST_INDEX);
    a.need[i] = need;
  }
  book_sync<N>();
  if (list_refused(a)) return;
  const int total = scan_needs(a, sums);
  int before, all;
  free_before<N>(a, c, before, all);
  if (total > all) {
    if (c == 0 && tid == 0) report(a, ST_PAGES);
    return;
  }
  each_bit(g, sums, first, before, total, free_word, [&](int r, int p) { a.list[r] = p; });
  book_sync<N>();
  for (int i = c * kWarps + (tid >> 5); i < a.n; i += N * kWarps) {
    const int r = a.row[i], old = a.lens[r], had = pages_of(a, old), need = a.need[i], off = a.offset[i];
    for (int j0 = lane; j0 < need; j0 += 32 * kAhead) {
      int p[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) p[x] = j0 + 32 * x < need ? a.list[off + j0 + 32 * x] : -1;
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (p[x] >= 0) {
          a.table[(size_t)r * a.max_pages + had + j0 + 32 * x] = p[x];
          a.refs[p[x]] = 1;
        }
    }
    __syncwarp();
    if (lane == 0) a.lens[r] = old + a.grow[i];
  }
}

template <int N> __global__ void __launch_bounds__(kThreads, 1) pages_free_kernel(PagesArgs a) {
  const int c = cluster_rank<N>(), lane = threadIdx.x & 31;
  const int w0 = c * kWarps + (threadIdx.x >> 5);
  clear_marks<N>(a, c);
  book_sync<N>();
  for (int i = w0; i < a.n; i += N * kWarps) {
    const int r = a.row[i];
    bool ok = row_ok(a, r) && len_ok(a, a.lens[r]);
    if (ok) ok = entries_ok(a, a.table + (size_t)r * a.max_pages, pages_of(a, a.lens[r]));
    if (lane == 0 && !(ok && first_mark(a, r))) report(a, ST_INDEX);
  }
  book_sync<N>();
  if (list_refused(a)) return;
  for (int i = w0; i < a.n; i += N * kWarps) {
    const int r = a.row[i], held = pages_of(a, a.lens[r]);
    int *entries = a.table + (size_t)r * a.max_pages;
    for (int j0 = lane; j0 < a.max_pages; j0 += 32 * kAhead) {
      int p[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) p[x] = j0 + 32 * x < held ? entries[j0 + 32 * x] : -1;
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        if (p[x] >= 0) atomicSub(a.refs + p[x], 1);
        if (j0 + 32 * x < a.max_pages) entries[j0 + 32 * x] = -1;
      }
    }
    __syncwarp();
    if (lane == 0) a.lens[r] = 0;
  }
}

// need[i]: 1 when the source's last page is part-filled; held[i]: length of
// the source as it was; snap: its table row as it was.
template <int N> __global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], first[kThreads];
  const int c = cluster_rank<N>(), tid = threadIdx.x, lane = tid & 31;
  const int w0 = c * kWarps + (tid >> 5);
  const Segment g = segment_of<N>(a, c);
  pdl_trigger();                                    // the copies' kernel may take its place and wait
  clear_marks<N>(a, c);
  if (c == 0 && tid == 0) a.count[kMost] = 0;       // no copies yet, whatever happens below
  read_live(a, g, bits);
  const auto free_word = [&](int w) { return ~bits[w]; };
  const int mine = count_bits(g, sums, free_word);
  if (tid == 0) a.count[c] = mine;
  book_sync<N>();
  for (int i = w0; i < a.n; i += N * kWarps) {
    const int r = a.row[i], x = a.src[i];
    bool ok = row_ok(a, r) && row_ok(a, x);
    int need = 0, n = 0;
    if (ok) {
      n = a.lens[x];
      const int old = a.lens[r];
      ok = len_ok(a, n) && len_ok(a, old);
      if (ok && r != x) {
        const int *from = a.table + (size_t)x * a.max_pages;
        const int held = pages_of(a, n);
        ok = entries_ok(a, from, held) && entries_ok(a, a.table + (size_t)r * a.max_pages, pages_of(a, old));
        for (int j = lane; j < held; j += 32) a.snap[(size_t)i * a.max_pages + j] = from[j];
        need = n % a.page != 0;
      }
    }
    if (lane == 0) {
      if (!(ok && first_mark(a, r))) report(a, ST_INDEX);
      a.need[i] = need;
      a.held[i] = n;
    }
  }
  book_sync<N>();
  if (list_refused(a)) return;
  const int total = scan_needs(a, sums);
  int before, all;
  free_before<N>(a, c, before, all);
  if (total > all) {
    if (c == 0 && tid == 0) report(a, ST_PAGES);
    return;
  }
  if (c == 0 && tid == 0) a.count[kMost] = total;   // the copies to make; none of a call that is refused
  each_bit(g, sums, first, before, total, free_word, [&](int r, int p) { a.list[r] = p; });
  // the shared pages' new holders, and what the replaced rows held
  for (int i = w0; i < a.n; i += N * kWarps) {
    const int r = a.row[i];
    if (r == a.src[i]) continue;
    const int whole = a.held[i] / a.page, old = pages_of(a, a.lens[r]);
    const int *was = a.table + (size_t)r * a.max_pages;
    for (int j = lane; j < whole; j += 32) atomicAdd(a.refs + a.snap[(size_t)i * a.max_pages + j], 1);
    for (int j = lane; j < old; j += 32) atomicSub(a.refs + was[j], 1);
  }
  book_sync<N>();
  for (int i = w0; i < a.n; i += N * kWarps) {
    const int r = a.row[i];
    if (r == a.src[i]) continue;
    const int n = a.held[i], whole = n / a.page;
    int *to = a.table + (size_t)r * a.max_pages;
    for (int j = lane; j < a.max_pages; j += 32) {
      int p = -1;
      if (j < whole) {
        p = a.snap[(size_t)i * a.max_pages + j];
      } else if (j == whole && n % a.page) {
        const int k = a.offset[i];
        p = a.list[k];
        a.refs[p] = 1;
        a.from[k] = a.snap[(size_t)i * a.max_pages + j];
        a.to[k] = p;
      }
      to[j] = p;
    }
    if (lane == 0) a.lens[r] = n;
  }
}

// list: new number of every live page; from / to: the pages that move;
// held: the moved pages' counts.
template <int N> __global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int sums[32], first[kThreads];
  const int c = cluster_rank<N>(), tid = threadIdx.x;
  const Segment g = segment_of<N>(a, c);
  pdl_trigger();                                   // the moves' kernel may take its place and wait
  if (c == 0 && tid == 0) *a.status = 0;
  read_live(a, g, bits);
  // bits past the pool: not live here
  const auto valid = [&](int w) { return g.hi - g.lo - w * 32 >= 32 ? ~0u : (1u << (g.hi - g.lo - w * 32)) - 1u; };
  const int mine = count_bits(g, sums, [&](int w) { return bits[w] & valid(w); });
  if (tid == 0) a.count[c] = mine;
  book_sync<N>();
  int before, live;
  free_before<N>(a, c, before, live);                 // live pages here
  const auto below = [&](int w) {                  // numbers below `live`
    const int n = live - (g.lo + w * 32);
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
  };
  const auto hole = [&](int w) { return ~bits[w] & below(w); };
  const auto high = [&](int w) { return bits[w] & valid(w) & ~below(w); };
  const int holes = count_bits(g, sums, hole), highs = count_bits(g, sums, high);
  if (tid == 0) a.count[kMost + c] = holes, a.count[2 * kMost + c] = highs;
  book_sync<N>();
  int hole0 = 0, high0 = 0, moves = 0;
  for (int x = 0; x < N; ++x) {
    const int h = a.count[kMost + x], o = a.count[2 * kMost + x];
    if (x < c) hole0 += h, high0 += o;
    moves += h;
  }
  each_bit(g, sums, first, hole0, INT_MAX, hole, [&](int r, int p) { a.to[r] = p; });
  each_bit(g, sums, first, high0, INT_MAX, high, [&](int r, int p) { a.from[r] = p; a.held[r] = a.refs[p]; });
  book_sync<N>();                                  // counts are read before they change (refs_out may be refs)
  if (c == 0 && tid == 0) a.count[3 * kMost] = moves;
  for (int p = g.lo + tid; p < g.hi; p += kThreads) {
    const bool on = (bits[(p - g.lo) >> 5] >> ((p - g.lo) & 31)) & 1u;
    if (p < live) {
      if (on) {
        a.list[p] = p;
        if (a.refs_out != a.refs) a.refs_out[p] = a.refs[p];
      } else {
        a.list[p] = -1;
      }
    } else {
      if (!on) a.list[p] = -1;
      a.refs_out[p] = 0;
    }
  }
  book_sync<N>();
  for (int k = c * kThreads + tid; k < moves; k += N * kThreads) {
    a.list[a.from[k]] = a.to[k];
    a.refs_out[a.to[k]] = a.held[k];
  }
}

// ------------------------------------------------------------- contents ---
// Copies page from[k] to to[k], k < *copies, in every layer, K and V; with a
// table, also gives its entries their pages' new numbers.  Sources and
// destinations are different pages.  A unit is 32 KB of a page in one layer, 128
// bytes under way per thread (32 bytes: 6.0 TB/s of a plain copy, 128: 6.25);
// neighbours in the list with one source (branches of one
// prompt) share its loads: 192 copies of 24 sources of 4 MB: 212 -> 175 us.
constexpr int kCopyThreads = 256, kCopyUnroll = 8, kRuns = 2048;

__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(PagesArgs a, const int *copies, int renumber) {
  __shared__ int heads[kRuns], warp_heads[kCopyThreads / 32];
  pdl_wait();
  const int n = *copies, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the list's runs of one source, where the copies are many bytes (finding
  // the runs costs 1.9 us; moves have no two alike)
  const bool merge = !renumber && n <= kRuns && (size_t)n * a.layers * 2 * a.page_bytes >= (size_t)32 << 20;
  int runs = n;
  if (merge) {
    runs = 0;
    for (int k0 = 0; k0 < n; k0 += kCopyThreads) {
      const int k = k0 + threadIdx.x;
      const bool head = k < n && (k == 0 || a.from[k] != a.from[k - 1]);
      const unsigned set = __ballot_sync(0xffffffffu, head);
      if (lane == 0) warp_heads[warp] = __popc(set);
      __syncthreads();
      int at = runs + __popc(set & ((1u << lane) - 1u));
      for (int w = 0; w < kCopyThreads / 32; ++w) {
        if (w < warp) at += warp_heads[w];
        runs += warp_heads[w];
      }
      if (head) heads[at] = k;
      __syncthreads();
    }
  }
  const size_t words = a.page_bytes / 16;                   // of one page in one layer
  const size_t chunk = (size_t)kCopyThreads * kCopyUnroll;
  const size_t per = (words + chunk - 1) / chunk;           // units of such a block
  const size_t blocks = (size_t)runs * a.layers * 2;
  for (size_t u = blockIdx.x; u < blocks * per; u += gridDim.x) {
    const size_t blk = u / per, off = (u % per) * chunk + threadIdx.x;
    const size_t x = blk / runs;
    const int run = (int)(blk % runs), k = merge ? heads[run] : run, end = !merge ? k + 1 : run + 1 < runs ? heads[run + 1] : n;
    uint4 *pool = static_cast<uint4 *>(x & 1 ? a.v_pages : a.k_pages) + (x >> 1) * a.num_pages * words;
    const uint4 *from = pool + (size_t)a.from[k] * words;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (off + i * kCopyThreads < words) v[i] = from[off + i * kCopyThreads];
    for (int r = k; r < end; ++r) {
      uint4 *to = pool + (size_t)a.to[r] * words;
#pragma unroll
      for (int i = 0; i < kCopyUnroll; ++i)
        if (off + i * kCopyThreads < words) to[off + i * kCopyThreads] = v[i];
    }
  }
  if (!renumber) return;
  const size_t entries = (size_t)a.rows * a.max_pages;
  bool bad = false;
  for (size_t e = (size_t)blockIdx.x * kCopyThreads + threadIdx.x; e < entries; e += (size_t)gridDim.x * kCopyThreads) {
    int p = a.table[e];
    if (p >= 0) {
      const int q = p < a.num_pages ? a.list[p] : -1;
      if (q < 0) bad = true;
      else p = q;
    }
    a.table_out[e] = p;
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) report(a, ST_INDEX);
}

template <int N> size_t bits_bytes(const PagesArgs &a) {
  return (size_t)((a.num_pages + N * 128 - 1) / (N * 128)) * 128 / 8;
}
template <int N, typename K> cudaError_t launch_n(K kernel, const PagesArgs &a, bool pool, cudaStream_t s) {
  const size_t smem = pool ? bits_bytes<N>(a) : 0;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = N;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(N);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = N > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
// One CTA where its 32 warps can take a row of the list each and the pool's
// counts are a few loads per thread; both sides measured on a B200 with 1 row
// of 16 and 2048 pages: free and reserve 10.7 us together, 15.8 on the cluster.
template <typename K1, typename K8>
cudaError_t launch_book(K1 one, K8 many, const PagesArgs &a, bool pool, cudaStream_t s) {
  return a.n <= kWarps && a.num_pages <= 16384 ? launch_n<1>(one, a, pool, s) : launch_n<kMost>(many, a, pool, s);
}
cudaError_t launch_move(const PagesArgs &a, const int *copies, bool renumber, cudaStream_t s) {
  return pdl_launch(pages_move_kernel, 8 * kSMs, kCopyThreads, 0, s, a, copies, renumber ? 1 : 0);
}

}  // namespace
}  // namespace paged

cudaError_t launch_pages_reserve(const PagesArgs &a, cudaStream_t s) {
  return paged::launch_book(paged::pages_reserve_kernel<1>, paged::pages_reserve_kernel<paged::kMost>, a, true, s);
}
cudaError_t launch_pages_free(const PagesArgs &a, cudaStream_t s) {
  return paged::launch_book(paged::pages_free_kernel<1>, paged::pages_free_kernel<paged::kMost>, a, false, s);
}
cudaError_t launch_pages_fork(const PagesArgs &a, cudaStream_t s) {
  const cudaError_t e =
      paged::launch_book(paged::pages_fork_kernel<1>, paged::pages_fork_kernel<paged::kMost>, a, true, s);
  if (e != cudaSuccess) return e;
  return paged::launch_move(a, a.count + paged::kMost, false, s);
}
cudaError_t launch_pages_compact(const PagesArgs &a, cudaStream_t s) {
  const cudaError_t e =
      paged::launch_book(paged::pages_compact_kernel<1>, paged::pages_compact_kernel<paged::kMost>, a, true, s);
  if (e != cudaSuccess) return e;
  return paged::launch_move(a, a.count + 3 * paged::kMost, true, s);
}

}  // namespace lz
