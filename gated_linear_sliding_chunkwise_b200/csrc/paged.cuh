// Paged attention: what its kernels share -- the call's arguments, the split
// of the work over CTAs, page lookup, and the exact row.
//
// Work.  An item is the new tokens [i0, i1) of one (sequence, key/value head)
// with all g = H / Hkv query heads of the group: its rows are (token, head),
// so every key tile that is read serves the whole group.  An item's keys are
// cut into tiles of KT tokens; tiles no row of it sees are not counted.  The
// tiles of all items form one list, in the order (sequence, head, item,
// tile), and CTA c of n takes the stretch [c share, (c + 1) share), whatever
// the lengths are: a long sequence is split over many CTAs and many short
// ones share one.  An item that lies in one CTA's stretch is finished there;
// a CTA keeps the unnormalised sums of an item's piece otherwise (at most two
// pieces per CTA: the item it starts inside and the item it ends inside), and
// a second kernel joins them in tile order.  The split depends on the
// lengths alone, so results do not change from run to run.
#pragma once

#include <float.h>
#include <limits.h>

#include <atomic>

#include "common.cuh"
#include "lizard_internal.h"

namespace lz {
namespace paged {

constexpr uint32_t ST_TIMEOUT = 1u, ST_INDEX = 4u;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoKey = -FLT_MAX;   // running maximum before any key was seen

// ------------------------------------------------ dependent launches ------
// A kernel launched with the programmatic attribute starts while the one
// before it still runs; pdl_wait returns once that one has completed and its
// writes are visible.
LZ_DEV void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// Orders what this thread has seen before it against all that it does after it,
// over the whole GPU, TMA loads included.
LZ_DEV void gpu_fence() { asm volatile("fence.acq_rel.gpu;\nfence.proxy.async;\n" ::: "memory"); }
LZ_DEV void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
// Raises a kernel's shared-memory limit, once per device.
struct SmemOnce {
  std::atomic<bool> done[64] = {};
  cudaError_t operator()(const void *kernel, size_t smem) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
  }
};
template <typename... P, typename... A>
cudaError_t pdl_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// 2^x in one instruction; results below 2^-126 become zero, which a weight may
// lose.
LZ_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
LZ_DEV float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(x)), "l"(reinterpret_cast<uint64_t &>(y)),
        "l"(reinterpret_cast<uint64_t &>(z)));
  return r;
}
LZ_DEV float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(x)), "l"(reinterpret_cast<uint64_t &>(y)));
  return r;
}

// Row r of an item (r < 512) is (token, head of the group): r / g and r mod g
// by a product with ginv = floor(2^16 / g) + 1.
LZ_DEV int token_of(const PagedArgs &a, int r) { return (r * a.ginv) >> 16; }
LZ_DEV int head_of(const PagedArgs &a, int r) { return r - token_of(a, r) * a.g; }

// ------------------------------------------------------------ sequences ---
struct __align__(16) Seq {
  int t0, n, s, row;   // first new token in q, new tokens, length with them, table row
};
// Sequence b of the batch, checked; n = 0 when there is nothing to do or
// something is not allowed (`bad` says so).  The prep kernel keeps the result
// in a.seqs for the kernels after it.
LZ_DEV Seq check_seq(const PagedArgs &a, int b, bool *bad = nullptr) {
  Seq q;
  const int t0 = a.cu_q[b], t1 = a.cu_q[b + 1];
  const int row = a.row ? a.row[b] : b;
  bool ok = t0 >= 0 && t1 >= t0 && t1 <= a.T && t1 - t0 <= a.max_q && row >= 0 && row < a.rows;
  int s = 0;
  if (ok) {
    s = a.lens[row];
    ok = s >= 0 && s <= (long long)a.max_pages * a.page;
  }
  q.t0 = t0;
  q.n = ok ? t1 - t0 : 0;
  q.s = ok ? s : 0;
  q.row = ok ? row : 0;
  if (bad) *bad = !ok;
  return q;
}

// ----------------------------------------------------------- key tiles ----
// Tiles of KT keys that the tokens [i0, i1) of a sequence see: the first
// `nsink` tiles from key 0, then the tiles from `first` on.
struct Tiles {
  int nsink, first, count;
};
template <int KT>
LZ_DEV Tiles tiles_of(const PagedArgs &a, const Seq &q, int i0, int i1) {
  Tiles t;
  const int base = q.s - q.n;
  const int end = max(base + i1, 0);                // keys below this one may be seen
  const int lo = a.window > 0 ? max(base + i0 - a.window + 1, 0) : 0;
  const int nt = (end + KT - 1) / KT;
  t.first = min(lo / KT, nt);
  t.nsink = a.window > 0 ? min((min(a.sinks, end) + KT - 1) / KT, t.first) : 0;
  // an item without any key still has its rows written (as zeros): one tile
  t.count = max(nt - t.first + t.nsink, 1);
  return t;
}
LZ_DEV int tile_index(const Tiles &t, int j) { return j < t.nsink ? j : t.first + (j - t.nsink); }

// Whether the token at position p sees key j.
LZ_DEV bool sees(const PagedArgs &a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}

// Page that holds tokens [pg * page, ...) of a row; -1 (and the status bit)
// when the table's entry is outside the pool.
LZ_DEV int page_id(const PagedArgs &a, uint32_t *status, int row, int pg) {
  int id = -1;
  if (pg < a.max_pages) id = a.table[(size_t)row * a.max_pages + pg];
  if ((unsigned)id >= (unsigned)a.num_pages) {
    atomicOr(status, ST_INDEX);
    id = -1;
  }
  return id;
}

// --------------------------------------------------------------- split ----
// For each class of sequences (class 0: few rows, class 1: the others).
struct Split {
  long long total, share;
};
// The work of a class: prefix[b] = tiles of the sequences before b.  Written
// by the prep kernel, or found by each CTA for itself (streaming kernel).
struct Work {
  const long long *prefix;
  const Seq *seqs;
  Split split;
};
LZ_DEV Work planned(const PagedArgs &a, int cls) {
  return Work{a.prefix + (size_t)cls * (a.B + 1), a.seqs, a.split[cls]};
}
// A CTA's share of `total` tiles over n CTAs.
LZ_DEV long long share_of(long long total, int n, int least) {
  const long long share = total < INT_MAX ? ((unsigned)total + n - 1u) / (unsigned)n : (total + n - 1) / n;
  return share > least ? share : least;
}
struct Piece {
  int b, h, item;        // sequence, key/value head, item within (b, h)
  int i0, i1;            // its tokens
  int j0, j1;            // its tiles in this CTA's stretch
  Seq q;
  Tiles t;
  int slot;              // partial slot, or -1: the piece is the whole item
};

// Whether a sequence of n tokens belongs to class 0 (few rows).
LZ_DEV bool few_rows(const PagedArgs &a, int n, int few) { return n * a.g <= few; }

// Item that begins in CTA c's stretch and goes on in those up to CTA `last`:
// entry c of a.items[class], rows = 0 when there is none.
struct __align__(16) JoinItem {
  int token, head, rows, last;
};

// Walks the pieces of one CTA's stretch.  All lanes of a warp call it
// together (the first search runs across the lanes).
template <int KT>
struct Cursor {
  const PagedArgs &a;
  const long long *prefix;
  const Seq *seqs;
  int tok;               // tokens per item
  long long u, end, share;
  int cta;
  Piece p;
  int nitem;
  // Latency counts here: every CTA starts with it.  The search for the
  // sequence probes 32 places at a time (one step for 32 sequences, two for
  // 1024), and its first probes do not wait for the split.
  LZ_DEV Cursor(const PagedArgs &a_, const Work &work, int tok_, int cta_)
      : a(a_), prefix(work.prefix), seqs(work.seqs), tok(tok_), cta(cta_) {
    const int lane = threadIdx.x & 31;
    int lo = 0, width = a.B;                      // the sequence is one of lo .. lo + width - 1
    int step = (width + 31) / 32;
    long long probe = prefix[min(lane * step, a.B)];
    const Split sp = work.split;
    share = sp.share;
    u = share * cta;
    end = min(u + share, sp.total);
    if (u >= end) return;
    for (;;) {
      // the last probed place that does not lie behind u (empty sequences share a place with the next)
      const unsigned below = __ballot_sync(0xffffffffu, lane * step < width && probe <= u);
      const int l = 31 - __clz(below);
      lo += l * step;
      width = min(step, width - l * step);
      if (width <= 1) break;
      step = (width + 31) / 32;
      probe = prefix[min(lo + lane * step, a.B)];
    }
    p.b = lo;
    const long long before = prefix[lo], all_tiles = prefix[lo + 1] - before;
    open_seq();
    long long rem = u - before;
    if (all_tiles < INT_MAX) {                    // 32-bit division where it does
      const unsigned per = (unsigned)all_tiles / (unsigned)a.Hkv;
      p.h = (unsigned)rem / per;
      rem = (unsigned)rem % per;
    } else {
      const long long per = all_tiles / a.Hkv;
      p.h = (int)(rem / per);
      rem %= per;
    }
    // the item: 32 at a time
    int it = 0;
    if (nitem > 1)
      for (;; it += 32) {
        int c = 0;
        if (it + lane < nitem) {
          const int i0 = (it + lane) * tok;
          c = tiles_of<KT>(a, p.q, i0, min(i0 + tok, p.q.n)).count;
        }
        int pre = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += x;
        }
        const int all = __shfl_sync(0xffffffffu, pre, 31);
        if (rem >= all && it + 32 < nitem) {
          rem -= all;
          continue;
        }
        const unsigned past = __ballot_sync(0xffffffffu, rem < pre);
        const int l = past ? __ffs(past) - 1 : 0;
        rem -= __shfl_sync(0xffffffffu, pre - c, l);
        it += l;
        break;
      }
    p.item = it;
    open_item((int)rem);
  }
  LZ_DEV bool valid() const { return u < end; }
  LZ_DEV void next() {
    u += p.j1 - p.j0;
    if (u >= end) return;
    if (++p.item == nitem) {
      p.item = 0;
      if (++p.h == a.Hkv) {
        p.h = 0;
        do ++p.b;
        while (prefix[p.b + 1] == prefix[p.b]);
        open_seq();
      }
    }
    open_item(0);
  }
  // What the join kernel needs to know of a split item that begins in this
  // CTA's stretch (always its last piece).
  LZ_DEV JoinItem join_item() const {
    JoinItem d{};
    if (p.slot == 2 * cta + 1) {
      d.rows = (p.i1 - p.i0) * a.g;
      d.token = p.q.t0 + p.i0;
      d.head = p.h * a.g;
      d.last = (int)((u + p.t.count - 1) / share);
    }
    return d;
  }

 private:
  LZ_DEV void open_seq() {
    p.q = seqs[p.b];
    nitem = (p.q.n + tok - 1) / tok;
  }
  LZ_DEV void open_item(int j0) {
    p.i0 = p.item * tok;
    p.i1 = min(p.i0 + tok, p.q.n);
    p.t = tiles_of<KT>(a, p.q, p.i0, p.i1);
    p.j0 = j0;
    p.j1 = (int)min((long long)p.t.count, j0 + (end - u));
    p.slot = j0 > 0 ? 2 * cta : p.j1 < p.t.count ? 2 * cta + 1 : -1;
  }
};

// Partial sums of a class: per slot `rows` rows of D fp32 sums, then per row
// (maximum in log2 units, sum).
struct Partial {
  float *o;      // [slots][rows][D]
  float2 *ml;    // [slots][rows]
};

// ------------------------------------------------------------ exact row ---
// One row of a piece, key by key with the mask applied to each: keys the row
// does not see are not touched at all.  The attention kernels multiply masked
// values by a zero weight, which is not zero when such a value is infinite or
// NaN; a row whose result is not finite is computed again here.  One warp;
// lane l gets elements l * D / 32 ...  It stops at a logit that is NaN: every
// element is NaN from there on.
template <typename T, int D>
__device__ __noinline__ void exact_row(const PagedArgs &a, uint32_t *status, const Piece &p, int KT, int r, float *acc,
                                       float &m_out, float &l_out) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int tok = p.i0 + token_of(a, r), head = p.h * a.g + head_of(a, r);
  const int pos = p.q.s - p.q.n + tok;
  const T *q = static_cast<const T *>(a.q) + ((size_t)(p.q.t0 + tok) * a.H + head) * D + lane * E;
  float qv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = to_f32(q[e]), acc[e] = 0.f;
  float m = kNoKey, l = 0.f;
  const float c = a.scale * kLog2e;
  for (int jt = p.j0; jt < p.j1 && !isnan(l); ++jt) {
    const int k0 = tile_index(p.t, jt) * KT;
    for (int j = k0; j < k0 + KT && j <= pos; ++j) {
      if (!sees(a, pos, j)) continue;
      const int id = page_id(a, status, p.q.row, j >> a.shift);
      if (id < 0) continue;
      const size_t at = ((((size_t)id * a.Hkv + p.h) << a.shift) + (j & (a.page - 1))) * D + lane * E;
      const T *k = static_cast<const T *>(a.k_pages) + at;
      const T *v = static_cast<const T *>(a.v_pages) + at;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(qv[e], to_f32(k[e]), s);
      s = warp_sum(s) * c;
      const float mn = s > m ? s : m;
      const float f = exp2f(m - mn), w = exp2f(s - mn);   // f = 0 at the first key
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * to_f32(v[e]);
      m = mn;
      if (isnan(l)) break;
    }
  }
  m_out = m;
  l_out = l;
}

// Recomputes a row and writes it where it belongs: the partial slot, or o and lse.
template <typename T, int D>
__device__ __noinline__ void exact_row_write(const PagedArgs &a, uint32_t *status, const Piece &p, int KT, int r,
                                             const Partial &part, int slot_rows) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float acc[E], m, l;
  exact_row<T, D>(a, status, p, KT, r, acc, m, l);
  if (p.slot >= 0) {
    const size_t at = (size_t)p.slot * slot_rows + r;
#pragma unroll
    for (int e = 0; e < E; ++e) part.o[at * D + lane * E + e] = acc[e];
    if (lane == 0) part.ml[at] = make_float2(m, l);
    return;
  }
  const int tok = p.i0 + token_of(a, r), head = p.h * a.g + head_of(a, r);
  const size_t at = (size_t)(p.q.t0 + tok) * a.H + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) static_cast<T *>(a.o)[at * D + lane * E + e] = from_f32<T>(l == 0.f ? 0.f : acc[e] * inv);
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The rows of a CTA's pieces whose results are not finite, as the kernel has
// written them: computed again, by all warps of the CTA, when its pieces are
// done.  That takes a warp 0.7 us per row and key (1500 tokens of a 16K prompt
// with 16 heads: 0.19 s), so it is not done between pieces: there the CTA's
// other warps are in waits that give up, and the pieces that follow may be
// other users'.  A kernel that calls this leaves something that is not finite
// in what it writes of every such row (an infinite sum of weights would make a
// zero of it).
template <typename T, int D, int KT>
__device__ __noinline__ void exact_rows(const PagedArgs &a, uint32_t *status, const Work &work, int tok, int cls,
                                        int slot_rows) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Partial part{a.part_o[cls], reinterpret_cast<float2 *>(a.part_ml[cls])};
  for (Cursor<KT> cur(a, work, tok, blockIdx.x); cur.valid(); cur.next()) {
    const Piece &p = cur.p;
    for (int r = warp; r < (p.i1 - p.i0) * a.g; r += warps) {
      bool fine = true;
      if (p.slot >= 0) {
        const size_t at = (size_t)p.slot * slot_rows + r;
        fine = isfinite(part.ml[at].y);
#pragma unroll
        for (int e = 0; e < E; ++e) fine = fine && isfinite(part.o[at * D + lane * E + e]);
      } else {
        const size_t at = (size_t)(p.q.t0 + p.i0 + token_of(a, r)) * a.H + p.h * a.g + head_of(a, r);
#pragma unroll
        for (int e = 0; e < E; ++e) fine = fine && isfinite(to_f32(static_cast<const T *>(a.o)[at * D + lane * E + e]));
      }
      if (__any_sync(0xffffffffu, !fine)) exact_row_write<T, D>(a, status, Piece(p), KT, r, part, slot_rows);
    }
  }
}
// 1 / sum of a row's weights: 0 for a row without keys, NaN for a sum that is
// not finite (see exact_rows).
LZ_DEV float inverse_sum(float l) { return !isfinite(l) ? NAN : l == 0.f ? 0.f : 1.f / l; }

}  // namespace paged
}  // namespace lz
