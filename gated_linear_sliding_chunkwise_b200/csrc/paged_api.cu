// Host side of the paged cache's entry points (include/lizard.h): argument
// checks, workspace layout, choice of kernels.
#include <limits.h>
#include <math.h>

#include "../../include/lizard.h"
#include "lizard_internal.h"

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kHeader = 256;   // status word region at the workspace start
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool ok_ptr(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename P> P *at(void *base, size_t off) { return reinterpret_cast<P *>(static_cast<char *>(base) + off); }
// Whether [x, x + n) and [y, y + m) share a byte.
bool overlap(const void *x, size_t n, const void *y, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + m && b < a + n;
}
lizard_status cuda_status(cudaError_t e) { return e == cudaSuccess ? LIZARD_OK : LIZARD_ERR_CUDA; }

// Sizes of the pool and the table.
lizard_status check_pool(int num_pages, int page, int rows, int max_pages) {
  if (num_pages < 1 || rows < 1 || max_pages < 1 || page < 1) return LIZARD_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return LIZARD_ERR_UNSUPPORTED;
  if (num_pages > (1 << 22) || (long long)rows * max_pages > INT_MAX || (long long)max_pages * page > (1 << 30))
    return LIZARD_ERR_UNSUPPORTED;
  return LIZARD_OK;
}
lizard_status check_contents(int layers, int num_pages, int Hkv, int page, int d, int dtype) {
  if (layers < 1 || Hkv < 1 || d < 1) return LIZARD_ERR_INVALID_ARG;
  if (dtype != LIZARD_BF16 && dtype != LIZARD_FP32) return LIZARD_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return LIZARD_ERR_UNSUPPORTED;
  if ((long long)num_pages * Hkv * page > INT_MAX) return LIZARD_ERR_UNSUPPORTED;
  return LIZARD_OK;
}

lizard_status check_sizes(const lizard_paged_args *a) {
  if (!a) return LIZARD_ERR_INVALID_ARG;
  if (a->B < 0 || a->T < 0 || a->H < 1 || a->max_q < 0 || a->window < 0 || a->sinks < 0) return LIZARD_ERR_INVALID_ARG;
  lizard_status st = check_pool(a->num_pages, a->page, a->rows, a->max_pages);
  if (st != LIZARD_OK) return st;
  st = check_contents(a->layers, a->num_pages, a->Hkv, a->page, a->d, a->dtype);
  if (st != LIZARD_OK) return st;
  if (a->layer < 0 || a->layer >= a->layers || a->H % a->Hkv != 0) return LIZARD_ERR_INVALID_ARG;
  if (a->impl < LIZARD_IMPL_AUTO || a->impl > LIZARD_IMPL_TC) return LIZARD_ERR_INVALID_ARG;
  if (!(a->softmax_scale >= 0.f) || !isfinite(a->softmax_scale)) return LIZARD_ERR_INVALID_ARG;
  if (a->H / a->Hkv > lz::paged::kMaxGroup) return LIZARD_ERR_UNSUPPORTED;
  if (a->impl == LIZARD_IMPL_TC && a->dtype != LIZARD_BF16) return LIZARD_ERR_UNSUPPORTED;
  return LIZARD_OK;
}

// bf16 on the tensor-core kernels.
bool on_tensor_cores(const lizard_paged_args *a) {
  return a->dtype == LIZARD_BF16 && a->impl != LIZARD_IMPL_SIMT;
}

// The split of the batch over kernels.  bf16: sequences of at most
// kStreamRows rows per key/value head go to the streaming kernel (class 0),
// the others, when the call can have any, to the tile kernel (class 1); fp32
// and impl SIMT: all of them to the portable kernel (class 1).
lz::PagedGeometry choose(const lizard_paged_args *a) {
  lz::PagedGeometry c{};
  const int g = a->H / a->Hkv;
  // Fewest tiles worth a CTA of their own, against the join of one more piece:
  // one token over 9 tiles takes 11.0 us with one as with two; 3 fp32 chunks
  // of 20 tokens 18.5 us with one, 25.9 with two (class 1).
  c.least[0] = 2;
  c.least[1] = 1;
  if (!on_tensor_cores(a)) {
    c.kt[0] = c.kt[1] = 64;
    c.tok[0] = c.tok[1] = lz::paged::kSimtRows / g;
    c.ctas[1] = lz::paged::kSimtCtas;
    c.slot_rows[1] = lz::paged::kSimtRows;
    return c;
  }
  c.few = lz::paged::kStreamRows;
  c.kt[0] = 64;
  c.tok[0] = lz::paged::kStreamRows;
  if (g <= c.few) {
    c.ctas[0] = lz::paged::kStreamCtas;
    c.slot_rows[0] = lz::paged::kStreamRows;
  }
  c.kt[1] = 128;
  c.tok[1] = 2 * (lz::paged::kTileRows2 / 2 / g);
  if ((long long)a->max_q * g > c.few) {
    c.ctas[1] = lz::paged::kTileCtas;
    c.slot_rows[1] = lz::paged::kTileRows2;
  } else {
    c.alone = a->B <= lz::paged::kAlone;
  }
  return c;
}

struct PagedLayout {
  size_t split, prefix, seqs, found, items[2], part_o[2], part_ml[2], total;
};
PagedLayout paged_layout(const lizard_paged_args *a, const lz::PagedGeometry &c) {
  PagedLayout l{};
  size_t off = kHeader;
  l.split = off; off += up(2 * 2 * sizeof(long long));
  l.prefix = off; off += up(2 * ((size_t)a->B + 1) * sizeof(long long));
  l.seqs = off; off += up((size_t)a->B * 4 * sizeof(int));
  l.found = off; off += up((size_t)c.ctas[0] * sizeof(uint32_t));
  for (int x = 0; x < 2; ++x) {
    l.items[x] = off; off += up((size_t)c.ctas[x] * 4 * sizeof(int));
    const size_t rows = 2 * (size_t)c.ctas[x] * c.slot_rows[x];
    l.part_o[x] = off; off += up(rows * a->d * sizeof(float));
    l.part_ml[x] = off; off += up(rows * 2 * sizeof(float));
  }
  l.total = off;
  return l;
}

}  // namespace

extern "C" {

size_t lizard_paged_attn_workspace_size(const lizard_paged_args *a) {
  if (check_sizes(a) != LIZARD_OK) return 0;
  return paged_layout(a, choose(a)).total;
}

lizard_status lizard_paged_attn(const lizard_paged_args *a, lizard_stream_t stream) {
  const lizard_status st = check_sizes(a);
  if (st != LIZARD_OK) return st;
  if ((a->k != nullptr) != (a->v != nullptr)) return LIZARD_ERR_INVALID_ARG;
  const bool some = a->T > 0 && a->B > 0;
  if (some && (!a->q || !a->k_pages || !a->v_pages || !a->table || !a->lens || !a->cu_q || !a->o || a->max_q < 1))
    return LIZARD_ERR_INVALID_ARG;
  const size_t row_bytes = (size_t)a->T * a->d * (a->dtype == LIZARD_BF16 ? 2 : 4);
  for (const void *x : {a->q, a->k, a->v}) {
    // a key or value is read before the output of its own token and head is
    // written: with as many of them as query heads, o may be k or v itself
    const bool itself = x != a->q && x == a->o && a->H == a->Hkv;
    if (some && x && !itself && overlap(a->o, row_bytes * a->H, x, row_bytes * (x == a->q ? a->H : a->Hkv)))
      return LIZARD_ERR_INVALID_ARG;
  }
  const void *ptrs[] = {a->q, a->k, a->v, a->k_pages, a->v_pages, a->table, a->lens, a->cu_q, a->row,
                        a->o, a->lse, a->workspace};
  for (const void *p : ptrs)
    if (!ok_ptr(p)) return LIZARD_ERR_INVALID_ARG;
  const lz::PagedGeometry c = choose(a);
  const PagedLayout lay = paged_layout(a, c);
  if (!a->workspace || a->workspace_bytes < lay.total) return LIZARD_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *ws = a->workspace;
  if (!some) return cuda_status(cudaMemsetAsync(ws, 0, sizeof(uint32_t), s));
  const bool bf16 = a->dtype == LIZARD_BF16;
  const size_t layer = (size_t)a->layer * a->num_pages * a->Hkv * a->page * a->d * (bf16 ? 2 : 4);
  lz::PagedArgs p{};
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.k_pages = at<void>(a->k_pages, layer); p.v_pages = at<void>(a->v_pages, layer);
  p.table = a->table; p.lens = a->lens; p.cu_q = a->cu_q; p.row = a->row;
  p.o = a->o; p.lse = a->lse;
  p.num_pages = a->num_pages; p.Hkv = a->Hkv; p.page = a->page; p.d = a->d;
  while (1 << p.shift < a->page) ++p.shift;
  p.rows = a->rows;
  p.max_pages = a->max_pages; p.B = a->B; p.T = a->T; p.H = a->H; p.g = a->H / a->Hkv;
  p.ginv = 65536 / p.g + 1;
  p.max_q = a->max_q;
  // lengths stay below 2^30: a wider window or more first tokens are all of them
  p.window = a->window < (1 << 30) ? a->window : 1 << 30;
  p.sinks = a->sinks < (1 << 30) ? a->sinks : 1 << 30;
  p.scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.f / sqrtf((float)a->d);
  p.status = static_cast<uint32_t *>(ws);
  p.split = at<lz::paged::Split>(ws, lay.split);
  p.prefix = at<long long>(ws, lay.prefix);
  p.seqs = at<lz::paged::Seq>(ws, lay.seqs);
  p.found = at<uint32_t>(ws, lay.found);
  for (int x = 0; x < 2; ++x) {
    p.items[x] = at<lz::paged::JoinItem>(ws, lay.items[x]);
    p.part_o[x] = at<float>(ws, lay.part_o[x]);
    p.part_ml[x] = at<float>(ws, lay.part_ml[x]);
  }
  if (!c.alone && lz::launch_paged_prep(p, c, bf16, s) != cudaSuccess) return LIZARD_ERR_CUDA;
  if (c.ctas[0] && lz::launch_paged_stream(p, c, s) != cudaSuccess) return LIZARD_ERR_CUDA;
  if (c.ctas[1] &&
      (on_tensor_cores(a) ? lz::launch_paged_tile(p, c, s) : lz::launch_paged_simt(p, c, bf16, s)) != cudaSuccess)
    return LIZARD_ERR_CUDA;
  return cuda_status(lz::launch_paged_join(p, c, bf16, s));
}

}  // extern "C"

// ----------------------------------------------------------- bookkeeping ---
namespace {

struct PagesLayout {
  size_t count, mark, need, offset, held, list, from, to, snap, total;
};
PagesLayout pages_layout(const lizard_pages_args *a) {
  PagesLayout l{};
  const size_t n = a->n, P = a->num_pages, most = n > P ? n : P;
  size_t off = kHeader;
  l.count = off; off += up(32 * sizeof(int));
  l.mark = off; off += up((size_t)a->rows * sizeof(int));
  l.need = off; off += up(n * sizeof(int));
  l.offset = off; off += up(n * sizeof(int));
  l.held = off; off += up(most * sizeof(int));
  l.list = off; off += up(P * sizeof(int));
  l.from = off; off += up(most * sizeof(int));
  l.to = off; off += up(most * sizeof(int));
  l.snap = off; off += up(n * a->max_pages * sizeof(int));
  l.total = off;
  return l;
}

lizard_status check_pages(const lizard_pages_args *a) {
  if (!a || a->n < 0) return LIZARD_ERR_INVALID_ARG;
  const lizard_status st = check_pool(a->num_pages, a->page, a->rows, a->max_pages);
  if (st != LIZARD_OK) return st;
  return a->n > a->rows ? LIZARD_ERR_INVALID_ARG : LIZARD_OK;   // the rows are all different
}

enum class Op { reserve, free, fork, compact };

lizard_status run_pages(const lizard_pages_args *a, Op op, lizard_stream_t stream) {
  lizard_status st = check_pages(a);
  if (st != LIZARD_OK) return st;
  const bool contents = op == Op::fork || op == Op::compact, list = op != Op::compact;
  if (contents) {
    st = check_contents(a->layers, a->num_pages, a->Hkv, a->page, a->d, a->dtype);
    if (st != LIZARD_OK) return st;
  }
  if (!a->table || !a->refs || (contents && (!a->k_pages || !a->v_pages))) return LIZARD_ERR_INVALID_ARG;
  if (list && (!a->lens || (a->n > 0 && !a->row))) return LIZARD_ERR_INVALID_ARG;
  if (a->n > 0 && ((op == Op::reserve && !a->grow) || (op == Op::fork && !a->src))) return LIZARD_ERR_INVALID_ARG;
  if (op == Op::compact && (!a->table_out || !a->refs_out)) return LIZARD_ERR_INVALID_ARG;
  const void *ptrs[] = {a->k_pages, a->v_pages, a->refs, a->table, a->lens, a->row, a->src, a->grow,
                        a->table_out, a->refs_out, a->workspace};
  for (const void *p : ptrs)
    if (!ok_ptr(p)) return LIZARD_ERR_INVALID_ARG;
  const PagesLayout lay = pages_layout(a);
  if (!a->workspace || a->workspace_bytes < lay.total) return LIZARD_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *ws = a->workspace;
  if (list && a->n == 0) return cuda_status(cudaMemsetAsync(ws, 0, sizeof(uint32_t), s));
  lz::PagesArgs p{};
  p.layers = a->layers; p.num_pages = a->num_pages; p.page = a->page; p.rows = a->rows;
  p.max_pages = a->max_pages; p.n = list ? a->n : 0;   // without a list, n has no say in the kernel's choice
  p.page_bytes = contents ? (size_t)a->Hkv * a->page * a->d * (a->dtype == LIZARD_BF16 ? 2 : 4) : 0;
  p.k_pages = a->k_pages; p.v_pages = a->v_pages;
  p.refs = a->refs; p.table = a->table; p.lens = a->lens;
  p.row = a->row; p.src = a->src; p.grow = a->grow;
  p.table_out = a->table_out; p.refs_out = a->refs_out;
  p.status = static_cast<uint32_t *>(ws);
  p.count = at<int>(ws, lay.count); p.mark = at<int>(ws, lay.mark); p.need = at<int>(ws, lay.need);
  p.offset = at<int>(ws, lay.offset); p.held = at<int>(ws, lay.held); p.list = at<int>(ws, lay.list);
  p.from = at<int>(ws, lay.from); p.to = at<int>(ws, lay.to); p.snap = at<int>(ws, lay.snap);
  switch (op) {
    case Op::reserve: return cuda_status(lz::launch_pages_reserve(p, s));
    case Op::free: return cuda_status(lz::launch_pages_free(p, s));
    case Op::fork: return cuda_status(lz::launch_pages_fork(p, s));
    case Op::compact: return cuda_status(lz::launch_pages_compact(p, s));
  }
  return LIZARD_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

size_t lizard_pages_workspace_size(const lizard_pages_args *a) {
  return check_pages(a) == LIZARD_OK ? pages_layout(a).total : 0;
}
lizard_status lizard_pages_reserve(const lizard_pages_args *a, lizard_stream_t s) { return run_pages(a, Op::reserve, s); }
lizard_status lizard_pages_free(const lizard_pages_args *a, lizard_stream_t s) { return run_pages(a, Op::free, s); }
lizard_status lizard_pages_fork(const lizard_pages_args *a, lizard_stream_t s) { return run_pages(a, Op::fork, s); }
lizard_status lizard_pages_compact(const lizard_pages_args *a, lizard_stream_t s) { return run_pages(a, Op::compact, s); }

}  // extern "C"
