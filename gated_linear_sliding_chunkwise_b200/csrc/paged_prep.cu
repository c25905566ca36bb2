// Paged attention, before and after the attention kernels: the batch's checks
// and the split of its work, the new tokens' way into their pages, and the
// join of split items.
#include "paged.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kPrepThreads = 512;

template <int KT>
LZ_DEV int item_tiles(const PagedArgs &a, const Seq &q, int tok, int it) {
  const int i0 = it * tok;
  return tiles_of<KT>(a, q, i0, min(i0 + tok, q.n)).count;
}
LZ_DEV int item_tiles_kt(const PagedArgs &a, const Seq &q, int kt, int tok, int it) {
  return kt == 64 ? item_tiles<64>(a, q, tok, it) : item_tiles<128>(a, q, tok, it);
}

// CTA 0.  Latency-bound (a few dependent loads and one block scan): a thread
// takes one sequence; a sequence of many items is summed by its whole warp.
__device__ void split_batch(const PagedArgs &a, const PagedGeometry &g) {
  __shared__ long long warp_sums[2][kPrepThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long base[2] = {0, 0};
  bool any_bad = false;
  for (int b0 = 0; b0 < a.B; b0 += kPrepThreads) {
    const int b = b0 + threadIdx.x;
    Seq q{};
    bool bad = false;
    if (b < a.B) {
      q = check_seq(a, b, &bad);
      a.seqs[b] = q;
    }
    any_bad |= bad;
    const int cls = few_rows(a, q.n, g.few) ? 0 : 1;
    const int nitem = q.n > 0 ? (q.n + g.tok[cls] - 1) / g.tok[cls] : 0;
    long long tiles = 0;
    if (nitem <= 4)
      for (int it = 0; it < nitem; ++it) tiles += item_tiles_kt(a, q, g.kt[cls], g.tok[cls], it);
    for (unsigned many = __ballot_sync(0xffffffffu, nitem > 4); many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      Seq w;
      w.n = __shfl_sync(0xffffffffu, q.n, l);
      w.s = __shfl_sync(0xffffffffu, q.s, l);
      const int wc = __shfl_sync(0xffffffffu, cls, l), wn = __shfl_sync(0xffffffffu, nitem, l);
      long long sum = 0;
      for (int it = lane; it < wn; it += 32) sum += item_tiles_kt(a, w, g.kt[wc], g.tok[wc], it);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == l) tiles = sum;
    }
    tiles *= a.Hkv;
    long long v[2] = {cls == 0 ? tiles : 0, cls == 1 ? tiles : 0}, inc[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      long long x = v[c];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      inc[c] = x;
      if (lane == 31) warp_sums[c][warp] = x;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      long long before = 0, all = 0;
      for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) before += warp_sums[c][w];
        all += warp_sums[c][w];
      }
      if (b < a.B) a.prefix[(size_t)c * (a.B + 1) + b] = base[c] + before + inc[c] - v[c];
      base[c] += all;
    }
    __syncthreads();
  }
  const int bad = __syncthreads_or(any_bad);
  if (threadIdx.x == 0) {
    *a.status = bad ? ST_INDEX : 0u;
    for (int c = 0; c < 2; ++c) {
      a.prefix[(size_t)c * (a.B + 1) + a.B] = base[c];
      a.split[c].total = base[c];
      a.split[c].share = share_of(base[c], g.ctas[c] > 0 ? g.ctas[c] : 1, g.least[c]);
    }
  }
}

// 16 bytes of one new token's k and v per thread.
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(PagedArgs a, PagedGeometry g, int row_chunks) {
  pdl_trigger();
  if (blockIdx.x == 0) {
    split_batch(a, g);
    return;
  }
  const size_t idx = (size_t)(blockIdx.x - 1) * kPrepThreads + threadIdx.x;
  const size_t per = (size_t)a.Hkv * row_chunks;
  if (idx >= a.T * per) return;
  const int t = (int)(idx / per), rest = (int)(idx % per);
  int lo = 0;
  if (t < a.B && a.cu_q[t] == t && a.cu_q[t + 1] == t + 1) {
    lo = t;                                    // one token per sequence
  } else {
    int hi = a.B;                              // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
  }
  const Seq q = check_seq(a, lo);
  const int i = t - q.t0;
  if (i < 0 || i >= q.n) return;               // between or behind the sequences
  const int p = q.s - q.n + i;
  if (p < 0) return;
  const int id = a.table[(size_t)q.row * a.max_pages + (p >> a.shift)];
  if ((unsigned)id >= (unsigned)a.num_pages) return;   // the attention kernels report it
  const int h = rest / row_chunks, c = rest % row_chunks;
  const size_t to = ((((size_t)id * a.Hkv + h) << a.shift) + (p & (a.page - 1))) * row_chunks + c;
  static_cast<uint4 *>(a.k_pages)[to] = static_cast<const uint4 *>(a.k)[idx];
  static_cast<uint4 *>(a.v_pages)[to] = static_cast<const uint4 *>(a.v)[idx];
}

// Joins a split item's pieces: o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// over the CTAs that the item spans, in order.  `parts` blocks take the item
// that begins in CTA `first`'s stretch, if one does, and go over its rows with
// their warps; a lane takes D / 32 columns.
template <typename T, int D>
__device__ void join(const PagedArgs &a, const PagedGeometry &g, int cls, int first, int part, int parts) {
  constexpr int E = D / 32;
  const int slot_rows = g.slot_rows[cls];
  const JoinItem d = a.items[cls][first];
  const int lane = threadIdx.x & 31;
  const float *po = a.part_o[cls];
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml[cls]);
  for (int r = part * 8 + (threadIdx.x >> 5); r < d.rows; r += parts * 8) {
    float m = kNoKey, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int x = first; x <= d.last; ++x) {
      const size_t at = (size_t)(x == first ? 2 * x + 1 : 2 * x) * slot_rows + r;
      const float2 v = ml[at];
      const float mn = v.x > m ? v.x : m;
      const float fo = ex2(m - mn), fn = ex2(v.x - mn);
      l = l * fo + v.y * fn;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * fo + po[at * D + lane * E + e] * fn;
      m = mn;
    }
    const size_t at = (size_t)(d.token + token_of(a, r)) * a.H + d.head + head_of(a, r);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
      static_cast<T *>(a.o)[at * D + lane * E + e] = from_f32<T>(l == 0.f ? 0.f : acc[e] * inv);
    if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// Blocks of an item of a class: 16 rows each (two per warp: the join waits for
// its loads, so more blocks beat one wave of larger ones: 64 rows each took
// 13 us longer on prompt chunks of four users).
LZ_DEV __host__ int join_parts(const PagedGeometry &g, int cls) { return (g.slot_rows[cls] + 15) / 16; }

// First the blocks of class 0, then those of class 1.  (The
// last CTA's stretch begins no item that goes on.)
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedArgs a, PagedGeometry g) {
  pdl_wait();
  if (g.alone && blockIdx.x == 0) {   // the CTAs' findings make the call's status
    uint32_t st = 0;
    for (int c = threadIdx.x; c < g.ctas[0]; c += 256) st |= a.found[c];
    const int index = __syncthreads_or(st & ST_INDEX), timeout = __syncthreads_or(st & ST_TIMEOUT);
    if (threadIdx.x == 0) *a.status = (index ? ST_INDEX : 0u) | (timeout ? ST_TIMEOUT : 0u);
  }
  int x = blockIdx.x, cls = 0;
  const int few = max(g.ctas[0] - 1, 0) * join_parts(g, 0);
  if (x >= few) {
    x -= few;
    cls = 1;
  }
  const int parts = join_parts(g, cls);
  join<T, D>(a, g, cls, x / parts, x % parts, parts);
}

template <typename T, int D> cudaError_t launch_join(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  int blocks = 0;
  for (int c = 0; c < 2; ++c)
    if (g.ctas[c] > 0) blocks += (g.ctas[c] - 1) * join_parts(g, c);
  return pdl_launch(paged_join_kernel<T, D>, blocks, 256, 0, s, a, g);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_prep(const PagedArgs &a, const PagedGeometry &g, bool bf16, cudaStream_t s) {
  const int row_chunks = a.d * (bf16 ? 2 : 4) / 16;
  const size_t chunks = a.k ? (size_t)a.T * a.Hkv * row_chunks : 0;
  const size_t blocks = 1 + (chunks + paged::kPrepThreads - 1) / paged::kPrepThreads;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  paged::paged_prep_kernel<<<(unsigned)blocks, paged::kPrepThreads, 0, s>>>(a, g, row_chunks);
  return cudaGetLastError();
}

cudaError_t launch_paged_join(const PagedArgs &a, const PagedGeometry &g, bool bf16, cudaStream_t s) {
  if (bf16) return a.d == 64 ? paged::launch_join<__nv_bfloat16, 64>(a, g, s) : paged::launch_join<__nv_bfloat16, 128>(a, g, s);
  return a.d == 64 ? paged::launch_join<float, 64>(a, g, s) : paged::launch_join<float, 128>(a, g, s);
}

}  // namespace lz
