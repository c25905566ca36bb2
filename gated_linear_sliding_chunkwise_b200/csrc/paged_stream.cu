// Paged attention for sequences with at most 16 rows per key/value head
// (decoding, a few tokens at a time), bf16.
//
// Bound by reading the cache: every key and value is used by at most 16 rows,
// 16 operations per byte.  So the kernel keeps loads in flight: a producer
// warp fetches tiles of 64 keys (32 KB of K and V at d = 128) by TMA into a
// ring of 3 (d = 128) or 6 stages, two CTAs per SM, which is 192 KB under way
// per SM where about 45 KB cover the latency at full bandwidth.  The products
// run on warp-level mma.sync m16n8k16: a tcgen05 tile has 128 rows, of which
// 112 or more would be empty here, and its round trip through TMEM would be
// longer than the 16 + 32 products that each of the four consumer warps needs
// per tile.  A warp takes 16 of the tile's keys in the first product and D / 4
// of the columns in the second, with the maxima and the weights handed over
// in shared memory (two barriers of 128 threads a tile): no warp holds another
// sum for the same output, so a piece ends without a join of the warps, which
// took 4.6 us of a call with one token.
//
// The weights' product with the values is taken twice, with a weight's bf16
// rounding and with what that leaves (also in bf16): the tensor pipe has the
// time (20% busy with one product), and the output's error is that of its own
// rounding, 1.66e-3 of it, where weights of one bf16 number gave 2.27e-3.  64
// decoding sequences 353 -> 349 us, one token 11.9 us as before.
//
// A call that only has such sequences, at most kAlone of them, needs no kernel
// before this one (ALONE): each CTA checks the batch and splits the work for
// itself in shared memory, and the CTA that holds a new token's tile puts its
// key and value into the page and into the tile it has just loaded (no other
// CTA reads that head's rows there).  One token at 517 keys: 13.7 -> 11.2 us.
#include "paged_tma.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kKeys = 64, kWarps = 4, kThreads = (kWarps + 1) * 32;

template <int D> constexpr int stages() { return D == 128 ? 3 : 6; }
template <int D> constexpr uint32_t tile_bytes() { return kKeys * D * 2; }   // K or V
template <int D> struct StreamSmem {
  unsigned char kv[stages<D>()][2][tile_bytes<D>()];   // 64-column regions of 64 rows, 128-byte swizzle
  unsigned char p[2][kStreamRows * 128];               // weights in two bf16 parts [row][key], 128-byte swizzle
  float m[kWarps][kStreamRows], l[kWarps][kStreamRows];
  long long prefix[kAlone + 1], warp_sums[kWarps + 1];   // the work, where there is no prep
  Seq seqs[kAlone];
  uint64_t full[stages<D>()], empty[stages<D>()];
  uint32_t dead, found, odd;                           // odd: some row is not finite
};

LZ_DEV uint32_t kv_offset(int row, int chunk) {   // 16-byte chunk of a row
  return (chunk >> 3) * (kKeys * 128) + tc::sw128_offset(row, (chunk & 7) * 8);
}
LZ_DEV void ldmatrix4(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
LZ_DEV void ldmatrix4_t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
LZ_DEV void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The batch's checks and the prefix of its tiles, by the whole CTA.
template <int D> LZ_DEV Work find_work(const PagedArgs &a, StreamSmem<D> &sm, int least) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    long long tiles = 0;
    if (b < a.B) {
      bool bad;
      const Seq q = check_seq(a, b, &bad);
      if (bad) atomicOr(&sm.found, ST_INDEX);
      sm.seqs[b] = q;
      if (q.n > 0) tiles = (long long)tiles_of<kKeys>(a, q, 0, q.n).count * a.Hkv;
    }
    long long x = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm.warp_sums[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
      if (w < warp) before += sm.warp_sums[w];
      all += sm.warp_sums[w];
    }
    if (b < a.B) sm.prefix[b] = total + before + x - tiles;
    total += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) sm.prefix[a.B] = total;
  __syncthreads();
  return Work{sm.prefix, sm.seqs, Split{total, share_of(total, gridDim.x, least)}};
}

template <int D>
__device__ void produce(const PagedArgs &a, const Work &work, const CUtensorMap *kmap, const CUtensorMap *vmap,
                        StreamSmem<D> &sm, const Waits &wait) {
  constexpr int S = stages<D>();
  const int lane = threadIdx.x & 31;
  const int box = min(a.page, 64), boxes = kKeys / box, per = boxes * (D / 64);
  int it = 0;
  for (Cursor<kKeys> cur(a, work, kStreamRows, blockIdx.x); cur.valid(); cur.next()) {
    const Piece &p = cur.p;
    const Range range(a, p);
    // lane i < 2 per loads box x of half `half` of K (i < per) or V
    const int x = lane % per % boxes, half = lane % per / boxes;
    const bool mine = lane < 2 * per;
    int row = mine ? box_row(a, wait.status, p, range, tile_index(p.t, p.j0) * kKeys + x * box, box) : 0;
    for (int j = p.j0; j < p.j1; ++j, ++it) {
      const int st = it % S;
      if (it >= S) wait(&sm.empty[st], (it / S - 1) & 1);
      if (*wait.dead) return;
      if (lane == 0) tc::mbar_expect_tx(&sm.full[st], 2 * tile_bytes<D>());
      __syncwarp();
      if (mine)
        tc::tma_load_3d(sm.kv[st][lane / per] + half * (kKeys * 128) + x * box * 128, lane < per ? kmap : vmap,
                        &sm.full[st], half * 64, row, 0);
      __syncwarp();                    // no lane runs ahead into the next wait, which would hold the others up
      if (mine && j + 1 < p.j1) row = box_row(a, wait.status, p, range, tile_index(p.t, j + 1) * kKeys + x * box, box);
    }
  }
}

template <int D, bool ALONE>
__device__ void consume(const PagedArgs &a, const Work &work, StreamSmem<D> &sm, const Waits &wait) {
  constexpr int S = stages<D>(), KS = D / 16, NT = D / 8 / kWarps;   // NT: 8-column blocks of this warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Partial part{a.part_o[0], reinterpret_cast<float2 *>(a.part_ml[0])};
  const float sc = a.scale * kLog2e;
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;       // fragment rows r0, r0 + 8; columns c0, c0 + 1
  int it = 0;
  JoinItem item{};
  for (Cursor<kKeys> cur(a, work, kStreamRows, blockIdx.x); cur.valid(); cur.next()) {
    const Piece &p = cur.p;
    item = cur.join_item();
    const Range range(a, p);
    const int rows = (p.i1 - p.i0) * a.g, base = p.q.s - p.q.n;
    uint32_t qf[KS][4];
    int pos[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = r0 + 8 * x;
      pos[x] = r < rows ? base + p.i0 + token_of(a, r) : -1;
      const uint32_t *q = reinterpret_cast<const uint32_t *>(
          static_cast<const __nv_bfloat16 *>(a.q) +
          ((size_t)(p.q.t0 + p.i0 + (r < rows ? token_of(a, r) : 0)) * a.H + p.h * a.g + (r < rows ? head_of(a, r) : 0)) * D + c0);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][x] = r < rows ? q[k * 8] : 0u;
        qf[k][2 + x] = r < rows ? q[k * 8 + 4] : 0u;
      }
    }
    float o[NT][4], m[2] = {kNoKey, kNoKey}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    const int first_pos = base + p.i0, last_pos = base + p.i1 - 1;
    for (int j = p.j0; j < p.j1; ++j, ++it) {
      const int st = it % S, k0 = tile_index(p.t, j) * kKeys, kw = k0 + warp * 16;   // this warp's first key
      wait(&sm.full[st], (it / S) & 1);
      const uint32_t ka = tc::smem_u32(sm.kv[st][0]), va = tc::smem_u32(sm.kv[st][1]);
      if (!range.whole(kw, 16)) {
        // values that no row sees may be anything: their weight is zero, so make them zero
        for (int x = lane; x < 16 * (D / 8); x += 32)
          if (!range.any(kw + x / (D / 8)))
            *reinterpret_cast<uint4 *>(sm.kv[st][1] + kv_offset(warp * 16 + x / (D / 8), x % (D / 8))) =
                make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async();       // before the stage is loaded again
      }
      if (ALONE && a.k && kw + 16 > max(base, 0) && kw < p.q.s) {
        // new tokens among this warp's keys: into their page and over what was loaded for them
        for (int j = max(kw, max(base, 0)); j < min(kw + 16, p.q.s); ++j) {
          constexpr int L = D / 8;               // 16-byte pieces of a row
          const size_t from = ((size_t)(p.q.t0 + j - base) * a.Hkv + p.h) * L;
          const int id = a.table[(size_t)p.q.row * a.max_pages + (j >> a.shift)];
          const size_t to = ((((size_t)id * a.Hkv + p.h) << a.shift) + (j & (a.page - 1))) * L;
          const bool there = (unsigned)id < (unsigned)a.num_pages;   // the producer reports it where it is not
          for (int x = lane; x < 2 * L; x += 32) {
            const bool v = x >= L;
            const int c = v ? x - L : x;
            const uint4 u = static_cast<const uint4 *>(v ? a.v : a.k)[from + c];
            *reinterpret_cast<uint4 *>(sm.kv[st][v] + kv_offset(j - k0, c)) = u;
            if (there) static_cast<uint4 *>(v ? a.v_pages : a.k_pages)[to + c] = u;
          }
        }
        tc::fence_proxy_async();       // before the stage is loaded again
        __syncwarp();
      }
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t b[4];
          ldmatrix4(ka + kv_offset(warp * 16 + n * 8 + (lane & 7), k * 2 + (lane >> 3)), b);
          mma16816(s[n], qf[k], b[0], b[1]);
          mma16816(s[n], qf[k + 1], b[2], b[3]);
        }
      }
      const bool all = kw + 15 <= first_pos && (a.window == 0 || kw > last_pos - a.window || kw + 15 < a.sinks);
      float mn[2] = {kNoKey, kNoKey};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[n][e] * sc;
          if (!all && !sees(a, pos[e >> 1], kw + n * 8 + c0 + (e & 1))) x = -INFINITY;
          s[n][e] = x;
          mn[e >> 1] = fmaxf(mn[e >> 1], x);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mn[x] = fmaxf(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], 1));
        mn[x] = fmaxf(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], 2));
        if ((lane & 3) == 0) sm.m[warp][r0 + 8 * x] = mn[x];
      }
      // every warp has read the last tile's maxima and weights
      tc::bar_sync(1, kWarps * 32);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mn[x] = m[x];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mn[x] = fmaxf(mn[x], sm.m[w][r0 + 8 * x]);
        const float f = ex2(m[x] - mn[x]);
        m[x] = mn[x];
        l[x] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][2 * x] *= f, o[n][2 * x + 1] *= f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float w0 = ex2(s[n][2 * x] - m[x]), w1 = ex2(s[n][2 * x + 1] - m[x]);
          l[x] += w0 + w1;
          // a weight goes to the second product as two bf16 numbers, which are off by at most 2^-16 of it
          const uint32_t hi = tc::pack_bf16(w0, w1);
          const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&hi));
          const uint32_t at = tc::sw128_offset(r0 + 8 * x, warp * 16 + n * 8 + c0);
          *reinterpret_cast<uint32_t *>(sm.p[0] + at) = hi;
          *reinterpret_cast<uint32_t *>(sm.p[1] + at) = tc::pack_bf16(w0 - h.x, w1 - h.y);
        }
      }
      tc::bar_sync(1, kWarps * 32);
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k) {
        uint32_t pf[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
          ldmatrix4(tc::smem_u32(sm.p[x]) + tc::sw128_offset(lane & 15, k * 16 + (lane >> 4) * 8), pf[x]);
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          ldmatrix4_t(va + kv_offset(k * 16 + (lane & 15), warp * NT + n + (lane >> 4)), b);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma16816(o[n], pf[x], b[0], b[1]);
            mma16816(o[n + 1], pf[x], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.empty[st]);
      __syncwarp();
    }
    // the sum over the warps' keys; the output's columns are this warp's own
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if ((lane & 3) == 0) sm.l[warp][r0 + 8 * x] = l[x];
    }
    tc::bar_sync(1, kWarps * 32);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = r0 + 8 * x;
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += sm.l[w][r];
      bool fine = isfinite(ll);
#pragma unroll
      for (int n = 0; n < NT; ++n) fine = fine && isfinite(o[n][2 * x]) && isfinite(o[n][2 * x + 1]);
      if (r >= rows) continue;
      if (!fine) sm.odd = 1;
      if (p.slot >= 0) {
        const size_t at = (size_t)p.slot * kStreamRows + r;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2 *>(part.o + at * D + (warp * NT + n) * 8 + c0) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
        if (warp == 0 && (lane & 3) == 0) part.ml[at] = make_float2(m[x], ll);
      } else {
        const size_t at = (size_t)(p.q.t0 + p.i0 + token_of(a, r)) * a.H + p.h * a.g + head_of(a, r);
        const float inv = inverse_sum(ll);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + (warp * NT + n) * 8 + c0) =
              tc::pack_bf16(o[n][2 * x] * inv, o[n][2 * x + 1] * inv);
        if (a.lse && warp == 0 && (lane & 3) == 0) a.lse[at] = ll == 0.f ? -INFINITY : (m[x] + log2f(ll)) * kLn2;
      }
    }
  }
  if (threadIdx.x == 0) a.items[0][blockIdx.x] = item;
}

template <int D, bool ALONE>
__global__ void __launch_bounds__(kThreads, 2)
    paged_stream_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int least) {
  constexpr int S = stages<D>();
  extern __shared__ unsigned char raw[];
  StreamSmem<D> &sm = *reinterpret_cast<StreamSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], kWarps);
    }
    sm.dead = sm.found = sm.odd = 0;
    tc::fence_barrier_init();
  }
  __syncthreads();
  if (!ALONE) {
    pdl_wait();
    gpu_fence();   // for the tile kernel, which starts on the triggers
  }
  pdl_trigger();
  const Waits wait{&sm.dead, ALONE ? &sm.found : a.status};
  const Work work = ALONE ? find_work<D>(a, sm, least) : planned(a, 0);
  if (warp == kWarps) produce<D>(a, work, &kmap, &vmap, sm, wait);
  else consume<D, ALONE>(a, work, sm, wait);
  __syncthreads();
  if (sm.odd) exact_rows<__nv_bfloat16, D, kKeys>(a, wait.status, work, kStreamRows, 0, kStreamRows);
  if (ALONE) {
    __syncthreads();
    if (threadIdx.x == 0) a.found[blockIdx.x] = sm.found;
  }
}

template <int D> cudaError_t launch(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  if (!make_pool_map(&kmap, a.k_pages, a) || !make_pool_map(&vmap, a.v_pages, a)) return cudaErrorInvalidValue;
  const size_t smem = sizeof(StreamSmem<D>) + 1024;
  static SmemOnce once, once_alone;
  if (!g.alone) {
    const cudaError_t e = once(reinterpret_cast<const void *>(paged_stream_kernel<D, false>), smem);
    if (e != cudaSuccess) return e;
    return pdl_launch(paged_stream_kernel<D, false>, g.ctas[0], kThreads, smem, s, a, kmap, vmap, g.least[0]);
  }
  const cudaError_t e = once_alone(reinterpret_cast<const void *>(paged_stream_kernel<D, true>), smem);
  if (e != cudaSuccess) return e;
  paged_stream_kernel<D, true><<<g.ctas[0], kThreads, smem, s>>>(a, kmap, vmap, g.least[0]);
  return cudaGetLastError();
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_stream(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  return a.d == 64 ? paged::launch<64>(a, g, s) : paged::launch<128>(a, g, s);
}

}  // namespace lz
