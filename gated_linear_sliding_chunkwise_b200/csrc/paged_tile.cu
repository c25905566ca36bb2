// Paged attention for sequences with more than 16 rows per key/value head
// (chunks of prompts), bf16, on tcgen05.
//
// A CTA holds two 128-row query tiles of one (sequence, key/value head): rows
// are (token, head of the group), so 128 / g tokens per tile.  Each tile has
// its warpgroup for its rows' softmax (thread = row = TMEM lane); one warp
// loads, one issues the products.  Per tile of 128 keys:
//
//   load    K, V by TMA, a page (or 64 rows of it) per box, into a ring of
//           tile-sized slots
//   MMA     S_q = Q_q K^T                       (128 x 128, TMEM)
//   rows    P_q = 2^(S scale log2 e - m) in bf16, over S_q's own columns,
//           64 keys at a time; sums in fp32 from the unrounded weights
//   MMA     O_q (+)= P_q V                      (128 x d, TMEM)
//
// The products of one query tile run while the other's rows are in the
// softmax: PV_0(j), QK_0(j+1), PV_1(j), QK_1(j+1), the first half of PV(j) as
// soon as the first half of P(j) is there.  S_q(j+1) is issued after PV_q(j),
// so the barrier that announces S_q(j+1) also says that O_q is complete up to
// j.
//
// The weights of a tile are formed with the m there is, while the tile's
// maximum is found: they need not stay below 1, since bf16 and fp32 have the
// range.  When the maximum has passed m by 2^8, m is moved before the next
// tile and O rescaled in TMEM.  A row whose maximum rises by more than 2^96
// within one tile could overflow: it is computed again, exactly, at the end.
//
// The weights' product takes them rounded to bf16 (half a step, 2^-8 of each),
// with which the output is 2.3e-3 of it off, 1.7e-3 of that its own rounding.
// As two bf16 numbers each, like the streaming kernel's, they cost nothing in
// accuracy, but the second product and the splitting are on the chain that
// bounds this kernel: 8192 tokens of a 16K prompt 1.58 -> 2.12 ms, prompt
// chunks of four users 141 -> 172 us.
//
// What it took (8192 tokens of a 16K prompt, 32 heads on 8): 1.91 ms with a
// maximum before the weights and the products issued by lane 0 (their
// descriptors then go through vector registers, 120 cycles per product
// instead of 64); 1.62 ms with an elected lane; 1.53 to 1.60 ms as it is now
// (several B200s), 1.03 to 1.07 PFLOP/s, 63 to 65% of the measured bf16 rate.
// Tried and left out: one S for both query tiles, so that QK_q(j+1)
// need not wait for PV_q(j) (1.63 ms: all 128 logits of a row then have to be
// in registers at once); sixteen softmax warps (1.55 ms, but a mixed batch 20%
// slower); an issuing warp for each query tile (1.70 ms: the two tiles'
// products interleave and both softmaxes wait); exp2 on the FMA pipe for a
// part of the weights (slower at any share).
//
// Bound by the chain softmax -> PV -> QK -> softmax of a query tile, which the
// other tile covers only in part: per 128 keys 3.65 K cycles, of which 1.6 K
// form the weights (16384 of them take at least 1024 cycles of the exp2 unit),
// 1.1 K wait for the products (at least 1024 cycles at d = 128; QK reads 128
// bytes of shared memory per cycle, all there is) and 0.9 K go into barriers,
// loads from TMEM and the tile's bookkeeping.
#include "paged_tma.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kKeys = 128, kThreads = 320;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;   // S_x (and P_x), O_x at 128 x from there
constexpr float kSlack = 8.f, kRange = 96.f;      // log2 of the weights from which m is moved, and of the largest

template <int D> constexpr uint32_t tile_bytes() { return 128 * D * 2; }
template <int D> constexpr int slots() { return 5; }   // two and a half tiles of K and V (10 at d = 64: no faster)
template <int D> struct TileSmem {
  unsigned char q[2][tile_bytes<D>()];
  unsigned char kv[slots<D>()][tile_bytes<D>()];  // K, V, K, V, ...
  uint64_t q_full, q_empty, kv_full[slots<D>()], kv_empty[slots<D>()], s_full[2], p_full[2][2], o_full[2];
  uint32_t tmem, dead, odd;                       // odd: some row is not finite
};

// One lane of a converged warp.  The issuing branches go by this and not by
// the lane's number: the compiler then knows that one thread is in them and
// keeps the products' descriptors in uniform registers.
LZ_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// 32 lanes x 32-bit, 32 consecutive columns per thread.
LZ_DEV void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Tokens of query tile x of a piece: [i0 + x tpt, ...), `rows` rows.
struct Half {
  int first, tokens, rows;
  LZ_DEV Half(const PagedArgs &a, const Piece &p, int tpt, int x) {
    first = p.i0 + x * tpt;
    tokens = max(0, min(tpt, p.i1 - first));
    rows = tokens * a.g;
  }
};

template <int D>
__device__ void produce(const PagedArgs &a, const CUtensorMap *qmap, const CUtensorMap *kmap, const CUtensorMap *vmap,
                        TileSmem<D> &sm, const Waits &wait, int tpt) {
  constexpr int S = slots<D>();
  const int lane = threadIdx.x & 31;
  // K or V tile: lane < per loads box x of 64-column half `half`
  const int box = min(a.page, 64), boxes = kKeys / box, per = boxes * (D / 64);
  const int x = lane % boxes, half = lane / boxes;
  const bool mine = lane < per;
  int it = 0, pieces = 0;
  for (Cursor<kKeys> cur(a, planned(a, 1), 2 * tpt, blockIdx.x); cur.valid(); cur.next(), ++pieces) {
    const Piece &p = cur.p;
    const Range range(a, p);
    if (pieces > 0) wait(&sm.q_empty, (pieces - 1) & 1);
    if (*wait.dead) return;
    if (lane == 0) {
      const int halves = p.i0 + tpt < p.i1 ? 2 : 1;
      tc::mbar_expect_tx(&sm.q_full, halves * tpt * a.g * D * 2);
      for (int h = 0; h < halves; ++h)
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_3d(sm.q[h] + c * tc::kReg, qmap, &sm.q_full, c * 64, p.h * a.g, p.q.t0 + p.i0 + h * tpt);
    }
    __syncwarp();
    int row = mine ? box_row(a, a.status, p, range, tile_index(p.t, p.j0) * kKeys + x * box, box) : 0;
    for (int j = p.j0; j < p.j1; ++j) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++it) {
        const int st = it % S;
        if (it >= S) wait(&sm.kv_empty[st], (it / S - 1) & 1);
        if (*wait.dead) return;
        if (lane == 0) tc::mbar_expect_tx(&sm.kv_full[st], tile_bytes<D>());
        __syncwarp();
        if (mine)
          tc::tma_load_3d(sm.kv[st] + half * tc::kReg + x * box * 128, kv ? vmap : kmap, &sm.kv_full[st], half * 64,
                          row, 0);
        __syncwarp();
      }
      if (mine && j + 1 < p.j1) row = box_row(a, a.status, p, range, tile_index(p.t, j + 1) * kKeys + x * box, box);
    }
  }
}

template <int D>
__device__ void multiply(const PagedArgs &a, TileSmem<D> &sm, const Waits &wait, uint32_t tmem, int tpt) {
  constexpr int S = slots<D>();
  constexpr uint32_t id_s = tc::idesc_bf16(128, 128, 0, 0), id_o = tc::idesc_bf16(128, D, 0, 1);
  uint32_t it = 0, pieces = 0, np[2] = {0, 0};
  // One lane issues; the others stay with it (__syncwarp): lanes that ran ahead
  // into the next wait would keep the warp in it and hold that lane up.
  const auto qk = [&](int x, uint32_t k) {
    if (elect_one()) {
      const uint32_t q = tc::smem_u32(sm.q[x]), kk = tc::smem_u32(sm.kv[k % S]);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        tc::mma_ss(tmem + kColS + x * 128, tc::desc_k(q, s), tc::desc_k(kk, s), id_s, s > 0);
      tc::mma_commit(&sm.s_full[x]);
    }
    __syncwarp();
  };
  const auto full = [&](uint32_t k) {
    wait(&sm.kv_full[k % S], (k / S) & 1);
    tc::tc_fence_after();
  };
  const auto release = [&](uint64_t *bar) {
    if (elect_one()) tc::mma_commit(bar);
    __syncwarp();
  };
  for (Cursor<kKeys> cur(a, planned(a, 1), 2 * tpt, blockIdx.x); cur.valid(); cur.next(), ++pieces) {
    const Piece &p = cur.p;
    const int halves = p.i0 + tpt < p.i1 ? 2 : 1, n = p.j1 - p.j0;
    wait(&sm.q_full, pieces & 1);
    full(it);
    for (int x = 0; x < halves; ++x) qk(x, it);
    release(&sm.kv_empty[it % S]);
    if (n == 1) release(&sm.q_empty);
    for (int j = 0; j < n; ++j, it += 2) {
      const bool more = j + 1 < n;
      if (*wait.dead) return;                 // no products over what did not arrive
      full(it + 1);
      if (more) full(it + 2);
      const uint32_t v = tc::smem_u32(sm.kv[(it + 1) % S]);
      for (int x = 0; x < halves; ++x) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wait(&sm.p_full[x][h], np[x] & 1);
          tc::tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int s = 4 * h; s < 4 * h + 4; ++s)
              tc::mma_ts(tmem + kColO + x * 128, tmem + kColS + x * 128 + s * 8, tc::desc_mn(v, s), id_o,
                         j > 0 || s > 0);
            if (h == 1 && !more) tc::mma_commit(&sm.o_full[x]);
          }
          __syncwarp();
        }
        ++np[x];
        if (more) qk(x, it + 2);
      }
      release(&sm.kv_empty[(it + 1) % S]);
      if (more) release(&sm.kv_empty[(it + 2) % S]);
      if (j + 2 == n) release(&sm.q_empty);
    }
  }
}

template <int D>
__device__ void softmax(const PagedArgs &a, TileSmem<D> &sm, const Waits &wait, uint32_t tmem, int tpt) {
  constexpr int S = slots<D>(), C = 64;       // columns at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = warp >> 2;
  const int wrow = (warp & 3) * 32, row = wrow + lane;
  const uint32_t lanes = (uint32_t)wrow << 16;
  const uint32_t ts = tmem + lanes + kColS + x * 128, to = tmem + lanes + kColO + x * 128;
  const Partial part{a.part_o[1], reinterpret_cast<float2 *>(a.part_ml[1])};
  const float sc = a.scale * kLog2e;
  uint32_t it = 0, ns = 0, no = 0;
  JoinItem item{};
  for (Cursor<kKeys> cur(a, planned(a, 1), 2 * tpt, blockIdx.x); cur.valid(); cur.next()) {
    const Piece &p = cur.p;
    item = cur.join_item();
    const Half hf(a, p, tpt, x);
    const int n = p.j1 - p.j0;
    if (hf.rows == 0) {
      it += 2 * n;
      continue;
    }
    const Range range(a, p);
    const int base = p.q.s - p.q.n, first = base + hf.first, last = first + hf.tokens - 1;
    const int pos = row < hf.rows ? first + token_of(a, row) : -1;
    const bool live = row < hf.rows, busy = wrow < hf.rows;   // this row, some row of the warp is one of the item's
    // tiles within [clear0, clear1) need no mask here and no zeroed values
    const int clear0 = a.window > 0 ? last - a.window + 1 : 0, clear1 = base + p.i0 + 1;
    int k0 = tile_index(p.t, p.j0) * kKeys;
    float m = kNoKey, l = 0.f, top = kNoKey;  // top: the largest logit so far
    for (int j = 0; j < n; ++j, it += 2) {
      if (j > 0) k0 = p.j0 + j == p.t.nsink ? p.t.first * kKeys : k0 + kKeys;
      const bool clear = k0 >= clear0 && k0 + kKeys <= clear1;
      if (x == 0 && !range.whole(k0, kKeys)) {
        // Values that no row sees may be anything: their weight is zero, so make
        // them zero.  The first query tile's warps do it for both: their weights
        // are waited for before either product with V.  (The second's must not:
        // they pass over pieces that have no rows for them, and a wait for a slot
        // so far ahead of its loads would take an earlier load for this one.)
        const uint32_t v = it + 1;
        wait(&sm.kv_full[v % S], (v / S) & 1);
        for (int e = threadIdx.x & 127; e < kKeys * (D / 8); e += 128)
          if (!range.any(k0 + e / (D / 8)))
            *tc::chunk_ptr(sm.kv[v % S], 0, e / (D / 8), e % (D / 8)) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async();
      }
      const int hi = pos - k0, lo = a.window > 0 ? hi - a.window : INT_MIN, sk = a.window > 0 ? a.sinks - k0 : 0;
      float s[C];
      const auto load = [&](int c) {
        tc::tmem_ld32x2(ts + c, ts + c + 32, s, s + 32);
        if (!clear) {
#pragma unroll
          for (int e = 0; e < C; ++e)
            if (!(c + e <= hi && (c + e > lo || c + e < sk))) s[e] = -INFINITY;
        }
      };
      const auto raise = [&]() {              // top over these columns
        float mx[2] = {s[0], s[1]};
#pragma unroll
        for (int e = 2; e < C; e += 2) mx[e >> 1 & 1] = fmaxf(fmaxf(mx[e >> 1 & 1], s[e]), s[e + 1]);
        top = fmaxf(top, fmaxf(mx[0], mx[1]) * sc);
      };
      wait(&sm.s_full[x], ns++ & 1);
      tc::tc_fence_after();
      if (busy) {
        // Only rows of the item are asked (the others' logits come from what
        // shared memory held before, and what is moved for one row shows in the
        // last bits of its neighbours).
        // a row sees its first keys
        if (__any_sync(0xffffffffu, live && m == kNoKey && hi >= 0 && (lo < kKeys - 1 || sk > 0))) {
          load(0);
          raise();
          load(C);
          raise();
        }
        if (__any_sync(0xffffffffu, live && top > m + kSlack)) {
          const float mn = fmaxf(m, top), f = ex2(m - mn);     // f = 0 at the first key
          m = mn;
          l *= f;
          if (j > 0) {
            float o[16];
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              tc::tmem_ld16(to + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tc::tmem_st8(to + c, reinterpret_cast<const uint32_t *>(o));
              tc::tmem_st8(to + c + 8, reinterpret_cast<const uint32_t *>(o + 8));
            }
          }
        }
      }
      const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (busy) {
          load(h * C);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float mx[2] = {s[0], s[1]};
          uint32_t pk[C / 2];
#pragma unroll
          for (int e = 0; e < C; e += 2) {
            if (e > 0) mx[e >> 1 & 1] = fmaxf(fmaxf(mx[e >> 1 & 1], s[e]), s[e + 1]);
            float2 w = fma2(make_float2(s[e], s[e + 1]), sc2, m2);
            w = make_float2(ex2(w.x), ex2(w.y));
            sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], w);
            // weights go to the second product in bf16 (see the top); the sum keeps 32 bits
            pk[e / 2] = tc::pack_bf16(w.x, w.y);
          }
          tmem_st32(ts + h * (C / 2), pk);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          top = fmaxf(top, fmaxf(mx[0], mx[1]) * sc);
          tc::tmem_st_wait();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.p_full[x][h]);
        __syncwarp();
      }
      if (top > m + kRange) l = NAN;
    }
    wait(&sm.o_full[x], no++ & 1);
    tc::tc_fence_after();
    if (!busy) continue;
    // out: 32 columns at a time, unnormalised sums for a split item
    const int r = x * tpt * a.g + row;
    const size_t at = p.slot >= 0 ? (size_t)p.slot * kTileRows2 + r
                                  : (size_t)(p.q.t0 + p.i0 + token_of(a, r)) * a.H + p.h * a.g + head_of(a, r);
    const float inv = inverse_sum(l);
    bool fine = isfinite(l);
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tc::tmem_ld32(to + c, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) fine = fine && isfinite(o[e]);
      if (!live) continue;
      if (p.slot >= 0) {
        float4 *out = reinterpret_cast<float4 *>(part.o + at * D + c);
#pragma unroll
        for (int e = 0; e < 32; e += 4) out[e / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + c);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
#pragma unroll
        for (int e = 0; e < 32; e += 8) out[e / 8] = tc::pack8(o + e);
      }
    }
    if (live) {
      if (p.slot >= 0) part.ml[at] = make_float2(m, l);
      else if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    if (live && !fine) sm.odd = 1;
    tc::tc_fence_before();
  }
  if (threadIdx.x == 0) a.items[1][blockIdx.x] = item;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int tpt, int beside) {
  constexpr int S = slots<D>();
  extern __shared__ __align__(1024) unsigned char raw[];
  TileSmem<D> &sm = *reinterpret_cast<TileSmem<D> *>(raw);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(&sm.kv_full[i], 1);
      tc::mbar_init(&sm.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i][0], 4);
      tc::mbar_init(&sm.p_full[i][1], 4);
      tc::mbar_init(&sm.o_full[i], 1);
    }
    sm.dead = sm.odd = 0;
    tc::fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // Beside the streaming kernel this one does not wait for it.  What it reads
  // are the prep kernel's split and pages: each CTA of the streaming kernel lets
  // this kernel start only after its own wait for the prep kernel, which has
  // then completed with its writes visible, and a fence on either side of the
  // start (there before the trigger, here) carries that over.  The start itself
  // is what the two fences meet at: that a kernel's CTAs run after the triggers
  // that let them start is how the launch works, not an order that the memory
  // model names.  CTAs take over SM by SM as the streaming kernel's leave (a
  // batch of 44 decoding and 4 chunked sequences: 54.4 -> 48.2 us; SMs set apart
  // for each of the two by their work: 58), and they wait for that kernel at
  // their end, so that the join, which waits for this one, follows both.
  if (beside) gpu_fence();
  else pdl_wait();
  pdl_trigger();
  const uint32_t tmem = sm.tmem;
  const Waits wait{&sm.dead, a.status};
  if (warp < 8) softmax<D>(a, sm, wait, tmem, tpt);
  else if (warp == 8) produce<D>(a, &qmap, &kmap, &vmap, sm, wait, tpt);
  else multiply<D>(a, sm, wait, tmem, tpt);
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 9) tc::tmem_dealloc(tmem, kTmemCols);
  if (sm.odd) exact_rows<__nv_bfloat16, D, kKeys>(a, a.status, planned(a, 1), 2 * tpt, 1, kTileRows2);
  if (beside) pdl_wait();
}

// q [T][H][d]: a box is 64 columns x the g heads of a group x tpt tokens.
bool make_query_map(CUtensorMap *map, const PagedArgs &a, int tpt) {
  tc::EncodeTiledFn fn = tc::encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.T};
  const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.H * a.d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)tpt}, estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D> cudaError_t launch(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  CUtensorMap qmap, kmap, vmap;
  const int tpt = g.tok[1] / 2;
  if (!make_query_map(&qmap, a, tpt) || !make_pool_map(&kmap, a.k_pages, a) || !make_pool_map(&vmap, a.v_pages, a))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(TileSmem<D>);
  static_assert(sizeof(TileSmem<D>) <= 232448, "227 KB of shared memory per CTA");
  static SmemOnce once;
  const cudaError_t e = once(reinterpret_cast<const void *>(paged_tile_kernel<D>), smem);
  if (e != cudaSuccess) return e;
  return pdl_launch(paged_tile_kernel<D>, g.ctas[1], kThreads, smem, s, a, qmap, kmap, vmap, tpt, g.ctas[0] > 0 ? 1 : 0);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_tile(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  return a.d == 64 ? paged::launch<64>(a, g, s) : paged::launch<128>(a, g, s);
}

}  // namespace lz
