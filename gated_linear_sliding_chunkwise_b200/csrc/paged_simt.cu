// Paged attention in fp32 on the CUDA cores: every sequence of the batch, any
// supported size, fp32 or bf16 activations.
//
// One pass over the keys with the running maximum and sum of the softmax.  An
// item is up to 64 rows (token, head of the group), a tile 64 keys.  128
// threads as 8 x 16: a thread holds 8 rows x 4 keys of the logits and 8 rows x
// D / 16 columns of the output.  It is bound by shared-memory reads (a 16-byte
// read takes four cycles of the SM's one port) and then by the FMA pipe, hence
// the tall blocks (12 reads for 128 products; 4 x 4 blocks, 8 for 64, took
// 50 of 102 K cycles for them alone) and the two products per instruction:
// pairs of dimensions in the first product, pairs of columns in the second.
// fp32 keys and values come by cp.async into padded rows, each while the other
// is in use, and the CTAs of an SM cover the rest of the latency.
//
// The tensor cores were tried for fp32, each operand as two tf32 numbers and
// three products (m16n8k8): no faster, and 1.7e-6 off the 64-bit result where
// this is 4e-7 off, because the tensor cores cut what they accumulate.
#include "paged.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kRows = kSimtRows, kKeys = 64, kThreads = 128;

template <int D> struct SimtSmem {
  float q[kRows][D + 4];
  float k[kKeys][D + 4];
  float v[kKeys][D + 4];
  float p[kKeys / 2][kRows + 4];   // weights [key][row], half a tile at a time
  int page[2][kKeys];              // page of each key of a tile, -1: no row sees it
};

LZ_DEV float4 load4(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(x.x, x.y, y.x, y.y);
}
// Four elements of a pool row into shared memory; zeros where there is no row.
LZ_DEV void put4(float *to, const float *from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(there ? 16 : 0)
               : "memory");
}
LZ_DEV void put4(float *to, const __nv_bfloat16 *from, bool there) {
  *reinterpret_cast<float4 *>(to) = there ? load4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
}
LZ_DEV void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> LZ_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) paged_simt_kernel(PagedArgs a, int tok) {
  constexpr int C = D / 16;                 // output columns per thread, in groups of four 64 apart
  extern __shared__ __align__(16) unsigned char raw[];
  SimtSmem<D> &sm = *reinterpret_cast<SimtSmem<D> *>(raw);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Partial part{a.part_o[1], reinterpret_cast<float2 *>(a.part_ml[1])};
  const float sc = a.scale * kLog2e;
  JoinItem item{};
  for (Cursor<kKeys> cur(a, planned(a, 1), tok, blockIdx.x); cur.valid(); cur.next()) {
    const Piece &p = cur.p;
    item = cur.join_item();
    const int rows = (p.i1 - p.i0) * a.g, base = p.q.s - p.q.n;
    // keys that some row of the item may see
    const int end = base + p.i1, low = a.window > 0 ? base + p.i0 - a.window + 1 : 0;
    const auto look = [&](int j) {
      if (tid < kKeys && j < p.j1) {
        const int key = tile_index(p.t, j) * kKeys + tid;
        sm.page[j & 1][tid] =
            key < end && (key >= low || key < a.sinks) ? page_id(a, a.status, p.q.row, key >> a.shift) : -1;
      }
    };
    const auto fetch = [&](int j, float(*to)[D + 4], const void *pool) {
      if (j < p.j1) {
        const int k0 = tile_index(p.t, j) * kKeys;
        const int c = tid % (D / 4) * 4;
#pragma unroll
        for (int i = 0; i < kKeys * (D / 4) / kThreads; ++i) {
          const int r = tid / (D / 4) + i * (kThreads / (D / 4)), id = sm.page[j & 1][r];
          const T *from = static_cast<const T *>(pool);
          if (id >= 0) from += ((((size_t)id * a.Hkv + p.h) << a.shift) + ((k0 + r) & (a.page - 1))) * D + c;
          put4(&to[r][c], from, id >= 0);
        }
      }
      cp_commit();
    };
    __syncthreads();                        // the last piece's reads
    look(p.j0);
    {
      const int c = tid % (D / 4) * 4;
      const T *from = static_cast<const T *>(a.q) + ((size_t)(p.q.t0 + p.i0) * a.H + p.h * a.g) * D + c;
#pragma unroll
      for (int i = 0; i < kRows * (D / 4) / kThreads; ++i) {
        const int r = tid / (D / 4) + i * (kThreads / (D / 4));
        put4(&sm.q[r][c], r < rows ? from + ((size_t)(token_of(a, r)) * a.H + head_of(a, r)) * D : from, r < rows);
      }
    }
    __syncthreads();
    fetch(p.j0, sm.k, a.k_pages);
    fetch(p.j0, sm.v, a.v_pages);
    float2 acc[8][C / 2];
    float m[8], l[8];
    int pos[8];                             // position of each row's token; -1: no row
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = ty * 8 + i;
      pos[i] = r < rows ? base + p.i0 + token_of(a, r) : -1;
      m[i] = kNoKey;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C / 2; ++c) acc[i][c] = make_float2(0.f, 0.f);
    }
    const bool busy = (tid >> 5) * 16 < rows;   // some row of this warp is one of the item's
    const int first = base + p.i0, last = base + p.i1 - 1;
    for (int j = p.j0; j < p.j1; ++j) {
      const int k0 = tile_index(p.t, j) * kKeys;
      look(j + 1);
      cp_wait<1>();                         // K of this tile
      __syncthreads();
      float s[8][4];                        // keys tx, tx + 16, tx + 32, tx + 48
      if (busy) {
        float2 s2[8][4];                    // even and odd dimensions
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s2[i][e] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int c = 0; c < D; c += 4) {
          float4 kk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) kk[e] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * e][c]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(&sm.q[ty * 8 + i][c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s2[i][e] = fma2(make_float2(q.x, q.y), make_float2(kk[e].x, kk[e].y), s2[i][e]);
              s2[i][e] = fma2(make_float2(q.z, q.w), make_float2(kk[e].z, kk[e].w), s2[i][e]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = s2[i][e].x + s2[i][e].y;
      }
      __syncthreads();                      // K has been read
      fetch(j + 1, sm.k, a.k_pages);
      if (busy) {
        const bool all = k0 + kKeys - 1 <= first && (a.window == 0 || k0 > last - a.window || k0 + kKeys - 1 < a.sinks);
        // m is moved, with shuffles over the row's 16 threads, only when some
        // maximum has grown by more than 2^8 since it was set
        float top[8];
        bool grown = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top[i] = kNoKey;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][e] = all || sees(a, pos[i], k0 + tx + 16 * e) ? s[i][e] * sc : -INFINITY;
            top[i] = fmaxf(top[i], s[i][e]);
          }
          grown = grown || top[i] > m[i] + 8.f;
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
            const float mx = fmaxf(m[i], top[i]), f = ex2(m[i] - mx);
            m[i] = mx;
            l[i] *= f;
#pragma unroll
            for (int c = 0; c < C / 2; ++c) acc[i][c].x *= f, acc[i][c].y *= f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][e] = ex2(s[i][e] - m[i]);
            l[i] += s[i][e];                // of this thread's keys
          }
      }
      cp_wait<1>();                         // V of this tile (K of the next may be under way)
      __syncthreads();
      if (busy) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {       // a row's weights are written and read by one half-warp
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
              *reinterpret_cast<float4 *>(&sm.p[tx + 16 * e][ty * 8 + i]) =
                  make_float4(s[i][2 * h + e], s[i + 1][2 * h + e], s[i + 2][2 * h + e], s[i + 3][2 * h + e]);
          __syncwarp();
#pragma unroll 4
          for (int y = 0; y < kKeys / 2; ++y) {
            const float4 p0 = *reinterpret_cast<const float4 *>(&sm.p[y][ty * 8]);
            const float4 p1 = *reinterpret_cast<const float4 *>(&sm.p[y][ty * 8 + 4]);
            const float pv[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int c = 0; c < C; c += 4) {
              const float4 v = *reinterpret_cast<const float4 *>(&sm.v[h * (kKeys / 2) + y][c * 16 + tx * 4]);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 pp = make_float2(pv[i], pv[i]);
                acc[i][c / 2] = fma2(pp, make_float2(v.x, v.y), acc[i][c / 2]);
                acc[i][c / 2 + 1] = fma2(pp, make_float2(v.z, v.w), acc[i][c / 2 + 1]);
              }
            }
          }
        }
      }
      __syncthreads();                      // V has been read
      fetch(j + 1, sm.v, a.v_pages);
    }
    cp_wait<0>();
    if (!busy) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = ty * 8 + i;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      bool fine = isfinite(l[i]);
#pragma unroll
      for (int c = 0; c < C / 2; ++c) fine = fine && isfinite(acc[i][c].x) && isfinite(acc[i][c].y);
      if (r < rows) {
        const size_t at = p.slot >= 0 ? (size_t)p.slot * kRows + r
                                      : (size_t)(p.q.t0 + p.i0 + token_of(a, r)) * a.H + p.h * a.g + head_of(a, r);
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          const size_t o = at * D + (c / 4) * 64 + tx * 4 + c % 4;
          const float2 v = acc[i][c / 2];
          if (p.slot >= 0) {
            *reinterpret_cast<float2 *>(part.o + o) = v;
          } else {
            static_cast<T *>(a.o)[o] = from_f32<T>(l[i] == 0.f ? 0.f : v.x * inv);
            static_cast<T *>(a.o)[o + 1] = from_f32<T>(l[i] == 0.f ? 0.f : v.y * inv);
          }
        }
        if (tx == 0) {
          if (p.slot >= 0) part.ml[at] = make_float2(m[i], l[i]);
          else if (a.lse) a.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
        }
      }
      const unsigned odd = __ballot_sync(0xffffffffu, r < rows && !fine);
      if (odd) __syncwarp();                // such a row is written a second time, by other lanes
      for (int half = 0; half < 2; ++half)
        if (odd & (0xffffu << (16 * half)))
          exact_row_write<T, D>(a, a.status, Piece(p), kKeys, ((tid >> 5) * 2 + half) * 8 + i, part, kRows);
    }
  }
  if (tid == 0) a.items[1][blockIdx.x] = item;
}

template <typename T, int D>
cudaError_t launch(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  static SmemOnce once;
  const cudaError_t e = once(reinterpret_cast<const void *>(paged_simt_kernel<T, D>), sizeof(SimtSmem<D>));
  if (e != cudaSuccess) return e;
  return pdl_launch(paged_simt_kernel<T, D>, g.ctas[1], kThreads, sizeof(SimtSmem<D>), s, a, g.tok[1]);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_simt(const PagedArgs &a, const PagedGeometry &g, bool bf16, cudaStream_t s) {
  if (bf16) return a.d == 64 ? paged::launch<__nv_bfloat16, 64>(a, g, s) : paged::launch<__nv_bfloat16, 128>(a, g, s);
  return a.d == 64 ? paged::launch<float, 64>(a, g, s) : paged::launch<float, 128>(a, g, s);
}

}  // namespace lz
