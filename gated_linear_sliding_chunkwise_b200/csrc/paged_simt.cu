// Paged attention in fp32 on the CUDA cores: every sequence of the batch, any
// supported size, fp32 or bf16 activations.
//
// One pass over the keys with the running maximum and sum of the softmax.  An
// item is up to 64 rows (token, head of the group); a tile is 64 keys.  256
// threads as 16 x 16: a thread holds a 4 x 4 block of the logits and 4 rows x
// D / 16 columns of the output, operands come from shared memory as 16-byte
// loads (two per 16 products), so the kernel is bound by the FMA pipe for
// long chunks and by the latency of its loads for few rows.
#include "paged.cuh"

namespace lz {
namespace paged {
namespace {

constexpr int kRows = kSimtRows, kKeys = 64, kPad = 4;

template <int D>
struct SimtSmem {
  float q[D][kRows + kPad];     // transposed
  union {
    float k[D][kKeys + kPad];     // transposed
    float p[kKeys][kRows + kPad]; // transposed weights, once every thread has its logits
  };
  float v[kKeys][D];
  int page[kKeys];              // page of each key, -1: no row sees it
};

template <typename T> LZ_DEV float4 load4(const T *p);
template <> LZ_DEV float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <> LZ_DEV float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(x.x, x.y, y.x, y.y);
}

template <typename T, int D>
__global__ void __launch_bounds__(256, 2) paged_simt_kernel(PagedArgs a, int tok) {
  constexpr int C = D / 16;                 // output columns per thread, in pairs of float4 64 columns apart
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
    __syncthreads();                        // the last piece's reads of q
    for (int x = tid; x < kRows * D / 4; x += 256) {
      const int r = x % kRows, c = x / kRows * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = load4(static_cast<const T *>(a.q) +
                  ((size_t)(p.q.t0 + p.i0 + r / a.g) * a.H + p.h * a.g + r % a.g) * D + c);
      sm.q[c][r] = v.x, sm.q[c + 1][r] = v.y, sm.q[c + 2][r] = v.z, sm.q[c + 3][r] = v.w;
    }
    float acc[4][C], m[4], l[4];
    int pos[4];                             // position of each row's token; -1: no row
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      pos[i] = r < rows ? base + p.i0 + r / a.g : -1;
      m[i] = kNoKey;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[i][c] = 0.f;
    }
    // keys that some row of the item may see
    const int end = base + p.i1, low = a.window > 0 ? base + p.i0 - a.window + 1 : 0;
    for (int jt = p.j0; jt < p.j1; ++jt) {
      const int k0 = tile_index(p.t, jt) * kKeys;
      __syncthreads();                      // the last tile's reads
      if (tid < kKeys) {
        const int j = k0 + tid;
        sm.page[tid] = j < end && (j >= low || j < a.sinks) ? page_id(a, a.status, p.q.row, j / a.page) : -1;
      }
      __syncthreads();
      for (int x = tid; x < kKeys * D / 4; x += 256) {
        const int j = x % kKeys, c = x / kKeys * 4, id = sm.page[j];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (id >= 0)
          v = load4(static_cast<const T *>(a.k_pages) +
                    (((size_t)id * a.Hkv + p.h) * a.page + (k0 + j) % a.page) * D + c);
        sm.k[c][j] = v.x, sm.k[c + 1][j] = v.y, sm.k[c + 2][j] = v.z, sm.k[c + 3][j] = v.w;
      }
      for (int x = tid; x < kKeys * D / 4; x += 256) {
        const int j = x / (D / 4), c = x % (D / 4) * 4, id = sm.page[j];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (id >= 0)
          v = load4(static_cast<const T *>(a.v_pages) +
                    (((size_t)id * a.Hkv + p.h) * a.page + (k0 + j) % a.page) * D + c);
        *reinterpret_cast<float4 *>(&sm.v[j][c]) = v;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
      for (int c = 0; c < D; ++c) {
        const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[c][ty * 4]);
        const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[c][tx * 4]);
        const float qv[4] = {q4.x, q4.y, q4.z, q4.w}, kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = fmaf(qv[i], kv[j], s[i][j]);
      }
      __syncthreads();                      // p takes k's place
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = sees(a, pos[i], k0 + tx * 4 + j) ? s[i][j] * sc : -INFINITY;
          mx = s[i][j] > mx ? s[i][j] : mx;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          const float y = __shfl_xor_sync(0xffffffffu, mx, o);
          mx = y > mx ? y : mx;
        }
        const float f = exp2f(m[i] - mx);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f(s[i][j] - mx);
          sum += s[i][j];
          sm.p[tx * 4 + j][ty * 4 + i] = s[i][j];
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c] *= f;
      }
      __syncwarp();                         // a row's weights are written and read by one warp
#pragma unroll 4
      for (int j = 0; j < kKeys; ++j) {
        const float4 p4 = *reinterpret_cast<const float4 *>(&sm.p[j][ty * 4]);
        const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 v4 = *reinterpret_cast<const float4 *>(&sm.v[j][c * 16 + tx * 4]);
          const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][c + e] = fmaf(pv[i], vv[e], acc[i][c + e]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      bool fine = isfinite(l[i]);
#pragma unroll
      for (int c = 0; c < C; ++c) fine = fine && isfinite(acc[i][c]);
      if (r < rows) {
        const size_t at = p.slot >= 0 ? (size_t)p.slot * kRows + r
                                      : (size_t)(p.q.t0 + p.i0 + r / a.g) * a.H + p.h * a.g + r % a.g;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int c = 0; c < C; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const size_t o = at * D + c * 16 + tx * 4 + e;
            if (p.slot >= 0) part.o[o] = acc[i][c + e];
            else static_cast<T *>(a.o)[o] = from_f32<T>(l[i] == 0.f ? 0.f : acc[i][c + e] * inv);
          }
        if (tx == 0) {
          if (p.slot >= 0) part.ml[at] = make_float2(m[i], l[i]);
          else if (a.lse) a.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
        }
      }
      const unsigned odd = __ballot_sync(0xffffffffu, r < rows && !fine);
      for (int half = 0; half < 2; ++half)
        if (odd & (0xffffu << (16 * half)))
          exact_row_write<T, D>(a, a.status, Piece(p), kKeys, ((tid >> 5) * 2 + half) * 4 + i, part, kRows);
    }
  }
  if (tid == 0) a.items[1][blockIdx.x] = item;
}

template <typename T, int D>
cudaError_t launch(const PagedArgs &a, const PagedGeometry &g, cudaStream_t s) {
  const size_t smem = sizeof(SimtSmem<D>);
  static SmemOnce once;
  const cudaError_t e = once(reinterpret_cast<const void *>(paged_simt_kernel<T, D>), smem);
  if (e != cudaSuccess) return e;
  return pdl_launch(paged_simt_kernel<T, D>, g.ctas[1], 256, smem, s, a, g.tok[1]);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_simt(const PagedArgs &a, const PagedGeometry &g, bool bf16, cudaStream_t s) {
  if (bf16) return a.d == 64 ? paged::launch<__nv_bfloat16, 64>(a, g, s) : paged::launch<__nv_bfloat16, 128>(a, g, s);
  return a.d == 64 ? paged::launch<float, 64>(a, g, s) : paged::launch<float, 128>(a, g, s);
}

}  // namespace lz
