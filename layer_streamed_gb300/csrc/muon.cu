// Orthogonalised updates of weight matrices (Muon): momentum, then an
// approximate polar factor of it by Newton-Schulz products, then the step.
//
//   M <- mu M + G,  U = G + mu M (Nesterov) or M
//   X <- U / (|U|_F + eps);  steps times:  A = X X^T,  X <- a X + (b A + c A^2) X
//   W <- W - lr (scale X + decay W)
//
// (A = X^T X and X (b A + c A^2) where there are more rows than columns: the
// square matrices are always as small as they can be, and nothing is
// transposed, the products read X by rows or by columns as they need it.)
//
// Numbers. The products' operands are fp16 with power-of-two scales (X 2^10,
// the square matrices 2^8: fp16's normal range then covers them from 2^-24
// and 2^-22 of their largest values up), the sums fp32. Two things keep an
// operand's rounding (2^-12) from being what the result is off by:
//  - X itself is carried as two fp16 values, hi + lo (22 bits). Only hi is
//    multiplied; a X is formed from both. Directions in which X is small grow
//    by a factor a a step (3.44^5 = 485): with hi alone their rounding would
//    grow with them, and it is what momentum of low rank ends in (4e-2 of the
//    result in a float64 model of these roundings, 1e-3 with both).
//  - A's and B = b A + c A^2's diagonals stay fp32, beside matrices whose
//    diagonal is zero: with D the diagonal and O the rest, A^2 = O^2 + (d_i +
//    d_j) O + D^2, and B X = (B's rest) X + d X. Diagonals are near to each
//    other and to 1, so their rounding errors would all point the same way
//    (2.7e-3 of the result in that model, 0.8e-3 so). lo gets half of d: all
//    of it where X is flat, none where B takes lo's direction to zero.
// Together 0.2e-3 to 1.4e-3 of the result against exact arithmetic (bf16
// products: 1e-2 to 3e-2, and 3e-1 at low rank), below what rounding the
// result to bf16 costs (1.7e-3).
//
// m n^2-like work: 3 m^2 n + m^3 operations a step (m <= n), the symmetric
// products made on and above the diagonal only and mirrored by the epilogue,
// which also forms every linear combination: nothing runs between products.
#include <algorithm>

#include <cuda_fp16.h>

#include "tile_product.cuh"

namespace mt {

MT_DEVICE_ERROR_READER(muon_take_device_error)

namespace {

constexpr float kXUp = 1024.f, kXDown = 1.f / 1024.f;  // X in fp16
constexpr float kAUp = 256.f, kADown = 1.f / 256.f;    // the square matrices

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) { return __half22float2(*(const __half2*)&w); }
__device__ __forceinline__ uint16_t f2h(float f) { return __half_as_ushort(__float2half_rn(f)); }
__device__ __forceinline__ float h2f(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// Eight fp16 values at a 16-byte boundary.
__device__ __forceinline__ void load8h(const uint16_t* p, float* v) {
  const uint4 w = *(const uint4*)p;
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_h2(ws[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ void store8h(uint16_t* p, const float* v) {
  *(uint4*)p = make_uint4(pack_h2(v[0], v[1]), pack_h2(v[2], v[3]), pack_h2(v[4], v[5]), pack_h2(v[6], v[7]));
}
// ---------------------------------------------------------------------------
// Momentum and the norm of the update
// ---------------------------------------------------------------------------
__device__ __forceinline__ float load1(const void* p, size_t i, bool bf16) {
  return bf16 ? bf2f(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void load4(const void* p, size_t i, bool bf16, float (&v)[4]) {
  if (bf16) {
    const uint2 w = *(const uint2*)((const uint16_t*)p + i);
    v[0] = bf2f(w.x & 0xffff), v[1] = bf2f(w.x >> 16), v[2] = bf2f(w.y & 0xffff), v[3] = bf2f(w.y >> 16);
  } else {
    const float4 w = *(const float4*)((const float*)p + i);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
}

__device__ __forceinline__ float block_sum256(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < 8 ? red[threadIdx.x] : 0.f;
  return warp_sum(v);  // in warp 0
}

// M <- mu M + G where there is an M, and a block's part of the sum of U^2.
// Block (x, y) takes every gridDim.x-th group of values of matrix y.
template <bool VEC>
__global__ void __launch_bounds__(256) momentum_kernel(const void* G, bool bf16, float* M, float mu, int nesterov,
                                                       int64_t n, float* part) {
  __shared__ float red[8];
  grid_wait();
  grid_release();
  constexpr int E = VEC ? 4 : 1;
  const size_t base = (size_t)blockIdx.y * n;
  const int64_t step = (int64_t)gridDim.x * 256 * E;
  float sum = 0.f;
#pragma unroll 4
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E; i < n; i += step) {
    float g[4], m[4];
    if (VEC) load4(G, base + i, bf16, g);
    else g[0] = load1(G, base + i, bf16);
    if (M) {
      if (VEC) load4(M, base + i, false, m);
      else m[0] = M[base + i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[e] = fmaf(mu, m[e], g[e]);
        g[e] = nesterov ? fmaf(mu, m[e], g[e]) : m[e];
      }
      if (VEC) *(float4*)(M + base + i) = make_float4(m[0], m[1], m[2], m[3]);
      else M[base + i] = m[0];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sum = fmaf(g[e], g[e], sum);
  }
  sum = block_sum256(sum, red);
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
}

// X = U / (|U| + eps) as hi + lo. VEC: rows are whole groups of eight values
// on their boundary.
template <bool VEC>
__global__ void __launch_bounds__(256)
    normalise_kernel(const void* G, bool bf16, const float* M, float mu, int nesterov, int rows, int cols, int64_t ld,
                     const float* part, int parts, float eps, uint16_t* hi, uint16_t* lo) {
  __shared__ float red[8];
  __shared__ float inv_s;
  grid_wait();
  grid_release();
  const size_t b = blockIdx.y;
  float s = 0.f;
  for (int i = threadIdx.x; i < parts; i += 256) s += part[b * parts + i];
  s = block_sum256(s, red);
  if (threadIdx.x == 0) {
    const float norm = sqrtf(s) + eps;
    // a zero matrix stays zero; an infinite norm (or a NaN) stands for NaN throughout
    inv_s = norm < INFINITY ? (norm > 0.f ? kXUp / norm : 0.f) : __uint_as_float(0x7fffffffu);
  }
  __syncthreads();
  const float inv = inv_s;
  const size_t in0 = b * rows * (size_t)cols, out0 = b * rows * (size_t)ld;
  const int per_row = (cols + 7) / 8;
  const int64_t all = (int64_t)rows * per_row;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += (int64_t)gridDim.x * 256) {
    const int r = (int)(u / per_row), c = (int)(u - (int64_t)r * per_row) * 8;
    const size_t at = in0 + (size_t)r * cols + c;
    float v[8], l[8];
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      float g[4], m[4];
      if (VEC) {
        load4(G, at + q, bf16, g);
        if (M) load4(M, at + q, false, m);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = c + q + e < cols;
          g[e] = in ? load1(G, at + q + e, bf16) : 0.f;
          m[e] = in && M ? M[at + q + e] : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[q + e] = M ? (nesterov ? fmaf(mu, m[e], g[e]) : m[e]) : g[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] *= inv;
      l[e] = v[e] - h2f(f2h(v[e]));
    }
    const size_t o = out0 + (size_t)r * ld + c;
    store8h(hi + o, v);
    store8h(lo + o, l);
  }
}

// ---------------------------------------------------------------------------
// Epilogues. Each works on slabs of 32 rows by 64 columns that come and go by
// TMA (tile_product.cuh): a warp has two pairs of 4 KB, one in work and one on
// its way. The square matrices' slabs leave twice, as they are and transposed.
// ---------------------------------------------------------------------------
constexpr int kSlab = 4096;

// The next slab's place: free once what left from there before has been read.
__device__ __forceinline__ uint8_t* next_slab(EpiWarp& w) {
  uint8_t* p = w.smem + (w.begun++ & 1) * 2 * kSlab;
  if (w.lane == 0) bulk_store_wait<1, true>();
  __syncwarp();
  return p;
}
// 32 columns (half 0 or 1 of a slab's) of this lane's row of a square matrix
// into the slab, and into its transposed image behind it: there a column of
// the slab is a row of 64 bytes, this lane's value at 2 * lane.
__device__ __forceinline__ void put_square(uint8_t* slab, int lane, int half, bool mirror, const float (&v)[32]) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = pack_h2(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *slab_piece(slab, lane, half * 4 + i) = make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
  if (mirror) {
    uint16_t* t = (uint16_t*)(slab + kSlab) + half * 1024 + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      t[64 * i] = (uint16_t)p[i];
      t[64 * i + 32] = (uint16_t)(p[i] >> 16);
    }
  }
}
__device__ __forceinline__ void send_square(const CUtensorMap* m, const CUtensorMap* mt, uint8_t* slab, int lane, int col,
                                            const TileAt& at) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(m, slab, col, at.row0, at.b);
    if (at.mirror) tma_store_3d(mt, slab + kSlab, at.row0, col, at.b);
    bulk_store_commit();
  }
}

// A = X X^T: the rest of A to fp16, its diagonal to fp32.
struct GramEpi : NoSlabs {
  static constexpr int WARPS = 4, SLABS = 4 * kSlab;
  struct Args {
    CUtensorMap O, OT;  // A's rest in slabs, and in transposed ones
    float* d;
    int64_t dpad;  // diagonal entries of a matrix
  };
  struct Row {};
  static __device__ __forceinline__ void load_row(const Args&, const ProductShape&, const TileAt&, Row&) {}
  // 32 columns from col of this lane's row, the diagonal taken out
  static __device__ __forceinline__ void values(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                                float (&v)[32]) {
    const int here = at.row - col;
    if (here >= 0 && here < 32) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        d = i == here ? v[i] : d;
        v[i] = i == here ? 0.f : v[i];
      }
      if (at.row < s.M) a.d[at.b * a.dpad + at.row] = d * (kXDown * kXDown);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= kAUp * kXDown * kXDown;
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row&,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
#pragma unroll 1
    for (int col = at.n0; col < at.n0 + BN && col < s.N; col += 64) {
      uint8_t* slab = next_slab(w);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32];
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
        values(a, s, at, col + 32 * half, v);
        put_square(slab, w.lane, half, at.mirror, v);
      }
      send_square(&a.O, &a.OT, slab, w.lane, col, at);
    }
  }
};

// B = b A + c A^2 from O O^T, O and the diagonal.
struct PolyEpi {
  static constexpr int WARPS = 4, SLABS = 4 * kSlab;
  struct Args {
    CUtensorMap O, B, BT;
    const float* d;
    float* db;
    int64_t dpad;
    float b, c;
  };
  struct Row {
    float d;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.d = at.row < s.M ? a.d[at.b * a.dpad + at.row] : 0.f;
  }
  static __device__ __forceinline__ void values(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                                int col, const float (&o)[32], const float* dj, float (&v)[32]) {
    const int here = at.row - col;
    if (here >= 0 && here < 32) {
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) sq = i == here ? v[i] : sq;
      if (at.row < s.M) a.db[at.b * a.dpad + at.row] = r.d * a.b + a.c * fmaf(r.d, r.d, sq * (kADown * kADown));
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = fmaf(a.c, fmaf(r.d + dj[i], o[i], v[i] * kADown), a.b * o[i]);
      v[i] = i == here ? 0.f : v[i];
    }
  }
  static __device__ __forceinline__ void request(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                                 EpiWarp& w) {
    if (w.lane == 0 && at.row0 < s.M) {
      uint64_t* bar = &w.bars[w.begun & 1];
      mbar_arrive_expect_tx(bar, kSlab);
      tma_load_3d(w.smem + (w.begun & 1) * 2 * kSlab, &a.O, bar, col, at.row0, at.b);
    }
  }
  static __device__ __forceinline__ void prefetch(const Args& a, const ProductShape& s, const TileAt& at, EpiWarp& w) {
    if (w.lane == 0) bulk_store_wait<0, true>();
    request(a, s, at, at.n0, w);
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    const float* dcol = a.d + at.b * a.dpad;
#pragma unroll 1
    for (int col = at.n0; col < at.n0 + BN && col < s.N; col += 64) {
      uint8_t* slab = w.smem + (w.begun & 1) * 2 * kSlab;
      mbar_wait(&w.bars[w.begun & 1], (w.begun >> 1) & 1, w.abort, kErrTimeoutEpi);
      ++w.begun;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32], o[32], dj[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) *(float4*)(dj + 4 * i) = ((const float4*)(dcol + col + 32 * half))[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) load8h((const uint16_t*)slab_piece(slab, w.lane, half * 4 + i), o + 8 * i);
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
        values(a, s, at, r, col + 32 * half, o, dj, v);
        put_square(slab, w.lane, half, at.mirror, v);
        if (half == 0 && col + 64 < at.n0 + BN && col + 64 < s.N) {
          // the other place: what left from it has been read meanwhile
          if (w.lane == 0) bulk_store_wait<0, true>();
          request(a, s, at, col + 64, w);
        }
      }
      send_square(&a.B, &a.BT, slab, w.lane, col, at);
    }
  }
};

// X <- a X + B X; the last step leaves the result or takes the weights' step.
template <bool LAST>
struct ApplyEpi {
  static constexpr int WARPS = 4, SLABS = 4 * kSlab;
  struct Args {
    CUtensorMap hi, lo, hi_out;  // lo in place; hi_out: not LAST
    const float* db;
    int64_t dpad;
    float a;
    int by_col;  // the diagonal runs along the columns (X B) or the rows (B X)
    // LAST: out [M, N] dense per matrix, out <- keep * out - step * X with
    // update, else X
    void* out;
    int out_bf16, update;
    float keep, step;
  };
  struct Row {
    float d;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.d = !a.by_col && at.row < s.M ? a.db[at.b * a.dpad + at.row] : 0.f;
  }
  // four neighbouring values of the new X (times kXUp)
  static __device__ __forceinline__ void step4(float a, const float* d, const float* h, const float* l, float* v) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = fmaf(a + d[e], h[e], fmaf(fmaf(0.5f, d[e], a), l[e], v[e] * kADown));
  }
  static __device__ __forceinline__ void request(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                                 EpiWarp& w) {
    if (w.lane == 0 && at.row0 < s.M) {
      uint64_t* bar = &w.bars[w.begun & 1];
      uint8_t* p = w.smem + (w.begun & 1) * 2 * kSlab;
      mbar_arrive_expect_tx(bar, 2 * kSlab);
      tma_load_3d(p, &a.hi, bar, col, at.row0, at.b);
      tma_load_3d(p + kSlab, &a.lo, bar, col, at.row0, at.b);
    }
  }
  static __device__ __forceinline__ void prefetch(const Args& a, const ProductShape& s, const TileAt& at, EpiWarp& w) {
    if (LAST) fence_proxy_async_smem();
    __syncwarp();
    if (!LAST && w.lane == 0) bulk_store_wait<0, true>();
    request(a, s, at, at.n0, w);
  }
  // LAST: 64 columns of 32 rows of results in the slab pair (fp32; of eight
  // columns the first four where their hi were, the others where their lo
  // were) to out, whole rows at a time: neighbouring lanes, neighbouring columns.
  static __device__ __forceinline__ void write_rows(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                                    uint8_t* slab, int lane) {
    const int rows = min(32, s.M - at.row0);
    const int c = col + 2 * lane;
    uint8_t* half = slab + (lane & 2 ? kSlab : 0);
    const size_t o0 = ((size_t)at.b * s.M + at.row0) * s.N + c;
    // pairs at a time where every row's pairs lie on their boundary
    const bool pairs = (s.N & 1) == 0 && ((uintptr_t)a.out & (a.out_bf16 ? 3 : 7)) == 0;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float2 old[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        old[i] = make_float2(0.f, 0.f);
        const size_t o = o0 + (size_t)(r0 + i) * s.N;
        if (a.update && r0 + i < rows && c < s.N) {
          if (pairs) {
            if (a.out_bf16) {
              const uint32_t u = *(const uint32_t*)((const uint16_t*)a.out + o);
              old[i] = make_float2(bf2f(u & 0xffff), bf2f(u >> 16));
            } else {
              old[i] = *(const float2*)((const float*)a.out + o);
            }
          } else {
            old[i].x = load1(a.out, o, a.out_bf16);
            if (c + 1 < s.N) old[i].y = load1(a.out, o + 1, a.out_bf16);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i >= rows || c >= s.N) break;
        const size_t o = o0 + (size_t)(r0 + i) * s.N;
        float2 x = ((const float2*)slab_piece(half, r0 + i, lane >> 2))[lane & 1];
        if (a.update) {
          x.x = fmaf(a.keep, old[i].x, -a.step * x.x);
          x.y = fmaf(a.keep, old[i].y, -a.step * x.y);
        }
        if (pairs) {
          if (a.out_bf16) *(uint32_t*)((uint16_t*)a.out + o) = pack_bf2(x.x, x.y);
          else *(float2*)((float*)a.out + o) = x;
        } else if (a.out_bf16) {
          ((uint16_t*)a.out)[o] = f2bf(x.x);
          if (c + 1 < s.N) ((uint16_t*)a.out)[o + 1] = f2bf(x.y);
        } else {
          ((float*)a.out)[o] = x.x;
          if (c + 1 < s.N) ((float*)a.out)[o + 1] = x.y;
        }
      }
    }
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    const float* dcol = a.db + at.b * a.dpad;
#pragma unroll 1
    for (int col = at.n0; col < at.n0 + BN && col < s.N; col += 64) {
      uint8_t* slab = w.smem + (w.begun & 1) * 2 * kSlab;
      mbar_wait(&w.bars[w.begun & 1], (w.begun >> 1) & 1, w.abort, kErrTimeoutEpi);
      ++w.begun;
      const bool more = col + 64 < at.n0 + BN && col + 64 < s.N;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32];
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* hp = slab_piece(slab, w.lane, half * 4 + i);
          uint4* lp = slab_piece(slab + kSlab, w.lane, half * 4 + i);
          float h[8], l[8], d[8];
          load8h((const uint16_t*)hp, h);
          load8h((const uint16_t*)lp, l);
          if (a.by_col) {
            *(float4*)d = ((const float4*)(dcol + col + 32 * half))[2 * i];
            *(float4*)(d + 4) = ((const float4*)(dcol + col + 32 * half))[2 * i + 1];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = r.d;
          }
          step4(a.a, d, h, l, v + 8 * i);
          step4(a.a, d + 4, h + 4, l + 4, v + 8 * i + 4);
          if (!LAST) {
            uint32_t p[4], q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = pack_h2(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
              const float2 f = unpack_h2(p[e]);
              q[e] = pack_h2(v[8 * i + 2 * e] - f.x, v[8 * i + 2 * e + 1] - f.y);
            }
            *hp = make_uint4(p[0], p[1], p[2], p[3]);
            *lp = make_uint4(q[0], q[1], q[2], q[3]);
          }
        }
        if (LAST) {
          // the half's own 32 columns: their hi and lo have been read, and the
          // other half's lie in the other half of the pieces
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            *slab_piece(slab, w.lane, half * 4 + i) =
                make_uint4(__float_as_uint(v[8 * i] * kXDown), __float_as_uint(v[8 * i + 1] * kXDown),
                           __float_as_uint(v[8 * i + 2] * kXDown), __float_as_uint(v[8 * i + 3] * kXDown));
            *slab_piece(slab + kSlab, w.lane, half * 4 + i) =
                make_uint4(__float_as_uint(v[8 * i + 4] * kXDown), __float_as_uint(v[8 * i + 5] * kXDown),
                           __float_as_uint(v[8 * i + 6] * kXDown), __float_as_uint(v[8 * i + 7] * kXDown));
          }
        }
        if (half == 0 && more) {
          if (!LAST && w.lane == 0) bulk_store_wait<0, true>();
          if (LAST) {  // the other place has been read by this warp's own loads
            fence_proxy_async_smem();
            __syncwarp();
          }
          request(a, s, at, col + 64, w);
        }
      }
      if (!LAST) {
        fence_proxy_async_smem();
        __syncwarp();
        if (w.lane == 0) {
          tma_store_3d(&a.hi_out, slab, col, at.row0, at.b);
          tma_store_3d(&a.lo, slab + kSlab, col, at.row0, at.b);
          bulk_store_commit();
        }
      } else {
        __syncwarp();
        write_rows(a, s, at, col, slab, w.lane);
        __syncwarp();
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Blocks that share the sum of a matrix's squares: one per 8192 values, as
// many as eight on every SM.
int norm_parts(int64_t n) { return (int)std::min<int64_t>((n + 8191) / 8192, 152 * 8); }

struct Ws {
  size_t part, hi[2], lo, o, b, d, db, total;
  int m, parts;
  int64_t ldx, lda, dpad;
};
Ws workspace(int batch, int rows, int cols) {
  Ws w;
  w.m = std::min(rows, cols);
  w.ldx = (int64_t)up(cols, 64);
  w.lda = (int64_t)up(w.m, 64);
  w.dpad = w.lda;
  w.parts = norm_parts((int64_t)rows * cols);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += up(n, 256);
    return r;
  };
  w.part = take((size_t)batch * w.parts * 4);
  const size_t x = (size_t)batch * rows * w.ldx * 2, a = (size_t)batch * w.m * w.lda * 2;
  w.hi[0] = take(x);
  w.hi[1] = take(x);
  w.lo = take(x);
  w.o = take(a);
  w.b = take(a);
  w.d = take((size_t)batch * w.dpad * 4);
  w.db = take((size_t)batch * w.dpad * 4);
  w.total = at;
  return w;
}

// D = A B^T of fp16 matrices in a batch, tiles by how many there are.
struct Operand {
  const void* p;
  int rows, cols;
  int64_t ld;
};
template <bool A_MN, bool B_MN, bool SYM, class E>
cudaError_t product(const Operand& A, const Operand& B, int M, int N, int K, int batch, const typename E::Args& args,
                    cudaStream_t st) {
  auto go = [&](auto cfg) {
    using C = decltype(cfg);
    CUtensorMap ta, tb;
    if (!product_map(&ta, A.p, A.rows, A.cols, A.ld, A.ld * A.rows, batch, a_box<C>(), true) ||
        !product_map(&tb, B.p, B.rows, B.cols, B.ld, B.ld * B.rows, batch, b_box<C>(), true))
      return cudaErrorUnknown;
    return launch_product<C, E>(ta, tb, product_shape<C>(M, N, K, batch), args, st);
  };
  using Wide = ProductCfg<256, true, A_MN, B_MN, true, SYM>;
  // 256 x 256 tiles on SM pairs where they fill half of the pairs, else 128 x 128 on single SMs
  const ProductShape w = product_shape<Wide>(M, N, K, batch);
  if ((int64_t)w.tiles * batch >= mt_host::num_sms() / 4) return go(Wide());
  return go(ProductCfg<128, false, A_MN, B_MN, true, SYM>());
}

}  // namespace

bool orthogonalize_dims(int batch, int rows, int cols) {
  return batch > 0 && rows > 0 && cols > 0 && batch <= 4096 && rows <= (1 << 16) && cols <= (1 << 16) &&
         (int64_t)rows * cols * batch <= ((int64_t)1 << 40);
}
size_t orthogonalize_workspace(int batch, int rows, int cols) { return workspace(batch, rows, cols).total; }

int orthogonalize(const void* G, bool g_bf16, float* M, float mu, bool nesterov, void* out, bool out_bf16, bool update,
                  float keep, float step, const float* coef, int steps, float eps, void* work, int batch, int rows,
                  int cols, cudaStream_t st) {
  const Ws w = workspace(batch, rows, cols);
  uint8_t* base = (uint8_t*)work;
  float* part = (float*)(base + w.part);
  uint16_t* hi[2] = {(uint16_t*)(base + w.hi[0]), (uint16_t*)(base + w.hi[1])};
  uint16_t *lo = (uint16_t*)(base + w.lo), *O = (uint16_t*)(base + w.o), *B = (uint16_t*)(base + w.b);
  float *d = (float*)(base + w.d), *db = (float*)(base + w.db);
  const int64_t n = (int64_t)rows * cols;
  const size_t gs = g_bf16 ? 8 : 16;
  const bool flat = n % 4 == 0 && al(G, gs) && al(M, 16);
  const dim3 pg((unsigned)w.parts, (unsigned)batch);
  cudaError_t e = mt_host::launch_early(flat ? momentum_kernel<true> : momentum_kernel<false>, pg, 256, 0, st, 1, G,
                                        g_bf16, M, mu, (int)nesterov, n, part);
  const bool whole = cols % 8 == 0 && al(G, gs) && al(M, 16);
  if (e == cudaSuccess)
    e = mt_host::launch_early(whole ? normalise_kernel<true> : normalise_kernel<false>, pg, 256, 0, st, 1, G, g_bf16,
                              (const float*)M, mu, (int)nesterov, rows, cols, w.ldx, (const float*)part, w.parts, eps,
                              hi[0], lo);
  count_launches(2);
  const bool tall = rows > cols;
  const int m = w.m;
  const Operand o{O, m, m, w.lda}, p{B, m, m, w.lda};
  // slabs of X and of the square matrices, these also as 64 rows of 32 columns
  CUtensorMap mX[2], mLo, mO, mOT, mB, mBT;
  const int64_t xa = w.ldx * rows, aa = w.lda * m;
  if (!product_map(&mX[0], hi[0], rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mX[1], hi[1], rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mLo, lo, rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mO, O, m, m, w.lda, aa, batch, 32, true) ||
      !product_map(&mOT, O, m, m, w.lda, aa, batch, 64, true, 32) ||
      !product_map(&mB, B, m, m, w.lda, aa, batch, 32, true) ||
      !product_map(&mBT, B, m, m, w.lda, aa, batch, 64, true, 32))
    return kLaunchFailed;
  for (int i = 0; i < steps && e == cudaSuccess; ++i) {
    const float *c = coef + 3 * i;
    const Operand x{hi[i & 1], rows, cols, w.ldx};
    const GramEpi::Args ga{mO, mOT, d, w.dpad};
    e = tall ? product<true, true, true, GramEpi>(x, x, m, m, rows, batch, ga, st)
             : product<false, false, true, GramEpi>(x, x, m, m, cols, batch, ga, st);
    if (e != cudaSuccess) break;
    e = product<false, false, true, PolyEpi>(o, o, m, m, m, batch, PolyEpi::Args{mO, mB, mBT, d, db, w.dpad, c[1], c[2]}, st);
    if (e != cudaSuccess) break;
    auto apply = [&](auto epi) {
      using E = decltype(epi);
      typename E::Args a{};
      a.hi = mX[i & 1];
      a.lo = mLo;
      a.hi_out = mX[(i + 1) & 1];
      a.db = db;
      a.dpad = w.dpad;
      a.a = c[0];
      a.by_col = tall;
      a.out = out;
      a.out_bf16 = out_bf16;
      a.update = update;
      a.keep = keep;
      a.step = step;
      return tall ? product<false, false, false, E>(x, p, rows, cols, m, batch, a, st)
                  : product<false, true, false, E>(p, x, rows, cols, m, batch, a, st);
    };
    e = i + 1 < steps ? apply(ApplyEpi<false>()) : apply(ApplyEpi<true>());
  }
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

}  // namespace mt
