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
// and 2^-22 of their largest values up; B less where a step's coefficients can
// take it past fp16, see b_scales), the sums fp32. Two things keep an
// operand's rounding (2^-12) from being what the result is off by:
//  - X itself is carried as two fp16 values, hi + lo (22 bits). Only hi is
//    multiplied; a X is formed from both. Directions in which X is small grow
//    by a factor a a step (3.44^5 = 485): with hi alone their rounding would
//    grow with them, and it is what momentum of low rank ends in (4e-2 of the
//    result in a float64 model of these roundings, 0.8e-3 to 2.1e-3 with both,
//    rank 4 and five steps; what is left is B's own rounding, about 0.3 / m of
//    the result for the shorter side m, twice that after six steps).
//  - A's and B = b A + c A^2's diagonals stay fp32, beside matrices whose
//    diagonal is zero: with D the diagonal and O the rest, A^2 = O^2 + (d_i +
//    d_j) O + D^2, and B X = (B's rest) X + d X. Diagonals are near to each
//    other and to 1, so their rounding errors would all point the same way
//    (2.7e-3 of a flat spectrum's result in that model, 0.6e-3 to 1.1e-3 so).
//    lo gets half of d: all of it is right where X is flat, none where B takes
//    lo's direction to zero.
// Together 0.1e-3 to 1.3e-3 of a result of full rank against exact arithmetic
// after five steps (bf16 products: 1e-2 to 3e-2, and 3e-1 at low rank);
// rounding the result to bf16 costs 1.7e-3. The tensor core's sums add what is
// seen with few directions and long sums alone: rank 2 of 4096 x 4096 1.4e-3
// after five steps and 7.5e-3 after six, where the roundings make 0.1e-3 and
// 0.2e-3; they come out up to 3e-5 short, and the polynomial takes a singular
// value's error up to five times as far near 1.2.
//
// Work: 3 m^2 n + m^3 operations a step (m <= n), the symmetric products made
// on and above the diagonal only and mirrored by the epilogue, which also
// forms every linear combination: nothing runs between products. Large
// matrices are bound by the tensor cores, the way from L2 to the SMs (the
// operands take 64 bytes a cycle of it, X's slabs come on top) and the board's
// power limit; the depth of the ring, bands of rows, staged whole-line stores
// and loads of the sums ahead of their use moved the times by no more than the
// clocks do. Small ones are bound by their chain of launches.
#include <algorithm>
#include <type_traits>

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

// The sum of an update's squares, twice: as it is, and of values kSmall times
// as large, which is what counts where squares end among fp32's subnormals or
// below them.
constexpr float kSmall = 0x1p60f;
struct Squares {
  float plain = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float u) {
    plain = fmaf(u, u, plain);
    small = fmaf(u * kSmall, u * kSmall, small);
  }
};
__device__ __forceinline__ Squares block_sum256(Squares v, float2* red) {
  v.plain = warp_sum(v.plain);
  v.small = warp_sum(v.small);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(v.plain, v.small);
  __syncthreads();
  const float2 w = threadIdx.x < 8 ? red[threadIdx.x] : make_float2(0.f, 0.f);
  v.plain = warp_sum(w.x);  // in warp 0
  v.small = warp_sum(w.y);
  return v;
}
// X is u * first * then for the values u of an update with these squares.
// Nothing (a zero matrix) stays nothing whatever eps is; an infinite norm (or
// a NaN) stands for NaN throughout. From 2^-60 on the plain sum's own losses,
// 2^-126 a value, are far below its rounding.
struct Factors {
  float first, then;
};
__device__ __forceinline__ Factors factors(const Squares& s, float eps) {
  if (s.plain < 0x1p-60f) return {kSmall, s.small > 0.f ? kXUp / (sqrtf(s.small) + eps * kSmall) : 0.f};
  const float norm = sqrtf(s.plain) + eps;
  return {1.f, norm < INFINITY ? kXUp / norm : __uint_as_float(0x7fffffffu)};
}

// M <- mu M + G where there is an M, and a block's part of the sum of U^2.
// Block (x, y) takes every gridDim.x-th group of values of matrix y.
template <bool VEC>
__global__ void __launch_bounds__(256, 5) momentum_kernel(const void* G, bool bf16, float* M, float mu, int nesterov,
                                                       int64_t n, float2* part) {
  __shared__ float2 red[8];
  grid_wait();
  grid_release();
  constexpr int E = VEC ? 4 : 1;
  const size_t base = (size_t)blockIdx.y * n;
  const int64_t step = (int64_t)gridDim.x * 256 * E;
  Squares sum;
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
    for (int e = 0; e < E; ++e) sum.add(g[e]);
  }
  sum = block_sum256(sum, red);
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = make_float2(sum.plain, sum.small);
}

// X = U / (|U| + eps) as hi + lo. VEC: rows are whole groups of eight values
// on their boundary.
template <bool VEC>
__global__ void __launch_bounds__(256)
    normalise_kernel(const void* G, bool bf16, const float* M, float mu, int nesterov, int rows, int cols, int64_t ld,
                     const float2* part, int parts, float eps, uint16_t* hi, uint16_t* lo) {
  __shared__ float2 red[8];
  __shared__ Factors all_threads;
  grid_wait();
  grid_release();
  const size_t b = blockIdx.y;
  Squares s;
  for (int i = threadIdx.x; i < parts; i += 256) {
    s.plain += part[b * parts + i].x;
    s.small += part[b * parts + i].y;
  }
  s = block_sum256(s, red);
  if (threadIdx.x == 0) all_threads = factors(s, eps);
  __syncthreads();
  const Factors f = all_threads;
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
      v[e] = v[e] * f.first * f.then;
      l[e] = v[e] - h2f(f2h(v[e]));
    }
    const size_t o = out0 + (size_t)r * ld + c;
    store8h(hi + o, v);
    store8h(lo + o, l);
  }
}

// ---------------------------------------------------------------------------
// Epilogues: eight warps, two to a row of the tile, each its half of the
// columns in slabs of 32 rows by 64. What a slab needs comes by TMA; it is
// taken into registers at once, so that the next one (of the next tile, often)
// is on its way while this one is worked on. Results leave from the lanes, 32
// bytes of a row at a time: whole sectors, and nothing waits for them. The
// square matrices' mirror images leave transposed, by TMA.
// (Results by TMA from where the operands came in, two places a warp, four
// warps: 13 us for a 256 x 256 tile of X against 11, the place being free again
// only when the store has read it. Results through the slab's place in whole
// 128-byte lines: 3 % slower, for it is the next slab that then waits.)
// ---------------------------------------------------------------------------
constexpr int kSlab = 4096;

// Eight fp16 values as they came.
__device__ __forceinline__ void unpack8h(const uint4& w, float* v) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_h2(ws[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}
// First column and one past the last of this warp's share of a tile.
template <int BN>
__device__ __forceinline__ void share(const TileAt& at, const ProductShape& s, const EpiWarp& w, int& c0, int& c1) {
  c0 = at.n0 + w.part * (BN / 2);
  c1 = min(c0 + BN / 2, s.N);
}

// 32 columns from col of this lane's row of a square matrix: the row itself
// (rows are padded to whole 64 columns, so 32 bytes that begin inside can be
// written whole), and into the transposed slab, where a column is 64 bytes and
// this lane's value lies at 2 * lane.
__device__ __forceinline__ void put_square(uint16_t* row, bool ok, uint8_t* slab, int lane, int col, int N, int half,
                                           bool mirror, const float (&v)[32]) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = pack_h2(v[2 * i], v[2 * i + 1]);
  if (ok) {
    if (col < N) store32(row + col, p);
    if (col + 16 < N) store32(row + col + 16, p + 8);
  }
  if (mirror) {
    uint16_t* t = (uint16_t*)slab + half * 1024 + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      t[64 * i] = (uint16_t)p[i];
      t[64 * i + 32] = (uint16_t)(p[i] >> 16);
    }
  }
}
// The same straight to memory, the mirror image a column at a time: the lanes'
// rows are neighbours there.
__device__ __forceinline__ void write_square(uint16_t* mat, int64_t ld, const TileAt& at, int col, int m,
                                             const float (&v)[32]) {
  if (at.row >= m) return;
  put_square(mat + (size_t)at.row * ld, true, nullptr, 0, col, m, 0, false, v);
  if (at.mirror) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i < m) mat[(size_t)(col + i) * ld + at.row] = f2h(v[i]);
  }
}
// 32 fp16 values of a padded row, as far as it has groups of 16 from col on.
__device__ __forceinline__ void load_row32(const uint16_t* row, int col, int N, uint32_t (&w)[16]) {
  load32(row + col, w);
  if (col + 16 < N) {
    load32(row + col + 16, w + 8);
  } else {
#pragma unroll
    for (int i = 8; i < 16; ++i) w[i] = 0;
  }
}
// The transposed slab's place is free when what left from it has been read.
__device__ __forceinline__ void mirror_free(const TileAt& at, int lane) {
  if (at.mirror) {
    if (lane == 0) bulk_store_wait<0, true>();
    __syncwarp();
  }
}
__device__ __forceinline__ void send_mirror(const CUtensorMap* mt, uint8_t* slab, int lane, int col, const TileAt& at) {
  if (at.mirror) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(mt, slab, at.row0, col, at.b);
      bulk_store_commit();
    }
  }
}

// A = X X^T: the rest of A to fp16, its diagonal to fp32.
struct GramEpi : NoSlabs {
  static constexpr int WARPS = 8, SLABS = kSlab;
  struct Args {
    CUtensorMap OT;  // A's rest in transposed slabs
    uint16_t* O;
    float* d;
    int64_t ld, dpad;  // row stride; diagonal entries of a matrix
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
    uint16_t* row = a.O + ((size_t)at.b * s.M + at.row) * a.ld;
    int c0, c1;
    share<BN>(at, s, w, c0, c1);
#pragma unroll 1
    for (int col = c0; col < c1; col += 64) {
      mirror_free(at, w.lane);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32];
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
        values(a, s, at, col + 32 * half, v);
        put_square(row, at.row < s.M, w.smem, w.lane, col + 32 * half, s.N, half, at.mirror, v);
      }
      send_mirror(&a.OT, w.smem, w.lane, col, at);
    }
  }
  struct Early {};
  static __device__ __forceinline__ void early(const Args&, const ProductShape&, const TileAt&, int, Early&) {}
  static __device__ __forceinline__ void chunk(const Args& a, const ProductShape& s, const TileAt& at, const Row&,
                                               const Early&, int col, float (&v)[32], uint8_t*) {
    values(a, s, at, col, v);
    write_square(a.O + (size_t)at.b * s.M * a.ld, a.ld, at, col, s.M, v);
  }
};

// B = b A + c A^2 from O O^T, O and the diagonal.
struct PolyEpi {
  static constexpr int WARPS = 8, SLABS = 2 * kSlab;  // O in, the mirror image out
  template <class A>
  static __device__ __forceinline__ void begin(const A&, int) {}
  struct Args {
    CUtensorMap O, BT;
    const uint16_t* O_rows;
    uint16_t* B;
    const float* d;
    float* db;
    int64_t ld, dpad;
    float b, c, undo;  // times B's scale / kAUp; its reciprocal, for the diagonal
  };
  struct Row {
    float d;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.d = at.row < s.M ? a.d[at.b * a.dpad + at.row] : 0.f;
  }
  static __device__ __forceinline__ void values(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                                int col, const float (&o)[32], const float* dcol, float (&v)[32]) {
    const int here = at.row - col;
    if (here >= 0 && here < 32) {
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) sq = i == here ? v[i] : sq;
      if (at.row < s.M) a.db[at.b * a.dpad + at.row] = (r.d * a.b + a.c * fmaf(r.d, r.d, sq * (kADown * kADown))) * a.undo;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 dj = *(const float4*)(dcol + col + i);
      const float d4[4] = {dj.x, dj.y, dj.z, dj.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = fmaf(a.c, fmaf(r.d + d4[e], o[i + e], v[i + e] * kADown), a.b * o[i + e]);
        v[i + e] = i + e == here ? 0.f : x;
      }
    }
  }
  static __device__ __forceinline__ void request(const Args& a, const TileAt& at, int col, EpiWarp& w) {
    if (w.lane == 0) {
      mbar_arrive_expect_tx(w.bar, kSlab);
      tma_load_3d(w.smem, &a.O, w.bar, col, at.row0, at.b);
    }
  }
  template <int BN>
  static __device__ __forceinline__ void prefetch(const Args& a, const ProductShape& s, const TileAt& at, EpiWarp& w) {
    int c0, c1;
    share<BN>(at, s, w, c0, c1);
    if (at.row0 < s.M && c0 < c1) request(a, at, c0, w);
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    const float* dcol = a.d + at.b * a.dpad;
    uint16_t* row = a.B + ((size_t)at.b * s.M + at.row) * a.ld;
    int c0, c1;
    share<BN>(at, s, w, c0, c1);
#pragma unroll 1
    for (int col = c0; col < c1; col += 64) {
      mbar_wait(w.bar, w.begun++ & 1, w.abort, kErrTimeoutEpi);
      uint4 raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = *slab_piece(w.smem, w.lane, i);
      fence_proxy_async_smem();
      mirror_free(at, w.lane);
      __syncwarp();
      if (col + 64 < c1) request(a, at, col + 64, w);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32], o[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack8h(raw[half * 4 + i], o + 8 * i);
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
        values(a, s, at, r, col + 32 * half, o, dcol, v);
        put_square(row, at.row < s.M, w.smem + kSlab, w.lane, col + 32 * half, s.N, half, at.mirror, v);
      }
      send_mirror(&a.BT, w.smem + kSlab, w.lane, col, at);
    }
  }
  struct Early {
    uint32_t o[16];
  };
  static __device__ __forceinline__ void early(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                               Early& e) {
    if (at.row < s.M) load_row32(a.O_rows + ((size_t)at.b * s.M + at.row) * a.ld, col, s.N, e.o);
  }
  static __device__ __forceinline__ void chunk(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                               const Early& e, int col, float (&v)[32], uint8_t*) {
    float o[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = unpack_h2(e.o[i]);
      o[2 * i] = f.x;
      o[2 * i + 1] = f.y;
    }
    values(a, s, at, r, col, o, a.d + at.b * a.dpad, v);
    write_square(a.B + (size_t)at.b * s.M * a.ld, a.ld, at, col, s.M, v);
  }
};

// X <- a X + B X; the last step leaves the result or takes the weights' step.
// (The last one's form for single SMs spills 208 bytes: ten warps leave it 168
// registers, and the way out by rows shares the kernel with the aligned one.)
template <bool LAST>
struct ApplyEpi {
  static constexpr int WARPS = 8, SLABS = 2 * kSlab;  // hi and lo in
  template <class A>
  static __device__ __forceinline__ void begin(const A&, int) {}
  struct Args {
    CUtensorMap hi, lo;
    const uint16_t* hi_rows;
    uint16_t *hi_out, *lo_out;  // lo_out is lo
    const float* db;
    int64_t ld, dpad;
    float a, down;  // down: 1 / B's scale
    int by_col;  // the diagonal runs along the columns (X B) or the rows (B X)
    // LAST: out [M, N] dense per matrix, out <- keep * out - step * X with
    // update, else X; vec: 32 bytes of a row at a time
    void* out;
    int out_bf16, update, vec;
    float keep, step;
  };
  struct Row {
    float d;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.d = !a.by_col && at.row < s.M ? a.db[at.b * a.dpad + at.row] : 0.f;
  }
  static __device__ __forceinline__ void request(const Args& a, const TileAt& at, int col, EpiWarp& w) {
    if (w.lane == 0) {
      mbar_arrive_expect_tx(w.bar, 2 * kSlab);
      tma_load_3d(w.smem, &a.hi, w.bar, col, at.row0, at.b);
      tma_load_3d(w.smem + kSlab, &a.lo, w.bar, col, at.row0, at.b);
    }
  }
  template <int BN>
  static __device__ __forceinline__ void prefetch(const Args& a, const ProductShape& s, const TileAt& at, EpiWarp& w) {
    int c0, c1;
    share<BN>(at, s, w, c0, c1);
    if (at.row0 < s.M && c0 < c1) request(a, at, c0, w);
    if (LAST && a.update && at.row < s.M) {  // the weights' lines into L2, while the sums are made
      const int e = a.out_bf16 ? 2 : 4;
      const char* line = (const char*)a.out + ((size_t)at.b * s.M + at.row) * s.N * e;
      for (int c = c0 * e; c < c1 * e; c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + c));
      if (c0 < c1) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + c1 * e - 1));
    }
  }
  // LAST: 16 results from `col` of this lane's row.
  static __device__ __forceinline__ void finish16(const Args& a, const ProductShape& s, size_t row, int col, float* x) {
    const size_t o = row + col;
    if (a.vec && col + 16 <= s.N) {
      if (a.out_bf16) {
        uint32_t u[8];
        if (a.update) {
          load32((uint16_t*)a.out + o, u);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[2 * e] = fmaf(a.keep, bf2f(u[e] & 0xffff), -a.step * x[2 * e]);
            x[2 * e + 1] = fmaf(a.keep, bf2f(u[e] >> 16), -a.step * x[2 * e + 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = pack_bf2(x[2 * e], x[2 * e + 1]);
        store32((uint16_t*)a.out + o, u);
      } else {
#pragma unroll
        for (int q = 0; q < 16; q += 8) {
          uint32_t u[8];
          if (a.update) {
            load32((float*)a.out + o + q, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[q + e] = fmaf(a.keep, __uint_as_float(u[e]), -a.step * x[q + e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(x[q + e]);
          store32((float*)a.out + o + q, u);
        }
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (col + e >= s.N) break;
      const float r = a.update ? fmaf(a.keep, load1(a.out, o + e, a.out_bf16), -a.step * x[e]) : x[e];
      if (a.out_bf16) ((uint16_t*)a.out)[o + e] = f2bf(r);
      else ((float*)a.out)[o + e] = r;
    }
  }
  // LAST where rows lie on no boundary: results wait in shared memory, 32 fp32
  // columns by 32 rows a slab, and leave a row at a time: fp32 a column a lane,
  // bf16 two a lane, at whole words wherever a row begins (lane 0 of a row that
  // begins between two has the first column and the last).
  // (Muon step of 8 x 936 x 7753, the last product: from the lanes' own rows,
  // value by value, took 1100 us; a column a lane 415; as here 271.)
  static __device__ __forceinline__ void hold16(uint8_t* slab, int lane, int k, const float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *(float4*)slab_piece(slab, lane, k + e) =
          make_float4(x[4 * e] * kXDown, x[4 * e + 1] * kXDown, x[4 * e + 2] * kXDown, x[4 * e + 3] * kXDown);
  }
  static __device__ __forceinline__ float held_at(uint8_t* slab, int row, int col) {  // of 64 columns in two slabs
    return ((const float*)slab_piece(slab + (col >> 5) * kSlab, row, (col & 31) >> 2))[col & 3];
  }
  // `cols` (32 or 64) columns from col
  static __device__ __forceinline__ void write_rows(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                                    uint8_t* slab, int lane, int cols) {
    const int rows = min(32, s.M - at.row0), end = min(s.N - col, cols);
    const size_t o0 = ((size_t)at.b * s.M + at.row0) * s.N + col;
    if (!a.out_bf16) {
      for (int c = lane; c < end; c += 32) {
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8) {
          float* p = (float*)a.out + o0 + (size_t)r0 * s.N + c;
          float old[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) old[i] = a.update && r0 + i < rows ? p[(size_t)i * s.N] : 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows) break;
            const float x = held_at(slab, r0 + i, c);
            p[(size_t)i * s.N] = a.update ? fmaf(a.keep, old[i], -a.step * x) : x;
          }
        }
      }
      return;
    }
    if (2 * lane >= cols) return;
    uint16_t* out = (uint16_t*)a.out;
    const size_t between = ((uintptr_t)out >> 1) & 1;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      // asked for together: nothing is made of a value before the last is on its way
      uint32_t both[8];
      uint16_t first[8], second[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        both[i] = 0;
        first[i] = second[i] = 0;
        const size_t o = o0 + (size_t)(r0 + i) * s.N;
        const int e = 2 * lane - (int)((o + between) & 1), f = e < 0 ? cols - 1 : e;
        const bool in = a.update && r0 + i < rows, word = e >= 0 && e + 1 < end;
        if (in && word) both[i] = *(const uint32_t*)(out + o + e);
        if (in && !word && f < end) first[i] = out[o + f];
        if (in && !word && e + 1 < end) second[i] = out[o + e + 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i >= rows) break;
        const size_t o = o0 + (size_t)(r0 + i) * s.N;
        const int e = 2 * lane - (int)((o + between) & 1), f = e < 0 ? cols - 1 : e;
        const bool word = e >= 0 && e + 1 < end;
        float x = f < end ? held_at(slab, r0 + i, f) : 0.f, y = e + 1 < end ? held_at(slab, r0 + i, e + 1) : 0.f;
        if (a.update) {
          x = fmaf(a.keep, bf2f(word ? (uint16_t)both[i] : first[i]), -a.step * x);
          y = fmaf(a.keep, bf2f(word ? (uint16_t)(both[i] >> 16) : second[i]), -a.step * y);
        }
        const uint32_t w = pack_bf2(x, y);
        if (word) *(uint32_t*)(out + o + e) = w;
        if (!word && f < end) out[o + f] = (uint16_t)w;
        if (!word && e + 1 < end) out[o + e + 1] = (uint16_t)(w >> 16);
      }
    }
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    const bool held = LAST && !a.vec;  // the results take the slabs' place for a while
    int c0, c1;
    share<BN>(at, s, w, c0, c1);
#pragma unroll 1
    for (int col = c0; col < c1; col += 64) {
      mbar_wait(w.bar, w.begun++ & 1, w.abort, kErrTimeoutEpi);
      uint4 rh[8], rl[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        rh[i] = *slab_piece(w.smem, w.lane, i);
        rl[i] = *slab_piece(w.smem + kSlab, w.lane, i);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (!held && col + 64 < c1) request(a, at, col + 64, w);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32];
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 *hq = rh + half * 4 + q * 2, *lq = rl + half * 4 + q * 2;
          const uint32_t h[8] = {hq[0].x, hq[0].y, hq[0].z, hq[0].w, hq[1].x, hq[1].y, hq[1].z, hq[1].w};
          const uint32_t l[8] = {lq[0].x, lq[0].y, lq[0].z, lq[0].w, lq[1].x, lq[1].y, lq[1].z, lq[1].w};
          new16(a, at, r, col + 32 * half + 16 * q, h, l, v + 16 * q);
          if (held) hold16(w.smem + half * kSlab, w.lane, 4 * q, v + 16 * q);
          else put16(a, s, at, col + 32 * half + 16 * q, v + 16 * q);
        }
      }
      if (held) {
        __syncwarp();
        write_rows(a, s, at, col, w.smem, w.lane, 64);
        fence_proxy_async_smem();
        __syncwarp();
        if (col + 64 < c1) request(a, at, col + 64, w);
      }
    }
  }
  // 16 values of the new X (times kXUp) from col of this lane's row
  static __device__ __forceinline__ void new16(const Args& a, const TileAt& at, const Row& r, int col,
                                               const uint32_t* hw, const uint32_t* lw, float* x) {
    const float* dcol = a.db + at.b * a.dpad + col;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float d[4] = {r.d, r.d, r.d, r.d};
      if (a.by_col) *(float4*)d = *(const float4*)(dcol + i);
      const float2 h0 = unpack_h2(hw[i / 2]), h1 = unpack_h2(hw[i / 2 + 1]), l0 = unpack_h2(lw[i / 2]),
                   l1 = unpack_h2(lw[i / 2 + 1]);
      const float h[4] = {h0.x, h0.y, h1.x, h1.y}, l[4] = {l0.x, l0.y, l1.x, l1.y};
#pragma unroll
      for (int f = 0; f < 4; ++f)
        x[i + f] = fmaf(a.a + d[f], h[f], fmaf(fmaf(0.5f, d[f], a.a), l[f], x[i + f] * a.down));
    }
  }
  static __device__ __forceinline__ void put16(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                               float* x) {
    if (at.row >= s.M || col >= s.N) return;
    const size_t row = (size_t)at.b * s.M + at.row;
    if (!LAST) {
      uint32_t p[8], l[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = pack_h2(x[2 * e], x[2 * e + 1]);
        const float2 f = unpack_h2(p[e]);
        l[e] = pack_h2(x[2 * e] - f.x, x[2 * e + 1] - f.y);
      }
      store32(a.hi_out + row * a.ld + col, p);
      store32(a.lo_out + row * a.ld + col, l);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= kXDown;
      finish16(a, s, row * s.N, col, x);
    }
  }
  struct Early {
    uint32_t h[16], l[16];
  };
  static __device__ __forceinline__ void early(const Args& a, const ProductShape& s, const TileAt& at, int col,
                                               Early& e) {
    if (at.row >= s.M) return;
    const size_t o = ((size_t)at.b * s.M + at.row) * a.ld;
    load_row32(a.hi_rows + o, col, s.N, e.h);
    load_row32(a.lo_out + o, col, s.N, e.l);
  }
  static __device__ __forceinline__ void chunk(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                               const Early& e, int col, float (&v)[32], uint8_t* room) {
    const bool held = LAST && !a.vec;
    const int lane = (int)lane_id();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      new16(a, at, r, col + 16 * q, e.h + 8 * q, e.l + 8 * q, v + 16 * q);
      if (held) hold16(room, lane, 4 * q, v + 16 * q);
      else put16(a, s, at, col + 16 * q, v + 16 * q);
    }
    if (held) {
      __syncwarp();
      write_rows(a, s, at, col, room, lane, 32);
    }
  }
};

// ---------------------------------------------------------------------------
// Matrices with a side of at most 128: everything in one launch. A cluster of
// S CTAs takes a matrix, each up to 256 of the long side's values (tall ones
// are taken transposed). X lives in tensor memory in fp32 (256 columns of 128
// lanes) and its fp16 copy in shared memory as blocks of 64 columns by 128
// rows of 128 bytes, which one matrix descriptor reads as X (K along the
// columns: the Gram product) and another one as X transposed (B X). A step is
// three rounds of MMAs with their epilogues by all sixteen warps, and between
// the first and the second the sum of the CTAs' parts of A: each CTA adds up
// 128 / S columns of it, from the others' shared memory, and sends them all
// that share of A's rest in fp16 and of its diagonal. Latency is all that
// counts here: 64 x 64 took 72 us as a chain of seventeen launches, 20 so.
// ---------------------------------------------------------------------------
struct NarrowArgs {
  const void* G;
  float* M;  // null: none
  void* out;
  int g_bf16, nesterov, out_bf16, update, steps, tall;
  int m, n, cols;  // short and long side; columns as stored
  float mu, keep, step, eps;
  float coef[96], up[32], down[32];  // B's scale / kAUp, 1 / B's scale of each step
};
constexpr int kXBlock = 128 * 128;  // bytes of 64 columns of X, of 64 columns of a square matrix
constexpr int kNarrowCols = 256;    // columns of X in a CTA
constexpr int kNarrowSmem = 4 * kXBlock + 2 * kXBlock + 65536 + 1024 /*align*/;

// 16-byte piece k (8 columns) of a row of such blocks.
__device__ __forceinline__ uint4* block_piece(uint8_t* blocks, int row, int k) {
  return slab_piece(blocks + (k >> 3) * kXBlock, row, k & 7);
}

// 32 values of this lane's row to tensor memory.
__device__ __forceinline__ void put_chunk(uint32_t t, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  __syncwarp();
  tmem_st32(t, r);
}

template <int S>
__global__ void __launch_bounds__(512, 1) narrow_kernel(const __grid_constant__ NarrowArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* xh = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // 4 blocks of X
  uint8_t* sq = xh + 4 * kXBlock;                                             // 2 blocks of O, then of B
  uint8_t* ex = sq + 2 * kXBlock;                                             // the others' parts: [S][128 / S / 4][128] float4
  __shared__ float dg[128], dbs[128];
  __shared__ float2 norms[S], red[16];
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, part = warp >> 2;  // lanes of tensor memory, quarter of the columns
  const int row = q * 32 + lane;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const size_t mat = (size_t)(blockIdx.x / S) * p.m * p.n;
  if (tid == 0) {
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 128) dg[tid] = dbs[tid] = 0.f;
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync();  // every CTA runs: its shared memory may be written
  tc_fence_after();
  const uint32_t tx = tmem_slot + ((uint32_t)(q * 32) << 16);  // X: columns 0 .. 255; sums: 256 ..
  const uint32_t td = tx + 256;
  grid_wait();
  grid_release();

  const int j0 = rank * kNarrowCols;
  const int mine = max(0, min(kNarrowCols, p.n - j0));  // columns of this CTA
  const int blocks = (mine + 63) / 64;
  // where X[row][j] lies, and whether four neighbours can be read at once
  const bool vec = !p.tall && p.cols % 4 == 0 && ((uintptr_t)p.G & (p.g_bf16 ? 7 : 15)) == 0 && ((uintptr_t)p.M & 15) == 0;
  const bool vec_out = !p.tall && p.cols % 4 == 0 && ((uintptr_t)p.out & (p.out_bf16 ? 7 : 15)) == 0;
  auto at = [&](int j) { return mat + (p.tall ? (size_t)j * p.cols + row : (size_t)row * p.cols + j); };

  // U into tensor memory, the sums of its squares. Rows on no boundary come a row
  // at a time, a column a lane, and wait in shared memory (the blocks' place,
  // not yet in use; a row is 257 words, so that neither side meets a bank
  // twice). 100 x 1001: 54 us, and 78 value by value from the lanes' own rows.
  Squares sum;
  float* rows = (float*)xh;
  constexpr int kRow = 257;
  const bool by_rows = !p.tall && !vec;
  if (by_rows) {
#pragma unroll 1
    for (int r = warp; r < p.m; r += 16) {
      float u[8], m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = lane + 32 * k;
        const size_t o = mat + (size_t)r * p.cols + j0 + c;
        u[k] = c < mine ? load1(p.G, o, p.g_bf16) : 0.f;
        m[k] = c < mine && p.M ? p.M[o] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = lane + 32 * k;
        if (p.M) {
          m[k] = fmaf(p.mu, m[k], u[k]);
          u[k] = p.nesterov ? fmaf(p.mu, m[k], u[k]) : m[k];
          if (c < mine) p.M[mat + (size_t)r * p.cols + j0 + c] = m[k];
        }
        rows[r * kRow + c] = u[k];
      }
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int col = part * 64 + c * 32;
    float u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = 0.f;
    if (by_rows && row < p.m) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        u[i] = rows[row * kRow + col + i];
        sum.add(u[i]);
      }
    } else if (row < p.m && col < mine) {
      float m[32];
      if (vec && col + 32 <= mine) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          load4(p.G, at(j0 + col + i), p.g_bf16, *(float(*)[4])(u + i));
          if (p.M) load4(p.M, at(j0 + col + i), false, *(float(*)[4])(m + i));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const bool in = col + i < mine;
          u[i] = in ? load1(p.G, at(j0 + col + i), p.g_bf16) : 0.f;
          m[i] = in && p.M ? p.M[at(j0 + col + i)] : 0.f;
        }
      }
      if (p.M) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          m[i] = fmaf(p.mu, m[i], u[i]);
          u[i] = p.nesterov ? fmaf(p.mu, m[i], u[i]) : m[i];
        }
        if (vec && col + 32 <= mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *(float4*)(p.M + at(j0 + col + i)) = make_float4(m[i], m[i + 1], m[i + 2], m[i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < mine) p.M[at(j0 + col + i)] = m[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) sum.add(u[i]);
    }
    put_chunk(tx + col, u);
  }
  tmem_st_wait();
  sum.plain = warp_sum(sum.plain);
  sum.small = warp_sum(sum.small);
  if (lane == 0) red[warp] = make_float2(sum.plain, sum.small);
  __syncthreads();
  if (tid < S) {
    Squares s;
    for (int i = 0; i < 16; ++i) {
      s.plain += red[i].x;
      s.small += red[i].y;
    }
    if (S > 1) {
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(&norms[rank], (uint32_t)tid)), "f"(s.plain),
                   "f"(s.small)
                   : "memory");
    } else {
      norms[0] = make_float2(s.plain, s.small);
    }
  }
  if (S > 1) cluster_sync();
  else __syncthreads();
  sum = Squares();
#pragma unroll
  for (int r = 0; r < S; ++r) {
    sum.plain += norms[r].x;
    sum.small += norms[r].y;
  }
  const Factors f = factors(sum, p.eps);

  // X (times kXUp) to tensor memory, its fp16 copy to the blocks
  auto keep_x = [&](int col, float (&x)[32]) {
    put_chunk(tx + col, x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *block_piece(xh, row, col / 8 + i) = make_uint4(pack_h2(x[8 * i], x[8 * i + 1]), pack_h2(x[8 * i + 2], x[8 * i + 3]),
                                                      pack_h2(x[8 * i + 4], x[8 * i + 5]), pack_h2(x[8 * i + 6], x[8 * i + 7]));
  };
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int col = part * 64 + c * 32;
    float x[32];
    tile_chunk(tx, part * 2 + c, x);
    // padding stays zero where the norm is not a number
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = row < p.m && col + i < mine ? x[i] * f.first * f.then : 0.f;
    keep_x(col, x);
  }
  tmem_st_wait();

  constexpr uint32_t kSquare = make_idesc(128, 128, false, false) & ~((1u << 7) | (1u << 10));
  const uint32_t times_x = make_idesc(128, blocks * 64, false, true) & ~((1u << 7) | (1u << 10));
  // Rows from m on and this CTA's columns behind its own are zeros: sums along
  // them end at the next whole 16, and chunks of 32 results that lie there
  // altogether are left out.
  const int deep = (p.m + 15) / 16;
  const bool square = part * 32 < p.m;  // this warp has columns of the square matrices
  uint32_t phase = 0;
  auto sync = [&] {  // shared and tensor memory as the other warps have left them, for the MMAs
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  auto wait = [&] {
    mbar_wait(&done, phase, &abort_flag, kErrTimeoutMma);
    phase ^= 1;
    tc_fence_after();
  };

#pragma unroll 1
  for (int step = 0; step < p.steps; ++step) {
    const float ca = p.coef[3 * step], cb = p.coef[3 * step + 1], cc = p.coef[3 * step + 2];
    const float up = p.up[step], down = p.down[step];
    // A = X X^T, this CTA's columns
    sync();
    if (tid == 0) {
      const uint32_t x = smem_u32(xh);
      for (int k = 0; k < blocks * 4; ++k) {
        const uint64_t d = make_sdesc(x + (k >> 2) * kXBlock + (k & 3) * 32, 16, 1024);
        tc_mma(tmem_slot + 256, d, d, kSquare, k != 0);
      }
      tc_commit(&done);
    }
    __syncwarp();
    wait();
    if (S > 1) {
      // eight columns at a time to the CTA that adds them up: [source][4 columns][row]
      constexpr int SHARE = 128 / S;
      if (square) {
        float v[32];
        tile_chunk(td, part, v);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          const int col = part * 32 + i;
          const uint32_t to = mapa_shared(ex + ((rank * SHARE + col % SHARE) / 4) * 2048, (uint32_t)(col / SHARE)) + row * 16;
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + e * 512),
                         "f"(blocks ? v[i + e] : 0.f), "f"(blocks ? v[i + e + 1] : 0.f), "f"(blocks ? v[i + e + 2] : 0.f),
                         "f"(blocks ? v[i + e + 3] : 0.f)
                         : "memory");
        }
      }
      tc_fence_before();
      cluster_sync();
      // this CTA's share: eight columns at a time to all
#pragma unroll 1
      for (int in = part * 8; in < SHARE; in += 32) {
        const int col = rank * SHARE + in;
        if (col / 32 * 32 >= p.m) break;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
        for (int r = 0; r < S; ++r) {
          const float4* e = (const float4*)(ex + ((r * SHARE + in) / 4) * 2048) + row;
          const float4 a = e[0], b = e[128];
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d = col + i == row ? v[i] * (kXDown * kXDown) : d;
          v[i] = col + i == row ? 0.f : v[i] * (kAUp * kXDown * kXDown);
        }
        const uint32_t w[4] = {pack_h2(v[0], v[1]), pack_h2(v[2], v[3]), pack_h2(v[4], v[5]), pack_h2(v[6], v[7])};
        uint4* to = block_piece(sq, row, col / 8);
#pragma unroll
        for (int r = 0; r < S; ++r) {
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mapa_shared(to, (uint32_t)r)), "r"(w[0]),
                       "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
          if (col <= row && row < col + 8)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(&dg[row], (uint32_t)r)), "f"(d) : "memory");
        }
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      cluster_sync();
    } else {
      if (square) {
        const int col = part * 32;
        float v[32];
        tile_chunk(td, part, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (col + i == row) dg[row] = v[i] * (kXDown * kXDown);
          v[i] = col + i == row ? 0.f : v[i] * (kAUp * kXDown * kXDown);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *block_piece(sq, row, col / 8 + i) = make_uint4(pack_h2(v[8 * i], v[8 * i + 1]), pack_h2(v[8 * i + 2], v[8 * i + 3]),
                                                          pack_h2(v[8 * i + 4], v[8 * i + 5]), pack_h2(v[8 * i + 6], v[8 * i + 7]));
      }
    }
    // A^2's rest, then B in A's place
    sync();
    if (tid == 0) {
      const uint32_t o = smem_u32(sq);
      for (int k = 0; k < deep; ++k) {
        const uint64_t d = make_sdesc(o + (k >> 2) * kXBlock + (k & 3) * 32, 16, 1024);
        tc_mma(tmem_slot + 256, d, d, kSquare, k != 0);
      }
      tc_commit(&done);
    }
    __syncwarp();
    wait();
    const float d = dg[row];
    if (square) {
      const int col = part * 32;
      float v[32], o[32];
      tile_chunk(td, part, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack8h(*block_piece(sq, row, col / 8 + i), o + 8 * i);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (col + i == row) dbs[row] = d * cb + cc * fmaf(d, d, v[i] * (kADown * kADown));
        v[i] = col + i == row ? 0.f : fmaf(cc * up, fmaf(d + dg[col + i], o[i], v[i] * kADown), cb * up * o[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *block_piece(sq, row, col / 8 + i) = make_uint4(pack_h2(v[8 * i], v[8 * i + 1]), pack_h2(v[8 * i + 2], v[8 * i + 3]),
                                                        pack_h2(v[8 * i + 4], v[8 * i + 5]), pack_h2(v[8 * i + 6], v[8 * i + 7]));
    }
    // X <- a X + B X
    sync();
    if (tid == 0) {
      const uint32_t b = smem_u32(sq), x = smem_u32(xh);
      for (int k = 0; k < deep && blocks; ++k)
        tc_mma(tmem_slot + 256, make_sdesc(b + (k >> 2) * kXBlock + (k & 3) * 32, 16, 1024),
               make_sdesc(x + k * 2048, kXBlock, 1024), times_x, k != 0);
      tc_commit(&done);
    }
    __syncwarp();
    wait();
    const float db = dbs[row], ah = ca + db, al_ = ca + 0.5f * db;
    const bool last = step + 1 == p.steps;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int col = part * 64 + c * 32;
      if (col >= mine) break;
      float v[32], x[32];
      tile_chunk(td, part * 2 + c, v);
      tile_chunk(tx, part * 2 + c, x);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float h = h2f(f2h(x[i]));
        x[i] = fmaf(ah, h, fmaf(al_, x[i] - h, v[i] * down));
      }
      if (!last) {
        keep_x(col, x);
      } else if (row < p.m && vec_out && col + 32 <= mine) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const size_t o = at(j0 + col + i);
          float r[4] = {x[i] * kXDown, x[i + 1] * kXDown, x[i + 2] * kXDown, x[i + 3] * kXDown};
          if (p.update) {
            float w[4];
            load4(p.out, o, p.out_bf16, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = fmaf(p.keep, w[e], -p.step * r[e]);
          }
          if (p.out_bf16) *(uint2*)((uint16_t*)p.out + o) = make_uint2(pack_bf2(r[0], r[1]), pack_bf2(r[2], r[3]));
          else *(float4*)((float*)p.out + o) = make_float4(r[0], r[1], r[2], r[3]);
        }
      } else if (!p.tall && !vec_out) {
#pragma unroll
        for (int i = 0; i < 32; ++i) rows[row * kRow + col + i] = x[i] * kXDown;  // the blocks have been read
      } else if (row < p.m) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (col + i >= mine) break;
          const size_t o = at(j0 + col + i);
          float r = x[i] * kXDown;
          if (p.update) r = fmaf(p.keep, load1(p.out, o, p.out_bf16), -p.step * r);
          if (p.out_bf16) ((uint16_t*)p.out)[o] = f2bf(r);
          else ((float*)p.out)[o] = r;
        }
      }
    }
    if (!last) tmem_st_wait();
  }
  if (!p.tall && !vec_out) {  // rows on no boundary leave as they come
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < p.m; r += 16) {
      const size_t o = mat + (size_t)r * p.cols + j0 + lane;
      float old[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) old[k] = p.update && lane + 32 * k < mine ? load1(p.out, o + 32 * k, p.out_bf16) : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (lane + 32 * k >= mine) break;
        float x = rows[r * kRow + lane + 32 * k];
        if (p.update) x = fmaf(p.keep, old[k], -p.step * x);
        if (p.out_bf16) ((uint16_t*)p.out)[o + 32 * k] = f2bf(x);
        else ((float*)p.out)[o + 32 * k] = x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// The scale of B = b A + c A^2 in each step: 2^8, or the largest power of two
// with which no value off B's diagonal can pass fp16. Such a value is at most
// half of the range of q(t) = b t + c t^2 over A's eigenvalues t = s^2. The
// singular values s begin below 1 and go through s (a + q(s^2)); past 15 the
// matrices themselves leave fp16, so no bound beyond that is of use. (Muon's
// quintic stays with 2^8; 5 X in one step and the quintic in the next has B up
// to 575.)
void b_scales(const float* coef, int steps, float* scale) {
  double s = 1.01;  // roundings
  for (int i = 0; i < steps; ++i) {
    const double a = coef[3 * i], b = coef[3 * i + 1], c = coef[3 * i + 2], top = s * s;
    auto q = [&](double t) { return (b + c * t) * t; };
    double lo = std::min(0.0, q(top)), hi = std::max(0.0, q(top));
    if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < top) {
      lo = std::min(lo, q(-b / (2.0 * c)));
      hi = std::max(hi, q(-b / (2.0 * c)));
    }
    scale[i] = kAUp;
    while ((hi - lo) * 0.5 * scale[i] > 60000.0) scale[i] *= 0.5f;
    // |s (a + q(s^2))| is largest at the end or where a + 3 b t + 5 c t^2 = 0
    double most = std::fabs(s * (a + q(top)));
    auto at = [&](double t) {
      if (t > 0.0 && t < top) most = std::max(most, std::fabs(std::sqrt(t) * (a + q(t))));
    };
    const double root = 9.0 * b * b - 20.0 * a * c;
    if (c == 0.0) {
      if (b != 0.0) at(-a / (3.0 * b));
    } else if (root >= 0.0) {
      at((-3.0 * b + std::sqrt(root)) / (10.0 * c));
      at((-3.0 * b - std::sqrt(root)) / (10.0 * c));
    }
    s = std::min(15.0, 1.01 * most);
  }
}

// Blocks that share the sum of a matrix's squares: one per 2048 values, as
// many as eight on every SM.
int norm_parts(int64_t n) { return (int)std::min<int64_t>((n + 2047) / 2048, 152 * 8); }

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
  w.part = take((size_t)batch * w.parts * 8);
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

// D = A B^T of fp16 matrices in a batch. Few tiles of 128 x 128: each shared by
// four CTAs where that leaves every CTA an SM (1024 x 1024: 152 us a call of
// five steps without, 138 so), by two where the sum is deep or, a little less
// deep, the result not symmetric (two CTAs for all: 2 x 1024 x 1024 172 us,
// 160 so; none: 1024 x 1024 153). One SM a tile up to as many as there are SMs
// (4 x 1024 x 1024: 235 us on pairs, 192 so), then 256 x 256 on SM pairs where
// they fill half of the pairs.
struct Operand {
  const void* p;
  int rows, cols;
  int64_t ld;
};
template <bool A_MN, bool B_MN, bool SYM, class E>
cudaError_t product(const Operand& A, const Operand& B, int M, int N, int K, int batch, const typename E::Args& args,
                    cudaStream_t st) {
  auto go = [&](auto cfg, auto split) {
    using C = decltype(cfg);
    constexpr int S = decltype(split)::value;
    CUtensorMap ta, tb;
    if (!product_map(&ta, A.p, A.rows, A.cols, A.ld, A.ld * A.rows, batch, a_box<C>(M, K), true) ||
        !product_map(&tb, B.p, B.rows, B.cols, B.ld, B.ld * B.rows, batch, b_box<C>(K), true))
      return cudaErrorUnknown;
    const ProductShape s = product_shape<C>(M, N, K, batch);
    if constexpr (S > 1) return launch_split<C, E, S>(ta, tb, s, args, st);
    else return launch_product<C, E>(ta, tb, s, args, st);
  };
  using Wide = ProductCfg<256, true, A_MN, B_MN, true, SYM>;
  using Small = ProductCfg<128, false, A_MN, B_MN, true, SYM>;
  const int sms = mt_host::num_sms();
  const int64_t wide = (int64_t)product_shape<Wide>(M, N, K, batch).tiles * batch;
  const int64_t small = (int64_t)product_shape<Small>(M, N, K, batch).tiles * batch;
  if (4 * small <= sms) return go(Small(), std::integral_constant<int, 4>());
  if (2 * small <= sms && K >= (SYM ? 2048 : 1024)) return go(Small(), std::integral_constant<int, 2>());
  if (small > sms && wide >= sms / 4) return go(Wide(), std::integral_constant<int, 1>());
  return go(Small(), std::integral_constant<int, 1>());
}

template <int S>
int launch_narrow(const NarrowArgs& a, int batch, cudaStream_t st) {
  auto k = narrow_kernel<S>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kNarrowSmem);
  if (S > 8 && e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = mt_host::launch_early(k, batch * S, 512, kNarrowSmem, st, S, a);
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
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
  const int sides[2] = {std::min(rows, cols), std::max(rows, cols)};
  float scale[32];
  b_scales(coef, steps, scale);
  if (sides[0] <= 128 && sides[1] <= 16 * kNarrowCols) {
    NarrowArgs a{};
    a.G = G;
    a.M = M;
    a.out = out;
    a.g_bf16 = g_bf16;
    a.nesterov = nesterov;
    a.out_bf16 = out_bf16;
    a.update = update;
    a.steps = steps;
    a.tall = rows > cols;
    a.m = sides[0];
    a.n = sides[1];
    a.cols = cols;
    a.mu = mu;
    a.keep = keep;
    a.step = step;
    a.eps = eps;
    std::copy(coef, coef + 3 * steps, a.coef);
    for (int i = 0; i < steps; ++i) {
      a.up[i] = scale[i] * kADown;
      a.down[i] = 1.f / scale[i];
    }
    const int ctas = (sides[1] + kNarrowCols - 1) / kNarrowCols;
    return ctas == 1   ? launch_narrow<1>(a, batch, st)
           : ctas == 2 ? launch_narrow<2>(a, batch, st)
           : ctas <= 4 ? launch_narrow<4>(a, batch, st)
           : ctas <= 8 ? launch_narrow<8>(a, batch, st)
                       : launch_narrow<16>(a, batch, st);
  }
  const Ws w = workspace(batch, rows, cols);
  uint8_t* base = (uint8_t*)work;
  float2* part = (float2*)(base + w.part);
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
                              (const float*)M, mu, (int)nesterov, rows, cols, w.ldx, (const float2*)part, w.parts, eps,
                              hi[0], lo);
  count_launches(2);
  const bool tall = rows > cols;
  const int m = w.m;
  const Operand o{O, m, m, w.lda}, p{B, m, m, w.lda};
  // slabs of X, of A, and transposed ones of A and of B (64 rows of 32 columns)
  CUtensorMap mX[2], mLo, mO, mOT, mBT;
  const int64_t xa = w.ldx * rows, aa = w.lda * m;
  if (!product_map(&mX[0], hi[0], rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mX[1], hi[1], rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mLo, lo, rows, cols, w.ldx, xa, batch, 32, true) ||
      !product_map(&mO, O, m, m, w.lda, aa, batch, 32, true) ||
      !product_map(&mOT, O, m, m, w.lda, aa, batch, 64, true, 32) ||
      !product_map(&mBT, B, m, m, w.lda, aa, batch, 64, true, 32))
    return kLaunchFailed;
  for (int i = 0; i < steps && e == cudaSuccess; ++i) {
    const float *c = coef + 3 * i;
    const Operand x{hi[i & 1], rows, cols, w.ldx};
    const GramEpi::Args ga{mOT, O, d, w.lda, w.dpad};
    e = tall ? product<true, true, true, GramEpi>(x, x, m, m, rows, batch, ga, st)
             : product<false, false, true, GramEpi>(x, x, m, m, cols, batch, ga, st);
    if (e != cudaSuccess) break;
    const float f = scale[i] * kADown;
    const PolyEpi::Args pa{mO, mBT, O, B, d, db, w.lda, w.dpad, c[1] * f, c[2] * f, 1.f / f};
    e = product<false, false, true, PolyEpi>(o, o, m, m, m, batch, pa, st);
    if (e != cudaSuccess) break;
    auto apply = [&](auto epi) {
      using E = decltype(epi);
      typename E::Args a{};
      a.hi = mX[i & 1];
      a.lo = mLo;
      a.hi_rows = hi[i & 1];
      a.hi_out = hi[(i + 1) & 1];
      a.lo_out = lo;
      a.db = db;
      a.ld = w.ldx;
      a.dpad = w.dpad;
      a.a = c[0];
      a.down = 1.f / scale[i];
      a.by_col = tall;
      a.out = out;
      a.out_bf16 = out_bf16;
      a.update = update;
      a.vec = cols % (out_bf16 ? 16 : 8) == 0 && al(out, 32);
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
