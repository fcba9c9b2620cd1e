// Cross entropy of a head over a large vocabulary from the head's inputs and
// weights: the logits are never stored.
//
//   z = scale X W^T,  lse = log sum_j e^{z_j}
//   loss = lse - (1 - e) z_y - e mean_j z_j + c lse^2     (smoothing e, penalty c)
//   dz_j = g ((1 + 2 c lse) p_j - (1 - e) [j = y] - e / V),  p = e^{z - lse}
//   dX = scale dz W,  dW = scale dz^T X
//
// Forward: one product whose epilogue reduces each tile's 256 (or 128)
// columns of a row to their maximum and their sum of 2^(z - max), from tensor
// memory; a second launch joins a row's tiles (V / 256 pairs a row). Backward:
// the vocabulary is taken in pieces of as many columns as keep a piece's dz
// within 2^28 values; a piece's logits are made again and leave as dz
// (rounded to bf16, as the operands of the next two products have to be), dX
// is summed over the pieces in fp32 and rounded once, dW's rows are the
// piece's own. 2 T V h operations forward and 6 T V h backward, all on the
// tensor cores, bound them.
//
// Rows that are not scored (label below 0) have dz = 0 whatever their inputs
// hold: the backward works on a copy of X in which they are zero, since 0
// times an infinity or a NaN would reach every row of dW.
#include <algorithm>

#include "tile_product.cuh"

namespace mt {

MT_DEVICE_ERROR_READER(linear_ce_take_device_error)

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------------------
// Forward epilogue: per row and tile the maximum of z log2(e) and the sum of
// 2^(. - maximum); with smoothing the sum of the accumulators too; the
// label's own logit.
// ---------------------------------------------------------------------------
struct StatsEpi {
  struct Args {
    const int32_t* labels;
    float2* part;  // [M][num_n]
    float* sums;   // [M][num_n] or null
    float* zlab;   // [M]
    float scale;
  };
  struct Row {
    int label;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.label = at.row < s.M ? a.labels[at.row] : -1;
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              uint32_t tb) {
    const float k = a.scale * kLog2e;
    float m = -INFINITY, sum = 0.f, plain = 0.f;
    const int here = r.label - at.n0;  // the label's column in this tile, if it is one
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      if (at.n0 + c * 32 >= s.N) break;  // the same in every lane
      float v[32];
      tile_chunk(tb, c, v);
      if (a.sums) {
        float p0 = 0.f, p1 = 0.f;  // columns past N hold zeros
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          p0 += v[i];
          p1 += v[i + 1];
        }
        plain += p0 + p1;
      }
      if (here >= c * 32 && here < c * 32 + 32 && at.row < s.M) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) z = here == c * 32 + i ? v[i] : z;
        a.zlab[at.row] = z * a.scale;
      }
      if (at.n0 + c * 32 + 32 > s.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (at.n0 + c * 32 + i >= s.N) v[i] = -INFINITY;
      }
      float cm = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) cm = fmaxf(cm, v[i]);
      cm *= k;
      const float mn = fmaxf(m, cm);
      const float ref = mn == -INFINITY ? 0.f : mn;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        s0 += ex2(fmaf(v[i], k, -ref));
        s1 += ex2(fmaf(v[i + 1], k, -ref));
      }
      sum = sum * ex2(m - ref) + (s0 + s1);
      m = mn;
    }
    if (at.row < s.M) {
      const size_t o = (size_t)at.row * s.num_n + at.nb;
      a.part[o] = make_float2(m, sum);
      if (a.sums) a.sums[o] = plain;
    }
  }
};

// One warp a row: the tiles' pairs joined, the loss.
__global__ void __launch_bounds__(256)
    join_rows_kernel(const float2* part, const float* sums, const float* zlab, const int32_t* labels, int T, int V,
                     int num_n, float scale, float smooth, float zc, float* loss, float* lse_out) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= T) return;
  const int label = labels[row];
  if (label < 0 || label >= V) {
    if (lane == 0) {
      if (label >= V) report_error(kErrBadArg);
      loss[row] = lse_out[row] = label < 0 ? 0.f : __uint_as_float(0x7fffffffu);
    }
    return;
  }
  const float2* p = part + (size_t)row * num_n;
  float m = -INFINITY, s = 0.f, plain = 0.f;
  for (int i = lane; i < num_n; i += 32) {
    const float2 v = p[i];
    const float mn = fmaxf(m, v.x), ref = mn == -INFINITY ? 0.f : mn;
    s = s * ex2(m - ref) + v.y * ex2(v.x - ref);
    m = mn;
    if (sums) plain += sums[(size_t)row * num_n + i];
  }
  const float top = warp_max(m), ref = top == -INFINITY ? 0.f : top;
  s = warp_sum(s * ex2(m - ref));
  if (sums) plain = warp_sum(plain);
  if (lane == 0) {
    const float lse = fmaf(top, kLn2, logf(s));
    float l = lse - (1.f - smooth) * zlab[row];
    if (sums) l -= smooth * (plain * scale / (float)V);
    loss[row] = l + zc * lse * lse;
    lse_out[row] = lse;
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// X with the rows that are not scored set to zero: eight values a thread.
__global__ void __launch_bounds__(256) scored_rows_kernel(const uint16_t* X, int64_t ldx, const int32_t* labels, int V,
                                                          uint16_t* out, int T, int h) {
  grid_wait();
  grid_release();
  const int n8 = h >> 3;
  const int64_t all = (int64_t)T * n8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / n8), c = (int)(i - (int64_t)t * n8);
    const int y = labels[t];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (y >= 0 && y < V) v = *(const uint4*)(X + t * ldx + 8 * c);
    *(uint4*)(out + (int64_t)t * h + 8 * c) = v;
  }
}

// Eight values at p (16-byte aligned) in either type.
__device__ __forceinline__ void load8(const void* base, size_t at, bool bf16, float (&v)[8]) {
  if (bf16) {
    const uint4 w = *(const uint4*)((const uint16_t*)base + at);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bf2f(ws[e] & 0xffff);
      v[2 * e + 1] = bf2f(ws[e] >> 16);
    }
  } else {
    const float4* p = (const float4*)((const float*)base + at);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}
__device__ __forceinline__ void store8(void* base, size_t at, bool bf16, const float* v) {
  if (bf16) {
    *(uint4*)((uint16_t*)base + at) =
        make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
  } else {
    float4* p = (float4*)((float*)base + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// A piece's dz in bf16 (without the factor `scale`, which the next products'
// epilogues apply), zero past its last column up to the row stride.
struct GradEpi {
  struct Args {
    const int32_t* labels;
    const float *lse, *g;
    uint16_t* dz;
    int64_t ld;
    int V, v0;  // vocabulary, the piece's first column
    float scale, smooth, zc;
  };
  struct Row {
    int label;      // in the piece's columns
    float lse2, cp, cl, c0;
    bool scored;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    const int y = at.row < s.M ? a.labels[at.row] : -1;
    r.scored = y >= 0 && y < a.V;
    r.label = y - a.v0;
    const float g = r.scored ? a.g[at.row] : 0.f, lse = r.scored ? a.lse[at.row] : 0.f;
    r.lse2 = lse * kLog2e;
    r.cp = g * (1.f + 2.f * a.zc * lse);
    r.cl = g * (1.f - a.smooth);
    r.c0 = g * a.smooth / (float)a.V;
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              uint32_t tb) {
    const float k = a.scale * kLog2e;
    const int here = r.label - at.n0;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      const int col = at.n0 + c * 32;
      if (col >= a.ld) break;
      float v[32];
      tile_chunk(tb, c, v);
      if (at.row >= s.M) continue;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = r.scored ? fmaf(r.cp, ex2(fmaf(v[i], k, -r.lse2)), -r.c0) : 0.f;
      if (here >= c * 32 && here < c * 32 + 32 && r.scored) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] -= here == c * 32 + i ? r.cl : 0.f;
      }
      if (col + 32 > s.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i >= s.N) v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + 8 * i < a.ld) store8(a.dz, (size_t)at.row * a.ld + col + 8 * i, true, v + 8 * i);
    }
  }
};

// out = scale * accumulator (+ what is there, or an fp32 sum), N a multiple of 8.
struct SumEpi {
  struct Args {
    void* out;
    const void* add;  // same row stride; null: nothing
    int64_t ld;
    float scale;
    int out_bf16, add_bf16;
  };
  struct Row {};
  static __device__ __forceinline__ void load_row(const Args&, const ProductShape&, const TileAt&, Row&) {}
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row&,
                                              uint32_t tb) {
    const bool ok = at.row < s.M;
    const size_t row = (size_t)at.row * a.ld;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      const int col = at.n0 + c * 32;
      if (col >= s.N) break;
      float add[4][8];
      if (a.add && ok) {  // asked for before the accumulator, which the stores below would hold up
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col + 8 * i < s.N) load8(a.add, row + col + 8 * i, a.add_bf16, add[i]);
      }
      float v[32];
      tile_chunk(tb, c, v);
      if (!ok) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col + 8 * i >= s.N) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] = a.add ? fmaf(v[8 * i + j], a.scale, add[i][j]) : v[8 * i + j] * a.scale;
        store8(a.out, row + col + 8 * i, a.out_bf16, v + 8 * i);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Tiles of 256 x 256 on SM pairs where they fill half of the pairs, else 128 x
// 128 on single SMs.
bool wide(int64_t M, int64_t N) {
  return ((M + 255) / 256) * ((N + 255) / 256) >= mt_host::num_sms() / 4;
}

// The columns of a piece: dz of a piece has at most 2^28 values (or 256
// columns), pieces are alike in size and whole tiles.
int piece_cols(int T, int V) {
  const int64_t most = std::max<int64_t>(256, ((int64_t)1 << 28) / T / 256 * 256);
  const int64_t pieces = (V + most - 1) / most;
  return (int)std::min<int64_t>(up((size_t)((V + pieces - 1) / pieces), 256), up(V, 64));
}

struct BwdWs {
  size_t x, dz, acc, total;
  int cols;
};
BwdWs bwd_ws(int T, int V, int h) {
  BwdWs o;
  o.cols = piece_cols(T, V);
  o.x = 0;
  o.dz = up((size_t)T * h * 2, 256);
  o.acc = o.dz + up((size_t)T * o.cols * 2, 256);
  o.total = o.acc + (o.cols < V ? up((size_t)T * h * 4, 256) : 0);
  return o;
}

template <bool A_MN, bool B_MN, class E>
cudaError_t product(const void* A, int64_t lda, const void* B, int64_t ldb, int M, int N, int K,
                    const typename E::Args& args, cudaStream_t st) {
  auto go = [&](auto cfg) {
    using C = decltype(cfg);
    CUtensorMap ta, tb;
    const int ar = A_MN ? K : M, ac = A_MN ? M : K, br = B_MN ? K : N, bc = B_MN ? N : K;
    if (!product_map(&ta, A, ar, ac, lda, lda, 1, a_box<C>(), false) ||
        !product_map(&tb, B, br, bc, ldb, ldb, 1, b_box<C>(), false))
      return cudaErrorUnknown;
    return launch_product<C, E>(ta, tb, product_shape<C>(M, N, K, 1), args, st);
  };
  if (wide(M, N)) return go(ProductCfg<256, true, A_MN, B_MN>());
  return go(ProductCfg<128, false, A_MN, B_MN>());
}

}  // namespace

bool linear_ce_dims(int T, int V, int h) {
  // counters of tiles and of the statistics stay within 31 bits
  return T > 0 && V > 0 && h > 0 && T <= (1 << 24) && V <= (1 << 24) && h <= (1 << 16) && h % 8 == 0 &&
         (int64_t)T * V <= ((int64_t)1 << 40);
}

size_t linear_ce_fwd_workspace(int T, int V) {
  const size_t n = (size_t)T * ((V + 127) / 128);
  return up(n * 8, 256) + up(n * 4, 256) + up((size_t)T * 4, 256);
}
size_t linear_ce_bwd_workspace(int T, int V, int h) { return bwd_ws(T, V, h).total; }

int linear_ce_fwd(const uint16_t* X, const uint16_t* W, const int32_t* labels, float scale, float smooth, float zc,
                  float* loss, float* lse, void* work, int T, int V, int h, int ldx, int ldw, cudaStream_t st) {
  const size_t n = (size_t)T * ((V + 127) / 128);
  StatsEpi::Args a;
  a.labels = labels;
  a.part = (float2*)work;
  a.sums = smooth != 0.f ? (float*)((uint8_t*)work + up(n * 8, 256)) : nullptr;
  a.zlab = (float*)((uint8_t*)work + up(n * 8, 256) + up(n * 4, 256));
  a.scale = scale;
  cudaError_t e = product<false, false, StatsEpi>(X, ldx, W, ldw, T, V, h, a, st);
  if (e != cudaSuccess) return kLaunchFailed;
  const int num_n = wide(T, V) ? (V + 255) / 256 : (V + 127) / 128;
  e = mt_host::launch_early(join_rows_kernel, (T + 7) / 8, 256, 0, st, 1, (const float2*)a.part, (const float*)a.sums,
                            (const float*)a.zlab, labels, T, V, num_n, scale, smooth, zc, loss, lse);
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

int linear_ce_bwd(const uint16_t* X, const uint16_t* W, const int32_t* labels, float scale, float smooth, float zc,
                  const float* lse, const float* g, void* dX, bool dx_bf16, void* dW, bool dw_bf16, bool accumulate,
                  void* work, int T, int V, int h, int ldx, int ldw, cudaStream_t st) {
  const BwdWs o = bwd_ws(T, V, h);
  uint16_t* xs = (uint16_t*)((uint8_t*)work + o.x);
  uint16_t* dz = (uint16_t*)((uint8_t*)work + o.dz);
  float* acc = dx_bf16 ? (float*)((uint8_t*)work + o.acc) : (float*)dX;
  const int64_t units = ((int64_t)T * (h / 8) + 255) / 256;
  cudaError_t e = mt_host::launch_early(scored_rows_kernel, (int)std::min<int64_t>(units, 152 * 16), 256, 0, st, 1, X,
                                        (int64_t)ldx, labels, V, xs, T, h);
  count_launches(1);
  for (int v0 = 0; v0 < V && e == cudaSuccess; v0 += o.cols) {
    const int n = std::min(o.cols, V - v0);
    const int64_t ld = (int64_t)up(n, 64);
    const uint16_t* Wp = W + (int64_t)v0 * ldw;
    GradEpi::Args a{labels, lse, g, dz, ld, V, v0, scale, smooth, zc};
    e = product<false, false, GradEpi>(xs, h, Wp, ldw, T, n, h, a, st);
    if (e == cudaSuccess && dX) {
      const bool last = v0 + n == V;
      SumEpi::Args s{last ? dX : acc, v0 ? acc : nullptr, h, scale, last && dx_bf16, 0};
      e = product<false, true, SumEpi>(dz, ld, Wp, ldw, T, h, n, s, st);
    }
    if (e == cudaSuccess && dW) {
      void* out = dw_bf16 ? (void*)((uint16_t*)dW + (int64_t)v0 * h) : (void*)((float*)dW + (int64_t)v0 * h);
      SumEpi::Args s{out, accumulate ? out : nullptr, h, scale, dw_bf16, dw_bf16};
      e = product<true, true, SumEpi>(dz, ld, xs, h, n, h, T, s, st);
    }
  }
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

bool linear_ce_aligned(const void* X, const void* W, const void* dX, const void* dW, const void* work) {
  return al(X, 16) && al(W, 16) && al(dX, 16) && al(dW, 16) && al(work, 256);
}

}  // namespace mt
