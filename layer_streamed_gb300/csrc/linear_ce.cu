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
// hold; dW is made from a copy of X in which they are zero, since 0 times an
// infinity or a NaN would reach every row of it.
#include <algorithm>
#include <type_traits>

#include "tile_product.cuh"

namespace mt {

namespace {

// Labels past the vocabulary. A word of its own: a bit in g_device_error would
// make every wait of this file's kernels give up until the host has read it.
static __device__ uint32_t g_bad_label = 0;
MT_DEVICE_ERROR_READER(take_timeouts)

}  // namespace

uint32_t linear_ce_take_device_error() {
  uint32_t bad = 0;
  const uint32_t e = take_timeouts(), zero = 0;
  if (cudaMemcpyFromSymbol(&bad, g_bad_label, 4) != cudaSuccess) return 0xffffffffu;
  if (bad) cudaMemcpyToSymbol(g_bad_label, &zero, 4);
  return e | bad;
}

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The label's logits of R tokens side by side, x and w their rows (x null:
// none), U pieces of a row asked for together: sums in fp32, h / 32 terms a
// lane and then a tree, the same bits wherever they are made. The tensor core's
// long sums come out a few 2^-24 of their terms short, 1.6e-6 of a loss at h =
// 4096, and the label's own is most of what counts of that: where its
// probability is high, in the log-sum-exp, and then in dz = p - 1. So both
// directions take it from here, and the products' column of the label is not
// used. By the epilogue's warps, while products run.
template <int R, int U>
__device__ __forceinline__ void label_logits(const uint16_t* const (&x)[R], const uint16_t* const (&w)[R], int h,
                                             float scale, float (&z)[R]) {
  const int n8 = h >> 3;
  float z0[R] = {}, z1[R] = {};
#pragma unroll 1
  for (int i0 = (int)lane_id(); i0 - (int)lane_id() < n8; i0 += 32 * U) {
    uint4 p[R][U], q[R][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        p[r][u] = q[r][u] = make_uint4(0, 0, 0, 0);
        if (x[r] && i0 + 32 * u < n8) {
          p[r][u] = ((const uint4*)x[r])[i0 + 32 * u];
          q[r][u] = ((const uint4*)w[r])[i0 + 32 * u];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t ps[4] = {p[r][u].x, p[r][u].y, p[r][u].z, p[r][u].w},
                       qs[4] = {q[r][u].x, q[r][u].y, q[r][u].z, q[r][u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z0[r] = fmaf(bf2f(ps[e] & 0xffff), bf2f(qs[e] & 0xffff), z0[r]);
          z1[r] = fmaf(bf2f(ps[e] >> 16), bf2f(qs[e] >> 16), z1[r]);
        }
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < R; ++r) z[r] = __fmul_rn(warp_sum(z0[r] + z1[r]), scale);
}

// ---------------------------------------------------------------------------
// Forward epilogue: per row and tile the maximum of z log2(e) and the sum of
// 2^(. - maximum) over all columns but the label's; with smoothing the sum of
// the accumulators too. The label's term joins the others' sum last
// (join_rows_kernel).
// ---------------------------------------------------------------------------
// Two warps a row of a tile, half of the columns each, hide each other's
// latencies: with one, 8 us a tile of 256 x 256 against 4.2 us of MMAs at h = 1024.
struct StatsEpi : NoSlabs {
  static constexpr int WARPS = 8, SLABS = 0;
  struct Args {
    const int32_t* labels;
    float2* part;  // [M][2 num_n]
    float* sums;   // [M][2 num_n] or null
    float* zlab;   // [M]: the label's logit
    float scale;
    const uint16_t *X, *W;
    int64_t ldx, ldw;
    int T, V, h;
  };
  static __device__ __forceinline__ void begin(const Args& a, int warp) {
    for (int t = (int)blockIdx.x * WARPS + warp; t < a.T; t += (int)gridDim.x * WARPS) {
      const int y = a.labels[t];
      if (y < 0 || y >= a.V) continue;
      float z[1];
      label_logits<1, 4>({a.X + t * a.ldx}, {a.W + y * a.ldw}, a.h, a.scale, z);
      if (lane_id() == 0) a.zlab[t] = z[0];
    }
  }
  struct Row {
    int label;
  };
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    r.label = at.row < s.M ? max(a.labels[at.row], -1) : -1;
  }
  // This warp's share of the columns: m = max v k, the sum of 2^(v k - m) and
  // (FAR = false, with sums) that of v. m is rounded, which is a factor of the
  // sum that goes with it; FAR, for logits so large that the factor could leave
  // fp32, takes the exponents from differences to the maximum itself.
  template <int BN, bool FAR>
  static __device__ __forceinline__ void scan(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              const EpiWarp& w, uint32_t tb, float& m_out, float& sum_out, float& plain) {
    const float k = a.scale * kLog2e;
    float top = -INFINITY, m = -INFINITY, sum = 0.f;
    const int here = r.label - at.n0;  // the label's column in this tile, if it is one
#pragma unroll 1
    for (int c = w.part * (BN / 64); c < (w.part + 1) * (BN / 64); ++c) {
      if (at.n0 + c * 32 >= s.N) break;  // the same in every lane
      float v[32];
      tile_chunk(tb, c, v);
      if (!FAR && a.sums) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};  // columns past N hold zeros
#pragma unroll
        for (int i = 0; i < 32; ++i) p[i & 3] += v[i];
        plain += (p[0] + p[1]) + (p[2] + p[3]);
      }
      if (here >= c * 32 && here < c * 32 + 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = here == c * 32 + i ? -INFINITY : v[i];
      }
      if (at.n0 + c * 32 + 32 > s.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (at.n0 + c * 32 + i >= s.N) v[i] = -INFINITY;
      }
      float cm[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < 32; ++i) cm[i & 3] = fmaxf(cm[i & 3], v[i]);
      const float here_top = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
      if (FAR) top = fmaxf(top, here_top);
      const float mn = FAR ? top * k : fmaxf(m, here_top * k);
      const float ref = mn == -INFINITY ? 0.f : mn, from = top == -INFINITY ? 0.f : top;
      float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i & 3] += ex2(FAR ? (v[i] - from) * k : fmaf(v[i], k, -ref));
      sum = sum * ex2(m - ref) + ((p[0] + p[1]) + (p[2] + p[3]));
      m = mn;
    }
    m_out = m;
    sum_out = sum;
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    float m, sum, plain = 0.f;
    scan<BN, false>(a, s, at, r, w, tb, m, sum, plain);
    // rows behind the last token hold what the ring held
    const bool far = at.row < s.M && fabsf(m) > 0x1p22f && m != -INFINITY;
    if (__any_sync(0xffffffffu, far)) {
      float m2, sum2;
      scan<BN, true>(a, s, at, r, w, tb, m2, sum2, plain);
      m = far ? m2 : m;
      sum = far ? sum2 : sum;
    }
    if (at.row < s.M) {
      const size_t o = (size_t)at.row * (2 * s.num_n) + 2 * at.nb + w.part;
      a.part[o] = make_float2(m, sum);  // (-inf, 0) where the half lies past N
      if (a.sums) a.sums[o] = plain;
    }
  }
};

// One warp a row: the tiles' pairs joined, then the label's term with them.
// With rest = s 2^top the others' sum, the loss without smoothing and penalty
// is log(1 + rest / e^z): never below 0, and with its own size's accuracy
// where the label holds nearly everything.
__global__ void __launch_bounds__(256)
    join_rows_kernel(const float2* part, const float* sums, const float* zlab, const int32_t* labels, int T, int V,
                     int parts, float scale, float smooth, float zc, float* loss, float* lse_out) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= T) return;
  const int label = labels[row];
  if (label < 0 || label >= V) {
    if (lane == 0) {
      if (label >= V) atomicOr(&g_bad_label, (uint32_t)kErrBadArg);
      loss[row] = lse_out[row] = label < 0 ? 0.f : __uint_as_float(0x7fffffffu);
    }
    return;
  }
  const float2* p = part + (size_t)row * parts;
  float m = -INFINITY, s = 0.f, plain = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = p[i];
    const float mn = fmaxf(m, v.x), ref = mn == -INFINITY ? 0.f : mn;
    s = s * ex2(m - ref) + v.y * ex2(v.x - ref);
    m = mn;
    if (sums) plain += sums[(size_t)row * parts + i];
  }
  const float top = warp_max(m);
  s = warp_sum(s * ex2(m - (top == -INFINITY ? 0.f : top)));
  if (sums) plain = warp_sum(plain);
  if (lane == 0) {
    const float z = zlab[row], d = fmaf(-kLog2e, z, top);
    const bool over = d > 0.f;
    // log(1 + r) of small r as log(u) r / (u - 1), u = 1 + r as rounded (Kahan's)
    const float r = s * ex2(over ? 0.f : d), u = over ? s + ex2(-d) : 1.f + r, lg = logf(u);
    const float more = over ? lg : u == 1.f ? r : lg * __fdividef(r, u - 1.f);
    const float lse = over ? fmaf(top, kLn2, lg) : z + more;
    float l = over ? fmaf(d, kLn2, lg) : more;
    if (!(z < INFINITY)) l = z - z;  // not a number
    if (sums) l += smooth * (z - plain * scale / (float)V);
    loss[row] = l + zc * lse * lse;
    lse_out[row] = lse;
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
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
// epilogues apply). Two warps a row as above, slabs of 64 columns out by TMA,
// one place a warp (two leave the ring a step shorter: 2 % slower).
struct GradEpi : NoSlabs {
  static constexpr int kSlab = 4096;
  static constexpr int WARPS = 8, SLABS = kSlab;
  static constexpr float kFar = 0x1p18f;
  struct Args {
    CUtensorMap dz;
    const int32_t* labels;
    const float *lse, *g;
    int V, v0;  // vocabulary, the piece's first column
    float scale, smooth, zc;
    // with the first piece: X with the rows that are not scored set to zero
    const uint16_t* X;
    uint16_t* xs;  // null: not wanted
    const uint16_t* W;  // the piece's rows
    int64_t ldx, ldw;
    int T, h;
  };
  // The copy of X is made by the epilogue's warps, which have nothing to do
  // until the first tile's products are there.
  static __device__ __forceinline__ void begin(const Args& a, int warp) {
    if (!a.xs) return;
    const int n8 = a.h >> 3;
    const int64_t all = (int64_t)a.T * n8, step = (int64_t)gridDim.x * (32 * WARPS);
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * (32 * WARPS) + warp * 32 + lane_id(); i < all; i += step) {
      const int t = (int)(i / n8), c = (int)(i - (int64_t)t * n8);
      const int y = a.labels[t];
      uint4 v = *(const uint4*)(a.X + t * a.ldx + 8 * c);
      if (y < 0 || y >= a.V) v = make_uint4(0, 0, 0, 0);
      *(uint4*)(a.xs + (int64_t)t * a.h + 8 * c) = v;
    }
  }
  struct Row {
    int label;  // in the piece's columns
    float lse2, cp, c0, dz;  // dz: the label's
    bool scored;
  };
  // The label's dz is made before its tile is there, by the warp whose columns
  // hold it (a row in V / 128 of them), from z - lse, which is exact where they
  // are near each other: its p - 1 may be all that is left of it. (Nothing to be
  // seen at vocabularies of 32000 and h of 1024 up, 2 % at h = 256; where every
  // row's label is in the one tile there is, V 256, 16384 tokens, 13 to 15 %,
  // which a launch of its own for all rows takes as well: 7 tokens, V 32000,
  // then 51.7 us, so 47.4.)
  static __device__ __forceinline__ void load_row(const Args& a, const ProductShape& s, const TileAt& at, Row& r) {
    const int y = at.row < s.M ? a.labels[at.row] : -1;
    r.scored = y >= 0 && y < a.V;
    r.label = r.scored ? y - a.v0 : -1;
    const float g = r.scored ? a.g[at.row] : 0.f, lse = r.scored ? a.lse[at.row] : 0.f;
    r.lse2 = lse * kLog2e;
    r.cp = g * (1.f + 2.f * a.zc * lse);
    r.c0 = g * a.smooth / (float)a.V;
    r.dz = 0.f;
    const int half = at.width / 2, c = r.label - at.n0 - ((int)(warp_id() - 2) >> 2) * half;
    const int lane = (int)lane_id();
    uint32_t left = __ballot_sync(0xffffffffu, c >= 0 && c < half && r.label < s.N);
    auto next = [&](auto rows) {  // the next rows of those left
      constexpr int R = decltype(rows)::value;
      const uint16_t *x[R], *w[R];
      int l[R];
      float z[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        l[k] = left ? __ffs(left) - 1 : -1;
        left &= left - 1;
        x[k] = l[k] < 0 ? nullptr : a.X + (at.row0 + l[k]) * a.ldx;
        w[k] = a.W + __shfl_sync(0xffffffffu, r.label, max(l[k], 0)) * (l[k] < 0 ? 0 : a.ldw);
      }
      label_logits<R, 8 / R>(x, w, a.h, a.scale, z);
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (lane == l[k]) r.dz = fmaf(r.cp, ex2(min_nan((z[k] - lse) * kLog2e, 0.f)), -r.c0) - g * (1.f - a.smooth);
    };
    while (left & (left - 1)) next(std::integral_constant<int, 4>());
    if (left) next(std::integral_constant<int, 1>());
  }
  // FAR: some row's logits are so large that their roundings would pass for p above 1
  template <int BN, bool FAR>
  static __device__ __forceinline__ void write(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                               EpiWarp& w, uint32_t tb) {
    const float k = a.scale * kLog2e, most = fabsf(r.lse2) > kFar ? 0.f : INFINITY;
    const int here = r.label - at.n0;
#pragma unroll 1
    for (int j = w.part * (BN / 128); j < (w.part + 1) * (BN / 128); ++j) {
      const int col = at.n0 + j * 64;
      if (col >= s.N) break;
      uint8_t* slab = w.smem;
      if (w.lane == 0) bulk_store_wait<0, true>();
      __syncwarp();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int c0 = j * 64 + half * 32;
        float v[32];
        tile_chunk(tb, 2 * j + half, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float e = fmaf(v[i], k, -r.lse2);
          v[i] = r.scored ? fmaf(r.cp, ex2(FAR ? min_nan(e, most) : e), -r.c0) : 0.f;
        }
        if (here >= c0 && here < c0 + 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = here == c0 + i ? r.dz : v[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *slab_piece(slab, w.lane, half * 4 + i) =
              make_uint4(pack_bf2(v[8 * i], v[8 * i + 1]), pack_bf2(v[8 * i + 2], v[8 * i + 3]),
                         pack_bf2(v[8 * i + 4], v[8 * i + 5]), pack_bf2(v[8 * i + 6], v[8 * i + 7]));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0) {
        tma_store_3d(&a.dz, slab, col, at.row0, 0);
        bulk_store_commit();
      }
    }
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row& r,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    if (__any_sync(0xffffffffu, fabsf(r.lse2) > kFar)) write<BN, true>(a, s, at, r, w, tb);
    else write<BN, false>(a, s, at, r, w, tb);
  }
};

// out = scale * accumulator, N a multiple of 8, by slabs of 64 bf16 or 32 fp32
// columns; or added to what is there or to an fp32 sum, 32 columns at a time
// straight to memory, the addend asked for ahead of the accumulator. Two warps
// a row as above. (From the lanes' rows, 32 bytes at a time: dW of 7 tokens, V
// 128256, h 4096, 397 us, so 353. Adding to dW goes that way still: a backward
// of 512 x 32000 x 1024 takes a third longer in bf16 and 58 % in fp32, of 8192 x
// 128256 x 4096 3 % and 1 %.)
struct SumEpi : NoSlabs {
  static constexpr int kSlab = 4096;
  static constexpr int WARPS = 8, SLABS = kSlab;
  struct Args {
    CUtensorMap map;  // of out
    void* out;
    const void* add;  // same row stride; null: nothing
    int64_t ld;
    float scale;
    int out_bf16, add_bf16;
  };
  struct Row {};
  static __device__ __forceinline__ void load_row(const Args&, const ProductShape&, const TileAt&, Row&) {}
  template <int BN, bool BF16>
  static __device__ __forceinline__ void written(const Args& a, const ProductShape& s, const TileAt& at, EpiWarp& w,
                                                 uint32_t tb) {
    constexpr int WIDE = BF16 ? 64 : 32;
    const int c0 = at.n0 + w.part * (BN / 2), c1 = min(c0 + BN / 2, s.N);
#pragma unroll 1
    for (int col = c0; col < c1; col += WIDE) {
      uint8_t* slab = w.smem;
      if (w.lane == 0) bulk_store_wait<0, true>();
      __syncwarp();
#pragma unroll
      for (int half = 0; half < WIDE / 32; ++half) {
        float v[32];
        tile_chunk(tb, (col - at.n0) / 32 + half, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= a.scale;
        if (BF16) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *slab_piece(slab, w.lane, half * 4 + i) =
                make_uint4(pack_bf2(v[8 * i], v[8 * i + 1]), pack_bf2(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf2(v[8 * i + 4], v[8 * i + 5]), pack_bf2(v[8 * i + 6], v[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *(float4*)slab_piece(slab, w.lane, i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0) {
        tma_store_3d(&a.map, slab, col, at.row0, at.b);
        bulk_store_commit();
      }
    }
  }
  template <int BN>
  static __device__ __forceinline__ void tile(const Args& a, const ProductShape& s, const TileAt& at, const Row&,
                                              EpiWarp& w, uint32_t tb) {
    if (at.row0 >= s.M) return;
    if (!a.add) {
      if (a.out_bf16) written<BN, true>(a, s, at, w, tb);
      else written<BN, false>(a, s, at, w, tb);
      return;
    }
    const bool ok = at.row < s.M;
    const size_t row = (size_t)at.row * a.ld;
#pragma unroll 1
    for (int c = w.part * (BN / 64); c < (w.part + 1) * (BN / 64); ++c) {
      const int col = at.n0 + c * 32;
      if (col >= s.N) break;
      float add[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ok && col + 8 * i < s.N) load8(a.add, row + col + 8 * i, a.add_bf16, add[i]);
      float v[32];
      tile_chunk(tb, c, v);
      if (!ok) continue;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], a.scale, add[i >> 3][i & 7]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + 8 * i < s.N) store8(a.out, row + col + 8 * i, a.out_bf16, v + 8 * i);
    }
  }
};

// A gradient from the partial sums of the ranges that its K was cut into, in
// their order, and what it is added to.
__global__ void __launch_bounds__(256)
    join_ranges_kernel(const float* part, int ranges, int64_t n, void* out, int bf16, int add) {
  grid_wait();
  grid_release();
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (add && bf16) {
      const uint2 o = *(const uint2*)((const uint16_t*)out + i);
      s = make_float4(bf2f(o.x & 0xffff), bf2f(o.x >> 16), bf2f(o.y & 0xffff), bf2f(o.y >> 16));
    } else if (add) {
      s = *(const float4*)((const float*)out + i);
    }
#pragma unroll 8
    for (int r = 0; r < ranges; ++r) {
      const float4 p = *(const float4*)(part + r * n + i);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    if (bf16) *(uint2*)((uint16_t*)out + i) = make_uint2(pack_bf2(s.x, s.y), pack_bf2(s.z, s.w));
    else *(float4*)((float*)out + i) = s;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kSms = 152;  // sizes the workspace, whatever machine asks
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Tiles of 256 x 256 on SM pairs where they fill half of the pairs; 128 x 128
// on single SMs for fewer of them, for few rows (M up to 128: half of a pair's
// tile would be empty; 128 tokens, V 32000, h 1024: dX 40 us on pairs, 36.4 on
// single SMs) and for shallow sums (K up to 128: what counts is how many warps
// write results; dW of V 32000, h 1024: 7 tokens 39.8 us on pairs, 33.6 so, 128
// tokens 41.9 and 39.4, 256 tokens 46.5 and 51.4).
bool wide(int64_t M, int64_t N, int64_t K) {
  return M > 128 && K > 128 && ((M + 255) / 256) * ((N + 255) / 256) >= mt_host::num_sms() / 4;
}

// The columns of a piece: dz of a piece has at most 2^28 values (or 256
// columns), pieces are alike in size and whole tiles.
int piece_cols(int T, int V) {
  const int64_t most = std::max<int64_t>(256, ((int64_t)1 << 28) / T / 256 * 256);
  const int64_t pieces = (V + most - 1) / most;
  return (int)std::min<int64_t>(up((size_t)((V + pieces - 1) / pieces), 256), up(V, 64));
}

// Ranges that the K of a gradient's product [M, N] is cut into: few tiles
// (few tokens, or a small vocabulary) leave most of the GPU idle otherwise.
// The number that takes the least time by a count of SM pairs' steps (512
// cycles for a 256 x 256 tile 64 deep; 300 for 128 x 128 on one SM), with what
// the partial sums cost to write and to read at 3500 bytes a cycle (dX of 7
// tokens, V 32000, h 1024: 141 us in one range, 17 in nineteen).
int ranges_of(int64_t M, int64_t N, int K) {
  const int64_t edge = M <= 128 ? 128 : 256, units = M <= 128 ? kSms : kSms / 2, step = M <= 128 ? 300 : 512;
  const int64_t tiles = ((M + edge - 1) / edge) * ((N + edge - 1) / edge), steps = (K + 63) / 64;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int64_t r = 1; r <= units && (r == 1 || (tiles < 4 * units && steps / r >= 4)); ++r) {
    const int64_t cycles =
        (tiles * r + units - 1) / units * ((steps + r - 1) / r) * step + (r > 1 ? 4000 + r * M * N * 8 / 3500 : 0);
    if (cycles < least) {
      least = cycles;
      best = (int)r;
    }
  }
  return best;
}

struct BwdWs {
  size_t x, dz, acc, total;
  int cols, dx_ranges, dw_ranges;
};
BwdWs bwd_ws(int T, int V, int h) {
  BwdWs o;
  o.cols = piece_cols(T, V);
  o.x = 0;
  o.dz = up((size_t)T * h * 2, 256);
  o.acc = o.dz + up((size_t)T * o.cols * 2, 256);
  const bool pieces = o.cols < V;
  o.dx_ranges = pieces ? 1 : ranges_of(T, h, V);
  o.dw_ranges = pieces ? 1 : ranges_of(V, h, T);
  // dX's sum over the pieces, or partial sums of either
  const size_t dx = pieces || o.dx_ranges > 1 ? (size_t)o.dx_ranges * T * h * 4 : 0;
  const size_t dw = o.dw_ranges > 1 ? (size_t)o.dw_ranges * V * h * 4 : 0;
  o.total = o.acc + up(std::max(dx, dw), 256);
  return o;
}

template <bool A_MN, bool B_MN, class E>
cudaError_t product(const void* A, int64_t lda, const void* B, int64_t ldb, int M, int N, int K,
                    const typename E::Args& args, cudaStream_t st, int ranges = 1) {
  auto go = [&](auto cfg) {
    using C = decltype(cfg);
    CUtensorMap ta, tb;
    const int ar = A_MN ? K : M, ac = A_MN ? M : K, br = B_MN ? K : N, bc = B_MN ? N : K;
    if (!product_map(&ta, A, ar, ac, lda, lda, 1, a_box<C>(M, K), false) ||
        !product_map(&tb, B, br, bc, ldb, ldb, 1, b_box<C>(K), false))
      return cudaErrorUnknown;
    ProductShape s = product_shape<C>(M, N, K, 1);
    if (ranges > 1) {
      const int steps = (K + C::BK - 1) / C::BK;
      s.split_kb = (steps + ranges - 1) / ranges;
      s.batch = (steps + s.split_kb - 1) / s.split_kb;
    }
    return launch_product<C, E>(ta, tb, s, args, st);
  };
  if (wide(M, N, K) || (ranges > 1 && M > 128)) return go(ProductCfg<256, true, A_MN, B_MN>());
  if constexpr (A_MN) {  // dW of few tokens
    if (K < 64) return go(ProductCfg<128, false, A_MN, B_MN, false, false, true>());
  }
  return go(ProductCfg<128, false, A_MN, B_MN>());
}

// out [M, N] = scale * (product over K) + add, dense, in `ranges` of K by way
// of partial sums (add is then out itself or nothing).
template <bool A_MN, bool B_MN>
cudaError_t gradient(const void* A, int64_t lda, const void* B, int64_t ldb, int M, int N, int K, int ranges,
                     float* part, void* out, bool bf16, const void* add, bool add_bf16, float scale, cudaStream_t st) {
  const int steps = (K + 63) / 64, each = (steps + ranges - 1) / ranges, used = (steps + each - 1) / each;
  const int64_t all = (int64_t)M * N;
  SumEpi::Args s{};
  s.out = ranges > 1 ? (void*)part : out;
  s.add = ranges > 1 ? nullptr : add;
  s.ld = N;
  s.scale = scale;
  s.out_bf16 = ranges == 1 && bf16;
  s.add_bf16 = add_bf16;
  const int64_t apart = used > 1 ? all : N;
  if (!(s.out_bf16 ? product_map(&s.map, s.out, M, N, N, apart, used, 32, false)
                   : product_map_f32(&s.map, s.out, M, N, N, apart, used)))
    return cudaErrorUnknown;
  cudaError_t e = product<A_MN, B_MN, SumEpi>(A, lda, B, ldb, M, N, K, s, st, ranges);
  if (ranges > 1 && e == cudaSuccess) {
    e = mt_host::launch_early(join_ranges_kernel, (int)std::min<int64_t>((all + 1023) / 1024, kSms * 8), 256, 0, st, 1,
                              (const float*)part, used, all, out, (int)bf16, (int)(add != nullptr));
    count_launches(1);
  }
  return e;
}

}  // namespace

bool linear_ce_dims(int T, int V, int h) {
  // counters of tiles and of the statistics stay within 31 bits
  return T > 0 && V > 0 && h > 0 && T <= (1 << 24) && V <= (1 << 24) && h <= (1 << 16) && h % 8 == 0 &&
         (int64_t)T * V <= ((int64_t)1 << 40);
}

size_t linear_ce_fwd_workspace(int T, int V) {
  const size_t n = (size_t)T * (2 * ((V + 127) / 128));
  return up(n * 8, 256) + up(n * 4, 256) + up((size_t)T * 4, 256);
}
size_t linear_ce_bwd_workspace(int T, int V, int h) { return bwd_ws(T, V, h).total; }

int linear_ce_fwd(const uint16_t* X, const uint16_t* W, const int32_t* labels, float scale, float smooth, float zc,
                  float* loss, float* lse, void* work, int T, int V, int h, int ldx, int ldw, cudaStream_t st) {
  const size_t n = (size_t)T * (2 * ((V + 127) / 128));
  StatsEpi::Args a{};
  a.labels = labels;
  a.part = (float2*)work;
  a.sums = smooth != 0.f ? (float*)((uint8_t*)work + up(n * 8, 256)) : nullptr;
  a.zlab = (float*)((uint8_t*)work + up(n * 8, 256) + up(n * 4, 256));
  a.scale = scale;
  a.X = X;
  a.W = W;
  a.ldx = ldx;
  a.ldw = ldw;
  a.T = T;
  a.V = V;
  a.h = h;
  cudaError_t e = product<false, false, StatsEpi>(X, ldx, W, ldw, T, V, h, a, st);
  if (e != cudaSuccess) return kLaunchFailed;
  const int parts = 2 * (wide(T, V, h) ? (V + 255) / 256 : (V + 127) / 128);
  e = mt_host::launch_early(join_rows_kernel, (T + 7) / 8, 256, 0, st, 1, (const float2*)a.part, (const float*)a.sums,
                            (const float*)a.zlab, labels, T, V, parts, scale, smooth, zc, loss, lse);
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

int linear_ce_bwd(const uint16_t* X, const uint16_t* W, const int32_t* labels, float scale, float smooth, float zc,
                  const float* lse, const float* g, void* dX, bool dx_bf16, void* dW, bool dw_bf16, bool accumulate,
                  void* work, int T, int V, int h, int ldx, int ldw, cudaStream_t st) {
  const BwdWs o = bwd_ws(T, V, h);
  uint16_t* xs = (uint16_t*)((uint8_t*)work + o.x);
  uint16_t* dz = (uint16_t*)((uint8_t*)work + o.dz);
  float* part = (float*)((uint8_t*)work + o.acc);
  float* acc = dx_bf16 ? part : (float*)dX;
  cudaError_t e = cudaSuccess;
  for (int v0 = 0; v0 < V && e == cudaSuccess; v0 += o.cols) {
    const int n = std::min(o.cols, V - v0);
    const int64_t ld = (int64_t)up(n, 64);
    const uint16_t* Wp = W + (int64_t)v0 * ldw;
    GradEpi::Args a{};
    if (!product_map(&a.dz, dz, T, n, ld, ld, 1, 32, false)) return kLaunchFailed;
    a.labels = labels;
    a.lse = lse;
    a.g = g;
    a.V = V;
    a.v0 = v0;
    a.scale = scale;
    a.smooth = smooth;
    a.zc = zc;
    a.X = X;
    a.xs = dW && v0 == 0 ? xs : nullptr;
    a.W = Wp;
    a.ldx = ldx;
    a.ldw = ldw;
    a.T = T;
    a.h = h;
    e = product<false, false, GradEpi>(X, ldx, Wp, ldw, T, n, h, a, st);
    if (e == cudaSuccess && dX) {
      const bool last = v0 + n == V;
      e = gradient<false, true>(dz, ld, Wp, ldw, T, h, n, o.dx_ranges, part, last ? dX : acc, last && dx_bf16,
                                v0 ? acc : nullptr, false, scale, st);
    }
    if (e == cudaSuccess && dW) {
      void* out = dw_bf16 ? (void*)((uint16_t*)dW + (int64_t)v0 * h) : (void*)((float*)dW + (int64_t)v0 * h);
      e = gradient<true, true>(dz, ld, xs, h, n, h, T, o.dw_ranges, part, out, dw_bf16, accumulate ? out : nullptr,
                               dw_bf16, scale, st);
    }
  }
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

bool linear_ce_aligned(const void* X, const void* W, const void* dX, const void* dW, const void* work) {
  return al(X, 16) && al(W, 16) && al(dX, 16) && al(dW, 16) && al(work, 256);
}

}  // namespace mt
