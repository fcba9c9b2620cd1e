// Embedding lookup with a scale, and the table's gradient by sorted tokens.
//
// Forward: out[t] = scale * table[id_t] (0 for a negative id: padding).
// Backward: dtable[v] = scale * sum of dout[t] over the positions t with
// id_t = v, in 32 bits and in a fixed order, so it is bitwise reproducible:
//  1. one cluster of eight blocks sorts the positions by id (stable radix
//     sort, so equal ids keep ascending positions) and writes, for every
//     vocabulary row, its range of sorted positions; ranges longer than 64
//     are cut into pieces;
//  2. the pieces are summed, each in position order;
//  3. every row of the table gets its sum (short ranges straight from dout,
//     long ones from their pieces in order) or zeros.
// The pieces keep a frequent id (or a constant batch) from leaving one block
// with all the work. HBM traffic bounds the whole: dout read once, the table's
// gradient written once.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mt {

MT_DEVICE_ERROR_READER(embedding_take_device_error)

namespace {

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// Four neighbouring values as fp32.
template <bool BF16>
__device__ __forceinline__ float4 load4(const void* p, size_t i) {
  if (BF16) {
    const uint2 u = *(const uint2*)((const uint16_t*)p + i);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
  return *(const float4*)((const float*)p + i);
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, size_t i, const float4& v) {
  if (BF16) *(uint2*)((uint16_t*)p + i) = make_uint2(pack_bf2(v.x, v.y), pack_bf2(v.z, v.w));
  else *(float4*)((float*)p + i) = v;
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, size_t i) {
  return BF16 ? bf2f(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, size_t i, float v) {
  if (BF16) ((uint16_t*)p)[i] = f2bf(v);
  else ((float*)p)[i] = v;
}
// N (4 or 1) values at column c.
template <bool BF16, int N>
__device__ __forceinline__ float4 loadn(const void* p, size_t i) {
  return N == 4 ? load4<BF16>(p, i) : make_float4(load1<BF16>(p, i), 0.f, 0.f, 0.f);
}
template <bool BF16, int N>
__device__ __forceinline__ void storen(void* p, size_t i, const float4& v) {
  if (N == 4) store4<BF16>(p, i, v);
  else store1<BF16>(p, i, v.x);
}
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 scaled(const float4& a, float s) {
  return make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
}

// A thread takes N columns of four rows; blockDim.y rows side by side.
constexpr int kFwdRows = 4;

template <bool TB, bool OB, int N>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* __restrict__ table,
                                                        const int32_t* __restrict__ ids, float scale,
                                                        void* __restrict__ out, int T, int V, int h) {
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * N;
  if (c >= h) return;
  const int step = gridDim.y * blockDim.y;
  for (int t0 = blockIdx.y * blockDim.y + threadIdx.y; t0 < T; t0 += step * kFwdRows) {
    int id[kFwdRows];
    float4 v[kFwdRows];
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) id[r] = t0 + r * step < T ? ids[t0 + r * step] : -1;
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      if (id[r] >= V) {
        report_error(kErrBadArg);
        id[r] = -1;
      }
      v[r] = id[r] >= 0 ? loadn<TB, N>(table, (size_t)id[r] * h + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      const int t = t0 + r * step;
      if (t < T) storen<OB, N>(out, (size_t)t * h + c, scaled(v[r], scale));
    }
  }
}

// ---------------------------------------------------------------------------
// Sort: one cluster of kSortCtas blocks of 32 warps. Every warp owns a
// contiguous part of the positions; a pass counts its digits per warp (equal
// digits of 32 neighbouring keys are found with match.any), turns the counts
// into offsets (digit, then block, then warp: a stable order) with one scan
// over the cluster, and walks its part again to place its keys.
// ---------------------------------------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 10;  // bits: 32 warps x 1024 counters in shared memory
constexpr int kShort = 64;     // longest range summed in one go

struct SortArgs {
  const int32_t* ids;
  int2 *a, *b;      // (key, position), ping-pong
  int2* range;      // [V]: sorted positions [x, y) of an id
  int32_t* piece0;  // [V]: first piece of a long range
  int4* pieces;     // (first, last) sorted position of a piece
  int32_t* n_pieces;
  int T, V, passes, digit;
};

// Positions a piece of a range of n covers: about the square root of n, so
// that summing a piece and adding up the pieces take equally long.
__host__ __device__ inline int piece_len(int n) {
  int l = kShort;
  while ((long long)l * l < n) l *= 2;
  return l;
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t cnt[];  // [kSortWarps][bins], then the block's totals [bins]
  __shared__ uint32_t scan[kSortWarps];
  const int bins = 1 << a.digit;
  uint32_t* tot = cnt + kSortWarps * bins;
  const uint32_t rank = cluster_rank(), warp = warp_id(), lane = lane_id();
  const int tid = threadIdx.x;
  uint32_t* mine = cnt + warp * bins;

  // empty ranges, while the first pass runs
  for (int v = (int)rank * kSortThreads + tid; v < a.V; v += kSortCtas * kSortThreads) a.range[v] = make_int2(0, 0);
  if (rank == 0 && tid == 0) *a.n_pieces = 0;

  // the warp's part: whole groups of 32 positions
  const int groups = (a.T + 31) / 32, all = kSortCtas * kSortWarps;
  const int wid = (int)rank * kSortWarps + (int)warp;
  const int lo = (int)((int64_t)groups * wid / all) * 32;
  const int hi = min(a.T, (int)((int64_t)groups * (wid + 1) / all) * 32);

  for (int p = 0; p < a.passes; ++p) {
    const int2* src = p == 0 ? nullptr : (p & 1) ? a.a : a.b;
    int2* dst = (p & 1) ? a.b : a.a;
    const int shift = p * a.digit;
    auto key_at = [&](int i) {
      if (src) return __ldcg(src + i);
      const int id = a.ids[i];
      if (id >= a.V) report_error(kErrBadArg);
      return make_int2(id < 0 || id >= a.V ? a.V : id, i);  // ids outside the table sort last
    };
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      const uint32_t d = on ? ((uint32_t)key_at(i + (int)lane).x >> shift) & (bins - 1) : 0xffffffffu;
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (on && (peers & ((1u << lane) - 1)) == 0) mine[d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    uint32_t own = 0;
    if (tid < bins) {
      for (int w = 0; w < kSortWarps; ++w) own += cnt[w * bins + tid];
      tot[tid] = own;
    }
    cluster_sync();
    uint32_t before = 0, total = 0;
    if (tid < bins) {
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        uint32_t x;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(tot + tid, r)) : "memory");
        if (r < rank) before += x;
        total += x;
      }
    }
    // exclusive sum of the digits' totals over the block
    uint32_t s = total;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
      if ((int)lane >= o) s += x;
    }
    if (lane == 31) scan[warp] = s;
    __syncthreads();
    if (warp == 0) {
      uint32_t x = scan[lane];
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)lane >= o) x += y;
      }
      scan[lane] = x;
    }
    __syncthreads();
    if (tid < bins) {
      uint32_t at = s - total + (warp ? scan[warp - 1] : 0u) + before;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t x = cnt[w * bins + tid];
        cnt[w * bins + tid] = at;
        at += x;
      }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      const int2 kv = on ? key_at(i + (int)lane) : make_int2(0, 0);
      const uint32_t d = on ? ((uint32_t)kv.x >> shift) & (bins - 1) : 0xffffffffu;
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const uint32_t below = __popc(peers & ((1u << lane) - 1));
      uint32_t at = 0;
      if (on) at = mine[d] + below;
      __syncwarp();
      if (on) {
        if (below == 0) mine[d] += __popc(peers);
        __stcg(dst + at, kv);
      }
      __syncwarp();
    }
    cluster_sync();  // the sorted keys (and, after the first pass, the empty ranges) are visible to the cluster
  }

  // ranges of equal ids
  const int2* s = (a.passes & 1) ? a.a : a.b;
  for (int i = (int)rank * kSortThreads + tid; i < a.T; i += kSortCtas * kSortThreads) {
    const int k = __ldcg(s + i).x;
    if (k >= a.V) continue;
    if (i == 0 || __ldcg(s + i - 1).x != k) __stcg(&a.range[k].x, i);
    if (i == a.T - 1 || __ldcg(s + i + 1).x != k) __stcg(&a.range[k].y, i + 1);
  }
  cluster_sync();
  // pieces of the long ones
  for (int i = (int)rank * kSortThreads + tid; i < a.T; i += kSortCtas * kSortThreads) {
    const int k = __ldcg(s + i).x;
    if (k >= a.V || (i > 0 && __ldcg(s + i - 1).x == k)) continue;
    const int end = __ldcg(&a.range[k].y), n = end - i;
    if (n <= kShort) continue;
    const int l = piece_len(n), np = (n + l - 1) / l;
    const int p0 = atomicAdd(a.n_pieces, np);  // where a range's pieces lie does not enter their sums
    a.piece0[k] = p0;
    for (int q = 0; q < np; ++q) a.pieces[p0 + q] = make_int4(i + q * l, min(end, i + (q + 1) * l), 0, 0);
  }
}

// Sum of dout over the sorted positions [i0, i1), N columns from c: eight
// rows' loads in flight, added in position order.
template <bool DB, int N>
__device__ __forceinline__ float4 sum_rows(const int2* s, int i0, int i1, const void* dout, int h, int c) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  int i = i0;
  for (; i + 8 <= i1; i += 8) {
    float4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = loadn<DB, N>(dout, (size_t)s[i + q].y * h + c);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc = add4(acc, v[q]);
  }
  for (; i < i1; ++i) acc = add4(acc, loadn<DB, N>(dout, (size_t)s[i].y * h + c));
  return acc;
}

template <bool DB, int N>
__global__ void __launch_bounds__(256) embed_pieces_kernel(const int2* __restrict__ s, const int4* __restrict__ pieces,
                                                           const int32_t* __restrict__ n_pieces,
                                                           const void* __restrict__ dout, float* __restrict__ part,
                                                           int h) {
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  if (c >= h) return;
  const int n = *n_pieces;
  for (int p = blockIdx.x; p < n; p += gridDim.x) {
    const int4 d = pieces[p];
    storen<false, N>(part, (size_t)p * h + c, sum_rows<DB, N>(s, d.x, d.y, dout, h, c));
  }
}

constexpr int kTableRows = 8;  // vocabulary rows of a block

template <bool DB, bool EB, int N>
__global__ void __launch_bounds__(256) embed_table_kernel(const int2* __restrict__ s, const int2* __restrict__ range,
                                                          const int32_t* __restrict__ piece0,
                                                          const float* __restrict__ part,
                                                          const void* __restrict__ dout, float scale, void* dtable,
                                                          int V, int h, int add) {
  __shared__ int2 sr[kTableRows];
  const int v0 = blockIdx.x * kTableRows, rows = min(kTableRows, V - v0);
  if ((int)threadIdx.x < rows) sr[threadIdx.x] = range[v0 + threadIdx.x];
  __syncthreads();
  for (int r = 0; r < rows; ++r) {
    const int2 d = sr[r];
    const int n = d.y - d.x;
    if (n == 0 && add) continue;
    const size_t at = (size_t)(v0 + r) * h;
    const int l = piece_len(n), np = (n + l - 1) / l;
    const int p0 = n > kShort ? piece0[v0 + r] : 0;
    for (int c = threadIdx.x * N; c < h; c += blockDim.x * N) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n > kShort) {
#pragma unroll 8
        for (int p = 0; p < np; ++p) acc = add4(acc, loadn<false, N>(part, (size_t)(p0 + p) * h + c));
      } else if (n > 0) {
        acc = sum_rows<DB, N>(s, d.x, d.y, dout, h, c);
      }
      acc = scaled(acc, scale);
      if (add) acc = add4(loadn<EB, N>(dtable, at + c), acc);
      storen<EB, N>(dtable, at + c, acc);
    }
  }
}

struct EmbedWs {
  size_t a, b, range, piece0, pieces, n_pieces, part, total;
};
EmbedWs embed_ws(int T, int V, int h) {
  EmbedWs o;
  size_t x = 0;
  auto take = [&](size_t bytes) {
    const size_t r = x;
    x += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t max_pieces = (size_t)T / 32 + 1;  // ranges over 64, pieces of 64 or more
  o.a = take((size_t)T * 8);
  o.b = take((size_t)T * 8);
  o.range = take((size_t)V * 8);
  o.piece0 = take((size_t)V * 4);
  o.pieces = take(max_pieces * 16);
  o.n_pieces = take(4);
  o.part = take(max_pieces * (size_t)h * 4);
  o.total = x;
  return o;
}

bool embed_dims_ok(int T, int V, int h) {
  return T > 0 && V > 0 && h > 0 && T <= (1 << 28) && V < (1 << 30) && h <= (1 << 24);
}
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

int embed_fwd(const void* table, bool tb, const int32_t* ids, float scale, void* out, bool ob, int T, int V, int h,
              cudaStream_t st) {
  if (!embed_dims_ok(T, V, h) || !al(table, tb ? 2 : 4) || !al(out, ob ? 2 : 4)) return -1;
  const bool vec = h % 4 == 0 && al(table, tb ? 8 : 16) && al(out, ob ? 8 : 16);
  const int units = vec ? h / 4 : h;
  int bx = 32;
  while (bx < units && bx < 256) bx *= 2;
  const int by = 256 / bx;
  const dim3 block((unsigned)bx, (unsigned)by);
  const dim3 grid((unsigned)((units + bx - 1) / bx), (unsigned)std::min((T + by * kFwdRows - 1) / (by * kFwdRows), 65535));
  auto go = [&](auto k) { k<<<grid, block, 0, st>>>(table, ids, scale, out, T, V, h); };
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (tb) ob ? go(embed_fwd_kernel<true, true, N>) : go(embed_fwd_kernel<true, false, N>);
    else ob ? go(embed_fwd_kernel<false, true, N>) : go(embed_fwd_kernel<false, false, N>);
  };
  if (vec) pick(std::integral_constant<int, 4>());
  else pick(std::integral_constant<int, 1>());
  count_launches(1);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

size_t embed_bwd_workspace(int T, int V, int h) { return embed_dims_ok(T, V, h) ? embed_ws(T, V, h).total : 0; }

int embed_bwd(const int32_t* ids, const void* dout, bool db, float scale, void* dtable, bool eb, bool add, void* work,
              int T, int V, int h, cudaStream_t st) {
  if (!embed_dims_ok(T, V, h) || !al(work, 256) || !al(dout, db ? 2 : 4) || !al(dtable, eb ? 2 : 4)) return -1;
  const EmbedWs o = embed_ws(T, V, h);
  uint8_t* w = (uint8_t*)work;
  SortArgs a;
  a.ids = ids;
  a.a = (int2*)(w + o.a);
  a.b = (int2*)(w + o.b);
  a.range = (int2*)(w + o.range);
  a.piece0 = (int32_t*)(w + o.piece0);
  a.pieces = (int4*)(w + o.pieces);
  a.n_pieces = (int32_t*)(w + o.n_pieces);
  a.T = T;
  a.V = V;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // keys 0..V
  a.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  a.digit = (bits + a.passes - 1) / a.passes;
  const int smem = ((kSortWarps + 1) << a.digit) * 4;
  if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ((kSortWarps + 1) << kMaxDigit) * 4) != cudaSuccess)
    return -1;
  embed_sort_kernel<<<kSortCtas, kSortThreads, smem, st>>>(a);
  const int2* s = (a.passes & 1) ? a.a : a.b;
  float* part = (float*)(w + o.part);
  const bool vec = h % 4 == 0 && al(dout, db ? 8 : 16) && al(dtable, eb ? 8 : 16);
  const int units = vec ? h / 4 : h;
  const int cols = (units + 255) / 256;
  const bool long_ranges = T > kShort;
  auto pieces = [&](auto k) {
    k<<<dim3((unsigned)std::min(T / 32 + 1, 2048), (unsigned)cols), 256, 0, st>>>(s, a.pieces, a.n_pieces, dout, part,
                                                                                 h);
  };
  auto table = [&](auto k) {
    k<<<(V + kTableRows - 1) / kTableRows, 256, 0, st>>>(s, a.range, a.piece0, part, dout, scale, dtable, V, h,
                                                        add ? 1 : 0);
  };
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (long_ranges) db ? pieces(embed_pieces_kernel<true, N>) : pieces(embed_pieces_kernel<false, N>);
    if (db) eb ? table(embed_table_kernel<true, true, N>) : table(embed_table_kernel<true, false, N>);
    else eb ? table(embed_table_kernel<false, true, N>) : table(embed_table_kernel<false, false, N>);
  };
  if (vec) pick(std::integral_constant<int, 4>());
  else pick(std::integral_constant<int, 1>());
  count_launches(long_ranges ? 3 : 2);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mt
