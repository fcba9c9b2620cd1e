// Embedding lookup with a scale, and the table's gradient by sorted tokens.
//
// Forward: out[t] = scale * table[id_t] (0 for a negative id: padding).
// Backward: dtable[v] = scale * sum of dout[t] over the positions t with
// id_t = v, in 32 bits and in a fixed order, so it is bitwise reproducible:
//  1. one cluster of eight blocks sorts the positions by id (stable radix
//     sort, so equal ids keep ascending positions) and lists the runs of
//     equal ids, those longer than 8 in pieces; meanwhile the other blocks of
//     the same launch clear the table's gradient;
//  2. blocks take the pieces in turn, then warps the short runs, and add
//     their rows in position order; the block that finishes a run's last
//     piece adds the pieces in order.
// The pieces keep a frequent id (or a constant batch) from leaving one block
// with all the work. HBM traffic bounds the whole: dout read once, the table's
// gradient written once (used rows twice). The sort (12 us for small batches)
// hides behind the clearing of all but small tables.
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
// N partial sums that another block wrote during this launch.
template <int N>
__device__ __forceinline__ float4 load_part(const float* p, size_t i) {
  return N == 4 ? __ldcg((const float4*)(p + i)) : make_float4(__ldcg(p + i), 0.f, 0.f, 0.f);
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
// over the cluster, and walks its part again to place its keys. The last step
// counts and lists the heads of runs the same way.
// ---------------------------------------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 10;  // bits: 32 warps x 1024 counters in shared memory
constexpr int kShort = 8;      // longest run summed by one warp
constexpr int kPiece = 32;     // least length of a longer run's pieces
constexpr int kClearBytes = 128 * 1024;  // cleared by one block

struct SortArgs {
  const int32_t* ids;
  int2 *a, *b;       // (key, position), ping-pong
  int32_t* head;     // first sorted position of each run, then the end
  int4* runs;        // of each run: sorted positions [x, y), id z, w: first position (short) or first partial sum
  int4* pieces;      // sorted positions [x, y), run z, partial sum w (-1: the piece is the run)
  int32_t* left;     // per run and column chunk: pieces not yet summed
  int32_t* n;        // [0] pieces, [1] partial sums, [2] runs
  void* clear;       // table gradient to clear (null: none)
  size_t clear_bytes;
  int T, V, passes, digit, chunks;
};

// Positions a piece of a run of n covers: about the square root of n, so that
// summing a piece and adding up the pieces take equally long.
__host__ __device__ inline int piece_len(int n) {
  int l = kPiece;
  while ((long long)l * l < n) l *= 2;
  return l;
}

// One block's share of clearing: 16-byte stores, 2-byte ones at the ends.
__device__ __forceinline__ void clear_share(void* base, size_t bytes, int block) {
  uint8_t* p = (uint8_t*)base;
  const size_t head = min((size_t)((16 - ((uintptr_t)p & 15)) & 15), bytes);
  const size_t vecs = (bytes - head) / 16;
  constexpr size_t per = kClearBytes / 16;
  const size_t lo = (size_t)block * per, hi = min(lo + per, vecs);
  uint4* v = (uint4*)(p + head);
  const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 8
  for (size_t i = lo + threadIdx.x; i < hi; i += kSortThreads) v[i] = z;
  if (block == 0) {
    uint16_t* e = (uint16_t*)p;
    const size_t tail = head + vecs * 16;
    if (threadIdx.x < head / 2) e[threadIdx.x] = 0;
    if (threadIdx.x < (bytes - tail) / 2) e[tail / 2 + threadIdx.x] = 0;
  }
}

// Exclusive sum of x over the block's threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* scratch) {
  const uint32_t lane = lane_id(), warp = warp_id();
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if ((int)lane >= o) s += y;
  }
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  if (warp == 0) {
    uint32_t v = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
      if ((int)lane >= o) v += y;
    }
    scratch[lane] = v;
  }
  __syncthreads();
  return s - x + (warp ? scratch[warp - 1] : 0u);
}
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, uint32_t rank) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(mapa_shared(p, rank)) : "memory");
  return x;
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t cnt[];  // [kSortWarps][bins], then the block's totals [bins]
  __shared__ uint32_t scratch[kSortWarps];
  __shared__ uint32_t heads[kSortWarps + 1];  // run heads of each warp's part, of the block
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sums wait for this launch's end themselves
  if (blockIdx.x >= kSortCtas) {
    clear_share(a.clear, a.clear_bytes, (int)blockIdx.x - kSortCtas);
    return;
  }
  const int bins = 1 << a.digit;
  uint32_t* tot = cnt + kSortWarps * bins;
  const uint32_t rank = cluster_rank(), warp = warp_id(), lane = lane_id(), below_mask = (1u << lane) - 1;
  const int tid = threadIdx.x;
  uint32_t* mine = cnt + warp * bins;
  if (rank == 0 && tid == 0) a.n[0] = a.n[1] = 0;

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
      if (i >= hi) return make_int2(0, 0);
      if (src) return __ldcg(src + i);
      const int id = a.ids[i];
      if (id >= a.V) report_error(kErrBadArg);
      return make_int2(id < 0 || id >= a.V ? a.V : id, i);  // ids outside the table sort last
    };
    int2 next = key_at(lo + (int)lane);
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      const uint32_t d = on ? ((uint32_t)next.x >> shift) & (bins - 1) : 0xffffffffu;
      next = key_at(i + 32 + (int)lane);
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (on && (peers & below_mask) == 0) mine[d] += __popc(peers);
      __syncwarp();
    }
    next = key_at(lo + (int)lane);
    __syncthreads();
    uint32_t own = 0;
    if (tid < bins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) own += cnt[w * bins + tid];
      tot[tid] = own;
    }
    cluster_sync();
    uint32_t before = 0, total = 0;
    if (tid < bins) {
#pragma unroll
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        const uint32_t x = peer_word(tot + tid, r);
        if (r < rank) before += x;
        total += x;
      }
    }
    const uint32_t base = block_scan(total, scratch);
    if (tid < bins) {
      uint32_t at = base + before;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t x = cnt[w * bins + tid];
        cnt[w * bins + tid] = at;
        at += x;
      }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      const int2 kv = next;
      const uint32_t d = on ? ((uint32_t)kv.x >> shift) & (bins - 1) : 0xffffffffu;
      next = key_at(i + 32 + (int)lane);
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const uint32_t below = __popc(peers & below_mask);
      uint32_t at = 0;
      if (on) at = mine[d] + below;
      __syncwarp();
      if (on) {
        if (below == 0) mine[d] += __popc(peers);
        __stcg(dst + at, kv);
      }
      __syncwarp();
    }
    cluster_sync();  // the sorted keys are visible to the cluster
  }

  // heads of runs of equal ids: counted, then listed in order
  const int2* s = (a.passes & 1) ? a.a : a.b;
  auto is_head = [&](int i) { return i < hi && (i == 0 || __ldcg(s + i).x != __ldcg(s + i - 1).x); };
  uint32_t h = 0;
  for (int i = lo; i < hi; i += 32) h += __popc(__ballot_sync(0xffffffffu, is_head(i + (int)lane)));
  if (lane == 0) heads[warp] = h;
  __syncthreads();
  if (tid == 0) {
    uint32_t sum = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t x = heads[w];
      heads[w] = sum;
      sum += x;
    }
    heads[kSortWarps] = sum;
  }
  cluster_sync();
  uint32_t at = heads[warp], runs = 0;
  for (uint32_t r = 0; r < kSortCtas; ++r) {
    const uint32_t x = peer_word(&heads[kSortWarps], r);
    if (r < rank) at += x;
    runs += x;
  }
  for (int i = lo; i < hi; i += 32) {
    const bool here = is_head(i + (int)lane);
    const uint32_t m = __ballot_sync(0xffffffffu, here);
    if (here) __stcg(a.head + at + __popc(m & below_mask), i + (int)lane);
    at += __popc(m);
  }
  if (rank == 0 && tid == 0) {
    __stcg(a.head + runs, a.T);
    a.n[2] = (int)runs;
  }
  cluster_sync();
  for (int r = (int)rank * kSortThreads + tid; r < (int)runs; r += kSortCtas * kSortThreads) {
    const int x = __ldcg(a.head + r), id = __ldcg(s + x).x;
    const int y = id < a.V ? __ldcg(a.head + r + 1) : x, n = y - x;  // ids outside the table: an empty run
    int w = 0;
    if (n > kShort) {
      const int l = piece_len(n), np = (n + l - 1) / l, p0 = atomicAdd(a.n, np);
      // where a run's pieces and partial sums lie does not enter their values
      w = np > 1 ? atomicAdd(a.n + 1, np) : -1;
      for (int q = 0; q < np; ++q)
        a.pieces[p0 + q] = make_int4(x + q * l, min(y, x + (q + 1) * l), r, np > 1 ? w + q : -1);
      if (np > 1)
        for (int c = 0; c < a.chunks; ++c) a.left[(size_t)r * a.chunks + c] = np;
    } else if (n > 0) {
      w = __ldcg(s + x).y;
    }
    a.runs[r] = make_int4(x, y, id, w);
  }
}

// ---------------------------------------------------------------------------
// Sums, 256 N columns at a time. A block adds a piece with a column group of
// N a thread and eight rows in flight. A warp adds a short run with eight
// column groups a thread, the next row requested under the sum of the last:
// most runs have one or two rows, and only many bytes in flight a warp hide
// the way from the run's entry to its rows and the table (one block a run,
// one group a thread: 166 against 106 us for 8192 tokens of 128256 x 4096,
// added to the table).
// ---------------------------------------------------------------------------
template <bool DB, int N>
__device__ __forceinline__ float4 sum_rows(const int2* s, int i0, int i1, const void* dout, int h, int c) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = i0; i < i1; i += 8) {
    float4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q < i1) v[q] = loadn<DB, N>(dout, (size_t)s[i + q].y * h + c);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (i + q < i1) acc = add4(acc, v[q]);
  }
  return acc;
}

template <bool DB, bool EB, int N>
__global__ void __launch_bounds__(256, 2) embed_sum_kernel(const int2* s, const int4* runs, const int4* pieces,
                                                           int32_t* left, const int32_t* n, float* part,
                                                           const void* __restrict__ dout, float scale, void* dtable,
                                                           int h, int add) {
  __shared__ int last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int chunk = blockIdx.y, n_pieces = n[0], n_runs = n[2];
  const int c = (chunk * 256 + (int)threadIdx.x) * N;
  auto finish = [&](int id, float4 acc) {
    acc = scaled(acc, scale);
    const size_t at = (size_t)id * h + c;
    if (add) acc = add4(loadn<EB, N>(dtable, at), acc);
    storen<EB, N>(dtable, at, acc);
  };
  for (int i = blockIdx.x; i < n_pieces; i += gridDim.x) {
    const int4 d = pieces[i];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < h) acc = sum_rows<DB, N>(s, d.x, d.y, dout, h, c);
    if (d.w < 0) {
      if (c < h) finish(runs[d.z].z, acc);
      continue;
    }
    if (c < h) storen<false, N>(part, (size_t)d.w * h + c, acc);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicSub(&left[(size_t)d.z * gridDim.y + chunk], 1) == 1;
    __syncthreads();
    if (last && c < h) {  // every piece of the run is there: add them in order
      __threadfence();
      const int4 r = runs[d.z];
      const int l = piece_len(r.y - r.x), k = (r.y - r.x + l - 1) / l;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < k; q += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (q + j < k) v[j] = load_part<N>(part, (size_t)(r.w + q + j) * h + c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (q + j < k) acc = add4(acc, v[j]);
      }
      finish(r.z, acc);
    }
    __syncthreads();  // `last` is read before the next piece sets it
  }

  // short runs
  const int lane = (int)lane_id(), step = gridDim.x * 8;
  const int c0 = chunk * 256 * N + lane * N;  // column groups c0 + 32 N k
  auto row = [&](int pos, float4 (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c0 + 32 * N * k < h) v[k] = loadn<DB, N>(dout, (size_t)pos * h + c0 + 32 * N * k);
  };
  auto entry = [&](int i) { return i < n_runs ? runs[i] : make_int4(0, 0, 0, 0); };
  int i = blockIdx.x * 8 + (int)warp_id();
  int4 next = entry(i);
  for (; i < n_runs; i += step) {
    const int4 d = next;
    next = entry(i + step);
    const int rows = d.y - d.x;
    if (rows == 0 || rows > kShort) continue;
    float4 acc[8], v[8];
    row(d.w, acc);
    const int pos = lane < rows ? s[d.x + lane].y : 0;
    if (rows > 1) row(__shfl_sync(0xffffffffu, pos, 1), v);
    for (int q = 1; q < rows; ++q) {
      const int p = __shfl_sync(0xffffffffu, pos, q + 1 < rows ? q + 1 : 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = add4(acc[k], v[k]);
      if (q + 1 < rows) row(p, v);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int cc = c0 + 32 * N * k;
      if (cc < h) {
        const size_t at = (size_t)d.z * h + cc;
        acc[k] = scaled(acc[k], scale);
        if (add) acc[k] = add4(loadn<EB, N>(dtable, at), acc[k]);
        storen<EB, N>(dtable, at, acc[k]);
      }
    }
  }
}

struct EmbedWs {
  size_t a, b, head, runs, pieces, left, n, part, total;
};
EmbedWs embed_ws(int T, int V, int h) {
  EmbedWs o;
  size_t x = 0;
  auto take = [&](size_t bytes) {
    const size_t r = x;
    x += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t max_pieces = (size_t)T / 8 + 1;  // runs over 8: one piece, or pieces of 32 or more
  const size_t max_parts = (size_t)T / 16 + 1;  // runs over 32
  const size_t max_runs = std::min((size_t)T, (size_t)V + 1);
  o.a = take((size_t)T * 8);
  o.b = take((size_t)T * 8);
  o.head = take((max_runs + 1) * 4);
  o.runs = take(max_runs * 16);
  o.pieces = take(max_pieces * 16);
  o.left = take(max_runs * (size_t)((h + 255) / 256) * 4);
  o.n = take(12);
  o.part = take(max_parts * (size_t)h * 4);
  o.total = x;
  return o;
}

bool embed_dims_ok(int T, int V, int h) {
  return T > 0 && V > 0 && h > 0 && T <= (1 << 28) && V < (1 << 30) && h <= (1 << 22);
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
  const bool vec = h % 4 == 0 && al(dout, db ? 8 : 16) && al(dtable, eb ? 8 : 16);
  const int units = vec ? h / 4 : h;
  SortArgs a;
  a.ids = ids;
  a.a = (int2*)(w + o.a);
  a.b = (int2*)(w + o.b);
  a.head = (int32_t*)(w + o.head);
  a.runs = (int4*)(w + o.runs);
  a.pieces = (int4*)(w + o.pieces);
  a.left = (int32_t*)(w + o.left);
  a.n = (int32_t*)(w + o.n);
  a.clear = add ? nullptr : dtable;
  a.clear_bytes = add ? 0 : (size_t)V * h * (eb ? 2 : 4);
  a.T = T;
  a.V = V;
  a.chunks = (units + 255) / 256;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // keys 0..V
  a.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  a.digit = (bits + a.passes - 1) / a.passes;
  const int smem = ((kSortWarps + 1) << a.digit) * 4;
  if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ((kSortWarps + 1) << kMaxDigit) * 4) != cudaSuccess)
    return -1;
  size_t clearers = (a.clear_bytes + kClearBytes - 1) / kClearBytes;
  clearers = (clearers + kSortCtas - 1) / kSortCtas * kSortCtas;
  if (clearers > (1u << 30)) return -1;
  embed_sort_kernel<<<(unsigned)(kSortCtas + clearers), kSortThreads, smem, st>>>(a);

  // as many blocks as run at once, launched while the last ones of the sort end
  const int most = std::max(T / 8 + 1, (std::min(T, V) + 7) / 8), fit = std::max(1, 152 * 2 / a.chunks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(most, fit), (unsigned)a.chunks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) {
    e = cudaLaunchKernelEx(&cfg, k, (const int2*)((a.passes & 1) ? a.a : a.b), (const int4*)a.runs,
                           (const int4*)a.pieces, a.left, (const int32_t*)a.n, (float*)(w + o.part), dout, scale,
                           dtable, h, add ? 1 : 0);
  };
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (db) eb ? go(embed_sum_kernel<true, true, N>) : go(embed_sum_kernel<true, false, N>);
    else eb ? go(embed_sum_kernel<false, true, N>) : go(embed_sum_kernel<false, false, N>);
  };
  if (vec) pick(std::integral_constant<int, 4>());
  else pick(std::integral_constant<int, 1>());
  count_launches(2);
  return e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mt
