// Embedding lookup with a scale, and the table's gradient by sorted tokens.
//
// Forward: out[t] = scale * table[id_t] (0 for a negative id: padding).
// Backward: dtable[v] = scale * sum of dout[t] over the positions t with
// id_t = v, in 32 bits and in a fixed order, so it is bitwise reproducible:
//  1. one cluster of eight blocks sorts the positions by id (stable radix
//     sort, so equal ids keep ascending positions) and marks the used rows;
//     meanwhile other blocks of the launch clear the first rows of the table;
//  2. warps stream over ranges of the sorted positions with the next rows
//     always in flight, add runs of equal ids and write their rows; a run
//     longer than 32 leaves a partial sum per range. Other warps clear the
//     unused rows that are left;
//  3. the partial sums of the long runs are added in order.
// Cutting long runs at fixed positions keeps a frequent id (or a constant
// batch) from leaving one warp with all the work. HBM traffic bounds the
// whole: dout read once, the table's gradient written once; the sort (some 10
// us for small batches) hides behind the first clearing. Measured: 8192 tokens
// of 128256 x 4096 fp32 (floor 329 us) 316-322 us, 16384 of 151936 x 4096 bf16
// (223) 226, 64 of 32000 x 1024 fp32 (19.3) 24; where nothing hides the sort,
// 8192 of 1000 x 4096 (22) 46 us, 131072 of 32000 x 1024 (98) 198. Rows of bf16:
// 8192 of 128256 x 4096 fp32 (319) 320, 16384 of 151936 x 4096 bf16 (203) 220.
// Added to the table: 8192 of 128256 x 4096 fp32 (39) 62, 16384 of 151936 x 4096
// bf16 (57) 107. Lookup from bf16, 8192 rows of 4096: 33 us to fp32 (30), 25 to
// bf16 (20).
#include <algorithm>
#include <cmath>
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

// p[i..] += v, one writer a value. fp32: a reduction in memory, which the
// thread does not wait for (reading the old row first stalled the stream of
// rows: 179 against 92 us for 8192 tokens of 128256 x 4096). bf16: added in
// fp32 and rounded once.
template <bool BF16, int N>
__device__ __forceinline__ void accumulate(void* p, size_t i, const float4& v) {
  if (BF16) {
    storen<true, N>(p, i, add4(loadn<true, N>(p, i), v));
  } else if (N == 4) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"((float*)p + i), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
  } else {
    atomicAdd((float*)p + i, v.x);
  }
}

// A thread takes N columns of four rows; blockDim.y rows side by side.
constexpr int kFwdRows = 4;

template <bool TB, bool OB, int N>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* table,
                                                        const int32_t* ids, float scale,
                                                        void* __restrict__ out, int T, int V, int h) {
  grid_wait();
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
      // (padding is 0 whatever the scale: an infinite one would make it NaN)
      if (t < T) storen<OB, N>(out, (size_t)t * h + c, scaled(v[r], id[r] >= 0 ? scale : 0.f));
    }
  }
}

// ---------------------------------------------------------------------------
// Sort: one cluster of eight blocks of 32 warps, or one block for few
// positions, where the barriers between blocks cost more than the work (a
// gradient added to 32000 x 192: 300 positions 9.4 us by one block, 10.7 by the
// cluster; 4096 17.9 and 13.5). Every warp owns a
// contiguous part of the positions; a pass counts its digits per warp, turns
// the counts into offsets (digit, then block, then warp: a stable order) with
// one scan over the cluster, and walks its part again to place its keys (equal
// digits of 32 neighbouring keys are found with a ballot a bit: match.any took
// 78 us for 131072 positions, counting with it included).
// ---------------------------------------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortOne = 1024;  // positions that one block sorts alone
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 10;  // bits: 32 warps x 1024 counters in shared memory
constexpr int kClearBytes = 128 * 1024;     // cleared by one block of the sort's launch
constexpr size_t kClearFirst = 64u << 20;   // and by all of them: what takes as long as the sort

struct SortArgs {
  const int32_t* ids;
  int2 *a, *b;       // (key, position), ping-pong
  uint8_t* used;     // [V] rows with a position (null: not wanted)
  int32_t* ctl;      // counters of the later steps, zeroed here: [0] long runs, [1] clearing
  void* clear;       // the part of the table's gradient to clear here
  size_t clear_bytes;
  int T, V, passes, digit, ctas;
  int warps;  // of a block that take positions (and have counters)
};

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

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t cnt[];  // [warps][bins], then the block's totals [bins]
  __shared__ uint32_t scratch[kSortWarps];
  grid_release();  // the sums wait for this launch's end themselves
  grid_wait();
  const int ctas = a.ctas;
  if ((int)blockIdx.x >= ctas) {
    clear_share(a.clear, a.clear_bytes, (int)blockIdx.x - ctas);
    return;
  }
  const int bins = 1 << a.digit;
  const int W = a.warps;
  uint32_t* tot = cnt + W * bins;
  const uint32_t rank = ctas > 1 ? cluster_rank() : 0u, warp = warp_id(), lane = lane_id(), below_mask = (1u << lane) - 1;
  const int tid = threadIdx.x;
  uint32_t* mine = cnt + warp * bins;  // a warp past W has no positions
  if (rank == 0 && tid < 2) a.ctl[tid] = 0;
  auto sync_all = [&] {  // what the cluster's blocks have written is visible to all of them
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  };
  if (a.used) {  // [V] rounded up to whole 16-byte words
    uint4* u = (uint4*)a.used;
    for (int i = (int)rank * kSortThreads + tid; i < (a.V + 15) / 16; i += ctas * kSortThreads)
      u[i] = make_uint4(0, 0, 0, 0);
    sync_all();
  }

  // the warp's part: whole groups of 32 positions
  const int groups = (a.T + 31) / 32, all = ctas * W;
  const int wid = (int)rank * W + (int)warp;
  const int lo = (int)((int64_t)groups * wid / all) * 32;
  const int hi = (int)warp < W ? min(a.T, (int)((int64_t)groups * (wid + 1) / all) * 32) : lo;

  for (int p = 0; p < a.passes; ++p) {
    const int2* src = p == 0 ? nullptr : (p & 1) ? a.a : a.b;
    int2* dst = (p & 1) ? a.b : a.a;
    const int shift = p * a.digit;
    auto key_at = [&](int i) {
      if (i >= hi) return make_int2(0, 0);
      if (src) return __ldcg(src + i);
      const int id = a.ids[i];
      if (id >= a.V) report_error(kErrBadArg);
      const bool off = id < 0 || id >= a.V;  // ids outside the table sort last
      if (!off && a.used) a.used[id] = 1;
      return make_int2(off ? a.V : id, i);
    };
    int2 next = key_at(lo + (int)lane);
    for (int i = tid; i < W * bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      if (on) atomicAdd(&mine[((uint32_t)next.x >> shift) & (bins - 1)], 1u);
      next = key_at(i + 32 + (int)lane);
    }
    next = key_at(lo + (int)lane);
    __syncthreads();
    uint32_t own = 0;
    if (tid < bins) {
#pragma unroll 8
      for (int w = 0; w < W; ++w) own += cnt[w * bins + tid];
      tot[tid] = own;
    }
    uint32_t before = 0, total = own;
    if (ctas > 1) {
      cluster_sync();
      total = 0;
      if (tid < bins) {
#pragma unroll
        for (uint32_t r = 0; r < kSortCtas; ++r) {
          const uint32_t x = peer_word(tot + tid, r);
          if (r < rank) before += x;
          total += x;
        }
      }
    }
    const uint32_t base = block_scan(total, scratch);
    if (tid < bins) {
      uint32_t at = base + before;
#pragma unroll 8
      for (int w = 0; w < W; ++w) {
        const uint32_t x = cnt[w * bins + tid];
        cnt[w * bins + tid] = at;
        at += x;
      }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32) {
      const bool on = i + (int)lane < hi;
      const int2 kv = next;
      const uint32_t d = ((uint32_t)kv.x >> shift) & (bins - 1);
      next = key_at(i + 32 + (int)lane);
      uint32_t peers = __ballot_sync(0xffffffffu, on);  // lanes with the same digit
#pragma unroll
      for (int b = 0; b < kMaxDigit; ++b)
        if (b < a.digit) {
          const bool set = (d >> b) & 1;
          const uint32_t m = __ballot_sync(0xffffffffu, set);
          peers &= set ? m : ~m;
        }
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
    sync_all();
  }

}

// ---------------------------------------------------------------------------
// Sums. A warp takes a range of L sorted positions and 32 N G columns (G
// groups of N a lane). Each lane copies its part of the rows into shared
// memory D rows ahead of the sums (cp.async: nothing to wait for but its own
// copies), so a row's way from memory is hidden however short the runs are.
// Runs of at most kShort belong whole to the range of their first position; a
// longer one is cut at the ranges' borders, each piece going to a partial sum:
// slot 2 j + 1 in the range j where the run begins, slot 2 j in the later ones.
// Measured for 8192 tokens of 128256 x 4096, added to the table: a block a
// run 136 us, blocks for pieces and warps for short runs 92 us, rows ahead in
// registers 76 us (and their unrolled code 18 us for 1266 tokens of 884 x 192,
// most of it instruction fetches).
// ---------------------------------------------------------------------------
constexpr int kShort = 32;

struct SumArgs {
  const int2* s;
  const void* dout;
  void* dtable;
  float* part;
  int2* longs;         // (range of the run's first position, id)
  const uint8_t* used;
  int32_t* ctl;
  float scale;
  int T, V, h, L, chunks, add;
  int words;  // bf16 rows of single columns: dout starts on a word
  int clear_row0, clear_rows;  // rows from clear_row0 on are cleared, clear_rows at a time (0: none)
};

// Bytes a lane copies at once: its N columns, or the word that a column lies in.
constexpr int sum_part(int N, bool bf16) { return N == 1 ? 4 : bf16 ? 8 : 16; }
constexpr int sum_depth(int G, int N) { return N == 1 ? 16 : G == 1 ? 8 : 6; }
constexpr int sum_smem(int G, int N, bool bf16) { return 8 * sum_depth(G, N) * G * 32 * sum_part(N, bf16); }

template <bool DB, bool EB, int N, int G>
__global__ void __launch_bounds__(256) embed_sum_kernel(SumArgs a) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kGroups = G, D = sum_depth(G, N), kPart = sum_part(N, DB);
  extern __shared__ __align__(16) uint8_t ring[];  // [warp][D][G][lane]: sum_part bytes
  uint8_t* mine_ring = ring + ((int)warp_id() * D * G * 32 + (int)lane_id()) * kPart;
  const int lane = (int)lane_id(), h = a.h;
  grid_wait();
  grid_release();
  const int ranges = (a.T + a.L - 1) / a.L, jobs = ranges * a.chunks;
  for (int job = blockIdx.x * 8 + (int)warp_id(); job < jobs; job += gridDim.x * 8) {
    const int j = job / a.chunks, chunk = job - j * a.chunks, lo = j * a.L;
    const int c0 = chunk * 32 * kGroups * N + lane * N;  // column groups c0 + 32 N k
    // keys (and positions) from 32 before the range to 64 past its start; -1 outside the table's
    auto at = [&](int i) {
      int2 kv = i >= 0 && i < a.T ? a.s[i] : make_int2(-1, 0);
      if (kv.x >= a.V) kv.x = -1;
      return kv;
    };
    const int kp = at(lo - 32 + lane).x;
    const int2 cur = at(lo + lane), fol = at(lo + 32 + lane);
    const int e = min(a.L, __popc(__ballot_sync(kAll, cur.x >= 0)));
    if (e == 0) continue;
    // bit i: position i starts a run
    int prev = __shfl_up_sync(kAll, cur.x, 1);
    const int before = __shfl_sync(kAll, kp, 31);
    if (lane == 0) prev = before;
    uint32_t m = __ballot_sync(kAll, cur.x != prev);
    uint64_t heads = m;
    prev = __shfl_up_sync(kAll, fol.x, 1);
    const int border = __shfl_sync(kAll, cur.x, 31);
    if (lane == 0) prev = border;
    m = __ballot_sync(kAll, fol.x != prev);
    heads |= (uint64_t)m << 32;
    auto next_head = [&](int i) {  // first head past i, 64 if none is in sight
      const uint64_t r = i < 63 ? heads >> (i + 1) : 0ull;
      return r ? i + __ffsll((long long)r) : 64;
    };
    int p0 = 0, pend;
    bool head_piece = false, tail_piece = false;
    if (!(heads & 1)) {  // a run that began earlier
      const int first = __shfl_sync(kAll, cur.x, 0), fwd = next_head(0) < 64 ? next_head(0) : 64;
      const int back = __clz(~__ballot_sync(kAll, kp == first));  // 32 where all of them are (clz of 0)
      if (back + fwd > kShort) head_piece = true;
      else p0 = fwd;
      pend = head_piece ? min(fwd, e) : fwd;
      if (fwd >= e && !head_piece) continue;
    } else {
      pend = 0;
    }
    const uint64_t mine = heads & ((e < 64 ? 1ull << e : 0ull) - 1ull) & ~((pend < 64 ? 1ull << pend : 0ull) - 1ull);
    if (mine) {  // runs that begin here; the last one decides where the range's work ends
      const int last = 63 - __clzll((long long)mine), n = next_head(last);
      tail_piece = n - last > kShort;
      pend = tail_piece ? e : n;
    }
    const int tail_from = tail_piece ? 63 - __clzll((long long)mine) : 64;
    float4 acc[kGroups];
    auto row_of = [&](int p) { return (size_t)__shfl_sync(kAll, p < 32 ? cur.y : fol.y, p & 31) * h + c0; };
    auto request = [&](int p, int slot) {
      if (p < pend) {
        const size_t base = row_of(p);
        if (EB && N == 4 && a.add) {  // the table's row that the run is added to
          const int id = __shfl_sync(kAll, p < 32 ? cur.x : fol.x, p & 31);
          if ((heads >> p) & 1)
#pragma unroll
            for (int k = 0; k < kGroups; ++k)
              if (c0 + 32 * N * k < h && lane % 8 == 0)
                asm volatile("prefetch.global.L2 [%0];" ::"l"((const uint16_t*)a.dtable + (size_t)id * h + c0 + 32 * N * k));
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          if (c0 + 32 * N * k < h) {
            const size_t i = base + 32 * N * k;
            const uint32_t to = smem_u32(mine_ring + (slot * G + k) * 32 * kPart);
            if (N == 4 || !DB) {
              const void* g = (const uint8_t*)a.dout + i * (DB ? 2 : 4);
              asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(g), "n"(kPart) : "memory");
            } else if (a.words) {  // the word with column i; nothing behind the last one is read
              const void* g = (const uint8_t*)a.dout + (i & ~(size_t)1) * 2;
              const int n = (i | 1) < (size_t)a.T * h ? 4 : 2;
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(g), "r"(n) : "memory");
            }
          }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto row_value = [&](int slot, int k, size_t base) {
      const uint8_t* at = mine_ring + (slot * G + k) * 32 * kPart;
      if (N == 4) return load4<DB>(at, 0);
      const size_t i = base + 32 * k;
      if (DB && !a.words) return loadn<DB, N>(a.dout, i);
      return loadn<DB, N>(at, DB ? i & 1 : 0);
    };
    bool fresh = true, in_head = head_piece;
    int slot = 0;
    for (int i = 0; i < D; ++i) request(p0 + i, i);
    for (int p = p0; p < pend; ++p) {
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      const size_t base = DB && N == 1 ? row_of(p) : 0;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
        if (c0 + 32 * N * k < h) {
          const float4 v = row_value(slot, k, base);
          acc[k] = fresh ? v : add4(acc[k], v);
        }
      request(p + D, slot);
      slot = slot + 1 == D ? 0 : slot + 1;
      fresh = p + 1 == pend || ((heads >> (p + 1)) & 1);
      if (!fresh) continue;
      const bool tail = p >= tail_from;
      if (in_head || tail) {
        float* dst = a.part + (size_t)(2 * j + (in_head ? 0 : 1)) * h + c0;
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          if (c0 + 32 * N * k < h) storen<false, N>(dst, 32 * N * k, acc[k]);
      } else {
        const int id = __shfl_sync(kAll, p < 32 ? cur.x : fol.x, p & 31);
        const size_t to = (size_t)id * h + c0;
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          if (c0 + 32 * N * k < h) {
            const float4 o = scaled(acc[k], a.scale);
            if (a.add) accumulate<EB, N>(a.dtable, to + 32 * N * k, o);
            else storen<EB, N>(a.dtable, to + 32 * N * k, o);
          }
      }
      in_head = false;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (tail_piece && chunk == 0) {
      const int id = __shfl_sync(kAll, cur.x, tail_from);
      if (lane == 0) a.longs[atomicAdd(a.ctl, 1)] = make_int2(j, id);  // their order does not enter the sums
    }
  }

  // what is left to clear, a few rows (32 at most) at a time: every warp's
  // first ones by its number, so that only a second turn waits for the counter
  // (8192 tokens of 128256 x 4096: 479 us with 16 KB at a time, 321 with 32,
  // 331 with 128)
  if (a.clear_rows == 0) return;
  constexpr int esz = EB ? 2 : 4;
  const int warps = gridDim.x * 8, end = (a.V - a.clear_row0 + a.clear_rows - 1) / a.clear_rows;
  int next = blockIdx.x + gridDim.x * (int)warp_id();
  while (next < end) {
    const int v_lo = a.clear_row0 + next * a.clear_rows, n = min(a.clear_rows, a.V - v_lo);
    if (end > warps && lane == 0) next = warps + atomicAdd(a.ctl + 1, 1);  // on its way during the stores
    uint32_t rows = __ballot_sync(kAll, lane < n && !a.used[v_lo + min(lane, n - 1)]);
    for (; rows; rows &= rows - 1) {
      uint8_t* row = (uint8_t*)a.dtable + (size_t)(v_lo + __ffs(rows) - 1) * h * esz;
      if (N == 4) {
#pragma unroll 4
        for (int c = lane; c < h / 4; c += 32) {
          if (EB) ((uint2*)row)[c] = make_uint2(0, 0);
          else ((uint4*)row)[c] = make_uint4(0, 0, 0, 0);
        }
      } else {
        for (int c = lane; c < h; c += 32) store1<EB>(row, c, 0.f);
      }
    }
    if (end <= warps) break;
    next = __shfl_sync(kAll, next, 0);
  }
}

// Long runs: their partial sums added in order by 1024 / CX groups of CX
// threads (a column each), every group an equal share, then the groups in
// order.
template <bool EB, int N>
__global__ void __launch_bounds__(1024) embed_long_kernel(SumArgs a, int CX) {
  __shared__ float4 share[1024];
  grid_wait();
  const int x = (int)threadIdx.x & (CX - 1), g = (int)threadIdx.x / CX, groups = 1024 / CX;
  const int c = ((int)blockIdx.y * CX + x) * N, h = a.h, n = a.ctl[0];
  for (int r = blockIdx.x; r < n; r += gridDim.x) {
    const int j0 = a.longs[r].x, id = a.longs[r].y;
    int k = 0;  // later ranges that the run reaches into
    while (true) {
      const int64_t i = (int64_t)(j0 + 1 + k + (int)threadIdx.x) * a.L;
      const int more = __syncthreads_count(i < a.T && a.s[i].x == id);
      k += more;
      if (more < 1024) break;
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < h) {
      const int lo = (int)((int64_t)k * g / groups), hi = (int)((int64_t)k * (g + 1) / groups);
      if (g == 0) acc = loadn<false, N>(a.part, (size_t)(2 * j0 + 1) * h + c);
      for (int q = lo; q < hi; q += 8) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (q + i < hi) v[i] = loadn<false, N>(a.part, (size_t)(2 * (j0 + 1 + q + i)) * h + c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (q + i < hi) acc = add4(acc, v[i]);
      }
    }
    share[threadIdx.x] = acc;
    __syncthreads();
    if (g == 0 && c < h) {
#pragma unroll 4
      for (int i = 1; i < groups; ++i) acc = add4(acc, share[i * CX + x]);
      acc = scaled(acc, a.scale);
      const size_t to = (size_t)id * h + c;
      if (a.add) accumulate<EB, N>(a.dtable, to, acc);
      else storen<EB, N>(a.dtable, to, acc);
    }
    __syncthreads();
  }
}

// Column groups a lane takes, and positions a range covers: 4 and 32 for many
// wide rows, fewer where that would leave warps without work.
struct SumShape {
  int G, L;
};
SumShape sum_shape(int T, int h) {
  SumShape s{4, 32};
  if (h <= 128 || (int64_t)(T / 16) * ((h + 511) / 512) < 2048) s.G = 1;
  const int chunks = (h + 128 * s.G - 1) / (128 * s.G);
  while (s.L > 4 && (int64_t)(T / s.L) * chunks < 2048) s.L /= 2;
  return s;
}

struct EmbedWs {
  size_t a, b, used, ctl, longs, part, total;
};
EmbedWs embed_ws(int T, int V, int h) {
  EmbedWs o;
  size_t x = 0;
  auto take = [&](size_t bytes) {
    const size_t r = x;
    x += (bytes + 255) / 256 * 256;
    return r;
  };
  const int L = sum_shape(T, h).L;
  o.a = take((size_t)T * 8);
  o.b = take((size_t)T * 8);
  o.used = take((size_t)V);
  o.ctl = take(8);
  o.longs = take(((size_t)T / kShort + 1) * 8);
  o.part = take((size_t)2 * ((T + L - 1) / L) * h * 4);
  o.total = x;
  return o;
}

bool embed_dims_ok(int T, int V, int h) {
  return T > 0 && V > 0 && h > 0 && T <= (1 << 28) && V < (1 << 30) && h <= (1 << 22);
}
// The sums' jobs are counted in 31 bits: ranges of at least four positions
// by chunks of at least 32 columns. The bound takes no alignment into
// account, so that the workspace query knows it too; 2^40 values fit no GPU.
bool embed_bwd_dims_ok(int T, int V, int h) {
  return embed_dims_ok(T, V, h) &&
         (int64_t)((T + sum_shape(T, h).L - 1) / sum_shape(T, h).L) * ((h + 31) / 32) <= (1 << 30);
}
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

int embed_fwd(const void* table, bool tb, const int32_t* ids, float scale, void* out, bool ob, int T, int V, int h,
              cudaStream_t st) {
  if (!embed_dims_ok(T, V, h) || !al(table, tb ? 2 : 4) || !al(out, ob ? 2 : 4)) return kRefused;
  const bool vec = h % 4 == 0 && al(table, tb ? 8 : 16) && al(out, ob ? 8 : 16);
  const int units = vec ? h / 4 : h;
  int bx = 32;
  while (bx < units && bx < 256) bx *= 2;
  const int by = 256 / bx;
  const dim3 block((unsigned)bx, (unsigned)by);
  const dim3 grid((unsigned)((units + bx - 1) / bx), (unsigned)std::min((T + by * kFwdRows - 1) / (by * kFwdRows), 65535));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, grid, block, 0, st, 1, table, ids, scale, out, T, V, h); };
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (tb) ob ? go(embed_fwd_kernel<true, true, N>) : go(embed_fwd_kernel<true, false, N>);
    else ob ? go(embed_fwd_kernel<false, true, N>) : go(embed_fwd_kernel<false, false, N>);
  };
  if (vec) pick(std::integral_constant<int, 4>());
  else pick(std::integral_constant<int, 1>());
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

size_t embed_bwd_workspace(int T, int V, int h) { return embed_bwd_dims_ok(T, V, h) ? embed_ws(T, V, h).total : 0; }

int embed_bwd(const int32_t* ids, const void* dout, bool db, float scale, void* dtable, bool eb, bool add, void* work,
              int T, int V, int h, cudaStream_t st) {
  if (!embed_bwd_dims_ok(T, V, h) || !al(work, 256) || !al(dout, db ? 2 : 4) || !al(dtable, eb ? 2 : 4)) return kRefused;
  const EmbedWs o = embed_ws(T, V, h);
  uint8_t* w = (uint8_t*)work;
  const bool vec = h % 4 == 0 && al(dout, db ? 8 : 16) && al(dtable, eb ? 8 : 16);
  const int units = vec ? h / 4 : h, esz = eb ? 2 : 4;
  const size_t row = (size_t)h * esz;
  SumShape shape = sum_shape(T, h);
  // a warp that adds to bf16 rows waits for them: more and narrower jobs
  // (16384 tokens of 151936 x 4096: 139 us with four groups a lane, 108 with one)
  if (add && eb) shape.G = 1;
  const int chunks = (units + 32 * shape.G - 1) / (32 * shape.G);
  const int64_t jobs = (int64_t)((T + shape.L - 1) / shape.L) * chunks;
  SortArgs a;
  a.ids = ids;
  a.a = (int2*)(w + o.a);
  a.b = (int2*)(w + o.b);
  a.ctl = (int32_t*)(w + o.ctl);
  const int first = add ? 0 : (int)std::min<size_t>((size_t)V, kClearFirst / row + 1);  // rows cleared beside the sort
  a.used = !add && first < V ? w + o.used : nullptr;
  a.clear = dtable;
  a.clear_bytes = first * row;
  a.T = T;
  a.V = V;
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // keys 0..V
  a.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  a.digit = (bits + a.passes - 1) / a.passes;
  a.ctas = T <= kSortOne ? 1 : kSortCtas;
  // Every warp more has 2^digit counters that are gone over four times a pass,
  // every group of 32 positions more is some hundred cycles of a warp's walk:
  // the groups a warp takes where the sum of both is least (1266 positions of
  // 884 rows 11.4 us with all warps, 10.5 so; 64 of 151936 10.2 and 8.7)
  const int groups = ((T + 31) / 32 + a.ctas - 1) / a.ctas;
  const double least = std::sqrt(groups * 8000.0 / (1 << a.digit));  // warps
  const int each = (int)std::lround(std::max(1.0, groups / least));
  a.warps = std::min(kSortWarps, (groups + each - 1) / each);
  const int smem = ((a.warps + 1) << a.digit) * 4;
  if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ((kSortWarps + 1) << kMaxDigit) * 4) != cudaSuccess)
    return kLaunchFailed;
  const size_t clearers = (a.clear_bytes + kClearBytes - 1) / kClearBytes;
  const dim3 sorters((unsigned)(a.ctas + (clearers + a.ctas - 1) / a.ctas * a.ctas));
  cudaError_t e = mt_host::launch_early(embed_sort_kernel, sorters, kSortThreads, smem, st, a.ctas, a);

  SumArgs b;
  b.s = (a.passes & 1) ? a.a : a.b;
  b.dout = dout;
  b.dtable = dtable;
  b.part = (float*)(w + o.part);
  b.longs = (int2*)(w + o.longs);
  b.used = a.used;
  b.ctl = a.ctl;
  b.scale = scale;
  b.T = T;
  b.V = V;
  b.h = h;
  b.L = shape.L;
  b.chunks = chunks;
  b.add = add ? 1 : 0;
  b.words = al(dout, 4) ? 1 : 0;
  b.clear_row0 = first;
  b.clear_rows = a.used ? (int)std::min<size_t>(32, std::max<size_t>(1, 32768 / row)) : 0;
  auto sums = [&](auto n, auto gr) {
    constexpr int N = decltype(n)::value, G = decltype(gr)::value;
    const int ring = sum_smem(G, N, db);
    const int resident = mt_host::num_sms() * std::min(6, (227 << 10) / (ring + 1024));  // blocks by their shared memory
    const dim3 grid((unsigned)(a.used ? resident : std::min<int64_t>(resident, (jobs + 7) / 8)));
    auto go = [&](auto k) {
      if (e == cudaSuccess && ring > 47 * 1024)
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
      if (e == cudaSuccess) e = mt_host::launch_early(k, grid, 256, ring, st, 1, b);
    };
    if (db) eb ? go(embed_sum_kernel<true, true, N, G>) : go(embed_sum_kernel<true, false, N, G>);
    else eb ? go(embed_sum_kernel<false, true, N, G>) : go(embed_sum_kernel<false, false, N, G>);
  };
  auto sums_n = [&](auto n) {
    if (shape.G == 4) sums(n, std::integral_constant<int, 4>());
    else sums(n, std::integral_constant<int, 1>());
  };
  if (vec) sums_n(std::integral_constant<int, 4>());
  else sums_n(std::integral_constant<int, 1>());
  if (T > kShort) {
    int CX = 32;
    while (CX < units && CX < 256) CX *= 2;
    const dim3 grid((unsigned)std::min(T / kShort + 1, mt_host::num_sms()), (unsigned)((units + CX - 1) / CX));
    auto longs = [&](auto n) {
      constexpr int N = decltype(n)::value;
      if (e != cudaSuccess) return;
      e = eb ? mt_host::launch_early(embed_long_kernel<true, N>, grid, 1024, 0, st, 1, b, CX)
             : mt_host::launch_early(embed_long_kernel<false, N>, grid, 1024, 0, st, 1, b, CX);
    };
    if (vec) longs(std::integral_constant<int, 4>());
    else longs(std::integral_constant<int, 1>());
  }
  count_launches(T > kShort ? 3 : 2);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

}  // namespace mt
