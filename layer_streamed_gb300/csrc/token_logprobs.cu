// Log probability of one given token per row of logits, with the row's
// log-sum-exp, entropy and k most likely tokens, and the gradient.
//
// For a row z and an inverse temperature c, with m = max z and d_j = c (z_j - m):
//   S = sum_j e^{d_j},  A = sum_j e^{d_j} d_j
//   lse = c m + ln S,  log p_j = d_j - ln S,  H = ln S - A / S
// Forward: one pass over the logits with a running (m, S, A) per thread, in
// 32 bits and log2 units (e^d = 2^{c2 (z - m)}, c2 = c log2 e; the difference
// is formed first, so large logits cost no accuracy). The k largest logits
// come from the maxima of that pass (see below). Backward: with p_j = e^{c z_j - lse},
//   dz_j = c (g_logp ([j = t] - p_j) - g_H p_j (log p_j + H)).
// Both directions are bound by reading the logits (and writing the gradient)
// where there are many; 16-bit logits come close to the issue rate too, so
// maxima and clamps are taken on packed pairs and sums on pairs of fp32.
// Measured: 8192 x 128256 fp32 (floor 618 us) forward 576-587 us, with the 8
// largest 589-599, gradient 1160 (floor 1236); 4095 x 151936 bf16 (183 and 366)
// 174-177, 184-188 and 355; 4096 x 32000 bf16 (39) 41 and 49. A few rows are
// bound by latency: one of 151936 4.8 us, with its 20 largest 9.4.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mt {

MT_DEVICE_ERROR_READER(token_logprobs_take_device_error)

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTop = 32;
// Logits at or below -kBig (-inf, a mask of the type's lowest value) are
// masked out; a row with one at or above kBig (or a NaN) has no distribution.
// 2^100 is a bf16 value too, and kBig * c stays finite for every allowed c.
constexpr float kBig = 1.2676506002282294e30f;
constexpr uint32_t kBigPair = 0xf180f180u;  // two bf16 -2^100
constexpr float kMinScale = 1e-6f, kMaxScale = 1e6f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t max_nan_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Statistics of a set of logits: the largest, and the sums of 2^d and 2^d d
// with d = c2 (z - m).
struct Stat {
  float m, s, a;
};
// Distance of two maxima, kept where 2^d is 0 but d times a count is finite
// (masked logits alone have the maximum -kBig and a count).
__device__ __forceinline__ float apart(float x, float m, float c2) { return fmaxf((x - m) * c2, -1024.f); }
__device__ __forceinline__ Stat merge(const Stat& x, const Stat& y, float c2) {
  const float m = fmaxf(x.m, y.m), dx = apart(x.m, m, c2), dy = apart(y.m, m, c2);
  const float ex = ex2(dx), ey = ex2(dy);
  return {m, x.s * ex + y.s * ey, (x.a + dx * x.s) * ex + (y.a + dy * y.s) * ey};
}

// Order-preserving whole number of a float (no NaN); both zeros get one.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kKeyNone = ~0xf1800000u;  // key of -kBig: masked out, or nothing there

// The lanes' sets joined: one maximum, each lane's sums brought to it, then
// plain sums in a fixed order.
__device__ __forceinline__ Stat warp_join(Stat x, float c2) {
  const float m = of_key(__reduce_max_sync(0xffffffffu, key_of(x.m))), d = apart(x.m, m, c2), e = ex2(d);
  x.a = (x.a + d * x.s) * e;
  x.s *= e;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x.s += __shfl_xor_sync(0xffffffffu, x.s, o);
    x.a += __shfl_xor_sync(0xffffffffu, x.a, o);
  }
  x.m = m;
  return x;
}

// The warp's 32 keys in descending order.
__device__ __forceinline__ uint32_t warp_sort(uint32_t key, uint32_t lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, key, o);
      key = ((lane & o) == 0) == ((lane & size) == 0) ? max(key, other) : min(key, other);
    }
  return key;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint32_t warp_merge(uint32_t a, uint32_t b, uint32_t lane) {
  uint32_t key = max(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, key, o);
    key = (lane & o) == 0 ? max(key, other) : min(key, other);
  }
  return key;
}

constexpr int kOneThreads = 128;  // a block alone with a row, at most
constexpr int kMaxThreads = 512;  // one of a cluster
constexpr int kVecs = 4;  // 16-byte vectors a thread holds at a time
constexpr int kMaxCluster = 8;
constexpr int kSegs = 32;

// A block's shared memory. cap: logits that may reach the bound before the
// slow search takes over.
struct Smem {
  uint2* cand;         // [cap]
  uint64_t* list;      // [C * k] key and ~index: k of each block, best first (the first block's is used)
  int* place;          // [C * k] places of the entries, where there are several blocks
  Stat* stat;          // [C * warps] (the first block's)
  uint32_t* key;       // [warps][32]
  float* seg;          // [segments][threads]
  uint16_t* hot;       // [cap] segment * threads + thread
};
__host__ __device__ inline size_t smem_layout(uint8_t* base, int NT, int C, int k, int cap, int segs, Smem* o) {
  size_t x = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + x;
    x += (bytes + 15) / 16 * 16;
    return p;
  };
  const int nw = NT / 32;
  Smem m;
  m.stat = (Stat*)take((size_t)C * nw * sizeof(Stat));
  if (k > 0) {
    m.cand = (uint2*)take((size_t)cap * 8);
    m.list = (uint64_t*)take((size_t)C * k * 8);
    m.place = (int*)take(C > 1 ? (size_t)C * k * 4 : 0);
    m.key = (uint32_t*)take((size_t)nw * 128);
    m.seg = (float*)take((size_t)segs * NT * 4);
    m.hot = (uint16_t*)take((size_t)cap * 2);
  }
  *o = m;
  return x;
}

struct FwdArgs {
  const void* z;
  const int32_t* ids;
  float *lse, *logp, *ent, *top_logp;
  int32_t* top_ids;
  int T, V, ld, k;
  float c;
  int C, G, cap, segs;  // blocks a row, chunks a segment, see Smem
};

// Vectors (16 bytes) of a row between its unaligned ends.
template <bool BF16>
struct RowView {
  static constexpr int E = BF16 ? 8 : 4, esz = BF16 ? 2 : 4;
  const uint8_t* p;
  int head, nv, tail0;  // logits [0, head) and [tail0, V) lie outside whole vectors
  __device__ __forceinline__ RowView(const void* base, size_t row, int ld, int V) {
    p = (const uint8_t*)base + row * (size_t)ld * esz;
    const int off = (int)((16u - ((uint32_t)(uintptr_t)p & 15u)) & 15u) / esz;
    head = min(off, V);
    nv = (V - head) / E;
    tail0 = head + nv * E;
  }
  __device__ __forceinline__ float at(int i) const {
    return BF16 ? bf2f(((const uint16_t*)p)[i]) : ((const float*)p)[i];
  }
  __device__ __forceinline__ const uint4* vec(int v) const { return (const uint4*)(p + (size_t)head * esz) + v; }
  // End logit e (0..7 the head's, 8..15 the tail's) of a block that owns those ends, or -1.
  __device__ __forceinline__ int end_index(int e, bool lo, bool hi, int V) const {
    if (e < 8) return lo && e < head ? e : -1;
    return hi && e < 16 && e - 8 < V - tail0 ? tail0 + (e - 8) : -1;  // (V may be 2^31 - 1)
  }
};
template <bool BF16>
__device__ __forceinline__ void spread(const uint4& u, float* out) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      out[i] = __uint_as_float(w[i]);
    }
  }
}

// A thread's running statistics, sums kept as pairs.
struct Run {
  float m;
  uint64_t s, a;
  bool bad;
};
// One chunk of kVecs vectors. Masked logits are raised to -kBig, where 2^d is
// 0 and 2^d d too.
template <bool BF16>
__device__ __forceinline__ float take(Run& r, uint4 (&u)[kVecs], float c2) {
  float cm;
  if (BF16) {
    uint32_t top = kBigPair;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      u[j].x = max_nan_bf2(u[j].x, kBigPair);
      u[j].y = max_nan_bf2(u[j].y, kBigPair);
      u[j].z = max_nan_bf2(u[j].z, kBigPair);
      u[j].w = max_nan_bf2(u[j].w, kBigPair);
      top = max_nan_bf2(top, max_nan_bf2(max_nan_bf2(u[j].x, u[j].y), max_nan_bf2(u[j].z, u[j].w)));
    }
    cm = max_nan(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
  } else {
    cm = -kBig;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      float* f = (float*)&u[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = max_nan(f[i], -kBig);
      cm = max3_nan(cm, f[0], f[1]);
      cm = max3_nan(cm, f[2], f[3]);
    }
  }
  r.bad |= !(cm < kBig);
  const float m = fmaxf(r.m, cm), d0 = apart(r.m, m, c2), e0 = ex2(d0);
  const uint64_t e02 = pair(e0, e0);
  r.a = mul2(fma2(pair(d0, d0), r.s, r.a), e02);
  r.s = mul2(r.s, e02);
  r.m = m;
  const uint64_t cc = pair(c2, c2), mm = pair(-m, -m);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float z[BF16 ? 8 : 4];
    spread<BF16>(u[j], z);
#pragma unroll
    for (int i = 0; i < (BF16 ? 8 : 4); i += 2) {
      const uint64_t d = mul2(add2(pair(z[i], z[i + 1]), mm), cc);
      float d0_, d1_;
      unpair(d, d0_, d1_);
      const uint64_t e = pair(ex2(d0_), ex2(d1_));
      r.s = add2(r.s, e);
      r.a = fma2(e, d, r.a);
    }
  }
  return cm;
}

// An entry's place is the number of entries before it: all compared with all,
// the threads beyond one an entry sharing the comparisons out (halving in
// each block's list took 4600 cycles for 8 x 20 entries, single comparisons
// 2400; two at a time 62 x 27089 with the 32 largest 15.6 -> 14.8 us).
__device__ __forceinline__ void places(const uint64_t* list, int* place, int n) {
  const int tid = (int)threadIdx.x, NT = (int)blockDim.x;
  const int wide = (n + 31) & ~31, shares = max(1, NT / wide), g = shares > 1 ? tid / wide : 0;
  const int pairs = n / 2, lo = pairs * g / shares, hi = pairs * (g + 1) / shares;  // n is even
  if (g >= shares) return;
  for (int i = tid - g * wide; i < n; i += NT) {
    const uint64_t e = list[i];
    int before = 0;
#pragma unroll 8
    for (int j = lo; j < hi; ++j) {
      const ulonglong2 f = ((const ulonglong2*)list)[j];
      before += (f.x > e ? 1 : 0) + (f.y > e ? 1 : 0);
    }
    if (shares > 1) atomicAdd(&place[i], before);
    else place[i] = before;
  }
}

// Forward. A cluster of C blocks a row (C = 1 for many rows; more where the
// rows alone would leave SMs idle), each over its part of the row's vectors;
// the blocks' results are joined in the first one's shared memory.
//
// The k largest: with the threads' maxima, the k-th largest of them is a
// value that at least k logits reach (kth below). Each thread also leaves the
// maxima of up to kSegs segments of its logits (G chunks each) in shared
// memory; the few segments that reach kth are read a second time, and their
// logits that reach it are collected and ranked by (value, index). Where more
// than cap do (rows of one value), the k are searched one by one.
// Sorted lists kept while streaming took 230 us more for k = 8 on 8192 x
// 128256 fp32 rows (828 against 598 us without a list), and reading all of
// the k best threads' logits again 137 us more, since DRAM moves 64 bytes for
// every 16 of them.
// ONE: a block a row (a.C = 1). Blocks an SM, by the registers a thread gets:
// 4095 x 151936 bf16 with the 8 largest 211 us unbounded, 203 with nine, 199
// with eight, 188 with seven, 191 with six; clusters (64 x 128256) 8.1 us
// unbounded, 6.9 with two of the largest block.
template <bool BF16, bool TOP, bool ONE>
__global__ void __launch_bounds__(ONE ? kOneThreads : kMaxThreads, ONE ? 7 : 2) token_logprobs_kernel(FwdArgs a) {
  using R = RowView<BF16>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ uint32_t sh_kth;
  __shared__ int sh_bad, sh_nhot, sh_n;
  const int C = ONE ? 1 : a.C, G = a.G, cap = a.cap;
  const int t = blockIdx.x / C, rank = blockIdx.x % C;
  const uint32_t lane = lane_id(), warp = warp_id();
  const int tid = (int)threadIdx.x, NT = (int)blockDim.x, nw = NT >> 5;
  Smem sm;
  smem_layout(smem_raw, NT, C, a.k, cap, a.segs, &sm);
  const R row(a.z, t, a.ld, a.V);
  const float c2 = a.c * kLog2e;
  const int v_lo = (int)((int64_t)row.nv * rank / C), v_hi = (int)((int64_t)row.nv * (rank + 1) / C);
  const bool lo_end = rank == 0, hi_end = rank == C - 1;
  const uint32_t none = BF16 ? kBigPair : 0xf1800000u;
  auto fetch = [&](int v, uint4 (&u)[kVecs]) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      u[j] = v + j * NT < v_hi ? __ldcs(row.vec(v + j * NT)) : make_uint4(none, none, none, none);
  };
  grid_wait();
  // the first chunk is requested before the row's token is known: their
  // latencies overlap
  uint4 next[kVecs];
  fetch(v_lo + tid, next);
  const int id = a.ids[t];
  if (id < 0 || id >= a.V) {  // the same for every block of the cluster
    if (rank == 0) {
      const float fill = id < 0 ? 0.f : __int_as_float(0x7fffffff);
      if (tid == 0) {
        a.lse[t] = fill;
        a.logp[t] = fill;
        if (a.ent) a.ent[t] = fill;
        if (id >= a.V) report_error(kErrBadArg);
      }
      if (TOP && tid < a.k) {
        a.top_ids[(size_t)t * a.k + tid] = -1;
        a.top_logp[(size_t)t * a.k + tid] = fill;
      }
    }
    return;
  }
  if (tid == 0) sh_bad = 0, sh_nhot = 0, sh_n = 0;
  if (TOP && C > 1)
    for (int i = tid; i < C * a.k; i += NT) sm.place[i] = 0;
  // every block's shared memory is set up before another one writes to it
  // (waited for just before the first such write)
  if (C > 1) {
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  float given = 0.f;  // the given token's logit
  if (rank == 0 && tid == 0) given = row.at(id);
  Run run{-kBig, 0ull, 0ull, false};
  {
    float seg = -kBig;  // largest of this segment
    int left = G, entry = tid;
    for (int v = v_lo + tid; v < v_hi; v += NT * kVecs) {  // the next chunk's loads run under this one's sums
      uint4 u[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) u[j] = next[j];
      fetch(v + NT * kVecs, next);
      const float cm = take<BF16>(run, u, c2);
      if (TOP) {
        seg = fmaxf(seg, cm);
        if (--left == 0) {
          sm.seg[entry] = seg;
          seg = -kBig;
          left = G;
          entry += NT;
        }
      }
    }
    if (TOP && left != G) sm.seg[entry] = seg;
  }
  const float tmax = run.m;  // of the whole vectors
  {  // the unaligned ends of the row: fewer than one vector each
    const int i = row.end_index(tid, lo_end, hi_end, a.V);
    if (i >= 0) {
      uint4 u[kVecs];
#pragma unroll
      for (int j = 0; j < kVecs; ++j) u[j] = make_uint4(none, none, none, none);
      u[0].x = BF16 ? (none & 0xffff0000u) | ((const uint16_t*)row.p)[i] : ((const uint32_t*)row.p)[i];
      take<BF16>(run, u, c2);
    }
  }

  // join: lanes, then warps (and blocks) in order
  float s0, s1, a0, a1;
  unpair(run.s, s0, s1);
  unpair(run.a, a0, a1);
  Stat st{run.m, s0 + s1, a0 + a1};
  st = warp_join(st, c2);
  const bool bad = __any_sync(0xffffffffu, run.bad);
  auto put = [rank](void* p, uint32_t v) {  // to the first block's shared memory
    if (rank == 0) *(volatile uint32_t*)p = v;
    else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(p, 0)), "r"(v) : "memory");
  };
  if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();  // sh_bad, sh_nhot and sh_n are set up
  if (lane == 0) {
    Stat* slot = &sm.stat[rank * nw + (int)warp];
    put(&slot->m, __float_as_uint(st.m));
    put(&slot->s, __float_as_uint(st.s));
    put(&slot->a, __float_as_uint(st.a));
    if (bad) put(&sh_bad, 1u);
  }

  if (TOP) {
    const uint32_t mine = max(key_of(tmax), kKeyNone);
    uint32_t key = warp_sort(mine, lane);
    for (int o = 1; o < nw; o *= 2) {  // the warps' lists joined pairwise
      if ((warp & (2 * o - 1)) == (uint32_t)o) sm.key[warp * 32 + lane] = key;
      __syncthreads();
      if ((warp & (2 * o - 1)) == 0) key = warp_merge(key, sm.key[(warp + o) * 32 + lane], lane);
    }
    if (warp == 0 && (int)lane == a.k - 1) sh_kth = max(key, kKeyNone + 1);
    __syncthreads();
    const uint32_t kth = sh_kth;
    const int chunks = v_lo + tid < v_hi ? (v_hi - v_lo - tid + NT * kVecs - 1) / (NT * kVecs) : 0;
    if (mine >= kth) {
      const float bound = of_key(kth);
      for (int e = tid, c = 0; c < chunks; e += NT, c += G)
        if (sm.seg[e] >= bound) {
          const int at = atomicAdd(&sh_nhot, 1);
          if (at < cap) sm.hot[at] = (uint16_t)e;
        }
    }
    __syncthreads();
    const int nhot = sh_nhot;
    auto offer = [&](float z, int i) {
      const uint32_t q = key_of(z);
      if (q >= kth) {
        const int at = atomicAdd(&sh_n, 1);
        if (at < cap) sm.cand[at] = make_uint2(q, (uint32_t)i);
      }
    };
    const int per = G * kVecs, all = min(nhot, cap) * per;  // vectors of the listed segments
    for (int q = tid; q < all; q += NT) {
      const int e = sm.hot[q / per], v = v_lo + (e & (NT - 1)) + (e / NT * per + q % per) * NT;
      if (v < v_hi) {
        const uint4 u = *row.vec(v);
        float z[R::E];
        spread<BF16>(u, z);
#pragma unroll
        for (int i = 0; i < R::E; ++i) offer(z[i], row.head + v * R::E + i);
      }
    }
    const int end = row.end_index(tid, lo_end, hi_end, a.V);
    if (end >= 0) offer(row.at(end), end);
    __syncthreads();
    const int found = sh_n, n = max(found, nhot);  // too many segments count as too many logits
    auto list = [&](int place, uint2 e) {  // empty entries follow the others, in an order of their own
      uint32_t* to = (uint32_t*)&sm.list[rank * a.k + place];
      put(to, ~(e.x > kKeyNone ? e.y : 0x80000000u + (uint32_t)(rank * a.k + place)));
      put(to + 1, e.x);
    };
    if (n <= cap) {
      for (int i = tid; i < found; i += NT) {
        const uint2 e = sm.cand[i];
        int better = 0;
#pragma unroll 8
        for (int j = 0; j < found; ++j) {
          const uint2 f = sm.cand[j];
          better += f.x > e.x || (f.x == e.x && f.y < e.y) ? 1 : 0;
        }
        if (better < a.k) list(better, e);
      }
      if (tid >= found && tid < a.k) list(tid, make_uint2(kKeyNone, 0xffffffffu));
    } else {
      uint2 last = make_uint2(0xffffffffu, 0u);
      for (int r = 0; r < a.k; ++r) {
        uint2 best = make_uint2(kKeyNone, 0xffffffffu);
        auto look = [&](float z, int i) {
          const uint32_t q = key_of(z);
          const bool open = q < last.x || (q == last.x && (uint32_t)i > last.y);
          if (open && (q > best.x || (q == best.x && (uint32_t)i < best.y)) && q > kKeyNone)
            best = make_uint2(q, (uint32_t)i);
        };
        for (int v = v_lo + tid; v < v_hi; v += NT) {
          float z[R::E];
          spread<BF16>(*row.vec(v), z);
#pragma unroll
          for (int i = 0; i < R::E; ++i) look(z[i], row.head + v * R::E + i);
        }
        if (end >= 0) look(row.at(end), end);
        const uint32_t wk = __reduce_max_sync(0xffffffffu, best.x);
        const uint32_t wi = __reduce_min_sync(0xffffffffu, best.x == wk ? best.y : 0xffffffffu);
        __syncthreads();  // the last round's entries have been read
        if (lane == 0) sm.cand[warp] = make_uint2(wk, wi);
        __syncthreads();
        last = make_uint2(kKeyNone, 0xffffffffu);
        for (int w = 0; w < nw; ++w) {
          const uint2 e = sm.cand[w];
          if (e.x > last.x || (e.x == last.x && e.y < last.y)) last = e;
        }
        if (tid == 0) list(r, last);
      }
    }
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0) return;

  const float nan = __int_as_float(0x7fffffff);
  const bool broken = sh_bad != 0;
  Stat f{-kBig, 0.f, 0.f};
  for (int i = (int)lane; i < C * nw; i += 32) f = merge(f, sm.stat[i], c2);
  f = warp_join(f, c2);
  const bool empty = f.m <= -kBig;  // every logit is masked out
  const float ln_s = logf(f.s);
  auto logp_of = [&](float z) { return broken ? nan : z <= -kBig ? -INFINITY : (z - f.m) * a.c - ln_s; };
  if (tid == 0) {
    a.lse[t] = broken ? nan : empty ? -INFINITY : fmaf(f.m, a.c, ln_s);
    a.logp[t] = logp_of(given);
    if (a.ent) a.ent[t] = broken ? nan : empty ? 0.f : fmaxf(ln_s - kLn2 * (f.a / f.s), 0.f);
  }
  if (TOP) {
    const int n = C * a.k;
    auto write = [&](int place, uint64_t e) {
      const uint32_t key = (uint32_t)(e >> 32);
      const bool there = key > kKeyNone && !broken;
      a.top_ids[(size_t)t * a.k + place] = there ? (int32_t)~(uint32_t)e : -1;
      a.top_logp[(size_t)t * a.k + place] = there ? logp_of(of_key(key)) : broken ? nan : -INFINITY;
    };
    if (C == 1) {
      if (tid < a.k) write(tid, sm.list[tid]);
    } else {
      places(sm.list, sm.place, n);
      __syncthreads();
      for (int i = tid; i < n; i += NT)
        if (sm.place[i] < a.k) write(sm.place[i], sm.list[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: a thread holds kBwdVecs vectors of neighbouring logits of one row.
// ---------------------------------------------------------------------------
struct BwdArgs {
  const void* z;
  const int32_t* ids;
  const float *lse, *ent, *g_logp, *g_ent;
  void* dz;
  int T, V, ld, ldd;
  float c;
};
constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 2;

// Blocks of blockDim.x threads along a row by blockDim.y rows (short rows
// share a block). A thread's logits are requested before the row's scalars,
// whose loads they do not depend on. VEC: logits and gradient come to a
// 16-byte boundary at the same columns of a row; a row's units then start at
// its first such column, and the first threads take the columns before it.
// (Six blocks an SM: the 40 registers spill 12 to 16 bytes of bf16 logits
// without VEC, and nothing else.)
template <bool BF16, bool OBF16, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, 6) token_logprobs_bwd_kernel(BwdArgs a) {
  constexpr int esz = BF16 ? 2 : 4;
  constexpr int W = kBwdVecs * (BF16 ? 8 : 4);  // logits a thread holds at a time
  grid_wait();
  const float cs = a.c * -0x1p-8f;
  const uint64_t ll = pair(-0x1p8f * kLog2e, -0x1p8f * kLog2e);
  const int unit = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  for (int t = blockIdx.y * blockDim.y + threadIdx.y; t < a.T; t += gridDim.y * blockDim.y) {
    const int head = VEC ? (int)((8 - ((size_t)t * a.ld & 7)) & 7) : 0;  // a unit of 8 starts on every boundary
    const int j = unit * W + head - (head ? W : 0);  // unit 0 holds the columns before the boundary
    if (j >= a.V) continue;
    const bool whole = VEC && j >= 0 && j + W <= a.V;
    const uint8_t* zr = (const uint8_t*)a.z + (size_t)t * a.ld * esz;
    uint8_t* dr = (uint8_t*)a.dz + (size_t)t * a.ldd * (OBF16 ? 2 : 4);
    uint4 u[kBwdVecs];
    if (whole) {
#pragma unroll
      for (int i = 0; i < kBwdVecs; ++i) u[i] = __ldcs((const uint4*)(zr + (size_t)j * esz) + i);
    }
    const int id = a.ids[t];
    const bool off = id < 0 || id >= a.V;
    const float l = a.lse[t];
    // a row without any logit left has no gradient; a NaN row's is NaN
    const bool zero = off || l == -INFINITY;
    const float gl = a.g_logp ? a.g_logp[t] : 0.f, ge = a.g_ent ? a.g_ent[t] : 0.f;
    const float h = a.g_ent ? a.ent[t] : 0.f;
    // dz = c (gl [j = t] - p (gl + ge (log p + H)))
    const float k0 = l == l ? -a.c * (gl + ge * h) : l, k1 = 0x1p8f * a.c * ge, ls = l * 0x1p-8f;
    const uint64_t kk0 = pair(k0, k0), kk1 = pair(k1, k1);
    float g[W];
    if (zero) {
#pragma unroll
      for (int i = 0; i < W; ++i) g[i] = 0.f;
    } else {
      float z[W];
      if (whole) {
#pragma unroll
        for (int i = 0; i < kBwdVecs; ++i) spread<BF16>(u[i], z + i * (W / kBwdVecs));
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          z[i] = j + i >= 0 && j + i < a.V ? (BF16 ? bf2f(((const uint16_t*)zr)[j + i]) : ((const float*)zr)[j + i]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        // -log p / 256 within [0, 1]: p is 0 at the one end, and no product
        // of its logarithm overflows; at the other, it is 1 at most
        const uint64_t y = pair(__saturatef(fmaf(z[i], cs, ls)), __saturatef(fmaf(z[i + 1], cs, ls)));
        float x0, x1;
        unpair(mul2(y, ll), x0, x1);  // log2 p
        unpair(mul2(pair(ex2(x0), ex2(x1)), fma2(kk1, y, kk0)), g[i], g[i + 1]);
      }
      if ((unsigned)(id - j) < (unsigned)W) {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (j + i == id) g[i] += a.c * gl;
      }
    }
    if (whole) {
      if (OBF16) {
#pragma unroll
        for (int i = 0; i < W; i += 8)
          __stcs((uint4*)(dr + (size_t)(j + i) * 2),
                 make_uint4(pack_bf2(g[i], g[i + 1]), pack_bf2(g[i + 2], g[i + 3]), pack_bf2(g[i + 4], g[i + 5]),
                            pack_bf2(g[i + 6], g[i + 7])));
      } else {
#pragma unroll
        for (int i = 0; i < W; i += 4)
          __stcs((float4*)(dr + (size_t)(j + i) * 4), make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (j + i >= 0 && j + i < a.V) {
          if (OBF16) ((uint16_t*)dr)[j + i] = f2bf(g[i]);
          else ((float*)dr)[j + i] = g[i];
        }
    }
  }
}

inline bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

int token_logprobs(const void* z, bool bf16, const int32_t* ids, float c, int k, float* lse, float* logp, float* ent,
                   int32_t* top_ids, float* top_logp, int T, int V, int ld, cudaStream_t st) {
  if (T <= 0 || V <= 0 || ld < V || k < 0 || k > kMaxTop || k > V || !(c >= kMinScale) || !(c <= kMaxScale) ||
      ((uintptr_t)z & (bf16 ? 1 : 3)) || T > (1 << 28))
    return kRefused;
  // Threads a block: the more rows, the more chunks each, so that a short row
  // needs no more than a warp or two (4227 x 12722 bf16 with the 8 largest: 37
  // us with four chunks each, 26 with sixteen; 2200 rows 21, 18 with eight);
  // else one. Blocks a row: where the rows alone do not fill the GPU twice over,
  // as many as leave every thread a chunk (two or four where lists are to be
  // joined: 141 x 7935 bf16 with the 8 largest 7.2 us with one, 5.4 with two; 62 x
  // 27089 fp32 with 20 10.6 and 8.4 with four), and larger blocks (up to 512
  // threads an SM: 64 x 128256 bf16 5.7 us, 6.6 with 1024) where even that does
  // not.
  const int chunk = kVecs * (bf16 ? 8 : 4), sms = mt_host::num_sms();
  const int each = T >= 16 * sms ? 16 * chunk : T >= 8 * sms ? 8 * chunk : chunk;
  int NT = 32, C = 1;
  while (NT < kOneThreads && NT * each < V) NT *= 2;
  while (C < kMaxCluster && (int64_t)T * C < 2 * sms && V > C * NT * chunk * (k > 8 ? 4 : k ? 2 : 1)) C *= 2;
  while (C == kMaxCluster && NT < kMaxThreads && 2 * NT * T * C <= 512 * sms && V > C * NT * chunk) NT *= 2;
  // a block's vectors, at most, in chunks a thread; segments of G chunks
  const int vecs = V / (bf16 ? 8 : 4) / C + 1, chunks = (vecs + NT * kVecs - 1) / (NT * kVecs);
  const int G = (chunks + kSegs - 1) / kSegs;
  const int segs = (chunks + G - 1) / G, cap = std::max(256, 4 * NT);
  FwdArgs a{z, ids, lse, logp, ent, top_logp, top_ids, T, V, ld, k, c, C, G, cap, segs};
  Smem unused;
  const size_t smem = smem_layout(nullptr, NT, C, k, cap, segs, &unused);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto f) {
    if (smem > 47 * 1024)  // with the static part past the default limit
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e == cudaSuccess) e = mt_host::launch_early(f, T * C, NT, smem, st, C, a);
  };
  auto pick = [&](auto one) {
    constexpr bool X = decltype(one)::value;
    if (k > 0) bf16 ? go(token_logprobs_kernel<true, true, X>) : go(token_logprobs_kernel<false, true, X>);
    else bf16 ? go(token_logprobs_kernel<true, false, X>) : go(token_logprobs_kernel<false, false, X>);
  };
  if (C == 1) pick(std::true_type());
  else pick(std::false_type());
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

int token_logprobs_bwd(const void* z, bool bf16, const int32_t* ids, float c, const float* lse, const float* ent,
                       const float* g_logp, const float* g_ent, void* dz, bool dz_bf16, int T, int V, int ld, int ldd,
                       cudaStream_t st) {
  // (row and column counters step past the last one by up to a round of the grid)
  if (T <= 0 || V <= 0 || ld < V || ldd < V || T > (1 << 30) || V > (1 << 30) || !(c >= kMinScale) ||
      !(c <= kMaxScale) || (g_ent && !ent) || ((uintptr_t)z & (bf16 ? 1 : 3)) ||
      ((uintptr_t)dz & (dz_bf16 ? 1 : 3)))
    return kRefused;
  BwdArgs a{z, ids, lse, ent, g_logp, g_ent, dz, T, V, ld, ldd, c};
  // every eighth element of both on a 16-byte boundary at the same columns
  const bool vec = al16(z) && al16(dz) && (ld - ldd) % 8 == 0;
  const int W = kBwdVecs * (bf16 ? 8 : 4), units = (V + W - 1) / W + (vec && ld % 8 ? 1 : 0);
  int bx = 8;
  while (bx < units && bx < kBwdThreads) bx *= 2;
  const int by = kBwdThreads / bx;
  const dim3 block((unsigned)bx, (unsigned)by);
  const dim3 grid((unsigned)((units + bx - 1) / bx), (unsigned)std::min((T + by - 1) / by, 65535));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, grid, block, 0, st, 1, a); };
  auto pick = [&](auto v) {
    constexpr bool X = decltype(v)::value;
    if (bf16) dz_bf16 ? go(token_logprobs_bwd_kernel<true, true, X>) : go(token_logprobs_bwd_kernel<true, false, X>);
    else dz_bf16 ? go(token_logprobs_bwd_kernel<false, true, X>) : go(token_logprobs_bwd_kernel<false, false, X>);
  };
  if (vec) pick(std::true_type());
  else pick(std::false_type());
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

}  // namespace mt
