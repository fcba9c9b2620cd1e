// Log probability of one given token per row of logits, with the row's
// log-sum-exp, entropy and k most likely tokens, and the gradient.
//
// For a row z and an inverse temperature c, with m = max z and d_j = c (z_j - m):
//   S = sum_j e^{d_j},  A = sum_j e^{d_j} d_j
//   lse = c m + ln S,  log p_j = d_j - ln S,  H = ln S - A / S
// Forward: one pass over the logits with a running (m, S, A) per thread, in
// 32 bits; differences from the maximum are formed before the scaling, so
// neither large logits nor masks of the type's lowest value overflow, and
// log p near 0 keeps its absolute accuracy. The k largest logits come from
// the same pass (see TopList). Backward: with p_j = e^{c z_j - lse},
//   dz_j = c (g_logp ([j = t] - p_j) - g_H p_j (log p_j + H)).
// Both directions are bound by reading the logits (and writing the gradient).
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
constexpr float kFar = -1000.f;  // 2^kFar is 0, and 0 * kFar too: stands for -inf in sums of e d
constexpr int kMaxTop = 32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Running statistics of a set of logits: largest, sum of 2^d, sum of 2^d d,
// d = c2 (z - m) in log2 units. The empty set has m = -FLT_MAX, s = 0.
struct Stat {
  float m, s, a;
};
__device__ __forceinline__ void rescale(Stat& x, float m, float c2) {
  const float d = fmaxf((x.m - m) * c2, kFar), r = ex2(d);
  x.a = (x.a + d * x.s) * r;
  x.s *= r;
  x.m = m;
}
__device__ __forceinline__ Stat merge(Stat x, Stat y, float c2) {
  const float m = fmaxf(x.m, y.m);
  rescale(x, m, c2);
  rescale(y, m, c2);
  return {m, x.s + y.s, x.a + y.a};
}

// Order-preserving whole number of a float (no NaN); both zeros get one.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// Logits at or below kMasked count as masked out, like -inf (a mask of the
// type's lowest value): probability 0, never listed.
constexpr float kMasked = -1e30f;
constexpr uint32_t kKeyNone = 0xeb60d35u;  // key of kMasked: an empty place of a list

// The k best (value, then lower index) that a warp has seen, place j in lane j.
struct TopList {
  uint32_t key, idx;
  __device__ __forceinline__ void insert(uint32_t k, uint32_t i, uint32_t lane) {
    const bool stays = key > k || (key == k && idx < i);
    const int at = __popc(__ballot_sync(0xffffffffu, stays));
    const uint32_t pk = __shfl_up_sync(0xffffffffu, key, 1), pi = __shfl_up_sync(0xffffffffu, idx, 1);
    if ((int)lane == at) {
      key = k;
      idx = i;
    } else if ((int)lane > at) {
      key = pk;
      idx = pi;
    }
  }
};

// The k-th largest of the warp's 32 keys.
__device__ __forceinline__ uint32_t warp_kth(uint32_t key, int k, uint32_t lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, key, o);
      const bool down = (lane & size) == 0;            // descending runs
      const bool low = (lane & o) == 0;
      key = (low == down) ? max(key, other) : min(key, other);
    }
  return __shfl_sync(0xffffffffu, key, k - 1);
}

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 16;  // logits a thread holds at a time
constexpr int kMaxCluster = 8;

struct FwdArgs {
  const void* z;
  const int32_t* ids;
  float *lse, *logp, *ent, *top_logp;
  int32_t* top_ids;
  int T, V, ld, k;
  float c;
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

// A cluster of C blocks per row (C = 1 for many rows; more where the rows
// alone would leave SMs idle), each over its part of the row's vectors; the
// blocks' statistics and lists are joined in the first one's shared memory.
template <bool BF16, bool TOP>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(FwdArgs a, int C) {
  using R = RowView<BF16>;
  constexpr int U = kChunk / R::E;  // vectors a thread holds at a time
  __shared__ Stat sh_stat[kMaxCluster * kWarps];
  __shared__ uint32_t sh_key[TOP ? kMaxCluster * kWarps : 1][kMaxTop], sh_idx[TOP ? kMaxCluster * kWarps : 1][kMaxTop];
  __shared__ int sh_bad;
  __shared__ uint32_t sh_thr;
  const int t = blockIdx.x / C, rank = blockIdx.x % C;
  const uint32_t lane = lane_id(), warp = warp_id();
  const int id = a.ids[t];
  if (id < 0 || id >= a.V) {  // the same for every block of the cluster
    if (rank == 0) {
      const float fill = id < 0 ? 0.f : __int_as_float(0x7fffffff);
      if (threadIdx.x == 0) {
        a.lse[t] = fill;
        a.logp[t] = fill;
        if (a.ent) a.ent[t] = fill;
        if (id >= a.V) report_error(kErrBadArg);
      }
      if (TOP && (int)threadIdx.x < a.k) {
        a.top_ids[(size_t)t * a.k + threadIdx.x] = -1;
        a.top_logp[(size_t)t * a.k + threadIdx.x] = fill;
      }
    }
    return;
  }
  if (threadIdx.x == 0) {
    sh_bad = 0;
    sh_thr = kKeyNone + 1;
  }
  __syncthreads();
  if (C > 1) cluster_sync();  // every block's shared memory is set up before another one writes to it
  const R row(a.z, t, a.ld, a.V);
  const float c2 = a.c * kLog2e;
  const int v_lo = (int)((int64_t)row.nv * rank / C), v_hi = (int)((int64_t)row.nv * (rank + 1) / C);
  Stat st{-FLT_MAX, 0.f, 0.f};
  bool bad = false;
  TopList top{kKeyNone, 0xffffffffu};
  uint32_t tkey = kKeyNone + 1;  // values below cannot enter
  float thr = of_key(kKeyNone + 1);
  bool first = true;

  // One chunk: z[i] is the logit of index index_of(i), -inf where there is none.
  auto take = [&](const float (&z)[kChunk], auto index_of) {
    float cm = z[0];
#pragma unroll
    for (int i = 1; i < kChunk; ++i) cm = max_nan(cm, z[i]);
    bad |= !(cm <= FLT_MAX);
    const float m = fmaxf(st.m, cm);
    rescale(st, m, c2);
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float d = fmaxf((z[i] - m) * c2, kFar);
      const float e = ex2(d);
      s += e;
      q = fmaf(e, d, q);
    }
    st.s += s;
    st.a += q;
    if (TOP) {
      if (first) {  // at least k logits of this chunk reach the k-th largest of the lanes' maxima
        first = false;
        tkey = max(tkey, warp_kth(key_of(cm), a.k, lane));
        thr = of_key(tkey);
      } else {
        const uint32_t shared = *(volatile uint32_t*)&sh_thr;
        if (shared > tkey) {
          tkey = shared;
          thr = of_key(tkey);
        }
      }
      if (__any_sync(0xffffffffu, cm >= thr)) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) bits |= z[i] >= thr ? 1u << i : 0u;
        while (true) {
          const uint32_t who = __ballot_sync(0xffffffffu, bits != 0);
          if (!who) break;
          const int src = __ffs(who) - 1;
          const int i = __ffs(bits) - 1;
          float v = z[0];
#pragma unroll
          for (int j = 1; j < kChunk; ++j) v = i == j ? z[j] : v;
          const uint32_t k = __shfl_sync(0xffffffffu, key_of(v), src);
          const uint32_t x = __shfl_sync(0xffffffffu, (uint32_t)index_of(i), src);
          if ((int)lane == src) bits &= bits - 1;
          top.insert(k, x, lane);
        }
        // later logits of this warp have higher indexes: they must exceed its
        // k-th best; another warp's must reach it
        const uint32_t kth = __shfl_sync(0xffffffffu, top.key, a.k - 1);
        if (kth > kKeyNone) {
          if (lane == 0) atomicMax(&sh_thr, kth);
          if (kth + 1 > tkey) {
            tkey = kth + 1;
            thr = of_key(tkey);
          }
        }
      }
    }
  };

  for (int v = v_lo + (int)warp * 32; v < v_hi; v += kThreads * U) {  // whole warps
    float z[kChunk];
    uint4 u[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int w = v + j * kThreads + (int)lane;
      if (w < v_hi) u[j] = __ldcs(row.vec(w));
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (v + j * kThreads + (int)lane < v_hi) {
        spread<BF16>(u[j], z + j * R::E);
      } else {
#pragma unroll
        for (int i = 0; i < R::E; ++i) z[j * R::E + i] = -INFINITY;
      }
    }
    take(z, [&](int i) { return row.head + (v + (i / R::E) * kThreads + (int)lane) * R::E + i % R::E; });
  }
  if (warp == 0) {  // the unaligned ends of the row: fewer than one vector each
    const bool lo = rank == 0, hi = rank == C - 1;
    int i0 = -1;
    if (lane < 8) i0 = lo && (int)lane < row.head ? (int)lane : -1;
    else if (lane < 16) i0 = hi && row.tail0 + (int)lane - 8 < a.V ? row.tail0 + (int)lane - 8 : -1;
    if (__any_sync(0xffffffffu, i0 >= 0)) {
      float z[kChunk];
#pragma unroll
      for (int i = 0; i < kChunk; ++i) z[i] = -INFINITY;
      if (i0 >= 0) z[0] = row.at(i0);
      // indexes below those already listed may tie with the k-th best
      if (TOP && !first) {
        const uint32_t kth = __shfl_sync(0xffffffffu, top.key, a.k - 1);
        if (tkey == kth + 1 && kth > kKeyNone) {
          tkey = kth;
          thr = of_key(tkey);
        }
      }
      take(z, [&](int) { return i0; });
    }
  }

  // join: lanes, then warps (and blocks) in order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat y{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
           __shfl_xor_sync(0xffffffffu, st.a, o)};
    st = merge(st, y, c2);
  }
  bad = __any_sync(0xffffffffu, bad);
  {
    // the first block's shared memory, as a cluster address where there is one
    const int slot = rank * kWarps + (int)warp;
    if (C == 1 || rank == 0) {
      if (lane == 0) {
        sh_stat[slot] = st;
        if (bad) sh_bad = 1;
      }
      if (TOP && (int)lane < a.k) {
        sh_key[slot][lane] = top.key;
        sh_idx[slot][lane] = top.idx;
      }
    } else {
      auto put = [](const void* p, uint32_t v) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(p, 0)), "r"(v) : "memory");
      };
      if (lane == 0) {
        put(&sh_stat[slot].m, __float_as_uint(st.m));
        put(&sh_stat[slot].s, __float_as_uint(st.s));
        put(&sh_stat[slot].a, __float_as_uint(st.a));
        if (bad) put(&sh_bad, 1u);
      }
      if (TOP && (int)lane < a.k) {
        put(&sh_key[slot][lane], top.key);
        put(&sh_idx[slot][lane], top.idx);
      }
    }
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0 || warp != 0) return;

  const int n = C * kWarps;
  Stat f{-FLT_MAX, 0.f, 0.f};
  for (int i = (int)lane; i < n; i += 32) f = merge(f, sh_stat[i], c2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat y{__shfl_xor_sync(0xffffffffu, f.m, o), __shfl_xor_sync(0xffffffffu, f.s, o),
           __shfl_xor_sync(0xffffffffu, f.a, o)};
    f = merge(f, y, c2);
  }
  const float nan = __int_as_float(0x7fffffff);
  const bool none = f.m <= kMasked;  // every logit is masked out
  const float ln_s = none ? 0.f : logf(f.s);
  auto logp_of = [&](float z) { return sh_bad ? nan : z <= kMasked ? -INFINITY : (z - f.m) * a.c - ln_s; };
  if (lane == 0) {
    a.lse[t] = sh_bad ? nan : none ? -INFINITY : fmaf(f.m, a.c, ln_s);
    a.logp[t] = logp_of(row.at(id));
    if (a.ent) a.ent[t] = sh_bad ? nan : none ? 0.f : fmaxf(ln_s - kLn2 * f.a / f.s, 0.f);
  }
  if (TOP) {
    // k rounds: the best head of the sorted lists (two a lane at most)
    int p0 = 0, p1 = 0;
    for (int r = 0; r < a.k; ++r) {
      uint32_t k0 = kKeyNone, x0 = 0xffffffffu, k1 = kKeyNone, x1 = 0xffffffffu;
      if ((int)lane < n && p0 < a.k) k0 = sh_key[lane][p0], x0 = sh_idx[lane][p0];
      if ((int)lane + 32 < n && p1 < a.k) k1 = sh_key[lane + 32][p1], x1 = sh_idx[lane + 32][p1];
      const bool second = k1 > k0 || (k1 == k0 && x1 < x0);
      const uint32_t kb = second ? k1 : k0, xb = second ? x1 : x0;
      const uint32_t best = __reduce_max_sync(0xffffffffu, kb);
      const uint32_t at = __reduce_min_sync(0xffffffffu, kb == best ? xb : 0xffffffffu);
      if (kb == best && xb == at) {
        if (second) ++p1;
        else ++p0;
      }
      if (lane == 0) {
        const bool there = best > kKeyNone && !sh_bad;
        a.top_ids[(size_t)t * a.k + r] = there ? (int32_t)at : -1;
        a.top_logp[(size_t)t * a.k + r] = there ? logp_of(of_key(best)) : sh_bad ? nan : -INFINITY;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: a block takes kThreads * kChunk logits of one row.
// ---------------------------------------------------------------------------
struct BwdArgs {
  const void* z;
  const int32_t* ids;
  const float *lse, *ent, *g_logp, *g_ent;
  void* dz;
  int T, V, ld, ldd;
  float c;
};

template <bool BF16, bool OBF16, bool VEC>
__global__ void __launch_bounds__(kThreads) token_logprobs_bwd_kernel(BwdArgs a) {
  constexpr int esz = BF16 ? 2 : 4;
  constexpr int W = 8;  // logits a thread holds at a time: 8 neighbours
  for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
    const int id = a.ids[t];
    const bool off = id < 0 || id >= a.V;
    const float l = off ? 0.f : a.lse[t];
    // a row without any finite logit has no gradient; a NaN row's is NaN
    const bool zero = off || l == -INFINITY;
    const float gl = zero || !a.g_logp ? 0.f : a.g_logp[t];
    const float ge = zero || !a.g_ent ? 0.f : a.g_ent[t];
    const float h = zero || !a.ent ? 0.f : a.ent[t];
    // dz = c (gl [j = t] - p (gl + ge (log p + H)))
    const float k0 = -a.c * (gl + ge * h), k1 = -a.c * ge;
    const uint8_t* zr = (const uint8_t*)a.z + (size_t)t * a.ld * esz;
    uint8_t* dr = (uint8_t*)a.dz + (size_t)t * a.ldd * (OBF16 ? 2 : 4);
    for (int j = (blockIdx.x * kThreads + (int)threadIdx.x) * W; j < a.V; j += gridDim.x * kThreads * W) {
      float z[W], g[W];
      const bool whole = VEC && j + W <= a.V;
      if (zero) {
#pragma unroll
        for (int i = 0; i < W; ++i) g[i] = 0.f;
      } else {
        if (whole) {
          const uint4* p = (const uint4*)(zr + (size_t)j * esz);
          spread<BF16>(__ldcs(p), z);
          if (!BF16) spread<BF16>(__ldcs(p + 1), z + 4);
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i)
            z[i] = j + i < a.V ? (BF16 ? bf2f(((const uint16_t*)zr)[j + i]) : ((const float*)zr)[j + i]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float d = fmaf(z[i], a.c, -l), p = ex2(d * kLog2e);  // log p, p
          g[i] = p * fmaf(k1, fmaxf(d, kFar), k0);
          if (j + i == id) g[i] += a.c * gl;
        }
      }
      if (whole) {
        if (OBF16) {
          __stcs((uint4*)(dr + (size_t)j * 2), make_uint4(pack_bf2(g[0], g[1]), pack_bf2(g[2], g[3]),
                                                          pack_bf2(g[4], g[5]), pack_bf2(g[6], g[7])));
        } else {
          __stcs((float4*)(dr + (size_t)j * 4), make_float4(g[0], g[1], g[2], g[3]));
          __stcs((float4*)(dr + (size_t)j * 4) + 1, make_float4(g[4], g[5], g[6], g[7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (j + i < a.V) {
            if (OBF16) ((uint16_t*)dr)[j + i] = f2bf(g[i]);
            else ((float*)dr)[j + i] = g[i];
          }
      }
    }
  }
}

inline bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

int token_logprobs(const void* z, bool bf16, const int32_t* ids, float c, int k, float* lse, float* logp, float* ent,
                   int32_t* top_ids, float* top_logp, int T, int V, int ld, cudaStream_t st) {
  if (T <= 0 || V <= 0 || ld < V || k < 0 || k > kMaxTop || k > V || !(c >= 1e-30f) || !(c <= 1e30f) ||
      ((uintptr_t)z & (bf16 ? 1 : 3)) || T > (1 << 28))
    return -1;
  // Blocks a row: enough that the rows fill the GPU twice over, while a block
  // keeps at least four chunks a thread.
  int C = 1;
  while (C < kMaxCluster && (int64_t)T * C < 2 * mt_host::num_sms() && V >= 2 * C * kThreads * kChunk) C *= 2;
  FwdArgs a{z, ids, lse, logp, ent, top_logp, top_ids, T, V, ld, k, c};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(T * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  cudaError_t e;
  if (k > 0)
    e = bf16 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<true, true>, a, C)
             : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<false, true>, a, C);
  else
    e = bf16 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<true, false>, a, C)
             : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<false, false>, a, C);
  count_launches(1);
  return e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int token_logprobs_bwd(const void* z, bool bf16, const int32_t* ids, float c, const float* lse, const float* ent,
                       const float* g_logp, const float* g_ent, void* dz, bool dz_bf16, int T, int V, int ld, int ldd,
                       cudaStream_t st) {
  if (T <= 0 || V <= 0 || ld < V || ldd < V || V > (1 << 30) || !(c >= 1e-30f) || !(c <= 1e30f) || (g_ent && !ent) ||
      ((uintptr_t)z & (bf16 ? 1 : 3)) || ((uintptr_t)dz & (dz_bf16 ? 1 : 3)))
    return -1;
  BwdArgs a{z, ids, lse, ent, g_logp, g_ent, dz, T, V, ld, ldd, c};
  const bool vec = al16(z) && al16(dz) && ld % (bf16 ? 8 : 4) == 0 && ldd % (dz_bf16 ? 8 : 4) == 0;
  const dim3 grid((unsigned)std::min((V + kThreads * 16 - 1) / (kThreads * 16), 65535), (unsigned)std::min(T, 65535));
  auto go = [&](auto k) { k<<<grid, kThreads, 0, st>>>(a); };
  auto pick = [&](auto v) {
    constexpr bool X = decltype(v)::value;
    if (bf16) dz_bf16 ? go(token_logprobs_bwd_kernel<true, true, X>) : go(token_logprobs_bwd_kernel<true, false, X>);
    else dz_bf16 ? go(token_logprobs_bwd_kernel<false, true, X>) : go(token_logprobs_bwd_kernel<false, false, X>);
  };
  if (vec) pick(std::true_type());
  else pick(std::false_type());
  count_launches(1);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mt
