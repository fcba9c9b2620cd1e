// The norm after a block, the block's gate, the scaled residual and the norm
// before the next block, as one pass over a row:
//
//   ra = 1 / rms(y),  u = w_post y ra,  x' = alpha x + sigmoid(s) u
//   rb = 1 / rms(x'), n = w_pre x' rb
//
// and backward from dn and the residual's own gradient dres:
//
//   d  = dres + rb (dn w_pre - x^ mean(dn w_pre x^)),  x^ = x' rb
//   dx = alpha d,  ds = d u sigmoid' (s),  k = d sigmoid(s)
//   dy = ra (k w_post - y^ mean(k w_post y^)),  y^ = y ra
//   dw_post = sum_t k y^,  dw_pre = sum_t dn x^
//
// HBM bounds both: forward 14 bytes a value (bf16 y and s), backward 24.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mt {

MT_DEVICE_ERROR_READER(sandwich_norm_take_device_error)

namespace {

// sigmoid by the hardware's exponential and reciprocal; below 2^-126 it is 0
__device__ __forceinline__ float sigmoid_of(float e) {  // e = e^-s
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float sigmoid(float s) { return sigmoid_of(__expf(-s)); }
// and 1 - sigmoid, from the exponential where it is the small one of the two
// (the difference of 1 and a rounded sigmoid is 0 from s = 17 on)
__device__ __forceinline__ float sigmoid(float s, float& rest) {
  const float e = __expf(-s), r = sigmoid_of(e);
  rest = e <= 1.f ? e * r : 1.f - r;
  return r;
}

// Four values of a row as they are stored, and as floats.
template <bool BF16>
struct Raw4;
template <>
struct Raw4<true> {
  uint2 w;
};
template <>
struct Raw4<false> {
  float4 w;
};
template <bool BF16>
__device__ __forceinline__ Raw4<BF16> fetch4(const void* row, int unit) {
  Raw4<BF16> r;
  if constexpr (BF16) r.w = ((const uint2*)row)[unit];
  else r.w = ((const float4*)row)[unit];
  return r;
}
template <bool BF16>
__device__ __forceinline__ float4 value4(const Raw4<BF16>& r) {
  if constexpr (BF16)
    return make_float4(bf2f(r.w.x & 0xffff), bf2f(r.w.x >> 16), bf2f(r.w.y & 0xffff), bf2f(r.w.y >> 16));
  else
    return r.w;
}
template <bool BF16>
__device__ __forceinline__ void put4(void* row, int unit, float4 v) {
  if constexpr (BF16) ((uint2*)row)[unit] = make_uint2(pack_bf2(v.x, v.y), pack_bf2(v.z, v.w));
  else ((float4*)row)[unit] = v;
}
template <bool BF16>
__device__ __forceinline__ char* row_of(const void* p, size_t t, int h) {
  return (char*)p + t * h * (BF16 ? 2 : 4);
}

// Sum over the block; red: one float a warp, a buffer of its own each call.
__device__ __forceinline__ float block_sum(float v, float* red, int nw) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f);
}

__device__ __forceinline__ float squares(float4 v) {
  return fmaf(v.w, v.w, fmaf(v.z, v.z, fmaf(v.y, v.y, v.x * v.x)));
}
// The sum over a row of a thread's G sums. Each goes through its warp by
// itself: with one group a thread or two, up to 32 warps' worth of groups are
// added up in the same order, so that a row's bits do not depend on which.
template <int G>
__device__ __forceinline__ float row_sum(const float (&v)[G], float* red, int nw) {
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float s = warp_sum(v[j]);
    if ((threadIdx.x & 31) == 0) red[j * nw + (threadIdx.x >> 5)] = s;
  }
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < G * nw ? red[threadIdx.x & 31] : 0.f);
}

// One block a row, the row in registers: V groups of four values a thread.
// 8192 x 4096, bf16 y and gate (floor 70.3 us): V = 2 70.1 us, V = 1 89.7,
// V = 4 81.2 with a thread's groups added up before its warp's; apart, as here,
// 1.7 % more with V = 2. Wider rows take V = 4, with a bf16 gate three blocks an
// SM (4095 x 5636: 53.7 us, 58.7 with two; without a gate 51.5 against 49.7),
// at the price of 24 bytes spilled.
template <bool BF16, bool GATE, int V>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, V == 4 && GATE && BF16 ? 3 : 1)
    sandwich_fwd_kernel(const float* x, const void* y, const void* gate, const float* w_post, const float* w_pre,
                        float alpha, float eps, float* x_out, uint16_t* n_out, float* rstd_post, float* rstd_pre,
                        int h) {
  __shared__ float red[2][32];
  grid_wait();
  grid_release();
  const int tid = threadIdx.x, NT = blockDim.x, nw = NT >> 5, n4 = h >> 2;
  const size_t t = blockIdx.x;
  const float inv_h = 1.f / (float)h;
  float4 xv[V];
  Raw4<BF16> yr[V], sr[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    if (i < n4) {
      yr[j] = fetch4<BF16>(row_of<BF16>(y, t, h), i);
      if (GATE) sr[j] = fetch4<BF16>(row_of<BF16>(gate, t, h), i);
      xv[j] = ((const float4*)(x + t * h))[i];
    }
  }
  constexpr int G = V > 2 ? 1 : V;
  float sum[G] = {};
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (tid + j * NT < n4) sum[j % G] += squares(value4<BF16>(yr[j]));
  const float ra = rsqrtf(row_sum(sum, red[0], nw) * inv_h + eps);
#pragma unroll
  for (int j = 0; j < G; ++j) sum[j] = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    if (i < n4) {
      const float4 w = ((const float4*)w_post)[i], v = value4<BF16>(yr[j]);
      float4 u = make_float4(v.x * ra * w.x, v.y * ra * w.y, v.z * ra * w.z, v.w * ra * w.w);
      if (GATE) {
        const float4 s = value4<BF16>(sr[j]);
        u.x *= sigmoid(s.x), u.y *= sigmoid(s.y), u.z *= sigmoid(s.z), u.w *= sigmoid(s.w);
      }
      float4& o = xv[j];
      o.x = fmaf(alpha, o.x, u.x), o.y = fmaf(alpha, o.y, u.y), o.z = fmaf(alpha, o.z, u.z), o.w = fmaf(alpha, o.w, u.w);
      ((float4*)(x_out + t * h))[i] = o;
      sum[j % G] += squares(o);
    }
  }
  const float rb = rsqrtf(row_sum(sum, red[1], nw) * inv_h + eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    if (i < n4) {
      const float4 w = ((const float4*)w_pre)[i], o = xv[j];
      put4<true>(row_of<true>(n_out, t, h), i, make_float4(o.x * rb * w.x, o.y * rb * w.y, o.z * rb * w.z, o.w * rb * w.w));
    }
  }
  if (tid == 0) {
    rstd_post[t] = ra;
    rstd_pre[t] = rb;
  }
}

// ---------------------------------------------------------------------------
// Backward: blocks take rows in turn (row t belongs to part t mod parts, so a
// part's sums have a fixed order) and hold their shares of both weights'
// gradients, and the weights, in registers. One thread requests whole rows of
// x', dn and dres stages - 1 rows ahead as bulk copies into shared memory;
// y and s, whose rows need not be whole 16-byte pieces, are loaded one row
// ahead. A row has two sums, one after the other.
// A thread has V groups of four columns. One up to 4096 columns (8192 x 4096,
// bf16 and gate, floor 120.5 us: 129). Up to 6144 two with up to 768 threads,
// three with up to 512 where there is a gate: more threads leave too few
// registers (4095 x 5636 fp32 without a gate, floor 82.9: 109 us spilling at
// the bound of 1024 threads, 87 at 768; bf16 with a gate 127, 102 and, with
// three, 92; fp32 with a gate spills 32 bytes there). Up to 8192 two, spilling
// 16 to 196 bytes (2000 x 8192 with a gate, floor 58.8: 83 us; four with 512
// threads 88).
// ---------------------------------------------------------------------------
constexpr int kMaxThreads = 1024, kMaxStages = 8;
constexpr int kMaxSms = 152;  // sizes the workspace, whatever machine asks

struct BwdShape {
  int threads, vecs, stages, an_sm;
  int parts(int T, int sms) const { return std::min(T, sms * an_sm); }
};
BwdShape bwd_shape(int h, bool gate) {
  BwdShape s;
  const int n4 = h / 4;
  s.vecs = h <= 4096 ? 1 : h <= 6144 && gate ? 3 : 2;
  s.threads = std::max(32, (n4 + s.vecs * 32 - 1) / (s.vecs * 32) * 32);
  s.an_sm = h > 4096 ? 1 : std::min(8, 1024 / s.threads);
  s.stages = std::min(kMaxStages, 222 * 1024 / s.an_sm / (12 * h));
  return s;
}

__device__ __forceinline__ void bulk_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <bool BF16, bool GATE, int V, int THREADS>
__global__ void __launch_bounds__(THREADS)
    sandwich_bwd_kernel(const float* x_out, const void* y, const void* gate, const float* w_post, const float* w_pre,
                        float alpha, const float* rstd_post, const float* rstd_pre, const float* dn, const float* dres,
                        float* dx, void* dy, void* dgate, float* part, int T, int h, int stages) {
  extern __shared__ __align__(128) uint8_t stage[];  // [stages]: x', dn, dres of a row
  __shared__ float red[4][kMaxThreads / 32];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_flag;
  const int n4 = h >> 2, tid = threadIdx.x, NT = blockDim.x, nw = NT >> 5;
  const float inv_h = 1.f / (float)h;
  const uint32_t row_bytes = (uint32_t)h * (dres ? 12u : 8u);
  auto request = [&](int t, int s) {  // one thread
    if (t >= T) return;
    uint8_t* p = stage + (size_t)s * row_bytes;
    mbar_arrive_expect_tx(&full[s], row_bytes);
    bulk_row(p, x_out + (size_t)t * h, 4u * h, &full[s]);
    bulk_row(p + 4 * h, dn + (size_t)t * h, 4u * h, &full[s]);
    if (dres) bulk_row(p + 8 * h, dres + (size_t)t * h, 4u * h, &full[s]);
  };
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_wait();
  if (tid == 0)
    for (int s = 0; s < stages - 1; ++s) request(blockIdx.x + s * gridDim.x, s);
  float4 acc_post[V], acc_pre[V], wa[V], wb[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    acc_post[j] = acc_pre[j] = wa[j] = wb[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n4) {
      wa[j] = ((const float4*)w_post)[i];
      wb[j] = ((const float4*)w_pre)[i];
    }
  }
  Raw4<BF16> y_next[V], s_next[V];
  float ra_next = 0.f, rb_next = 0.f;
  auto ahead = [&](int t) {
    if (t < T) {
      ra_next = rstd_post[t];
      rb_next = rstd_pre[t];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = tid + j * NT;
        if (i < n4) {
          y_next[j] = fetch4<BF16>(row_of<BF16>(y, t, h), i);
          if (GATE) s_next[j] = fetch4<BF16>(row_of<BF16>(gate, t, h), i);
        }
      }
    }
  };
  ahead(blockIdx.x);
  int flip = 0, st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int t = blockIdx.x; t < T; t += gridDim.x, flip ^= 2) {
    const float ra = ra_next, rb = rb_next;
    Raw4<BF16> yr[V], sr[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      yr[j] = y_next[j];
      if (GATE) sr[j] = s_next[j];
    }
    ahead(t + gridDim.x);
    if (!mbar_wait(&full[st], phase, &abort_flag, kErrTimeoutTma)) break;
    const uint8_t* p = stage + (size_t)st * row_bytes;
    float4 xh[V], g[V];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        xh[j] = ((const float4*)p)[i];
        g[j] = ((const float4*)(p + 4 * h))[i];
        float4& x = xh[j];
        x.x *= rb, x.y *= rb, x.z *= rb, x.w *= rb;
        acc_pre[j].x += g[j].x * x.x, acc_pre[j].y += g[j].y * x.y, acc_pre[j].z += g[j].z * x.z, acc_pre[j].w += g[j].w * x.w;
        g[j].x *= wb[j].x, g[j].y *= wb[j].y, g[j].z *= wb[j].z, g[j].w *= wb[j].w;
        dot += g[j].x * x.x + g[j].y * x.y + g[j].z * x.z + g[j].w * x.w;
      }
    }
    // four buffers in turn: a barrier a sum is enough
    const float mb = block_sum(dot, red[flip], nw) * inv_h;
    // that barrier also says that the last row's stage has been read
    if (tid == 0) request(t + (stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
    dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        float4 d = make_float4(rb * (g[j].x - xh[j].x * mb), rb * (g[j].y - xh[j].y * mb),
                               rb * (g[j].z - xh[j].z * mb), rb * (g[j].w - xh[j].w * mb));
        if (dres) {
          const float4 e = ((const float4*)(p + 8 * h))[i];
          d.x += e.x, d.y += e.y, d.z += e.z, d.w += e.w;
        }
        ((float4*)(dx + (size_t)t * h))[i] = make_float4(alpha * d.x, alpha * d.y, alpha * d.z, alpha * d.w);
        float4 yh = value4<BF16>(yr[j]);
        yh.x *= ra, yh.y *= ra, yh.z *= ra, yh.w *= ra;
        if (GATE) {
          float4 s = value4<BF16>(sr[j]), c;
          s = make_float4(sigmoid(s.x, c.x), sigmoid(s.y, c.y), sigmoid(s.z, c.z), sigmoid(s.w, c.w));
          const float4 k = make_float4(d.x * s.x, d.y * s.y, d.z * s.z, d.w * s.w);
          put4<BF16>(row_of<BF16>(dgate, t, h), i,
                     make_float4(k.x * (yh.x * wa[j].x) * c.x, k.y * (yh.y * wa[j].y) * c.y,
                                 k.z * (yh.z * wa[j].z) * c.z, k.w * (yh.w * wa[j].w) * c.w));
          d = k;
        }
        acc_post[j].x += d.x * yh.x, acc_post[j].y += d.y * yh.y, acc_post[j].z += d.z * yh.z, acc_post[j].w += d.w * yh.w;
        g[j] = make_float4(d.x * wa[j].x, d.y * wa[j].y, d.z * wa[j].z, d.w * wa[j].w);
        xh[j] = yh;
        dot += g[j].x * yh.x + g[j].y * yh.y + g[j].z * yh.z + g[j].w * yh.w;
      }
    }
    const float ma = block_sum(dot, red[flip + 1], nw) * inv_h;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4)
        put4<BF16>(row_of<BF16>(dy, t, h), i,
                   make_float4(ra * (g[j].x - xh[j].x * ma), ra * (g[j].y - xh[j].y * ma),
                               ra * (g[j].z - xh[j].z * ma), ra * (g[j].w - xh[j].w * ma)));
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
  grid_release();
  if (*(volatile int*)&abort_flag) {  // a wait ran out: give the copies in flight time to land
    for (int k = 0; k < stages - 1; ++k) {
      for (int spin = 0; spin < (1 << 20) && !mbar_try_wait(smem_u32(&full[st]), phase); ++spin) {
      }
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    if (i < n4) {
      ((float4*)(part + (size_t)blockIdx.x * 2 * h))[i] = acc_post[j];
      ((float4*)(part + (size_t)blockIdx.x * 2 * h + h))[i] = acc_pre[j];
    }
  }
}

// Both weights' gradients: column c of [parts][2 h] summed in a fixed order,
// 32 columns a block.
__global__ void __launch_bounds__(1024) sum_both_kernel(const float* part, int nparts, int h, float* dw_post,
                                                        float* dw_pre) {
  __shared__ float red[32][33];
  grid_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * h) {
#pragma unroll 8
    for (int p = w; p < nparts; p += 32) s += part[(size_t)p * 2 * h + c];
  }
  red[w][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][w]);
  const int o = blockIdx.x * 32 + w;
  if (lane == 0 && o < 2 * h) (o < h ? dw_post + o : dw_pre + (o - h))[0] = s;
}

inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

}  // namespace

bool sandwich_norm_dims(int T, int h) {
  // a block's row counter goes up to stages rounds of the grid past T
  return T > 0 && T <= (1 << 30) && h > 0 && h % 4 == 0 && h <= 8192;
}
size_t sandwich_norm_bwd_partials(int T, int h) { return (size_t)bwd_shape(h, false).parts(T, kMaxSms) * 2 * h; }

int sandwich_norm_fwd(const float* x, const void* y, const void* gate, bool bf16, const float* w_post,
                      const float* w_pre, float alpha, float eps, float* x_out, uint16_t* n_out, float* rstd_post,
                      float* rstd_pre, int T, int h, cudaStream_t st) {
  const size_t ya = bf16 ? 8 : 16;
  if (!sandwich_norm_dims(T, h) || !al(x, 16) || !al(y, ya) || !al(gate, ya) || !al(w_post, 16) || !al(w_pre, 16) ||
      !al(x_out, 16) || !al(n_out, 8))
    return kRefused;
  const int n4 = h / 4;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k, int v) {
    const int threads = std::max(32, (n4 + v * 32 - 1) / (v * 32) * 32);
    e = mt_host::launch_early(k, T, threads, 0, st, 1, x, y, gate, w_post, w_pre, alpha, eps, x_out, n_out, rstd_post,
                              rstd_pre, h);
  };
  auto pick = [&](auto b, auto g) {
    constexpr bool B = decltype(b)::value, G = decltype(g)::value;
    // one group a thread is the shortest way through few rows; more keep more of
    // many rows in flight
    if (n4 <= 1024 && T <= kMaxSms * 2) go(sandwich_fwd_kernel<B, G, 1>, 1);
    else if (n4 <= 1024) go(sandwich_fwd_kernel<B, G, 2>, 2);
    else go(sandwich_fwd_kernel<B, G, 4>, 4);
  };
  auto pick_g = [&](auto b) { gate ? pick(b, std::true_type()) : pick(b, std::false_type()); };
  bf16 ? pick_g(std::true_type()) : pick_g(std::false_type());
  count_launches(1);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

int sandwich_norm_bwd(const float* x_out, const void* y, const void* gate, bool bf16, const float* w_post,
                      const float* w_pre, float alpha, const float* rstd_post, const float* rstd_pre, const float* dn,
                      const float* dres, float* dx, void* dy, void* dgate, float* dw_post, float* dw_pre, float* work,
                      int T, int h, cudaStream_t st) {
  const size_t ya = bf16 ? 8 : 16;
  if (!sandwich_norm_dims(T, h) || !al(x_out, 16) || !al(y, ya) || !al(gate, ya) || !al(w_post, 16) ||
      !al(w_pre, 16) || !al(dn, 16) || !al(dres, 16) || !al(dx, 16) || !al(dy, ya) || !al(dgate, ya) || !al(work, 16))
    return kRefused;
  BwdShape shape = bwd_shape(h, gate != nullptr);
  const int parts = shape.parts(T, std::min(mt_host::num_sms(), kMaxSms));
  shape.stages = std::min(shape.stages, (T + parts - 1) / parts + 1);  // no more than there are rows for
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) {
    const int smem = shape.stages * h * (dres ? 12 : 8);
    if (smem > 47 * 1024)  // with the static part past the default limit
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
    if (e == cudaSuccess)
      e = mt_host::launch_early(k, parts, shape.threads, smem, st, 1, x_out, y, gate, w_post, w_pre, alpha, rstd_post,
                                rstd_pre, dn, dres, dx, dy, dgate, work, T, h, shape.stages);
  };
  auto pick = [&](auto b, auto g) {
    constexpr bool B = decltype(b)::value, G = decltype(g)::value;
    if (shape.vecs == 1) go(sandwich_bwd_kernel<B, G, 1, 1024>);
    else if (h > 6144) go(sandwich_bwd_kernel<B, G, 2, 1024>);
    else if constexpr (G) go(sandwich_bwd_kernel<B, G, 3, 512>);
    else go(sandwich_bwd_kernel<B, G, 2, 768>);
  };
  auto pick_g = [&](auto b) { gate ? pick(b, std::true_type()) : pick(b, std::false_type()); };
  bf16 ? pick_g(std::true_type()) : pick_g(std::false_type());
  if (e == cudaSuccess)
    e = mt_host::launch_early(sum_both_kernel, (2 * h + 31) / 32, 1024, 0, st, 1, (const float*)work, parts, h, dw_post,
                              dw_pre);
  count_launches(2);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}

}  // namespace mt
