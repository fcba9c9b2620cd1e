// Activation checkpoints in 8 bits and their use in the backward pass.
//
// Block form: the columns of a row are cut into blocks of 32 (the last one
// may be shorter); a block keeps one scale 2^(b-127), its byte b, and one
// 8-bit code per value. b is the least byte with max|x| <= limit * 2^(b-127),
// limit = 127 for int8 codes (x / scale rounded to the nearest whole number)
// and 448 for e4m3 codes (x / scale rounded to e4m3), ties to even. Because
// the scale is a power of two, x / scale and code * scale are exact: the one
// rounding is the code's, and nothing ever saturates. A block that holds an
// infinity or a NaN has b = 255 and codes 0, and stands for NaN throughout
// (the same convention as the OCP microscaling formats' E8M0 scale).
//
// int8 steps evenly (error <= max|x| / 127 of the block's maximum when the
// scale is tight, twice that at worst); e4m3 keeps 2^-4 relative error down
// to 2^-14 of the block's maximum, so a block with one outlier keeps its
// other values.
//
// All kernels here are bound by HBM traffic: every operand is read once and
// every result written once, loads are 16 or 32 bytes a thread, and a
// block's maximum is a shuffle reduction over the four or eight lanes that
// hold it.
#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace mt {

MT_DEVICE_ERROR_READER(ckpt8_take_device_error)

namespace {

enum { FMT_I8 = 1, FMT_E4M3 = 2 };

// Scale byte of a block from the bit pattern of max|x| (as an unsigned
// integer it orders like the value, infinities and NaN above all numbers).
// SHIFT: fraction bits of the pattern (23, or 7 for a bf16). The exponent
// goes up by one where the fraction is past the limit's (127 = 1.984375 * 2^6,
// 448 = 1.75 * 2^8): a carry out of the fraction.
template <int FMT, int SHIFT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  constexpr int off = FMT == FMT_I8 ? 6 : 8;
  constexpr uint32_t ones = (1u << SHIFT) - 1;
  constexpr uint32_t top = FMT == FMT_I8 ? 126u << (SHIFT - 7) : 96u << (SHIFT - 7);
  const int b = max((int)((amax_bits + (ones - top)) >> SHIFT) - off, 0);
  return amax_bits >= (255u << SHIFT) ? 255u : (uint32_t)b;
}
__device__ __forceinline__ float scale_up(uint32_t b) {  // 2^(b-127); 2^-127 is subnormal
  return __uint_as_float(b == 255u ? 0x7fffffffu : b ? b << 23 : 0x00400000u);
}
// 2^(127-b), b <= 249; 0 for a block that stands for NaN, whose codes come out 0
__device__ __forceinline__ float scale_down(uint32_t b) {
  return __uint_as_float(b == 255u ? 0u : (254u - b) << 23);
}

// Four values to four code bytes. inv = 0 gives 0 even for infinities and NaN
// in int8; e4m3 clears them.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(uint64_t ab, uint64_t cd, float inv) {
  const uint64_t ii = pair(inv, inv);
  if (FMT == FMT_I8) {
    // adding 1.5 * 2^23 leaves the nearest whole number (ties to even) in the low bits
    constexpr float magic = 12582912.f;
    const uint64_t mm = pair(magic, magic), x = fma2(ab, ii, mm), y = fma2(cd, ii, mm);
    return __byte_perm(__byte_perm((uint32_t)x, (uint32_t)(x >> 32), 0x0040),
                       __byte_perm((uint32_t)y, (uint32_t)(y >> 32), 0x0040), 0x5410);
  }
  float a, b, c, d;
  unpair(mul2(ab, ii), a, b);
  unpair(mul2(cd, ii), c, d);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Four code bytes to the two pairs of values they stand for.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float s, uint64_t& ab, uint64_t& cd) {
  const uint64_t ss = pair(s, s);
  if (FMT == FMT_I8) {
    // byte + 128 in the low bits of 2^23; the subtraction is exact
    w ^= 0x80808080u;
    constexpr float bias = -8388736.f;  // -(2^23 + 128)
    const uint64_t bb = pair(bias, bias);
    ab = mul2(add2(pair(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)),
                        __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))), bb), ss);
    cd = mul2(add2(pair(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)),
                        __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443))), bb), ss);
    return;
  }
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
  const float2 l = __half22float2(*(const __half2*)&lo), h = __half22float2(*(const __half2*)&hi);
  ab = mul2(pair(l.x, l.y), ss);
  cd = mul2(pair(h.x, h.y), ss);
}
template <int FMT>
__device__ __forceinline__ float4 decode4(uint32_t w, float s) {
  uint64_t ab, cd;
  decode4<FMT>(w, s, ab, cd);
  float4 v;
  unpair(ab, v.x, v.y);
  unpair(cd, v.z, v.w);
  return v;
}

// Maximum over aligned groups of G lanes.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 32-byte accesses (one instruction for eight fp32).
__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void store8f(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Eight consecutive values of a row from column c; columns at or past n read
// as 0. VEC: one 16-byte (bf16) or 32-byte (fp32) load.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_unit(const void* row, int c, int n, float (&v)[8]) {
  if (VEC && c + 8 <= n) {
    if (BF16) {
      const uint4 u = __ldcs((const uint4*)((const uint16_t*)row + c));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      load8f((const float*)row + c, v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = c + i < n ? (BF16 ? bf2f(((const uint16_t*)row)[c + i]) : ((const float*)row)[c + i]) : 0.f;
}
// E code bytes (E / 4 words) to columns c.. of a row of codes.
template <int E, bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int n, const uint32_t (&w)[E / 4]) {
  if (VEC && c + E <= n) {
    if (E == 8) *(uint2*)(row + c) = make_uint2(w[0], w[E / 4 - 1]);
    else *(uint32_t*)(row + c) = w[0];
    return;
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (c + i < n) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}
template <int E, bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* row, int c, int n, uint32_t (&w)[E / 4]) {
  if (VEC && c + E <= n) {
    if (E == 8) {
      const uint2 u = __ldcs((const uint2*)(row + c));
      w[0] = u.x;
      w[E / 4 - 1] = u.y;
    } else {
      w[0] = __ldcs((const uint32_t*)(row + c));
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < E / 4; ++k) w[k] = 0;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (c + i < n) w[i >> 2] |= (uint32_t)row[c + i] << (8 * (i & 3));
}

// Codes of one thread's E values under a block's scale byte.
template <int FMT, int E>
__device__ __forceinline__ void encode_unit(uint32_t b, const float (&v)[E], uint32_t (&w)[E / 4]) {
  const float inv = scale_down(b);
#pragma unroll
  for (int k = 0; k < E / 4; ++k) {
    w[k] = encode4<FMT>(pair(v[4 * k], v[4 * k + 1]), pair(v[4 * k + 2], v[4 * k + 3]), inv);
    if (b == 255u) w[k] = 0;
  }
}
// Scale byte of the block that G lanes hold, from each lane's E values.
template <int FMT, int E>
__device__ __forceinline__ uint32_t block_byte(const float (&v)[E]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < E; i += 2) m = max3_nan(m, fabsf(v[i]), fabsf(v[i + 1]));
  return scale_byte<FMT, 23>(group_max<32 / E>(__float_as_uint(m)));
}
// Larger of each half's magnitudes over eight bf16 (magnitudes order like
// whole numbers, two at a time).
__device__ __forceinline__ uint32_t amax_bf16x8(const uint4& u) {
  constexpr uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vimax3_u16x2(u.x & m, u.y & m, u.z & m), u.w & m);
}

// ---------------------------------------------------------------------------
// Pack and unpack. A thread owns one unit of eight values in each of kRows
// rows (their loads are in flight together); a 2D block covers blockDim.x
// units of blockDim.y rows at a time, so narrow matrices still fill a block.
// ---------------------------------------------------------------------------
constexpr int kRows = 4;

template <int FMT, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_pack_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales, int T, int n, int ldx, int ldc,
                                                         int nb) {
  constexpr int E = 8, G = 32 / E, esz = BF16 ? 2 : 4;
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * E;
  const int step = gridDim.y * blockDim.y;
  // the whole block leaves the loop together: shuffles need every lane
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kRows) {
    float v[kRows][E];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      load_unit<BF16, VEC>((const uint8_t*)x + (size_t)t * ldx * esz, c, t < T ? n : 0, v[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      uint32_t w[E / 4];
      const uint32_t b = block_byte<FMT, E>(v[r]);
      encode_unit<FMT, E>(b, v[r], w);
      if (t < T) {
        store_codes<E, VEC>(codes + (size_t)t * ldc, c, n, w);
        if ((threadIdx.x & (G - 1)) == 0 && c < n) scales[(size_t)t * nb + c / 32] = (uint8_t)b;
      }
    }
  }
}

template <int FMT, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_unpack_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, void* __restrict__ x,
                                                           int T, int n, int ldc, int ldx, int nb) {
  constexpr int E = 8;
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * E;
  if (c >= n) return;
  const int step = gridDim.y * blockDim.y;
  for (int t0 = blockIdx.y * blockDim.y + threadIdx.y; t0 < T; t0 += step * kRows) {
    uint32_t w[kRows][E / 4];
    uint32_t b[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step;
      if (t < T) {
        load_codes<E, VEC>(codes + (size_t)t * ldc, c, n, w[r]);
        b[r] = scales[(size_t)t * nb + c / 32];
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step;
      if (t >= T) break;
      const float s = scale_up(b[r]);
      float v[E];
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        const float4 f = decode4<FMT>(w[r][k], s);
        v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
      }
      if (BF16) {
        uint16_t* dst = (uint16_t*)x + (size_t)t * ldx + c;
        if (VEC && c + E <= n) {
          *(uint4*)dst = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[E - 4], v[E - 3]),
                                    pack_bf2(v[E - 2], v[E - 1]));
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (c + i < n) dst[i] = f2bf(v[i]);
        }
      } else {
        float* dst = (float*)x + (size_t)t * ldx + c;
        if (VEC && c + E <= n) {
          store8f(dst, v);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (c + i < n) dst[i] = v[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// RMSNorm forward that keeps its input: one pass over x writes y, rstd and
// the 8-bit block form (7 bytes a value instead of the 6 of the plain
// forward). A block per row; a thread holds V units of eight columns of the
// row in registers, four neighbouring lanes hold a block of 32 columns.
// ---------------------------------------------------------------------------
// Measured at 8192 x 4096 (floor 34.5 us): 256 threads 37.8 us, 128 threads
// 38.9, four columns a unit 41.2.
template <int FMT, int NT, int V, bool VEC>
__global__ void __launch_bounds__(NT)
    rmsnorm_fwd_ckpt8_kernel(const float* __restrict__ x, const float* __restrict__ w, uint16_t* __restrict__ y,
                             float* __restrict__ rstd, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                             int h, int nb, float eps) {
  __shared__ float red[NT / 32];
  const size_t t = blockIdx.x;
  const float* xr = x + t * h;
  const int tid = threadIdx.x;
  float v[V][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) load_unit<false, VEC>(xr, (tid + k * NT) * 8, h, v[k]);
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      ss += v[k][i] * v[k][i] + v[k][i + 1] * v[k][i + 1] + v[k][i + 2] * v[k][i + 2] + v[k][i + 3] * v[k][i + 3];
  ss = warp_sum(ss);
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  // the checkpoint does not need the norm: its stores go out during the reduction
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (tid + k * NT) * 8;
    uint32_t q[2];
    const uint32_t b = block_byte<FMT, 8>(v[k]);
    encode_unit<FMT, 8>(b, v[k], q);
    if (c < h) {
      store_codes<8, VEC>(codes + t * h, c, h, q);
      if ((tid & 3) == 0) scales[t * nb + c / 32] = (uint8_t)b;
    }
  }
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) ss += red[i];
  const float r = rsqrtf(ss / (float)h + eps);
  if (tid == 0) rstd[t] = r;
  uint16_t* yr = y + t * h;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (tid + k * NT) * 8;
    float g[8];
    uint32_t o[4];
    if (VEC && c + 8 <= h) {
      const float4 g0 = *(const float4*)(w + c), g1 = *(const float4*)(w + c + 4);
      g[0] = g0.x, g[1] = g0.y, g[2] = g0.z, g[3] = g0.w, g[4] = g1.x, g[5] = g1.y, g[6] = g1.z, g[7] = g1.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = c + i < h ? w[c + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf2(v[k][2 * i] * r * g[2 * i], v[k][2 * i + 1] * r * g[2 * i + 1]);
    if (VEC && c + 8 <= h) {
      *(uint4*)(yr + c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < h) yr[c + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// RMSNorm backward that reads its input from the 8-bit form:
//   xh = x' rstd, dx = resid + rstd (dy w - xh mean(dy w xh)), dw = sum_t dy xh,
// x' the checkpoint's values. Blocks take rows in turn (row t belongs to part
// t mod parts, so a part's sum has a fixed order) and hold their share of dw
// in registers; a second kernel adds the parts in order.
// ---------------------------------------------------------------------------
// A block holds a row: V float4 a thread (two where h > 4096), w and the
// sums of dw in registers. One thread requests whole rows of codes, dy and
// resid stages - 1 rows ahead as bulk copies into shared memory, so loads
// stay in flight across a row's reduction and hold no registers; rows that
// are not whole 16-byte pieces (BULK false) are loaded by the threads.
// Measured at 8192 x 4096 (504 MB, floor 74 us) with the sum of the parts:
// per-thread loads 103 us, per-thread cp.async staging 128 us (its 4-byte
// copies and second reads cost more than the loads it hides), bulk copies
// with two blocks an SM and three stages 87 us, one block and five 82 us.
// ---------------------------------------------------------------------------
constexpr int kBwdMaxThreads = 1024;
constexpr int kBwdMaxStages = 8;

struct BwdShape {
  int threads, vecs, stages, parts;
};
// 1024 threads an SM where the rows allow, the shared memory shared out among
// their blocks as stages of 9 h bytes (5 h without a residual).
BwdShape bwd_shape(int T, int h) {
  BwdShape s;
  const int n4 = h / 4;
  s.vecs = h > 4096 ? 2 : 1;
  s.threads = std::max(32, (n4 + s.vecs * 32 - 1) / (s.vecs * 32) * 32);
  const int an_sm = std::min(8, 1024 / s.threads);
  s.stages = std::min(kBwdMaxStages, 222 * 1024 / an_sm / (9 * h));
  s.parts = std::min(T, 152 * an_sm);
  return s;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int FMT, int V, bool BULK>
__global__ void __launch_bounds__(kBwdMaxThreads)
    rmsnorm_bwd_ckpt8_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                             const float* __restrict__ w, const float* __restrict__ rstd,
                             const float* __restrict__ dy, const float* resid, float* dx, uint16_t* __restrict__ dxb,
                             float* __restrict__ part, int T, int h, int nb, int stages) {
  extern __shared__ __align__(128) uint8_t stage[];  // [stages]: dy, resid, codes of a row
  __shared__ float red[2][kBwdMaxThreads / 32];
  __shared__ uint64_t full[kBwdMaxStages];
  __shared__ int abort_flag;
  const int n4 = h >> 2, tid = threadIdx.x, NT = blockDim.x, nw = NT >> 5;
  const float inv_h = 1.f / (float)h;
  const uint32_t row_bytes = (uint32_t)h * (resid ? 9u : 5u);
  auto request = [&](int t, int s) {  // one thread
    if (t >= T) return;
    uint8_t* p = stage + (size_t)s * row_bytes;
    mbar_arrive_expect_tx(&full[s], row_bytes);
    bulk_load(p, dy + (size_t)t * h, 4u * h, &full[s]);
    if (resid) bulk_load(p + 4 * h, resid + (size_t)t * h, 4u * h, &full[s]);
    bulk_load(p + row_bytes - h, codes + (size_t)t * h, (uint32_t)h, &full[s]);
  };
  if (BULK) {
    if (tid == 0) {
      abort_flag = 0;
      for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
      fence_barrier_init();
    }
    __syncthreads();
    if (tid == 0)
      for (int s = 0; s < stages - 1; ++s) request(blockIdx.x + s * gridDim.x, s);
  }
  float4 acc[V], wv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    wv[j] = i < n4 ? ((const float4*)w)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // a row's scales and rstd, requested one row ahead
  uint32_t b_next[V];
  float r_next = 0.f;
  auto small = [&](int t) {
    if (t < T) {
      r_next = rstd[t];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = tid + j * NT;
        if (i < n4) b_next[j] = scales[(size_t)t * nb + i / 8];
      }
    }
  };
  small(blockIdx.x);
  int flip = 0, st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
    const float r = r_next;
    float4 g[V], e[V], x[V];
    uint32_t q[V];
    if (BULK) {
      if (!mbar_wait(&full[st], phase, &abort_flag, kErrTimeoutTma)) break;
    }
    const uint8_t* p = stage + (size_t)st * row_bytes;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        if (BULK) {
          g[j] = ((const float4*)p)[i];
          q[j] = ((const uint32_t*)(p + row_bytes - h))[i];
        } else {
          g[j] = __ldcs((const float4*)(dy + (size_t)t * h) + i);
          q[j] = __ldcs((const uint32_t*)(codes + (size_t)t * h) + i);
          if (resid) e[j] = ((const float4*)(resid + (size_t)t * h))[i];
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        x[j] = decode4<FMT>(q[j], scale_up(b_next[j]));
        dot += g[j].x * wv[j].x * x[j].x + g[j].y * wv[j].y * x[j].y + g[j].z * wv[j].z * x[j].z +
               g[j].w * wv[j].w * x[j].w;
      }
    }
    small(t + gridDim.x);
    dot = warp_sum(dot);
    if ((tid & 31) == 0) red[flip][tid >> 5] = dot;
    // two buffers in turn: one barrier a row is enough; it also says that the
    // last row's stage has been read
    __syncthreads();
    if (BULK && tid == 0) request(t + (stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
    dot = (tid & 31) < nw ? red[flip][tid & 31] : 0.f;
    const float mean = warp_sum(dot) * r * inv_h;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        const float4 xh = make_float4(x[j].x * r, x[j].y * r, x[j].z * r, x[j].w * r);
        float4 o = make_float4(r * (g[j].x * wv[j].x - xh.x * mean), r * (g[j].y * wv[j].y - xh.y * mean),
                               r * (g[j].z * wv[j].z - xh.z * mean), r * (g[j].w * wv[j].w - xh.w * mean));
        if (resid) {
          if (BULK) e[j] = ((const float4*)(p + 4 * h))[i];
          o.x += e[j].x;
          o.y += e[j].y;
          o.z += e[j].z;
          o.w += e[j].w;
        }
        ((float4*)(dx + (size_t)t * h))[i] = o;
        if (dxb) ((uint2*)(dxb + (size_t)t * h))[i] = make_uint2(pack_bf2(o.x, o.y), pack_bf2(o.z, o.w));
        acc[j].x += g[j].x * xh.x;
        acc[j].y += g[j].y * xh.y;
        acc[j].z += g[j].z * xh.z;
        acc[j].w += g[j].w * xh.w;
      }
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (BULK && *(volatile int*)&abort_flag) {  // a wait ran out: give the copies in flight time to land
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
    if (i < n4) ((float4*)(part + (size_t)blockIdx.x * h))[i] = acc[j];
  }
}

// out[c] = sum over the parts, in a fixed order: 32 warps take the parts in
// turn for 32 columns, then their sums are added by a shuffle tree.
// Launched while the kernel that writes the parts still runs (it waits for
// that kernel's end here), so its own launch costs nothing.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* part, int nparts, int n,
                                                         float* __restrict__ out) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int p = w; p < nparts; p += 32) s += part[(size_t)p * n + c];
  }
  red[w][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][w]);  // warp w: column w of the 32
  if (lane == 0 && blockIdx.x * 32 + w < n) out[blockIdx.x * 32 + w] = s;
}

// ---------------------------------------------------------------------------
// SwiGLU forward and backward around an 8-bit g|u. Columns of g and of u are
// cut into blocks of 32 separately. A thread owns 8 columns of g and the
// same 8 of u, four lanes a block.
// ---------------------------------------------------------------------------
// 1 / (1 + e^-g) of two values with the hardware's exponential and
// reciprocal (the exact division and the subnormal range of both cost more
// instructions than the rest of the formula): results below 2^-126 are 0.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  constexpr float k = -1.4426950408889634f;
  float a, b;
  unpair(mul2(g, pair(k, k)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  unpair(add2(pair(a, b), pair(1.f, 1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pair(a, b);
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  unpair(v, a, b);
  return pack_bf2(a, b);
}
__device__ __forceinline__ void spread8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Eight bf16 from column c; columns at or past n read as 0.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int n) {
  if (VEC && c + 8 <= n) return __ldcs((const uint4*)(row + c));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
constexpr int kSwRows = 2;

template <int FMT, bool VEC>
__global__ void __launch_bounds__(256, 5) swiglu_fwd_ckpt8_kernel(const uint16_t* __restrict__ gu,
                                                               uint16_t* __restrict__ act,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, int T, int F, int ld,
                                                               int nb) {
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const int step = gridDim.y * blockDim.y;
  // the whole block leaves the loop together: shuffles need every lane
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kSwRows) {
    uint4 gq[kSwRows], uq[kSwRows];
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const uint16_t* row = gu + (size_t)t * 2 * ld;
      gq[r] = load8<VEC>(row, c, t < T ? F : 0);
      uq[r] = load8<VEC>(row + ld, c, t < T ? F : 0);
    }
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      // the maxima of g and u, a half of a word each, go through the shuffles together
      const uint32_t mg = amax_bf16x8(gq[r]), mu = amax_bf16x8(uq[r]);
      uint32_t m = __vmaxu2(__byte_perm(mg, mu, 0x5410), __byte_perm(mg, mu, 0x7632));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      float g[8], u[8];
      spread8(gq[r], g);
      spread8(uq[r], u);
      uint32_t wg[2], wu[2];
      const uint32_t bg = scale_byte<FMT, 7>(m & 0xffffu), bu = scale_byte<FMT, 7>(m >> 16);
      encode_unit<FMT, 8>(bg, g, wg);
      encode_unit<FMT, 8>(bu, u, wu);
      if (t < T) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t g2 = pair(g[2 * i], g[2 * i + 1]), u2 = pair(u[2 * i], u[2 * i + 1]);
          a[i] = pack_pair(mul2(mul2(g2, sigmoid2(g2)), u2));
        }
        uint8_t* crow = codes + (size_t)t * 2 * ld;
        uint16_t* arow = act + (size_t)t * ld;
        // columns F..ld-1 are padding: codes and act are 0 there (the loads gave 0)
        store_codes<8, VEC>(crow, c, ld, wg);
        store_codes<8, VEC>(crow + ld, c, ld, wu);
        if (VEC && c + 8 <= ld) {
          *(uint4*)(arow + c) = make_uint4(a[0], a[1], a[2], a[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < ld) arow[c + i] = (uint16_t)(a[i >> 1] >> (16 * (i & 1)));
        }
        if ((threadIdx.x & 3) == 0 && c < F) {
          scales[(size_t)t * 2 * nb + c / 32] = (uint8_t)bg;
          scales[(size_t)t * 2 * nb + nb + c / 32] = (uint8_t)bu;
        }
      }
    }
  }
}

// dg = dact u silu'(g), du = dact silu(g), with g and u from the 8-bit form.
template <int FMT, bool VEC>
__global__ void __launch_bounds__(256) swiglu_bwd_ckpt8_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales,
                                                               const uint16_t* __restrict__ dact,
                                                               uint16_t* __restrict__ dgu, int T, int F, int ld,
                                                               int nb) {
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (c >= ld) return;
  const int step = gridDim.y * blockDim.y;
  for (int t0 = blockIdx.y * blockDim.y + threadIdx.y; t0 < T; t0 += step * kSwRows) {
    uint32_t wg[kSwRows][2], wu[kSwRows][2], bg[kSwRows], bu[kSwRows];
    uint4 dq[kSwRows];
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step;
      if (t < T) {
        const uint8_t* crow = codes + (size_t)t * 2 * ld;
        load_codes<8, VEC>(crow, c, F, wg[r]);
        load_codes<8, VEC>(crow + ld, c, F, wu[r]);
        dq[r] = load8<VEC>(dact + (size_t)t * ld, c, F);
        // a unit that lies in the padding has no block of its own
        bg[r] = c < F ? scales[(size_t)t * 2 * nb + c / 32] : 0u;
        bu[r] = c < F ? scales[(size_t)t * 2 * nb + nb + c / 32] : 0u;
      }
    }
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step;
      if (t >= T) break;
      const float sg = scale_up(bg[r]), su = scale_up(bu[r]);
      float d[8];
      spread8(dq[r], d);
      uint32_t og[4], ou[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint64_t g2[2], u2[2];
        decode4<FMT>(wg[r][k], sg, g2[0], g2[1]);
        decode4<FMT>(wu[r][k], su, u2[0], u2[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = 4 * k + 2 * i;
          const uint64_t s = sigmoid2(g2[i]), ds = mul2(pair(d[e], d[e + 1]), s), du = mul2(ds, g2[i]);
          // dact u s (1 + g (1 - s)); dact g s
          const uint64_t rest = fma2(s, pair(-1.f, -1.f), pair(1.f, 1.f));
          og[2 * k + i] = pack_pair(mul2(u2[i], fma2(du, rest, ds)));
          ou[2 * k + i] = pack_pair(du);
        }
      }
      uint16_t* row = dgu + (size_t)t * 2 * ld;
      if (VEC && c + 8 <= F) {
        *(uint4*)(row + c) = make_uint4(og[0], og[1], og[2], og[3]);
        *(uint4*)(row + ld + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < ld) {  // padding columns carry no gradient
            row[c + i] = c + i < F ? (uint16_t)(og[i >> 1] >> (16 * (i & 1))) : (uint16_t)0;
            row[ld + c + i] = c + i < F ? (uint16_t)(ou[i >> 1] >> (16 * (i & 1))) : (uint16_t)0;
          }
      }
    }
  }
}

// Block and grid of the 2D kernels: units of 8 columns along x, rows along y.
struct Shape2 {
  dim3 grid, block;
};
Shape2 shape2(int T, int units, int rows) {
  int bx = 8;
  while (bx < units && bx < 256) bx *= 2;
  // narrower blocks where the last one along a row would idle by a quarter or more
  while (bx > 32 && (units + bx - 1) / bx * bx - units >= units / 4) bx /= 2;
  const int by = 256 / bx;
  const int gy = (T + by * rows - 1) / (by * rows);
  return {dim3((unsigned)((units + bx - 1) / bx), (unsigned)std::min(gy, 65535)), dim3((unsigned)bx, (unsigned)by)};
}

inline int blocks32(int n) { return (n + 31) / 32; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int done(int launches) {
  count_launches(launches);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}
// Sizes: row and column counters stay within 31 bits with room for a grid's step.
inline bool dims_ok(int T, int n, int ld) { return T > 0 && n > 0 && ld >= n && T <= (1 << 30) && ld <= (1 << 29); }
inline bool fmt_ok(int fmt) { return fmt == FMT_I8 || fmt == FMT_E4M3; }

}  // namespace

int ckpt8_pack(const void* x, bool bf16, int fmt, uint8_t* codes, uint8_t* scales, int T, int n, int ldx, int ldc,
               cudaStream_t st) {
  if (!dims_ok(T, n, ldx) || !dims_ok(T, n, ldc) || !fmt_ok(fmt) || !al(x, bf16 ? 2 : 4)) return -1;
  const int nb = blocks32(n);
  const Shape2 s = shape2(T, (n + 7) / 8, kRows);
  // whole loads and stores of eight values where every row starts on their boundary
  const bool vec = al(x, bf16 ? 16 : 32) && ldx % 8 == 0 && al(codes, 8) && ldc % 8 == 0;
  auto go = [&](auto k) { k<<<s.grid, s.block, 0, st>>>(x, codes, scales, T, n, ldx, ldc, nb); };
  if (fmt == FMT_I8) {
    if (bf16) vec ? go(ckpt8_pack_kernel<FMT_I8, true, true>) : go(ckpt8_pack_kernel<FMT_I8, true, false>);
    else vec ? go(ckpt8_pack_kernel<FMT_I8, false, true>) : go(ckpt8_pack_kernel<FMT_I8, false, false>);
  } else {
    if (bf16) vec ? go(ckpt8_pack_kernel<FMT_E4M3, true, true>) : go(ckpt8_pack_kernel<FMT_E4M3, true, false>);
    else vec ? go(ckpt8_pack_kernel<FMT_E4M3, false, true>) : go(ckpt8_pack_kernel<FMT_E4M3, false, false>);
  }
  return done(1);
}

int ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int fmt, void* x, bool bf16, int T, int n, int ldc,
                 int ldx, cudaStream_t st) {
  if (!dims_ok(T, n, ldx) || !dims_ok(T, n, ldc) || !fmt_ok(fmt) || !al(x, bf16 ? 2 : 4)) return -1;
  const int nb = blocks32(n);
  const Shape2 s = shape2(T, (n + 7) / 8, kRows);
  const bool vec = al(x, bf16 ? 16 : 32) && ldx % 8 == 0 && al(codes, 8) && ldc % 8 == 0;
  auto go = [&](auto k) { k<<<s.grid, s.block, 0, st>>>(codes, scales, x, T, n, ldc, ldx, nb); };
  if (fmt == FMT_I8) {
    if (bf16) vec ? go(ckpt8_unpack_kernel<FMT_I8, true, true>) : go(ckpt8_unpack_kernel<FMT_I8, true, false>);
    else vec ? go(ckpt8_unpack_kernel<FMT_I8, false, true>) : go(ckpt8_unpack_kernel<FMT_I8, false, false>);
  } else {
    if (bf16) vec ? go(ckpt8_unpack_kernel<FMT_E4M3, true, true>) : go(ckpt8_unpack_kernel<FMT_E4M3, true, false>);
    else vec ? go(ckpt8_unpack_kernel<FMT_E4M3, false, true>) : go(ckpt8_unpack_kernel<FMT_E4M3, false, false>);
  }
  return done(1);
}

int rmsnorm_fwd_ckpt8(const float* x, const float* w, uint16_t* y, float* rstd, uint8_t* codes, uint8_t* scales,
                      int fmt, int T, int h, float eps, cudaStream_t st) {
  if (T <= 0 || h <= 0 || (h & 3) || h > 8192 || !fmt_ok(fmt) || !al(x, 16) || !al(w, 16) ||
      !al(y, 8) || !al(codes, 4))
    return -1;
  const int units = (h + 7) / 8, nb = blocks32(h);
  // whole units where every row starts on a 32-byte boundary
  const bool vec = h % 8 == 0 && al(x, 32) && al(y, 16) && al(codes, 8);
  auto go = [&](auto k, int threads) { k<<<T, threads, 0, st>>>(x, w, y, rstd, codes, scales, h, nb, eps); };
  auto pick = [&](auto f, auto v) {
    constexpr int F = decltype(f)::value;
    constexpr bool X = decltype(v)::value;
    if (units <= 128) go(rmsnorm_fwd_ckpt8_kernel<F, 128, 1, X>, 128);
    else if (units <= 256) go(rmsnorm_fwd_ckpt8_kernel<F, 256, 1, X>, 256);
    else if (units <= 512) go(rmsnorm_fwd_ckpt8_kernel<F, 256, 2, X>, 256);
    else go(rmsnorm_fwd_ckpt8_kernel<F, 256, 4, X>, 256);
  };
  auto pick_f = [&](auto f) { vec ? pick(f, std::true_type()) : pick(f, std::false_type()); };
  if (fmt == FMT_I8) pick_f(std::integral_constant<int, FMT_I8>());
  else pick_f(std::integral_constant<int, FMT_E4M3>());
  return done(1);
}

size_t rmsnorm_bwd_ckpt8_partials(int T, int h) { return (size_t)bwd_shape(T, h).parts * h; }

int rmsnorm_bwd_ckpt8(const uint8_t* codes, const uint8_t* scales, int fmt, const float* w, const float* rstd,
                      const float* dy, const float* resid, float* dx, uint16_t* dx_bf16, float* dw, float* work,
                      int T, int h, cudaStream_t st) {
  if (T <= 0 || h <= 0 || (h & 3) || h > 8192 || !fmt_ok(fmt) || !al(codes, 4) || !al(w, 16) ||
      !al(dy, 16) || !al(resid, 16) || !al(dx, 16) || !al(dx_bf16, 8) || !al(work, 16))
    return -1;
  const int nb = blocks32(h);
  const BwdShape shape = bwd_shape(T, h);
  const bool bulk = h % 16 == 0 && al(codes, 16);  // every row of codes starts and ends on 16 bytes
  bool ok = true;
  auto go = [&](auto k, bool staged) {
    const int smem = staged ? shape.stages * h * (resid ? 9 : 5) : 0;
    if (smem > 48 * 1024)
      ok = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024) == cudaSuccess;
    if (ok)
      k<<<shape.parts, shape.threads, smem, st>>>(codes, scales, w, rstd, dy, resid, dx, dx_bf16, work, T, h, nb,
                                                  shape.stages);
  };
  auto pick = [&](auto f) {
    constexpr int F = decltype(f)::value;
    if (shape.vecs == 1) bulk ? go(rmsnorm_bwd_ckpt8_kernel<F, 1, true>, true) : go(rmsnorm_bwd_ckpt8_kernel<F, 1, false>, false);
    else bulk ? go(rmsnorm_bwd_ckpt8_kernel<F, 2, true>, true) : go(rmsnorm_bwd_ckpt8_kernel<F, 2, false>, false);
  };
  if (fmt == FMT_I8) pick(std::integral_constant<int, FMT_I8>());
  else pick(std::integral_constant<int, FMT_E4M3>());
  if (!ok) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((h + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, sum_parts_kernel, (const float*)work, shape.parts, h, dw) != cudaSuccess) return -1;
  return done(2);
}

int swiglu_fwd_ckpt8(const uint16_t* gu, uint16_t* act, uint8_t* codes, uint8_t* scales, int fmt, int T, int F,
                     int ld, cudaStream_t st) {
  if (!dims_ok(T, F, ld) || !fmt_ok(fmt) || !al(gu, 2) || !al(act, 2)) return -1;
  const Shape2 s = shape2(T, (ld + 7) / 8, kSwRows);
  const bool vec = ld % 8 == 0 && al(gu, 16) && al(act, 16) && al(codes, 8);
  auto go = [&](auto k) { k<<<s.grid, s.block, 0, st>>>(gu, act, codes, scales, T, F, ld, blocks32(F)); };
  if (fmt == FMT_I8) vec ? go(swiglu_fwd_ckpt8_kernel<FMT_I8, true>) : go(swiglu_fwd_ckpt8_kernel<FMT_I8, false>);
  else vec ? go(swiglu_fwd_ckpt8_kernel<FMT_E4M3, true>) : go(swiglu_fwd_ckpt8_kernel<FMT_E4M3, false>);
  return done(1);
}

int swiglu_bwd_ckpt8(const uint8_t* codes, const uint8_t* scales, int fmt, const uint16_t* dact, uint16_t* dgu,
                     int T, int F, int ld, cudaStream_t st) {
  if (!dims_ok(T, F, ld) || !fmt_ok(fmt) || !al(dact, 2) || !al(dgu, 2)) return -1;
  const Shape2 s = shape2(T, (ld + 7) / 8, kSwRows);
  const bool vec = ld % 8 == 0 && al(dact, 16) && al(dgu, 16) && al(codes, 8);
  auto go = [&](auto k) { k<<<s.grid, s.block, 0, st>>>(codes, scales, dact, dgu, T, F, ld, blocks32(F)); };
  if (fmt == FMT_I8) vec ? go(swiglu_bwd_ckpt8_kernel<FMT_I8, true>) : go(swiglu_bwd_ckpt8_kernel<FMT_I8, false>);
  else vec ? go(swiglu_bwd_ckpt8_kernel<FMT_E4M3, true>) : go(swiglu_bwd_ckpt8_kernel<FMT_E4M3, false>);
  return done(1);
}

}  // namespace mt
