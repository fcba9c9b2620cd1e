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
// int8 steps evenly (error, half a step: at most max|x| / 254 of the block's
// maximum when the scale is tight, max|x| / 127 at worst); e4m3 keeps 2^-4
// relative error down to 2^-14 of the block's maximum, so a block with one
// outlier keeps its other values.
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
MT_DEVICE_ERROR_PEEKER(ckpt8_peek_device_error)

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

// ---------------------------------------------------------------------------
// A unit is eight neighbouring columns, as WORDS 32-bit words: codes (2),
// bf16 (4) or fp32 (8). VEC: every row's units start on their own boundary
// and move in one access. Otherwise rows start anywhere: a unit is read as
// the aligned blocks that cover it (BLK bytes each, within the tensor) and
// shifted into place, and written as the aligned blocks that start in it,
// completed by the next lane's words; only a row's first and last bytes go
// one element at a time. The next lane has to hold the next unit, so a warp
// then takes 28 units of its own and the first four (one scale block) of the
// next warp's. (SwiGLU 4690 x 8001: forward 174 us element by element, 74 us
// so; backward 215 and 87 us.)
// ---------------------------------------------------------------------------
template <int WORDS>
constexpr int block_bytes() { return WORDS == 2 ? 8 : 16; }
template <int WORDS>
constexpr int elem_bytes() { return WORDS / 2; }
constexpr int kOwnUnits = 28;

__device__ __forceinline__ void load_block(const uint8_t* p, uint32_t (&w)[2]) {
  const uint2 u = __ldcs((const uint2*)p);
  w[0] = u.x, w[1] = u.y;
}
__device__ __forceinline__ void load_block(const uint8_t* p, uint32_t (&w)[4]) {
  const uint4 u = __ldcs((const uint4*)p);
  w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
}
__device__ __forceinline__ void load_block(const uint8_t* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store_block(uint8_t* p, const uint32_t (&w)[2]) { *(uint2*)p = make_uint2(w[0], w[1]); }
__device__ __forceinline__ void store_block(uint8_t* p, const uint32_t (&w)[4]) {
  *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_block(uint8_t* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// WORDS words from byte offset o (less than a block, the same in the whole
// warp: a warp's units lie in one row) of NX words.
template <int WORDS, int K, int NX>
__device__ __forceinline__ void shift_from(const uint32_t (&x)[NX], uint32_t bits, uint32_t (&w)[WORDS]) {
#pragma unroll
  for (int i = 0; i < WORDS; ++i) w[i] = __funnelshift_r(x[i + K], i + K + 1 < NX ? x[i + K + 1] : 0u, bits);
}
template <int WORDS, int NX>
__device__ __forceinline__ void shift_words(const uint32_t (&x)[NX], uint32_t o, uint32_t (&w)[WORDS]) {
  const uint32_t bits = (o & 3) * 8;
  if constexpr (block_bytes<WORDS>() == 8) {
    if (o & 4) shift_from<WORDS, 1>(x, bits, w);
    else shift_from<WORDS, 0>(x, bits, w);
  } else {
    switch (o >> 2) {
      case 0: shift_from<WORDS, 0>(x, bits, w); break;
      case 1: shift_from<WORDS, 1>(x, bits, w); break;
      case 2: shift_from<WORDS, 2>(x, bits, w); break;
      default: shift_from<WORDS, 3>(x, bits, w);
    }
  }
}
template <int WORDS>
__device__ __forceinline__ void load_elem(const uint8_t* p, int i, uint32_t (&w)[WORDS]) {
  if (WORDS == 2) w[(i >> 2) % WORDS] |= (uint32_t)p[i] << (8 * (i & 3));
  else if (WORDS == 4) w[(i >> 1) % WORDS] |= (uint32_t)((const uint16_t*)p)[i] << (16 * (i & 1));
  else w[i % WORDS] = ((const uint32_t*)p)[i];
}
template <int WORDS>
__device__ __forceinline__ void store_elem(uint8_t* p, int i, const uint32_t (&w)[WORDS]) {
  if (WORDS == 2) p[i] = (uint8_t)(w[(i >> 2) % WORDS] >> (8 * (i & 3)));
  else if (WORDS == 4) ((uint16_t*)p)[i] = (uint16_t)(w[(i >> 1) % WORDS] >> (16 * (i & 1)));
  else ((uint32_t*)p)[i] = w[i % WORDS];
}
// Element i (ES bytes) of a block's words.
template <int ES, int BW>
__device__ __forceinline__ void store_elem_of(uint8_t* p, int i, const uint32_t (&y)[BW]) {
  if (ES == 1) p[i] = (uint8_t)(y[(i >> 2) % BW] >> (8 * (i & 3)));
  else if (ES == 2) ((uint16_t*)p)[i] = (uint16_t)(y[(i >> 1) % BW] >> (16 * (i & 1)));
  else ((uint32_t*)p)[i] = y[i % BW];
}
// Whether the blocks that cover a row of `bytes` bytes lie within the
// tensor's bytes [lo, hi) (the blocks reach 15 bytes back and 31 on).
__device__ __forceinline__ bool inside(const void* row, size_t bytes, const void* lo, const void* hi) {
  return (const uint8_t*)row - (const uint8_t*)lo >= 16 && (const uint8_t*)hi - (const uint8_t*)row >= (int64_t)bytes + 32;
}
// Unit u of a row of n columns, 0 past them. in: the row's blocks all lie
// inside the tensor; else (its first and last rows) units go by elements.
template <int WORDS, bool VEC>
__device__ __forceinline__ void load_cols(const void* row, int u, int n, bool in, uint32_t (&w)[WORDS]) {
  constexpr int BLK = block_bytes<WORDS>(), BW = BLK / 4, NB = WORDS / BW + 1;
  const uint8_t* p = (const uint8_t*)row + (size_t)u * (WORDS * 4);
  if (VEC && u * 8 + 8 <= n) {
    load_block(p, w);
    return;
  }
  if (!VEC && in && u * 8 + 8 <= n) {
    const uint32_t o = (uint32_t)(uintptr_t)p & (BLK - 1);
    const uint8_t* q = p - o;
    uint32_t x[NB * BW];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      uint32_t y[BW];
      load_block(q + k * BLK, y);
#pragma unroll
      for (int i = 0; i < BW; ++i) x[k * BW + i] = y[i];
    }
    shift_words<WORDS>(x, o, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (u * 8 + i < n) load_elem(p, i, w);
}
// Unit u of a row of n columns. Without VEC the whole warp calls it; `own`:
// this lane's unit is the warp's to write (and there is a row to write to).
template <int WORDS, bool VEC>
__device__ __forceinline__ void store_cols(void* row, int u, int n, const uint32_t (&w)[WORDS], bool own) {
  constexpr int BLK = block_bytes<WORDS>(), BW = BLK / 4, ES = elem_bytes<WORDS>();
  uint8_t* p = (uint8_t*)row + (size_t)u * (WORDS * 4);
  if constexpr (VEC) {
    if (!own) return;
    if (u * 8 + 8 <= n) {
      store_block(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (u * 8 + i < n) store_elem(p, i, w);
    }
  } else {
    uint32_t x[WORDS + BW], v[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) x[i] = w[i];
#pragma unroll
    for (int i = 0; i < BW; ++i) x[WORDS + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
    const uint32_t o = (0u - (uint32_t)(uintptr_t)p) & (BLK - 1);  // bytes before the first boundary
    shift_words<WORDS>(x, o, v);
    if (!own) return;
    const int first = u * 8 + (int)o / ES;  // column of the boundary
#pragma unroll
    for (int k = 0; k < WORDS / BW; ++k) {
      const int c = first + k * (BLK / ES);
      uint32_t y[BW];
#pragma unroll
      for (int i = 0; i < BW; ++i) y[i] = v[k * BW + i];
      if (c + BLK / ES <= n) {
        store_block(p + o + k * BLK, y);
      } else if (c < n) {
#pragma unroll
        for (int i = 0; i < BLK / ES; ++i)
          if (c + i < n) store_elem_of<ES>(p + o + k * BLK, i, y);
      }
    }
    if (u == 0 && o) {
#pragma unroll
      for (int i = 0; i < BLK / ES; ++i)
        if (i < (int)o / ES && i < n) store_elem(p, i, w);
    }
  }
}
// The unit of a thread that is the x-th along its row, and whether it is its own.
template <bool VEC>
__device__ __forceinline__ int unit_of(int x, bool& own) {
  if (VEC) {
    own = true;
    return x;
  }
  own = (x & 31) < kOwnUnits;
  return (x >> 5) * kOwnUnits + (x & 31);
}
template <int WORDS>
__device__ __forceinline__ void to_floats(const uint32_t (&w)[WORDS], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (WORDS == 4) {
      v[2 * i] = __uint_as_float(w[i % WORDS] << 16);
      v[2 * i + 1] = __uint_as_float(w[i % WORDS] & 0xffff0000u);
    } else {
      v[2 * i] = __uint_as_float(w[(2 * i) % WORDS]);
      v[2 * i + 1] = __uint_as_float(w[(2 * i + 1) % WORDS]);
    }
  }
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
__device__ __forceinline__ uint32_t amax_bf16x8(const uint32_t (&w)[4]) {
  constexpr uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vimax3_u16x2(w[0] & m, w[1] & m, w[2] & m), w[3] & m);
}

// ---------------------------------------------------------------------------
// Pack and unpack. A thread owns one unit of eight values in each of kRows
// rows (their loads are in flight together); a 2D block covers blockDim.x
// units of blockDim.y rows at a time, so narrow matrices still fill a block.
// Measured for 8192 x 4096 fp32 (floor 24.7 us): pack 25.1 us, unpack 26.6;
// ragged 14783 x 777 (8.5): 12.6 with two rows a thread, 14.8 and 12.9 with
// four; four are the faster for whole rows of bf16 (unpack 13.8, 14.5 us).
// Ragged rows are bound by the issue of instructions (4172 x 4525 bf16, floor
// 8.4: 17 us each way, issue slots 75-80 % used): the shifts into place, and
// four lanes of 32 that repeat the next warp's units.
// ---------------------------------------------------------------------------
constexpr int pk_rows(bool vec) { return vec ? 4 : 2; }

template <int FMT, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_pack_kernel(const void* x, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales, int T, int n, int ldx, int ldc,
                                                         int nb) {
  constexpr int kRows = pk_rows(VEC);
  constexpr int W = BF16 ? 4 : 8, esz = BF16 ? 2 : 4;
  grid_wait();
  bool own;
  const int u = unit_of<VEC>(blockIdx.x * blockDim.x + threadIdx.x, own);
  const int step = gridDim.y * blockDim.y;
  const void* hi = (const uint8_t*)x + ((size_t)(T - 1) * ldx + n) * esz;
  // the whole block leaves the loop together: shuffles need every lane
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kRows) {
    uint32_t xw[kRows][W];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const uint8_t* row = (const uint8_t*)x + (size_t)t * ldx * esz;
      load_cols<W, VEC>(row, u, t < T ? n : 0, !VEC && inside(row, (size_t)n * esz, x, hi), xw[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      float v[8];
      to_floats(xw[r], v);
      uint32_t w[2];
      const uint32_t b = block_byte<FMT, 8>(v);
      encode_unit<FMT, 8>(b, v, w);
      store_cols<2, VEC>(codes + (size_t)t * ldc, u, n, w, own && t < T);
      if (t < T && (u & 3) == 0 && u * 8 < n) scales[(size_t)t * nb + u / 4] = (uint8_t)b;
    }
  }
}

template <int FMT, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_unpack_kernel(const uint8_t* codes,
                                                           const uint8_t* scales, void* __restrict__ x,
                                                           int T, int n, int ldc, int ldx, int nb) {
  constexpr int kRows = pk_rows(VEC);
  constexpr int W = BF16 ? 4 : 8, esz = BF16 ? 2 : 4;
  grid_wait();
  bool own;
  const int u = unit_of<VEC>(blockIdx.x * blockDim.x + threadIdx.x, own);
  const int step = gridDim.y * blockDim.y;
  const void* hi = codes + (size_t)(T - 1) * ldc + n;
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kRows) {
    uint32_t w[kRows][2];
    uint32_t b[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const uint8_t* row = codes + (size_t)t * ldc;
      load_cols<2, VEC>(row, u, t < T ? n : 0, !VEC && inside(row, n, codes, hi), w[r]);
      b[r] = t < T && u * 8 < n ? scales[(size_t)t * nb + u / 4] : 0u;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const float s = scale_up(b[r]);
      const float4 f = decode4<FMT>(w[r][0], s), g = decode4<FMT>(w[r][1], s);
      uint32_t o[W];
      if (BF16) {
        o[0] = pack_bf2(f.x, f.y), o[1] = pack_bf2(f.z, f.w), o[2] = pack_bf2(g.x, g.y), o[3] = pack_bf2(g.z, g.w);
      } else {
        const float v[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = __float_as_uint(v[i]);
      }
      store_cols<W, VEC>((uint8_t*)x + (size_t)t * ldx * esz, u, n, o, own && t < T);
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
// 38.9, four columns a unit 41.2; with the SM's 2048 threads and launched early
// 36.0, 512 threads of one unit 38.6. 4096 x 8192: 36.6, 256 threads of four
// units 38.3. Two units do not quite fit the 32 registers that 2048 threads
// leave: 4 to 8 bytes a thread spill at h = 4096, 8 to 24 above.
template <int FMT, int NT, int V, bool VEC>
__global__ void __launch_bounds__(NT, 2048 / NT)
    rmsnorm_fwd_ckpt8_kernel(const float* x, const float* w, uint16_t* __restrict__ y,
                             float* __restrict__ rstd, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                             int h, int nb, float eps) {
  __shared__ float red[NT / 32];
  grid_wait();
  const size_t t = blockIdx.x;
  const float* xr = x + t * h;
  const int tid = threadIdx.x;
  float v[V][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (tid + k * NT) * 8;
    if (VEC && c + 8 <= h) {
      uint32_t q[8];
      load_block((const uint8_t*)(xr + c), q);
      to_floats(q, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 f = c + i < h ? __ldcs((const float4*)(xr + c + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[k][i] = f.x, v[k][i + 1] = f.y, v[k][i + 2] = f.z, v[k][i + 3] = f.w;
      }
    }
  }
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
      if (VEC) {
        *(uint2*)(codes + t * h + c) = make_uint2(q[0], q[1]);
      } else {
        *(uint32_t*)(codes + t * h + c) = q[0];
        if (c + 4 < h) *(uint32_t*)(codes + t * h + c + 4) = q[1];
      }
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
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 g = c + i < h ? *(const float4*)(w + c + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      o[i / 2] = pack_bf2(v[k][i] * r * g.x, v[k][i + 1] * r * g.y);
      o[i / 2 + 1] = pack_bf2(v[k][i + 2] * r * g.z, v[k][i + 3] * r * g.w);
    }
    if (VEC) {
      if (c < h) *(uint4*)(yr + c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      if (c < h) *(uint2*)(yr + c) = make_uint2(o[0], o[1]);
      if (c + 4 < h) *(uint2*)(yr + c + 4) = make_uint2(o[2], o[3]);
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
// sums of dw in registers. One thread requests whole rows of dy and resid
// stages - 1 rows ahead as bulk copies into shared memory, so loads stay in
// flight across a row's reduction and hold no registers; codes and scales,
// whose rows need not be whole 16-byte pieces, are loaded one row ahead.
// Measured at 8192 x 4096 (504 MB, floor 74 us) with the sum of the parts:
// per-thread loads 103 us, per-thread cp.async staging 128 us (its 4-byte
// copies and second reads cost more than the loads it hides), bulk copies
// with two blocks an SM and three stages 87 us, one block and five 83 us.
// ---------------------------------------------------------------------------
constexpr int kBwdMaxThreads = 1024;
constexpr int kBwdMaxStages = 8;

// The SMs of the GPU that this is built for: sizes the workspace, so that it
// does not depend on the machine that asks (a budget is computed without one).
constexpr int kMaxSms = 152;

struct BwdShape {
  int threads, vecs, stages, an_sm;
  int parts(int T, int sms) const { return std::min(T, sms * an_sm); }
};
// 1024 threads an SM where the rows allow, the shared memory shared out among
// their blocks as stages of 8 h bytes (4 h without a residual).
BwdShape bwd_shape(int h) {
  BwdShape s;
  const int n4 = h / 4;
  s.vecs = h > 4096 ? 2 : 1;
  s.threads = std::max(32, (n4 + s.vecs * 32 - 1) / (s.vecs * 32) * 32);
  s.an_sm = std::min(8, 1024 / s.threads);
  s.stages = std::min(kBwdMaxStages, 222 * 1024 / s.an_sm / (8 * h));
  return s;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int FMT, int V>
__global__ void __launch_bounds__(kBwdMaxThreads)
    rmsnorm_bwd_ckpt8_kernel(const uint8_t* codes, const uint8_t* scales,
                             const float* w, const float* rstd,
                             const float* dy, const float* resid, float* dx, uint16_t* __restrict__ dxb,
                             float* __restrict__ part, int T, int h, int nb, int stages) {
  extern __shared__ __align__(128) uint8_t stage[];  // [stages]: dy, resid of a row
  __shared__ float red[2][kBwdMaxThreads / 32];
  __shared__ uint64_t full[kBwdMaxStages];
  __shared__ int abort_flag;
  const int n4 = h >> 2, tid = threadIdx.x, NT = blockDim.x, nw = NT >> 5;
  const float inv_h = 1.f / (float)h;
  const uint32_t row_bytes = (uint32_t)h * (resid ? 8u : 4u);
  auto request = [&](int t, int s) {  // one thread
    if (t >= T) return;
    uint8_t* p = stage + (size_t)s * row_bytes;
    mbar_arrive_expect_tx(&full[s], row_bytes);
    bulk_load(p, dy + (size_t)t * h, 4u * h, &full[s]);
    if (resid) bulk_load(p + 4 * h, resid + (size_t)t * h, 4u * h, &full[s]);
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
  float4 acc[V], wv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * NT;
    acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    wv[j] = i < n4 ? ((const float4*)w)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // a row's codes, scales and rstd, requested one row ahead
  uint32_t q_next[V], b_next[V];
  float r_next = 0.f;
  auto small = [&](int t) {
    if (t < T) {
      r_next = rstd[t];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = tid + j * NT;
        if (i < n4) {
          q_next[j] = __ldcs((const uint32_t*)(codes + (size_t)t * h) + i);
          b_next[j] = scales[(size_t)t * nb + i / 8];
        }
      }
    }
  };
  small(blockIdx.x);
  int flip = 0, st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
    const float r = r_next;
    float4 g[V], x[V];
    if (!mbar_wait(&full[st], phase, &abort_flag, kErrTimeoutTma)) break;
    const uint8_t* p = stage + (size_t)st * row_bytes;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * NT;
      if (i < n4) {
        g[j] = ((const float4*)p)[i];
        x[j] = decode4<FMT>(q_next[j], scale_up(b_next[j]));
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
    if (tid == 0) request(t + (stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
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
          const float4 e = ((const float4*)(p + 4 * h))[i];
          o.x += e.x;
          o.y += e.y;
          o.z += e.z;
          o.w += e.w;
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
  grid_wait();
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
// HBM bounds whole rows (8192 x 14336, floor 139 us each way: forward 139-140
// us, backward 137-139; with exact divisions and single maxima 242 and 243),
// the issue of instructions ragged ones (4690 x 8001, floor 44: 74 and 87 us;
// issue slots 83 and 80 % used). Whole rows: two a thread, five blocks an SM
// forward, six backward (146 us with the four that its registers allowed).
// Ragged: one row, eight blocks (two rows at five and four: 85 and 118 us).
// These bounds make the backward spill: 4 to 24 bytes a thread whole, 8 ragged.
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
constexpr int sw_rows(bool vec) { return vec ? 2 : 1; }

template <int FMT, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 5 : 8) swiglu_fwd_ckpt8_kernel(const uint16_t* gu,
                                                                  uint16_t* __restrict__ act,
                                                                  uint8_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales, int T, int F, int ld,
                                                                  int nb) {
  grid_wait();
  constexpr int kSwRows = sw_rows(VEC);
  bool own;
  const int x = unit_of<VEC>(blockIdx.x * blockDim.x + threadIdx.x, own);
  const int step = gridDim.y * blockDim.y;
  const void* hi = gu + (2 * (size_t)T - 1) * ld + F;
  // the whole block leaves the loop together: shuffles need every lane
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kSwRows) {
    uint32_t gq[kSwRows][4], uq[kSwRows][4];
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const uint16_t* row = gu + (size_t)t * 2 * ld;
      const bool in = !VEC && inside(row, ((size_t)ld + F) * 2, gu, hi);
      load_cols<4, VEC>(row, x, t < T ? F : 0, in, gq[r]);
      load_cols<4, VEC>(row + ld, x, t < T ? F : 0, in, uq[r]);
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
      to_floats(gq[r], g);
      to_floats(uq[r], u);
      uint32_t wg[2], wu[2], a[4];
      const uint32_t bg = scale_byte<FMT, 7>(m & 0xffffu), bu = scale_byte<FMT, 7>(m >> 16);
      encode_unit<FMT, 8>(bg, g, wg);
      encode_unit<FMT, 8>(bu, u, wu);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t g2 = pair(g[2 * i], g[2 * i + 1]), u2 = pair(u[2 * i], u[2 * i + 1]);
        a[i] = pack_pair(mul2(mul2(g2, sigmoid2(g2)), u2));
      }
      const bool write = own && t < T;
      uint8_t* crow = codes + (size_t)t * 2 * ld;
      // columns F..ld-1 are padding: codes and act are 0 there (the loads gave 0)
      store_cols<2, VEC>(crow, x, ld, wg, write);
      store_cols<2, VEC>(crow + ld, x, ld, wu, write);
      store_cols<4, VEC>(act + (size_t)t * ld, x, ld, a, write);
      if (t < T && (x & 3) == 0 && x * 8 < F) {
        scales[(size_t)t * 2 * nb + x / 4] = (uint8_t)bg;
        scales[(size_t)t * 2 * nb + nb + x / 4] = (uint8_t)bu;
      }
    }
  }
}

// dg = dact u silu'(g), du = dact silu(g), with g and u from the 8-bit form.
template <int FMT, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 6 : 8) swiglu_bwd_ckpt8_kernel(const uint8_t* codes,
                                                               const uint8_t* scales,
                                                               const uint16_t* dact,
                                                               uint16_t* __restrict__ dgu, int T, int F, int ld,
                                                               int nb) {
  grid_wait();
  constexpr int kSwRows = sw_rows(VEC);
  bool own;
  const int x = unit_of<VEC>(blockIdx.x * blockDim.x + threadIdx.x, own);
  const int step = gridDim.y * blockDim.y;
  const void *chi = codes + (2 * (size_t)T - 1) * ld + F, *dhi = dact + (size_t)(T - 1) * ld + F;
  for (int t0 = blockIdx.y * blockDim.y; t0 < T; t0 += step * kSwRows) {
    uint32_t wg[kSwRows][2], wu[kSwRows][2], bg[kSwRows], bu[kSwRows], dq[kSwRows][4];
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step + threadIdx.y, n = t < T ? F : 0;
      const uint8_t* crow = codes + (size_t)t * 2 * ld;
      const uint16_t* drow = dact + (size_t)t * ld;
      const bool in = !VEC && inside(crow, (size_t)ld + F, codes, chi) && inside(drow, (size_t)F * 2, dact, dhi);
      load_cols<2, VEC>(crow, x, n, in, wg[r]);
      load_cols<2, VEC>(crow + ld, x, n, in, wu[r]);
      load_cols<4, VEC>(drow, x, n, in, dq[r]);
      // a unit that lies in the padding has no block of its own
      bg[r] = x * 8 < n ? scales[(size_t)t * 2 * nb + x / 4] : 0u;
      bu[r] = x * 8 < n ? scales[(size_t)t * 2 * nb + nb + x / 4] : 0u;
    }
#pragma unroll
    for (int r = 0; r < kSwRows; ++r) {
      const int t = t0 + r * step + threadIdx.y;
      const float sg = scale_up(bg[r]), su = scale_up(bu[r]);
      float d[8];
      to_floats(dq[r], d);
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
      if (x * 8 + 8 > F) {  // padding columns carry no gradient (a NaN block reaches into them)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (x * 8 + i >= F) {
            const uint32_t keep = (i & 1) ? 0x0000ffffu : 0xffff0000u;
            og[i >> 1] &= keep;
            ou[i >> 1] &= keep;
          }
      }
      const bool write = own && t < T;
      uint16_t* row = dgu + (size_t)t * 2 * ld;
      store_cols<4, VEC>(row, x, ld, og, write);
      store_cols<4, VEC>(row + ld, x, ld, ou, write);
    }
  }
}

// Block and grid of the 2D kernels: units of 8 columns along x, rows along y.
struct Shape2 {
  dim3 grid, block;
};
Shape2 shape2(int T, int units, int rows, bool vec) {
  if (!vec) units = (units + kOwnUnits - 1) / kOwnUnits * 32;  // threads along a row
  int bx = vec ? 8 : 32;
  while (bx < units && bx < 256) bx *= 2;
  // narrower blocks where the last one along a row would idle by a quarter or more
  while (bx > 32 && (units + bx - 1) / bx * bx - units >= units / 4) bx /= 2;
  const int by = 256 / bx;
  const int gy = (T + by * rows - 1) / (by * rows);
  return {dim3((unsigned)((units + bx - 1) / bx), (unsigned)std::min(gy, 65535)), dim3((unsigned)bx, (unsigned)by)};
}

inline int blocks32(int n) { return (n + 31) / 32; }
inline bool al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int done(int launches, cudaError_t e) {
  count_launches(launches);
  return e == cudaSuccess ? 0 : kLaunchFailed;
}
// Sizes: row and column counters stay within 31 bits with room for a grid's step.
inline bool dims_ok(int T, int n, int ld) { return T > 0 && n > 0 && ld >= n && T <= (1 << 30) && ld <= (1 << 29); }
inline bool fmt_ok(int fmt) { return fmt == FMT_I8 || fmt == FMT_E4M3; }

}  // namespace

int ckpt8_pack(const void* x, bool bf16, int fmt, uint8_t* codes, uint8_t* scales, int T, int n, int ldx, int ldc,
               cudaStream_t st) {
  if (!dims_ok(T, n, ldx) || !dims_ok(T, n, ldc) || !fmt_ok(fmt) || !al(x, bf16 ? 2 : 4)) return kRefused;
  const int nb = blocks32(n);
  // whole loads and stores of eight values where every row starts on their boundary
  const bool vec = al(x, bf16 ? 16 : 32) && ldx % 8 == 0 && al(codes, 8) && ldc % 8 == 0;
  const Shape2 s = shape2(T, (n + 7) / 8, pk_rows(vec), vec);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, s.grid, s.block, 0, st, 1, x, codes, scales, T, n, ldx, ldc, nb); };
  if (fmt == FMT_I8) {
    if (bf16) vec ? go(ckpt8_pack_kernel<FMT_I8, true, true>) : go(ckpt8_pack_kernel<FMT_I8, true, false>);
    else vec ? go(ckpt8_pack_kernel<FMT_I8, false, true>) : go(ckpt8_pack_kernel<FMT_I8, false, false>);
  } else {
    if (bf16) vec ? go(ckpt8_pack_kernel<FMT_E4M3, true, true>) : go(ckpt8_pack_kernel<FMT_E4M3, true, false>);
    else vec ? go(ckpt8_pack_kernel<FMT_E4M3, false, true>) : go(ckpt8_pack_kernel<FMT_E4M3, false, false>);
  }
  return done(1, e);
}

int ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int fmt, void* x, bool bf16, int T, int n, int ldc,
                 int ldx, cudaStream_t st) {
  if (!dims_ok(T, n, ldx) || !dims_ok(T, n, ldc) || !fmt_ok(fmt) || !al(x, bf16 ? 2 : 4)) return kRefused;
  const int nb = blocks32(n);
  const bool vec = al(x, bf16 ? 16 : 32) && ldx % 8 == 0 && al(codes, 8) && ldc % 8 == 0;
  const Shape2 s = shape2(T, (n + 7) / 8, pk_rows(vec), vec);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, s.grid, s.block, 0, st, 1, codes, scales, x, T, n, ldc, ldx, nb); };
  if (fmt == FMT_I8) {
    if (bf16) vec ? go(ckpt8_unpack_kernel<FMT_I8, true, true>) : go(ckpt8_unpack_kernel<FMT_I8, true, false>);
    else vec ? go(ckpt8_unpack_kernel<FMT_I8, false, true>) : go(ckpt8_unpack_kernel<FMT_I8, false, false>);
  } else {
    if (bf16) vec ? go(ckpt8_unpack_kernel<FMT_E4M3, true, true>) : go(ckpt8_unpack_kernel<FMT_E4M3, true, false>);
    else vec ? go(ckpt8_unpack_kernel<FMT_E4M3, false, true>) : go(ckpt8_unpack_kernel<FMT_E4M3, false, false>);
  }
  return done(1, e);
}

int rmsnorm_fwd_ckpt8(const float* x, const float* w, uint16_t* y, float* rstd, uint8_t* codes, uint8_t* scales,
                      int fmt, int T, int h, float eps, cudaStream_t st) {
  if (T <= 0 || h <= 0 || (h & 3) || h > 8192 || !fmt_ok(fmt) || !al(x, 16) || !al(w, 16) ||
      !al(y, 8) || !al(codes, 4))
    return kRefused;
  const int units = (h + 7) / 8, nb = blocks32(h);
  // whole units where every row starts on a 32-byte boundary, else their halves
  const bool vec = h % 8 == 0 && al(x, 32) && al(y, 16) && al(codes, 8);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k, int threads) {
    e = mt_host::launch_early(k, T, threads, 0, st, 1, x, w, y, rstd, codes, scales, h, nb, eps);
  };
  auto pick = [&](auto f, auto v) {
    constexpr int F = decltype(f)::value;
    constexpr bool X = decltype(v)::value;
    if (units <= 128) go(rmsnorm_fwd_ckpt8_kernel<F, 128, 1, X>, 128);
    else if (units <= 256) go(rmsnorm_fwd_ckpt8_kernel<F, 256, 1, X>, 256);
    else if (units <= 512) go(rmsnorm_fwd_ckpt8_kernel<F, 256, 2, X>, 256);
    else go(rmsnorm_fwd_ckpt8_kernel<F, 512, 2, X>, 512);
  };
  auto pick_f = [&](auto f) { vec ? pick(f, std::true_type()) : pick(f, std::false_type()); };
  if (fmt == FMT_I8) pick_f(std::integral_constant<int, FMT_I8>());
  else pick_f(std::integral_constant<int, FMT_E4M3>());
  return done(1, e);
}

bool rmsnorm_bwd_ckpt8_dims(int T, int h) {
  // a block's row counter goes up to stages rounds of the grid past T
  return T > 0 && T <= (1 << 30) && h > 0 && h % 4 == 0 && h <= 8192;
}

size_t rmsnorm_bwd_ckpt8_partials(int T, int h) { return (size_t)bwd_shape(h).parts(T, kMaxSms) * h; }

int rmsnorm_bwd_ckpt8(const uint8_t* codes, const uint8_t* scales, int fmt, const float* w, const float* rstd,
                      const float* dy, const float* resid, float* dx, uint16_t* dx_bf16, float* dw, float* work,
                      int T, int h, cudaStream_t st) {
  if (!rmsnorm_bwd_ckpt8_dims(T, h) || !fmt_ok(fmt) || !al(codes, 4) || !al(w, 16) || !al(dy, 16) ||
      !al(resid, 16) || !al(dx, 16) || !al(dx_bf16, 8) || !al(work, 16))
    return kRefused;
  const int nb = blocks32(h);
  const BwdShape shape = bwd_shape(h);
  const int parts = shape.parts(T, std::min(mt_host::num_sms(), kMaxSms));
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) {
    const int smem = shape.stages * h * (resid ? 8 : 4);
    if (smem > 47 * 1024)  // with the static part past the default limit
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
    if (e == cudaSuccess)
      e = mt_host::launch_early(k, parts, shape.threads, smem, st, 1, codes, scales, w, rstd, dy, resid, dx,
                                dx_bf16, work, T, h, nb, shape.stages);
  };
  auto pick = [&](auto f) {
    constexpr int F = decltype(f)::value;
    if (shape.vecs == 1) go(rmsnorm_bwd_ckpt8_kernel<F, 1>);
    else go(rmsnorm_bwd_ckpt8_kernel<F, 2>);
  };
  if (fmt == FMT_I8) pick(std::integral_constant<int, FMT_I8>());
  else pick(std::integral_constant<int, FMT_E4M3>());
  if (e == cudaSuccess)
    e = mt_host::launch_early(sum_parts_kernel, (h + 31) / 32, 1024, 0, st, 1, (const float*)work, parts, h, dw);
  return done(2, e);
}

int swiglu_fwd_ckpt8(const uint16_t* gu, uint16_t* act, uint8_t* codes, uint8_t* scales, int fmt, int T, int F,
                     int ld, cudaStream_t st) {
  if (!dims_ok(T, F, ld) || !fmt_ok(fmt) || !al(gu, 2) || !al(act, 2)) return kRefused;
  const bool vec = ld % 8 == 0 && al(gu, 16) && al(act, 16) && al(codes, 8);
  const Shape2 s = shape2(T, (ld + 7) / 8, sw_rows(vec), vec);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, s.grid, s.block, 0, st, 1, gu, act, codes, scales, T, F, ld, blocks32(F)); };
  if (fmt == FMT_I8) vec ? go(swiglu_fwd_ckpt8_kernel<FMT_I8, true>) : go(swiglu_fwd_ckpt8_kernel<FMT_I8, false>);
  else vec ? go(swiglu_fwd_ckpt8_kernel<FMT_E4M3, true>) : go(swiglu_fwd_ckpt8_kernel<FMT_E4M3, false>);
  return done(1, e);
}

int swiglu_bwd_ckpt8(const uint8_t* codes, const uint8_t* scales, int fmt, const uint16_t* dact, uint16_t* dgu,
                     int T, int F, int ld, cudaStream_t st) {
  if (!dims_ok(T, F, ld) || !fmt_ok(fmt) || !al(dact, 2) || !al(dgu, 2)) return kRefused;
  const bool vec = ld % 8 == 0 && al(dact, 16) && al(dgu, 16) && al(codes, 8);
  const Shape2 s = shape2(T, (ld + 7) / 8, sw_rows(vec), vec);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto k) { e = mt_host::launch_early(k, s.grid, s.block, 0, st, 1, codes, scales, dact, dgu, T, F, ld, blocks32(F)); };
  if (fmt == FMT_I8) vec ? go(swiglu_bwd_ckpt8_kernel<FMT_I8, true>) : go(swiglu_bwd_ckpt8_kernel<FMT_I8, false>);
  else vec ? go(swiglu_bwd_ckpt8_kernel<FMT_E4M3, true>) : go(swiglu_bwd_ckpt8_kernel<FMT_E4M3, false>);
  return done(1, e);
}

}  // namespace mt
