// Tensor-core products whose results are used where they are made: D = A B^T
// over a batch, bf16 or fp16 operands, fp32 accumulators in tensor memory,
// and an epilogue type E that sees every output tile there and decides what
// leaves the SM (the statistics of a softmax, a gradient, a polynomial of a
// matrix). The plain products of the decoder's layers are gemm.cu's.
//
// A tile is TM x BN outputs: 256 x 256 by a pair of SMs (tcgen05.mma
// cta_group::2; each CTA holds 128 rows of A and 128 of B, 32 KB a 64-deep
// step, five or six steps in flight) where there are enough of them for the
// GPU, else 128 x 128 by one SM. Warp 0 fills the ring by TMA, one thread of
// warp 1 issues the MMAs, the E::WARPS warps behind them drain the two
// accumulators, so one tile's epilogue overlaps the next one's products. CTAs
// are persistent and take tiles in a fixed order; each output is one fixed
// sum, whatever the grid.
//
// What an epilogue reads beside the sums comes by TMA in slabs of 32 rows by
// 64 columns, each warp its own, asked for as soon as the one before is in
// registers: for the next tile while its products run. Results leave from the
// lanes in whole 32-byte sectors, or by TMA where shared memory gathers them
// anyway. (Four warps with plain 16-byte loads and stores took 24 us for a 256
// x 256 tile that reads and writes two fp16 matrices, against 7 us of MMAs at
// K = 1536; eight so 11, most of it the way to and from L2, which the operands
// share.)
//
// Rows, columns and depth need not be multiples of anything: TMA fills zeros
// outside a matrix and drops what is stored there, and the epilogues look at
// M and N.
#pragma once
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace mt {

struct ProductShape {
  int M, N, K;
  int batch;     // matrices, one after another (the tensor maps' third axis)
  int num_m, num_n, tiles;  // of one matrix; set by product_shape
  int group_m;   // row blocks that share a sweep over the columns
  int a_rows;    // rows of A that a CTA loads: 128, or fewer where M is (single SMs, K contiguous)
  int k_rows;    // rows of a step of an operand with K along its rows: 64, or fewer where K is
  int split_kb;  // not 0: one matrix, `batch` counts ranges of split_kb 64-deep steps of its K
};

// BN: tile columns; PAIR: two SMs a tile; A_MN / B_MN: the operand is stored
// with its outputs' axis contiguous ([K, M] and [K, N]) rather than K; F16:
// fp16 operands; SYM: A = B and D symmetric, only tiles on and above the
// diagonal are made (the epilogue mirrors them); SHALLOW: K is below 64 and
// operands with K along their rows are loaded and multiplied no deeper (a kind
// of its own: the test of it in the MMAs' loop costs the others 4 %).
template <int BN_, bool PAIR_, bool A_MN_, bool B_MN_, bool F16_ = false, bool SYM_ = false, bool SHALLOW_ = false>
struct ProductCfg {
  static constexpr int BN = BN_;
  static constexpr bool PAIR = PAIR_, A_MN = A_MN_, B_MN = B_MN_, F16 = F16_, SYM = SYM_,
                        SHALLOW = SHALLOW_;
  static constexpr int BM = 128, BK = 64;
  static constexpr int TM = PAIR ? 2 * BM : BM;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // rows of B in one CTA
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;
};
// Ring depth and shared memory of a product with epilogue E, which gets
// E::SLABS bytes of it a warp (each a multiple of 1024).
template <class C, class E>
struct ProductSmem {
  static constexpr int SLABS = E::WARPS * E::SLABS;
  static constexpr int STAGES = SLABS > 32 * 1024 ? 5 : 6;
  static constexpr int TOTAL = STAGES * C::STAGE_BYTES + SLABS + 1024 /*align*/ + 512 /*barriers*/;
};

// What an epilogue knows of its tile: this lane's row of D, the warp's first
// row, the tile's first column, its columns and its matrix.
struct TileAt {
  int row, row0, n0, width, nb, b;
  bool mirror;  // SYM: the tile lies above the diagonal
};

template <class C>
__device__ __forceinline__ void product_tile(const ProductShape& s, int tile, int& mb, int& nb, int& b) {
  b = tile / s.tiles;
  const int t = tile - b * s.tiles;
  if (C::SYM) {  // column nb holds nb + 1 tiles
    nb = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (nb * (nb + 1) / 2 > t) --nb;
    while ((nb + 1) * (nb + 2) / 2 <= t) ++nb;
    mb = t - nb * (nb + 1) / 2;
  } else {
    const int per_group = s.group_m * s.num_n;
    const int g = t / per_group;
    const int first = g * s.group_m;
    const int size = min(s.num_m - first, s.group_m);
    const int r = t - g * per_group;
    mb = first + r % size;
    nb = r / size;
  }
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int x, int y,
                                                 int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}

// Bytes that a CTA's loads of one step bring.
template <class C>
__device__ __forceinline__ uint32_t step_bytes(const ProductShape& s) {
  const int k = C::SHALLOW ? s.k_rows : C::BK;
  return (C::A_MN ? C::BM / 64 * k : C::PAIR ? C::BM : s.a_rows) * 128 + (C::B_MN ? C::B_ROWS / 64 * k : C::B_ROWS) * 128;
}
template <class C>
__host__ __device__ constexpr uint32_t product_idesc() {
  return make_idesc(C::TM, C::BN, C::A_MN, C::B_MN) & (C::F16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}
// Matrix descriptors of an operand's first step; a later place in the ring is
// its distance / 16 further, the low bits being the address / 16.
template <bool MN>
__device__ __forceinline__ uint64_t first_desc(const void* ring) {
  return MN ? make_sdesc(smem_u32(ring), 8192, 1024) : make_sdesc(smem_u32(ring), 16, 1024);
}
// One 64-deep step: four MMAs of depth 16, fewer where K has fewer `rows`.
template <class C>
__device__ __forceinline__ void product_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool first,
                                            int rows) {
#pragma unroll
  for (int kk = 0; kk < C::BK / 16; ++kk) {
    if (C::SHALLOW && kk * 16 >= rows) break;
    const uint64_t ad = a + kk * ((C::A_MN ? 2048 : 32) >> 4), bd = b + kk * ((C::B_MN ? 2048 : 32) >> 4);
    if (C::PAIR) tc_mma2(d_tmem, ad, bd, idesc, !first || kk != 0);
    else tc_mma(d_tmem, ad, bd, idesc, !first || kk != 0);
  }
}

// Slabs: tiles of shared memory that TMA reads from or writes to.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)map),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until all but the last N groups of this thread's stores have been read out
// of shared memory (READ) or are complete.
template <int N, bool READ>
__device__ __forceinline__ void bulk_store_wait() {
  if (READ) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
  else asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
// 16-byte piece k of this lane's row of a slab of 128-byte rows (128-byte swizzle).
__device__ __forceinline__ uint4* slab_piece(uint8_t* slab, int row, int k) {
  return (uint4*)(slab + row * 128 + ((k ^ (row & 7)) << 4));
}

// What an epilogue warp keeps from tile to tile: its slabs and their barrier,
// how many slabs it has begun, its share of the columns.
struct EpiWarp {
  uint8_t* smem;
  uint64_t* bar;
  volatile int* abort;
  int lane, part;
  uint32_t begun;
};
// For epilogues without slabs coming in, and without work of their own before
// the first tile.
struct NoSlabs {
  template <class A>
  static __device__ __forceinline__ void begin(const A&, int) {}
  template <int BN, class A>
  static __device__ __forceinline__ void prefetch(const A&, const ProductShape&, const TileAt&, EpiWarp&) {}
};

template <class C>
__device__ __forceinline__ TileAt tile_at(const ProductShape& s, int tile, int rank, int q, int lane) {
  int mb, nb;
  TileAt at;
  product_tile<C>(s, tile, mb, nb, at.b);
  at.row0 = mb * C::TM + rank * C::BM + q * 32;
  at.row = at.row0 + lane;
  at.nb = nb;
  at.n0 = nb * C::BN;
  at.width = C::BN;
  at.mirror = C::SYM && mb != nb;
  return at;
}

template <class C, class E>
__global__ void __launch_bounds__(64 + 32 * E::WARPS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ ProductShape s, const __grid_constant__ typename E::Args args) {
  constexpr int BN = C::BN, BM = C::BM, BK = C::BK;
  constexpr bool PAIR = C::PAIR;
  constexpr int STAGES = ProductSmem<C, E>::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * C::A_BYTES;
  uint8_t* slabs = smem + STAGES * C::STAGE_BYTES;
  uint64_t* full = (uint64_t*)(slabs + ProductSmem<C, E>::SLABS);  // PAIR: the even CTA's, for both halves
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // PAIR: the even CTA's, both CTAs drained
  uint64_t* slab_bars = tempty + 2;  // one a warp
  uint32_t* tmem_slot = (uint32_t*)(slab_bars + E::WARPS);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);

  const uint32_t warp = warp_id(), lane = lane_id();
  const int rank = PAIR ? (int)cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], (PAIR ? 2 : 1) * E::WARPS);
    }
    for (int i = 0; i < E::WARPS; ++i) mbar_init(&slab_bars[i], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc2(tmem_slot, C::TMEM_COLS);
      tmem_relinquish2();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_wait();
  grid_release();

  const int all = s.tiles * s.batch;
  const int first = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int step = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int all_kb = (s.K + BK - 1) / BK;
  // K steps of a tile, and the first one
  auto steps_of = [&](int b) { return s.split_kb ? min(s.split_kb, all_kb - b * s.split_kb) : all_kb; };
  auto first_of = [&](int b) { return s.split_kb ? b * s.split_kb : 0; };

  if (warp == 0) {
    if (lane == 0) {  // TMA producer
      const uint32_t full0 = PAIR ? mapa_shared(full, 0) : 0;
      const uint32_t stage_bytes = (PAIR ? 2 : 1) * step_bytes<C>(s);
      int stage = 0;
      uint32_t phase = 0;
      for (int tile = first; tile < all; tile += step) {
        int mb, nb, b;
        product_tile<C>(s, tile, mb, nb, b);
        const int m0 = mb * C::TM + rank * BM, n0 = nb * BN + rank * C::B_ROWS;
        const int k0 = first_of(b), num_kb = steps_of(b), z = s.split_kb ? 0 : b;
        for (int kb = k0; kb < k0 + num_kb; ++kb) {
          mbar_wait<PAIR>(&empty[stage], phase ^ 1, abort_flag, kErrTimeoutTma);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], stage_bytes);
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if (PAIR) tma_load_3d_pair(dst, map, full0 + stage * 8, x, y, z);
            else tma_load_3d(dst, map, &full[stage], x, y, z);
          };
          uint8_t* a_dst = sA + stage * C::A_BYTES;
          uint8_t* b_dst = sB + stage * C::B_BYTES;
          if (!C::A_MN) {
            load(a_dst, &tmA, kb * BK, m0);
          } else {
#pragma unroll
            for (int j = 0; j < BM / 64; ++j) load(a_dst + j * 8192, &tmA, m0 + 64 * j, kb * BK);
          }
          if (!C::B_MN) {
            load(b_dst, &tmB, kb * BK, n0);
          } else {
#pragma unroll
            for (int j = 0; j < C::B_ROWS / 64; ++j) load(b_dst + j * 8192, &tmB, n0 + 64 * j, kb * BK);
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // MMA issuer
      constexpr uint32_t IDESC = product_idesc<C>();
      const uint64_t a0 = first_desc<C::A_MN>(sA), b0 = first_desc<C::B_MN>(sB);
      int stage = 0, local = 0;
      uint32_t phase = 0;
      for (int tile = first; tile < all; tile += step, ++local) {
        const int acc = local & 1;
        const int num_kb = steps_of(tile / s.tiles);
        mbar_wait<PAIR>(&tempty[acc], ((local >> 1) & 1) ^ 1, abort_flag, kErrTimeoutMma);
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < num_kb; ++kb) {
          mbar_wait(&full[stage], phase, abort_flag, kErrTimeoutMma);
          tc_fence_after();
          product_mma<C>(d_tmem, a0 + stage * (C::A_BYTES >> 4), b0 + stage * (C::B_BYTES >> 4), IDESC, kb == 0, s.k_rows);
          if (PAIR) tc_commit2(&empty[stage], 0x3);
          else tc_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (PAIR) tc_commit2(&tfull[acc], 0x3);
        else tc_commit(&tfull[acc]);
      }
    }
    __syncwarp();
  } else {  // epilogue: warp w reads tensor memory lanes 32 (w % 4) ..
    const int q = (int)(warp & 3);
    const uint32_t tempty0 = PAIR ? mapa_shared(tempty, 0) : 0;
    EpiWarp w;
    w.smem = slabs + (warp - 2) * E::SLABS;
    w.bar = slab_bars + (warp - 2);
    w.abort = abort_flag;
    w.lane = (int)lane;
    w.part = (int)(warp - 2) >> 2;
    w.begun = 0;
    E::begin(args, (int)(warp - 2));
    if (first < all) E::template prefetch<BN>(args, s, tile_at<C>(s, first, rank, q, (int)lane), w);
    int local = 0;
    for (int tile = first; tile < all; tile += step, ++local) {
      const int acc = local & 1;
      const TileAt at = tile_at<C>(s, tile, rank, q, (int)lane);
      // per-row values that the epilogue needs are loaded while the products run
      typename E::Row row_in;
      E::load_row(args, s, at, row_in);
      mbar_wait<PAIR>(&tfull[acc], (local >> 1) & 1, abort_flag, kErrTimeoutEpi);
      tc_fence_after();
      E::template tile<BN>(args, s, at, row_in, w, tmem_base + ((q * 32) << 16) + acc * BN);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(tempty0 + acc * 8);
        else mbar_arrive(&tempty[acc]);
      }
      if (tile + step < all) E::template prefetch<BN>(args, s, tile_at<C>(s, tile + step, rank, q, (int)lane), w);
    }
    if (lane == 0) bulk_store_wait<0, false>();
  }
  if (*abort_flag) {  // a wait ran out: give the copies in flight time to land
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 24)) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the peer may still address this CTA's barriers or tensor memory
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc2(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// 32 bytes at a 32-byte boundary: a whole sector.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
// 32 accumulator columns of this lane's row.
__device__ __forceinline__ void tile_chunk(uint32_t tb, int c, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();
  tmem_ld32(tb + c * 32, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------------------
// The form for few tiles: a cluster of S CTAs (2 or 4) shares one 128 x 128
// tile, each a range of K; then each gets a 128 / S wide share of its columns
// from the others through distributed shared memory, adds the parts in rank
// order and runs the epilogue on it, 32 columns of a row a thread.
// E::early asks for what E::chunk needs beside the sums, while these are made;
// E::chunk has 4 KB of shared memory a warp.
// Four 32 KB steps are in flight and the parts have 64 KB of their own: one CTA
// an SM. (1024 x 4096 orthogonalised in 183 us so when it was built; with three
// steps, so that the CTAs of two launches fit on an SM, 210; with more steps no
// faster.)
// ---------------------------------------------------------------------------
struct SplitSmem {
  static constexpr int STAGES = 4;
  static constexpr int PART = 128 * 32 * 4;  // 128 rows of a 32-column chunk
};

template <class C, class E, int S>
__global__ void __launch_bounds__(192, 1)
    product_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ ProductShape s, const __grid_constant__ typename E::Args args) {
  constexpr int BN = C::BN, BM = C::BM, BK = C::BK, STAGES = SplitSmem::STAGES;
  static_assert(!C::PAIR && BN == 128 && (S == 2 || S == 4), "one SM a CTA, chunks of 32 columns");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * C::A_BYTES;
  uint8_t* parts = smem + STAGES * C::STAGE_BYTES;  // [source][chunk of this CTA's share]
  uint64_t* full = (uint64_t*)(parts + 4 * SplitSmem::PART);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);

  const uint32_t warp = warp_id(), lane = lane_id();
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA runs: its shared memory may be written
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_wait();
  grid_release();

  const int tile = (int)blockIdx.x / S;
  const int all_kb = (s.K + BK - 1) / BK, each = (all_kb + S - 1) / S;
  const int k0 = min(all_kb, rank * each), k1 = min(all_kb, k0 + each);
  int mb, nb, b;
  product_tile<C>(s, tile, mb, nb, b);
  constexpr int CHUNKS = 4 / S;  // of this CTA's share

  if (warp == 0) {
    if (lane == 0) {
      for (int kb = k0; kb < k1; ++kb) {
        const int stage = (kb - k0) % STAGES;
        mbar_wait(&empty[stage], (((kb - k0) / STAGES) & 1) ^ 1, abort_flag, kErrTimeoutTma);
        mbar_arrive_expect_tx(&full[stage], step_bytes<C>(s));
        uint8_t* a_dst = sA + stage * C::A_BYTES;
        uint8_t* b_dst = sB + stage * C::B_BYTES;
        if (!C::A_MN) {
          tma_load_3d(a_dst, &tmA, &full[stage], kb * BK, mb * BM, b);
        } else {
#pragma unroll
          for (int j = 0; j < BM / 64; ++j)
            tma_load_3d(a_dst + j * 8192, &tmA, &full[stage], mb * BM + 64 * j, kb * BK, b);
        }
        if (!C::B_MN) {
          tma_load_3d(b_dst, &tmB, &full[stage], kb * BK, nb * BN, b);
        } else {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j)
            tma_load_3d(b_dst + j * 8192, &tmB, &full[stage], nb * BN + 64 * j, kb * BK, b);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t IDESC = product_idesc<C>();
      const uint64_t a0 = first_desc<C::A_MN>(sA), b0 = first_desc<C::B_MN>(sB);
      for (int kb = k0; kb < k1; ++kb) {
        const int stage = (kb - k0) % STAGES;
        mbar_wait(&full[stage], ((kb - k0) / STAGES) & 1, abort_flag, kErrTimeoutMma);
        tc_fence_after();
        product_mma<C>(tmem_base, a0 + stage * (C::A_BYTES >> 4), b0 + stage * (C::B_BYTES >> 4), IDESC, kb == k0, s.k_rows);
        tc_commit(&empty[stage]);
      }
      tc_commit(done);  // with no steps: arrives at once
    }
    __syncwarp();
  }
  // warps 2 ..: lanes 32 (w % 4) .. of tensor memory
  const int q = (int)(warp & 3);
  TileAt at;
  at.row0 = mb * BM + q * 32;
  at.row = at.row0 + (int)lane;
  at.nb = nb;
  at.n0 = nb * BN;
  at.width = BN;
  at.b = b;
  at.mirror = C::SYM && mb != nb;
  const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
  const bool finish = warp >= 2 && at.row0 < s.M;
  typename E::Row row_in;
  typename E::Early early[CHUNKS];
  if (warp >= 2) {
    E::load_row(args, s, at, row_in);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int col = at.n0 + 32 * (rank * CHUNKS + c);
      if (finish && col < s.N) E::early(args, s, at, col, early[c]);
    }
    mbar_wait(done, 0, abort_flag, kErrTimeoutEpi);
    tc_fence_after();
  }
  if (warp >= 2) {
#pragma unroll 1
    for (int j = 1; j < S; ++j) {  // each CTA begins with another one's share
      const int owner = (rank + j) % S;
#pragma unroll 1
      for (int c = 0; c < CHUNKS; ++c) {
        const int chunk = owner * CHUNKS + c;
        if (at.n0 + 32 * chunk >= s.N) break;
        float v[32];
        if (k0 < k1) {
          tile_chunk(tb, chunk, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        // [source][chunk of the owner's share][4 columns][row]
        const uint32_t to =
            mapa_shared(parts + (rank * CHUNKS + c) * SplitSmem::PART, (uint32_t)owner) + (q * 32 + lane) * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + i * 128 * 16), "f"(v[4 * i]),
                       "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                       : "memory");
      }
    }
    __syncwarp();
  }
  cluster_sync();  // the parts are there
  if (finish) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int chunk = rank * CHUNKS + c;
      if (at.n0 + 32 * chunk >= s.N) break;
      float v[32], sum[32];
      if (k0 < k1) {
        tile_chunk(tb, chunk, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[i] = 0.f;
#pragma unroll
      for (int r = 0; r < S; ++r) {
        if (r == rank) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[i] += v[i];
        } else {
          const float4* p = (const float4*)(parts + (r * CHUNKS + c) * SplitSmem::PART) + q * 32 + lane;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 w = p[i * 128];
            sum[4 * i] += w.x, sum[4 * i + 1] += w.y, sum[4 * i + 2] += w.z, sum[4 * i + 3] += w.w;
          }
        }
      }
      // 4 KB of the place that this CTA's own part does not need
      uint8_t* room = parts + (rank * CHUNKS + c) * SplitSmem::PART + q * 4096;
      E::chunk(args, s, at, row_in, early[c], at.n0 + 32 * chunk, sum, room);
    }
  }
  if (*abort_flag) {
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 24)) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, BN);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// A batch of matrices [rows, cols] of 16-bit values, row stride ld, matrices
// `apart` elements from each other; boxes of 64 columns by `box_rows`.
inline bool product_map(CUtensorMap* m, const void* base, int rows, int cols, int64_t ld, int64_t apart, int batch,
                        int box_rows, bool f16, int box_cols = 64) {
  const uint64_t gdim[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)batch};
  const uint64_t gstride[2] = {(uint64_t)ld * 2, (uint64_t)apart * 2};
  const uint32_t box[3] = {(uint32_t)box_cols, (uint32_t)box_rows, 1};
  return mt_host::encode_tiled(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base,
                               gdim, gstride, box,
                               box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE) ==
         CUDA_SUCCESS;
}
// The same for fp32 results, in slabs of 32 columns by 32 rows.
inline bool product_map_f32(CUtensorMap* m, const void* base, int rows, int cols, int64_t ld, int64_t apart, int batch) {
  const uint64_t gdim[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)batch};
  const uint64_t gstride[2] = {(uint64_t)ld * 4, (uint64_t)apart * 4};
  const uint32_t box[3] = {32, 32, 1};
  return mt_host::encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, gdim, gstride, box,
                               CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}
// Box heights of an operand: the tile's rows where K is contiguous, K steps
// else. Fewer rows of A than a tile has are loaded alone: what lies behind
// them in the ring is never zeroed and makes rows of D that nobody reads. A
// shallow K's rows are loaded to the next whole 16, as deep as the MMAs then
// go. (Boxes that TMA has to fill with zeros cost time: 128256 x 4096
// times 7 rows took 248 us, times 64 rows 181.)
template <class C>
int k_box(int K) { return C::SHALLOW ? std::min(64, (K + 15) / 16 * 16) : 64; }
template <class C>
int a_box(int M, int K) { return C::A_MN ? k_box<C>(K) : C::PAIR ? C::BM : std::min(C::BM, (M + 7) / 8 * 8); }
template <class C>
int b_box(int K) { return C::B_MN ? k_box<C>(K) : C::B_ROWS; }

template <class C>
ProductShape product_shape(int M, int N, int K, int batch) {
  ProductShape s;
  s.M = M;
  s.N = N;
  s.K = K;
  s.batch = batch;
  s.a_rows = C::A_MN ? C::BM : a_box<C>(M, K);
  s.k_rows = k_box<C>(K);
  s.split_kb = 0;
  s.num_m = (M + C::TM - 1) / C::TM;
  s.num_n = (N + C::BN - 1) / C::BN;
  s.tiles = C::SYM ? s.num_m * (s.num_m + 1) / 2 : s.num_m * s.num_n;
  // the rows of A that a sweep over the columns shares stay in L2: 32 MB, as measured for the layers' products
  const size_t band = (size_t)C::TM * K * 2;
  s.group_m = (int)std::min<size_t>(s.num_m, std::max<size_t>(1, ((size_t)32 << 20) / band));
  return s;
}

template <class C, class E>
cudaError_t launch_product(const CUtensorMap& a, const CUtensorMap& b, const ProductShape& s,
                           const typename E::Args& args, cudaStream_t st) {
  auto kern = product_kernel<C, E>;
  constexpr int smem = ProductSmem<C, E>::TOTAL;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t all = (int64_t)s.tiles * s.batch;
  const int sms = mt_host::num_sms();
  const int grid = C::PAIR ? 2 * (int)std::min<int64_t>(all, std::max(1, sms / 2)) : (int)std::min<int64_t>(all, sms);
  e = mt_host::launch_early(kern, grid, 64 + 32 * E::WARPS, smem, st, C::PAIR ? 2 : 1, a, b, s, args);
  count_launches(1);
  return e;
}

template <class C, class E, int S>
cudaError_t launch_split(const CUtensorMap& a, const CUtensorMap& b, const ProductShape& s,
                         const typename E::Args& args, cudaStream_t st) {
  auto kern = product_split_kernel<C, E, S>;
  constexpr int smem = SplitSmem::STAGES * C::STAGE_BYTES + 4 * SplitSmem::PART + 1024 + 128;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = mt_host::launch_early(kern, s.tiles * s.batch * S, 192, smem, st, S, a, b, s, args);
  count_launches(1);
  return e;
}

}  // namespace mt
