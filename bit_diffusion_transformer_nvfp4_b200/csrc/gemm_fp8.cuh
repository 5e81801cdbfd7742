// gemm_fp8.cuh -- the FP8 linear layer: E4M3 codes of both operands with one
// fp32 scale per row of each, and bias, activation and residual in the
// epilogue,
//   Y[m,n] = bf16( act( s_a[m] s_w[n] sum_k dec(A[m,k]) dec(W[n,k]) + bias[n] ) + R[m,n] ).
// The scales are constant along k, so the products run on the codes as they
// are (tcgen05.mma kind::f8f6f4, fp32 accumulation in TMEM) and the scales
// multiply the finished sum.
//
// Two kernels:
//   gemm_fp8_pair_kernel   many rows: persistent CTA pairs, 256 x BN tiles.
//                          Bound by the FP8 tensor pipe (81 % active under
//                          ncu) and its power: 4608 x 6144 x 6144 118 us (2940
//                          TFLOP/s) a few at a time, 145 us in a long run.
//                          One wave of tiles is bound by L2, some 50 bytes a
//                          cycle and SM (256 x 256: 625 cycles a K step of
//                          512 in the pipe), and by 5 us of beginning and end.
//   gemm_fp8_small_kernel  few rows: bound by streaming the weight once, so
//                          the weight rows are the 128-row operand, the
//                          tokens the narrow one, K is split over a cluster
//                          and the partial sums meet in shared memory.  One
//                          token times 36864 x 6144: 38.2 us, 5.93 TB/s.
#pragma once

#include "attention.cuh"
#include "gemm.cuh"
#include "sm100_warp.cuh"

namespace w4a4 {

struct Fp8GemmParams {
  int M, N, K;
  int m_group;               // row tiles swept together over all columns (pair kernel)
  const float* s_a;
  int s_a_step;              // 1: one scale per row of A, 0: one for all
  const float* s_w;
  const __nv_bfloat16* bias; // or nullptr
  const __nv_bfloat16* R;    // or nullptr
  __nv_bfloat16* Y;
  int64_t ldr, ldy;
  int epi;
  int* status;
};

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ------------------------------------------------------------------ many rows
// Two SMs share a 256 x BN tile; each CTA loads its 128 rows of A and BN / 2
// rows of W per 128-deep K step (128-byte swizzled boxes; past the end of K
// TMA fills zeros).  TMEM holds two accumulators, so the epilogue of a tile
// runs under the next tile's products.  Warp 0 TMA producer, warp 1 TMEM
// owner and (even CTA) MMA issuer, warps 2-3 spare, warps 4-11 epilogue: a
// warp owns 32 rows x BN / 2 columns and a staging box of 32 x 32 bf16 per 32
// columns, which receives the residual by TMA while the products run, is
// overwritten in place and leaves by a TMA store.
template <int BN_, int STAGES_>
struct Fp8PairCfg {
  static constexpr int BN = BN_, BH = BN / 2, STAGES = STAGES_;
  static constexpr int BM = 128, BK = 128;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BH * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int NUM_ACC = 2;
  static constexpr int TMEM_COLS = NUM_ACC * BN;
  static constexpr int EPI_WARPS = 8, EPI_WARP0 = 4;
  static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int HALF = BN / 2, BOXES = HALF / 32;
  static constexpr int BOX_BYTES = 32 * 64;
  static constexpr int EPI_BYTES = EPI_WARPS * BOXES * BOX_BYTES;
  static constexpr int BAR_BYTES = (8 * (2 * STAGES + 2 * NUM_ACC + EPI_WARPS + 1) + 8 + 127) / 128 * 128;
  static constexpr int SMEM = STAGE_BYTES * STAGES + EPI_BYTES + BAR_BYTES + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "TMEM budget");
  static_assert(HALF % 32 == 0 && STAGE_BYTES % 1024 == 0, "tile shape");
};

constexpr long long kFp8SettleCycles = 1 << 18;  // some 0.1 ms

// Tile `tile` of a product in row and column tiles: groups of `group` row
// tiles, each swept over all columns with the row tiles fastest, so that a
// group's rows of A stay in L2 while W streams past them.
__device__ __forceinline__ void fp8_tile_at(int tile, int m_tiles, int n_tiles, int group, int& m, int& n) {
  const int g = tile / (group * n_tiles), r = tile - g * group * n_tiles;
  const int rows = min(group, m_tiles - g * group);
  n = r / rows;
  m = g * group + r - n * rows;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                         const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_y,
                         const Fp8GemmParams p) {
  constexpr int BN = C::BN, STAGES = C::STAGES;
  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi_smem = smem + C::STAGE_BYTES * STAGES;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi_smem + C::EPI_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + C::NUM_ACC;
  uint64_t* res_full = acc_empty + C::NUM_ACC;  // [EPI_WARPS] the warp's residual boxes have landed
  uint64_t* drain = res_full + C::EPI_WARPS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < C::NUM_ACC; ++a) {
      mbar_init(smem_u32(&acc_full[a]), 1);
      mbar_init(smem_u32(&acc_empty[a]), 2 * C::EPI_WARPS);
    }
    for (int w = 0; w < C::EPI_WARPS; ++w) mbar_init(smem_u32(&res_full[w]), 1);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_y);
    if (p.R != nullptr) tma_prefetch_desc(&tm_r);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();

  const int m_tiles = (p.M + 2 * C::BM - 1) / (2 * C::BM);
  const int n_tiles = (p.N + BN - 1) / BN;
  const int total = m_tiles * n_tiles;
  const int nkb = (p.K + C::BK - 1) / C::BK;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ A/W producer (both CTAs)
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += pairs) {
        int tm, tn;
        fp8_tile_at(tile, m_tiles, n_tiles, p.m_group, tm, tn);
        const int m0 = tm * 2 * C::BM + static_cast<int>(rank) * C::BM;
        const int n0 = tn * BN + static_cast<int>(rank) * C::BH;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(smem_u32(&empty[s]), ((it / STAGES) & 1) ^ 1, abort_flag, p.status)) { ok = false; break; }
          uint8_t* st = smem + s * C::STAGE_BYTES;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * C::STAGE_BYTES);
          tma_load_2d_pair(smem_u32(st), &tm_a, bar, kb * C::BK, m0);
          tma_load_2d_pair(smem_u32(st + C::A_BYTES), &tm_w, bar, kb * C::BK, n0);
        }
      }
      // the even CTA's ring barriers count both CTAs' bytes: the newest fills
      // land before the shared memory goes away
      if (leader) {
        const uint32_t first = it > static_cast<uint32_t>(STAGES) ? it - STAGES : 0u;
        for (uint32_t j = first; j < it; ++j) mbar_wait_drain(smem_u32(&full[j % STAGES]), (j / STAGES) & 1);
      } else if (!ok) {
        // after a wait that gave up the even CTA may not have counted this one's
        // newest fills: the time in which any copy lands
        const long long start = clock64();
        while (clock64() - start < kFp8SettleCycles) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // (the whole warp in uniform control flow, one elected lane issuing)
    if (leader) {
      constexpr uint32_t kIdesc = idesc_e4m3(256, BN);
      const uint64_t a_desc = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t w_desc = smem_desc(smem_u32(smem + C::A_BYTES), 16, 1024, kSwizzle128B);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += pairs, ++tcount) {
        const uint32_t acc = tcount % C::NUM_ACC;
        if (!(ok = mbar_wait_warp(smem_u32(&acc_empty[acc]), ((tcount / C::NUM_ACC) & 1) ^ 1, abort_flag, p.status)))
          break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % STAGES;
          if (!(ok = mbar_wait_warp(smem_u32(&full[s]), (it / STAGES) & 1, abort_flag, p.status))) break;
          tc_fence_after();
          const uint64_t ad = a_desc + s * (C::STAGE_BYTES >> 4), wd = w_desc + s * (C::STAGE_BYTES >> 4);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < C::BK / 32; ++j)
              mma_e4m3_pair(d, ad + (32 * j >> 4), wd + (32 * j >> 4), kIdesc, (kb > 0 || j > 0) ? 1u : 0u);
            tc_commit_pair_mc(smem_u32(&empty[s]), 0x3);
            if (kb == nkb - 1) tc_commit_pair_mc(smem_u32(&acc_full[acc]), 0x3);
          }
          __syncwarp();
        }
      }
      if (elect_one()) tc_commit_pair(smem_u32(drain));
      __syncwarp();
      mbar_wait_drain(smem_u32(drain), 0);
      // the other CTA's last arrivals are in before this one may go
      for (uint32_t t = tcount > C::NUM_ACC ? tcount - C::NUM_ACC : 0u; ok && t < tcount; ++t)
        ok = mbar_wait_warp(smem_u32(&acc_empty[t % C::NUM_ACC]), (t / C::NUM_ACC) & 1, abort_flag, p.status);
    }
  } else if (warp >= C::EPI_WARP0) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int ew = warp - C::EPI_WARP0;
    const int q = warp & 3;    // TMEM lane quarter: rows 32q .. 32q+31 of this CTA
    const int h = ew >> 2;     // column half
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint8_t* boxes = epi_smem + ew * C::BOXES * C::BOX_BYTES;
    const uint32_t res_bar = smem_u32(&res_full[ew]);
    uint32_t loads = 0, used = 0;  // residual fills asked for and waited for
    auto load_residual = [&](int tile) {
      int tm, tn;
      fp8_tile_at(tile, m_tiles, n_tiles, p.m_group, tm, tn);
      const int row0 = tm * 2 * C::BM + static_cast<int>(rank) * C::BM + q * 32;
      const int n0 = tn * BN + h * C::HALF;
      if (lane == 0) {
        mbar_arrive_expect_tx(res_bar, C::BOXES * C::BOX_BYTES);
#pragma unroll
        for (int c = 0; c < C::BOXES; ++c)
          tma_load_2d(smem_u32(boxes + c * C::BOX_BYTES), &tm_r, res_bar, n0 + 32 * c, row0);
      }
      ++loads;
    };
    // Scales and biases of 32 columns (the same for every lane), asked for a
    // box ahead: under the products, then under the previous box's stores
    // (asked for where they are used, each group of eight waits for L2: 2000
    // cycles a box; handed round by shuffles 950; this way 570).
    // (columns past N read the last ones'; the store drops their outputs)
    float4 sw[8];
    uint4 bw[4] = {};
    auto load_columns = [&](int n) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4* w = reinterpret_cast<const float4*>(p.s_w + min(n + 8 * g, p.N - 8));
        sw[2 * g] = __ldg(w);
        sw[2 * g + 1] = __ldg(w + 1);
      }
      if (p.bias != nullptr) {
#pragma unroll
        for (int g = 0; g < 4; ++g) bw[g] = __ldg(reinterpret_cast<const uint4*>(p.bias + min(n + 8 * g, p.N - 8)));
      }
    };
    if (p.R != nullptr && pair < total) load_residual(pair);
    uint32_t tcount = 0;
    for (int tile = pair; tile < total; tile += pairs, ++tcount) {
      int tm, tn;
      fp8_tile_at(tile, m_tiles, n_tiles, p.m_group, tm, tn);
      const int row0 = tm * 2 * C::BM + static_cast<int>(rank) * C::BM + q * 32;
      const int n0 = tn * BN + h * C::HALF;
      const uint32_t acc = tcount % C::NUM_ACC;
      // (rows past M read the last row's scale; the store drops their outputs)
      const float sa = __ldg(p.s_a + static_cast<int64_t>(min(row0 + lane, p.M - 1)) * p.s_a_step);
      load_columns(n0);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[acc]), (tcount / C::NUM_ACC) & 1, abort_flag,
                                             p.status)))
        break;
      tc_fence_after();
      if (p.R != nullptr) {
        if (!__all_sync(0xffffffffu, mbar_wait(res_bar, used & 1, abort_flag, p.status))) break;
        ++used;
      } else if (tcount > 0) {
        // the previous tile's stores have read their boxes
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
      }
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + h * C::HALF;
#pragma unroll 1
      for (int c = 0; c < C::BOXES; ++c) {
        uint32_t r[32];
        tmem_ld_32cols(taddr + 32 * c, r);
        tmem_ld_wait();
        if (c == C::BOXES - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8 * acc);
        }
        uint8_t* box = boxes + c * C::BOX_BYTES;
        const int n = n0 + 32 * c;
        float y[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b0 = j & 1 ? bw[j >> 1].z : bw[j >> 1].x, b1 = j & 1 ? bw[j >> 1].w : bw[j >> 1].y;
          y[4 * j] = fmaf(__uint_as_float(r[4 * j]) * sa, sw[j].x, bf16_lo(b0));
          y[4 * j + 1] = fmaf(__uint_as_float(r[4 * j + 1]) * sa, sw[j].y, bf16_hi(b0));
          y[4 * j + 2] = fmaf(__uint_as_float(r[4 * j + 2]) * sa, sw[j].z, bf16_lo(b1));
          y[4 * j + 3] = fmaf(__uint_as_float(r[4 * j + 3]) * sa, sw[j].w, bf16_hi(b1));
        }
        if (c + 1 < C::BOXES) load_columns(n + 32);
        if (p.epi == 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = gelu_tanh_f32(y[j]);
        }
        uint4* line = reinterpret_cast<uint4*>(box + lane * 64);
        const int flip = (lane >> 1) & 3;  // the box's 64-byte swizzle
        if (p.R != nullptr) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint4 rr = line[g ^ flip];
            const uint32_t rs[4] = {rr.x, rr.y, rr.z, rr.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[8 * g + 2 * j] += bf16_lo(rs[j]);
              y[8 * g + 2 * j + 1] += bf16_hi(rs[j]);
            }
          }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
          line[g ^ flip] = make_uint4(pack_bf16x2(y[8 * g], y[8 * g + 1]), pack_bf16x2(y[8 * g + 2], y[8 * g + 3]),
                                      pack_bf16x2(y[8 * g + 4], y[8 * g + 5]), pack_bf16x2(y[8 * g + 6], y[8 * g + 7]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_y, smem_u32(box), n, row0);
          bulk_commit_group();
        }
      }
      if (p.R != nullptr && tile + pairs < total) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        load_residual(tile + pairs);
      }
    }
    // no residual fill may still be landing, no store still be reading
    if (lane == 0) {
      for (; used < loads; ++used) mbar_wait_drain(res_bar, used & 1);
      bulk_wait_group_all();
    }
    __syncwarp();
  }

  tc_fence_before();
  cluster_meet();  // no CTA leaves while its peer may still signal it or read its TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------ few rows
// At most TN tokens: the weight is read once and nothing else matters, so its
// rows are the MMA's 128-row operand and the tokens its N.  A CTA takes 128
// weight rows and one of gridDim.y / cluster-many slices of K, streams them
// through a TMA ring (two CTAs an SM keep about 180 KB in flight), and leaves
// its fp32 sums [token][weight row] in shared memory; after a cluster barrier
// every CTA of the cluster adds up its share of the tokens over the slices, in
// slice order, and writes them.  128 threads: warp 0 TMA producer and TMEM
// owner, warp 1 MMA issuer, all four warps the epilogue (one weight row a
// thread).
template <int TN_, int STAGES_>
struct Fp8SmallCfg {
  static constexpr int TN = TN_, STAGES = STAGES_, BM = 128, BK = 128;
  static constexpr int W_BYTES = BM * BK, X_BYTES = TN * BK, STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int TMEM_COLS = TN < 32 ? 32 : TN;
  static constexpr int THREADS = 128;
  static constexpr int PART_BYTES = TN * BM * 4;  // reuses the ring
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
  static constexpr int BAR_BYTES = (8 * (2 * STAGES + 1) + 8 + 127) / 128 * 128;
  static constexpr int SMEM = RING_BYTES + BAR_BYTES + 1024;
  static_assert(PART_BYTES <= RING_BYTES, "the partial sums fit the ring");
  static_assert(STAGE_BYTES % 1024 == 0 && SMEM <= 113 * 1024, "two CTAs per SM");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 2)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                          const Fp8GemmParams p) {
  constexpr int STAGES = C::STAGES;
  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const int splits = gridDim.x;               // the cluster spans the K slices of one weight tile
  const int split = blockIdx.x;
  const int n0 = blockIdx.y * C::BM;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();

  // K steps [k0, k1): the slices differ by one step at most (the launch never
  // has more slices than steps)
  const int nkb = (p.K + C::BK - 1) / C::BK;
  const int k0 = static_cast<int>(static_cast<int64_t>(nkb) * split / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(nkb) * (split + 1) / splits);
  const int steps = k1 - k0;
  if (warp == 0 && lane == 0) {
    int it = 0;
    for (; it < steps; ++it) {
      const int s = it % STAGES;
      if (!mbar_wait(smem_u32(&empty[s]), ((it / STAGES) & 1) ^ 1, abort_flag, p.status)) break;
      uint8_t* st = smem + s * C::STAGE_BYTES;
      const uint32_t bar = smem_u32(&full[s]);
      mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
      tma_load_2d(smem_u32(st), &tm_w, bar, (k0 + it) * C::BK, n0);
      tma_load_2d(smem_u32(st + C::W_BYTES), &tm_x, bar, (k0 + it) * C::BK, 0);
    }
    for (int j = max(0, it - STAGES); j < it; ++j) mbar_wait_drain(smem_u32(&full[j % STAGES]), (j / STAGES) & 1);
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = idesc_e4m3(C::BM, C::TN);
    const uint64_t w_desc = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t x_desc = smem_desc(smem_u32(smem + C::W_BYTES), 16, 1024, kSwizzle128B);
    for (int it = 0; it < steps; ++it) {
      const uint32_t s = it % STAGES;
      if (!mbar_wait_warp(smem_u32(&full[s]), (it / STAGES) & 1, abort_flag, p.status)) break;
      tc_fence_after();
      const uint64_t wd = w_desc + s * (C::STAGE_BYTES >> 4), xd = x_desc + s * (C::STAGE_BYTES >> 4);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < C::BK / 32; ++j)
          mma_e4m3(tmem, wd + (32 * j >> 4), xd + (32 * j >> 4), kIdesc, (it > 0 || j > 0) ? 1u : 0u);
        tc_commit(smem_u32(&empty[s]));
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(smem_u32(done));  // completes once every MMA above has, abort or not
  }
  __syncwarp();
  // the outputs' column scales and biases (four weight rows a lane), under the products
  const int n = n0 + 4 * lane;
  float4 sw = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  uint2 bw = make_uint2(0u, 0u);
  if (n < p.N) {  // N % 8 == 0: all four are valid
    sw = __ldg(reinterpret_cast<const float4*>(p.s_w + n));
    if (p.bias != nullptr) bw = __ldg(reinterpret_cast<const uint2*>(p.bias + n));
  }
  const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(done), 0, abort_flag, p.status));
  if (!ok) mbar_wait_drain(smem_u32(done), 0);
  tc_fence_after();
  // every fill has landed and been read: the ring now holds the partial sums
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);  // [token][128 weight rows]
  const int row = threadIdx.x;                    // weight row of the tile, and TMEM lane
#pragma unroll 1
  for (int c = 0; c < C::TN && c < p.M; c += 16) {
    uint32_t r[16];
    tmem_ld_16cols(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) part[(c + j) * C::BM + row] = ok ? __uint_as_float(r[j]) : 0.0f;
  }
  cluster_sync();
  // Outputs: a token per warp, four weight rows a lane.  Two tokens at a time,
  // all their partial sums asked for before the first is added (one load
  // after the other, a row a thread, took 128 tokens 12 us).
  if (ok && n < p.N) {
    const uint32_t mine = smem_u32(part + 4 * lane);
    const int stride = 4 * splits;  // tokens from one of a warp's to its next
    for (int m0 = split + warp * splits; m0 < p.M; m0 += 2 * stride) {
      float4 v[2][8];
      float sa[2];
      uint2 res[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = m0 + i * stride;
        const bool on = m < p.M;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          v[i][s] = on && s < splits ? ld_cluster_f32x4(mapa_shared(mine + static_cast<uint32_t>(m) * C::BM * 4,
                                                                    static_cast<uint32_t>(s)))
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        sa[i] = on ? __ldg(p.s_a + static_cast<int64_t>(m) * p.s_a_step) : 0.0f;
        // (a plain load: Y may be the residual itself)
        res[i] = on && p.R != nullptr ? *reinterpret_cast<const uint2*>(p.R + static_cast<int64_t>(m) * p.ldr + n)
                                      : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = m0 + i * stride;
        if (m >= p.M) break;
        float4 acc = v[i][0];
#pragma unroll
        for (int s = 1; s < 8; ++s) {  // in slice order; zeros past the last
          acc.x += v[i][s].x;
          acc.y += v[i][s].y;
          acc.z += v[i][s].z;
          acc.w += v[i][s].w;
        }
        float y[4] = {fmaf(acc.x * sa[i], sw.x, bf16_lo(bw.x)), fmaf(acc.y * sa[i], sw.y, bf16_hi(bw.x)),
                      fmaf(acc.z * sa[i], sw.z, bf16_lo(bw.y)), fmaf(acc.w * sa[i], sw.w, bf16_hi(bw.y))};
        if (p.epi == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = gelu_tanh_f32(y[e]);
        }
        *reinterpret_cast<uint2*>(p.Y + static_cast<int64_t>(m) * p.ldy + n) =
            make_uint2(pack_bf16x2(y[0] + bf16_lo(res[i].x), y[1] + bf16_hi(res[i].x)),
                       pack_bf16x2(y[2] + bf16_lo(res[i].y), y[3] + bf16_hi(res[i].y)));
      }
    }
  }
  tc_fence_before();
  cluster_meet();  // the peers have read this CTA's partial sums
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace w4a4
