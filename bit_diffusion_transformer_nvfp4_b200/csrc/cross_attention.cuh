// cross_attention.cuh -- bf16 attention of one token sequence to another of
// its own length (an encoder's states), on the sm_100a tensor cores.
//
// Per query row and head, over the keys j that the length and the key mask
// leave:  o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),
// c = scale log2 e, the sums and the running offset m in fp32; a row without
// keys gives 0.  m moves only when a half tile's maximum passes it by more
// than kXSlack binades (the accumulator and the sum are then rescaled), which
// is exact: numerator and denominator share the offset, the rounded product of
// c and the largest score.  Where that rounding would be a binade (from |m| =
// kXLarge up) the exponents are c times the scores' differences instead
// (xattn_ahead).  The probabilities are rounded to bf16 for the second product,
// at most 2^-8 each, random in sign, against the same bound of the output's own
// rounding.
//
// A work tile is 128 rows of one key/value head: queries times the heads that
// share it (the largest power of two of them, so that a group of heads reads
// its keys once), loaded by one 4-D TMA box whose row order is token-major.
// S = Q K^T and O += P V are tcgen05.mma kind::f16 with both accumulators in
// TMEM; P goes back into S's columns as the A operand of the second product,
// V is its MN-major B operand as it lies in memory.
//
// A stream of softmax (a warpgroup, one row a thread) takes a 128-key tile in
// two halves of 64 with a score buffer each: when a half's probabilities are
// there its product goes out, and behind it the next tile's scores for the
// same buffer, so that scores are always ahead.  The issuing thread's MMAs run
// in order: the scores may follow the product that reads the buffer, and one
// commit covers both.  Measured on 16384 queries, 4096 keys, 16 heads of 128:
// one buffer of 128 keys a stream 440 us (the softmax, 1800 cycles a tile, and
// the MMAs, 1600 with their latency, in turn), this 427 us although the
// narrower scores cost the pipe more (128 x 64 x 16: 48 cycles from shared
// memory where 128 x 128 x 16 takes 64); two threads a row, with one buffer,
// 449 us (a barrier between their halves).
//
// Roles (512 threads): a warp each for loading keys and values, loading
// queries (a query tile waits for the scores of the tile before and would hold
// up the keys behind it) and issuing each stream's MMAs; two softmax
// warpgroups; an epilogue warpgroup that normalises and stores a finished tile
// under the next one.
//
// Two forms:
//   SPLIT = false  many rows: the streams are two row tiles over the same keys,
//                  persistent CTAs, one per SM.  Bound by the tensor pipe and
//                  the exponentials in turn (57 and 50 % of the active cycles
//                  under ncu), at full load by the power cap: 16384 queries x
//                  4096 keys, 16 heads of 128, 1150 to 1240 TFLOP/s in runs of
//                  3 ms, 1075 sustained, against 1646 and 1388 measured for a
//                  large matrix product.
//   SPLIT = true   few rows: the streams are the even and odd key tiles of one
//                  row tile, and a cluster of CTAs splits the keys; the
//                  partial sums meet in (distributed) shared memory.  Bound by
//                  the key and value bytes and about 7 us of latency (4 x 1
//                  query, 4109 keys, 32 heads on 8: 17.1 us, 3.94 TB/s).
#pragma once

#include "attention.cuh"
#include "sm100_warp.cuh"
#include "xattn_ring.h"

namespace w4a4 {

constexpr int kXTile = 128;       // rows per stream, keys of a ring slot
constexpr int kXSub = 64;         // keys of a score buffer
constexpr int kXThreads = 512;    // control warpgroup, a softmax warpgroup a stream, epilogue warpgroup
constexpr float kXSlack = 8.0f;   // binades a tile's maximum may pass the offset
constexpr float kXLarge = 0x1p24f;  // offsets up to here are rounded (by half a binade at most)
constexpr int kXChunk = 16;       // scores taken together through the exponential
// Of 16 pairs of exponentials, how many on the FMA pipes instead of the MUFU
// (0, 2, 4 and 6: 443, 427, 425 and 428 us on the long case; fewer take less power).
constexpr int kXPolyPairs = 2;
constexpr int kXRegsCtrl = 80, kXRegsSoftmax = 168, kXRegsEpi = 96;  // of 128 at launch
static_assert(128 * (kXRegsCtrl + kXRegsEpi) + 256 * kXRegsSoftmax <= kXThreads * 128,
              "register budgets fit the launch allocation");

struct XAttnParams {
  int Sq, Skv, heads, kv_heads, D;
  int pack;                 // heads of a group that share a row tile (power of two <= 32)
  int batch, kv_batch;
  int row_tiles;            // work tiles along the queries (128 or 256 rows each)
  int tiles;                // work tiles in all
  int head_blocks;          // heads / pack
  int step, step_rt, step_hb, step_b;  // tiles from one of a CTA's to its next, and the same as a decoded tile
  uint32_t hb_magic;        // hb / (head blocks of a key/value head) = umulhi(hb, hb_magic); 0 for a divisor of 1
  const int* kv_len;        // [kv_batch] or nullptr
  const uint8_t* key_mask;  // [kv_batch, ld_mask] or nullptr; 0: not attended to
  int64_t ld_mask;
  float scale;
  __nv_bfloat16* O;
  int64_t ldo;
  int* status;
};

template <int DB_, bool SPLIT_>
struct XAttnCfg {
  static constexpr int DB = DB_;           // 64-column blocks of a head
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int TILE_BYTES = DB * kXTile * 128;  // 128 rows of a head
  static constexpr int NQ = SPLIT ? 1 : 2;              // query tiles held
  static constexpr int SLOTS = (SPLIT ? 12 : 8) / DB;   // ring of key and value tiles
  static constexpr int RINGS = SPLIT ? 2 : 1;           // one for both streams, or one each
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = NQ * TILE_BYTES;
  static constexpr int O_OFF = KV_OFF + SLOTS * TILE_BYTES;
  static constexpr int O_BYTES = SPLIT ? 0 : 8 * 32 * 128;       // two 32 x 64 bf16 boxes per epilogue warp
  static constexpr int PART_PITCH = DB * 64 + 4;                 // floats; SPLIT: over Q and the ring
  static constexpr int STAT_OFF = 2 * kXTile * PART_PITCH * 4;   // behind them m, l and x, [2 streams][3][128]
  static constexpr int F_OFF = O_OFF + O_BYTES;                  // the rows' final factors, [2 streams][128]
  static constexpr int BAR_OFF = F_OFF + (SPLIT ? 0 : 2 * kXTile * 4);
  static constexpr int BARS = 2 * SLOTS + 2 * 10;
  static constexpr int SMEM = BAR_OFF + 8 * BARS + 8;  // (no slack: the kernel checks its base)
  static constexpr int TMEM_COLS = 512;
  static constexpr int O_COL = 256;        // S of stream t at 128 t, O at 256 + 128 t
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SLOTS % RINGS == 0, "rings of equal size");
  static_assert(!SPLIT || STAT_OFF + 6 * kXTile * 4 <= O_OFF, "the partial sums fit over Q and the ring");
};

// D(tmem) (+)= A(tmem) * B(smem), bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// max(a, b, c), NaN if any of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The factor of a row's sums at the end: 1 / l, 0 for a row without keys
// (whose largest score is still -infinity), NaN where l is.
__device__ __forceinline__ float xattn_factor(float x, float l) {
  return x == -INFINITY && l == l ? 0.0f : 1.0f / l;
}

// Offsets.  A row whose largest score is x has the offset m = c x, rounded to
// fp32 up to kXLarge and taken as the exact product beyond: there its rounding
// would be a binade and more, and 2^(c s - m) would leave fp32's range from
// |m| = 2^31 on.
__device__ __forceinline__ bool xattn_large(float m) { return !(fabsf(m) <= kXLarge); }

// The offset of largest score a less that of b, rounded once.
__device__ __forceinline__ float xattn_ahead(float a, float b, float c) {
  const float ma = __fmul_rn(a, c), mb = __fmul_rn(b, c);  // (as the offsets were: never fused)
  if (xattn_large(ma)) return xattn_large(mb) ? (a - b) * c : fmaf(a, c, -mb);
  return xattn_large(mb) ? fmaf(-b, c, ma) : ma - mb;
}

// What a work tile index stands for.
struct XTileAt {
  int row0;  // first row (token-major, `pack` heads a token) of the tile's first stream
  int h0;    // first query head
  int hk;    // key/value head
  int b, kb; // sequence and its key/value batch
  int len;   // keys
};

// A role's walk over a CTA's work tiles, gridDim.x apart in the persistent
// form.  Only the first is decoded by division; each tile's key length is
// loaded a tile ahead (with five divisions and the load in every tile a
// batch of short prompts took 86.7 us, this way 84.5).
struct XWalk {
  int tile, rt, hb, b;  // work tile: row tile, head block, sequence
  int len, len1;        // its key length as loaded, and that of the tile behind

  __device__ __forceinline__ int load(const XAttnParams& p, int seq) const {
    return p.kv_len != nullptr && seq < p.batch ? p.kv_len[p.kv_batch == 1 ? 0 : seq] : p.Skv;
  }
  // (row tile, head block, sequence) of the tile behind
  __device__ __forceinline__ void behind(const XAttnParams& p, int& rt1, int& hb1, int& b1) const {
    rt1 = rt + p.step_rt;
    hb1 = hb + p.step_hb;
    b1 = b + p.step_b;
    if (rt1 >= p.row_tiles) {
      rt1 -= p.row_tiles;
      ++hb1;
    }
    if (hb1 >= p.head_blocks) {
      hb1 -= p.head_blocks;
      ++b1;
    }
  }
  __device__ __forceinline__ void look_ahead(const XAttnParams& p) {
    int rt1, hb1, b1;
    behind(p, rt1, hb1, b1);
    len1 = load(p, b1);
  }
  __device__ __forceinline__ XWalk(const XAttnParams& p, int first) : tile(first) {
    rt = first % p.row_tiles;
    const int heads = first / p.row_tiles;
    hb = heads % p.head_blocks;
    b = heads / p.head_blocks;
    len = load(p, b);
    look_ahead(p);
  }
  __device__ __forceinline__ bool live(const XAttnParams& p) const { return tile < p.tiles; }
  __device__ __forceinline__ void next(const XAttnParams& p) {
    behind(p, rt, hb, b);
    tile += p.step;
    len = len1;
    look_ahead(p);
  }
  __device__ __forceinline__ int keys(const XAttnParams& p) const { return min(max(len, 0), p.Skv); }
  __device__ __forceinline__ XTileAt at(const XAttnParams& p, int rows) const {
    XTileAt a;
    a.row0 = rt * rows;
    a.h0 = hb * p.pack;
    a.hk = static_cast<int>(p.hb_magic != 0 ? __umulhi(static_cast<uint32_t>(hb), p.hb_magic) : static_cast<uint32_t>(hb));
    a.b = b;
    a.kb = p.kv_batch == 1 ? 0 : b;
    a.len = keys(p);
    return a;
  }
};

// Key tiles [j0, j1) of `len` keys that fall to one of `splits` CTAs.
__device__ __forceinline__ void xattn_key_range(int len, int split, int splits, int& j0, int& j1) {
  const int n = (len + kXTile - 1) / kXTile;
  j0 = static_cast<int>(static_cast<int64_t>(n) * split / splits);
  j1 = static_cast<int>(static_cast<int64_t>(n) * (split + 1) / splits);
}

template <class C>
__global__ void __launch_bounds__(kXThreads, 1)
    cross_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                           const XAttnParams p) {
  constexpr int DB = C::DB, SLOTS = C::SLOTS;
  constexpr bool SPLIT = C::SPLIT;
  constexpr int kRows = SPLIT ? kXTile : 2 * kXTile;  // rows of a work tile
  grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    // the swizzled tiles need 1024-byte alignment; every CTA sees the same
    // base, so all return here before any barrier or TMEM use
    grid_dependency_wait();
    if (threadIdx.x == 0 && p.status) atomicExch(p.status, kStatusMisaligned);
    return;
  }
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;                                 // [SLOTS]
  uint64_t* q_full = kv_empty + SLOTS;                                  // [2] query tiles (SPLIT: the first)
  uint64_t* q_empty = q_full + 2;                                       // [2] the tile's last scores are done
  uint64_t* s_full = q_empty + 2;                                       // [2][2] per stream and buffer: scores
  uint64_t* p_full = s_full + 4;                                        // [2][2] probabilities, O rescaled
  uint64_t* o_done = p_full + 4;                                        // [2] the tile's last product is done
  uint64_t* f_full = o_done + 2;                                        // [2] its rows' factors are there
  uint64_t* o_free = f_full + 2;                                        // [2] its sums and factors have been read
  uint64_t* drain = o_free + 2;                                         // [2] the issuers' last commits
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), SPLIT ? 1 : 2);  // the streams that read the slot
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&q_full[t]), 1);
      mbar_init(smem_u32(&q_empty[t]), 1);
      for (int w = 0; w < 2; ++w) {
        mbar_init(smem_u32(&s_full[2 * t + w]), 1);
        mbar_init(smem_u32(&p_full[2 * t + w]), 4);
      }
      mbar_init(smem_u32(&o_done[t]), 1);
      mbar_init(smem_u32(&f_full[t]), 4);
      mbar_init(smem_u32(&o_free[t]), 4);
    }
    for (int t = 0; t < 2; ++t) mbar_init(smem_u32(&drain[t]), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (!SPLIT) tma_prefetch_desc(&tm_o);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();

  // this CTA's work tiles: first, first + step, ...; SPLIT: one tile, of whose
  // key tiles it takes the cluster rank's share
  const int splits = SPLIT ? static_cast<int>(gridDim.x) : 1;
  const int split = SPLIT ? static_cast<int>(blockIdx.x) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.x);

  if (warp < 4) {
    regs_release_to<kXRegsCtrl>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- keys and values
      uint32_t fills[2] = {0u, 0u};
      bool ok = true;
      auto load = [&](const CUtensorMap* map, const XTileAt& a, int j, int ring_of) {
        const XRing ring = xattn_ring(SLOTS, C::RINGS, ring_of);
        uint32_t& fill = fills[ring_of];
        const uint32_t s = ring.slot(fill);
        if (!ok || !(ok = mbar_wait(smem_u32(&kv_empty[s]), ring.parity(fill) ^ 1, abort_flag, p.status))) return;
        const uint32_t bar = smem_u32(&kv_full[s]);
        mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
        for (int d = 0; d < DB; ++d)
          tma_load_4d(smem_u32(smem + C::KV_OFF + s * C::TILE_BYTES + d * (kXTile * 128)), map, bar, 64 * d, a.hk,
                      j * kXTile, a.kb);
        ++fill;
      };
      for (XWalk w(p, first); w.live(p) && ok; w.next(p)) {
        const XTileAt a = w.at(p, kRows);
        int j0, j1;
        xattn_key_range(a.len, split, splits, j0, j1);
        for (int j = j0; j < j1 && ok; j += C::RINGS) {
#pragma unroll
          for (int t = 0; t < C::RINGS; ++t)
            if (j + t < j1) load(&tm_k, a, j + t, t);
#pragma unroll
          for (int t = 0; t < C::RINGS; ++t)
            if (j + t < j1) load(&tm_v, a, j + t, t);
        }
      }
      // every fill issued lands before the shared memory is released
#pragma unroll
      for (int t = 0; t < C::RINGS; ++t) {
        const XRing ring = xattn_ring(SLOTS, C::RINGS, t);
        for (uint32_t j = fills[t] > ring.slots ? fills[t] - ring.slots : 0u; j < fills[t]; ++j)
          mbar_wait_drain(smem_u32(&kv_full[ring.slot(j)]), ring.parity(j));
      }
    } else if (warp == 3 && lane == 0) {
      // ---------------------------------------------------------- queries
      // (a thread of their own: a query tile waits for the scores of the
      // work tile before, and would hold up the keys and values behind it)
      uint32_t fills[2] = {0u, 0u};
      bool ok = true;
      for (XWalk w(p, first); w.live(p) && ok; w.next(p)) {
        const XTileAt a = w.at(p, kRows);
        int j0, j1;
        xattn_key_range(a.len, split, splits, j0, j1);
        if (j0 == j1) continue;
#pragma unroll
        for (int t = 0; t < (SPLIT ? 1 : 2); ++t) {
          if (!ok || !(ok = mbar_wait(smem_u32(&q_empty[t]), (fills[t] & 1) ^ 1, abort_flag, p.status))) break;
          const uint32_t bar = smem_u32(&q_full[t]);
          mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
          for (int d = 0; d < DB; ++d)
            tma_load_4d(smem_u32(smem + C::Q_OFF + t * C::TILE_BYTES + d * (kXTile * 128)), &tm_q, bar, 64 * d, a.h0,
                        (a.row0 + t * kXTile) / p.pack, a.b);
          ++fills[t];
        }
        if (!SPLIT && w.tile + p.step < p.tiles) {
          // the next tile's towards L2 meanwhile
          int rt1, hb1, b1;
          w.behind(p, rt1, hb1, b1);
          for (int t = 0; t < 2; ++t) {
            const int token = (rt1 * kRows + t * kXTile) / p.pack;
            if (token < p.Sq)
              for (int d = 0; d < DB; ++d) tma_prefetch_4d(&tm_q, 64 * d, hb1 * p.pack, token, b1);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (fills[t] > 0) mbar_wait_drain(smem_u32(&q_full[t]), (fills[t] - 1) & 1);
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------- MMA issuers, one a stream
      // (the whole warp in uniform control flow, one elected lane issuing)
      const int t = warp - 1;
      constexpr uint32_t kIdescS = idesc_bf16(kXTile, kXSub);
      constexpr uint32_t kIdescO = idesc_bf16(kXTile, DB * 64) | (1u << 16);  // B (the values) MN-major
      const uint32_t t_s = tmem + 128 * t, t_o = tmem + C::O_COL + 128 * t;
      const uint64_t q_desc =
          smem_desc(smem_u32(smem + C::Q_OFF + (SPLIT ? 0 : t) * C::TILE_BYTES), 16, 1024, kSwizzle128B);
      const uint64_t k_desc = smem_desc(smem_u32(smem + C::KV_OFF), 16, 1024, kSwizzle128B);
      const uint64_t v_desc = smem_desc(smem_u32(smem + C::KV_OFF), kXTile * 128, 1024, kSwizzle128B);
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait_warp(smem_u32(bar), parity & 1, abort_flag, p.status);
      };
      const XRing ring = xattn_ring(SLOTS, C::RINGS, SPLIT ? t : 0);
      auto slot_wait = [&](uint32_t fill) -> bool { return wait(&kv_full[ring.slot(fill)], ring.parity(fill)); };
      // The two halves of a key tile have a score buffer each.  As soon as
      // the probabilities of a half are there, its product goes out and behind
      // it the next key tile's scores for the same buffer: two half tiles of
      // scores are always ahead of the softmax.
      struct Next {
        bool live;       // there is a next key tile
        uint32_t fill;   // its keys
        bool new_q;      // it opens a work tile
        bool last;       // it closes one
      };
      uint32_t opened = 0;  // work tiles opened
      auto ready = [&](const Next& k) -> bool {
        return (!k.new_q || wait(&q_full[SPLIT ? 0 : t], opened)) && slot_wait(k.fill);
      };
      auto scores = [&](uint64_t kd, int h) {
#pragma unroll
        for (int i = 0; i < DB * 4; ++i)  // (columns past the head's are zeros in both)
          mma_bf16(t_s + kXSub * h, q_desc + (((i / 4) * (kXTile * 128) + 32 * (i % 4)) >> 4),
                   kd + (((i / 4) * (kXTile * 128) + 32 * (i % 4) + h * kXSub * 128) >> 4), kIdescS, i > 0 ? 1u : 0u);
      };
      auto open = [&](const Next& k) -> bool {  // the first scores of all
        if (!ready(k)) return false;
        const uint32_t k_slot = ring.slot(k.fill);
        const uint64_t kd = k_desc + k_slot * (C::TILE_BYTES >> 4);
        tc_fence_after();
        if (elect_one()) {
          scores(kd, 0);
          tc_commit(smem_u32(&s_full[2 * t]));
          scores(kd, 1);
          tc_commit(smem_u32(&s_full[2 * t + 1]));
          tc_commit(smem_u32(&kv_empty[k_slot]));
          if (k.last) tc_commit(smem_u32(&q_empty[t]));
        }
        __syncwarp();
        ++opened;
        return true;
      };
      uint32_t it = 0, summed = 0;  // key tiles done, work tiles begun
      auto advance = [&](uint32_t v_fill, bool fresh, const Next& k) -> bool {
        if (!slot_wait(v_fill)) return false;
        // the first product of a tile overwrites the sums of the one before
        if (!SPLIT && fresh && summed++ > 0 && !wait(&o_free[t], summed)) return false;
        const uint32_t v_slot = ring.slot(v_fill), k_slot = ring.slot(k.fill);
        const uint64_t vd = v_desc + v_slot * (C::TILE_BYTES >> 4);
        const uint64_t kd = k_desc + k_slot * (C::TILE_BYTES >> 4);
        const uint32_t v_bar = smem_u32(&kv_empty[v_slot]), k_bar = smem_u32(&kv_empty[k_slot]);
        const uint32_t add = fresh ? 0u : 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(&p_full[2 * t + h], it)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kXSub / 16; ++i)
              mma_bf16_ts(t_o, t_s + kXSub * h + 8 * i, vd + ((2048 * i + h * kXSub * 128) >> 4), kIdescO,
                          (h > 0 || i > 0) ? 1u : add);
            if (h == 1) tc_commit(v_bar);
          }
          __syncwarp();
          if (h == 0 && k.live && !ready(k)) return false;
          tc_fence_after();
          if (elect_one()) {
            if (k.live) scores(kd, h);
            // (without scores behind it too: the product is done)
            tc_commit(smem_u32(&s_full[2 * t + h]));
            if (h == 1) {
              if (k.live) tc_commit(k_bar);
              if (k.live && k.last) tc_commit(smem_u32(&q_empty[t]));
              if (!k.live || k.new_q) tc_commit(smem_u32(&o_done[t]));
            }
          }
          __syncwarp();
        }
        ++it;
        if (k.live && k.new_q) ++opened;
        return true;
      };
      if (SPLIT) {
        const XWalk w(p, first);
        if (w.live(p)) {
          int j0, j1;
          xattn_key_range(w.keys(p), split, splits, j0, j1);
          // this stream takes every second key tile
          const int n = (j1 - j0 + 1 - t) / 2;
          if (n > 0 && open(Next{true, xattn_fill_k(0), true, false}))
            for (int k = 0; k < n; ++k)
              if (!advance(xattn_fill_v(k), k == 0, Next{k + 1 < n, xattn_fill_k(k + 1), false, false})) break;
        }
      } else {
        // the ring holds K0 V0 K1 V1 ... of the tiles with keys in turn
        XWalk w(p, first);  // stands on the tile behind
        auto next_keys = [&]() -> int {  // key tiles of the next tile with keys, 0: none
          int n = 0;
          for (; n == 0 && w.live(p); w.next(p)) n = (w.keys(p) + kXTile - 1) / kXTile;
          return n;
        };
        int n = next_keys();
        bool ok = n > 0 && open(Next{true, xattn_fill_k(0), true, n == 1});
        uint32_t k = 0;  // key tiles of all work tiles
        while (ok && n > 0) {
          const int n_next = next_keys();
          for (int j = 0; ok && j < n; ++j, ++k) {
            const bool more = j + 1 < n;
            ok = advance(xattn_fill_v(k), j == 0,
                         Next{more || n_next > 0, xattn_fill_k(k + 1), !more, more ? j + 2 == n : n_next == 1});
          }
          n = n_next;
        }
      }
      if (elect_one()) tc_commit(smem_u32(&drain[t]));
      __syncwarp();
      mbar_wait_drain(smem_u32(&drain[t]), 0);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax: a row per thread
    regs_grow_to<kXRegsSoftmax>();
    const int t = (warp >> 2) - 1;  // stream
    const int q = warp & 3;         // TMEM lane quarter
    const int r = q * 32 + lane;    // row of the stream's tile
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t t_s = tmem + 128 * t + lane_base, t_o = tmem + C::O_COL + 128 * t + lane_base;
    const float c = p.scale * 1.4426950408889634f;  // log2 e
    uint32_t it = 0;                // key tiles done
    uint32_t keyed = 0, closed = 0; // key tiles of the work tiles before, work tiles with keys done
    const XRing ring = xattn_ring(SLOTS, C::RINGS, SPLIT ? t : 0);
    bool ok = true;
    auto got = [&](uint64_t* bar, uint32_t parity) -> bool {
      return mbar_wait_warp(smem_u32(bar), parity & 1, abort_flag, p.status);
    };
    for (XWalk w(p, first); w.live(p) && ok; w.next(p)) {
      const XTileAt a = w.at(p, kRows);
      int j0, j1;
      xattn_key_range(a.len, split, splits, j0, j1);
      const int n = j1 - j0;
      const bool some = SPLIT ? t < n : n > 0;  // this stream has keys here
      // the offset (log2 domain), the score that it stands for, the sum of 2^(c s - offset)
      float m_used = -INFINITY, x_used = -INFINITY, l = 0.0f;
      bool begun = false;
      // half key tiles (SPLIT: of every second key tile)
      for (int u = SPLIT ? 2 * t : 0; u < 2 * n; u += SPLIT && (u & 1) ? 3 : 1) {
        const int h = u & 1;
        const int key0 = j0 * kXTile + u * kXSub;
        // the keys of this half that count, one bit each, 32 from key0 + k on
        auto counted = [&](int k) -> uint32_t {
          const int left = a.len - (key0 + k);
          uint32_t bits = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
          if (p.key_mask != nullptr) {
            const int key = key0 + k + lane;
            const bool on = key < p.Skv && p.key_mask[static_cast<int64_t>(a.kb) * p.ld_mask + key] != 0;
            bits &= __ballot_sync(0xffffffffu, on);
          }
          return bits;
        };
        const uint32_t keep[2] = {counted(0), counted(32)};
        const uint32_t t_buf = t_s + kXSub * h;
        if (!got(&s_full[2 * t + h], it)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sv[kXSub];
        tmem_ld_32cols(t_buf, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld_32cols(t_buf + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld_wait();
        if ((keep[0] & keep[1]) != 0xffffffffu) {
          // The values of keys that do not count may hold anything (0 times
          // NaN is NaN): cleared once the tile has landed and before this
          // stream's probabilities let its product start, two threads a key
          // with half of its columns each.  (Past the last key of all, TMA
          // has filled zeros.)  Streams that share a value tile both do it
          // (the second writes zeros over zeros).
          const bool clear = !((q & 1 ? keep[1] : keep[0]) >> lane & 1) && key0 + (r & 63) < p.Skv;
          if (__any_sync(0xffffffffu, clear)) {
            const uint32_t fill = xattn_fill_v(SPLIT ? u >> 2 : keyed + (u >> 1));
            if (!got(&kv_full[ring.slot(fill)], ring.parity(fill))) {
              ok = false;
              break;
            }
            if (clear) {
              uint8_t* row = smem + C::KV_OFF + ring.slot(fill) * C::TILE_BYTES + (kXSub * h + (r & 63)) * 128 +
                             (r >> 6) * (DB == 2 ? kXTile * 128 : 64);
              // (in an order that spreads the lanes' rows over the banks)
#pragma unroll
              for (int e = 0; e < 4 * DB; ++e)
                *reinterpret_cast<uint4*>(row + 16 * ((e ^ lane) & (4 * DB - 1))) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!(keep[0] >> e & 1)) sv[e] = 0xff800000u;  // -inf: no weight
            if (!(keep[1] >> e & 1)) sv[32 + e] = 0xff800000u;
          }
          if ((keep[0] | keep[1]) == 0u) {
            // no key of this half counts: no probabilities, nothing to sum
            const uint32_t zero[16] = {};
            tmem_st_16cols(t_buf, zero);
            tmem_st_16cols(t_buf + 16, zero);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * t + h]));
            begun = true;
            it += h;
            continue;
          }
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          mx[e] = max3_nan(__uint_as_float(sv[e]), __uint_as_float(sv[e + 8]), __uint_as_float(sv[e + 16]));
#pragma unroll
        for (int e = 24; e < 56; e += 16)
#pragma unroll
          for (int w = 0; w < 8; ++w)
            mx[w] = max3_nan(mx[w], __uint_as_float(sv[e + w]), __uint_as_float(sv[e + w + 8]));
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = max3_nan(mx[e], __uint_as_float(sv[56 + e]), mx[e]);
        const float x_tile =
            max3_nan(max3_nan(mx[0], mx[1], mx[2]), max3_nan(mx[3], mx[4], mx[5]), max3_nan(mx[6], mx[7], mx[7]));
        // a score that is NaN or +infinity makes its row NaN (the polynomial
        // below would drop it)
        if (!(x_tile < INFINITY)) l = __int_as_float(0x7fffffff);
        const float m_tile = __fmul_rn(x_tile, c);
        if (__any_sync(0xffffffffu, m_tile > m_used + kXSlack || xattn_large(m_used))) {
          // (two scores can differ by many binades under one rounded large offset)
          const bool moves = m_tile > m_used + kXSlack || (xattn_large(m_used) && x_tile > x_used);
          float f = 1.0f;
          if (moves) {
            f = x_used == -INFINITY ? 0.0f : ex2_approx(xattn_ahead(x_used, x_tile, c));
            x_used = x_tile;
            m_used = m_tile;
            l *= f;
          }
          if (begun) {
            // O at rest: the half before is done when its buffer is full
            // again (phase it + 1 of the first, phase it of the second)
            if (!got(&s_full[2 * t + (h ^ 1)], h == 1 ? it + 1 : it)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < DB * 4; ++cc) {
              uint32_t v[16];
              tmem_ld_16cols(t_o + 16 * cc, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
              tmem_st_16cols(t_o + 16 * cc, v);
            }
          }
          if (__builtin_expect(__any_sync(0xffffffffu, x_used > -INFINITY && xattn_large(m_used)), 0)) {
            // A large row: exponents from the scores' differences, in a loop of
            // its own over the scores as they lie in TMEM (woven into the one
            // below they cost every call a tenth).
            const bool large = x_used > -INFINITY && xattn_large(m_used);
            const float off = x_used == -INFINITY ? 0.0f : m_used;
            float la = 0.0f, lb = 0.0f;
#pragma unroll 1
            for (int w32 = 0; w32 < 2; ++w32) {
              uint32_t sw[32], bw[16];
              tmem_ld_32cols(t_buf + 32 * w32, sw);
              tmem_ld_wait();
              const uint32_t on = counted(32 * w32);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float s = on >> (e + i) & 1 ? __uint_as_float(sw[e + i]) : -INFINITY;
                  y[i] = ex2_approx(large ? (s - x_used) * c : fmaf(s, c, -off));
                }
                bw[e / 2] = pack_bf16x2(y[0], y[1]);
                la += y[0];
                lb += y[1];
              }
              tmem_st_16cols(t_buf + 16 * w32, bw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * t + h]));
            l += la + lb;
            begun = true;
            it += h;
            continue;
          }
        }
        begun = true;
        const float off = x_used == -INFINITY ? 0.0f : m_used;
        float la = 0.0f, lb = 0.0f, lc = 0.0f, ld = 0.0f;
        uint32_t b[kXSub / 2];
#pragma unroll
        for (int c0 = 0; c0 < kXSub; c0 += kXChunk) {
          float y[kXChunk];
#pragma unroll
          for (int e = 0; e < kXChunk; e += 2)
            fma2_rn(y[e], y[e + 1], __uint_as_float(sv[c0 + e]), __uint_as_float(sv[c0 + e + 1]), c, c, -off, -off);
#pragma unroll
          for (int e = 0; e < kXChunk; e += 2) {
            if (((c0 + e) >> 1) % 16 >= 16 - kXPolyPairs) {
              exp2_poly2(y[e], y[e + 1], y[e], y[e + 1]);
            } else {
              y[e] = ex2_approx(y[e]);
              y[e + 1] = ex2_approx(y[e + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < kXChunk; e += 2) b[(c0 + e) / 2] = pack_bf16x2(y[e], y[e + 1]);
#pragma unroll
          for (int e = 0; e < kXChunk; e += 4) {
            add2_rn(la, lb, la, lb, y[e], y[e + 1]);
            add2_rn(lc, ld, lc, ld, y[e + 2], y[e + 3]);
          }
          if ((c0 + kXChunk) % 32 == 0)
            tmem_st_16cols(t_buf + 16 * (c0 / 32), *reinterpret_cast<uint32_t(*)[16]>(&b[16 * (c0 / 32)]));
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * t + h]));
        l += (la + lc) + (lb + ld);
        it += h;
      }
      if (!ok) break;
      keyed += n;
      if constexpr (SPLIT) {
        // both streams' last products are done, the ring is read
        if ((some && !got(&o_done[t], 0)) || ((t == 0 ? n > 1 : n > 0) && !got(&o_done[t ^ 1], 0))) break;
        tc_fence_after();
        float* stat = reinterpret_cast<float*>(smem + C::STAT_OFF) + 3 * kXTile * t;
        stat[r] = x_used > -INFINITY && xattn_large(m_used) ? __int_as_float(0x7fffffff) : m_used;  // NaN: see x
        stat[kXTile + r] = l;
        stat[2 * kXTile + r] = x_used;
        float* part = reinterpret_cast<float*>(smem) + (t * kXTile + r) * C::PART_PITCH;
        const bool live = a.row0 + r < p.Sq * p.pack;
        if (__any_sync(0xffffffffu, live)) {
#pragma unroll 1
          for (int cc = 0; cc < DB; ++cc) {
            uint32_t v[64];
            if (some) {
              tmem_ld_32cols(t_o + 64 * cc, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
              tmem_ld_32cols(t_o + 64 * cc + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int e = 0; e < 64; ++e) v[e] = 0u;
            }
            if (live) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                *reinterpret_cast<uint4*>(part + 64 * cc + 4 * e) =
                    make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
        }
      } else {
        if (!some) continue;
        // the epilogue takes the sums over; it has read the factors of the
        // tile before
        if (closed > 0 && !got(&o_free[t], closed - 1)) break;
        ++closed;
        reinterpret_cast<float*>(smem + C::F_OFF)[t * kXTile + r] = xattn_factor(x_used, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&f_full[t]));
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue: a row per thread
    regs_release_to<kXRegsEpi>();
    const int q = warp & 3;  // TMEM lane quarter
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint8_t* boxes = smem + C::O_OFF + q * (2 * 32 * 128);
    uint32_t closed = 0;  // tiles with keys done
    bool ok = !SPLIT;
    for (XWalk w(p, first); w.live(p) && ok; w.next(p)) {
      const XTileAt a = w.at(p, kRows);
      const bool some = a.len > 0;
      for (int t = 0; t < 2 && ok; ++t) {
        float f = 0.0f;
        if (some) {
          if (!mbar_wait_warp(smem_u32(&f_full[t]), closed & 1, abort_flag, p.status) ||
              !mbar_wait_warp(smem_u32(&o_done[t]), closed & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          f = reinterpret_cast<const float*>(smem + C::F_OFF)[t * kXTile + q * 32 + lane];
        }
        // out of TMEM and into the boxes as fast as it goes: the next tile's
        // first product waits to overwrite the sums
        if (lane == 0) bulk_wait_group_read<0>();  // the boxes' last stores have been read
        __syncwarp();
#pragma unroll
        for (int hh = 0; hh < DB * 2; ++hh) {
          uint32_t v[32];
          if (some) {
            tmem_ld_32cols(tmem + C::O_COL + 128 * t + lane_base + 32 * hh, v);
            tmem_ld_wait();
            if (hh == DB * 2 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&o_free[t]));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
          uint8_t* row = boxes + (hh >> 1) * (32 * 128) + lane * 128;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float o0, o1;
              mul2_rn(o0, o1, __uint_as_float(v[8 * u + 2 * e]), __uint_as_float(v[8 * u + 2 * e + 1]), f, f);
              b[e] = pack_bf16x2(o0, o1);
            }
            *reinterpret_cast<uint4*>(row + (((4 * (hh & 1) + u) ^ (lane & 7)) << 4)) =
                make_uint4(b[0], b[1], b[2], b[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        const int tok0 = (a.row0 + t * kXTile + q * 32) / p.pack;
        if (lane == 0) {
          if (tok0 < p.Sq)
#pragma unroll
            for (int d = 0; d < DB; ++d)
              tma_store_4d(&tm_o, smem_u32(boxes + d * (32 * 128)), 64 * d, a.h0, tok0, a.b);
          bulk_commit_group();
        }
      }
      if (some) ++closed;
    }
    if (!SPLIT && lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  if constexpr (SPLIT) {
    cluster_sync();  // every CTA's partial sums are in its shared memory
    if (warp >= 4 && warp < 12 && first < p.tiles && *abort_flag == 0) {
      // rows of the tile times groups of four columns, shared out evenly over the cluster
      const XTileAt a = XWalk(p, first).at(p, kRows);
      const int groups = p.D / 4, total = min(kXTile, p.Sq * p.pack - a.row0) * groups;
      const int end = total * (split + 1) / splits;
      const uint32_t part0 = smem_u32(smem), stat0 = smem_u32(smem + C::STAT_OFF);
      for (int e = total * split / splits + threadIdx.x - 128; e < end; e += 256) {
        const int row = e / groups, g = e % groups;
        // every stream of every CTA: all offsets, and eight streams' sums and
        // columns at a time, asked for before the first is used
        auto stat = [&](int s, int i) {
          return ld_cluster_f32(mapa_shared(stat0 + 4u * (((s & 1) * 3 + i) * kXTile + row), s >> 1));
        };
        auto cols = [&](int s) {
          return ld_cluster_f32x4(
              mapa_shared(part0 + 4u * (((s & 1) * kXTile + row) * C::PART_PITCH + 4 * g), s >> 1));
        };
        float ms[16], ls[8], m = -INFINITY, l = 0.0f, top;
        float4 v[8], o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto fetch = [&](int s0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int s = s0 + i;
            ls[i] = 0.0f;
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s < 2 * splits) {
              ls[i] = stat(s, 1);
              v[i] = cols(s);
            }
          }
        };
        auto join = [&](float w, float ls, const float4& v) {
          l = fmaf(w, ls, l);
          o.x = fmaf(w, v.x, o.x);
          o.y = fmaf(w, v.y, o.y);
          o.z = fmaf(w, v.z, o.z);
          o.w = fmaf(w, v.w, o.w);
        };
        auto add = [&](int s0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) join(ms[s0 + i] == m ? 1.0f : ex2_approx(ms[s0 + i] - m), ls[i], v[i]);
        };
#pragma unroll
        for (int s = 0; s < 16; ++s) ms[s] = s < 2 * splits ? stat(s, 0) : -INFINITY;
        fetch(0);
#pragma unroll
        for (int s = 0; s < 16; s += 2) m = max3_nan(m, ms[s], ms[s + 1]);
        top = m;
        if (__builtin_expect(m == m, 1)) {
          add(0);
          if (splits > 4) {
            fetch(8);
            add(8);
          }
        } else {  // a large offset among them
          const float c = p.scale * 1.4426950408889634f;
          top = -INFINITY;
#pragma unroll 1
          for (int s = 0; s < 2 * splits; ++s) top = fmaxf(top, stat(s, 2));
#pragma unroll 1
          for (int s = 0; s < 2 * splits; ++s) {
            const float x = stat(s, 2);
            join(x == top ? 1.0f : ex2_approx(xattn_ahead(x, top, c)), stat(s, 1), cols(s));
          }
        }
        const float f = xattn_factor(top, l);
        const int token = (a.row0 + row) / p.pack, head = a.h0 + (a.row0 + row) % p.pack;
        *reinterpret_cast<uint2*>(p.O + (static_cast<int64_t>(a.b) * p.Sq + token) * p.ldo + head * p.D + 4 * g) =
            make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
      }
    }
    tc_fence_before();
    cluster_meet();  // the peers have read this CTA's sums
  } else {
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace w4a4
