// cross_attention.cuh -- bf16 attention of one token sequence to another of
// its own length (an encoder's states), on the sm_100a tensor cores.
//
// Per query row and head, over the keys j that the length and the key mask
// leave:  o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),
// c = scale log2 e, the sums and the running offset m in fp32; a row without
// keys gives 0.  m moves only when a tile's maximum passes it by more than
// kXSlack binades (the accumulator and the sum are then rescaled), which is
// exact: numerator and denominator share the offset.  The probabilities are
// rounded to bf16 for the second product, a relative 2^-9 each, random in
// sign, against the 2^-9 of the output's own rounding.
//
// A work tile is 128 rows of one key/value head: queries times the heads that
// share it (the largest power of two of them, so that a group of heads reads
// its keys once), loaded by one 4-D TMA box whose row order is token-major.
// S = Q K^T and O += P V are tcgen05.mma kind::f16 with both accumulators in
// TMEM; P goes back into S's columns as the A operand of the second product,
// V is its MN-major B operand as it lies in memory.  MMAs of the issuing
// thread run in order, so S of the next key tile may follow the product that
// reads P, and a commit that covers S covers the product before it too.
//
// Two forms, each with two streams of softmax (a warpgroup each, one row a
// thread) that alternate on the tensor cores:
//   SPLIT = false  many rows: the streams are two row tiles over the same keys,
//                  persistent CTAs, one per SM; the next tile's first scores
//                  are computed under this tile's epilogue.
//   SPLIT = true   few rows: the streams are the even and odd key tiles of one
//                  row tile, and a cluster of CTAs splits the keys; the
//                  partial sums meet in (distributed) shared memory.
#pragma once

#include "attention.cuh"
#include "sm100.cuh"

namespace w4a4 {

constexpr int kXTile = 128;       // rows per stream, keys per step
constexpr int kXThreads = 384;    // control warpgroup, two softmax warpgroups
constexpr float kXSlack = 8.0f;   // binades a tile's maximum may pass the offset
constexpr int kXRegsCtrl = 48, kXRegsSoftmax = 224;
static_assert(128 * kXRegsCtrl + 256 * kXRegsSoftmax <= kXThreads * 168, "register budgets fit the launch allocation");

struct XAttnParams {
  int Sq, Skv, heads, kv_heads, D;
  int pack;                 // heads of a group that share a row tile (power of two <= 32)
  int batch, kv_batch;
  int row_tiles;            // work tiles along the queries (128 or 256 rows each)
  int tiles;                // work tiles in all
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
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = NQ * TILE_BYTES;
  static constexpr int O_OFF = KV_OFF + SLOTS * TILE_BYTES;
  static constexpr int O_BYTES = SPLIT ? 0 : 8 * 32 * 128;       // a 32 x 64 bf16 box per softmax warp
  static constexpr int PART_PITCH = DB * 64 + 4;                 // floats; SPLIT: over Q and the ring
  static constexpr int STAT_OFF = 2 * kXTile * PART_PITCH * 4;   // behind them m and l, [2 streams][2][128]
  static constexpr int BAR_OFF = O_OFF + O_BYTES;
  static constexpr int BARS = 2 * SLOTS + 2 * 5 + 1;
  static constexpr int SMEM = BAR_OFF + 8 * BARS + 16 + 1024;
  static constexpr int TMEM_COLS = 512;
  static constexpr int O_COL = 256;        // S of stream t at 128 t, O at 256 + 128 t
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(!SPLIT || STAT_OFF + 4 * kXTile * 4 <= O_OFF, "the partial sums fit over Q and the ring");
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
// (whose offset never moved), NaN where l is.
__device__ __forceinline__ float xattn_factor(float m, float l) {
  return m == -INFINITY && l == l ? 0.0f : 1.0f / l;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// What a work tile index stands for.
struct XTileAt {
  int row0;  // first row (token-major, `pack` heads a token) of the tile's first stream
  int h0;    // first query head
  int hk;    // key/value head
  int b, kb; // sequence and its key/value batch
  int len;   // keys
};

__device__ __forceinline__ XTileAt xattn_tile(const XAttnParams& p, int tile, int rows) {
  XTileAt a;
  const int blocks = p.heads / p.pack;
  const int rt = tile % p.row_tiles;
  const int hb = (tile / p.row_tiles) % blocks;
  a.b = tile / (p.row_tiles * blocks);
  a.row0 = rt * rows;
  a.h0 = hb * p.pack;
  a.hk = a.h0 / (p.heads / p.kv_heads);
  a.kb = p.kv_batch == 1 ? 0 : a.b;
  a.len = p.Skv;
  if (p.kv_len != nullptr) a.len = min(max(p.kv_len[a.kb], 0), p.Skv);
  return a;
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
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;                                 // [SLOTS]
  uint64_t* q_full = kv_empty + SLOTS;                                  // [2] query tiles (SPLIT: the first)
  uint64_t* q_empty = q_full + 2;                                       // [2] the tile's last scores are done
  uint64_t* s_full = q_empty + 2;                                       // [2] per stream: scores in TMEM
  uint64_t* p_full = s_full + 2;                                        // [2] probabilities in TMEM, O rescaled
  uint64_t* o_done = p_full + 2;                                        // [2] the tile's last product is done
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&q_full[t]), 1);
      mbar_init(smem_u32(&q_empty[t]), 1);
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[t]), 4);
      mbar_init(smem_u32(&o_done[t]), 1);
    }
    mbar_init(smem_u32(drain), 1);
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
  const int step = SPLIT ? p.tiles : static_cast<int>(gridDim.x);
  // key tiles [j0, j1) of a tile with `len` keys
  auto key_range = [&](int len, int& j0, int& j1) {
    const int n = (len + kXTile - 1) / kXTile;
    j0 = SPLIT ? static_cast<int>(static_cast<int64_t>(n) * split / splits) : 0;
    j1 = SPLIT ? static_cast<int>(static_cast<int64_t>(n) * (split + 1) / splits) : n;
  };

  if (warp < 4) {
    regs_release_to<kXRegsCtrl>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      uint32_t fill = 0, nonempty = 0;
      bool ok = true;
      auto load_kv = [&](const CUtensorMap* map, const XTileAt& a, int j) {
        const uint32_t s = fill % SLOTS;
        if (!ok || !(ok = mbar_wait(smem_u32(&kv_empty[s]), ((fill / SLOTS) & 1) ^ 1, abort_flag, p.status))) return;
        const uint32_t bar = smem_u32(&kv_full[s]);
        mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
        for (int d = 0; d < DB; ++d)
          tma_load_4d(smem_u32(smem + C::KV_OFF + s * C::TILE_BYTES + d * (kXTile * 128)), map, bar, 64 * d, a.hk,
                      j * kXTile, a.kb);
        ++fill;
      };
      uint32_t q_fills = 0;
      auto load_q = [&](const XTileAt& a, int t) {
        if (!ok || !(ok = mbar_wait(smem_u32(&q_empty[t]), (nonempty & 1) ^ 1, abort_flag, p.status))) return;
        const uint32_t bar = smem_u32(&q_full[t]);
        mbar_arrive_expect_tx(bar, C::TILE_BYTES);
#pragma unroll
        for (int d = 0; d < DB; ++d)
          tma_load_4d(smem_u32(smem + C::Q_OFF + t * C::TILE_BYTES + d * (kXTile * 128)), &tm_q, bar, 64 * d, a.h0,
                      (a.row0 + t * kXTile) / p.pack, a.b);
        q_fills |= 1u << t;
      };
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const XTileAt a = xattn_tile(p, tile, kRows);
        int j0, j1;
        key_range(a.len, j0, j1);
        if (j0 == j1) continue;
        q_fills = 0;
        load_q(a, 0);
        if (SPLIT) {
          // consumed in the order K0 K1 V0 K2 V1 K3 ...
          for (int j = j0; j <= j1 && ok; ++j) {
            if (j < j1) load_kv(&tm_k, a, j);
            if (j > j0) load_kv(&tm_v, a, j - 1);
          }
        } else {
          for (int j = j0; j < j1 && ok; ++j) {
            load_kv(&tm_k, a, j);
            if (j == j0) load_q(a, 1);
            load_kv(&tm_v, a, j);
          }
        }
        if (ok) ++nonempty;
      }
      // every fill issued lands before the shared memory is released
      for (uint32_t j = fill > SLOTS ? fill - SLOTS : 0u; j < fill; ++j)
        mbar_wait_drain(smem_u32(&kv_full[j % SLOTS]), (j / SLOTS) & 1);
      if (!ok)
        for (int t = 0; t < 2; ++t)
          if (q_fills >> t & 1) mbar_wait_drain(smem_u32(&q_full[t]), nonempty & 1);
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdescS = idesc_bf16(kXTile, kXTile);
      constexpr uint32_t kIdescO = idesc_bf16(kXTile, DB * 64) | (1u << 16);  // B (the values) MN-major
      const int d_steps = (p.D + 15) / 16;
      uint32_t use = 0;  // ring slots consumed
      bool ok = true;
      auto slot_wait = [&](uint32_t n) -> bool {
        return mbar_wait(smem_u32(&kv_full[n % SLOTS]), (n / SLOTS) & 1, abort_flag, p.status);
      };
      auto slot_base = [&](uint32_t n) -> uint32_t {
        return smem_u32(smem + C::KV_OFF + (n % SLOTS) * C::TILE_BYTES);
      };
      auto scores = [&](int t, uint32_t n) {  // S_t = Q K^T, keys in ring slot n
        tc_fence_after();
        const uint32_t q = smem_u32(smem + C::Q_OFF + (SPLIT ? 0 : t) * C::TILE_BYTES), k = slot_base(n);
#pragma unroll
        for (int i = 0; i < DB * 4; ++i)
          if (i < d_steps)
            mma_bf16(tmem + 128 * t, smem_desc(q + (i / 4) * (kXTile * 128) + 32 * (i % 4), 16, 1024, kSwizzle128B),
                     smem_desc(k + (i / 4) * (kXTile * 128) + 32 * (i % 4), 16, 1024, kSwizzle128B), kIdescS,
                     i > 0 ? 1u : 0u);
        tc_commit(smem_u32(&s_full[t]));
      };
      auto product = [&](int t, uint32_t n, bool fresh) {  // O_t (+)= P_t V, values in ring slot n
        tc_fence_after();
        const uint32_t v = slot_base(n);
#pragma unroll
        for (int i = 0; i < kXTile / 16; ++i)
          mma_bf16_ts(tmem + C::O_COL + 128 * t, tmem + 128 * t + 8 * i,
                      smem_desc(v + 2048 * i, kXTile * 128, 1024, kSwizzle128B), kIdescO,
                      (!fresh || i > 0) ? 1u : 0u);
      };
      uint32_t p_phase = 0;  // bit t: parity of the next phase of p_full[t]
      auto p_wait = [&](int t) -> bool {
        const bool r = mbar_wait(smem_u32(&p_full[t]), (p_phase >> t) & 1, abort_flag, p.status);
        p_phase ^= 1u << t;
        return r;
      };
      if (SPLIT) {
        if (first < p.tiles) {
          const XTileAt a = xattn_tile(p, first, kRows);
          int j0, j1;
          key_range(a.len, j0, j1);
          const int n = j1 - j0;
          ok = n == 0 || mbar_wait(smem_u32(&q_full[0]), 0, abort_flag, p.status);
          for (int t = 0; t < 2 && t < n && ok; ++t, ++use) {
            if (!(ok = slot_wait(use))) break;
            scores(t, use);
            tc_commit(smem_u32(&kv_empty[use % SLOTS]));
          }
          for (int i = 0; i < n && ok; ++i) {
            const int t = i & 1;
            if (!(ok = slot_wait(use) && p_wait(t))) break;
            product(t, use, i < 2);
            tc_commit(smem_u32(&kv_empty[use % SLOTS]));
            ++use;
            if (i + 2 >= n) {
              tc_commit(smem_u32(&o_done[t]));
            } else {
              if (!(ok = slot_wait(use))) break;
              scores(t, use);
              tc_commit(smem_u32(&kv_empty[use % SLOTS]));
              ++use;
            }
          }
        }
      } else {
        // the tiles with keys, one ahead: a tile's first scores are issued
        // behind the last product of the tile before
        auto next_tile = [&](int tile, int& n) -> int {
          for (; tile < p.tiles; tile += step) {
            int j0, j1;
            key_range(xattn_tile(p, tile, kRows).len, j0, j1);
            n = j1 - j0;
            if (n > 0) break;
          }
          return tile;
        };
        uint32_t count = 0;  // tiles with keys begun
        int n = 0;
        int tile = next_tile(first, n);
        auto begin = [&](int t) -> bool {  // the first scores of the tile `count`, keys in slot `use`
          if (!mbar_wait(smem_u32(&q_full[t]), count & 1, abort_flag, p.status) || !slot_wait(use)) return false;
          scores(t, use);
          return true;
        };
        if (tile < p.tiles) {
          for (int t = 0; t < 2 && ok; ++t)
            if ((ok = begin(t)) && n == 1) tc_commit(smem_u32(&q_empty[t]));
          if (ok) tc_commit(smem_u32(&kv_empty[use % SLOTS]));
          ++use;
          ++count;
        }
        while (tile < p.tiles && ok) {
          int n_next = 0;
          const int tile_next = next_tile(tile + step, n_next);
          for (int j = 0; j < n && ok; ++j) {
            const uint32_t v = use, k = use + 1;
            const bool more = j + 1 < n, follow = !more && tile_next < p.tiles;
            for (int t = 0; t < 2 && ok; ++t) {
              if (!(ok = slot_wait(v) && p_wait(t))) break;
              product(t, v, j == 0);
              if (t == 1) tc_commit(smem_u32(&kv_empty[v % SLOTS]));
              if (!more) tc_commit(smem_u32(&o_done[t]));
              if (more) {
                if (!(ok = slot_wait(k))) break;
                scores(t, k);
                if (j + 2 == n) tc_commit(smem_u32(&q_empty[t]));
              } else if (follow) {
                use = k;
                ok = begin(t);
                use = v;
                if (ok && n_next == 1) tc_commit(smem_u32(&q_empty[t]));
              }
              if (t == 1 && ok && (more || follow)) tc_commit(smem_u32(&kv_empty[k % SLOTS]));
            }
            use += (more || follow) ? 2 : 1;
            if (follow) ++count;
          }
          tile = tile_next;
          n = n_next;
        }
      }
      tc_commit(smem_u32(drain));
      mbar_wait_drain(smem_u32(drain), 0);
    }
  } else {
    // ------------------------------------------------------------ softmax: a row per thread
    regs_grow_to<kXRegsSoftmax>();
    const int t = (warp >> 2) - 1;  // stream
    const int q = warp & 3;         // TMEM lane quarter
    const int r = q * 32 + lane;    // row of the stream's tile
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t t_s = tmem + 128 * t + lane_base, t_o = tmem + C::O_COL + 128 * t + lane_base;
    const float c = p.scale * 1.4426950408889634f;  // log2 e
    uint32_t sc = 0, oc = 0;        // phases of s_full and o_done waited for
    uint32_t fills = 0;             // ring fills of the tiles before
    bool ok = true;
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      const XTileAt a = xattn_tile(p, tile, kRows);
      int j0, j1;
      key_range(a.len, j0, j1);
      const int n = j1 - j0;
      float m_used = -INFINITY, l = 0.0f;  // offset (log2 domain) and sum of 2^(c s - offset)
      bool begun = false;
      for (int i = SPLIT ? t : 0; i < n; i += SPLIT ? 2 : 1) {
        const int j = j0 + i;
        // the keys of this tile that count, one bit each
        uint32_t keep[4];
        bool all = true;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int left = a.len - (j * kXTile + 32 * w);
          keep[w] = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
          if (p.key_mask != nullptr) {
            const int key = j * kXTile + 32 * w + lane;
            const bool on = key < p.Skv && p.key_mask[static_cast<int64_t>(a.kb) * p.ld_mask + key] != 0;
            keep[w] &= __ballot_sync(0xffffffffu, on);
          }
          all = all && keep[w] == 0xffffffffu;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[t]), sc & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        ++sc;
        tc_fence_after();
        uint32_t sv[kXTile];
#pragma unroll
        for (int cc = 0; cc < kXTile / 32; ++cc)
          tmem_ld_32cols(t_s + 32 * cc, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * cc]));
        tmem_ld_wait();
        if (!all) {
          // Keys that do not count: no weight, and zeros for their values,
          // which may hold anything (0 times NaN is NaN).  One of the streams
          // that share a value tile clears them, once the tile has landed
          // and before its probabilities let the product start.
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int b = 0; b < 32; ++b)
              if (!(keep[w] >> b & 1)) sv[32 * w + b] = 0xff800000u;  // -inf
          if (SPLIT || t == 0) {
            const uint32_t v = SPLIT ? (i < n - 1 ? 2u * i + 2u : 2u * n - 1u) : fills + 2u * i + 1u;
            if (!__all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&kv_full[v % SLOTS]), (v / SLOTS) & 1, abort_flag, p.status))) {
              ok = false;
              break;
            }
            const uint32_t mine = q == 0 ? keep[0] : q == 1 ? keep[1] : q == 2 ? keep[2] : keep[3];
            if (!(mine >> lane & 1)) {
              uint8_t* row = smem + C::KV_OFF + (v % SLOTS) * C::TILE_BYTES + r * 128;
#pragma unroll
              for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  *reinterpret_cast<uint4*>(row + d * (kXTile * 128) + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kXTile; e += 2)
          mx4[(e >> 1) & 3] = max3_nan(mx4[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
        const float m_tile = max3_nan(max3_nan(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]) * c;
        // a score that is NaN or +infinity makes its row NaN (the polynomial
        // below would drop it)
        if (!(m_tile < INFINITY)) l = __int_as_float(0x7fffffff);
        const bool moves = m_tile > m_used + kXSlack;
        const float f = moves ? ex2_approx(m_used - m_tile) : 1.0f;
        if (moves) {
          m_used = m_tile;
          l *= f;
        }
        if (begun && __any_sync(0xffffffffu, moves)) {
          // (the scores' commit covers the product before them: O is at rest)
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
        begun = true;
        const float off = m_used == -INFINITY ? 0.0f : m_used;
        float la = 0.0f, lb = 0.0f;
#pragma unroll
        for (int cc = 0; cc < kXTile / 32; ++cc) {
          uint32_t b[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t* v = &sv[32 * cc + 4 * e];
            float x0, x1, x2, x3, p0, p1;
            fma2_rn(x0, x1, __uint_as_float(v[0]), __uint_as_float(v[1]), c, c, -off, -off);
            fma2_rn(x2, x3, __uint_as_float(v[2]), __uint_as_float(v[3]), c, c, -off, -off);
            if ((e & 1) == 0) {  // one pair in four on the FMA pipes
              exp2_poly2(p0, p1, x0, x1);
            } else {
              p0 = ex2_approx(x0);
              p1 = ex2_approx(x1);
            }
            const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
            b[2 * e] = pack_bf16x2(p0, p1);
            b[2 * e + 1] = pack_bf16x2(p2, p3);
            float s0, s1;
            add2_rn(s0, s1, p0, p1, p2, p3);
            add2_rn(la, lb, la, lb, s0, s1);
          }
          tmem_st_16cols(t_s + 16 * cc, b);
        }
        l += la + lb;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[t]));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (n > 0 && (!SPLIT || t < n)) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[t]), oc & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        ++oc;
        tc_fence_after();
      }
      fills += 2u * n;
      if constexpr (SPLIT) {
        // the other stream's products have read the ring too
        if (t == 0 ? n > 1 : n > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[t ^ 1]), 0, abort_flag, p.status))) {
            ok = false;
            break;
          }
        }
        float* stat = reinterpret_cast<float*>(smem + C::STAT_OFF);
        stat[t * 2 * kXTile + r] = m_used;
        stat[t * 2 * kXTile + kXTile + r] = l;
        float* part = reinterpret_cast<float*>(smem) + (t * kXTile + r) * C::PART_PITCH;
        const bool live = a.row0 + r < p.Sq * p.pack;
#pragma unroll 1
        for (int cc = 0; cc < DB * 4; ++cc) {
          uint32_t v[16];
          if (t < n) {
            tmem_ld_16cols(t_o + 16 * cc, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0u;
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(part + 16 * cc + 4 * e) =
                  make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
      } else {
        const float f = n == 0 ? 0.0f : xattn_factor(m_used, l);
        uint8_t* box = smem + C::O_OFF + (warp - 4) * (32 * 128);
        const int tok0 = (a.row0 + t * kXTile + q * 32) / p.pack;
#pragma unroll 1
        for (int d = 0; d < DB; ++d) {
          if (lane == 0) bulk_wait_group_read<0>();  // the box's last store has been read
          __syncwarp();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t v[32];
            if (n > 0) {
              tmem_ld_32cols(t_o + 64 * d + 32 * hh, v);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0u;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint4 w;
              w.x = pack_bf16x2(__uint_as_float(v[8 * u]) * f, __uint_as_float(v[8 * u + 1]) * f);
              w.y = pack_bf16x2(__uint_as_float(v[8 * u + 2]) * f, __uint_as_float(v[8 * u + 3]) * f);
              w.z = pack_bf16x2(__uint_as_float(v[8 * u + 4]) * f, __uint_as_float(v[8 * u + 5]) * f);
              w.w = pack_bf16x2(__uint_as_float(v[8 * u + 6]) * f, __uint_as_float(v[8 * u + 7]) * f);
              *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * hh + u) ^ (lane & 7)) << 4)) = w;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && tok0 < p.Sq) {
            tma_store_4d(&tm_o, smem_u32(box), 64 * d, a.h0, tok0, a.b);
            bulk_commit_group();
          }
        }
        // (O is read: the next tile's first product waits for this thread's
        // next probabilities)
        tc_fence_before();
      }
    }
    if (!SPLIT && lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  if constexpr (SPLIT) {
    cluster_sync();  // every CTA's partial sums are in its shared memory
    if (warp >= 4 && first < p.tiles && *abort_flag == 0) {
      // rows of the tile times groups of four columns, shared out over the cluster
      const XTileAt a = xattn_tile(p, first, kRows);
      const int rows = min(kXTile, p.Sq * p.pack - a.row0), groups = p.D / 4;
      const uint32_t part0 = smem_u32(smem), stat0 = smem_u32(smem + C::STAT_OFF);
      for (int e = split * 256 + threadIdx.x - 128; e < rows * groups; e += splits * 256) {
        const int row = e / groups, g = e % groups;
        float m = -INFINITY;
        for (int s = 0; s < 2 * splits; ++s)
          m = fmaxf(m, ld_cluster_f32(mapa_shared(stat0 + 4u * ((s & 1) * 2 * kXTile + row), s >> 1)));
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < 2 * splits; ++s) {
          const uint32_t st = mapa_shared(stat0 + 4u * ((s & 1) * 2 * kXTile + row), s >> 1);
          const float ms = ld_cluster_f32(st);
          const float w = ms == m ? 1.0f : ex2_approx(ms - m);
          l = fmaf(w, ld_cluster_f32(st + 4u * kXTile), l);
          const float4 v =
              ld_cluster_f32x4(mapa_shared(part0 + 4u * (((s & 1) * kXTile + row) * C::PART_PITCH + 4 * g), s >> 1));
          o.x = fmaf(w, v.x, o.x);
          o.y = fmaf(w, v.y, o.y);
          o.z = fmaf(w, v.z, o.z);
          o.w = fmaf(w, v.w, o.w);
        }
        const float f = xattn_factor(m, l);
        const int token = (a.row0 + row) / p.pack, head = a.h0 + (a.row0 + row) % p.pack;
        *reinterpret_cast<uint2*>(p.O + (static_cast<int64_t>(a.b) * p.Sq + token) * p.ldo + head * p.D + 4 * g) =
            make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
      }
    }
    tc_fence_before();
    cluster_sync();  // the peers have read this CTA's sums
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
