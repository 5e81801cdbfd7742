// plan.h -- which kernel a call takes, by sizes and the device's SM count: plain
// arithmetic, for the entry points and for host programs that check it.
#pragma once

#include <algorithm>
#include <climits>
#include <cstdint>

namespace w4a4 {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// K slices of the kernel for few rows: a power of two up to a cluster of
// eight, at most one per 128-deep step, while the CTAs still fit on the device
// at once: two per SM, but clusters of four and eight do not pack that densely
// (9216 x 3200 at one token: 144 CTAs in pairs 8.2 us, 288 in fours 12.2 us;
// 6144 x 6144: 192 in fours 11.2 us, 96 in pairs 11.7 us).
inline int fp8_small_splits(int64_t n_tiles, int64_t k_steps, int64_t sms) {
  int s = 1;
  while (s < 8 && 2 * s <= k_steps && n_tiles * 2 * s <= (s == 1 ? 2 * sms : sms + sms / 2)) s *= 2;
  return s;
}

// Which FP8 kernel a product takes, by its time on one B200 in units of 10 ns,
// fitted to products of 24 to 9216 rows, 280 to 18432 columns and K from 512
// to 8192 (most within 10 %).  Pairs: a beginning and end, and waves of tiles,
// each of its K steps or, where K is short, of the tile's epilogue.  Few rows:
// the K steps of a slice, dearer with more tokens a tile and with more than
// one CTA on an SM, and the exchange of the partial sums.
// Measured on both sides: 64 x 18432 x 6144 25.7 us by the weight, 27.5 by
// pairs, 100 x 9216 x 3200 13.3 and 10.6; 333 x 2056 x 4112 13.4, 15.4 and 18.8
// with tiles 64, 128 and 256 wide, 9216 x 640 x 512 11.3, 10.3 and 10.3, 640 x
// 6144 x 6144 40.8, 27.7 and 25.0, 1729 x 4528 x 1536 23.0, 18.5 and 14.5.
// Returns 0 for the kernel for few rows, else the tile width.
inline int fp8_gemm_plan(int64_t M, int64_t N, int64_t K, int64_t sms) {
  const int64_t k_steps = ceil_div(K, 128), n_tiles = ceil_div(N, 128);
  int best = 256;
  int64_t cost = INT64_MAX;
  const int width[3] = {64, 128, 256}, ends[3] = {508, 498, 542}, step[3] = {19, 24, 37}, epilogue[3] = {131, 210, 343};
  for (int i = 0; i < 3; ++i) {
    const int64_t waves = ceil_div(ceil_div(M, 256) * ceil_div(N, width[i]), sms / 2);
    const int64_t c = ends[i] + waves * std::max<int64_t>(k_steps * step[i], epilogue[i]);
    if (c < cost) {
      cost = c;
      best = width[i];
    }
  }
  if (M <= 128 && n_tiles <= 65535) {
    const int64_t ctas = n_tiles * fp8_small_splits(n_tiles, k_steps, sms);
    const int64_t steps = ceil_div(k_steps * n_tiles, ctas);
    const int64_t c = 500 + 460 * M / 128 + steps * (19 + 11 * M / 128) * std::max(ctas, sms) / sms +
                      910 * M / 128 * std::max<int64_t>(ctas - sms, 0) / sms;
    if (M <= 16 || c < cost) best = 0;
  }
  return best;
}

// Which form a problem takes: 0 the persistent one (256 rows a work tile), else
// the split one (128 rows) with that many CTAs of a cluster on the keys of a
// tile, by their time on one B200 in units of 0.1 us.  Persistent: 1.7 us a
// key tile and 3 us a work tile, one after the other on an SM.  Split: 7 us
// and 1.4 us a key tile, in waves of the clusters that are resident at once
// (B200: 74 of two, 33 of four, 15 of eight).
// Measured: 4 x 1 query, 4109 keys, 32 heads on 8: 17.5 us in fours; 1 query,
// 4096 keys, 16 heads: 12.8 us in one wave of clusters, 21.5 in two of eights.
// clusters[s]: clusters of s CTAs resident at once.
inline int xattn_splits(int64_t rows, int64_t head_blocks, int64_t key_tiles, int64_t sms, const int* clusters) {
  int best = 0;
  int64_t cost = ceil_div(ceil_div(rows, 256) * head_blocks, sms) * (17 * key_tiles + 30) + 30;
  const int64_t units = ceil_div(rows, 128) * head_blocks;
  if (units > 65535) return best;
  for (int s = 1; s <= 8 && s <= key_tiles; ++s) {
    const int64_t c = ceil_div(units, clusters[s]) * (14 * ceil_div(key_tiles, s) + 70);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

}  // namespace w4a4
