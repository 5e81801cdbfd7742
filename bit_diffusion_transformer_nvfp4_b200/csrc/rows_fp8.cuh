// rows_fp8.cuh -- E4M3 codes with one fp32 scale per row: of a tensor as it
// stands, or of its root-mean-square norm after the residual's addition.
//
// Per row m of D columns, in fp32 and rounded once at each output:
//   h = x + r                      (r optional; hidden = bf16(h) optional)
//   v = h * w                      (w optional)
//   i = 1 / sqrt(sum(h^2) / D + eps)   (1 without the norm)
//   s = i * max|v| / 448           (1 when that is not a normal number)
//   code = E4M3_rn_satfinite(v * (i * (1 / s)))
//   normed = bf16(v * i)           (optional)
// The factor i is common to the row, so the sum of squares and max|v| come
// from one pass and one reduction, and the row stays in registers: every
// input is read once and every output written once.  That traffic (for
// x, r, hidden and codes 7 bytes an element) is the bound: norm of 16896 x
// 6144 107.5 us (6.8 TB/s), its codes alone 46.3 us (6.7 TB/s).  Short rows are
// bound by instruction issue (36888 x 128 without a residual: 3.6 us, 3.9 TB/s).
//
// Rows whose squares leave fp32's range (|h| from about 2^52 up, or below 2^-45
// with an eps that small) take their sum again, scaled by a power of two, from
// the inputs: a branch that other rows do not enter (rows_far).
//
// Two shapes: short rows (up to 1024 columns for the norm, which keeps the
// residual too, 2048 for the codes alone) take a power of two of lanes of one
// warp (shuffles only); wider ones a block of their own.  A thread holds V
// 16-byte vectors of the row.
#pragma once

#include "sm100.cuh"

namespace w4a4 {

constexpr int kRowsWarpThreads = 256;   // block size of the warp-per-row shape
constexpr int kRowsWarpVecs = 8;        // 16-byte vectors a lane holds at most
constexpr int kRowsBlockThreads = 512;  // most threads of the block-per-row shape
constexpr int kRowsMaxCols = kRowsBlockThreads * 8 * 8;

struct RowsFp8Params {
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;   // or nullptr
  const __nv_bfloat16* w;   // or nullptr
  __nv_bfloat16* hidden;    // or nullptr; may be x or r itself
  __nv_bfloat16* normed;    // or nullptr
  uint8_t* codes;           // or nullptr (then scales is unused)
  float* scales;
  int64_t rows, ldx, ldr, ldh, ldn, ldo;
  int cols;
  float eps, inv_cols;      // 1 / cols
  float sum_min;            // smallest sum of squares that counts as ordinary: kRowsSumMin, 0 where eps hides it
};

// A thread whose part of the sum is ordinary (kRowsSumMin .. kRowsSumMax) writes
// its hidden at once; one that is late waits until the row's sum is known, so
// that its inputs can be read again (hidden may be one of them).  A row is far
// where sum / cols + eps leaves kRowsMeanMin .. kRowsMeanMax.  In one that is far
// above, the threads that are not late have no more than 512 x 2^60, which is
// nothing beside 2^104; in one that is far below (sum < 2^-75) every thread is late.
constexpr float kRowsSumMin = 0x1p-60f, kRowsSumMax = 0x1p60f;
constexpr float kRowsMeanMin = 0x1p-90f, kRowsMeanMax = 0x1p104f;
constexpr float kRowsEpsMin = 0x1p-80f;  // from here up eps keeps every row from far below
static_assert(kRowsMaxCols <= 1 << 15, "far rows below have late threads only");

struct RowStats {
  float sum, top;  // sum of h^2, max |v|
};

// This thread's vectors t0, t0 + step, ... of a row, as loaded.
template <int V>
struct RowRaw {
  uint4 x[V], r[V];
};

template <int V, bool NORM>
__device__ __forceinline__ void rows_fetch(const RowsFp8Params& p, int64_t row, bool live, int t0, int step,
                                           RowRaw<V>& raw) {
  const int nv = p.cols >> 3;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + row * p.ldx);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int t = t0 + i * step;
    raw.x[i] = live && t < nv ? xr[t] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (NORM && p.r != nullptr) {
    const uint4* rr = reinterpret_cast<const uint4*>(p.r + row * p.ldr);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int t = t0 + i * step;
      raw.r[i] = live && t < nv ? rr[t] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

__device__ __forceinline__ void rows_hidden(const RowsFp8Params& p, int64_t row, int t, const float* h) {
  reinterpret_cast<uint4*>(p.hidden + row * p.ldh)[t] = make_uint4(
      pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]), pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
}

// v and the partial statistics, and hidden unless the thread is late.
template <int V, bool NORM>
__device__ __forceinline__ RowStats rows_take(const RowsFp8Params& p, int64_t row, bool live, int t0, int step,
                                              const RowRaw<V>& raw, float (&v)[8 * V], bool& late) {
  const int nv = p.cols >> 3;
  RowStats st = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t xs[4] = {raw.x[i].x, raw.x[i].y, raw.x[i].z, raw.x[i].w};
    float* vi = v + 8 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vi[2 * j] = bf16_lo(xs[j]);
      vi[2 * j + 1] = bf16_hi(xs[j]);
    }
    if (NORM) {
      if (p.r != nullptr) {
        const uint32_t rs[4] = {raw.r[i].x, raw.r[i].y, raw.r[i].z, raw.r[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          vi[2 * j] += bf16_lo(rs[j]);
          vi[2 * j + 1] += bf16_hi(rs[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) st.sum = fmaf(vi[j], vi[j], st.sum);
    }
  }
  late = NORM && !(st.sum >= p.sum_min && st.sum <= kRowsSumMax);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int t = t0 + i * step;
    float* vi = v + 8 * i;
    if (NORM) {
      if (p.hidden != nullptr && live && t < nv && !late) rows_hidden(p, row, t, vi);
      if (p.w != nullptr && t < nv) {
        const uint4 ww = __ldg(reinterpret_cast<const uint4*>(p.w) + t);
        const uint32_t wsv[4] = {ww.x, ww.y, ww.z, ww.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          vi[2 * j] *= bf16_lo(wsv[j]);
          vi[2 * j + 1] *= bf16_hi(wsv[j]);
        }
      }
    }
    st.top = fmaxf(st.top, fmaxf(fmaxf(fmaxf(fabsf(vi[0]), fabsf(vi[1])), fmaxf(fabsf(vi[2]), fabsf(vi[3]))),
                                 fmaxf(fmaxf(fabsf(vi[4]), fabsf(vi[5])), fmaxf(fabsf(vi[6]), fabsf(vi[7])))));
  }
  return st;
}

__device__ __forceinline__ bool rows_far(const RowsFp8Params& p, float sum) {
  const float mean = fmaf(sum, p.inv_cols, p.eps);
  return !(mean >= kRowsMeanMin && mean <= kRowsMeanMax);
}

// What the values of a row are multiplied with: pre is 1 except in rows that are
// far below, whose factor alone may leave fp32's range.
struct RowFactor {
  float pre, inv;
};

// The factor of a row that is far, and hidden of the threads that are late.
// With h and eps scaled by 2^-76 or 2^76 the sum stays between 2^-114 and 2^119.
// (A block comes here as a whole for a far row, its late threads alone for
// others; a warp for any of its lanes.)
template <bool BLOCK>
__device__ __forceinline__ RowFactor rows_far_factor(const RowsFp8Params& p, int64_t row, int t0, int step, bool late,
                                                     bool far, float sum, float* red) {
  const int nv = p.cols >> 3;
  const bool above = fmaf(sum, p.inv_cols, p.eps) > 1.0f;
  const float scale = above ? 0x1p-76f : 0x1p76f;
  float part = 0.0f;
  // (two elements at a time: the registers that this branch needs are the kernel's)
#pragma unroll 1
  for (int t = 4 * t0; late && t < 4 * nv; t += (t & 3) == 3 ? 4 * step - 3 : 1) {
    const uint32_t x = reinterpret_cast<const uint32_t*>(p.x + row * p.ldx)[t];
    float h0 = bf16_lo(x), h1 = bf16_hi(x);
    if (p.r != nullptr) {
      const uint32_t r = reinterpret_cast<const uint32_t*>(p.r + row * p.ldr)[t];
      h0 += bf16_lo(r);
      h1 += bf16_hi(r);
    }
    part = fmaf(h0 * scale, h0 * scale, part);
    part = fmaf(h1 * scale, h1 * scale, part);
    if (p.hidden != nullptr) reinterpret_cast<uint32_t*>(p.hidden + row * p.ldh)[t] = pack_bf16x2(h0, h1);
  }
  if (BLOCK && !far) return RowFactor{1.0f, 1.0f};
  for (int o = (BLOCK ? 32 : step) >> 1; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (BLOCK) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = part;
    __syncthreads();
    part = lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f;
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  }
  const float f = rsqrtf(fmaf(part, p.inv_cols, p.eps * scale * scale));
  return above ? RowFactor{1.0f, f * scale} : RowFactor{scale, f};
}

// The row's factor and scale, then this thread's outputs.
template <int V, bool NORM>
__device__ __forceinline__ void rows_store(const RowsFp8Params& p, int64_t row, int t0, int step, bool first,
                                           RowStats st, RowFactor by, float (&v)[8 * V]) {
  const int nv = p.cols >> 3;
  // the norm's quotients by the hardware's reciprocals (a few units of the 23rd
  // bit; the plain codes' are exact divisions, whose steps their definition
  // fixes): every lane of a short row does these
  float inv = NORM ? by.inv : 1.0f;
  if (NORM && (by.pre != 1.0f || !(st.top >= 0x1p-118f && st.top <= 0x1p125f))) {
    // 448 / max|v| would leave fp32's range or __fdividef's: the factor first,
    // and 1 / s below
#pragma unroll
    for (int i = 0; i < 8 * V; ++i) v[i] = v[i] * by.pre * inv;
    st.top = st.top * by.pre * inv;
    inv = 1.0f;
  }
  if (p.codes != nullptr) {
    float s = NORM ? st.top * inv * (1.0f / 448.0f) : st.top / 448.0f;
    const bool normal = s >= 1.17549435e-38f && s < INFINITY;
    if (!normal) s = 1.0f;
    if (first) p.scales[row] = s;
    // (i / s = 448 / max|v|)
    const float f = !normal ? inv
                    : NORM  ? __fdividef(inv != 1.0f ? 448.0f : 1.0f, inv != 1.0f ? st.top : s)
                            : 1.0f / s;
    uint2* out = reinterpret_cast<uint2*>(p.codes + row * p.ldo);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int t = t0 + i * step;
      const float* vi = v + 8 * i;
      if (t < nv)
        out[t] = make_uint2(cvt_e4m3x2(vi[1] * f, vi[0] * f) | (cvt_e4m3x2(vi[3] * f, vi[2] * f) << 16),
                            cvt_e4m3x2(vi[5] * f, vi[4] * f) | (cvt_e4m3x2(vi[7] * f, vi[6] * f) << 16));
    }
  }
  if (NORM && p.normed != nullptr) {
    uint4* out = reinterpret_cast<uint4*>(p.normed + row * p.ldn);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int t = t0 + i * step;
      const float* vi = v + 8 * i;
      if (t < nv)
        out[t] = make_uint4(pack_bf16x2(vi[0] * inv, vi[1] * inv), pack_bf16x2(vi[2] * inv, vi[3] * inv),
                            pack_bf16x2(vi[4] * inv, vi[5] * inv), pack_bf16x2(vi[6] * inv, vi[7] * inv));
    }
  }
}

// A row per `lanes` lanes (a power of two up to 32) of a warp: no barriers, and
// four vectors a lane (six or eight where that fills the warp, for the codes
// alone), so that the reduction and the row's quotients are shared by many
// elements (a 128-column row on 16 lanes of one vector took 7.2 us for 36888
// rows).
template <int V, bool NORM>
__global__ void __launch_bounds__(kRowsWarpThreads) rows_fp8_warp_kernel(const RowsFp8Params p, int lanes) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowsWarpThreads / lanes) + threadIdx.x / lanes;
  const int t0 = threadIdx.x & (lanes - 1);
  const bool live = row < p.rows;  // (the shuffles take whole warps)
  RowRaw<V> raw;
  rows_fetch<V, NORM>(p, row, live, t0, lanes, raw);
  float v[8 * V];
  bool late;
  RowStats st = rows_take<V, NORM>(p, row, live, t0, lanes, raw, v, late);
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    if (NORM) st.sum += __shfl_xor_sync(0xffffffffu, st.sum, o);
    st.top = fmaxf(st.top, __shfl_xor_sync(0xffffffffu, st.top, o));
  }
  RowFactor by = {1.0f, NORM ? rsqrtf(fmaf(st.sum, p.inv_cols, p.eps)) : 1.0f};
  if (NORM) {
    const bool far = rows_far(p, st.sum);
    if (__any_sync(0xffffffffu, far || late)) {
      const RowFactor f = rows_far_factor<false>(p, row, t0, lanes, late && live, far, st.sum, nullptr);
      if (far) by = f;
    }
  }
  if (live) rows_store<V, NORM>(p, row, t0, lanes, t0 == 0, st, by, v);
}

// A row per block.
template <int V, bool NORM>
__global__ void __launch_bounds__(kRowsBlockThreads) rows_fp8_block_kernel(const RowsFp8Params p) {
  __shared__ float red_sum[32], red_top[32], red_far[32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  RowRaw<V> raw;
  rows_fetch<V, NORM>(p, row, true, threadIdx.x, blockDim.x, raw);
  float v[8 * V];
  bool late;
  RowStats st = rows_take<V, NORM>(p, row, true, threadIdx.x, blockDim.x, raw, v, late);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (NORM) st.sum += __shfl_xor_sync(0xffffffffu, st.sum, o);
    st.top = fmaxf(st.top, __shfl_xor_sync(0xffffffffu, st.top, o));
  }
  if (lane == 0) {
    if (NORM) red_sum[warp] = st.sum;
    red_top[warp] = st.top;
  }
  __syncthreads();
  st.sum = NORM && lane < warps ? red_sum[lane] : 0.0f;
  st.top = lane < warps ? red_top[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (NORM) st.sum += __shfl_xor_sync(0xffffffffu, st.sum, o);
    st.top = fmaxf(st.top, __shfl_xor_sync(0xffffffffu, st.top, o));
  }
  RowFactor by = {1.0f, NORM ? rsqrtf(fmaf(st.sum, p.inv_cols, p.eps)) : 1.0f};
  if (NORM) {
    // (every thread has added the same numbers in the same pairs, so they agree
    // on whether the row is far)
    const bool far = rows_far(p, st.sum);
    if (far || late) {
      const RowFactor f = rows_far_factor<true>(p, row, threadIdx.x, blockDim.x, late, far, st.sum, red_far);
      if (far) by = f;
    }
  }
  rows_store<V, NORM>(p, row, threadIdx.x, blockDim.x, threadIdx.x == 0, st, by, v);
}

}  // namespace w4a4
