// Device helpers shared by the product and exchange kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ccl.h"
#include "products.h"

namespace ccl {
namespace prod {

typedef __bf16 bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ inline float widen(bf16 v) { return float(v); }
__device__ inline float widen(float v) { return v; }
template <typename T>
__device__ inline T narrow(float v) {
  return T(v);  // nearest-even
}

__device__ inline float act_value(float z, int act) {
  switch (act) {
    case CCL_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case CCL_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case CCL_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    case CCL_ACT_SILU: return z / (1.0f + expf(-z));
  }
  return z;
}

__device__ inline float act_slope(float z, int act) {
  switch (act) {
    case CCL_ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case CCL_ACT_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    case CCL_ACT_GELU_TANH: {
      const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
      return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * 0.79788456080286536f * (1.0f + 0.134145f * z * z);
    }
    case CCL_ACT_SILU: {
      const float p = 1.0f / (1.0f + expf(-z));
      return p * (1.0f + z * (1.0f - p));
    }
  }
  return 1.0f;
}

// One tile of rows of a group.
struct RowTile {
  int group;    // `groups` for the rows behind the last group, -1 past the last tile
  int index;    // tile number over all groups
  int64_t row;  // first row
  int64_t end;  // end of the group
};

// The tile-th tile of `height` rows when every group is cut into tiles of its own. Runs
// on whole waves: lane l reads offset l, a running maximum makes the bounds monotone
// (offset 0 counts as 0, values are clamped to [0, rows]), a prefix sum counts tiles.
// With at most 64 groups that is one round of loads and 12 shuffles; more groups take a
// round for every 64.
__device__ inline RowTile find_tile(const int32_t* offsets, int groups, int64_t rows, int height, int tile,
                                    bool with_rest) {
  const int lane = threadIdx.x & 63;
  if (offsets == nullptr) {
    const int64_t row = int64_t(tile) * height;
    return {row < rows ? 0 : -1, tile, row, rows};
  }
  int carry_tiles = 0, carry_max = 0;
  const int last = with_rest ? groups : groups - 1;
  for (int base = 0; base <= last; base += 64) {
    const int e = base + lane;
    int hi = 0;
    if (e < groups)
      hi = max(0, min(offsets[e + 1], int(rows)));
    else
      hi = int(rows);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(hi, d);
      if (lane >= d) hi = max(hi, v);
    }
    hi = max(hi, carry_max);
    int lo = __shfl_up(hi, 1);
    if (lane == 0) lo = carry_max;
    int tiles = e <= last ? int((int64_t(hi) - lo + height - 1) / height) : 0;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    upto += carry_tiles;
    const unsigned long long hit = __ballot(tile < upto);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      const int first = __shfl(upto - tiles, l);
      const int64_t row = int64_t(__shfl(lo, l)) + int64_t(tile - first) * height;
      return {base + l, tile, row, int64_t(__shfl(hi, l))};
    }
    carry_tiles = __shfl(upto, 63);
    carry_max = __shfl(hi, 63);
  }
  return {-1, tile, 0, 0};
}

// Bounds of one group, with the same reading of the offsets.
__device__ inline void group_bounds(const int32_t* offsets, int64_t rows, int group, int64_t& lo, int64_t& hi) {
  if (offsets == nullptr) {
    lo = 0;
    hi = rows;
    return;
  }
  const int lane = threadIdx.x & 63;
  int top = 0;  // running maximum of the offsets up to the group's begin
  for (int e = 1 + lane; e <= group; e += 64) top = max(top, min(offsets[e], int(rows)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d));
  lo = top;
  hi = max(top, min(offsets[group + 1], int(rows)));
}

}  // namespace prod
}  // namespace ccl
