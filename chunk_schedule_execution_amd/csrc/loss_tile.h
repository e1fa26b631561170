// Products of the cross entropy for gfx950: tiles of logits that are reduced to a row's
// maximum and sum, or turned into their gradient, before they leave the registers.
#pragma once

#include <climits>
#include <cmath>

#include "layers.h"
#include "product_tile.h"

namespace ccl {
namespace prod {
namespace {

constexpr float kLog2e = 1.44269504088896341f;

// exp(z - base) by the hardware's power of 2: one rounding of the argument, so off by 2^-24 of
// |z - base| and of |base| and a step. Where base log2(e) may be past fp32's range, values are
// 2^102 apart and more: z is base or so far off that any power is 1 or 0.
struct ExpFrom {
  float scale, base2;
  __device__ inline explicit ExpFrom(float base)
      : scale(fabsf(base) < 0x1p126f ? kLog2e : 1.0f), base2(base * scale) {}
  __device__ inline float operator()(float z) const { return __builtin_amdgcn_exp2f(fmaf(z, scale, -base2)); }
};

// Column of a target, negative where there is none.
__device__ inline int target_column(int target, int first) { return target < 0 ? -1 : max(-1, target - first); }

// A lane holds, of every 16 rows, row lane & 15 and, of every 16 columns, four from
// 4 (lane >> 4) on. The column of value q of fragment j, counted from the wave's first.
__device__ inline int held_column(int lane, int j, int q) { return j * 16 + (lane >> 4) * 4 + q; }

// Leaves per row the maximum of a wave's columns and the sum of exp(z - maximum): 8 bytes for
// 64 logits. The maximum is the wave's own, so no wave waits for another.
struct RowSums {
  static constexpr bool kTakes = true, kAdds = false, kPlainStores = false;
  LossArgs loss;

  template <int FM>
  struct Rows {
    int at[FM];
    __device__ inline void load(const RowSums& s, const ProductArgs&, const TileJob& job, int wm) {
      const int lane = here(threadIdx.x & 63);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int in = wm + i * 16 + (lane & 15);
        const int target = in < job.m_end - job.row ? s.loss.targets[int64_t(job.row) + in] : -1;
        at[i] = target_column(target, s.loss.first);
      }
    }
  };

  template <int FM, int FN>
  __device__ inline void take(f32x4 (&acc)[FM][FN], const Rows<FM>& rows, const ProductArgs& g, const TileJob& job,
                              int wm, int wn) const {
    const int lane = here(threadIdx.x & 63);
    const int left = int(g.n) - job.col - wn;  // columns of this wave and behind it
    if (left <= 0) return;
    float* const to = loss.sums + int64_t((job.col + wn) / (FN * 16)) * g.m * 2;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int in = wm + i * 16 + (lane & 15);
      if (left < FN * 16) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (held_column(lane, j, q) >= left) acc[i][j][q] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, acc[i][j][q]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const ExpFrom exp_from(m == -INFINITY ? 0.0f : m);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += exp_from(acc[i][j][q]);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (in >= job.m_end - job.row) continue;
      const int64_t row = int64_t(job.row) + in;
      if (lane < 16) *reinterpret_cast<float2*>(to + row * 2) = make_float2(m, sum);
      const int at = rows.at[i] < g.n ? rows.at[i] - job.col - wn : -1;
      if (at < 0 || at >= FN * 16) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (held_column(lane, j, q) == at) loss.picked[row] = acc[i][j][q];
    }
  }
  template <int FM, int FN>
  __device__ inline void change(f32x4 (&)[FM][FN], const Rows<FM>&, const ProductArgs&, const TileJob&, int) const {}
  __device__ inline int64_t columns(const ProductArgs& g) const { return g.n; }
};

// Turns logits into their gradient, which is then written as a product's results are.
struct LossSlope {
  static constexpr bool kTakes = false, kAdds = false, kPlainStores = true;
  LossArgs loss;
  int64_t padded;

  template <int FM>
  struct Rows {
    int at[FM];  // INT_MIN: left out
    float lse[FM], d[FM];
    __device__ inline void load(const LossSlope& s, const ProductArgs&, const TileJob& job, int wm) {
      const int lane = here(threadIdx.x & 63);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int in = wm + i * 16 + (lane & 15);
        const bool there = in < job.m_end - job.row;
        const int64_t row = int64_t(job.row) + in;
        const int target = there ? s.loss.targets[row] : -1;
        at[i] = unsigned(target) >= s.loss.end ? INT_MIN : target_column(target, s.loss.first);
        lse[i] = there ? s.loss.lse[row] : 0.0f;
        d[i] = there ? s.loss.dloss[row] : 0.0f;
      }
    }
  };

  template <int FM, int FN>
  __device__ inline void change(f32x4 (&acc)[FM][FN], const Rows<FM>& rows, const ProductArgs& g, const TileJob& job,
                                int wn) const {
    const int lane = here(threadIdx.x & 63);
    const int first = job.col + wn, left = int(g.n) - first;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const bool out = rows.at[i] == INT_MIN;
      const ExpFrom exp_from(rows.lse[i]);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = out ? 0.0f : rows.d[i] * exp_from(acc[i][j][q]);
      const int at = out ? -1 : rows.at[i] - first;
      if (__ballot(at >= 0 && at < FN * 16)) {  // of a row's columns few waves hold the target
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (held_column(lane, j, q) == at) acc[i][j][q] -= rows.d[i];
      }
    }
    if (left < FN * 16) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (held_column(lane, j, q) >= left) acc[i][j][q] = 0.0f;
    }
  }
  __device__ inline int64_t columns(const ProductArgs&) const { return padded; }
};

template <typename T, bool ByK, class End>
int launch_end(const ProductArgs& g, const End& end, ProductKind kind, int splits, hipStream_t s, std::string* err) {
  if constexpr (sizeof(T) == 2)
    if (kind == kTile256) return launch_tile_as<T, false, ByK, 256, 256, 2, 4>(kPlain, g, end, splits, s, err);
  if (kind == kTile64) return launch_tile_as<T, false, ByK, 64, 64, 2, 2>(kPlain, g, end, splits, s, err);
  return launch_tile_as<T, false, ByK, 128, 128, 2, 2>(kPlain, g, end, splits, s, err);
}

}  // namespace
}  // namespace prod
}  // namespace ccl
