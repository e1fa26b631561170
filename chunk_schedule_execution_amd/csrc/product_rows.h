// Products with few rows (single tokens, small groups of an expert) for gfx950: bound by
// reading the weights once.
#pragma once

#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

// 16 bytes of a row from element k on, zeros from k_end on. Vec: rows on the 16-byte grid
// and k_end a multiple of the vector.
template <typename T, bool Vec>
__device__ inline auto load_k(const T* row, int k, int k_end) {
  constexpr int V = 16 / int(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(V)));
  vec v;
  // a load from the row's begin in place of none: no branch, so all loads start together
  if constexpr (Vec) {
    v = *reinterpret_cast<const vec*>(row + (k < k_end ? k : 0));
    const vec zero = {};
    v = k < k_end ? v : zero;
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const T x = row[k + q < k_end ? k + q : 0];
      v[q] = k + q < k_end ? x : T(0.0f);
    }
  }
  return v;
}

// A workgroup computes 16 rows by 16 FN columns. Its four waves split the summed
// dimension by lines of 128 bytes, every operand value goes straight from memory into the
// registers of a matrix instruction (nothing is used twice within a workgroup, so LDS
// would only add a trip), and Deep lines per wave are in flight together. The waves' sums
// meet in LDS in the order of the waves. Bound by reading the weights: the 41 used of 64
// matrices of 2048 x 1024 bf16 in 26 us warm and 33 cold, 5.2 TB/s. Two sets of registers in
// flight instead of more waves lost (1 x 4096 x 16384: 41 us and 35). The summed dimension may also be split over
// gridDim.y workgroups, whose fp32 sums a second kernel adds up.
template <typename T, int FN, bool Vec, int Deep>
__device__ inline void product_rows(const ProductArgs& g, int slabs) {
  constexpr int V = 16 / int(sizeof(T)), kLine = 8 * V;  // values per line of 128 bytes
  __shared__ float sums[4][16][FN * 16 + 4];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int band = uniform(blockIdx.x / slabs);
  const int64_t col = int64_t(blockIdx.x - band * slabs) * (16 * FN);
  const RowTile t = find_tile(g.offsets, g.groups, g.m, 16, band);
  if (t.group < 0) return;
  const bool nothing = g.offsets && t.group == g.groups;
  const T* A = static_cast<const T*>(g.a);
  const T* B = static_cast<const T*>(g.b) + (nothing ? 0 : t.group * g.b_stride);
  f32x4 acc[FN] = {};
  if (!nothing) {
    const int k_end = int(g.k), lines = (k_end + kLine - 1) / kLine;
    const int first = int(int64_t(lines) * blockIdx.y / gridDim.y), last = int(int64_t(lines) * (blockIdx.y + 1) / gridDim.y);
    // rows behind the end repeat the last one: their results are not stored
    const T* row = A + min(t.row + (lane & 15), t.end - 1) * g.lda;
    const T* cols[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) cols[j] = B + min(col + j * 16 + (lane & 15), g.n - 1) * g.ldb;
    const int part = (lane >> 4) * V;
    typedef decltype(load_k<T, Vec>(A, 0, 0)) vec;
    for (int l0 = first + wave; l0 < last; l0 += 4 * Deep) {
      vec a[Deep][2], b[Deep][2][FN];
#pragma unroll
      for (int d = 0; d < Deep; ++d) {
        const int k = (l0 + 4 * d) * kLine + part, end = l0 + 4 * d < last ? k_end : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < FN; ++j) b[d][h][j] = load_k<T, Vec>(cols[j], k + h * 4 * V, end);
          a[d][h] = load_k<T, Vec>(row, k + h * 4 * V, end);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // loads stay ahead of all products
#pragma unroll
      for (int d = 0; d < Deep; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[j] = multiply(b[d][h][j], a[d][h], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4*>(&sums[wave][lane & 15][j * 16 + (lane >> 4) * 4]) = acc[j];
    __syncthreads();
  }
  for (int e = threadIdx.x; e < FN * 256; e += 256) {
    const int r = e / (FN * 16), c = e % (FN * 16);
    const int64_t at = t.row + r, n = col + c;
    if (at >= t.end || n >= g.n) continue;
    const float z = nothing ? 0.0f : (sums[0][r][c] + sums[1][r][c]) + (sums[2][r][c] + sums[3][r][c]);
    if (g.partial) *partial_at(g, blockIdx.y, at, n) = z;
    else finish_one<T>(g, z, at, n, t.group, nothing);
  }
}

template <typename T, int FN, bool Vec, int Deep>
__global__ __launch_bounds__(256) void product_rows_kernel(ProductArgs g, int slabs) {
  product_rows<T, FN, Vec, Deep>(g, slabs);
}

}  // namespace
}  // namespace prod
}  // namespace ccl
