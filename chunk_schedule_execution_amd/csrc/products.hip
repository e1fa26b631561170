// Products beside the collectives for gfx950: C = act(A B^T + bias) + residual, plain or
// grouped by expert with ragged sizes, for the forward pass and both gradients.
#include <algorithm>
#include <cmath>

#include "products_device.h"

namespace ccl {
namespace prod {

// Defined with their kernels in product_tile_*.hip and product_rows.hip.
int launch_tile_bf16(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, const ProductPlan& plan,
                     hipStream_t s, std::string* err);
int launch_tile_f32(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, const ProductPlan& plan,
                    hipStream_t s, std::string* err);
int launch_rows(int dtype, const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err);

namespace {

// ---- operands off the 16-byte grid ------------------------------------------------------
// Rows copied to a stride of whole vectors, zeros behind their end: one pass over the
// operand, 5 us for the 1111 x 1001 of an odd product. Both operands in one launch.
struct Regrid {
  const void* src = nullptr;
  void* dst = nullptr;
  int64_t ld = 0, rows = 0, len = 0, ld_dst = 0;
};

template <typename T>
__global__ __launch_bounds__(256) void regrid_kernel(Regrid first, Regrid second) {
  const Regrid g = blockIdx.z ? second : first;
  const T* src = static_cast<const T*>(g.src);
  T* dst = static_cast<T*>(g.dst);
  const int64_t c = int64_t(blockIdx.y) * 1024 + threadIdx.x;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = c + i * 256;
      if (at < g.ld_dst) dst[r * g.ld_dst + at] = at < g.len ? src[r * g.ld + at] : T(0.0f);
    }
}

int regrid(int dtype, const Regrid& first, const Regrid& second, hipStream_t s, std::string* err) {
  const dim3 grid(unsigned(std::min<int64_t>(std::max(first.rows, second.rows), 1 << 20)),
                  unsigned((std::max(first.ld_dst, second.ld_dst) + 1023) / 1024), second.rows ? 2 : 1);
  if (dtype == CCL_BF16) hipLaunchKernelGGL(regrid_kernel<bf16>, grid, dim3(256), 0, s, first, second);
  else hipLaunchKernelGGL(regrid_kernel<float>, grid, dim3(256), 0, s, first, second);
  return hip_status("regrid launch", err);
}

// ---- joining the splits of the summed dimension -------------------------------------------
// A workgroup takes 16 rows of a group by 256 columns, 8 columns per thread, and adds the
// splits in order.
constexpr int kJoinRows = 16;

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs g, int splits) {
  const RowTile t = find_tile(g.offsets, g.groups, g.m, kJoinRows, blockIdx.x);
  const int64_t c = int64_t(blockIdx.y) * 256 + (threadIdx.x & 31) * 8;
  if (t.group < 0 || c >= g.n) return;
  const bool nothing = g.offsets && t.group == g.groups;
  const int64_t end = min(t.end, t.row + kJoinRows);
  const int n = int(min(int64_t(8), g.n - c));
  const int64_t first = t.row + (threadIdx.x >> 5);
  Finish<T> finish(g, static_cast<T*>(g.c), first, 8, c, n, t.group, nothing);
  for (int64_t r = first; r < end; r += 8) {
    float z[8] = {};
    if (!nothing) {
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        float v[8];
        load8(partial_at(g, s, r, c), true, n, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) z[q] += v[q];
      }
    }
    finish.row(z);
    finish.next();
  }
}

int join(int dtype, const ProductArgs& g, int splits, hipStream_t s, std::string* err) {
  const dim3 grid(unsigned((g.m + kJoinRows - 1) / kJoinRows + (g.offsets ? g.groups : 0)), unsigned((g.n + 255) / 256));
  if (dtype == CCL_BF16) hipLaunchKernelGGL(join_kernel<bf16>, grid, dim3(256), 0, s, g, splits);
  else hipLaunchKernelGGL(join_kernel<float>, grid, dim3(256), 0, s, g, splits);
  return hip_status("join launch", err);
}

// ---- slope and bias gradient ---------------------------------------------------------
// One pass over dout and preact: a workgroup takes a tile of rows of one group by 256
// columns, 8 columns (16 or 32 bytes) per thread, and leaves one fp32 sum per column and
// tile; a second kernel adds the tiles of a group in order, so the sums do not depend on
// the order in which workgroups run. Bound by memory: 8192 x 4096 bf16 (two reads, one
// write, 201 MB) in 42 us, 4.8 TB/s. Both operands are read around the caches, which leaves
// those to dz for the products behind it: with them 443 us for 449.
constexpr int kSlopeLanes = 8;  // rows that a workgroup has in hand at a time

// Rows of a tile: 64, fewer where those would not fill the chip, more where a grid could
// not hold the tiles.
int slope_height(int64_t rows, int64_t n) {
  if (rows >= int64_t(1) << 26) return 4096;
  return rows / 64 * ((n + 255) / 256) < 1024 ? 16 : 64;
}

template <typename T>
__global__ __launch_bounds__(256) void slope_kernel(SlopeArgs g, int height, bool vec_o, bool vec_p) {
  __shared__ float sums[kSlopeLanes][256];
  const RowTile t = find_tile(g.offsets, g.groups, g.rows, height, blockIdx.x);
  if (t.group < 0) return;
  const int64_t c = int64_t(blockIdx.y) * 256 + (threadIdx.x & 31) * 8;
  const int n = int(min(int64_t(8), g.n - c)), lane = threadIdx.x >> 5;
  const T* dout = static_cast<const T*>(g.dout);
  const T* preact = static_cast<const T*>(g.preact);
  T* dz = static_cast<T*>(g.dz);
  const bool nothing = g.offsets && t.group == g.groups;
  const int64_t end = min(t.end, t.row + height);
  float sum[8] = {};
#pragma unroll 2
  for (int64_t r = t.row + lane; r < end; r += kSlopeLanes) {
    float v[8] = {};
    if (!nothing && n > 0) {
      load8<true>(dout + r * g.ldo + c, vec_o, n, v);
      if (g.act != CCL_ACT_NONE) {
        float z[8];
        load8<true>(preact + r * g.ldp + c, vec_p, n, z);
        slope8(v, z, g.act);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < n ? v[q] : 0.0f;
      }
    }
    // the rounding of dz to the operands' type: what a stored gradient has everywhere
    if (dz && c < g.ldz) store8(dz + r * g.ldz + c, true, int(min(int64_t(8), g.ldz - c)), v);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] += v[q];
  }
  if (!g.dbias || nothing) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) sums[lane][(threadIdx.x & 31) * 8 + q] = sum[q];
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int l = 0; l < kSlopeLanes; ++l) total += sums[l][threadIdx.x];
  const int64_t at = int64_t(blockIdx.y) * 256 + threadIdx.x;
  if (at < g.n) g.partial[int64_t(t.index) * g.n + at] = total;
}

// dbias[group][c]: the partial sums of the group's tiles, 4 interleaved runs of them and
// then those, always in the same order. A workgroup: 64 columns.
template <typename T>
__global__ __launch_bounds__(256) void bias_sum_kernel(SlopeArgs g, int height) {
  __shared__ float sums[4][64];
  const int64_t c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int run = threadIdx.x >> 6;
  int64_t first, last;
  group_tiles(g.offsets, g.groups, g.rows, height, blockIdx.y, first, last);
  float sum = 0.0f;
  if (c < g.n) {
#pragma unroll 8
    for (int64_t tile = first + run; tile < last; tile += 4) sum += g.partial[tile * g.n + c];
  }
  sums[run][threadIdx.x & 63] = sum;
  __syncthreads();
  if (run == 0 && c < g.n)
    static_cast<T*>(g.dbias)[int64_t(blockIdx.y) * g.n + c] =
        narrow<T>((sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]));
}

template <typename T>
int slope_t(const SlopeArgs& g, hipStream_t s, std::string* err) {
  const int height = slope_height(g.rows, g.n);
  auto grid16 = [](const void* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(T) % 16 == 0;
  };
  if (g.rows > 0 && (g.dz || g.dbias))
    hipLaunchKernelGGL(slope_kernel<T>,
                       dim3(unsigned(slope_tiles(g.rows, g.n, g.offsets ? g.groups : 0)), unsigned((std::max(g.n, g.ldz) + 255) / 256)),
                       dim3(256), 0, s, g, height, grid16(g.dout, g.ldo), grid16(g.preact, g.ldp));
  if (g.dbias)
    hipLaunchKernelGGL(bias_sum_kernel<T>, dim3(unsigned((g.n + 63) / 64), unsigned(g.groups)), dim3(256), 0, s, g, height);
  return hip_status("bias gradient launch", err);
}

}  // namespace
}  // namespace prod

int64_t slope_tiles(int64_t rows, int64_t n, int groups) {
  const int height = prod::slope_height(rows, n);
  return (rows + height - 1) / height + groups;
}

int launch_slope(int dtype, const SlopeArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::slope_t<prod::bf16>(args, s, err) : prod::slope_t<float>(args, s, err);
}

namespace {

// The tile size and the number of splits that should take least time. A workgroup's step
// (128 bytes of the summed dimension) takes, by the number of workgroups on its compute
// unit at a time, measured at 1024^2, 2048^2 and 4096^2 by 4096 (us):
//             alone   more of them                  start and end of a tile
//   bf16  64   0.41   0.68 for 4                    4
//   bf16 128   0.62   0.98 for 2                    5
//   bf16 256   1.40   (its LDS fills the unit)      10
//   fp32  64   0.60   0.50 each                     4
//   fp32 128   1.90   1.90 each                     5
// fp32 is bound by the matrix instructions in either size; in bf16 a larger tile reads
// less per product but leaves units idle: 2048^2 x 4096 takes 47 us in 64s or 128s and
// 87 in 256s, 4096^2 x 4096 189, 130 and 112. Splits cost a second kernel (5 us) and the
// partial sums' way through memory (written and read at 3.5 TB/s): 512^2 x 4096 takes 31 us
// unsplit and 17 in 4 splits of 64s, 1024^2 x 1024 11 and 16 in 2. Operands from memory are
// read at 5.6 TB/s at best, and slower by few workgroups, whose two steps in flight are too
// little: 32 x 4096 x 16384 in 64s takes 54 us unsplit (one workgroup per unit), 42 in 2
// splits and 36 in 4.
void choose_tile(int dtype, ProductMode mode, const ProductArgs& g, ProductPlan& p) {
  struct Size {
    ProductKind kind;
    int edge, resident;
    double alone, full, ends;
  };
  static constexpr Size kBf16[] = {{kTile64, 64, 4, 0.41, 0.68, 4}, {kTile128, 128, 2, 0.62, 0.98, 5}, {kTile256, 256, 1, 1.4, 1.4, 10}};
  static constexpr Size kF32[] = {{kTile64, 64, 4, 0.60, 2.0, 4}, {kTile128, 128, 2, 1.9, 3.8, 5}};
  const Size* sizes = dtype == CCL_BF16 ? kBf16 : kF32;
  const int count = dtype == CCL_BF16 ? 3 : 2;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  constexpr int64_t kUnits = 256;
  const double summed = double(mode == kRaggedK ? g.k / std::max(1, g.groups) : g.k);
  const double steps = std::max(1.0, std::ceil(summed * (dtype == CCL_BF16 ? 2 : 4) / 128));
  const double weights = double(g.n) * double(g.k) * (mode == kRaggedM ? g.groups : 1);
  const double bytes = (double(g.m) * double(g.k) + weights) * (dtype == CCL_BF16 ? 2 : 4);
  double best = 0;
  for (int i = 0; i < count; ++i) {
    const Size& z = sizes[i];
    // groups of rows end in half a tile on average
    const double bands = mode == kRaggedM && g.groups > 1 ? double(g.m) / z.edge + 0.5 * std::min<int64_t>(g.groups, g.m)
                                                          : double(up(g.m, z.edge));
    const double tiles = std::max(1.0, bands) * double(up(g.n, z.edge)) * (mode == kRaggedK ? g.groups : 1);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (mode == kRaggedK || steps < 4 * splits)) break;
      const int64_t each = int64_t(std::ceil(tiles * splits / kUnits));  // workgroups per compute unit
      auto step = [&](int64_t n) { return z.resident == 1 || n <= 1 ? z.alone * n : z.alone + (z.full - z.alone) * (n - 1) / (z.resident - 1); };
      const double rounds = double(each / z.resident);
      double us = std::ceil(steps / splits) * (rounds * step(z.resident) + step(each % z.resident));
      const double rate = std::min(5.6, 1.4 + 1.4 * z.edge / 64 * double(std::min<int64_t>(each, z.resident)));  // MB per us
      us = std::max(us, bytes / (rate * 1e6)) + z.ends * (rounds + (each % z.resident != 0));
      if (splits > 1) us += 5 + 2.0 * splits * double(g.m) * double(g.n) * 4 / 3.5e6;
      if (best == 0 || us < best) {
        best = us;
        p.kind = z.kind;
        p.splits = splits;
      }
    }
  }
}

// Workgroups of 256 threads that one dimension of a grid holds: fewer than 2^32 threads.
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 24) - 1;

}  // namespace

int64_t rows16_workgroups(ProductMode mode, const ProductArgs& g, int columns) {
  const int64_t bands = (g.m + 15) / 16 + (mode == kPlain ? 0 : g.groups);
  return bands * ((g.n + 16 * columns - 1) / (16 * columns));
}

ProductPlan plan_product(int dtype, bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g,
                         OperandGrid a_grid, OperandGrid b_grid) {
  ProductPlan p;
  const int64_t size = dtype == CCL_BF16 ? 2 : 4, v = 16 / size;
  const bool on_a = a_grid == kPadded || (a_grid == kByStrides && g.lda % v == 0 && (a_by_k ? g.m : g.k) % v == 0);
  const bool on_b = b_grid == kPadded || (b_grid == kByStrides && g.ldb % v == 0 && (b_by_k ? g.n : g.k) % v == 0);
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  // Few rows (16, or on average 8 in a group) are bound by reading the weights, and there
  // the kernel without LDS has less to wait for: 64 rows over 64 groups of 2048 x 1024 bf16
  // take 37 us and 45 in tiles of 64, 512 rows 57 and 65, 1 x 4096 x 16384 fp32 64 and 80, 4 x
  // 1024 x 1024 bf16 4.5 and 9. One large bf16 matrix the tiles read faster (1 x 4096 x 16384:
  // 32 us and 35). Weights off the 16-byte grid this kernel reads as they are, uncopied.
  // Its grid has a workgroup for every tile of 16 rows, one more per group, and holds fewer
  // than 2^32 threads; beyond that the tiles, whose grid does not grow, take the call.
  const int64_t mean = g.m / g.groups;
  const bool few = g.groups > 1 ? mean <= 8 : g.m <= 16;
  if (!a_by_k && !b_by_k && mode != kRaggedK && few && rows16_workgroups(mode, g, 2) <= kMaxWorkgroups &&
      (dtype == CCL_F32 || g.groups > 1 || !on_a || !on_b || g.n * g.k * size <= (32 << 20))) {
    p.kind = kRows16;
    p.vec = on_a && on_b;
    const int64_t bands = up(g.m, 16) + (g.groups > 1 ? std::min<int64_t>(g.groups, g.m) : 0);
    p.columns = bands * up(g.n, 32) >= 512 ? 2 : 1;
    const int64_t wgs = std::max<int64_t>(1, bands * up(g.n, 16 * p.columns));
    p.splits = int(std::max<int64_t>(1, std::min<int64_t>(512 / wgs, g.k * size / 4096)));
  } else {
    choose_tile(dtype, mode, g, p);
    p.copy_a = !on_a;
    p.copy_b = !on_b;
    p.ld_a = up(a_by_k ? g.m : g.k, v) * v;
    p.ld_b = up(b_by_k ? g.n : g.k, v) * v;
  }
  // bytes of the copies: every stored row
  const int64_t rows_a = a_by_k ? g.k : g.m;
  const int64_t rows_b = (b_by_k ? g.k : g.n) * (mode == kRaggedM ? g.groups : 1);
  p.at_b = p.copy_a ? up(rows_a * p.ld_a * size, 16) * 16 : 0;
  p.at_partial = p.at_b + (p.copy_b ? up(rows_b * p.ld_b * size, 16) * 16 : 0);
  p.bytes = p.at_partial + (p.splits > 1 ? p.splits * g.m * partial_ld(g.n) * 4 : 0);
  return p;
}

int launch_product(int dtype, bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& args,
                   const ProductPlan& plan, void* workspace, void* stream, std::string* err) {
  using namespace prod;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  ProductArgs g = args;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Regrid copy[2];
  int copies = 0;
  if (plan.copy_a) {
    copy[copies++] = {g.a, ws, g.lda, a_by_k ? g.k : g.m, a_by_k ? g.m : g.k, plan.ld_a};
    g.a = ws;
    g.lda = plan.ld_a;
  }
  if (plan.copy_b) {
    // the groups' matrices follow each other, so their rows are one run of rows
    const int64_t rows = (b_by_k ? g.k : g.n) * (mode == kRaggedM ? g.groups : 1);
    copy[copies++] = {g.b, ws + plan.at_b, g.ldb, rows, b_by_k ? g.n : g.k, plan.ld_b};
    g.b = ws + plan.at_b;
    g.ldb = plan.ld_b;
    g.b_stride = (b_by_k ? g.k : g.n) * plan.ld_b;
  }
  // (no rows: the gradient of no rows, whose products are empty sums)
  if (copies && std::max(copy[0].rows, copy[1].rows) > 0)
    if (int rc = regrid(dtype, copy[0], copy[1], s, err)) return rc;
  if (plan.splits > 1) g.partial = reinterpret_cast<float*>(ws + plan.at_partial);
  int rc;
  if (plan.kind == kRows16) rc = launch_rows(dtype, g, plan, s, err);
  else if (dtype == CCL_BF16) rc = launch_tile_bf16(a_by_k, b_by_k, mode, g, plan, s, err);
  else rc = launch_tile_f32(a_by_k, b_by_k, mode, g, plan, s, err);
  if (rc || plan.splits == 1) return rc;
  return join(dtype, g, plan.splits, s, err);
}

}  // namespace ccl
