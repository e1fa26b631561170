// The cross entropy's sums joined over blocks of columns and over shards, for gfx950.
#include <algorithm>
#include <cmath>

#include "layers.h"
#include "products_device.h"

namespace ccl {
namespace prod {

// Defined with their kernels in loss_tile_*.hip.
int loss_sums_bf16(const ProductArgs& g, const LossArgs& loss, ProductKind kind, hipStream_t s, std::string* err);
int loss_sums_f32(const ProductArgs& g, const LossArgs& loss, ProductKind kind, hipStream_t s, std::string* err);
int loss_slope_bf16(const ProductArgs& g, const LossArgs& loss, int64_t padded, ProductKind kind, hipStream_t s,
                    std::string* err);
int loss_slope_f32(const ProductArgs& g, const LossArgs& loss, int64_t padded, ProductKind kind, hipStream_t s,
                   std::string* err);
int product_onto_bf16(const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err);
int product_onto_f32(const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err);

namespace {

// A sum of exponentials, sum exp(top); top -inf: of nothing, or of zeros.
struct Sum {
  float top = -INFINITY, sum = 0.0f;
  __device__ inline void add(float t, float s) {
    const float m = fmaxf(top, t), base = m == -INFINITY ? 0.0f : m;
    sum = sum * exp_of_minus(base - top) + s * exp_of_minus(base - t);
    top = m;
  }
  __device__ inline float log() const { return (top == -INFINITY ? 0.0f : top) + logf(sum); }
};

// A workgroup: In rows, whose blocks are dealt out to 1024 / In runs, joined in order. 16 rows
// read whole lines; with few rows, 4 bring four times the workgroups (64 rows of 1024 blocks:
// 7.0 us in sixteens).
template <int In>
__global__ __launch_bounds__(1024) void loss_join_kernel(LossJoinArgs a) {
  constexpr int Runs = 1024 / In;
  __shared__ float tops[Runs][In], sums[Runs][In], picks[Runs][In];
  const int in = threadIdx.x % In, run = threadIdx.x / In;
  const int64_t row = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * In + in;
  Sum s;
  float pick = 0.0f;
  if (row < a.rows) {
    if (a.pairs) {
#pragma unroll 8
      for (int64_t b = run; b < a.blocks; b += Runs) {
        const float2 v = reinterpret_cast<const float2*>(a.pairs)[b * a.rows + row];
        s.add(v.x, v.y);
      }
    } else {
      for (int64_t b = run; b < a.blocks; b += Runs) {
        s.add(a.lse_parts[b * a.rows + row], 1.0f);
        pick += a.picked_parts[b * a.rows + row];
      }
    }
  }
  tops[run][in] = s.top;
  sums[run][in] = s.sum;
  picks[run][in] = pick;
  __syncthreads();
  for (int d = Runs / 2; d >= 1; d >>= 1) {
    if (run < d) {
      s.add(tops[run + d][in], sums[run + d][in]);
      pick += picks[run + d][in];
      tops[run][in] = s.top;
      sums[run][in] = s.sum;
      picks[run][in] = pick;
    }
    __syncthreads();
  }
  if (run || row >= a.rows) return;
  const float lse = s.log();
  const int target = a.targets[row];
  if (a.pairs) {
    const int at = target < 0 ? -1 : target - a.first;
    pick = at >= 0 && at < a.n ? a.picked[row] : 0.0f;
    a.picked[row] = pick;
  }
  a.lse[row] = lse;
  if (a.loss) a.loss[row] = unsigned(target) >= a.end ? 0.0f : lse - pick;
}

// ---- logits through memory ---------------------------------------------------------------
// Where a product is small enough to be split (or to have 16 rows at most), its fp32 sums go
// through the workspace, whose size the split outputs bound.

// One logit, or four neighbours, from the splits in order.
__device__ inline float4 logits4(const LossRowsArgs& a, int64_t row, int64_t c) {
  const int64_t ld = partial_ld(a.n);
  const float* p = a.partial + row * ld + c;
  float4 z = *reinterpret_cast<const float4*>(p);
  for (int s = 1; s < a.splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(p + int64_t(s) * a.rows * ld);
    z.x += v.x;
    z.y += v.y;
    z.z += v.z;
    z.w += v.w;
  }
  return z;
}

// A workgroup a row.
template <int Threads>
__global__ __launch_bounds__(Threads) void loss_rows_kernel(LossRowsArgs a, LossArgs loss) {
  __shared__ float tops[Threads / 64], sums[Threads / 64], pick;
  const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  if (row >= a.rows) return;
  const int target = loss.targets[row];
  const int at = target < 0 || target - loss.first >= a.n ? -1 : target - loss.first;
  if (threadIdx.x == 0) pick = 0.0f;
  __syncthreads();
  Sum s;
  for (int64_t c = threadIdx.x * 4; c < a.n; c += Threads * 4) {
    const float4 z = logits4(a, row, c);
    float v[4] = {z.x, z.y, z.z, z.w};
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (c + q == at) pick = v[q];
      if (c + q >= a.n) v[q] = -INFINITY;
      m = fmaxf(m, v[q]);
    }
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int q = 0; q < 4; ++q) sum += exp_of_minus(base - v[q]);
    s.add(m, sum);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const float t = __shfl_xor(s.top, d), u = __shfl_xor(s.sum, d);
    s.add(t, u);
  }
  if (threadIdx.x % 64 == 0) {
    tops[threadIdx.x / 64] = s.top;
    sums[threadIdx.x / 64] = s.sum;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < Threads / 64; ++w) s.add(tops[w], sums[w]);
  const float lse = s.log();
  a.lse_out[row] = lse;
  if (loss.picked) loss.picked[row] = pick;
  if (a.loss_out) a.loss_out[row] = unsigned(target) >= loss.end ? 0.0f : lse - pick;
}

// Four columns a thread; zeros in the columns from n up to ldz.
template <typename T>
__global__ __launch_bounds__(256) void loss_rows_slope_kernel(LossRowsArgs a, LossArgs loss) {
  typedef T four __attribute__((ext_vector_type(4)));
  const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t c = (int64_t(blockIdx.z) * 256 + threadIdx.x) * 4;
  if (row >= a.rows || c >= a.ldz) return;
  const int target = loss.targets[row];
  const bool out = unsigned(target) >= loss.end;
  const int at = out || target < loss.first ? -1 : target - loss.first;
  float v[4] = {};
  if (!out && c < a.n) {
    const float4 z = logits4(a, row, c);
    const float d = loss.dloss[row], lse = loss.lse[row];
    const float w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < a.n) v[q] = d * (exp_of_minus(lse - w[q]) - (c + q == at ? 1.0f : 0.0f));
  }
  four o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = narrow<T>(v[q]);
  *reinterpret_cast<four*>(static_cast<T*>(a.dz) + row * a.ldz + c) = o;
}

}  // namespace
}  // namespace prod

int loss_block(ProductKind kind) { return kind == kTile64 ? 32 : 64; }

int launch_loss_sums(int dtype, const ProductArgs& g, const LossArgs& loss, ProductKind kind, void* stream,
                     std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::loss_sums_bf16(g, loss, kind, s, err) : prod::loss_sums_f32(g, loss, kind, s, err);
}

int launch_loss_slope(int dtype, const ProductArgs& g, const LossArgs& loss, int64_t padded, ProductKind kind,
                      void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::loss_slope_bf16(g, loss, padded, kind, s, err)
                           : prod::loss_slope_f32(g, loss, padded, kind, s, err);
}

int launch_product_onto(int dtype, const ProductArgs& g, const ProductPlan& plan, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::product_onto_bf16(g, plan, s, err) : prod::product_onto_f32(g, plan, s, err);
}

int launch_loss_rows(const LossRowsArgs& args, const LossArgs& loss, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid = prod::flat_grid(args.rows);
  if (args.n > 4096) hipLaunchKernelGGL(prod::loss_rows_kernel<1024>, grid, dim3(1024), 0, s, args, loss);
  else hipLaunchKernelGGL(prod::loss_rows_kernel<256>, grid, dim3(256), 0, s, args, loss);
  return prod::hip_status("cross entropy launch", err);
}

int launch_loss_rows_slope(int dtype, const LossRowsArgs& args, const LossArgs& loss, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  dim3 grid = prod::flat_grid(args.rows);
  grid.z = unsigned((args.ldz + 1023) / 1024);
  if (dtype == CCL_BF16) hipLaunchKernelGGL(prod::loss_rows_slope_kernel<prod::bf16>, grid, dim3(256), 0, s, args, loss);
  else hipLaunchKernelGGL(prod::loss_rows_slope_kernel<float>, grid, dim3(256), 0, s, args, loss);
  return prod::hip_status("cross entropy gradient launch", err);
}

int launch_loss_join(const LossJoinArgs& args, void* stream, std::string* err) {
  const int in = args.rows < 1024 ? 4 : 16;
  hipLaunchKernelGGL(in == 4 ? prod::loss_join_kernel<4> : prod::loss_join_kernel<16>,
                     prod::flat_grid((args.rows + in - 1) / in), dim3(1024), 0, reinterpret_cast<hipStream_t>(stream), args);
  return prod::hip_status("cross entropy launch", err);
}

}  // namespace ccl
