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
int product_onto_bf16(const ProductArgs& g, const ProductPlan& plan, bool fresh, hipStream_t s, std::string* err);
int product_onto_f32(const ProductArgs& g, const ProductPlan& plan, bool fresh, hipStream_t s, std::string* err);

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

int launch_product_onto(int dtype, const ProductArgs& g, const ProductPlan& plan, bool fresh, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::product_onto_bf16(g, plan, fresh, s, err) : prod::product_onto_f32(g, plan, fresh, s, err);
}

int launch_loss_join(const LossJoinArgs& args, void* stream, std::string* err) {
  const int in = args.rows < 1024 ? 4 : 16;
  const int64_t n = (args.rows + in - 1) / in, x = std::min<int64_t>(n, 1 << 20);
  hipLaunchKernelGGL(in == 4 ? prod::loss_join_kernel<4> : prod::loss_join_kernel<16>,
                     dim3(unsigned(x), unsigned((n + x - 1) / x)), dim3(1024), 0, reinterpret_cast<hipStream_t>(stream), args);
  return prod::hip_status("cross entropy launch", err);
}

}  // namespace ccl
