// Instances of the few-row product kernel.
#include "product_rows.h"

namespace ccl {
namespace prod {
namespace {

template <typename T, int FN, int Deep>
int go(const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err) {
  const int64_t slabs = (g.n + 16 * FN - 1) / (16 * FN);
  // the plan has seen to it that a grid holds them
  const dim3 grid(unsigned(rows16_workgroups(g.offsets ? kRaggedM : kPlain, g, FN)), plan.splits);
  if (plan.vec)
    hipLaunchKernelGGL((product_rows_kernel<T, FN, true, Deep>), grid, dim3(256), 0, s, g, int(slabs));
  else
    hipLaunchKernelGGL((product_rows_kernel<T, FN, false, Deep>), grid, dim3(256), 0, s, g, int(slabs));
  return hip_status("product launch", err);
}

template <typename T>
int pick(const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err) {
  return plan.columns == 1 ? go<T, 1, 4>(g, plan, s, err) : go<T, 2, 4>(g, plan, s, err);
}

}  // namespace

int launch_rows(int dtype, const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err) {
  return dtype == CCL_BF16 ? pick<bf16>(g, plan, s, err) : pick<float>(g, plan, s, err);
}

}  // namespace prod
}  // namespace ccl
