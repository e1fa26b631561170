// fp32 instances of the cross entropy's products.
#include "loss_tile.h"

namespace ccl {
namespace prod {

int loss_sums_f32(const ProductArgs& g, const LossArgs& loss, ProductKind kind, hipStream_t s, std::string* err) {
  return launch_end<float, false>(g, RowSums{loss}, kind, 1, s, err);
}
int loss_slope_f32(const ProductArgs& g, const LossArgs& loss, int64_t padded, ProductKind kind, hipStream_t s,
                    std::string* err) {
  return launch_end<float, false>(g, LossSlope{loss, padded}, kind, 1, s, err);
}
int product_onto_f32(const ProductArgs& g, const ProductPlan& plan, hipStream_t s, std::string* err) {
  return launch_end<float, true>(g, AddedSums(), plan.kind, plan.splits, s, err);
}

}  // namespace prod
}  // namespace ccl
