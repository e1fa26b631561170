// fp32 instances of the tiled product kernel.
#include "product_tile.h"

namespace ccl {
namespace prod {

int launch_tile_f32(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, const ProductPlan& plan,
                    hipStream_t s, std::string* err) {
  return plan.kind == kTile128 ? launch_tile<float, 128, 128, 2, 2>(a_by_k, b_by_k, mode, g, plan.splits, s, err)
                               : launch_tile<float, 64, 64, 2, 2>(a_by_k, b_by_k, mode, g, plan.splits, s, err);
}

}  // namespace prod
}  // namespace ccl
