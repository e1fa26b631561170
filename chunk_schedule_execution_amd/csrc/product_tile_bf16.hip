// bf16 instances of the tiled product kernel.
#include "product_tile.h"

namespace ccl {
namespace prod {

int launch_tile_bf16(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, const ProductPlan& plan,
                     hipStream_t s, std::string* err) {
  switch (plan.kind) {
    case kTile256: return launch_tile<bf16, 256, 256, 2, 4>(a_by_k, b_by_k, mode, g, plan.splits, s, err);
    case kTile128: return launch_tile<bf16, 128, 128, 2, 2>(a_by_k, b_by_k, mode, g, plan.splits, s, err);
    default: return launch_tile<bf16, 64, 64, 2, 2>(a_by_k, b_by_k, mode, g, plan.splits, s, err);
  }
}

}  // namespace prod
}  // namespace ccl
