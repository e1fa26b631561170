// bf16 instances of the tiled product kernel and the choice among them.
#include "product_tile.h"

namespace ccl {
namespace prod {

int launch_tile_bf16(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, hipStream_t s,
                     std::string* err) {
  const int64_t tiles = ((g.m + 255) / 256) * ((g.n + 255) / 256) * (mode == kRaggedK ? g.groups : 1);
  if (tiles >= 200) return launch_tile<bf16, 256, 256, 2, 4>(a_by_k, b_by_k, mode, g, s, err);
  return launch_tile<bf16, 128, 128, 2, 2>(a_by_k, b_by_k, mode, g, s, err);
}

}  // namespace prod
}  // namespace ccl
