// Kernels of the layer's operators around the products: the arguments that the entry
// points (layers.cpp) hand to the launches.
#pragma once

#include <cstdint>
#include <string>

#include "products.h"

namespace ccl {

// The choice of experts and its gradient.
struct SelectArgs {
  const void* logits = nullptr;
  const float* bias = nullptr;
  int32_t* ids = nullptr;        // read by the gradient
  float* gates = nullptr;
  const float* dgates = nullptr;
  void* dlogits = nullptr;
  int64_t tokens = 0, ld = 0, ldd = 0;
  int experts = 0, choices = 0, groups = 1, kept = 1, best = 1, score = 0;
  bool renorm = false;
  float scale = 1.0f;
  // of the groups: experts in each, 2^20 / that + 1, and the lanes of 16 that share one as a
  // power of 2
  int per = 0, magic = 0, parts_log2 = 0;
};
int launch_select(int dtype, const SelectArgs& args, void* stream, std::string* err);
int launch_select_backward(int dtype, const SelectArgs& args, void* stream, std::string* err);

// Layer norm and its gradients.
struct NormArgs {
  const void* x = nullptr;        // the backward pass: what was normalised
  const void* residual = nullptr;
  const void* weight = nullptr;
  const void* bias = nullptr;
  void* out = nullptr;
  void* total = nullptr;
  float* mean = nullptr;          // read by the gradients
  float* rstd = nullptr;
  const void* dout = nullptr;
  const void* dtotal = nullptr;
  void* dx = nullptr;
  void* dweight = nullptr;
  void* dbias = nullptr;
  float* partial = nullptr;       // norm_partials() rows of dweight's and of dbias's sums, each `width` values
  int64_t rows = 0, width = 0;
  int64_t ld_x = 0, ld_residual = 0, ld_out = 0, ld_total = 0, ld_dtotal = 0, ld_dx = 0;  // ld_out: dout's too
  float eps = 0.0f;
};
int launch_norm(int dtype, const NormArgs& args, void* stream, std::string* err);
// Rows of partial sums that the gradients leave, at most.
int64_t norm_partials(int64_t rows);
int launch_norm_backward(int dtype, const NormArgs& args, void* stream, std::string* err);

// The cross entropy of z = x w^T. A row's target is column target - first of z; it is none
// where that lies outside the columns. Rows whose target, as an unsigned number, is `end` or
// above are left out: the vocabulary's end, or 2^31 where only negative ones are.
struct LossArgs {
  const int32_t* targets = nullptr;
  int first = 0;
  unsigned end = 0;
  const float* lse = nullptr;    // the gradient's: of the whole vocabulary
  const float* dloss = nullptr;
  float* sums = nullptr;         // (maximum, sum of exp(z - maximum)) by [block of columns][row]
  float* picked = nullptr;       // the targets' logits
};
// Columns that one pair of LossArgs::sums covers.
int loss_block(ProductKind kind);
// A product's sums by row; nothing else of it is kept.
int launch_loss_sums(int dtype, const ProductArgs& g, const LossArgs& loss, ProductKind kind, void* stream,
                     std::string* err);
// dz = dloss (exp(z - lse) - 1 at the target), 0 for rows left out and in the columns from
// g.n up to `padded`.
int launch_loss_slope(int dtype, const ProductArgs& g, const LossArgs& loss, int64_t padded, ProductKind kind,
                      void* stream, std::string* err);
// The same two from the fp32 sums of `splits` splits of a product in g.partial.
struct LossRowsArgs {
  const float* partial = nullptr;
  int64_t rows = 0, n = 0, ldz = 0;  // ldz: dz's
  int splits = 1;
  float* loss_out = nullptr;         // NULL: not wanted
  float* lse_out = nullptr;
  void* dz = nullptr;
};
int launch_loss_rows(const LossRowsArgs& args, const LossArgs& loss, void* stream, std::string* err);
int launch_loss_rows_slope(int dtype, const LossRowsArgs& args, const LossArgs& loss, void* stream, std::string* err);
// A b_by_k product whose sums are added to what is in g.partial.
int launch_product_onto(int dtype, const ProductArgs& g, const ProductPlan& plan, void* stream, std::string* err);

// Joins parts of the rows' sums: `blocks` rows of pairs in `pairs`, or (pairs NULL) `blocks`
// rows of lse_parts and picked_parts, which are one shard's each. n: the columns that targets
// may lie in, for `picked` (NULL: not wanted). loss: NULL where it is not wanted.
struct LossJoinArgs {
  const float* pairs = nullptr;
  const float* lse_parts = nullptr;
  const float* picked_parts = nullptr;
  const int32_t* targets = nullptr;
  int64_t blocks = 0, rows = 0;
  int first = 0, n = 0;
  unsigned end = 0;              // as in LossArgs
  float* loss = nullptr;
  float* lse = nullptr;
  float* picked = nullptr;       // in: the targets' logits where there is one
};
int launch_loss_join(const LossJoinArgs& args, void* stream, std::string* err);

}  // namespace ccl
