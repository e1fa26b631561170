// Kernels of the products and the row exchange beside the collectives: the arguments
// that the entry points (products.cpp) hand to the launches.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

namespace ccl {

// How the rows of a product are cut into groups by the device array `offsets`.
enum ProductMode : int {
  kPlain = 0,    // one product
  kRaggedM = 1,  // the groups cut the rows of A and C; B, bias: one per group
  kRaggedK = 2,  // the groups cut the summed dimension; C: one per group
};

// C[i, j] = epilogue(sum over k of A(i, k) B(j, k)). A is stored by rows i (A(i, k) at
// a[i lda + k]) or, with a_by_k, by rows k (a[k lda + i]); B likewise.
struct ProductArgs {
  const void* a = nullptr;
  const void* b = nullptr;
  void* c = nullptr;
  int64_t lda = 0, ldb = 0, ldc = 0;
  int64_t b_stride = 0, c_stride = 0, bias_stride = 0;  // elements between groups
  int64_t m = 0, n = 0, k = 0;                          // kRaggedM: m, kRaggedK: k counts all groups' rows
  const int32_t* offsets = nullptr;
  int groups = 1;
  const void* bias = nullptr;
  const void* residual = nullptr;
  void* preact = nullptr;
  int64_t ldr = 0, ldp = 0;
  int act = 0;
  float* partial = nullptr;  // set: the splits' fp32 sums go here, [split][m][partial_ld(n)], and nothing else happens
};
#ifdef __HIPCC__
__host__ __device__
#endif
inline int64_t partial_ld(int64_t n) { return (n + 3) / 4 * 4; }

// How a product is run, from its sizes alone.
enum ProductKind : int { kRows16, kTile64, kTile128, kTile256 };
struct ProductPlan {
  ProductKind kind = kTile128;
  int columns = 1;                   // kRows16: 16-column fragments per workgroup
  int splits = 1;                    // of the summed dimension
  bool vec = true;                   // kRows16: both operands lie on the 16-byte grid
  bool copy_a = false, copy_b = false;  // tiles: operands that are first copied onto that grid
  int64_t ld_a = 0, ld_b = 0;        // of the copies
  int64_t at_b = 0, at_partial = 0, bytes = 0;  // workspace layout: the copy of a, of b, the splits' sums
};
// Where an operand's stored rows lie: on the 16-byte grid if strides and lengths are whole
// vectors; off it, its base pointer being unaligned; or on it with zeros up to the vector.
enum OperandGrid : int { kByStrides, kOffGrid, kPadded };
ProductPlan plan_product(int dtype, bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& args,
                         OperandGrid a_grid, OperandGrid b_grid);
// The few-row kernel's grid, in its first dimension.
int64_t rows16_workgroups(ProductMode mode, const ProductArgs& args, int columns);
int launch_product(int dtype, bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& args,
                   const ProductPlan& plan, void* workspace, void* stream, std::string* err);

// dz = dout act'(preact) (skipped when dz is NULL; zeros behind a row up to ldz) and its
// column sums by group (skipped when dbias is NULL). partial: fp32, slope_tiles() x n.
struct SlopeArgs {
  const void* dout = nullptr;
  const void* preact = nullptr;
  void* dz = nullptr;
  void* dbias = nullptr;
  float* partial = nullptr;
  int64_t ldo = 0, ldp = 0, ldz = 0;
  int64_t rows = 0, n = 0;
  const int32_t* offsets = nullptr;  // NULL: one group
  int groups = 1;
  int act = 0;
};
int64_t slope_tiles(int64_t rows, int64_t n, int groups);  // groups: 0 without offsets
int launch_slope(int dtype, const SlopeArgs& args, void* stream, std::string* err);

int64_t route_workspace(int64_t slots, int experts);
int launch_route(const int32_t* ids, int64_t slots, int experts, int32_t* offsets, int32_t* positions, int32_t* slot_of,
                 void* workspace, void* stream, std::string* err);
int launch_dispatch(int dtype, const void* x, int64_t ldx, const int32_t* slots, int64_t tokens, int choices,
                    int64_t width, void* rows, int64_t ldr, void* stream, std::string* err);
int launch_combine(int dtype, const void* h, int64_t ldh, const int32_t* positions, const float* gates, int64_t tokens,
                   int choices, int64_t width, void* out, int64_t ldo, void* stream, std::string* err);
int launch_combine_backward(int dtype, const void* dout, int64_t ldo, const void* h, int64_t ldh,
                            const int32_t* positions, const int32_t* slots, const float* gates, int64_t tokens,
                            int choices, int64_t width, void* dh, int64_t lddh, float* dgates, void* stream,
                            std::string* err);

}  // namespace ccl
