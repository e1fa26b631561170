// C ABI entry points of the layer's operators around the products: the choice of experts,
// layer norm and the vocabulary's cross entropy. Argument checks, workspace layout and the
// order of the launches.
#include "layers.h"

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "args.h"

using namespace ccl;

namespace {

// A pointer that may be NULL.
void optional_elements(int size, const void* p, const char* name) {
  if (p) elements(size, p, name);
}

// ---- the choice of experts ---------------------------------------------------------------
SelectArgs select_args(const ccl_select_desc* d) {
  require(d != nullptr, "null descriptor");
  elem_size(d->dtype);
  if (d->score != CCL_SCORE_SOFTMAX && d->score != CCL_SCORE_SIGMOID) fail(CCL_ERR_UNSUPPORTED, "unknown score");
  require(d->tokens >= 0 && d->tokens <= 0x7fffffff, "tokens: 0 .. 2^31 - 1");
  require(d->experts >= 1 && d->experts <= 1024, "experts: 1 .. 1024");
  require(d->choices >= 1 && d->choices <= 64 && d->choices <= d->experts, "choices: 1 .. 64, at most the experts");
  require(d->groups >= 1 && d->groups <= 64 && d->experts % d->groups == 0,
          "groups: 1 .. 64, of equal numbers of experts");
  require(d->kept_groups >= 1 && d->kept_groups <= d->groups, "kept_groups: 1 .. groups");
  require(d->group_best == 1 || d->group_best == 2, "group_best: 1 or 2");
  require(d->renormalise == 0 || d->renormalise == 1, "renormalise: 0 or 1");
  require(std::isfinite(d->scale), "scale: a finite number wanted");
  SelectArgs a;
  a.tokens = d->tokens;
  a.experts = d->experts;
  a.choices = d->choices;
  a.groups = d->groups;
  a.kept = d->kept_groups;
  a.best = d->group_best;
  a.per = d->experts / d->groups;
  a.magic = (1 << 20) / a.per + 1;
  while ((a.groups << (a.parts_log2 + 1)) <= 16) ++a.parts_log2;
  a.score = d->score;
  a.renorm = d->renormalise != 0;
  a.scale = d->scale;
  a.ld = stride_of(d->ld_logits, d->experts, "ld_logits");
  a.ldd = stride_of(d->ld_dlogits, d->experts, "ld_dlogits");
  return a;
}

// ---- layer norm ----------------------------------------------------------------------------
NormArgs norm_args(const ccl_norm_desc* d) {
  require(d != nullptr, "null descriptor");
  elem_size(d->dtype);
  require(d->rows >= 0 && d->rows <= 0x7fffffff, "rows: 0 .. 2^31 - 1");
  require(d->width >= 1 && d->width <= kMaxFeatures, "width: 1 .. 2^20");
  require(d->eps >= 0.0f && std::isfinite(d->eps), "eps: a finite number from 0 on wanted");
  NormArgs a;
  a.rows = d->rows;
  a.width = d->width;
  a.eps = d->eps;
  a.ld_x = stride_of(d->ld_x, d->width, "ld_x");
  a.ld_residual = stride_of(d->ld_residual, d->width, "ld_residual");
  a.ld_out = stride_of(d->ld_out, d->width, "ld_out");
  a.ld_total = stride_of(d->ld_total, d->width, "ld_total");
  a.ld_dtotal = stride_of(d->ld_dtotal, d->width, "ld_dtotal");
  a.ld_dx = stride_of(d->ld_dx, d->width, "ld_dx");
  return a;
}

// Whether two matrices of `rows` rows of `width` bytes, their rows ld_p and ld_q bytes apart,
// have a byte in common. Rows side by side in one buffer do not.
bool share_memory(const void* p, int64_t ld_p, const void* q, int64_t ld_q, int64_t rows, int64_t width) {
  const int64_t from = int64_t(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p));
  if (from >= (rows - 1) * ld_p + width || -from >= (rows - 1) * ld_q + width) return false;
  auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
  if (ld_p == ld_q) {  // rows of p this many behind q's, or one more
    const int64_t behind = floor_div(from, ld_p), off = from - behind * ld_p;
    return (std::abs(behind) < rows && off < width) || (std::abs(behind + 1) < rows && ld_p - off < width);
  }
  for (int64_t row = 0; row < rows; ++row) {
    // the first of p's rows that ends behind this one of q's begins
    const int64_t at = from + row * ld_q, first = std::max<int64_t>(0, floor_div(at - width, ld_p) + 1);
    if (first < rows && first * ld_p < at + width) return true;
  }
  return false;
}
// The norm's outputs may take its inputs' places whole, and otherwise no memory of theirs or of
// each other: rows are read by one workgroup while others write.
void in_place_or_apart(const NormArgs& a, int size) {
  auto share = [&](const void* p, int64_t ld_p, const void* q, int64_t ld_q) {
    return p && q && share_memory(p, ld_p * size, q, ld_q * size, a.rows, a.width * size);
  };
  auto taken = [&](const void* p, int64_t ld_p, const void* q, int64_t ld_q) {
    return !(p == q && (ld_p == ld_q || a.rows == 1)) && share(p, ld_p, q, ld_q);
  };
  require(!share(a.out, a.ld_out, a.total, a.ld_total), "out and total: the same memory");
  require(!taken(a.out, a.ld_out, a.x, a.ld_x), "out: memory of x, but not x itself");
  require(!taken(a.out, a.ld_out, a.residual, a.ld_residual), "out: memory of residual, but not residual itself");
  require(!taken(a.total, a.ld_total, a.x, a.ld_x), "total: memory of x, but not x itself");
  require(!taken(a.total, a.ld_total, a.residual, a.ld_residual), "total: memory of residual, but not residual itself");
}
int64_t norm_workspace(const NormArgs& a) { return align16(norm_partials(a.rows) * 2 * a.width * 4); }

// ---- cross entropy ---------------------------------------------------------------------------
ccl_cross_entropy_desc checked(const ccl_cross_entropy_desc* d) {
  require(d != nullptr, "null descriptor");
  ccl_cross_entropy_desc r = *d;
  elem_size(r.dtype);
  require(r.rows >= 0 && r.rows <= 0x7fffffff, "rows: 0 .. 2^31 - 1");
  require(r.in_features >= 1 && r.in_features <= kMaxFeatures, "in_features: 1 .. 2^20");
  require(r.vocabulary >= 1 && r.vocabulary <= kMaxFeatures, "vocabulary: 1 .. 2^20");
  require(r.first >= -1 && r.first <= 0x7fffffff - r.vocabulary, "first: -1, or a shard's first row below 2^31");
  require((r.flags & ~CCL_LINEAR_UNALIGNED) == 0, "unknown flags");
  r.ld_x = stride_of(r.ld_x, r.in_features, "ld_x");
  r.ld_w = stride_of(r.ld_w, r.in_features, "ld_w");
  r.ld_dx = stride_of(r.ld_dx, r.in_features, "ld_dx");
  r.ld_dw = stride_of(r.ld_dw, r.in_features, "ld_dw");
  return r;
}
void aligned(const ccl_cross_entropy_desc& d, const void* p, const char* name) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (a % elem_size(d.dtype)) fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": not aligned to its elements");
  if (!(d.flags & CCL_LINEAR_UNALIGNED) && a % 16)
    fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": not 16-byte aligned; set CCL_LINEAR_UNALIGNED");
}

// Columns of the vocabulary whose gradients of logits are kept at a time: 512 MiB of them, at
// least 8192, in pieces of nearly equal size. Adding a piece's dx up moves 8 bytes per value of
// dx and split, where the products of 8192 columns take 49152 operations per value: at most 5 %
// of their time unsplit. Both gradients per 1000 columns, bf16: 8192 x 4096 over 32768, one piece,
// 155.8 us, over 131072, four, 156.1; 4096 x 4096 over 65536, one, 78.9, over 65792, two, 80.4;
// 65536 x 4096 over 8192, one, 1258, over 32768, four of that size, 1270 (dx alone 832 and 868).
int64_t piece_columns(const ccl_cross_entropy_desc& d) {
  const int64_t most = std::max<int64_t>(8192, (int64_t(512) << 20) / std::max<int64_t>(1, d.rows * elem_size(d.dtype)));
  const int64_t pieces = (d.vocabulary + most - 1) / most;
  return ((d.vocabulary + pieces - 1) / pieces + 255) / 256 * 256;
}

// Where the parts of a call's workspace lie and how its products are run.
struct LossPlan {
  bool copy_x = false, copy_w = false;  // onto the 16-byte grid, or x for its zeroed rows
  int64_t ld_x = 0, ld_w = 0;
  int64_t at_w = 0, at_sums = 0, at_picked = 0;              // forward
  int64_t at_dz = 0, at_dx = 0, at_product = 0, ld_dz = 0;   // backward
  int64_t piece = 0;
  bool onto = false;  // dx is summed up over the pieces
  ProductPlan logits, dx;
  int64_t total = 0;
};

ProductArgs logits_args(const ccl_cross_entropy_desc& d, const LossPlan& p, int64_t columns) {
  ProductArgs g;
  g.lda = p.ld_x;
  g.ldb = p.ld_w;
  g.m = d.rows;
  g.n = columns;
  g.k = d.in_features;
  return g;
}
// dx = dz w: the summed dimension is the vocabulary.
ProductArgs dx_args(const ccl_cross_entropy_desc& d, const LossPlan& p, int64_t columns) {
  ProductArgs g;
  g.lda = p.ld_dz;
  g.ldb = p.ld_w;
  g.ldc = d.ld_dx;
  g.m = d.rows;
  g.n = d.in_features;
  g.k = columns;
  return g;
}
// dw = dz^T x: the summed dimension is the rows.
ProductArgs dw_args(const ccl_cross_entropy_desc& d, const LossPlan& p, int64_t columns) {
  ProductArgs g;
  g.lda = p.ld_dz;
  g.ldb = p.ld_x;
  g.ldc = d.ld_dw;
  g.m = columns;
  g.n = d.in_features;
  g.k = d.rows;
  return g;
}
ProductPlan dw_plan(const ccl_cross_entropy_desc& d, const LossPlan& p, int64_t columns) {
  return plan_product(d.dtype, true, true, kPlain, dw_args(d, p, columns), kPadded, kPadded);
}

// Of a piece of the backward pass, whose operands lie on the grid.
ProductPlan logits_plan(const ccl_cross_entropy_desc& d, const LossPlan& p, int64_t columns) {
  return plan_product(d.dtype, false, false, kPlain, logits_args(d, p, columns), kPadded, kPadded);
}

// Whether a product's logits go through the workspace instead of staying in registers: where
// it has few rows and a kernel without tiles (3 x 1190 x 11136 fp32: 50 us in tiles, whose
// operands have to be copied first), and where its tiles are fewer than the compute units and
// its sums are split, or most units would idle (113 x 1984 x 4562 fp32: 41 us unsplit). Both
// come for logits that are small beside the operands. With tiles for all units the split no
// longer pays (64 x 4096 x 32768 bf16: 57 us unsplit, 65 in 2 splits).
bool through_memory(const ProductPlan& p, const ProductArgs& g) {
  return p.kind == kRows16 || (p.splits > 1 && ((g.m + 63) / 64) * ((g.n + 63) / 64) < 256);
}
int64_t logits_bytes(const ProductPlan& p, const ProductArgs& g) {
  return p.at_partial + p.splits * g.m * partial_ld(g.n) * 4;
}

// What a call gives: the loss, or gradients.
struct LossGives {
  bool backward = false, dx = false, dw = false;
};

LossPlan loss_plan(const ccl_cross_entropy_desc& d, const LossGives& gives) {
  LossPlan p;
  const bool backward = gives.backward;
  const int64_t size = elem_size(d.dtype), v = 16 / size;
  auto up = [&](int64_t n) { return (n + v - 1) / v * v; };
  const bool off = d.flags & CCL_LINEAR_UNALIGNED;
  if (!backward) {
    p.ld_x = d.ld_x;
    p.ld_w = d.ld_w;
    const OperandGrid grid = off ? kOffGrid : kByStrides;
    const ProductArgs g = logits_args(d, p, d.vocabulary);
    p.logits = plan_product(d.dtype, false, false, kPlain, g, grid, grid);
    if (through_memory(p.logits, g)) {
      p.total = align16(logits_bytes(p.logits, g));
      return p;
    }
  }
  // dw's x is always a copy, with zeros in the rows that are left out: their dz is 0, but 0 times
  // what a row of padding may hold, NaN or infinite, would reach dw. (dz itself is set to 0 in
  // such rows, whatever their logits.)
  p.copy_x = gives.dw || off || d.ld_x % v || d.in_features % v;
  p.copy_w = off || d.ld_w % v || d.in_features % v;
  p.ld_x = p.copy_x ? up(d.in_features) : d.ld_x;
  p.ld_w = p.copy_w ? up(d.in_features) : d.ld_w;
  p.at_w = p.copy_x ? align16(d.rows * p.ld_x * size) : 0;
  const int64_t copied = p.at_w + (p.copy_w ? align16(d.vocabulary * p.ld_w * size) : 0);
  if (!backward) {
    const int64_t block = loss_block(unsplit_tile(d.dtype, logits_args(d, p, d.vocabulary)));
    p.at_sums = copied;
    p.at_picked = p.at_sums + align16((d.vocabulary + block - 1) / block * d.rows * 8);
    p.total = p.at_picked + align16(d.rows * 4);
    return p;
  }
  p.piece = piece_columns(d);
  p.ld_dz = up(std::min(p.piece, d.vocabulary));
  p.onto = gives.dx && p.piece < d.vocabulary;
  p.at_dz = copied;
  p.dx = plan_product(d.dtype, false, true, kPlain, dx_args(d, p, std::min(p.piece, d.vocabulary)), kPadded, kPadded);
  p.at_dx = p.at_dz + align16(d.rows * p.ld_dz * size);
  p.at_product = p.at_dx + (p.onto ? p.dx.splits * d.rows * partial_ld(d.in_features) * 4 : 0);
  int64_t most = p.onto || !gives.dx ? 0 : p.dx.bytes;
  for (int64_t lo = 0; lo < d.vocabulary; lo += p.piece) {
    const int64_t n = std::min(p.piece, d.vocabulary - lo);
    if (gives.dw) most = std::max(most, dw_plan(d, p, n).bytes);
    const ProductPlan logits = logits_plan(d, p, n);
    if (through_memory(logits, logits_args(d, p, n))) most = std::max(most, logits_bytes(logits, logits_args(d, p, n)));
  }
  p.total = p.at_product + most;
  return p;
}

// x and w, or their copies on the 16-byte grid, x's without the rows that l (or NULL) leaves out.
void operands(const ccl_cross_entropy_desc& d, const LossPlan& p, const LossArgs* l, unsigned char* space, void* stream,
              const void** x, const void** w) {
  Regrid copy[2];
  int copies = 0;
  if (p.copy_x) {
    copy[copies++] = {*x, space, d.ld_x, d.rows, d.in_features, p.ld_x, l ? l->targets : nullptr, l ? l->end : 0};
    *x = space;
  }
  if (p.copy_w) {
    copy[copies++] = {*w, space + p.at_w, d.ld_w, d.vocabulary, d.in_features, p.ld_w};
    *w = space + p.at_w;
  }
  std::string err;
  if (copies) launched(launch_regrid(d.dtype, copy[0], copy[1], stream, &err), err);
}

LossArgs loss_args(const ccl_cross_entropy_desc& d, const int32_t* targets) {
  LossArgs l;
  l.targets = targets;
  l.first = int(std::max<int64_t>(0, d.first));
  l.end = d.first < 0 ? unsigned(d.vocabulary) : 1u << 31;
  return l;
}

int loss_forward(const ccl_cross_entropy_desc* desc, const void* x, const void* w, const int32_t* targets, float* loss,
                 float* lse, float* picked, void* ws, size_t ws_bytes, void* stream) {
  const ccl_cross_entropy_desc d = checked(desc);
  if (d.rows == 0) return CCL_OK;
  require(x && w, "null x or w");
  aligned(d, x, "x");
  aligned(d, w, "w");
  elements(4, targets, "targets: null or misaligned");
  elements(4, lse, "lse: null or misaligned");
  optional_elements(4, loss, "loss: misaligned");
  optional_elements(4, picked, "picked: misaligned");
  require(!loss || d.first < 0, "loss: of a whole vocabulary only; join the shards' sums first");
  const LossPlan p = loss_plan(d, {});
  check_workspace(ws, ws_bytes, p.total);
  unsigned char* const space = static_cast<unsigned char*>(ws);
  std::string err;
  ProductArgs g = logits_args(d, p, d.vocabulary);
  LossArgs l = loss_args(d, targets);
  if (through_memory(p.logits, g)) {
    g.a = x;
    g.b = w;
    g.partial = reinterpret_cast<float*>(space + p.logits.at_partial);
    launched(launch_product_sums(d.dtype, false, false, kPlain, g, p.logits, space, stream, &err), err);
    LossRowsArgs r;
    r.partial = g.partial;
    r.rows = d.rows;
    r.n = d.vocabulary;
    r.splits = p.logits.splits;
    r.loss_out = loss;
    r.lse_out = lse;
    l.picked = picked;
    launched(launch_loss_rows(r, l, stream, &err), err);
    return CCL_OK;
  }
  operands(d, p, nullptr, space, stream, &x, &w);
  const ProductKind kind = unsplit_tile(d.dtype, g);
  g.a = x;
  g.b = w;
  l.sums = reinterpret_cast<float*>(space + p.at_sums);
  l.picked = picked ? picked : reinterpret_cast<float*>(space + p.at_picked);
  launched(launch_loss_sums(d.dtype, g, l, kind, stream, &err), err);
  LossJoinArgs j;
  j.pairs = l.sums;
  j.targets = targets;
  j.blocks = (d.vocabulary + loss_block(kind) - 1) / loss_block(kind);
  j.rows = d.rows;
  j.first = l.first;
  j.n = int(d.vocabulary);
  j.end = l.end;
  j.loss = loss;
  j.lse = lse;
  j.picked = l.picked;
  launched(launch_loss_join(j, stream, &err), err);
  return CCL_OK;
}

int loss_backward(const ccl_cross_entropy_desc* desc, const float* dloss, const void* x, const void* w,
                  const int32_t* targets, const float* lse, void* dx, void* dw, void* ws, size_t ws_bytes,
                  void* stream) {
  const ccl_cross_entropy_desc d = checked(desc);
  if (!dx && !dw) return CCL_OK;
  if (d.rows > 0) {
    require(x && w, "null x or w");
    elements(4, dloss, "dloss: null or misaligned");
    elements(4, targets, "targets: null or misaligned");
    elements(4, lse, "lse: null or misaligned");
  }
  aligned(d, x, "x");
  aligned(d, w, "w");
  aligned(d, dx, "dx");
  aligned(d, dw, "dw");
  const LossPlan p = loss_plan(d, {true, dx != nullptr, dw != nullptr});
  check_workspace(ws, ws_bytes, p.total);
  unsigned char* const space = static_cast<unsigned char*>(ws);
  std::string err;
  LossArgs l = loss_args(d, targets);
  if (d.rows > 0) operands(d, p, dw ? &l : nullptr, space, stream, &x, &w);
  const int64_t size = elem_size(d.dtype), v = 16 / size;
  l.lse = lse;
  l.dloss = dloss;
  const int first = l.first;
  for (int64_t lo = 0; lo < d.vocabulary; lo += p.piece) {
    const int64_t n = std::min(p.piece, d.vocabulary - lo);
    const char* const wp = static_cast<const char*>(w) + (d.rows > 0 ? lo * p.ld_w * size : 0);
    if (d.rows > 0) {
      ProductArgs g = logits_args(d, p, n);
      g.a = x;
      g.b = wp;
      g.c = space + p.at_dz;
      g.ldc = p.ld_dz;
      l.first = int(first + lo);
      const ProductPlan logits = logits_plan(d, p, n);
      if (through_memory(logits, g)) {
        g.partial = reinterpret_cast<float*>(space + p.at_product + logits.at_partial);
        launched(launch_product_sums(d.dtype, false, false, kPlain, g, logits, space + p.at_product, stream, &err), err);
        LossRowsArgs r;
        r.partial = g.partial;
        r.rows = d.rows;
        r.n = n;
        r.splits = logits.splits;
        r.dz = space + p.at_dz;
        r.ldz = p.ld_dz;
        launched(launch_loss_rows_slope(d.dtype, r, l, stream, &err), err);
      } else {
        launched(launch_loss_slope(d.dtype, g, l, (n + v - 1) / v * v, unsplit_tile(d.dtype, g), stream, &err), err);
      }
    }
    if (dx && d.rows > 0) {
      ProductArgs g = dx_args(d, p, n);
      g.a = space + p.at_dz;
      g.b = wp;
      g.c = dx;
      if (!p.onto) {
        launched(launch_product(d.dtype, false, true, kPlain, g, p.dx, space + p.at_product, stream, &err), err);
      } else {
        g.partial = reinterpret_cast<float*>(space + p.at_dx);
        launched(lo == 0 ? launch_product_sums(d.dtype, false, true, kPlain, g, p.dx, nullptr, stream, &err)
                         : launch_product_onto(d.dtype, g, p.dx, stream, &err), err);
        if (lo + n == d.vocabulary) launched(launch_join(d.dtype, g, p.dx.splits, stream, &err), err);
      }
    }
    if (dw) {
      ProductArgs g = dw_args(d, p, n);
      g.a = space + p.at_dz;
      g.b = x;
      g.c = static_cast<char*>(dw) + lo * d.ld_dw * size;
      launched(launch_product(d.dtype, true, true, kPlain, g, dw_plan(d, p, n), space + p.at_product, stream, &err), err);
    }
  }
  return CCL_OK;
}

}  // namespace

extern "C" {

int ccl_expert_select(const ccl_select_desc* desc, const void* logits, const float* bias, int32_t* ids, float* gates,
                      void* stream) {
  return api_guarded([&] {
    SelectArgs a = select_args(desc);
    if (a.tokens == 0) return CCL_OK;
    elements(elem_size(desc->dtype), logits, "logits: null or misaligned");
    optional_elements(4, bias, "bias: misaligned");
    elements(4, ids, "ids: null or misaligned");
    elements(4, gates, "gates: null or misaligned");
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.gates = gates;
    std::string err;
    launched(launch_select(desc->dtype, a, stream, &err), err);
    return CCL_OK;
  });
}

int ccl_expert_select_backward(const ccl_select_desc* desc, const float* dgates, const void* logits,
                               const int32_t* ids, void* dlogits, void* stream) {
  return api_guarded([&] {
    SelectArgs a = select_args(desc);
    if (a.tokens == 0) return CCL_OK;
    elements(4, dgates, "dgates: null or misaligned");
    elements(elem_size(desc->dtype), logits, "logits: null or misaligned");
    elements(4, ids, "ids: null or misaligned");
    elements(elem_size(desc->dtype), dlogits, "dlogits: null or misaligned");
    a.dgates = dgates;
    a.logits = logits;
    a.ids = const_cast<int32_t*>(ids);
    a.dlogits = dlogits;
    std::string err;
    launched(launch_select_backward(desc->dtype, a, stream, &err), err);
    return CCL_OK;
  });
}

int ccl_layer_norm(const ccl_norm_desc* desc, const void* x, const void* residual, const void* weight,
                   const void* bias, void* out, void* total, float* mean, float* rstd, void* stream) {
  return api_guarded([&] {
    NormArgs a = norm_args(desc);
    if (a.rows == 0) return CCL_OK;
    const int size = elem_size(desc->dtype);
    elements(size, x, "x: null or misaligned");
    optional_elements(size, residual, "residual: misaligned");
    optional_elements(size, weight, "weight: misaligned");
    optional_elements(size, bias, "bias: misaligned");
    elements(size, out, "out: null or misaligned");
    optional_elements(size, total, "total: misaligned");
    require(!total || residual, "total: without a residual it is x");
    optional_elements(4, mean, "mean: misaligned");
    optional_elements(4, rstd, "rstd: misaligned");
    require(!mean == !rstd, "mean and rstd: both or neither");
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.bias = bias;
    a.out = out;
    a.total = total;
    a.mean = mean;
    a.rstd = rstd;
    in_place_or_apart(a, size);
    std::string err;
    launched(launch_norm(desc->dtype, a, stream, &err), err);
    return CCL_OK;
  });
}

int64_t ccl_layer_norm_backward_workspace(const ccl_norm_desc* desc) {
  int64_t bytes = 0;
  const int rc = api_guarded([&] {
    bytes = norm_workspace(norm_args(desc));
    return CCL_OK;
  });
  return rc ? rc : bytes;
}

int ccl_layer_norm_backward(const ccl_norm_desc* desc, const void* dout, const void* x, const float* mean,
                            const float* rstd, const void* weight, const void* dtotal, void* dx, void* dweight,
                            void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  return api_guarded([&] {
    NormArgs a = norm_args(desc);
    const int size = elem_size(desc->dtype);
    if (!dx && !dweight && !dbias) return CCL_OK;
    if (a.rows > 0) {
      elements(size, dout, "dout: null or misaligned");
      elements(size, x, "x: null or misaligned");
      elements(4, mean, "mean: null or misaligned");
      elements(4, rstd, "rstd: null or misaligned");
    }
    optional_elements(size, weight, "weight: misaligned");
    optional_elements(size, dtotal, "dtotal: misaligned");
    optional_elements(size, dx, "dx: misaligned");
    optional_elements(size, dweight, "dweight: misaligned");
    optional_elements(size, dbias, "dbias: misaligned");
    if (dweight || dbias) check_workspace(workspace, workspace_bytes, norm_workspace(a));
    a.dout = dout;
    a.x = x;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.weight = weight;
    a.dtotal = dtotal;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.partial = static_cast<float*>(workspace);
    std::string err;
    launched(launch_norm_backward(desc->dtype, a, stream, &err), err);
    return CCL_OK;
  });
}

int64_t ccl_linear_cross_entropy_workspace(const ccl_cross_entropy_desc* desc, int backward) {
  int64_t bytes = 0;
  const int rc = api_guarded([&] {
    const bool any = backward != 0;
    bytes = loss_plan(checked(desc), {any, any && backward != CCL_GRADIENT_DW, any && backward != CCL_GRADIENT_DX}).total;
    return CCL_OK;
  });
  return rc ? rc : bytes;
}

int ccl_linear_cross_entropy(const ccl_cross_entropy_desc* desc, const void* x, const void* w, const int32_t* targets,
                             float* loss, float* lse, float* picked, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return api_guarded(
      [&] { return loss_forward(desc, x, w, targets, loss, lse, picked, workspace, workspace_bytes, stream); });
}

int ccl_linear_cross_entropy_backward(const ccl_cross_entropy_desc* desc, const float* dloss, const void* x,
                                      const void* w, const int32_t* targets, const float* lse, void* dx, void* dw,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  return api_guarded(
      [&] { return loss_backward(desc, dloss, x, w, targets, lse, dx, dw, workspace, workspace_bytes, stream); });
}

int ccl_cross_entropy_join(int shards, int64_t rows, const float* lse_parts, const float* picked_parts,
                           const int32_t* targets, float* loss, float* lse, void* stream) {
  return api_guarded([&] {
    require(shards >= 1 && shards <= 65536, "shards: 1 .. 2^16");
    require(rows >= 0 && rows <= 0x7fffffff, "rows: 0 .. 2^31 - 1");
    if (rows == 0) return CCL_OK;
    elements(4, lse_parts, "lse_parts: null or misaligned");
    elements(4, picked_parts, "picked_parts: null or misaligned");
    elements(4, targets, "targets: null or misaligned");
    elements(4, loss, "loss: null or misaligned");
    elements(4, lse, "lse: null or misaligned");
    LossJoinArgs j;
    j.lse_parts = lse_parts;
    j.picked_parts = picked_parts;
    j.targets = targets;
    j.blocks = shards;
    j.rows = rows;
    j.end = 1u << 31;
    j.loss = loss;
    j.lse = lse;
    std::string err;
    launched(launch_loss_join(j, stream, &err), err);
    return CCL_OK;
  });
}

}  // extern "C"
