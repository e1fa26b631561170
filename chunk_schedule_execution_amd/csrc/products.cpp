// C ABI entry points of the products and the row exchange beside the collectives:
// argument checks, workspace layout and the order of the launches.
#include "products.h"

#include <algorithm>
#include <string>

#include "ccl_internal.h"

using namespace ccl;

namespace {

void require(bool ok, const char* what) {
  if (!ok) fail(CCL_ERR_INVALID_ARGUMENT, what);
}

constexpr int64_t kMaxFeatures = int64_t(1) << 20, kMaxLd = int64_t(1) << 22;

int elem_size(int dtype) {
  if (dtype == CCL_F32) return 4;
  if (dtype == CCL_BF16) return 2;
  fail(CCL_ERR_UNSUPPORTED, "products take fp32 and bf16");
}

int64_t stride_of(int64_t ld, int64_t width, const char* name) {
  if (ld == 0) return width;
  if (ld < width || ld > kMaxLd) fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": a row stride below the row's length or above 2^22");
  return ld;
}

// A descriptor with its strides filled in.
ccl_linear_desc checked(const ccl_linear_desc* d, bool grouped) {
  require(d != nullptr, "null descriptor");
  ccl_linear_desc r = *d;
  elem_size(r.dtype);
  if (r.activation < CCL_ACT_NONE || r.activation > CCL_ACT_SILU) fail(CCL_ERR_UNSUPPORTED, "unknown activation");
  require(r.rows >= 0 && r.rows <= 0x7fffffff, "rows: 0 .. 2^31 - 1");
  require(r.in_features >= 1 && r.in_features <= kMaxFeatures, "in_features: 1 .. 2^20");
  require(r.out_features >= 1 && r.out_features <= kMaxFeatures, "out_features: 1 .. 2^20");
  if (grouped) require(r.experts >= 1 && r.experts <= 4096, "experts: 1 .. 4096");
  else require(r.experts == 0 || r.experts == 1, "experts belong to the grouped calls");
  require((r.flags & ~CCL_LINEAR_UNALIGNED) == 0, "unknown flags");
  r.ld_x = stride_of(r.ld_x, r.in_features, "ld_x");
  r.ld_w = stride_of(r.ld_w, r.in_features, "ld_w");
  r.ld_out = stride_of(r.ld_out, r.out_features, "ld_out");
  r.ld_residual = stride_of(r.ld_residual, r.out_features, "ld_residual");
  r.ld_preact = stride_of(r.ld_preact, r.out_features, "ld_preact");
  r.ld_dx = stride_of(r.ld_dx, r.in_features, "ld_dx");
  r.ld_dw = stride_of(r.ld_dw, r.in_features, "ld_dw");
  if (!grouped) r.experts = 1;
  return r;
}

void aligned(const ccl_linear_desc& d, const void* p, const char* name) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (a % elem_size(d.dtype)) fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": not aligned to its elements");
  if (!(d.flags & CCL_LINEAR_UNALIGNED) && a % 16)
    fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": not 16-byte aligned; set CCL_LINEAR_UNALIGNED");
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// The products of a call, without pointers where only sizes are asked for.
ProductArgs forward_args(const ccl_linear_desc& d) {
  ProductArgs g;
  g.lda = d.ld_x;
  g.ldb = d.ld_w;
  g.ldc = d.ld_out;
  g.m = d.rows;
  g.n = d.out_features;
  g.k = d.in_features;
  g.groups = d.experts;
  g.b_stride = d.out_features * d.ld_w;
  g.bias_stride = d.out_features;
  g.ldr = d.ld_residual;
  g.ldp = d.ld_preact;
  g.act = d.activation;
  return g;
}
// dx = dz w: the summed dimension is out_features, along w's rows.
ProductArgs dx_args(const ccl_linear_desc& d, int64_t ld_dz) {
  ProductArgs g;
  g.lda = ld_dz;
  g.ldb = d.ld_w;
  g.ldc = d.ld_dx;
  g.m = d.rows;
  g.n = d.in_features;
  g.k = d.out_features;
  g.groups = d.experts;
  g.b_stride = d.out_features * d.ld_w;
  return g;
}
// dw = dz^T x: the summed dimension is the rows.
ProductArgs dw_args(const ccl_linear_desc& d, int64_t ld_dz) {
  ProductArgs g;
  g.lda = ld_dz;
  g.ldb = d.ld_x;
  g.ldc = d.ld_dw;
  g.m = d.out_features;
  g.n = d.in_features;
  g.k = d.rows;
  g.groups = d.experts;
  g.c_stride = d.out_features * d.ld_dw;
  return g;
}
OperandGrid grid_of(const ccl_linear_desc& d) { return d.flags & CCL_LINEAR_UNALIGNED ? kOffGrid : kByStrides; }

// Workspace of a backward call: dz, the partial sums of the bias gradient, and what the
// two products need, one after the other.
struct BackwardPlan {
  bool own_dz = false;  // dz is written: there is an activation, or dout lies off the 16-byte grid
  int64_t ld_dz = 0, at_partial = 0, at_product = 0, total = 0;
  ProductPlan dx, dw;
};
BackwardPlan backward_plan(const ccl_linear_desc& d, bool grouped) {
  BackwardPlan s;
  const int size = elem_size(d.dtype);
  const int64_t padded = align16(d.out_features * size) / size;
  s.own_dz = d.activation != CCL_ACT_NONE || grid_of(d) == kOffGrid || d.ld_out * size % 16 || padded != d.out_features;
  s.ld_dz = s.own_dz ? padded : d.ld_out;
  s.at_partial = s.own_dz ? align16(d.rows * padded * size) : 0;
  s.at_product = s.at_partial + align16(slope_tiles(d.rows, d.out_features, grouped ? d.experts : 0) * d.out_features * 4);
  const OperandGrid dz = s.own_dz ? kPadded : kByStrides;
  s.dx = plan_product(d.dtype, false, true, grouped ? kRaggedM : kPlain, dx_args(d, s.ld_dz), dz, grid_of(d));
  s.dw = plan_product(d.dtype, true, true, grouped ? kRaggedK : kPlain, dw_args(d, s.ld_dz), dz, grid_of(d));
  s.total = s.at_product + std::max(s.dx.bytes, s.dw.bytes);
  return s;
}
ProductPlan forward_plan(const ccl_linear_desc& d, bool grouped) {
  return plan_product(d.dtype, false, false, grouped ? kRaggedM : kPlain, forward_args(d), grid_of(d), grid_of(d));
}

int64_t workspace_bytes_of(const ccl_linear_desc& d, bool grouped, bool backward) {
  return backward ? backward_plan(d, grouped).total : forward_plan(d, grouped).bytes;
}

ccl_product_info info_of(const ProductPlan& p) {
  const int edge = p.kind == kTile64 ? 64 : p.kind == kTile128 ? 128 : 256;
  return {p.kind == kRows16 ? 16 : edge, p.kind == kRows16 ? 16 * p.columns : edge, p.splits, int(p.copy_a) + int(p.copy_b)};
}

void check_workspace(const void* ws, size_t have, int64_t need) {
  if (need == 0) return;
  if (!ws || int64_t(have) < need)
    fail(CCL_ERR_INVALID_ARGUMENT, "workspace: " + std::to_string(need) + " bytes needed, " + std::to_string(have) + " given");
  require(reinterpret_cast<uintptr_t>(ws) % 16 == 0, "workspace: not 16-byte aligned");
}

void launched(int rc, const std::string& err) {
  if (rc) fail(rc, err);
}

int forward(const ccl_linear_desc* desc, bool grouped, const int32_t* offsets, const void* x, const void* w,
            const void* bias, const void* residual, void* out, void* preact, void* ws, size_t ws_bytes, void* stream) {
  const ccl_linear_desc d = checked(desc, grouped);
  if (d.rows == 0) return CCL_OK;
  require(x && w && out, "null x, w or out");
  require(!grouped || offsets, "null offsets");
  require(reinterpret_cast<uintptr_t>(offsets) % 4 == 0, "offsets: not aligned to its elements");
  aligned(d, x, "x");
  aligned(d, w, "w");
  aligned(d, bias, "bias");
  aligned(d, residual, "residual");
  aligned(d, out, "out");
  aligned(d, preact, "preact");
  const ProductPlan plan = forward_plan(d, grouped);
  check_workspace(ws, ws_bytes, plan.bytes);
  ProductArgs g = forward_args(d);
  g.a = x;
  g.b = w;
  g.c = out;
  g.offsets = offsets;
  g.bias = bias;
  g.residual = residual;
  g.preact = preact;
  std::string err;
  launched(launch_product(d.dtype, false, false, grouped ? kRaggedM : kPlain, g, plan, ws, stream, &err), err);
  return CCL_OK;
}

int backward(const ccl_linear_desc* desc, bool grouped, const int32_t* offsets, const void* dout, const void* x,
             const void* w, const void* preact, void* dx, void* dw, void* dbias, void* ws, size_t ws_bytes,
             void* stream) {
  const ccl_linear_desc d = checked(desc, grouped);
  require(!grouped || offsets, "null offsets");
  require(reinterpret_cast<uintptr_t>(offsets) % 4 == 0, "offsets: not aligned to its elements");
  if (d.rows > 0) {
    require(dout != nullptr, "null dout");
    require(!dx || w, "dx needs w");
    require(!dw || x, "dw needs x");
    require(d.activation == CCL_ACT_NONE || preact, "the activation's gradient needs preact");
  }
  aligned(d, dout, "dout");
  aligned(d, x, "x");
  aligned(d, w, "w");
  aligned(d, preact, "preact");
  aligned(d, dx, "dx");
  aligned(d, dw, "dw");
  aligned(d, dbias, "dbias");
  const BackwardPlan plan = backward_plan(d, grouped);
  check_workspace(ws, ws_bytes, plan.total);
  unsigned char* const space = static_cast<unsigned char*>(ws);
  std::string err;
  SlopeArgs sl;
  sl.dout = dout;
  sl.preact = preact;
  sl.ldo = d.ld_out;
  sl.ldp = d.ld_preact;
  sl.rows = d.rows;
  sl.n = d.out_features;
  sl.offsets = offsets;
  sl.groups = d.experts;
  sl.act = d.activation;
  sl.dbias = dbias;
  sl.partial = reinterpret_cast<float*>(space + plan.at_partial);
  if (plan.own_dz && (dx || dw)) {
    sl.dz = space;
    sl.ldz = plan.ld_dz;
  }
  launched(launch_slope(d.dtype, sl, stream, &err), err);
  const void* dz = plan.own_dz ? space : dout;
  if (dx && d.rows > 0) {
    ProductArgs g = dx_args(d, plan.ld_dz);
    g.a = dz;
    g.b = w;
    g.c = dx;
    g.offsets = offsets;
    launched(launch_product(d.dtype, false, true, grouped ? kRaggedM : kPlain, g, plan.dx, space + plan.at_product, stream, &err),
             err);
  }
  if (dw) {
    ProductArgs g = dw_args(d, plan.ld_dz);
    g.a = dz;
    g.b = x;
    g.c = dw;
    g.offsets = offsets;
    launched(launch_product(d.dtype, true, true, grouped ? kRaggedK : kPlain, g, plan.dw, space + plan.at_product, stream, &err),
             err);
  }
  return CCL_OK;
}

// Number of slots.
int64_t exchange_checked(int dtype, int64_t tokens, int choices, int64_t width) {
  elem_size(dtype);
  require(tokens >= 0 && choices >= 1 && choices <= 1024, "tokens >= 0 and choices in 1 .. 1024 wanted");
  require(tokens <= 0x7fffffff / choices, "tokens * choices: below 2^31");
  require(width >= 1 && width <= kMaxFeatures, "width: 1 .. 2^20");
  return tokens * choices;
}
void elements(int size, const void* p, const char* name) {
  require(p != nullptr, name);
  require(reinterpret_cast<uintptr_t>(p) % size == 0, name);
}

}  // namespace

extern "C" {

int64_t ccl_linear_workspace(const ccl_linear_desc* desc, int grouped, int backward) {
  int64_t bytes = 0;
  const int rc = api_guarded([&] {
    bytes = workspace_bytes_of(checked(desc, grouped != 0), grouped != 0, backward != 0);
    return CCL_OK;
  });
  return rc ? rc : bytes;
}

int ccl_linear_info(const ccl_linear_desc* desc, int grouped, int backward, ccl_product_info* info) {
  return api_guarded([&] {
    const ccl_linear_desc d = checked(desc, grouped != 0);
    require(info != nullptr, "null info");
    if (backward) {
      const BackwardPlan p = backward_plan(d, grouped != 0);
      info[0] = info_of(p.dx);
      info[1] = info_of(p.dw);
    } else {
      info[0] = info_of(forward_plan(d, grouped != 0));
    }
    return CCL_OK;
  });
}

int ccl_linear(const ccl_linear_desc* desc, const void* x, const void* w, const void* bias, const void* residual,
               void* out, void* preact, void* workspace, size_t workspace_bytes, void* stream) {
  return api_guarded([&] {
    return forward(desc, false, nullptr, x, w, bias, residual, out, preact, workspace, workspace_bytes, stream);
  });
}

int ccl_linear_backward(const ccl_linear_desc* desc, const void* dout, const void* x, const void* w,
                        const void* preact, void* dx, void* dw, void* dbias, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return api_guarded([&] {
    return backward(desc, false, nullptr, dout, x, w, preact, dx, dw, dbias, workspace, workspace_bytes, stream);
  });
}

int ccl_grouped_linear(const ccl_linear_desc* desc, const int32_t* offsets, const void* x, const void* w,
                       const void* bias, void* out, void* preact, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return api_guarded([&] {
    return forward(desc, true, offsets, x, w, bias, nullptr, out, preact, workspace, workspace_bytes, stream);
  });
}

int ccl_grouped_linear_backward(const ccl_linear_desc* desc, const int32_t* offsets, const void* dout, const void* x,
                                const void* w, const void* preact, void* dx, void* dw, void* dbias, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return api_guarded([&] {
    return backward(desc, true, offsets, dout, x, w, preact, dx, dw, dbias, workspace, workspace_bytes, stream);
  });
}

int64_t ccl_expert_route_workspace(int64_t tokens, int choices, int experts) {
  int64_t bytes = 0;
  const int rc = api_guarded([&] {
    const int64_t count = exchange_checked(CCL_F32, tokens, choices, 1);
    require(experts >= 1 && experts <= 1024, "experts: 1 .. 1024");
    bytes = route_workspace(count, experts);
    return CCL_OK;
  });
  return rc ? rc : bytes;
}

int ccl_expert_route(const int32_t* ids, int64_t tokens, int choices, int experts, int32_t* offsets,
                     int32_t* positions, int32_t* slots, void* workspace, size_t workspace_bytes, void* stream) {
  return api_guarded([&] {
    const int64_t count = exchange_checked(CCL_F32, tokens, choices, 1);
    require(experts >= 1 && experts <= 1024, "experts: 1 .. 1024");
    elements(4, offsets, "offsets: null or misaligned");
    if (count) {
      elements(4, ids, "ids: null or misaligned");
      elements(4, positions, "positions: null or misaligned");
      elements(4, slots, "slots: null or misaligned");
    }
    check_workspace(workspace, workspace_bytes, route_workspace(count, experts));
    std::string err;
    launched(launch_route(ids, count, experts, offsets, positions, slots, workspace, stream, &err), err);
    return CCL_OK;
  });
}

int ccl_expert_dispatch(int dtype, const void* x, int64_t ld_x, const int32_t* slots, int64_t tokens, int choices,
                        int64_t width, void* rows, int64_t ld_rows, void* stream) {
  return api_guarded([&] {
    const int64_t count = exchange_checked(dtype, tokens, choices, width);
    ld_x = stride_of(ld_x, width, "ld_x");
    ld_rows = stride_of(ld_rows, width, "ld_rows");
    if (count == 0) return CCL_OK;
    elements(elem_size(dtype), x, "x: null or misaligned");
    elements(4, slots, "slots: null or misaligned");
    elements(elem_size(dtype), rows, "rows: null or misaligned");
    std::string err;
    launched(launch_dispatch(dtype, x, ld_x, slots, tokens, choices, width, rows, ld_rows, stream, &err), err);
    return CCL_OK;
  });
}

int ccl_expert_combine(int dtype, const void* h, int64_t ld_h, const int32_t* positions, const float* gates,
                       int64_t tokens, int choices, int64_t width, void* out, int64_t ld_out, void* stream) {
  return api_guarded([&] {
    const int64_t count = exchange_checked(dtype, tokens, choices, width);
    ld_h = stride_of(ld_h, width, "ld_h");
    ld_out = stride_of(ld_out, width, "ld_out");
    if (count == 0) return CCL_OK;
    elements(elem_size(dtype), h, "h: null or misaligned");
    elements(4, positions, "positions: null or misaligned");
    if (gates) elements(4, gates, "gates: misaligned");
    elements(elem_size(dtype), out, "out: null or misaligned");
    std::string err;
    launched(launch_combine(dtype, h, ld_h, positions, gates, tokens, choices, width, out, ld_out, stream, &err), err);
    return CCL_OK;
  });
}

int ccl_expert_combine_backward(int dtype, const void* dout, int64_t ld_dout, const void* h, int64_t ld_h,
                                const int32_t* positions, const int32_t* slots, const float* gates, int64_t tokens,
                                int choices, int64_t width, void* dh, int64_t ld_dh, float* dgates, void* stream) {
  return api_guarded([&] {
    const int64_t count = exchange_checked(dtype, tokens, choices, width);
    ld_dout = stride_of(ld_dout, width, "ld_dout");
    ld_h = stride_of(ld_h, width, "ld_h");
    ld_dh = stride_of(ld_dh, width, "ld_dh");
    if (count == 0 || (!dh && !dgates)) return CCL_OK;
    elements(elem_size(dtype), dout, "dout: null or misaligned");
    elements(4, positions, "positions: null or misaligned");
    elements(4, slots, "slots: null or misaligned");
    if (gates) elements(4, gates, "gates: misaligned");
    if (dh) elements(elem_size(dtype), dh, "dh: misaligned");
    if (dgates) {
      elements(4, dgates, "dgates: misaligned");
      elements(elem_size(dtype), h, "h: null or misaligned");
    }
    std::string err;
    launched(launch_combine_backward(dtype, dout, ld_dout, h, ld_h, positions, slots, gates, tokens, choices, width,
                                     dh, ld_dh, dgates, stream, &err),
             err);
    return CCL_OK;
  });
}

}  // extern "C"
