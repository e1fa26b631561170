// Device helpers shared by the product and exchange kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/ccl.h"
#include "products.h"

namespace ccl {
namespace prod {

typedef __bf16 bf16;
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The status of the launches before it.
inline int hip_status(const char* what, std::string* err) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return CCL_OK;
  *err = std::string(what) + ": " + hipGetErrorString(e);
  return CCL_ERR_HIP;
}

__device__ inline float widen(bf16 v) { return float(v); }
__device__ inline float widen(float v) { return v; }
template <typename T>
__device__ inline T narrow(float v) {
  return T(v);  // nearest-even
}

// One step of the summed dimension of a 16 x 16 tile: 32 values in bf16, 16 in fp32.
__device__ inline f32x4 multiply(bf16x8 x, bf16x8 y, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc, 0, 0, 0);
}
__device__ inline f32x4 multiply(f32x4 x, f32x4 y, f32x4 acc) {
#pragma unroll
  for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[q], y[q], acc, 0, 0, 0);
  return acc;
}

// exp(-v) and 1 / v by the hardware's own instructions (one fp32 step each).
__device__ inline float exp_of_minus(float v) { return __builtin_amdgcn_exp2f(v * -1.44269504088896341f); }
__device__ inline float reciprocal(float v) { return __builtin_amdgcn_rcpf(v); }

// erfc(s / sqrt 2) / 2, the normal distribution's tail beyond s >= 0, as e t Q(t) with
// e = exp(-s^2 / 2), t = 1 / (1 + 0.305 s) and a polynomial Q of degree 7, fitted to
// erfcx(s / sqrt 2) / (2 t) on 0 <= s <= 14 for the least relative error (0.94e-7; the scale
// 0.305 is where that is smallest). In fp32 the tail is off by 0.4e-6 of itself below s = 2,
// by 2e-6 at 6, where exp's argument is what rounds. Relative, since gelu is -s times the
// tail at z = -s: an approximation good to 1e-7 of 1 is 5e-5 off there at 3 and 1 % at 7.
__device__ inline float normal_tail(float s, float e) {
  const float t = reciprocal(fmaf(0.305f, s, 1.0f));
  float q = 0.0366991609f;
  q = fmaf(q, t, -0.152988181f);
  q = fmaf(q, t, 0.185716659f);
  q = fmaf(q, t, -0.0379766189f);
  q = fmaf(q, t, 0.121021569f);
  q = fmaf(q, t, 0.103420898f);
  q = fmaf(q, t, 0.122466817f);
  q = fmaf(q, t, 0.121639736f);
  return e * t * q;
}

// (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u)), so gelu_tanh and silu are both z / (1 + exp(-v)).
__device__ inline float gelu_tanh_arg(float z) { return 1.59576912160573071f * (z + 0.044715f * z * z * z); }

__device__ inline float act_value(float z, int act) {
  switch (act) {
    case CCL_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case CCL_ACT_GELU: {
      // z times the distribution function is max(z, 0) - |z| tail(|z|); the bound on |z|, where
      // the tail is 0, keeps an infinite z
      const float tail = normal_tail(fabsf(z), exp_of_minus(0.5f * z * z));
      return fmaxf(z, 0.0f) - fminf(fabsf(z), 64.0f) * tail;
    }
    case CCL_ACT_GELU_TANH: return z * reciprocal(1.0f + exp_of_minus(gelu_tanh_arg(z)));
    case CCL_ACT_SILU: return z * reciprocal(1.0f + exp_of_minus(z));
  }
  return z;
}

__device__ inline float act_slope(float z, int act) {
  switch (act) {
    case CCL_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case CCL_ACT_GELU: {
      const float e = exp_of_minus(0.5f * z * z), tail = normal_tail(fabsf(z), e);
      return (z < 0.0f ? tail : 1.0f - tail) + z * e * 0.39894228040143268f;
    }
    case CCL_ACT_GELU_TANH:
    case CCL_ACT_SILU: {
      // p = 1 / (1 + exp(-v)): p + z p (1 - p) v'; 1 - p without cancellation
      const float v = act == CCL_ACT_SILU ? z : gelu_tanh_arg(z);
      const float dv = act == CCL_ACT_SILU ? 1.0f : 1.59576912160573071f * (1.0f + 0.134145f * z * z);
      const float e = exp_of_minus(v), p = reciprocal(1.0f + e);
      return p + z * p * (v > 0.0f ? e * p : 1.0f - p) * dv;
    }
  }
  return 1.0f;
}

// A value that all lanes share, for the compiler to keep in scalar registers.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <typename P>
__device__ inline P* uniform(P* p) {
  const unsigned long long v = reinterpret_cast<unsigned long long>(p);
  const unsigned long long lo = unsigned(uniform(int(v))), hi = unsigned(uniform(int(v >> 32)));
  return reinterpret_cast<P*>(hi << 32 | lo);
}

// The same value, from which nothing is computed ahead of here: keeps what a loop needs at
// its end out of the registers of its middle.
__device__ inline int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// One tile of rows of a group.
struct RowTile {
  int group;    // `groups` for the rows behind the last group, -1 past the last tile
  int index;    // tile number over all groups
  int64_t row;  // first row
  int64_t end;  // end of the group
};

// The groups' bounds and tiles when every group is cut into tiles of `height` rows of its
// own, 64 groups at a time on a whole wave: lane l reads offset base + l, a running maximum
// makes the bounds monotone (offset 0 counts as 0, values are clamped to [0, rows]), a prefix
// sum counts tiles. Group `groups` is the rows behind the last group. With at most 64 groups
// that is one round of loads and 12 shuffles.
struct GroupScan {
  int lo = 0, hi = 0;        // this lane's group
  int tiles = 0, upto = 0;   // its tiles; those up to and with its own
  int tiles_before = 0, top = 0;  // of the rounds before

  __device__ inline void round(const int32_t* offsets, int groups, int64_t rows, int height, int base, int lane) {
    const int e = base + lane;
    hi = e < groups ? max(0, min(offsets[e + 1], int(rows))) : int(rows);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(hi, d);
      if (lane >= d) hi = max(hi, v);
    }
    hi = max(hi, top);
    lo = __shfl_up(hi, 1);
    if (lane == 0) lo = top;
    tiles = e <= groups ? int((int64_t(hi) - lo + height - 1) / height) : 0;
    upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    upto += tiles_before;
  }
  // carries on to the next round
  __device__ inline void carry() {
    tiles_before = __builtin_amdgcn_readlane(upto, 63);
    top = __builtin_amdgcn_readlane(hi, 63);
  }
};

// The tile-th tile of `height` rows of the groups and the rows behind them.
__device__ inline RowTile find_tile(const int32_t* offsets, int groups, int64_t rows, int height, int tile) {
  const int lane = here(threadIdx.x & 63);
  if (offsets == nullptr) {
    const int64_t row = int64_t(tile) * height;
    return {row < rows ? 0 : -1, tile, row, rows};
  }
  GroupScan s;
  for (int base = 0; base <= groups; base += 64, s.carry()) {
    s.round(offsets, groups, rows, height, base, lane);
    const unsigned long long hit = __ballot(tile < s.upto);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      const int first = __builtin_amdgcn_readlane(s.upto - s.tiles, l);
      const int64_t row = int64_t(__builtin_amdgcn_readlane(s.lo, l)) + int64_t(tile - first) * height;
      return {base + l, tile, row, int64_t(__builtin_amdgcn_readlane(s.hi, l))};
    }
  }
  return {-1, tile, 0, 0};
}

// Bounds of one group, with the same reading of the offsets.
__device__ inline void group_bounds(const int32_t* offsets, int64_t rows, int group, int64_t& lo, int64_t& hi) {
  if (offsets == nullptr) {
    lo = 0;
    hi = rows;
    return;
  }
  const int lane = here(threadIdx.x & 63);
  int top = 0;  // running maximum of the offsets up to the group's begin
  for (int e = 1 + lane; e <= group; e += 64) top = max(top, min(offsets[e], int(rows)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, __shfl_xor(top, d));
  top = uniform(top);
  lo = top;
  hi = max(top, min(offsets[group + 1], int(rows)));
}

// How many tiles find_tile knows.
__device__ inline int count_tiles(const int32_t* offsets, int groups, int64_t rows, int height) {
  if (offsets == nullptr) return int((rows + height - 1) / height);
  GroupScan s;
  for (int base = 0; base <= groups; base += 64, s.carry()) s.round(offsets, groups, rows, height, base, threadIdx.x & 63);
  return uniform(s.tiles_before);
}

// The numbers of a group's tiles of `height` rows, [first, last).
__device__ inline void group_tiles(const int32_t* offsets, int groups, int64_t rows, int height, int group,
                                   int64_t& first, int64_t& last) {
  first = 0;
  if (offsets == nullptr) {
    last = (rows + height - 1) / height;
    return;
  }
  GroupScan s;
  int base = 0;
  for (;; base += 64, s.carry()) {
    s.round(offsets, groups, rows, height, base, threadIdx.x & 63);
    if (group < base + 64) break;
  }
  last = __builtin_amdgcn_readlane(s.upto, group - base);
  first = last - __builtin_amdgcn_readlane(s.tiles, group - base);
}

// ---- results -----------------------------------------------------------------------------
// 8 neighbouring values of a row; `vec`: the row lies on the 16-byte grid; `n`: how many of
// them exist. Stream: around the caches, for what is read once.
template <bool Stream = false, typename T>
__device__ inline void load8(const T* p, bool vec, int n, float* v) {
  if (vec && n >= 8) {
    constexpr int V = 16 / int(sizeof(T));
    typedef T pack __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      pack x;
      if constexpr (Stream) x = __builtin_nontemporal_load(reinterpret_cast<const pack*>(p) + h);
      else x = reinterpret_cast<const pack*>(p)[h];
#pragma unroll
      for (int q = 0; q < V; ++q) v[h * V + q] = widen(x[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = q < n ? widen(p[q]) : 0.0f;
  }
}

// Stream: around the caches, for what is not read again soon. 33 MB of results per round of
// tiles otherwise push the operands out of the L2s: 16384 rows over 32 experts of 2048 x
// 4096 take 351 us, and 390 with plain stores.
template <bool Stream = false, typename T>
__device__ inline void store8(T* p, bool vec, int n, const float* v) {
  if (vec && n >= 8) {
    constexpr int V = 16 / int(sizeof(T));
    typedef T pack __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      pack x;
#pragma unroll
      for (int q = 0; q < V; ++q) x[q] = narrow<T>(v[h * V + q]);
      if constexpr (Stream) __builtin_nontemporal_store(x, reinterpret_cast<pack*>(p) + h);
      else reinterpret_cast<pack*>(p)[h] = x;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = narrow<T>(v[q]);
  }
}
// The activation of 8 values: the branch is taken once for them.
__device__ inline void act8(float* v, int act) {
#define CCL_ACT8(A)                                            \
  case A:                                                      \
    _Pragma("unroll") for (int q = 0; q < 8; ++q) v[q] = act_value(v[q], A); \
    break;
  switch (act) {
    CCL_ACT8(CCL_ACT_RELU)
    CCL_ACT8(CCL_ACT_GELU)
    CCL_ACT8(CCL_ACT_GELU_TANH)
    CCL_ACT8(CCL_ACT_SILU)
    default: break;
  }
#undef CCL_ACT8
}
// v times the slopes at z.
__device__ inline void slope8(float* v, const float* z, int act) {
#define CCL_SLOPE8(A)                                                            \
  case A:                                                                        \
    _Pragma("unroll") for (int q = 0; q < 8; ++q) v[q] *= act_slope(z[q], A);    \
    break;
  switch (act) {
    CCL_SLOPE8(CCL_ACT_RELU)
    CCL_SLOPE8(CCL_ACT_GELU)
    CCL_SLOPE8(CCL_ACT_GELU_TANH)
    CCL_SLOPE8(CCL_ACT_SILU)
    default: break;
  }
#undef CCL_SLOPE8
}

template <typename T>
__device__ inline bool on_vectors(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(T) % 16 == 0;
}

// Bias, activation, residual and stores of results: 8 columns (c .. c + n - 1, n <= 8) of
// rows that lie a fixed step apart.
template <typename T>
struct Finish {
  const T* residual;
  T* preact;
  T* out;
  int64_t step_r, step_p, step_c;  // elements from one of its rows to the next
  float bias[8];
  int n, act;
  bool vec_c, vec_r, vec_p, with_bias;

  // nothing: rows of no group, whose results are zeros (z has to be 0)
  __device__ inline Finish(const ProductArgs& g, T* to, int64_t row, int step, int64_t c, int count, int group,
                           bool nothing)
      : residual(static_cast<const T*>(g.residual)), preact(static_cast<T*>(g.preact)), out(to + row * g.ldc + c),
        step_r(step * g.ldr), step_p(step * g.ldp), step_c(step * g.ldc), n(count),
        act(nothing ? CCL_ACT_NONE : g.act) {
    vec_c = on_vectors<T>(to, g.ldc);
    vec_r = on_vectors<T>(residual, g.ldr);
    vec_p = on_vectors<T>(preact, g.ldp);
    if (residual) residual += row * g.ldr + c;
    if (preact) preact += row * g.ldp + c;
    with_bias = g.bias != nullptr && !nothing;
    if (with_bias && n > 0) load8(static_cast<const T*>(g.bias) + group * g.bias_stride + c, false, n, bias);
  }
  __device__ inline void row(float* z) const {
    if (with_bias) {
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] += bias[q];
    }
    if (preact) store8<true>(preact, vec_p, n, z);
    act8(z, act);
    if (residual) {
      float w[8];
      load8(residual, vec_r, n, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] += w[q];
    }
    store8<true>(out, vec_c, n, z);
  }
  __device__ inline void next() {
    out += step_c;
    if (preact) preact += step_p;
    if (residual) residual += step_r;
  }
};

// The same for a single result.
template <typename T>
__device__ inline void finish_one(const ProductArgs& g, float z, int64_t row, int64_t c, int group, bool nothing) {
  float v = 0.0f;
  if (!nothing) {
    if (g.bias) z += widen(static_cast<const T*>(g.bias)[group * g.bias_stride + c]);
    v = act_value(z, g.act);
  }
  if (g.preact) static_cast<T*>(g.preact)[row * g.ldp + c] = narrow<T>(nothing ? 0.0f : z);
  if (g.residual) v += widen(static_cast<const T*>(g.residual)[row * g.ldr + c]);
  static_cast<T*>(g.c)[row * g.ldc + c] = narrow<T>(v);
}

// Where split `s`'s fp32 sum of a result goes; rows of whole 16-byte vectors.
__device__ inline float* partial_at(const ProductArgs& g, int s, int64_t row, int64_t c) {
  return g.partial + (int64_t(s) * g.m + row) * partial_ld(g.n) + c;
}

}  // namespace prod
}  // namespace ccl
