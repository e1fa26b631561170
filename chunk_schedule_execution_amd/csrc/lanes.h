// Sums and extremes over the lanes of a wave, or over 16 neighbours of them.
#pragma once

#include <hip/hip_runtime.h>

namespace ccl {
namespace prod {

// Lane l's value of the lane n further on within the 16 of a row, around its end.
template <int N>
__device__ inline int turned(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xf, 0xf, true);  // every lane has a source
}
template <int N>
__device__ inline float turned(float v) {
  return __int_as_float(turned<N>(__float_as_int(v)));
}
template <int N>
__device__ inline double turned(double v) {
  return __hiloint2double(turned<N>(__double2hiint(v)), turned<N>(__double2loint(v)));
}
// In every lane f over the L lanes that are taken together (16 or 64).
template <int L, typename V, typename F>
__device__ inline V over(V v, F f) {
  v = f(v, turned<8>(v));
  v = f(v, turned<4>(v));
  v = f(v, turned<2>(v));
  v = f(v, turned<1>(v));
  if constexpr (L == 64) {
    v = f(v, V(__shfl_xor(v, 16)));
    v = f(v, V(__shfl_xor(v, 32)));
  }
  return v;
}
template <int L, typename V>
__device__ inline V over_max(V v) {  // not of NaN
  return over<L>(v, [](V a, V b) {
    if constexpr (sizeof(V) == 4) return __builtin_fmaxf(a, b);
    else return a > b ? a : b;
  });
}
template <int L, typename V>
__device__ inline V over_sum(V v) {
  return over<L>(v, [](V a, V b) { return a + b; });
}

}  // namespace prod
}  // namespace ccl
