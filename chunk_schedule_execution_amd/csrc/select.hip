// The choice of experts for gfx950: scores, groups, the highest `choices` of a token's
// experts and their gates, and the gradient of the gates.
//
// L lanes take a token (16 up to 256 experts, 64 above), lane l its experts l, L + l, ... in
// registers. A choice is a maximum over the lane's values, one over the lanes, and the
// lowest index that has it; the chosen one leaves. No token waits for another.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lanes.h"
#include "layers.h"
#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

constexpr int kThreads = 256, kMaxChoices = 64, kMaxGroups = 64;

constexpr float kClosed = -INFINITY;

// A score times a factor that the chosen experts of a token share: exp(-m) for softmax (m
// their highest logit, or the row's), exp(-m) with m = min(0, highest) for sigmoid, so that a
// ratio of scores is right also where the scores themselves are too small for fp32. m = 0
// gives the sigmoid itself.
__device__ inline float scaled_score(float x, float m, bool soft) {
  return soft ? expf(x - m) : 1.0f / (expf(m) + expf(m - x));
}
__device__ inline float shared_top(float highest, bool soft) {
  return highest == -INFINITY ? 0.0f : soft ? highest : fminf(0.0f, highest);
}

// The row's maximum, 0 where there is none to subtract.
template <int L, int NE>
__device__ inline float row_top(const float (&x)[NE]) {
  float m = kClosed;
#pragma unroll
  for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
  m = over_max<L>(m);
  return m == kClosed ? 0.0f : m;
}

template <typename T, int L, int NE>
__device__ inline void load_row(const SelectArgs& a, int64_t t, int lane, float (&x)[NE]) {
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * L + lane;
    x[i] = t < a.tokens && e < a.experts ? widen(row[e]) : kClosed;
  }
}

// ---- the choice ----------------------------------------------------------------------------
// Takes the keys of experts outside the kept groups away. A lane takes a group, in LDS.
template <typename Key, int L, int NE>
struct Groups {
  Key value[kThreads / L][L * NE];
  Key best[kThreads / L][kMaxGroups];
  bool kept[kThreads / L][kMaxGroups];

  __device__ inline void keep(const SelectArgs& a, int slot, int lane, const Key (&v)[NE], Key (&key)[NE]) {
    const int per = a.experts / a.groups;
#pragma unroll
    for (int i = 0; i < NE; ++i) value[slot][i * L + lane] = v[i];
    __builtin_amdgcn_wave_barrier();
    for (int g = lane; g < a.groups; g += L) {
      Key first = kClosed, second = kClosed;
      for (int q = 0; q < per; ++q) {
        const Key w = value[slot][g * per + q];
        second = w > first ? first : w > second ? w : second;
        first = w > first ? w : first;
      }
      best[slot][g] = a.best == 2 && second > Key(kClosed) ? first + second : first;
    }
    __builtin_amdgcn_wave_barrier();
    for (int g = lane; g < a.groups; g += L) {
      const Key mine = best[slot][g];
      int before = 0;
      for (int h = 0; h < a.groups; ++h) before += best[slot][h] > mine || (best[slot][h] == mine && h < g);
      kept[slot][g] = before < a.kept;
    }
    __builtin_amdgcn_wave_barrier();
    // e / per without a division: e and per are at most 2^10
    const unsigned magic = (1u << 20) / per + 1;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const unsigned e = i * L + lane;
      if (e < unsigned(a.experts) && !kept[slot][e * magic >> 20]) key[i] = kClosed;
    }
  }
};
struct NoGroups {};

// Key double: scores and bias are added and compared in 64 bits, since fp32 would take the
// wrong one of two experts a rounding apart. Key float: the logits themselves are compared
// (no bias: the scores rise with them).
template <typename T, typename Key, bool Grouped, int L, int NE>
__global__ __launch_bounds__(kThreads) void select_kernel(SelectArgs a) {
  constexpr bool Scored = std::is_same<Key, double>::value;
  __shared__ int chosen[kThreads / L][kMaxChoices];
  __shared__ typename std::conditional<Grouped, Groups<Key, L, NE>, NoGroups>::type groups;
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / L) + slot;
  const Key closed = Key(kClosed);
  float x[NE];
  load_row<T, L>(a, t, lane, x);
  const float top = row_top<L>(x);

  Key key[NE];
  if constexpr (Scored) {
    double v[NE], total = 0.0;
    const bool soft = a.score == CCL_SCORE_SOFTMAX;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      v[i] = soft ? exp(double(x[i]) - double(top)) : 1.0 / (1.0 + exp(-double(x[i])));
      total += v[i];
    }
    if (soft) {
      total = over_sum<L>(total);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] /= total;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * L + lane;
      if (a.bias) v[i] += e < a.experts ? double(a.bias[e]) : 0.0;
      if (!(v[i] == v[i])) v[i] = INFINITY;
      if (x[i] == kClosed || (a.bias && e < a.experts && a.bias[e] == kClosed)) v[i] = closed;
      key[i] = a.bias || v[i] == closed ? v[i] : x[i] == x[i] ? double(x[i]) : INFINITY;
    }
    if constexpr (Grouped) groups.keep(a, slot, lane, v, key);
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = x[i] == x[i] ? x[i] : INFINITY;
    if constexpr (Grouped) {
      Key v[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = key[i];
      groups.keep(a, slot, lane, v, key);
    }
  }

  for (int c = 0; c < a.choices; ++c) {
    Key m = closed;
    int at = a.experts;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i * L + lane;
      }
    const Key best = over_max<L>(m);
    const int first = over<L>(m == best ? at : a.experts, [](int p, int q) { return min(p, q); });
    if (lane == 0) chosen[slot][c] = first < a.experts ? first : -1;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (first == i * L + lane) key[i] = closed;
  }
  __builtin_amdgcn_wave_barrier();

  // gates: of the chosen logits, read again (they are in the caches)
  constexpr int Each = kMaxChoices / L;
  const bool soft = a.score == CCL_SCORE_SOFTMAX;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  int id[Each];
  float q[Each], m = kClosed, total = 1.0f;
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    const int c = j * L + lane;
    id[j] = c < a.choices && t < a.tokens ? chosen[slot][c] : -1;
    q[j] = id[j] >= 0 ? widen(row[id[j]]) : kClosed;
    m = fmaxf(m, q[j]);
  }
  if (a.renorm) m = shared_top(over_max<L>(m), soft);
  else m = soft ? top : 0.0f;
#pragma unroll
  for (int j = 0; j < Each; ++j) q[j] = id[j] >= 0 ? scaled_score(q[j], m, soft) : 0.0f;
  if (a.renorm) {
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < Each; ++j) total += q[j];
    total = over_sum<L>(total);
  } else if (soft) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) total += expf(x[i] - m);
    total = over_sum<L>(total);
  }
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    const int c = j * L + lane;
    if (c >= a.choices || t >= a.tokens) continue;
    a.ids[t * a.choices + c] = id[j];
    a.gates[t * a.choices + c] = id[j] < 0 ? 0.0f : a.scale * (q[j] / total);
  }
}

// ---- the gradient --------------------------------------------------------------------------
// dx_e = p_e (d_e - sum p d) for softmax, d_e p_e (1 - p_e) for sigmoid, d the scores'
// gradients, zero but at the chosen experts; where the gates were divided by their sum the
// others have no part in them. The gradients of choices with the same id are added in their
// order.
template <typename T, int L, int NE>
__global__ __launch_bounds__(kThreads) void select_backward_kernel(SelectArgs a) {
  constexpr int Each = kMaxChoices / L;
  __shared__ int chosen[kThreads / L][kMaxChoices];
  __shared__ float grad[kThreads / L][kMaxChoices];
  __shared__ float spread[kThreads / L][L * NE];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / L) + slot;
  const bool soft = a.score == CCL_SCORE_SOFTMAX, whole = soft && !a.renorm;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float x[NE], m = 0.0f, total = 1.0f;
  if (whole) {  // p of every expert
    load_row<T, L>(a, t, lane, x);
    m = row_top<L>(x);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      x[i] = expf(x[i] - m);
      total += x[i];
    }
    total = over_sum<L>(total);
    if (total == 0.0f) total = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) spread[slot][i * L + lane] = 0.0f;

  int id[Each];
  float d[Each], p[Each], xs[Each];
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    const int c = j * L + lane;
    const bool there = c < a.choices && t < a.tokens;
    id[j] = there ? a.ids[t * a.choices + c] : -1;
    if (id[j] < 0 || id[j] >= a.experts) id[j] = -1;
    d[j] = id[j] >= 0 ? a.scale * a.dgates[t * a.choices + c] : 0.0f;
    xs[j] = id[j] >= 0 ? widen(row[id[j]]) : kClosed;
  }
  if (a.renorm) {
    m = kClosed;
#pragma unroll
    for (int j = 0; j < Each; ++j) m = fmaxf(m, xs[j]);
    m = shared_top(over_max<L>(m), soft);
  }
#pragma unroll
  for (int j = 0; j < Each; ++j) p[j] = id[j] < 0 ? 0.0f : scaled_score(xs[j], m, soft) / total;
  if (a.renorm) {
    float sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int j = 0; j < Each; ++j) sum += p[j];
    sum = over_sum<L>(sum);
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < Each; ++j) mean += d[j] * (p[j] * inverse);
    mean = over_sum<L>(mean);
#pragma unroll
    for (int j = 0; j < Each; ++j) d[j] = (d[j] - mean) * inverse * p[j];
  } else {
#pragma unroll
    for (int j = 0; j < Each; ++j) d[j] *= p[j];
  }
  float flow = 0.0f;  // sum p d
  if (whole) {
#pragma unroll
    for (int j = 0; j < Each; ++j) flow += d[j];
    flow = over_sum<L>(flow);
  }
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    const int c = j * L + lane;
    if (!soft && id[j] >= 0) d[j] *= scaled_score(-xs[j], 0.0f, false);
    chosen[slot][c] = id[j];
    grad[slot][c] = d[j];
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    if (id[j] < 0) continue;
    float sum = 0.0f;
    bool first = true;
    for (int c = 0; c < a.choices; ++c)
      if (chosen[slot][c] == id[j]) {
        if (c < j * L + lane) first = false;
        sum += grad[slot][c];
      }
    if (first) spread[slot][id[j]] = sum;
  }
  __builtin_amdgcn_wave_barrier();
  if (t >= a.tokens) return;
  T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * L + lane;
    if (e < a.experts) out[e] = narrow<T>(spread[slot][e] - (whole ? x[i] / total * flow : 0.0f));
  }
}

template <int L>
dim3 token_grid(int64_t tokens) {
  const int64_t n = (tokens + kThreads / L - 1) / (kThreads / L), x = std::min<int64_t>(n, 1 << 20);
  return dim3(unsigned(x), unsigned((n + x - 1) / x));
}

// Calls f with the lanes per token and the values per lane that hold the experts.
template <typename F>
void by_experts(int experts, F f) {
  using std::integral_constant;
  auto with = [&](auto lanes, auto each) { f(lanes, each); };
  if (experts <= 32) with(integral_constant<int, 16>(), integral_constant<int, 2>());
  else if (experts <= 64) with(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (experts <= 128) with(integral_constant<int, 16>(), integral_constant<int, 8>());
  else if (experts <= 256) with(integral_constant<int, 16>(), integral_constant<int, 16>());
  else if (experts <= 512) with(integral_constant<int, 64>(), integral_constant<int, 8>());
  else with(integral_constant<int, 64>(), integral_constant<int, 16>());
}

template <typename T>
int select_t(const SelectArgs& a, hipStream_t s, std::string* err) {
  const bool grouped = a.kept < a.groups, scored = a.bias || (grouped && a.best == 2);
  by_experts(a.experts, [&](auto lanes, auto each) {
    constexpr int L = decltype(lanes)::value, NE = decltype(each)::value;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_grid<L>(a.tokens), dim3(kThreads), 0, s, a); };
    if (scored && grouped) go(select_kernel<T, double, true, L, NE>);
    else if (scored) go(select_kernel<T, double, false, L, NE>);
    else if (grouped) go(select_kernel<T, float, true, L, NE>);
    else go(select_kernel<T, float, false, L, NE>);
  });
  return hip_status("expert selection launch", err);
}

template <typename T>
int select_backward_t(const SelectArgs& a, hipStream_t s, std::string* err) {
  by_experts(a.experts, [&](auto lanes, auto each) {
    constexpr int L = decltype(lanes)::value, NE = decltype(each)::value;
    hipLaunchKernelGGL((select_backward_kernel<T, L, NE>), token_grid<L>(a.tokens), dim3(kThreads), 0, s, a);
  });
  return hip_status("expert selection gradient launch", err);
}

}  // namespace
}  // namespace prod

int launch_select(int dtype, const SelectArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::select_t<prod::bf16>(args, s, err) : prod::select_t<float>(args, s, err);
}

int launch_select_backward(int dtype, const SelectArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::select_backward_t<prod::bf16>(args, s, err)
                           : prod::select_backward_t<float>(args, s, err);
}

}  // namespace ccl
