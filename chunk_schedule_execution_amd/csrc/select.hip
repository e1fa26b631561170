// The choice of experts for gfx950: scores, groups, the highest `choices` of a token's
// experts and their gates, and the gradient of the gates.
//
// What has to be right to the last bit is the order of p + bias in 64 bits; what would be
// slow is computing all of it there. So 16 lanes take a token, its experts in their registers,
// and find in fp32 the few experts that may be among the highest: those not below the
// choices-th highest of the lanes' maxima, less what fp32 may be off (11 of 256 for 8 choices).
// Their values are computed in 64 bits, one per lane, and each counts how many come before it.
// A softmax with a bias takes the sum that its scores share in 64 bits too, an exponential for
// every expert. 16384 x 256 fp32, sigmoids with a bias and groups: 15.7 us, 40 with all values and
// 8 maxima in turn in 64 bits; the logits alone would take 3.4. 1174 vector instructions a wave
// are half of the time (four waves a SIMD); the rest is one wave's chain of them, 10 us by itself.
// Softmax with a bias, no groups: 16 us (bf16 14), sigmoids 13, without a bias 11.
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

// exp to two steps of fp32: the argument's rounding on its way to a power of 2 is carried
// along. NaN stays; beyond +-200 the result is 0 or infinite either way.
__device__ inline float exp_exact(float x) {
  x = x < -200.0f ? -200.0f : x > 200.0f ? 200.0f : x;
  const float t = x * 1.44269504088896341f;
  const float rest = fmaf(x, 1.44269504088896341f, -t) + x * 1.92596299e-8f;
  return __builtin_amdgcn_exp2f(t) * fmaf(rest, 0.693147180559945309f, 1.0f);
}

// A score times a factor that the chosen experts of a token share: exp(-m) for softmax (m
// their highest logit, or the row's), exp(-m) with m = min(0, highest) for sigmoid, so that a
// ratio of scores is right also where the scores themselves are too small for fp32. m = 0
// gives the sigmoid itself.
__device__ inline float scaled_score(float x, float m, bool soft) {
  return soft ? exp_exact(x - m) : 1.0f / (exp_exact(m) + exp_exact(m - x));
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

// Which expert a lane's value i is: V neighbours of each 16-byte (or shorter) vector in turn,
// a quarter of the lanes further with every vector, so that the experts of a group, which are
// neighbours, fall to all lanes about equally.
template <int L, int V>
__device__ inline int expert_at(int i, int lane) {
  return V == 1 ? i * L + lane : i / V * (L * V) + ((lane + i / V * (L / 4)) & (L - 1)) * V + i % V;
}
// V > 1: row and ends lie on the grid of V values.
template <int L, int V, int NE, typename T>
__device__ inline void load_row(const T* row, int lane, int experts, float fill, float (&x)[NE]) {
  typedef T pack __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = expert_at<L, V>(i, lane);
    if constexpr (V == 1) {
      x[i] = e < experts ? widen(row[e]) : fill;
    } else {
      pack v = {};
      if (e < experts) v = *reinterpret_cast<const pack*>(row + e);
#pragma unroll
      for (int q = 0; q < V; ++q) x[i + q] = e < experts ? widen(v[q]) : fill;
    }
  }
}

// What an expert is ranked by, in 64 bits. total: of the row's exp(x - top), softmax only.
__device__ inline double score_of(float x, float top, double total, bool soft) {
  return soft ? exp(double(x) - double(top)) / total : 1.0 / (1.0 + exp(-double(x)));
}
template <typename V>
__device__ inline V nan_first(V v) {
  return v == v ? v : V(INFINITY);
}

// Which groups stay: a group's value is that of its best experts; ties go to the lower group.
template <typename V>
__device__ inline int groups_before(const V* best, int groups, int g) {
  int before = 0;
#pragma unroll 4
  for (int h = 0; h < groups; ++h) before += best[h] > best[g] || (best[h] == best[g] && h < g);
  return before;
}
// The group of expert e < 2^10, by magic = 2^20 / per + 1: without a division.
__device__ inline int group_of(int e, int magic) { return int(__umul24(e, magic) >> 20); }

// ---- a wave for a token -----------------------------------------------------------------------
template <int NE>
struct WholeSpace {
  double value[64 * NE];
  double best[kMaxGroups];
  bool kept[kMaxGroups];
};

// The choice by maxima in turn, all in 64 bits: for more experts (above 512), choices or groups
// than 16 lanes take, and for tokens whose order fp32 could not tell. 16384 x 512 sigmoids with
// a bias: 46 us this way, 19 by 16 lanes; 16384 x 1024: 72 us (bf16 87), 53 without a bias, which
// needs no scores; 16 of 256: 39.
template <typename T, int NE>
__device__ inline void choose_whole(const SelectArgs& a, int64_t t, WholeSpace<NE>& space, int* chosen) {
  const int lane = threadIdx.x & 63;
  const double closed = kClosed;
  float x[NE];
  load_row<64, 1>(static_cast<const T*>(a.logits) + t * a.ld, lane, a.experts, kClosed, x);
  const bool soft = a.score == CCL_SCORE_SOFTMAX, grouped = a.kept < a.groups;
  const bool scored = a.bias || grouped;
  const float top = row_top<64>(x);
  double total = 0.0;
  if (scored && soft) {
#pragma unroll
    for (int i = 0; i < NE; ++i) total += exp(double(x[i]) - double(top));
    total = over_sum<64>(total);
  }
  double key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * 64 + lane;
    const float b = a.bias && e < a.experts ? a.bias[e] : 0.0f;
    double v = nan_first(double(x[i]));
    if (scored) v = nan_first(score_of(x[i], top, total, soft) + double(b));
    if (x[i] == kClosed || b == kClosed) v = closed;
    if (grouped) space.value[e] = v;
    key[i] = a.bias || v == closed ? v : nan_first(double(x[i]));
  }
  if (grouped) {
    const int per = a.per;
    __builtin_amdgcn_wave_barrier();
    double first = closed, second = closed;
    if (lane < a.groups)
      for (int q = 0; q < per; ++q) {
        const double w = space.value[lane * per + q];
        second = w > first ? first : w > second ? w : second;
        first = w > first ? w : first;
      }
    space.best[lane] = a.best == 2 && second > closed ? first + second : first;
    __builtin_amdgcn_wave_barrier();
    if (lane < a.groups) space.kept[lane] = groups_before(space.best, a.groups, lane) < a.kept;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 64 + lane;
      if (e < a.experts && !space.kept[group_of(e, a.magic)]) key[i] = closed;
    }
  }
  for (int c = 0; c < a.choices; ++c) {
    double m = closed;
    int at = a.experts;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i * 64 + lane;
      }
    const double best = over_max<64>(m);
    const int first = over<64>(m == best ? at : a.experts, [](int p, int q) { return min(p, q); });
    if (lane == 0) chosen[c] = first < a.experts ? first : -1;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (first == i * 64 + lane) key[i] = closed;
  }
  __builtin_amdgcn_wave_barrier();
}

// ---- gates -----------------------------------------------------------------------------------
// x, top: the row and its maximum; logit(e): one of the row's by its number.
template <int L, int Each, int NE, typename F>
__device__ inline void write_gates(const SelectArgs& a, int64_t t, int lane, const int* chosen, const float (&x)[NE],
                                   float top, F logit) {
  const bool soft = a.score == CCL_SCORE_SOFTMAX;
  int id[Each];
  float q[Each], m = kClosed, total = 1.0f;
#pragma unroll
  for (int j = 0; j < Each; ++j) {
    const int c = j * L + lane;
    id[j] = c < a.choices && t < a.tokens ? chosen[c] : -1;
    q[j] = id[j] >= 0 ? logit(id[j]) : kClosed;
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
    for (int i = 0; i < NE; ++i) total += exp_exact(x[i] - top);
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

template <typename T, int NE>
__global__ __launch_bounds__(kThreads) void select_whole_kernel(SelectArgs a) {
  __shared__ WholeSpace<NE> space[kThreads / 64];
  __shared__ int chosen[kThreads / 64][kMaxChoices];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / 64) + wave;
  if (t >= a.tokens) return;  // a whole wave
  choose_whole<T, NE>(a, t, space[wave], chosen[wave]);
  float x[NE];
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  load_row<64, 1>(row, lane, a.experts, kClosed, x);
  write_gates<64, 1>(a, t, lane, chosen[wave], x, row_top<64>(x), [&](int e) { return widen(row[e]); });
}

// ---- 16 lanes for a token ----------------------------------------------------------------------
constexpr int kCandidates = 48;
// Choices that the kernel of 16 lanes takes. Beyond, more experts than kCandidates reach the
// choices-th highest of 16 maxima too often: 41 of 256 on average for 16 choices.
constexpr int kFewChoices = 12;
constexpr int kFewGroups = 32;  // a word of bits

// LDS of a wave: four tokens.
template <int NE>
struct FewSpace {
  static constexpr int kRow = 18 * NE + 2;  // four values more every 32: groups of 32 in different banks
  int chosen[4][16];
  int whole_chosen[kMaxChoices];
  double value[4][kCandidates];
  int expert[4][kCandidates];
  union {
    struct {
      float row[4][kRow];  // the experts' values, while groups are ranked; then their logits
      float best[4][kFewGroups];
    } few;
    WholeSpace<(NE + 3) / 4> whole;
  };
  static __device__ inline int at(int e) { return e + (e >> 5) * 4; }
  static __device__ inline int at_pair(int p) { return 2 * (p + (p >> 3)); }
};

// What a value in fp32 may be off by, but for the addition of its bias (2^-24 of the sum). In a
// sigmoid p: p (1 - p) (2 + |x|) 2^-24 by the exponential and its argument, below 2^-24, and 3
// times 2^-24 p by the sum and the reciprocal. In a softmax: p |x| 2^-24 with p |x| < 0.4 by the
// argument, and 2^-24 p for each of the sum's at most 35 additions and for the functions. The
// bound is one for all sizes of p: of peaked rows it takes in experts whose p are smaller still,
// and with more than kCandidates of them the token is done in 64 bits. 16384 x 256 fp32, a bias of
// zeros: 17 us with logits of deviation 1.5, 30 with 4, 44 with 8, 57 with 16.
__device__ inline float value_off(bool soft) { return soft ? 0x1p-18f : 0x1p-22f; }

// Whether scores differ in 64 bits where the logits do, high > low: they come in the logits'
// order, but sigmoids near 1, terms of a softmax near 0 and any two of nearly the same logit
// round to the same value. In a softmax the scores' quotient is above 1 + high - low, and each
// is off by 2^-53 of low - top and a few steps of 2^-53. Sigmoids differ by a sixteenth of the
// logits' difference (1 at most) of p (1 - p) at least, each off by a few steps.
__device__ inline bool scores_differ(float high, float low, float top, bool soft) {
  const float gap = high - low;
  if (soft) return low - top > -600.0f && gap > 0x1p-48f * (2.0f + (top - low));
  return low > -600.0f && fminf(gap, 1.0f) * exp_exact(-fmaxf(low, 0.0f)) > 0x1p-45f;
}

// Takes the keys of experts outside the kept groups away; true where fp32 cannot tell which
// those are. v: the experts' values, or (not Scored) their logits, whose order groups of one
// best score have too, but for equal scores. top: the row's highest logit.
template <bool Scored, int V, int NE>
__device__ inline bool keep_groups(const SelectArgs& a, FewSpace<NE>& space, int token, int lane, const float (&v)[NE],
                                   float (&key)[NE], float top) {
  auto& s = space.few;
  const int groups = a.groups, parts = 1 << a.parts_log2;
  const bool vectors = V > 1 && a.per % V == 0;  // no vector lies in two groups
  if (vectors) {
    // the two best of a vector, from registers
#pragma unroll
    for (int i = 0; i < NE; i += V) {
      float first = fmaxf(v[i], v[i + 1]), second = fminf(v[i], v[i + 1]);
#pragma unroll
      for (int q = 2; q < V; q += 2) {
        const float high = fmaxf(v[i + q], v[i + q + 1]), low = fminf(v[i + q], v[i + q + 1]);
        second = fmaxf(fmaxf(second, low), fminf(first, high));
        first = fmaxf(first, high);
      }
      *reinterpret_cast<float2*>(&s.row[token][space.at_pair(expert_at<16, V>(i, lane) / V)]) = make_float2(first, second);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) s.row[token][space.at(expert_at<16, V>(i, lane))] = v[i];
  }
  __builtin_amdgcn_wave_barrier();
  // the lanes share out the groups, or parts of a group where those are few
  float size = 0.0f;  // of the values that groups' values are made of
  for (int j = lane; j < groups * parts; j += 16) {
    const int g = j >> a.parts_log2, part = j & (parts - 1);
    float first = kClosed, second = kClosed;
    if (vectors) {
      const int per = a.per / V;
#pragma unroll 4
      for (int e = g * per + part; e < g * per + per; e += parts) {
        const float2 w = *reinterpret_cast<const float2*>(&s.row[token][space.at_pair(e)]);
        second = fmaxf(fmaxf(second, w.y), fminf(first, w.x));
        first = fmaxf(first, w.x);
      }
    } else {
#pragma unroll 4
      for (int e = g * a.per + part; e < g * a.per + a.per; e += parts) {
        const float w = s.row[token][space.at(e)];
        second = fmaxf(second, fminf(first, w));
        first = fmaxf(first, w);
      }
    }
    for (int p = 1; p < parts; p *= 2) {  // groups x parts lanes, all of them here
      const float w = __shfl_xor(first, p), u = __shfl_xor(second, p);
      second = fmaxf(fmaxf(second, u), fminf(first, w));
      first = fmaxf(first, w);
    }
    const bool two = a.best == 2 && second > kClosed;
    s.best[token][g] = two ? first + second : first;
    if (Scored && first > kClosed) size = fmaxf(size, fabsf(first) + (two ? fabsf(second) : 0.0f));
  }
  __builtin_amdgcn_wave_barrier();
  float lowest = INFINITY, highest = kClosed;  // of the groups that stay, of the others
  unsigned kept = 0;
  for (int g = lane; g < 16 * ((groups + 15) / 16); g += 16) {
    const bool stays = g < groups && groups_before(s.best[token], groups, g) < a.kept;
    if (stays) lowest = fminf(lowest, s.best[token][g]);
    else if (g < groups) highest = fmaxf(highest, s.best[token][g]);
    kept |= (unsigned(__ballot(stays) >> (token * 16)) & 0xffff) << (g & 16);
  }
  // past the last expert keys are closed already, whatever their group would be
  auto stays = [&](int i) { return kept >> (group_of(expert_at<16, V>(i, lane), a.magic) & 31) & 1; };
  if (vectors) {
#pragma unroll
    for (int i = 0; i < NE; i += V) {
      const bool out = !stays(i);
#pragma unroll
      for (int q = 0; q < V; ++q) key[i + q] = out ? kClosed : key[i + q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (!stays(i)) key[i] = kClosed;
  }
  lowest = -over_max<16>(-lowest);
  highest = over_max<16>(highest);
  if constexpr (!Scored) {
    // No group that goes may have the score of one that stays by a higher logit. The nearest
    // such pairs: the lowest that stays above the highest that goes, and the reverse; one pair,
    // but where the two are the same. 16384 x 256 fp32 softmax, 4 of 8 groups: 14.7 -> 15.7 us.
    const bool soft = a.score == CCL_SCORE_SOFTMAX;
    float above = INFINITY, below = kClosed, best = kClosed;
    for (int g = lane; g < groups; g += 16) {
      const float w = s.best[token][g];
      best = fmaxf(best, w);
      if (w > highest) above = fminf(above, w);
      if (w < lowest) below = fmaxf(below, w);
    }
    above = -over_max<16>(-above);
    below = over_max<16>(below);
    best = over_max<16>(best);
    // infinite: or NaN, which ranks as that
    return best == INFINITY || (highest > kClosed && above < INFINITY && !scores_differ(above, highest, top, soft)) ||
           (below > kClosed && !scores_differ(lowest, below, top, soft));
  }
  size = over_max<16>(size);
  // on either side two values and their sum: 2 offs, and 2^-24 of the size for each addition
  return highest > kClosed && !(lowest - highest > 4 * value_off(a.score == CCL_SCORE_SOFTMAX) + 0x1p-22f * size);
}

// Scored: experts are ranked by p + bias, or groups by sums of p. Otherwise both by their
// logits, which fp32 holds as they are.
template <typename T, bool Scored, bool Grouped, int NE, int V>
__global__ __launch_bounds__(kThreads) void select_kernel(SelectArgs a) {
  __shared__ FewSpace<NE> spaces[kThreads / 64];
  FewSpace<NE>& space = spaces[threadIdx.x >> 6];
  const int lane = threadIdx.x & 15, token = (threadIdx.x & 63) >> 4;
  const int64_t t0 = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 6) * 4;
  const int64_t t = t0 + token;
  const bool soft = a.score == CCL_SCORE_SOFTMAX;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float x[NE];
  load_row<16, V>(row, lane, t < a.tokens ? a.experts : 0, kClosed, x);
  const float top = soft ? row_top<16>(x) : 0.0f;

  double total = 0.0;  // softmax with a bias: the sum is part of what is compared
  float key[NE];
  bool doubt = false;
  if constexpr (Scored) {
    float v[NE], lower[NE], sum = 0.0f;  // lower: of the logit and the bias, -inf where one is
    if (soft) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        v[i] = __builtin_amdgcn_exp2f((x[i] - top) * 1.44269504088896341f);
        sum += v[i];
      }
      sum = over_sum<16>(sum);
      const float inverse = sum != 0.0f ? reciprocal(sum) : 0.0f;  // 0: all closed
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] *= inverse;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = reciprocal(1.0f + __builtin_amdgcn_exp2f(x[i] * -1.44269504088896341f));
    }
    sum = 0.0f;
    if (a.bias) {
      float b[NE];
      load_row<16, V>(a.bias, lane, a.experts, 0.0f, b);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        v[i] += b[i];
        key[i] = v[i];
        sum += v[i];
        lower[i] = fminf(x[i], b[i]);
      }
      if (soft) {
#pragma unroll
        for (int i = 0; i < NE; ++i) total += exp(double(x[i]) - double(top));
        total = over_sum<16>(total);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        key[i] = lower[i] = x[i];
        sum += v[i];
      }
    }
    float lowest = lower[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) lowest = fminf(lowest, lower[i]);
    if (__ballot(lowest == kClosed)) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lower[i] == kClosed) key[i] = v[i] = kClosed;
    }
    doubt = !(sum == sum);  // a NaN somewhere
    if constexpr (Grouped) doubt = keep_groups<Scored, V>(a, space, token, lane, v, key, top) || doubt;
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = nan_first(x[i]);
    if constexpr (Grouped) {
      float v[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = key[i];
      doubt = keep_groups<Scored, V>(a, space, token, lane, v, key, top);
    }
  }

  // (a wave's LDS accesses are in order: nothing of the groups is overwritten before it is read)
#pragma unroll
  for (int i = 0; i < NE; ++i) space.few.row[token][space.at(expert_at<16, V>(i, lane))] = x[i];

  // the choices-th highest of the lanes' maxima: at least `choices` experts reach it
  float most = key[0];
#pragma unroll
  for (int i = 1; i < NE; ++i) most = fmaxf(most, key[i]);
  int above = 0;
#define CCL_MEET(N) above += turned<N>(most) > most;
  CCL_MEET(1) CCL_MEET(2) CCL_MEET(3) CCL_MEET(4) CCL_MEET(5) CCL_MEET(6) CCL_MEET(7) CCL_MEET(8)
  CCL_MEET(9) CCL_MEET(10) CCL_MEET(11) CCL_MEET(12) CCL_MEET(13) CCL_MEET(14) CCL_MEET(15)
#undef CCL_MEET
  float reach = -over_max<16>(above < a.choices ? -most : kClosed);
  if (Scored && a.bias && fabsf(reach) < INFINITY) reach -= 2 * value_off(soft) + 0x1p-22f * fabsf(reach);
  reach = fmaxf(reach, -__FLT_MAX__);  // closed ones never do

  // their numbers, lane by lane
  unsigned hits = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) hits |= key[i] >= reach ? 1u << i : 0u;
  const int mine = __popc(hits);
  int place = mine;  // up to and with this lane's
#define CCL_UPTO(N) place += __builtin_amdgcn_update_dpp(0, place, 0x110 + N, 0xf, 0xf, true);
  CCL_UPTO(1) CCL_UPTO(2) CCL_UPTO(4) CCL_UPTO(8)
#undef CCL_UPTO
  int count = over<16>(place, [](int p, int q) { return max(p, q); });
  place -= mine;
  while (hits) {
    const int i = __ffs(hits) - 1;
    hits &= hits - 1;
    if (place < kCandidates) space.expert[token][place] = expert_at<16, V>(i, lane);
    ++place;
  }
  doubt = doubt || count > kCandidates;
  count = min(count, kCandidates);
  if (lane >= count && lane < a.choices) space.chosen[token][lane] = -1;
  __builtin_amdgcn_wave_barrier();
  for (int c = lane; c < count; c += 16) {
    const int e = space.expert[token][c];
    const float logit = space.few.row[token][space.at(e)];
    space.value[token][c] =
        nan_first(Scored && a.bias ? score_of(logit, top, total, soft) + double(a.bias[e]) : double(logit));
  }
  __builtin_amdgcn_wave_barrier();
  for (int c = lane; c < count; c += 16) {
    const double v = space.value[token][c];
    const int e = space.expert[token][c];
    int rank = 0;
#pragma unroll 4
    for (int d = 0; d < count; ++d) {
      const double w = space.value[token][d];
      rank += w > v || (w == v && space.expert[token][d] < e);
    }
    if (rank < a.choices) space.chosen[token][rank] = e;
  }
  __builtin_amdgcn_wave_barrier();

  const unsigned long long doubts = __ballot(doubt && t < a.tokens);
  if (doubts) {  // takes the place of the logits in LDS
#pragma nounroll
    for (int j = 0; j < 4; ++j) {
      if (!((doubts >> (j * 16)) & 0xffff)) continue;
      choose_whole<T, (NE + 3) / 4>(a, t0 + j, space.whole, space.whole_chosen);
      if (token == j && lane < a.choices) space.chosen[j][lane] = space.whole_chosen[lane];
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) space.few.row[token][space.at(expert_at<16, V>(i, lane))] = x[i];
    __builtin_amdgcn_wave_barrier();
  }
  write_gates<16, 1>(a, t, lane, space.chosen[token], x, top,
                     [&](int e) { return space.few.row[token][space.at(e)]; });
}

// ---- the gradient --------------------------------------------------------------------------
// dx_e = p_e (d_e - sum p d) for softmax, d_e p_e (1 - p_e) for sigmoid, d the scores'
// gradients, zero but at the chosen experts; where the gates were divided by their sum the
// others have no part in them. The gradients of choices with the same id are added in their
// order.
// 16384 x 256 fp32: 9.1 us for 33.5 MB.
template <typename T, int L, int NE, int V, int Each>
__global__ __launch_bounds__(kThreads) void select_backward_kernel(SelectArgs a) {
  __shared__ int chosen[kThreads / L][L * Each];
  __shared__ float grad[kThreads / L][L * Each];
  __shared__ float spread[kThreads / L][L * NE];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kThreads / L) + slot;
  const bool soft = a.score == CCL_SCORE_SOFTMAX, whole = soft && !a.renorm;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float x[NE], m = 0.0f, total = 1.0f;
  if (whole) {  // p of every expert
    load_row<L, V>(row, lane, t < a.tokens ? a.experts : 0, kClosed, x);
    m = row_top<L>(x);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      x[i] = exp_exact(x[i] - m);
      total += x[i];
    }
    total = over_sum<L>(total);
    if (total == 0.0f) total = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) spread[slot][expert_at<L, V>(i, lane)] = 0.0f;

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
  const float share = whole ? flow / total : 0.0f;
  typedef T pack __attribute__((ext_vector_type(V)));
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = expert_at<L, V>(i, lane);
    if (e >= a.experts) continue;
    pack o;
#pragma unroll
    for (int q = 0; q < V; ++q) o[q] = narrow<T>(whole ? fmaf(-x[i + q], share, spread[slot][e + q]) : spread[slot][e + q]);
    *reinterpret_cast<pack*>(out + e) = o;
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
  const integral_constant<int, 16> few;
  const integral_constant<int, 64> wave;
  if (experts <= 32) f(few, integral_constant<int, 2>());
  else if (experts <= 64) f(few, integral_constant<int, 4>());
  else if (experts <= 128) f(few, integral_constant<int, 8>());
  else if (experts <= 256) f(few, integral_constant<int, 16>());
  else if (experts <= 512) f(few, integral_constant<int, 32>());
  else f(wave, integral_constant<int, 16>());
}

// Whether rows of `experts` values are whole vectors of V.
template <typename T, int V>
bool on_grid(const void* p, int64_t ld, int experts) {
  return reinterpret_cast<uintptr_t>(p) % (V * sizeof(T)) == 0 && ld % V == 0 && experts % V == 0;
}
template <typename T, int NE>
constexpr int vector_of() {
  return NE < 16 / int(sizeof(T)) ? NE : 16 / int(sizeof(T));
}

template <typename T, int NE, int V>
void select_few(const SelectArgs& a, hipStream_t s) {
  const bool grouped = a.kept < a.groups, scored = a.bias || (grouped && a.best == 2);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_grid<16>(a.tokens), dim3(kThreads), 0, s, a); };
  if (scored && grouped) go(select_kernel<T, true, true, NE, V>);
  else if (scored) go(select_kernel<T, true, false, NE, V>);
  else if (grouped) go(select_kernel<T, false, true, NE, V>);
  else go(select_kernel<T, false, false, NE, V>);
}

template <typename T>
int select_t(const SelectArgs& a, hipStream_t s, std::string* err) {
  by_experts(a.experts, [&](auto lanes, auto each) {
    constexpr int L = decltype(lanes)::value, NE = decltype(each)::value;
    auto whole = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_grid<64>(a.tokens), dim3(kThreads), 0, s, a); };
    if constexpr (L == 16) {
      constexpr int V = vector_of<T, NE>();
      if (a.choices > kFewChoices || (a.kept < a.groups && a.groups > kFewGroups)) whole(select_whole_kernel<T, (NE + 3) / 4>);
      else if (on_grid<T, V>(a.logits, a.ld, a.experts) && reinterpret_cast<uintptr_t>(a.bias) % (V * 4) == 0) select_few<T, NE, V>(a, s);
      else select_few<T, NE, 1>(a, s);
    } else {
      whole(select_whole_kernel<T, NE>);
    }
  });
  return hip_status("expert selection launch", err);
}

template <typename T>
int select_backward_t(const SelectArgs& a, hipStream_t s, std::string* err) {
  by_experts(a.experts, [&](auto lanes, auto each) {
    constexpr int L = decltype(lanes)::value, NE = decltype(each)::value, V = vector_of<T, NE>();
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, token_grid<L>(a.tokens), dim3(kThreads), 0, s, a); };
    const bool vec = on_grid<T, V>(a.logits, a.ld, a.experts) && on_grid<T, V>(a.dlogits, a.ldd, a.experts);
    if constexpr (L == 64) {
      if (vec) go(select_backward_kernel<T, L, NE, V, 1>);
      else go(select_backward_kernel<T, L, NE, 1, 1>);
    } else {
      if (a.choices > 16) go(select_backward_kernel<T, L, NE, 1, kMaxChoices / L>);
      else if (vec) go(select_backward_kernel<T, L, NE, V, 1>);
      else go(select_backward_kernel<T, L, NE, 1, 1>);
    }
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
