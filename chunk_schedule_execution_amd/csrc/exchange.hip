// The row exchange around an expert-parallel layer's AllToAlls for gfx950: routing (a
// stable counting sort of the choices by expert), dispatch, combine and its gradients.
// All of it is memory traffic; rows move as 16-byte vectors where they lie on that grid.
// 16384 tokens of 4 choices and 4096 bf16: combine 671 MB in 123 us, 5.5 TB/s; its gradient
// 1.21 GB in 221 us, 5.5 TB/s (a plain copy of 1 GB reaches 4.9).
#include <algorithm>

#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

constexpr int kMaxExperts = 1024;

// ---- routing ---------------------------------------------------------------------------
// The slots are cut into chunks, one wave each. A wave walks its chunk 64 slots at a time
// in order; lanes with the same expert find each other by ballots over the bits of the id,
// so a slot's place among its wave's earlier slots of the expert is a running count plus
// the number of lower lanes with the same id: stable without atomics.
__device__ inline unsigned long long same_id(int id, int bits) {
  unsigned long long m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const unsigned long long set = __ballot((id >> b) & 1);
    m &= ((id >> b) & 1) ? set : ~set;
  }
  return m;
}

// count[] += the chunk's slots by expert; with `positions`, count[] holds the next row of
// every expert and the slots get their rows.
template <bool Place>
__device__ inline void walk_chunk(const int32_t* ids, int64_t lo, int64_t hi, int experts, int bits, int* count,
                                  int32_t* positions, int32_t* slot_of) {
  const int lane = threadIdx.x & 63;
  for (int64_t s0 = lo; s0 < hi; s0 += 64) {
    const int64_t s = s0 + lane;
    int id = s < hi ? ids[s] : -1;
    const bool here = id >= 0 && id < experts;
    id = here ? id : experts;  // bits covers this value too
    const unsigned long long m = same_id(id, bits);
    const int before = __popcll(m & ((1ull << lane) - 1));
    int base = here ? count[id] : 0;
    if (Place && s < hi) {
      positions[s] = here ? base + before : -1;
      if (here) slot_of[base + before] = int32_t(s);
    }
    __builtin_amdgcn_wave_barrier();
    if (here && before == 0) count[id] = base + __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

__global__ __launch_bounds__(64) void route_count_kernel(const int32_t* ids, int64_t slots, int64_t chunk, int experts,
                                                         int bits, int32_t* counts) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < experts; e += 64) count[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk;
  walk_chunk<false>(ids, lo, min(slots, lo + chunk), experts, bits, count, nullptr, nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += 64) counts[int64_t(blockIdx.x) * experts + e] = count[e];
}

// counts[chunk][expert] -> first row of the chunk's slots of that expert; offsets.
__global__ __launch_bounds__(1024) void route_scan_kernel(int32_t* counts, int chunks, int experts, int32_t* offsets) {
  __shared__ int total[kMaxExperts];
  const int e = threadIdx.x;
  int sum = 0;
  if (e < experts)
    for (int c = 0; c < chunks; ++c) sum += counts[int64_t(c) * experts + e];
  total[e] = e < experts ? sum : 0;
  __syncthreads();
  for (int d = 1; d < kMaxExperts; d <<= 1) {
    const int v = e >= d ? total[e - d] : 0;
    __syncthreads();
    total[e] += v;
    __syncthreads();
  }
  if (e < experts) {
    int row = total[e] - sum;
    if (e == 0) offsets[0] = 0;
    offsets[e + 1] = total[e];
    for (int c = 0; c < chunks; ++c) {
      const int n = counts[int64_t(c) * experts + e];
      counts[int64_t(c) * experts + e] = row;
      row += n;
    }
  }
}

__global__ __launch_bounds__(64) void route_place_kernel(const int32_t* ids, int64_t slots, int64_t chunk, int experts,
                                                         int bits, const int32_t* first, const int32_t* offsets,
                                                         int32_t* positions, int32_t* slot_of) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < experts; e += 64) count[e] = first[int64_t(blockIdx.x) * experts + e];
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = min(slots, lo + chunk);
  walk_chunk<true>(ids, lo, hi, experts, bits, count, positions, slot_of);
  const int64_t used = offsets[experts];  // the rows behind the last expert's have no slot
  for (int64_t i = max(lo, used) + threadIdx.x; i < hi; i += 64) slot_of[i] = -1;
}

// A whole route in one workgroup, for few slots: the chunks are its 16 waves'.
__global__ __launch_bounds__(1024) void route_small_kernel(const int32_t* ids, int slots, int experts, int bits,
                                                           int32_t* offsets, int32_t* positions, int32_t* slot_of) {
  __shared__ int count[16][kMaxExperts];
  __shared__ int wave_total[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = lane; e < experts; e += 64) count[wave][e] = 0;
  const int chunk = ((slots + 15) / 16 + 63) / 64 * 64;
  const int lo = min(slots, wave * chunk), hi = min(slots, lo + chunk);
  __builtin_amdgcn_wave_barrier();
  walk_chunk<false>(ids, lo, hi, experts, bits, count[wave], nullptr, nullptr);
  __syncthreads();
  int sum = 0;
  if (tid < experts)
    for (int w = 0; w < 16; ++w) sum += count[w][tid];
  int upto = sum;  // of this and the earlier experts
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) wave_total[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += wave_total[w];
  if (tid < experts) {
    int row = upto - sum;
    if (tid == 0) offsets[0] = 0;
    offsets[tid + 1] = upto;
    for (int w = 0; w < 16; ++w) {
      const int n = count[w][tid];
      count[w][tid] = row;
      row += n;
    }
  }
  int used = 0;
  for (int w = 0; w < 16; ++w) used += wave_total[w];
  __syncthreads();
  walk_chunk<true>(ids, lo, hi, experts, bits, count[wave], positions, slot_of);
  for (int i = used + tid; i < slots; i += 1024) slot_of[i] = -1;
}
// One kernel takes 3.3 us at 192 slots and 13.5 at 8192, where a wave walks 8 rounds of 64
// slots. The three of a long route take 6, 8 and 5.4 us at 8196 slots, and the scan, which
// walks the chunks' counts one after another, grows with their number: 41 us at 65536 slots,
// 78 from 131072 on, where there are 256 chunks; the other two 55 and 59 at 1600000.
constexpr int64_t kSmallRoute = 8192;

struct RoutePlan {
  int64_t chunk;
  int chunks;
};
// At most 256 chunks, since the scan walks them one by one, of at least 512 slots.
RoutePlan route_plan(int64_t slots) {
  int64_t chunk = (slots + 255) / 256;
  chunk = std::max<int64_t>(512, (chunk + 63) / 64 * 64);
  return {chunk, int((slots + chunk - 1) / chunk)};
}

// ---- rows --------------------------------------------------------------------------------
// V elements as they move: 16 bytes, or one element where rows are off that grid.
template <typename T, int V>
struct __attribute__((aligned(sizeof(T) * V))) Pack {
  T v[V];
};

// A store around the caches, for rows that are written once and whole.
template <typename T, int V>
__device__ inline void stream(Pack<T, V>* to, const Pack<T, V>& x) {
  if constexpr (sizeof(x) == 16) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, x), reinterpret_cast<u32x4*>(to));
  } else {
    *to = x;
  }
}

// A load around the caches, of rows that are read once: 6 us of the 129 that combine takes
// with plain loads at 16384 tokens of 4 choices and 4096 bf16, 29 of its gradient's 250.
template <typename T, int V>
__device__ inline Pack<T, V> load_once(const Pack<T, V>* from) {
  if constexpr (sizeof(Pack<T, V>) == 16) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(Pack<T, V>, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from)));
  } else {
    return *from;
  }
}

template <typename T, int V>
__global__ __launch_bounds__(256) void dispatch_kernel(const T* x, int64_t ldx, const int32_t* slots, int64_t count,
                                                       int choices, int64_t width, T* rows, int64_t ldr) {
  using P = Pack<T, V>;
  const int64_t i = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= count) return;
  const int slot = slots[i];
  const bool here = slot >= 0 && slot < count;
  const P* src = reinterpret_cast<const P*>(x + (here ? slot / choices : 0) * ldx);
  P* dst = reinterpret_cast<P*>(rows + i * ldr);
  const int64_t n = width / V;
  const P zero = {};
  for (int64_t c = threadIdx.x & 63; c < n; c += 64) stream(dst + c, here ? src[c] : zero);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void combine_kernel(const T* h, int64_t ldh, const int32_t* positions,
                                                      const float* gates, int64_t tokens, int choices, int64_t width,
                                                      T* out, int64_t ldo) {
  using P = Pack<T, V>;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t c = int64_t(blockIdx.z) * blockDim.x + threadIdx.x;
  if (t >= tokens || c >= width / V) return;
  const int64_t count = tokens * choices;
  float sum[V] = {};
  for (int j = 0; j < choices; ++j) {
    const int p = positions[t * choices + j];
    if (p < 0 || p >= count) continue;
    const float gate = gates ? gates[t * choices + j] : 1.0f;
    const P v = load_once(reinterpret_cast<const P*>(h + p * ldh) + c);
#pragma unroll
    for (int q = 0; q < V; ++q) sum[q] += gate * widen(v.v[q]);
  }
  P o;
#pragma unroll
  for (int q = 0; q < V; ++q) o.v[q] = narrow<T>(sum[q]);
  stream(reinterpret_cast<P*>(out + t * ldo) + c, o);
}

// One wave per token: Held packs of dout's row per lane are read once and stay in registers
// (a wave per row of h read them once per choice: 3 % more), longer rows take several rounds;
// then for each choice h's row is read, its product with dout summed and dh's row written.
// Held is 4: 16384 tokens of 4 choices and 4096 bf16 take 221 us (with 8, fewer waves, 276;
// with 2, shorter pieces of rows, 280; two rows of h at a time 224). The blocks behind the
// tokens' look for rows that no slot has and clear them.
template <typename T, int V, int Held>
__global__ __launch_bounds__(256) void combine_backward_kernel(const T* dout, int64_t ldo, const T* h, int64_t ldh,
                                                               const int32_t* positions, const int32_t* slots,
                                                               const float* gates, int64_t tokens, int choices,
                                                               int64_t width, T* dh, int64_t lddh, float* dgates) {
  using P = Pack<T, V>;
  const int64_t count = tokens * choices, n = width / V, token_blocks = (tokens + 3) / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t block = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  if (block >= token_blocks) {
    if (!dh) return;
    const int64_t first = (block - token_blocks) * 256 + wave * 64;
    const int slot = first + lane < count ? slots[first + lane] : 0;
    unsigned long long empty = __ballot(slot < 0 || slot >= count);
    const P zero = {};
    while (empty) {
      const int l = __ffsll(empty) - 1;
      empty &= empty - 1;
      P* dst = reinterpret_cast<P*>(dh + (first + l) * lddh);
      for (int64_t c = lane; c < n; c += 64) dst[c] = zero;
    }
    return;
  }
  const int64_t t = block * 4 + wave;
  if (t >= tokens) return;
  const P* src = reinterpret_cast<const P*>(dout + t * ldo);
  for (int j0 = 0; j0 < choices; j0 += 64) {  // lanes hold the choices' rows, gates and sums
    const bool mine = j0 + lane < choices;
    const int64_t at = t * choices + j0 + lane;
    int row = mine ? positions[at] : -1;
    if (row >= count) row = -1;
    const float gate = mine && row >= 0 && gates ? gates[at] : 1.0f;
    float dot = 0.0f;
    const int here = min(64, choices - j0);
    for (int64_t c0 = 0; c0 < n; c0 += 64 * Held) {
      P d[Held];
#pragma unroll
      for (int i = 0; i < Held; ++i)
        if (c0 + i * 64 + lane < n) d[i] = src[c0 + i * 64 + lane];
      for (int j = 0; j < here; ++j) {
        const int r = __builtin_amdgcn_readlane(row, j);
        if (r < 0) continue;
        const float scale = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gate), j));
        float sum = 0.0f;
        if (dgates) {
          const P* hrow = reinterpret_cast<const P*>(h + r * ldh);
          P v[Held];
#pragma unroll
          for (int i = 0; i < Held; ++i)
            if (c0 + i * 64 + lane < n) v[i] = load_once(hrow + c0 + i * 64 + lane);
#pragma unroll
          for (int i = 0; i < Held; ++i)
            if (c0 + i * 64 + lane < n)
#pragma unroll
              for (int q = 0; q < V; ++q) sum += widen(d[i].v[q]) * widen(v[i].v[q]);
#pragma unroll
          for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
          if (lane == j) dot += sum;
        }
        if (dh) {
          P* dst = reinterpret_cast<P*>(dh + r * lddh);
#pragma unroll
          for (int i = 0; i < Held; ++i)
            if (c0 + i * 64 + lane < n) {
              P o;
#pragma unroll
              for (int q = 0; q < V; ++q) o.v[q] = narrow<T>(scale * widen(d[i].v[q]));
              stream(dst + c0 + i * 64 + lane, o);
            }
        }
      }
    }
    if (mine && dgates) dgates[at] = dot;
  }
}

// Whether rows of `width` elements at base p, ld apart, are whole 16-byte vectors.
inline bool on_grid(const void* p, int64_t ld, int64_t width, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && width * size % 16 == 0;
}

}  // namespace
}  // namespace prod

using namespace prod;

int64_t route_workspace(int64_t slots, int experts) {
  return slots <= kSmallRoute ? 0 : int64_t(route_plan(slots).chunks) * experts * 4;
}

int launch_route(const int32_t* ids, int64_t slots, int experts, int32_t* offsets, int32_t* positions, int32_t* slot_of,
                 void* workspace, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const RoutePlan p = route_plan(slots);
  int bits = 1;
  while ((1 << bits) <= experts) ++bits;
  if (slots <= kSmallRoute) {
    hipLaunchKernelGGL(route_small_kernel, dim3(1), dim3(1024), 0, s, ids, int(slots), experts, bits, offsets, positions,
                       slot_of);
    return hip_status("route launch", err);
  }
  int32_t* counts = static_cast<int32_t*>(workspace);
  hipLaunchKernelGGL(route_count_kernel, dim3(p.chunks), dim3(64), 0, s, ids, slots, p.chunk, experts, bits, counts);
  hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(kMaxExperts), 0, s, counts, p.chunks, experts, offsets);
  hipLaunchKernelGGL(route_place_kernel, dim3(p.chunks), dim3(64), 0, s, ids, slots, p.chunk, experts, bits, counts,
                     offsets, positions, slot_of);
  return hip_status("route launch", err);
}

template <typename T>
static int dispatch_t(const void* x, int64_t ldx, const int32_t* slots, int64_t tokens, int choices, int64_t width,
                      void* rows, int64_t ldr, hipStream_t s, std::string* err) {
  constexpr int V = 16 / int(sizeof(T));
  const int64_t count = tokens * choices;
  const dim3 grid = flat_grid((count + 3) / 4);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, static_cast<const T*>(x), ldx, slots, count, choices, width,
                       static_cast<T*>(rows), ldr);
  };
  if (on_grid(x, ldx, width, sizeof(T)) && on_grid(rows, ldr, width, sizeof(T))) go(dispatch_kernel<T, V>);
  else go(dispatch_kernel<T, 1>);
  return hip_status("dispatch launch", err);
}

int launch_dispatch(int dtype, const void* x, int64_t ldx, const int32_t* slots, int64_t tokens, int choices,
                    int64_t width, void* rows, int64_t ldr, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? dispatch_t<bf16>(x, ldx, slots, tokens, choices, width, rows, ldr, s, err)
                           : dispatch_t<float>(x, ldx, slots, tokens, choices, width, rows, ldr, s, err);
}

template <typename T>
static int combine_t(const void* h, int64_t ldh, const int32_t* positions, const float* gates, int64_t tokens,
                     int choices, int64_t width, void* out, int64_t ldo, hipStream_t s, std::string* err) {
  constexpr int V = 16 / int(sizeof(T));
  const bool wide = on_grid(h, ldh, width, sizeof(T)) && on_grid(out, ldo, width, sizeof(T));
  const int64_t n = wide ? width / V : width;
  int bx = 64;  // whole waves along a row; short rows share a workgroup
  while (bx < 256 && bx < n) bx *= 2;
  const dim3 block(bx, 256 / bx);
  dim3 grid = flat_grid((tokens + block.y - 1) / block.y);
  grid.z = unsigned((n + bx - 1) / bx);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, static_cast<const T*>(h), ldh, positions, gates, tokens, choices,
                       width, static_cast<T*>(out), ldo);
  };
  if (wide) go(combine_kernel<T, V>);
  else go(combine_kernel<T, 1>);
  return hip_status("combine launch", err);
}

int launch_combine(int dtype, const void* h, int64_t ldh, const int32_t* positions, const float* gates, int64_t tokens,
                   int choices, int64_t width, void* out, int64_t ldo, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? combine_t<bf16>(h, ldh, positions, gates, tokens, choices, width, out, ldo, s, err)
                           : combine_t<float>(h, ldh, positions, gates, tokens, choices, width, out, ldo, s, err);
}

template <typename T>
static int combine_backward_t(const void* dout, int64_t ldo, const void* h, int64_t ldh, const int32_t* positions,
                              const int32_t* slots, const float* gates, int64_t tokens, int choices, int64_t width,
                              void* dh, int64_t lddh, float* dgates, hipStream_t s, std::string* err) {
  constexpr int V = 16 / int(sizeof(T));
  const dim3 grid = flat_grid((tokens + 3) / 4 + (tokens * choices + 255) / 256);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, static_cast<const T*>(dout), ldo, static_cast<const T*>(h), ldh,
                       positions, slots, gates, tokens, choices, width, static_cast<T*>(dh), lddh, dgates);
  };
  const bool wide = on_grid(dout, ldo, width, sizeof(T)) && (!dgates || on_grid(h, ldh, width, sizeof(T))) &&
                    (!dh || on_grid(dh, lddh, width, sizeof(T)));
  if (wide) go(combine_backward_kernel<T, V, 4>);
  else go(combine_backward_kernel<T, 1, 4>);
  return hip_status("combine gradient launch", err);
}

int launch_combine_backward(int dtype, const void* dout, int64_t ldo, const void* h, int64_t ldh,
                            const int32_t* positions, const int32_t* slots, const float* gates, int64_t tokens,
                            int choices, int64_t width, void* dh, int64_t lddh, float* dgates, void* stream,
                            std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? combine_backward_t<bf16>(dout, ldo, h, ldh, positions, slots, gates, tokens, choices,
                                                      width, dh, lddh, dgates, s, err)
                           : combine_backward_t<float>(dout, ldo, h, ldh, positions, slots, gates, tokens, choices,
                                                       width, dh, lddh, dgates, s, err);
}

}  // namespace ccl
