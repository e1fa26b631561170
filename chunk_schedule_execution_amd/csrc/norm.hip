// Layer norm with the residual's addition for gfx950, and its gradients. Memory bounds both:
// a row is read once and stays in registers for its mean, its variance and its result.
#include <algorithm>

#include "lanes.h"
#include "layers.h"
#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

// V elements as they move: 16 bytes, or one element where rows are off that grid.
template <typename T, int V>
struct __attribute__((aligned(sizeof(T) * V))) Pack {
  T v[V];
};

// Rows are read and written once: around the caches.
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
__device__ inline void store_once(Pack<T, V>* to, const Pack<T, V>& x) {
  if constexpr (sizeof(x) == 16) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, x), reinterpret_cast<u32x4*>(to));
  } else {
    *to = x;
  }
}

// All waves' LDS accesses before this point are done; loads from memory stay in flight.
__device__ inline void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ inline int64_t flat_block() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }
inline dim3 flat_grid(int64_t n) {
  const int64_t x = std::min<int64_t>(n, 1 << 20);
  return dim3(unsigned(x), unsigned((n + x - 1) / x));
}

// ---- forward -------------------------------------------------------------------------------
// The sum of v over the R threads of a row: a wave, or the workgroup's four.
template <int R>
__device__ inline float row_sum(float v, float* parts) {
  v = over_sum<64>(v);
  if constexpr (R == 64) {
    return v;
  } else {
    if (threadIdx.x % 64 == 0) parts[threadIdx.x / 64] = v;
    lds_barrier();
    return (parts[0] + parts[1]) + (parts[2] + parts[3]);
  }
}

// R threads hold a row, Held packs each. The variance is the mean of squared differences
// from the mean, from registers: nothing cancels.
template <typename T, int V, int Held, int R>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  using P = Pack<T, V>;
  __shared__ float parts[2][4];
  const int lane = threadIdx.x % R;
  const int64_t row = flat_block() * (256 / R) + threadIdx.x / R;
  if (row >= a.rows) return;  // a whole wave, or the workgroup
  const int n = int(a.width / V);
  const P* x = reinterpret_cast<const P*>(static_cast<const T*>(a.x) + row * a.ld_x);
  float h[Held][V];
  float sum = 0.0f;
  if (a.residual) {
    const P* r = reinterpret_cast<const P*>(static_cast<const T*>(a.residual) + row * a.ld_residual);
    P px[Held], pr[Held];
#pragma unroll
    for (int i = 0; i < Held; ++i)
      if (i * R + lane < n) {
        px[i] = load_once(x + i * R + lane);
        pr[i] = load_once(r + i * R + lane);
      }
    P* total = reinterpret_cast<P*>(static_cast<T*>(a.total) + row * a.ld_total);
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      const bool in = i * R + lane < n;
#pragma unroll
      for (int q = 0; q < V; ++q) h[i][q] = in ? widen(px[i].v[q]) + widen(pr[i].v[q]) : 0.0f;
      if (in && a.total) {
        P o;
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = narrow<T>(h[i][q]);
        store_once(total + i * R + lane, o);
      }
    }
  } else {
    P px[Held];
#pragma unroll
    for (int i = 0; i < Held; ++i)
      if (i * R + lane < n) px[i] = load_once(x + i * R + lane);
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) h[i][q] = i * R + lane < n ? widen(px[i].v[q]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < Held; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q) sum += h[i][q];
  const float mean = row_sum<R>(sum, parts[0]) / float(a.width);
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < Held; ++i)
    if (i * R + lane < n)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        h[i][q] -= mean;
        squares = fmaf(h[i][q], h[i][q], squares);
      }
  const float rstd = 1.0f / sqrtf(row_sum<R>(squares, parts[1]) / float(a.width) + a.eps);
  if (a.mean && lane == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  P* out = reinterpret_cast<P*>(static_cast<T*>(a.out) + row * a.ld_out);
#pragma unroll
  for (int i = 0; i < Held; ++i) {
    const int c = i * R + lane;
    if (c >= n) continue;
    P o, pw, pb;
    if (w) pw = w[c];
    if (b) pb = b[c];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      float v = h[i][q] * rstd;
      if (w) v *= widen(pw.v[q]);
      if (b) v += widen(pb.v[q]);
      o.v[q] = narrow<T>(v);
    }
    store_once(out + c, o);
  }
}

// Rows that registers do not hold: read three times, the second and third time from the
// caches as far as they go. 1024 threads a row, 8 columns each at a time.
template <typename T>
__device__ inline float block_sum(float v, float* parts) {
  v = over_sum<64>(v);
  if (threadIdx.x % 64 == 0) parts[threadIdx.x / 64] = v;
  lds_barrier();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += parts[i];
  return s;
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
  __shared__ float parts[2][16];
  const int64_t row = flat_block(), step = 1024 * 8;
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ld_residual : nullptr;
  const bool vec_x = on_vectors<T>(x, 0), vec_r = on_vectors<T>(r, 0), vec_w = on_vectors<T>(a.weight, 0),
             vec_b = on_vectors<T>(a.bias, 0);
  T* out = static_cast<T*>(a.out) + row * a.ld_out;
  T* total = a.total ? static_cast<T*>(a.total) + row * a.ld_total : nullptr;
  const bool vec_o = on_vectors<T>(out, 0), vec_t = on_vectors<T>(total, 0);
  auto read = [&](int64_t c, int n, float (&h)[8]) {
    load8(x + c, vec_x, n, h);
    if (r) {
      float v[8];
      load8(r + c, vec_r, n, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] += v[q];
    }
  };
  float sum = 0.0f, squares = 0.0f, h[8];
  for (int64_t c = threadIdx.x * 8; c < a.width; c += step) {
    const int n = int(min(int64_t(8), a.width - c));
    read(c, n, h);
    if (total) store8(total + c, vec_t, n, h);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum += h[q];
  }
  const float mean = block_sum<T>(sum, parts[0]) / float(a.width);
  for (int64_t c = threadIdx.x * 8; c < a.width; c += step) {
    const int n = int(min(int64_t(8), a.width - c));
    read(c, n, h);
#pragma unroll
    for (int q = 0; q < 8; ++q) squares += q < n ? (h[q] - mean) * (h[q] - mean) : 0.0f;
  }
  const float rstd = 1.0f / sqrtf(block_sum<T>(squares, parts[1]) / float(a.width) + a.eps);
  if (a.mean && threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  for (int64_t c = threadIdx.x * 8; c < a.width; c += step) {
    const int n = int(min(int64_t(8), a.width - c));
    float v[8];
    read(c, n, h);
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = (h[q] - mean) * rstd;
    if (a.weight) {
      load8(static_cast<const T*>(a.weight) + c, vec_w, n, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] *= v[q];
    }
    if (a.bias) {
      load8(static_cast<const T*>(a.bias) + c, vec_b, n, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] += v[q];
    }
    store8(out + c, vec_o, n, h);
  }
}

// ---- gradients -----------------------------------------------------------------------------
// With g = dout w and y = (x - mean) rstd: dx = rstd (g - mean(g) - y mean(g y)) + dtotal,
// dw = sum over the rows of dout y, db of dout. A workgroup walks rows, Held packs of a row
// per thread, always the same columns, whose share of dw and db stays in registers: one pass
// over the rows gives all three. Each workgroup leaves its share in `partial`.
template <typename T, int V, int Held, int Threads>
__global__ __launch_bounds__(Threads) void norm_backward_kernel(NormArgs a) {
  using P = Pack<T, V>;
  constexpr int Waves = Threads / 64;
  __shared__ float parts[2][Waves][2];
  const int tid = threadIdx.x, n = int(a.width / V);
  float dw[Held][V] = {}, db[Held][V] = {}, w[Held][V];
#pragma unroll
  for (int i = 0; i < Held; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q)
      w[i][q] = a.weight && i * Threads + tid < n ? widen(static_cast<const P*>(a.weight)[i * Threads + tid].v[q]) : 1.0f;
  P px[Held], pd[Held], pt[Held];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
    const P* x = reinterpret_cast<const P*>(static_cast<const T*>(a.x) + row * a.ld_x);
    const P* d = reinterpret_cast<const P*>(static_cast<const T*>(a.dout) + row * a.ld_out);
    mean = a.mean[row];
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < Held; ++i)
      if (i * Threads + tid < n) {
        px[i] = load_once(x + i * Threads + tid);
        pd[i] = load_once(d + i * Threads + tid);
      }
    if (a.dtotal) {
      const P* t = reinterpret_cast<const P*>(static_cast<const T*>(a.dtotal) + row * a.ld_dtotal);
#pragma unroll
      for (int i = 0; i < Held; ++i)
        if (i * Threads + tid < n) pt[i] = load_once(t + i * Threads + tid);
    }
  };
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    load(row);
    float y[Held][V], g[Held][V], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const bool in = i * Threads + tid < n;
        const float d = in ? widen(pd[i].v[q]) : 0.0f;
        y[i][q] = in ? (widen(px[i].v[q]) - mean) * rstd : 0.0f;
        dw[i][q] = fmaf(d, y[i][q], dw[i][q]);
        db[i][q] += d;
        g[i][q] = d * w[i][q];
        sum += g[i][q];
        dot = fmaf(g[i][q], y[i][q], dot);
      }
    if (!a.dx) continue;  // the same for all
    sum = over_sum<64>(sum);
    dot = over_sum<64>(dot);
    if (tid % 64 == 0) {
      parts[turn][tid / 64][0] = sum;
      parts[turn][tid / 64][1] = dot;
    }
    // one barrier a row: the other half of `parts` may still be read
    lds_barrier();
    sum = dot = 0.0f;
#pragma unroll
    for (int k = 0; k < Waves; ++k) {
      sum += parts[turn][k][0];
      dot += parts[turn][k][1];
    }
    sum /= float(a.width);
    dot /= float(a.width);
    P* dx = reinterpret_cast<P*>(static_cast<T*>(a.dx) + row * a.ld_dx);
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      if (i * Threads + tid >= n) continue;
      P o;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        float v = rstd * (g[i][q] - sum - y[i][q] * dot);
        if (a.dtotal) v += widen(pt[i].v[q]);
        o.v[q] = narrow<T>(v);
      }
      store_once(dx + i * Threads + tid, o);
    }
  }
  if (!a.partial) return;
  float* to = a.partial + int64_t(blockIdx.x) * 2 * a.width;
#pragma unroll
  for (int i = 0; i < Held; ++i)
    if (i * Threads + tid < n)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int64_t c = int64_t(i * Threads + tid) * V + q;
        to[c] = dw[i][q];
        to[a.width + c] = db[i][q];
      }
}

// Rows that registers do not hold. dx: a workgroup a row, read twice.
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(NormArgs a) {
  __shared__ float parts[2][16];
  const int64_t row = flat_block(), step = 1024 * 8;
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* d = static_cast<const T*>(a.dout) + row * a.ld_out;
  const T* t = a.dtotal ? static_cast<const T*>(a.dtotal) + row * a.ld_dtotal : nullptr;
  T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
  const bool vec_x = on_vectors<T>(x, 0), vec_d = on_vectors<T>(d, 0), vec_t = on_vectors<T>(t, 0),
             vec_w = on_vectors<T>(a.weight, 0), vec_o = on_vectors<T>(dx, 0);
  const float mean = a.mean[row], rstd = a.rstd[row];
  auto read = [&](int64_t c, int n, float (&y)[8], float (&g)[8]) {
    load8(x + c, vec_x, n, y);
    load8(d + c, vec_d, n, g);
    float w[8];
    if (a.weight) load8(static_cast<const T*>(a.weight) + c, vec_w, n, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      y[q] = (y[q] - mean) * rstd;
      if (a.weight) g[q] *= w[q];
    }
  };
  float sum = 0.0f, dot = 0.0f, y[8], g[8];
  for (int64_t c = threadIdx.x * 8; c < a.width; c += step) {
    const int n = int(min(int64_t(8), a.width - c));
    read(c, n, y, g);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) {
        sum += g[q];
        dot = fmaf(g[q], y[q], dot);
      }
  }
  sum = block_sum<T>(sum, parts[0]) / float(a.width);
  dot = block_sum<T>(dot, parts[1]) / float(a.width);
  for (int64_t c = threadIdx.x * 8; c < a.width; c += step) {
    const int n = int(min(int64_t(8), a.width - c));
    read(c, n, y, g);
    float v[8] = {};
    if (t) load8(t + c, vec_t, n, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += rstd * (g[q] - sum - y[q] * dot);
    store8(dx + c, vec_o, n, v);
  }
}

// dw's and db's share of a band of rows: 256 columns, 8 per thread, 8 rows at a time.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs a, int64_t height) {
  __shared__ float sums[2][8][256];
  const int64_t c = int64_t(blockIdx.y) * 256 + (threadIdx.x & 31) * 8;
  const int n = int(min(int64_t(8), a.width - c)), lane = threadIdx.x >> 5;
  const bool vec_x = on_vectors<T>(a.x, a.ld_x), vec_d = on_vectors<T>(a.dout, a.ld_out);
  const int64_t first = blockIdx.x * height, end = min(a.rows, first + height);
  float dw[8] = {}, db[8] = {};
  if (n > 0)
    for (int64_t r = first + lane; r < end; r += 8) {
      float x[8], d[8];
      load8(static_cast<const T*>(a.x) + r * a.ld_x + c, vec_x, n, x);
      load8(static_cast<const T*>(a.dout) + r * a.ld_out + c, vec_d, n, d);
      const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        dw[q] = fmaf(d[q], (x[q] - mean) * rstd, dw[q]);
        db[q] += d[q];
      }
    }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    sums[0][lane][(threadIdx.x & 31) * 8 + q] = dw[q];
    sums[1][lane][(threadIdx.x & 31) * 8 + q] = db[q];
  }
  __syncthreads();
  float w = 0.0f, b = 0.0f;
#pragma unroll
  for (int l = 0; l < 8; ++l) {
    w += sums[0][l][threadIdx.x];
    b += sums[1][l][threadIdx.x];
  }
  const int64_t at = int64_t(blockIdx.y) * 256 + threadIdx.x;
  if (at >= a.width) return;
  float* to = a.partial + int64_t(blockIdx.x) * 2 * a.width;
  to[at] = w;
  to[a.width + at] = b;
}

// The shares added up, 16 interleaved runs of them and then those, always in that order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs a, int64_t shares) {
  __shared__ float sums[16][64];
  const int64_t c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int run = threadIdx.x >> 6;
  T* to = static_cast<T*>(blockIdx.y ? a.dbias : a.dweight);
  if (!to) return;
  const float* from = a.partial + blockIdx.y * a.width + c;
  float sum = 0.0f;
  if (c < a.width) {
#pragma unroll 8
    for (int64_t i = run; i < shares; i += 16) sum += from[i * 2 * a.width];
  }
  sums[run][threadIdx.x & 63] = sum;
  __syncthreads();
  if (run || c >= a.width) return;
#pragma unroll
  for (int r = 1; r < 16; ++r) sum += sums[r][threadIdx.x];
  to[c] = narrow<T>(sum);
}

// ---- choice of kernels -----------------------------------------------------------------------
template <typename T>
bool on_grid(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(T) % 16 == 0;
}

template <typename T, int V>
bool norm_held(const NormArgs& a, hipStream_t s) {
  const int64_t n = a.width / V;
  auto go = [&](auto kernel, int rows) {
    hipLaunchKernelGGL(kernel, flat_grid((a.rows + rows - 1) / rows), dim3(256), 0, s, a);
    return true;
  };
  // a wave a row where there are rows enough for all units
  if (a.rows >= 1024) {
    if (n <= 64) return go(norm_kernel<T, V, 1, 64>, 4);
    if (n <= 128) return go(norm_kernel<T, V, 2, 64>, 4);
    if (n <= 256) return go(norm_kernel<T, V, 4, 64>, 4);
    if (n <= 512) return go(norm_kernel<T, V, 8, 64>, 4);
  }
  if (n <= 256) return go(norm_kernel<T, V, 1, 256>, 1);
  if (n <= 512) return go(norm_kernel<T, V, 2, 256>, 1);
  if (n <= 1024) return go(norm_kernel<T, V, 4, 256>, 1);
  if (n <= 2048) return go(norm_kernel<T, V, 8, 256>, 1);
  if constexpr (V == 1)
    if (n <= 4096) return go(norm_kernel<T, V, 16, 256>, 1);
  return false;
}

template <typename T>
int norm_t(const NormArgs& a, hipStream_t s, std::string* err) {
  constexpr int V = 16 / int(sizeof(T));
  const bool wide = a.width % V == 0 && on_grid<T>(a.x, a.ld_x) && on_grid<T>(a.residual, a.ld_residual) &&
                    on_grid<T>(a.out, a.ld_out) && on_grid<T>(a.total, a.ld_total) && on_grid<T>(a.weight, 0) &&
                    on_grid<T>(a.bias, 0);
  if (!(wide ? norm_held<T, V>(a, s) : norm_held<T, 1>(a, s)))
    hipLaunchKernelGGL(norm_long_kernel<T>, flat_grid(a.rows), dim3(1024), 0, s, a);
  return hip_status("layer norm launch", err);
}

// Workgroups that walk the rows.
int64_t walkers(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(512, (rows + 3) / 4)); }
int64_t band_height(int64_t rows) { return std::max<int64_t>(64, (rows + 511) / 512); }

template <typename T, int V>
bool norm_backward_held(const NormArgs& a, hipStream_t s) {
  const int64_t n = a.width / V;
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(walkers(a.rows))), dim3(threads), 0, s, a);
    return true;
  };
  if (n <= 256) return go(norm_backward_kernel<T, V, 1, 256>, 256);
  if (n <= 512) return go(norm_backward_kernel<T, V, 2, 256>, 256);
  if (n <= 1024) return go(norm_backward_kernel<T, V, 2, 512>, 512);
  if (n <= 2048) return go(norm_backward_kernel<T, V, 2, 1024>, 1024);
  if constexpr (V == 1)
    if (n <= 4096) return go(norm_backward_kernel<T, V, 4, 1024>, 1024);
  return false;
}

template <typename T>
int norm_backward_t(const NormArgs& args, hipStream_t s, std::string* err) {
  constexpr int V = 16 / int(sizeof(T));
  NormArgs a = args;
  const bool sums = a.dweight || a.dbias;
  if (!sums) a.partial = nullptr;
  const bool wide = a.width % V == 0 && on_grid<T>(a.x, a.ld_x) && on_grid<T>(a.dout, a.ld_out) &&
                    on_grid<T>(a.dtotal, a.ld_dtotal) && on_grid<T>(a.dx, a.ld_dx) && on_grid<T>(a.weight, 0);
  int64_t shares = walkers(a.rows);
  if (a.rows > 0 && !(wide ? norm_backward_held<T, V>(a, s) : norm_backward_held<T, 1>(a, s))) {
    if (a.dx) hipLaunchKernelGGL(norm_backward_long_kernel<T>, flat_grid(a.rows), dim3(1024), 0, s, a);
    const int64_t height = band_height(a.rows);
    shares = (a.rows + height - 1) / height;
    if (sums)
      hipLaunchKernelGGL(norm_columns_kernel<T>, dim3(unsigned(shares), unsigned((a.width + 255) / 256)), dim3(256), 0, s,
                         a, height);
  }
  if (sums)
    hipLaunchKernelGGL(norm_sum_kernel<T>, dim3(unsigned((a.width + 63) / 64), 2), dim3(1024), 0, s, a,
                       a.rows > 0 ? shares : 0);
  return hip_status("layer norm gradient launch", err);
}

}  // namespace
}  // namespace prod

int launch_norm(int dtype, const NormArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::norm_t<prod::bf16>(args, s, err) : prod::norm_t<float>(args, s, err);
}

int64_t norm_partials(int64_t rows, int64_t) {
  const int64_t height = prod::band_height(rows);
  return std::max(prod::walkers(rows), (rows + height - 1) / height);
}

int launch_norm_backward(int dtype, const NormArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::norm_backward_t<prod::bf16>(args, s, err)
                           : prod::norm_backward_t<float>(args, s, err);
}

}  // namespace ccl
