// Layer norm with the residual's addition for gfx950, and its gradients. Memory bounds both:
// a row is read once and stays in registers for its mean, its variance and its result, and
// workgroups walk rows, so that the next row's loads run beside this one's sums.
#include <algorithm>
#include <type_traits>

#include "lanes.h"
#include "layers.h"
#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

// 16 bytes of a row wherever they lie: loads and stores of vectors need no alignment beyond
// the element's, and a row's last vector may be cut short (`left` values to its end). Rows are
// read and written once: around the caches.
template <typename T>
struct Pack {
  static constexpr int kValues = 16 / int(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(kValues), aligned(sizeof(T))));
  vec v;

  __device__ inline void zero() { v = vec(T(0.0f)); }
  // The same values, from which nothing is kept that was computed before.
  __device__ inline void renew() {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    u32x4 bits = __builtin_bit_cast(u32x4, v);
    asm volatile("" : "+v"(bits));
    v = __builtin_bit_cast(vec, bits);
  }
  template <bool Once = true>
  __device__ inline void load(const T* p, int left) {
    if (left >= kValues) {
      if constexpr (Once) v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
      else v = *reinterpret_cast<const vec*>(p);
    } else {
#pragma unroll
      for (int q = 0; q < kValues; ++q) v[q] = q < left ? p[q] : T(0.0f);
    }
  }
  template <bool Once = true>
  __device__ inline void store(T* p, int left) const {
    if (left >= kValues) {
      if constexpr (Once) __builtin_nontemporal_store(v, reinterpret_cast<vec*>(p));
      else *reinterpret_cast<vec*>(p) = v;
    } else {
#pragma unroll
      for (int q = 0; q < kValues; ++q)
        if (q < left) p[q] = v[q];
    }
  }
};

// All waves' LDS accesses before this point are done; loads from memory stay in flight.
__device__ inline void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ inline int64_t flat_block() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

// How the threads share out rows of packs: R threads to a row, `Held` packs each, and as many
// rows side by side as a workgroup of 256 holds. One wave to a row needs no barrier.
template <int R>
struct Sharing {
  static constexpr int kThreads = R < 256 ? 256 : R, kRows = kThreads / R, kWaves = R / 64;
};

// The sum of v over the R threads of a row. parts: LDS that is not used again before the
// workgroup's next barrier but one.
template <int R>
__device__ inline float row_sum(float v, float* parts) {
  v = over_sum<64>(v);
  if constexpr (R > 64) {
    if (threadIdx.x % 64 == 0) parts[threadIdx.x / 64] = v;
    lds_barrier();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < R / 64; ++i) v += parts[i];
  }
  return v;
}

// Of two values with one barrier.
template <int R>
__device__ inline void row_sums(float& v, float& w, float (*parts)[Sharing<R>::kWaves]) {
  v = over_sum<64>(v);
  w = over_sum<64>(w);
  if constexpr (R > 64) {
    if (threadIdx.x % 64 == 0) {
      parts[0][threadIdx.x / 64] = v;
      parts[1][threadIdx.x / 64] = w;
    }
    lds_barrier();
    v = w = 0.0f;
#pragma unroll
    for (int i = 0; i < R / 64; ++i) {
      v += parts[0][i];
      w += parts[1][i];
    }
  }
}

// ---- forward -------------------------------------------------------------------------------
// The variance is the mean of squared differences from the mean, from registers: nothing
// cancels. 16384 x 4096 bf16 with residual and both outputs (537 MB): 95 us, 5.7 TB/s; 106 with
// a wave to each row and no walk. A copy of 1 GB reaches 5.1.
template <typename T, int Held, int R>
__global__ __launch_bounds__(Sharing<R>::kThreads) void norm_kernel(NormArgs a) {
  using P = Pack<T>;
  constexpr int V = P::kValues, Rows = Sharing<R>::kRows;
  __shared__ float parts[2][2][Sharing<R>::kWaves];
  const int lane = threadIdx.x % R, width = int(a.width);
  P pw[Held], pb[Held], px[Held], pr[Held];
#pragma unroll
  for (int i = 0; i < Held; ++i) {
    const int c = (i * R + lane) * V;
    pw[i].zero();
    pb[i].zero();
    px[i].zero();
    pr[i].zero();
    if (a.weight) pw[i].template load<false>(static_cast<const T*>(a.weight) + c, width - c);
    if (a.bias) pb[i].template load<false>(static_cast<const T*>(a.bias) + c, width - c);
  }
  auto load = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* r = static_cast<const T*>(a.residual) + row * a.ld_residual;
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      const int c = (i * R + lane) * V;
      px[i].load(x + c, width - c);
      if (a.residual) pr[i].load(r + c, width - c);
    }
  };
  const int64_t step = int64_t(gridDim.x) * Rows;
  int64_t row = int64_t(blockIdx.x) * Rows + threadIdx.x / R;
  int turn = 0;
  if (row < a.rows) load(row);
  for (; row < a.rows; row += step, turn ^= 1) {
    float h[Held][V], sum = 0.0f, squares = 0.0f;
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        h[i][q] = widen(px[i].v[q]);
        if (a.residual) h[i][q] += widen(pr[i].v[q]);
        sum += h[i][q];
      }
    if (row + step < a.rows) load(row + step);
    if (a.total) {
      T* total = static_cast<T*>(a.total) + row * a.ld_total;
#pragma unroll
      for (int i = 0; i < Held; ++i) {
        const int c = (i * R + lane) * V;
        P o;
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = narrow<T>(h[i][q]);
        o.store(total + c, width - c);
      }
    }
    const float mean = row_sum<R>(sum, parts[turn][0]) / float(width);
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        h[i][q] -= mean;
        squares += (i * R + lane) * V + q < width ? h[i][q] * h[i][q] : 0.0f;
      }
    const float rstd = 1.0f / sqrtf(row_sum<R>(squares, parts[turn][1]) / float(width) + a.eps);
    if (a.mean && lane == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.ld_out;
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      const int c = (i * R + lane) * V;
      P o;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        float v = h[i][q] * rstd;
        if (a.weight) v *= widen(pw[i].v[q]);
        if (a.bias) v += widen(pb[i].v[q]);
        o.v[q] = narrow<T>(v);
      }
      o.store(out + c, width - c);
    }
  }
}

// Rows that registers do not hold: read three times, the second and third time from the
// caches as far as they go, and nothing is written before the third, so that total and out may
// take the inputs' places. 1024 threads a row, 8 columns each at a time.
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
    if (total) store8(total + c, vec_t, n, h);
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
// dw = sum over the rows of dout y, db of dout. A thread keeps to its columns, whose share of dw
// and db stays in registers: one pass over the rows gives all three, and each workgroup leaves
// its share in `partial`. 16384 x 4096 bf16 with dtotal (537 MB): 90 to 94 us, 5.7 TB/s; 134
// without the next row's loads ahead.
template <typename T, int Held, int R>
__global__ __launch_bounds__(Sharing<R>::kThreads) void norm_backward_kernel(NormArgs a) {
  using P = Pack<T>;
  constexpr int V = P::kValues, Rows = Sharing<R>::kRows;
  constexpr bool Ahead = Held * V < 32;  // more values of three tensors twice do not fit the registers
  __shared__ float parts[2][2][Sharing<R>::kWaves];
  const int lane = threadIdx.x % R, width = int(a.width);
  float dw[Held][V] = {}, db[Held][V] = {};
  P pw[Held], px[Held], pd[Held], pt[Held];
#pragma unroll
  for (int i = 0; i < Held; ++i) {
    const int c = (i * R + lane) * V;
    pw[i].zero();
    px[i].zero();
    pd[i].zero();
    pt[i].zero();
    if (a.weight) pw[i].template load<false>(static_cast<const T*>(a.weight) + c, width - c);
  }
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* d = static_cast<const T*>(a.dout) + row * a.ld_out;
    const T* t = static_cast<const T*>(a.dtotal) + row * a.ld_dtotal;
    mean = a.mean[row];
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      const int c = (i * R + lane) * V;
      px[i].load(x + c, width - c);
      pd[i].load(d + c, width - c);
      if (a.dtotal) pt[i].load(t + c, width - c);
    }
  };
  const int64_t step = int64_t(gridDim.x) * Rows;
  int64_t row = int64_t(blockIdx.x) * Rows + threadIdx.x / R;
  int turn = 0;
  if (Ahead && row < a.rows) load(row);
  for (; row < a.rows; row += step, turn ^= 1) {
    if (!Ahead) load(row);
    P cx[Held], cd[Held], ct[Held];
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      cx[i] = px[i];
      cd[i] = pd[i];
      ct[i] = pt[i];
    }
    const float m = mean, r = rstd;
    if (Ahead && row + step < a.rows) load(row + step);
    // dout is 0 past the row's end, so nothing there reaches a sum
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float d = widen(cd[i].v[q]), y = (widen(cx[i].v[q]) - m) * r;
        dw[i][q] = fmaf(d, y, dw[i][q]);
        db[i][q] += d;
        const float g = a.weight ? d * widen(pw[i].v[q]) : d;
        sum += g;
        dot = fmaf(g, y, dot);
      }
    if (!a.dx) continue;  // the same for all
    row_sums<R>(sum, dot, parts[turn]);
    sum /= float(width);
    dot /= float(width);
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
#pragma unroll
    for (int i = 0; i < Held; ++i) {
      const int c = (i * R + lane) * V;
      if (Held * V >= 16) {  // y and g again rather than in registers, which they would overflow
        cx[i].renew();
        cd[i].renew();
      }
      P o;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float d = widen(cd[i].v[q]), y = (widen(cx[i].v[q]) - m) * r;
        const float g = a.weight ? d * widen(pw[i].v[q]) : d;
        float v = r * (g - sum - y * dot);
        if (a.dtotal) v += widen(ct[i].v[q]);
        o.v[q] = narrow<T>(v);
      }
      o.store(dx + c, width - c);
    }
  }
  if (!a.partial) return;
  float* to = a.partial + int64_t(blockIdx.x) * 2 * width;
  if constexpr (Rows > 1) {  // the rows side by side, in order
    __shared__ float sums[2][Rows - 1][Held * R * V];
    const int mine = threadIdx.x / R;
#pragma unroll
    for (int i = 0; i < Held; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q)
        if (mine) {
          sums[0][mine - 1][(i * V + q) * R + lane] = dw[i][q];
          sums[1][mine - 1][(i * V + q) * R + lane] = db[i][q];
        }
    __syncthreads();
    if (mine) return;
    for (int k = 0; k < Rows - 1; ++k)
#pragma unroll
      for (int i = 0; i < Held; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          dw[i][q] += sums[0][k][(i * V + q) * R + lane];
          db[i][q] += sums[1][k][(i * V + q) * R + lane];
        }
  }
#pragma unroll
  for (int i = 0; i < Held; ++i)
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const int c = (i * R + lane) * V + q;
      Pack<float> w, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w.v[j] = dw[i][q + j];
        b.v[j] = db[i][q + j];
      }
      w.template store<false>(to + c, width - c);  // read again at once
      b.template store<false>(to + width + c, width - c);
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
// Calls f with the threads to a row and the packs of each that hold a row of n packs; false
// where none do: there rows are read again instead (2048 x 16384 bf16 gradients, the widest in
// registers, 86 us; 1024 x 20000, read again, 66 for 0.6 times the bytes). A wave a row needs no
// barrier, but has all of the row's latency: only up to two packs a lane. Eight packs only in
// fp32, where they are as many values as four in bf16.
template <typename T, typename F>
bool by_width(int64_t n, F f) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, 512> most;
  if (n <= 64) f(integral_constant<int, 64>(), one);
  else if (n <= 128) f(integral_constant<int, 64>(), two);
  else if (n <= 256) f(integral_constant<int, 256>(), one);
  else if (n <= 512) f(integral_constant<int, 256>(), two);
  else if (n <= 1024) f(most, two);
  else if (n <= 2048) f(most, integral_constant<int, 4>());
  else if (sizeof(T) == 4 && n <= 4096) f(most, integral_constant<int, sizeof(T) == 4 ? 8 : 4>());
  else return false;
  return true;
}
template <typename T>
int64_t packs(int64_t width) {
  return (width * int64_t(sizeof(T)) + 15) / 16;
}
// Workgroups that walk `rows` rows, `side` of them side by side, at most `most`.
int64_t walkers(int64_t rows, int side, int64_t most) {
  return std::max<int64_t>(1, std::min<int64_t>(most, (rows + side - 1) / side));
}

template <typename T>
int norm_t(const NormArgs& a, hipStream_t s, std::string* err) {
  const bool held = by_width<T>(packs<T>(a.width), [&](auto threads, auto each) {
    constexpr int R = decltype(threads)::value, Held = decltype(each)::value;
    hipLaunchKernelGGL((norm_kernel<T, Held, R>),
                       dim3(unsigned(walkers(a.rows, Sharing<R>::kRows, 256 * 1024 / Sharing<R>::kThreads))),
                       dim3(Sharing<R>::kThreads), 0, s, a);
  });
  if (!held) hipLaunchKernelGGL(norm_long_kernel<T>, flat_grid(a.rows), dim3(1024), 0, s, a);
  return hip_status("layer norm launch", err);
}

// Workgroups of the gradients: as many as are resident (half of 512 threads: 4096 x 8192 bf16
// takes 64 us in 256 shares and 76 in 512), and each with four rows at least, or the shares of dw
// and db would be as much to write and add up as the rows (1111 x 4096 bf16: 19 us, 28 with a
// workgroup a row).
constexpr int64_t kMostShares = 512, kRowsEach = 4;
int64_t band_height(int64_t rows) { return std::max<int64_t>(64, (rows + kMostShares - 1) / kMostShares); }

template <typename T>
int norm_backward_t(const NormArgs& args, hipStream_t s, std::string* err) {
  NormArgs a = args;
  const bool sums = a.dweight || a.dbias;
  if (!sums) a.partial = nullptr;
  int64_t shares = 0;
  if (a.rows > 0) {
    const bool held = by_width<T>(packs<T>(a.width), [&](auto threads, auto each) {
      constexpr int R = decltype(threads)::value, Held = decltype(each)::value;
      shares = walkers((a.rows + kRowsEach - 1) / kRowsEach, Sharing<R>::kRows, kMostShares / (R > 256 ? 2 : 1));
      hipLaunchKernelGGL((norm_backward_kernel<T, Held, R>), dim3(unsigned(shares)), dim3(Sharing<R>::kThreads), 0, s, a);
    });
    if (!held) {
      if (a.dx) hipLaunchKernelGGL(norm_backward_long_kernel<T>, flat_grid(a.rows), dim3(1024), 0, s, a);
      const int64_t height = band_height(a.rows);
      shares = (a.rows + height - 1) / height;
      if (sums)
        hipLaunchKernelGGL(norm_columns_kernel<T>, dim3(unsigned(shares), unsigned((a.width + 255) / 256)), dim3(256), 0,
                           s, a, height);
    }
  }
  if (sums)
    hipLaunchKernelGGL(norm_sum_kernel<T>, dim3(unsigned((a.width + 63) / 64), 2), dim3(1024), 0, s, a, shares);
  return hip_status("layer norm gradient launch", err);
}

}  // namespace
}  // namespace prod

int launch_norm(int dtype, const NormArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::norm_t<prod::bf16>(args, s, err) : prod::norm_t<float>(args, s, err);
}

int64_t norm_partials(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(prod::kMostShares, rows)); }

int launch_norm_backward(int dtype, const NormArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::norm_backward_t<prod::bf16>(args, s, err)
                           : prod::norm_backward_t<float>(args, s, err);
}

}  // namespace ccl
