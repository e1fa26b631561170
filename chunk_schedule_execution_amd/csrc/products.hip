// Products beside the collectives for gfx950: C = act(A B^T + bias) + residual, plain or
// grouped by expert with ragged sizes, for the forward pass and both gradients.
#include "product_tile.h"

namespace ccl {
namespace prod {
namespace {

int hip_status(const char* what, std::string* err) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return CCL_OK;
  *err = std::string(what) + ": " + hipGetErrorString(e);
  return CCL_ERR_HIP;
}

// ---- one 64 x 64 tile per workgroup -------------------------------------------------
// Four waves, each 32 x 32 by matrix instructions of 16 x 16. Elements are loaded one by
// one into LDS rows of 64 bytes along k (80 apart: rows 16 apart then lie on different
// banks), so any stride and alignment is right. A lane of the matrix instructions holds
// row (lane & 15) of both operands and the same k values of them: which ones is free as
// long as A and B agree, so each lane takes 16 consecutive bytes at (lane >> 4) * 16.
template <typename T, bool AByK, bool BByK>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs g, ProductMode mode, int tiles_n, int tiles_m) {
  constexpr int BM = 64, BN = 64, BK = 64 / int(sizeof(T)), LD = 80 / int(sizeof(T));
  constexpr int PER = BM * BK / 256;  // elements per thread and operand
  __shared__ __attribute__((aligned(16))) T sa[BM * LD];
  __shared__ __attribute__((aligned(16))) T sb[BN * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const T* A = static_cast<const T*>(g.a);
  const T* B = static_cast<const T*>(g.b);
  T* C = static_cast<T*>(g.c);
  const int64_t tile = blockIdx.x;
  int group = 0;
  int64_t row = 0, m_end = g.m, col = 0, k_lo = 0, k_hi = g.k;
  if (mode == kRaggedK) {
    const int64_t per = int64_t(tiles_m) * tiles_n;
    group = int(tile / per);
    row = (tile % per) / tiles_n * BM;
    col = (tile % per) % tiles_n * BN;
    group_bounds(g.offsets, g.k, group, k_lo, k_hi);
    C += group * g.c_stride;
  } else {
    const RowTile t = find_tile(g.offsets, g.groups, g.m, BM, int(tile / tiles_n), true);
    if (t.group < 0) return;
    group = t.group;
    row = t.row;
    m_end = t.end;
    col = tile % tiles_n * BN;
    if (group == g.groups) k_hi = 0;  // rows of no group: zeros
    else B += group * g.b_stride;
  }
  const bool nothing = mode == kRaggedM && group == g.groups;
  f32x4 acc[2][2] = {};
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += BK) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (AByK) {
        const int kk = (i * 256 + tid) / BM, r = (i * 256 + tid) % BM;
        const bool in = k0 + kk < k_hi && row + r < m_end;
        sa[r * LD + kk] = in ? A[(k0 + kk) * g.lda + row + r] : T(0.0f);
      } else {
        const int kk = (i * 256 + tid) % BK, r = (i * 256 + tid) / BK;
        const bool in = k0 + kk < k_hi && row + r < m_end;
        sa[r * LD + kk] = in ? A[(row + r) * g.lda + k0 + kk] : T(0.0f);
      }
      if (BByK) {
        const int kk = (i * 256 + tid) / BN, r = (i * 256 + tid) % BN;
        const bool in = k0 + kk < k_hi && col + r < g.n;
        sb[r * LD + kk] = in ? B[(k0 + kk) * g.ldb + col + r] : T(0.0f);
      } else {
        const int kk = (i * 256 + tid) % BK, r = (i * 256 + tid) / BK;
        const bool in = k0 + kk < k_hi && col + r < g.n;
        sb[r * LD + kk] = in ? B[(col + r) * g.ldb + k0 + kk] : T(0.0f);
      }
    }
    __syncthreads();
    constexpr int V = 16 / int(sizeof(T));
    const int at = (lane & 15) * LD + (lane >> 4) * V;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // first operand: columns of C, so that a lane ends up with 4 consecutive columns
        if constexpr (sizeof(T) == 2) {
          const bf16x8 x = *reinterpret_cast<const bf16x8*>(&sb[(wn + j * 16) * LD + at]);
          const bf16x8 y = *reinterpret_cast<const bf16x8*>(&sa[(wm + i * 16) * LD + at]);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc[i][j], 0, 0, 0);
        } else {
          const f32x4 x = *reinterpret_cast<const f32x4*>(&sb[(wn + j * 16) * LD + at]);
          const f32x4 y = *reinterpret_cast<const f32x4*>(&sa[(wm + i * 16) * LD + at]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[q], y[q], acc[i][j], 0, 0, 0);
        }
      }
    __syncthreads();
  }
  const T* bias = g.bias && !nothing ? static_cast<const T*>(g.bias) + group * g.bias_stride : nullptr;
  const T* residual = static_cast<const T*>(g.residual);
  T* preact = static_cast<T*>(g.preact);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t r = row + wm + i * 16 + (lane & 15);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t c = col + wn + j * 16 + (lane >> 4) * 4 + q;
        if (r >= m_end || c >= g.n) continue;
        float z = acc[i][j][q];
        if (bias) z += widen(bias[c]);
        if (preact) preact[r * g.ldp + c] = narrow<T>(z);
        float v = nothing ? 0.0f : act_value(z, g.act);
        if (residual) v += widen(residual[r * g.ldr + c]);
        C[r * g.ldc + c] = narrow<T>(v);
      }
    }
}

template <typename T>
int launch_any(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, hipStream_t s, std::string* err) {
  const int64_t tiles_n = (g.n + 63) / 64, tiles_m = (g.m + 63) / 64;
  // kRaggedM: every group and the rest may end in a tile of their own
  const int64_t grid = mode == kRaggedK ? g.groups * tiles_m * tiles_n
                       : mode == kRaggedM ? (tiles_m + g.groups) * tiles_n : tiles_m * tiles_n;
  if (grid > 0x7fffffff) {
    *err = "product: more than 2^31 tiles";
    return CCL_ERR_INVALID_ARGUMENT;
  }
  if (grid == 0) return CCL_OK;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(256), 0, s, g, mode, int(tiles_n), int(tiles_m));
  };
  if (a_by_k && b_by_k) go(product_any_kernel<T, true, true>);
  else if (b_by_k) go(product_any_kernel<T, false, true>);
  else go(product_any_kernel<T, false, false>);
  return hip_status("product launch", err);
}

// ---- slope and bias gradient ---------------------------------------------------------
constexpr int kSlopeRows = 64;

template <typename T>
__global__ __launch_bounds__(256) void slope_kernel(SlopeArgs g) {
  const RowTile t = find_tile(g.offsets, g.groups, g.rows, kSlopeRows, blockIdx.x, true);
  const int64_t c = int64_t(blockIdx.y) * 256 + threadIdx.x;
  if (t.group < 0 || c >= g.n) return;
  const T* dout = static_cast<const T*>(g.dout);
  const T* preact = static_cast<const T*>(g.preact);
  T* dz = static_cast<T*>(g.dz);
  float sum = 0.0f;
  const bool nothing = g.offsets && t.group == g.groups;
  const int64_t end = min(t.end, t.row + kSlopeRows);
  for (int64_t r = t.row; r < end; ++r) {
    float v = nothing ? 0.0f : widen(dout[r * g.ldo + c]);
    if (!nothing && g.act != CCL_ACT_NONE) v *= act_slope(widen(preact[r * g.ldp + c]), g.act);
    if (dz) dz[r * g.ldz + c] = narrow<T>(v);
    sum += v;
  }
  if (g.dbias && !nothing) g.partial[int64_t(t.index) * g.n + c] = sum;
}

// dbias[group][c]: the partial sums of the group's tiles, in the order of the tiles.
template <typename T>
__global__ __launch_bounds__(256) void bias_sum_kernel(SlopeArgs g) {
  const int group = blockIdx.y;
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  // first tile of the group: tiles of all earlier groups
  int64_t tile = 0, lo = 0, hi = g.rows;
  if (g.offsets) {
    hi = 0;
    for (int e = 0; e <= group; ++e) {
      tile += (hi - lo + kSlopeRows - 1) / kSlopeRows;
      lo = hi;
      hi = max(lo, int64_t(max(0, min(g.offsets[e + 1], int(g.rows)))));
    }
  }
  if (c >= g.n) return;
  const int64_t last = tile + (hi - lo + kSlopeRows - 1) / kSlopeRows;
  float sum = 0.0f;
  for (; tile < last; ++tile) sum += g.partial[tile * g.n + c];
  static_cast<T*>(g.dbias)[int64_t(group) * g.n + c] = narrow<T>(sum);
}

template <typename T>
int slope_t(const SlopeArgs& g, hipStream_t s, std::string* err) {
  const unsigned cols = unsigned((g.n + 255) / 256);
  if (g.rows > 0 && (g.dz || g.dbias))
    hipLaunchKernelGGL(slope_kernel<T>, dim3(unsigned(slope_tiles(g.rows, g.offsets ? g.groups : 0)), cols), dim3(256),
                       0, s, g);
  if (g.dbias) hipLaunchKernelGGL(bias_sum_kernel<T>, dim3(cols, unsigned(g.groups)), dim3(256), 0, s, g);
  return hip_status("bias gradient launch", err);
}

__global__ __launch_bounds__(256) void fill_zero_kernel(unsigned char* p, int64_t bytes) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < bytes; i += int64_t(gridDim.x) * 256) p[i] = 0;
}

// Whether an operand's stored rows are whole 16-byte vectors.
bool on_grid(int dtype, bool by_k, const void* p, int64_t ld, int64_t rows, int64_t k) {
  const int64_t v = dtype == CCL_BF16 ? 8 : 4;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % v == 0 && (by_k ? rows : k) % v == 0;
}

}  // namespace
}  // namespace prod

int64_t slope_tiles(int64_t rows, int groups) { return (rows + prod::kSlopeRows - 1) / prod::kSlopeRows + groups; }

int launch_slope(int dtype, const SlopeArgs& args, void* stream, std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == CCL_BF16 ? prod::slope_t<prod::bf16>(args, s, err) : prod::slope_t<float>(args, s, err);
}

int launch_product(int dtype, bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& args, void* stream,
                   std::string* err) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (prod::on_grid(dtype, a_by_k, args.a, args.lda, args.m, args.k) &&
      prod::on_grid(dtype, b_by_k, args.b, args.ldb, args.n, args.k))
    return dtype == CCL_BF16 ? prod::launch_tile_bf16(a_by_k, b_by_k, mode, args, s, err)
                             : prod::launch_tile_f32(a_by_k, b_by_k, mode, args, s, err);
  return dtype == CCL_BF16 ? prod::launch_any<prod::bf16>(a_by_k, b_by_k, mode, args, s, err)
                           : prod::launch_any<float>(a_by_k, b_by_k, mode, args, s, err);
}

int launch_fill_zero(void* p, int64_t bytes, void* stream, std::string* err) {
  if (bytes <= 0) return CCL_OK;
  const unsigned grid = unsigned(std::min<int64_t>(1024, (bytes + 255) / 256));
  hipLaunchKernelGGL(prod::fill_zero_kernel, dim3(grid), dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                     static_cast<unsigned char*>(p), bytes);
  return prod::hip_status("fill launch", err);
}

}  // namespace ccl
