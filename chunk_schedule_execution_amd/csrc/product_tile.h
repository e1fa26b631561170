// The tiled product kernel for gfx950: operands whose rows lie on the 16-byte grid.
#pragma once

#include <algorithm>

#include "products_device.h"

namespace ccl {
namespace prod {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

// ---- operand tiles in LDS -------------------------------------------------------------
// A step of the summed dimension is 128 bytes of a row: 64 bf16 or 32 fp32 values. Tiles
// come straight from memory by 16-byte buffer loads into LDS (no registers in between),
// whose destination is lane-linear, so the layouts below permute the source addresses.
//
// Stored by rows (ByK false): tile [R rows][8 chunks of 16 bytes], chunk c of row r at
// position c ^ (r & 7). A matrix instruction's lanes read chunk c of 16 neighbouring
// rows: any 8 of them hit 8 different positions, all 128 bytes of the banks.
//
// Stored by k (ByK true): tile [step rows of k][R values]. bf16: the transposing read
// takes from 16 lanes 4 rows of k by 16 values and hands each lane 4 k values of its
// column; rows are R * 2 bytes apart, so the 32-byte windows are permuted by (k & 3).
// fp32: lanes read single values of 4 rows four apart; 64-byte windows permuted by
// (k >> 2) & 3.
//
// Which k values a lane of a matrix instruction holds is free as long as both operands
// agree: lane group g = lane >> 4 takes the step's bytes [64 h + 16 g, 64 h + 16 g + 16)
// of half h, for both layouts.
template <typename T, bool ByK, int R, int Threads>
struct OperandTile {
  static constexpr int kSize = sizeof(T), kStep = 128 / kSize, kVec = 16 / kSize;
  static constexpr int kLoads = R * 8 / Threads;
  static constexpr int kChunks = ByK ? R / kVec : 8;  // per stored row
  static_assert(kLoads * Threads == R * 8 && kLoads >= 1, "whole loads");

  // All byte counts within a tile are below 2^32: a stride is at most 2^22 values, so 256
  // rows of bf16 or 128 of fp32 span 2^31 bytes.
  const char* base;   // first value of the tile at the current step
  unsigned records;   // readable bytes from base (by rows), or in the last row of k (by k)
  unsigned ld_bytes;
  int voff[kLoads];
  int kc;  // by rows: first k value of this lane's chunk

  // What does not depend on the tile.
  __device__ inline void init(int64_t ld) {
    const int tid = threadIdx.x;
    ld_bytes = unsigned(ld * kSize);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = i * Threads + tid, r = q / kChunks;  // stored row
      const int c = (q % kChunks) ^ (ByK ? swizzle(r) : r & 7);
      voff[i] = int(unsigned(r) * ld_bytes) + c * 16;
      kc = c * kVec;  // by rows the same for every i: rows differ by multiples of 8
    }
  }

  // row: first row (or column) of the tile, end: one past the last; k_lo, k_hi: the summed
  // range. The vector around the last value is read whole.
  __device__ inline void place(const T* p, int row, int end, int k_lo, int k_hi) {
    if constexpr (ByK) {
      base = reinterpret_cast<const char*>(p + row) + int64_t(k_lo) * ld_bytes;
      records = unsigned(min(R, end - row) + kVec - 1) / kVec * 16;  // whole vectors
    } else {
      base = reinterpret_cast<const char*>(p + k_lo) + int64_t(row) * ld_bytes;
      records = unsigned(min(R, end - row) - 1) * ld_bytes + unsigned(k_hi - k_lo + kVec - 1) / kVec * 16;
    }
    base = uniform(base);
    records = uniform(int(records));
  }

  static __device__ inline int swizzle(int k) { return kSize == 2 ? (k & 3) << 1 : ((k >> 2) & 3) << 2; }

  // Starts the loads of the step whose `left` summed values remain, into `lds`, and moves
  // on to the next step. Reads out of range (all of them when none remain) give zeros.
  __device__ inline void load(T* lds, int left) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned to = unsigned((uintptr_t)(lds_ptr)lds) + wave * 1024;
    asm volatile("" : "+s"(to));
    const unsigned rest = ByK ? unsigned(min(kStep, left) - 1) * ld_bytes + records : records;
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, uniform(left > 0 ? int(rest) : 0), 0x00020000);
    // by rows, the last step: chunks behind the row's end would be the next row's values
    const bool out = !ByK && left < kStep && kc >= left;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(uintptr_t)(to + i * Threads * 16), 16, out ? -1 : voff[i], 0, 0, 0);
    base += ByK ? int64_t(ld_bytes) * kStep : 128;
    if (!ByK) records -= 128;
  }
};

// A wave's reads of one operand: F fragments of 16 rows from row r0 of the tile.
template <typename T, bool ByK, int R, int F>
struct FragmentReader {
  static constexpr int kSize = sizeof(T);
  static constexpr int kOffsets = ByK ? (F < 4 ? F : 4) : 2;
  static_assert(!ByK || F <= 4 || F % 4 == 0, "whole windows");
  int off[kOffsets];

  __device__ inline void init(int r0) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    if constexpr (!ByK) {
#pragma unroll
      for (int h = 0; h < 2; ++h) off[h] = (r0 + (lane & 15)) * 128 + (((h * 4 + g) ^ (lane & 7)) * 16);
    } else if constexpr (kSize == 2) {
      const int j = (lane >> 2) & 3;  // row of k within the lane group's 4
#pragma unroll
      for (int i = 0; i < kOffsets; ++i) {
        const int chunk = ((r0 / 8 + 2 * i) ^ (j << 1)) + ((lane & 3) >> 1);
        off[i] = (g * 8 + j) * (R * 2) + chunk * 16 + (lane & 1) * 8;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kOffsets; ++i) {
        const int chunk = ((r0 / 4 + 4 * i) ^ (g << 2)) + ((lane & 15) >> 2);
        off[i] = g * 4 * (R * 4) + chunk * 16 + (lane & 3) * 4;
      }
    }
  }

  // Half h of fragment i: 16 bytes of k values per lane.
  __device__ inline auto read(const T* lds, int i, int h) const {
    const char* p = reinterpret_cast<const char*>(lds);
    if constexpr (!ByK) {
      typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
      return *reinterpret_cast<const vec*>(p + off[h] + i * 2048);
    } else if constexpr (kSize == 2) {
      const char* at = p + off[i & 3] + (i >> 2) * 128 + h * 32 * (R * 2);
      typedef __attribute__((address_space(3))) s16x4* tr_ptr;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(at + 4 * (R * 2)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(bf16x8, v);
    } else {
      const char* at = p + off[i & 3] + (i >> 2) * 256 + h * 16 * (R * 4);
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const float*>(at + q * (R * 4));
      return v;
    }
  }
};

// All waves' reads of LDS before this point are done and their loads into LDS have arrived.
__device__ inline void steps_arrived() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Which tile a workgroup computes. Workgroups go round the 8 XCDs, each with an L2 of its
// own, so XCD x takes the x-th eighth of the tiles; within it kBands bands (rows of tiles)
// are walked together, column by column, so that the 32 workgroups that run there at a time
// share, with 8 bands, 8 row and 4 column tiles: 3 % of 8192^3 (bf16, 760 us) against the
// order of the columns. From each such set to the next the bands turn by one, or a workgroup
// would meet the same band again and again, and the last bands of groups are shorter than
// others: 16384 rows over 32 groups, 2048 x 4096, take 340 to 353 us for 346 to 361.
template <int kBands>
__device__ inline void place_tile(unsigned id, unsigned tiles, int tiles_n, int& band, int& column) {
  constexpr unsigned kXcds = 8;
  const unsigned x = id % kXcds, whole = tiles / kXcds, rest = tiles % kXcds;
  const int l = int(x * whole + min(x, rest) + id / kXcds);
  // quotients are computed in vector registers: uniform() brings them back
  const int slab = uniform(l / (kBands * tiles_n)), in = l - slab * kBands * tiles_n;
  const int bands = min(kBands, int(tiles) / tiles_n - slab * kBands);
  column = uniform(in / bands);
  const int turned = in - column * bands + column / (32 / kBands);
  band = slab * kBands + turned - uniform(turned / bands) * bands;
}

// ---- the kernel ---------------------------------------------------------------------------
// What a workgroup computes next; all of it uniform.
struct TileJob {
  int group = 0;         // `groups`: rows of no group
  bool there = false;    // false: no such tile
  int row = 0, m_end = 0, col = 0, k_lo = 0, k_hi = 0;  // all below 2^31
};

template <int BM, int BN, int Step>
__device__ inline TileJob find_job(const ProductArgs& g, ProductMode mode, unsigned id, unsigned tiles, int tiles_m,
                                   int tiles_n) {
  TileJob j;
  if (id >= tiles) return j;
  int band, column;
  int64_t row = 0, m_end = g.m, k_lo = 0, k_hi = g.k;
  if (mode == kRaggedK) {
    // Group after group, each spread over all XCDs: their lengths differ, and with them the
    // work. 16 groups of 512 rows +- 30 %, 2048 x 2048, take 104 us; 130 with two whole groups
    // per XCD, though now every L2 reads the groups' rows. 4 bands by 2 columns of a group's
    // 64 tiles read less of them than 8 by 1: 3 us.
    const unsigned per = unsigned(tiles_m) * unsigned(tiles_n);
    j.group = uniform(int(id / per));
    place_tile<4>(id - unsigned(j.group) * per, per, tiles_n, band, column);
    row = int64_t(band) * BM;
    group_bounds(g.offsets, g.k, j.group, k_lo, k_hi);
  } else {
    place_tile<8>(id, tiles, tiles_n, band, column);
    const RowTile t = find_tile(g.offsets, g.groups, g.m, BM, band);
    j.group = uniform(t.group);
    row = t.row;
    m_end = t.end;
    if (mode == kRaggedM && j.group == g.groups) k_hi = 0;  // rows of no group: zeros
  }
  j.there = true;
  j.col = column * BN;
  j.row = uniform(int(row));
  j.m_end = uniform(int(m_end));
  j.k_lo = uniform(int(k_lo));
  j.k_hi = uniform(int(k_hi));
  if (gridDim.y > 1) {  // this workgroup's share of the summed dimension, in whole steps
    // The steps end up to Step - 1 values past the range, which may be past 31 bits; times
    // the 16 splits there are at most, their number stays below 2^31.
    const unsigned range = max(0, j.k_hi - j.k_lo), steps = (range + Step - 1) / Step;
    const unsigned lo = uniform(int(steps * blockIdx.y / gridDim.y)) * Step;
    const unsigned hi = uniform(int(steps * (blockIdx.y + 1) / gridDim.y)) * Step;
    j.k_hi = j.k_lo + int(min(range, hi));
    j.k_lo += int(min(range, lo));
  }
  return j;
}

// The usual end of a tile: bias, activation, residual and stores, or the splits' sums.
struct Results {
  static constexpr bool kTakes = false, kAdds = false, kPlainStores = false;
  template <int FM>
  struct Rows {
    __device__ inline void load(const Results&, const ProductArgs&, const TileJob&, int) {}
  };
  template <int FM, int FN>
  __device__ inline void change(f32x4 (&)[FM][FN], const Rows<FM>&, const ProductArgs&, const TileJob&, int) const {}
  __device__ inline int64_t columns(const ProductArgs& g) const { return g.n; }
};
// Sums that are added onto those that an earlier part of the summed dimension left in
// `partial`.
struct AddedSums : Results {
  static constexpr bool kAdds = true;
};

// BM x BN values per tile, WM x WN waves, each (BM / WM) x (BN / WN) by matrix instructions
// of 16 x 16. Two LDS buffers, one barrier per step. A workgroup computes tile after tile:
// the loads of a tile's first two steps start before the results of the tile before it are
// written, so they arrive while bias, activation and stores run.
//
// In bf16 8192^3 takes 760 us, 1.45 PFLOP/s (the library 690), with the matrix pipes busy 60 %
// of the cycles at a clock that power holds near 1.9 GHz. A step of a 256 x 256 tile is 2048
// cycles of products and takes about 2800: what is lost goes to the barrier, where eight
// waves meet. A tile's start and end cost 10 us, 4.5 of them arithmetic of the epilogue (15
// with gelu and the argument kept), which nothing overlaps while one workgroup fills the
// unit's LDS. Lost against this: matrix instructions of 32 x 32 (810 us), two workgroups of
// 256 x 128 per unit on half steps (as much matrix work, but 1.5 times the loads: 990 us),
// four waves of 128 x 128 (registers spill).
//
// What becomes of a tile is End's: it may read what it needs of the tile's rows (`rows`),
// change the sums in registers, or take them and leave no results.
template <typename T, bool AByK, bool BByK, int BM, int BN, int WM, int WN, class End>
__device__ inline void product_tiles(const ProductArgs& g, const End& ending, ProductMode mode, int tiles_m, int tiles_n,
                                     unsigned all) {
  constexpr int Threads = WM * WN * 64, FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int kStep = 128 / int(sizeof(T));  // also the values per row of a stored tile
  constexpr int WTN = BN / WN;                 // columns of a wave
  __shared__ __attribute__((aligned(1024))) T a0[BM * kStep];
  __shared__ __attribute__((aligned(1024))) T b0[BN * kStep];
  __shared__ __attribute__((aligned(1024))) T a1[BM * kStep];
  __shared__ __attribute__((aligned(1024))) T b1[BN * kStep];
  __shared__ __attribute__((aligned(1024))) float stages[WM * WN * 16 * WTN];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN * (BM / WM), wn = wave % WN * WTN;
  // groups leave some of the tiles unused: only those that exist are spread over the XCDs
  const unsigned tiles = mode == kRaggedM ? unsigned(count_tiles(g.offsets, g.groups, g.m, BM)) * tiles_n : all;

  OperandTile<T, AByK, BM, Threads> ta;
  OperandTile<T, BByK, BN, Threads> tb;
  FragmentReader<T, AByK, BM, FM> ra;
  FragmentReader<T, BByK, BN, FN> rb;
  ta.init(g.lda);
  tb.init(g.ldb);
  ra.init(wm);
  rb.init(wn);
  auto begin = [&](const TileJob& j) {
    const int left = j.k_hi - j.k_lo;
    if (!j.there || left <= 0) return;
    const T* B = static_cast<const T*>(g.b) + (mode == kRaggedM ? j.group * g.b_stride : 0);
    ta.place(static_cast<const T*>(g.a), j.row, j.m_end, j.k_lo, j.k_hi);
    tb.place(B, j.col, int(g.n), j.k_lo, j.k_hi);
    ta.load(a0, left);
    tb.load(b0, left);
    ta.load(a1, left - kStep);
    tb.load(b1, left - kStep);
  };

  unsigned id = blockIdx.x;
  TileJob job = find_job<BM, BN, kStep>(g, mode, id, tiles, tiles_m, tiles_n);
  begin(job);
  while (job.there) {
    f32x4 acc[FM][FN] = {};
    int left = job.k_hi - job.k_lo;  // of the step being multiplied
    if (left > 0) {
      // A step is 2 FM rows of fragments (both halves), multiplied one after another. Reads
      // run Ahead rows ahead: a buffer's last read is done that many rows before its last
      // products, and there the step's only barrier stands. Behind it the next buffer is
      // read and the loads of the step after next may overwrite this one, with a whole step
      // to arrive; the rows still to be multiplied cover the barrier and the first reads.
      // Loads behind the end give zeros and nothing multiplies them, so no step branches.
      typedef decltype(ra.read(a0, 0, 0)) vec;
      constexpr int Rows = 2 * FM, Ahead = FM < 4 ? FM : 4, Ring = 2 * Ahead;
      static_assert(Rows % Ring == 0, "a ring of fragments");
      vec fa[Ring], fb[2][FN];
      auto read_a = [&](const T* la, int r) { fa[r % Ring] = ra.read(la, r % FM, r / FM % 2); };
      auto read_b = [&](const T* lb, int h) {
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[h][j] = rb.read(lb, j, h);
      };
      auto products = [&](int r) {
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[r % FM][j] = multiply(fb[r / FM][j], fa[r % Ring], acc[r % FM][j]);
      };
      steps_arrived();
      read_b(b0, 0);
#pragma unroll
      for (int r = 0; r < Ahead; ++r) read_a(a0, r);
      auto step = [&](T* la, T* lb, const T* na, const T* nb) {
        // the scheduling barriers keep reads from sinking back to their uses
#pragma unroll
        for (int r = 0; r < Rows - Ahead; ++r) {
          if (r == FM - Ahead) read_b(lb, 1);
          read_a(la, r + Ahead);
          products(r);
          __builtin_amdgcn_sched_barrier(0);
        }
        steps_arrived();
        read_b(nb, 0);
#pragma unroll
        for (int r = 0; r < Ahead; ++r) {
          read_a(na, r);
          products(Rows - Ahead + r);
          if (r == 0) ta.load(la, left - 2 * kStep);
          if (r == 1) tb.load(lb, left - 2 * kStep);
          __builtin_amdgcn_sched_barrier(0);
        }
        left -= kStep;
      };
      while (true) {
        step(a0, b0, a1, b1);
        if (left <= 0) break;
        step(a1, b1, a0, b0);
        if (left <= 0) break;
      }
      __builtin_amdgcn_s_waitcnt(0x0F70);  // this wave's loads behind the end, before its next ones
    }
    id += gridDim.x;
    const TileJob next = find_job<BM, BN, kStep>(g, mode, id, tiles, tiles_m, tiles_n);

    // Results go through LDS, 16 rows of a wave at a time and to itself alone, so that rows
    // are read and written in 16-byte vectors.
    constexpr int kChunks = WTN / 4;  // 16-byte chunks of fp32 per row
    constexpr int kLanesPerRow = WTN / 8, kRowsPerPass = 64 / kLanesPerRow;
    const int lane = here(tid & 63);
    float* const stage = stages + wave * (16 * WTN);
    const bool nothing = mode == kRaggedM && job.group == g.groups;
    T* const C = static_cast<T*>(g.c) + (mode == kRaggedK ? job.group * g.c_stride : 0);
    const int64_t c = job.col + wn + (lane % kLanesPerRow) * 8;
    const int n = int(min(int64_t(8), ending.columns(g) - c));
    // loads the bias: before the next tile's loads
    Finish<T> finish(g, C, int64_t(job.row) + wm + lane / kLanesPerRow, kRowsPerPass, c, n, job.group, nothing);
    typename End::template Rows<FM> rows;
    rows.load(ending, g, job, wm);
    // the last reads of this tile's values were before the last barrier, so every wave may
    // load the next tile's
    begin(next);
    if constexpr (End::kTakes) {
      ending.take(acc, rows, g, job, wm, wn);
      job = next;
      continue;
    }
    ending.change(acc, rows, g, job, wn);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int r = lane & 15, chunk = j * 4 + (lane >> 4);
        *reinterpret_cast<f32x4*>(stage + r * WTN + ((chunk ^ r) % kChunks) * 4) = acc[i][j];
      }
      __builtin_amdgcn_wave_barrier();
#pragma nounroll
      for (int r = lane / kLanesPerRow; r < 16; r += kRowsPerPass, finish.next()) {
        // counted from the tile's first row: a last tile may end past 31 bits
        const int in = wm + i * 16 + r;
        if (in >= job.m_end - job.row || n <= 0) continue;
        const int chunk = (lane % kLanesPerRow) * 2;
        float v[8];
        *reinterpret_cast<f32x4*>(v) = *reinterpret_cast<const f32x4*>(stage + r * WTN + ((chunk ^ r) % kChunks) * 4);
        *reinterpret_cast<f32x4*>(v + 4) =
            *reinterpret_cast<const f32x4*>(stage + r * WTN + (((chunk + 1) ^ r) % kChunks) * 4);
        if constexpr (End::kAdds) {
          float* const sums = partial_at(g, blockIdx.y, int64_t(job.row) + in, c);
          float before[8];
          load8(sums, true, n, before);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] += before[q];
          store8(sums, true, n, v);
        } else if (g.partial) {
          store8(partial_at(g, blockIdx.y, int64_t(job.row) + in, c), true, n, v);
        } else if constexpr (End::kPlainStores) {
          store8<false>(finish.out, finish.vec_c, n, v);
        } else {
          finish.row(v);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    job = next;
  }
}

// Two waves per SIMD: half of the registers each.
template <typename T, bool AByK, bool BByK, int BM, int BN, int WM, int WN, class End>
__global__ __launch_bounds__(WM* WN * 64, 2) void product_tile_kernel(ProductArgs g, End ending, ProductMode mode,
                                                                      int tiles_m, int tiles_n, unsigned tiles) {
  product_tiles<T, AByK, BByK, BM, BN, WM, WN>(g, ending, mode, tiles_m, tiles_n, tiles);
}

template <typename T, bool AByK, bool BByK, int BM, int BN, int WM, int WN, class End>
int launch_tile_as(ProductMode mode, const ProductArgs& g, const End& ending, int splits, hipStream_t s,
                   std::string* err) {
  constexpr int kUnits = 256, kXcds = 8;
  constexpr int kResident = 163840 / ((BM + BN) * 256 + WM * BN * 64);  // by LDS
  const int64_t tiles_n = (g.n + BN - 1) / BN, tiles_m = (g.m + BM - 1) / BM;
  const int64_t tiles = mode == kRaggedK ? g.groups * tiles_m * tiles_n
                        : mode == kRaggedM ? (tiles_m + g.groups) * tiles_n : tiles_m * tiles_n;
  if (tiles > 0x7fffffff) {
    *err = "product: more than 2^31 tiles";
    return CCL_ERR_INVALID_ARGUMENT;
  }
  if (tiles == 0) return CCL_OK;
  // as many workgroups as are resident at a time, a multiple of the XCDs
  const int64_t grid = std::min<int64_t>(tiles, std::max<int64_t>(kXcds, kUnits * kResident / splits / kXcds * kXcds));
  hipLaunchKernelGGL((product_tile_kernel<T, AByK, BByK, BM, BN, WM, WN, End>), dim3(unsigned(grid), splits),
                     dim3(WM * WN * 64), 0, s, g, ending, mode, int(tiles_m), int(tiles_n), unsigned(tiles));
  return hip_status("product launch", err);
}

template <typename T, int BM, int BN, int WM, int WN>
int launch_tile(bool a_by_k, bool b_by_k, ProductMode mode, const ProductArgs& g, int splits, hipStream_t s,
                std::string* err) {
  if (a_by_k && b_by_k) return launch_tile_as<T, true, true, BM, BN, WM, WN>(mode, g, Results(), splits, s, err);
  if (b_by_k) return launch_tile_as<T, false, true, BM, BN, WM, WN>(mode, g, Results(), splits, s, err);
  return launch_tile_as<T, false, false, BM, BN, WM, WN>(mode, g, Results(), splits, s, err);
}

}  // namespace

}  // namespace prod
}  // namespace ccl
