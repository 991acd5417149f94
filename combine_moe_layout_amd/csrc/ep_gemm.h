// ep_gemm.h -- what the matrix-product kernels of libep.so share: the problem
// description, the search for a workgroup's tile among ragged groups, loads
// from memory straight into LDS, and the epilogue's activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"
#include "ep_gemm_index.h"
#include "ep_internal.h"

namespace ep {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes that read as zero in every element type: what a load takes its
// data from where a tile reaches past the last element of a reduction.
static __device__ const uint4 g_zero16[1] = {};

// --------------------------------------------------------------------------
// LDS by address.  A workgroup's LDS is one array; kernels keep byte offsets.
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// A wave-wide load of 64 x 16 bytes from memory into LDS, without registers:
// lane l's 16 bytes go to lds + 16 l.  `lds` is the same in every lane.  The
// load is counted by vmcnt and the compiler does not know that it writes LDS:
// the reader waits with wait_loads<>() and a barrier, both of which order LDS
// accesses in the program.  (The builtin of this instruction makes the
// compiler wait for all loads in flight before every LDS read, which undoes
// the prefetch.)  One instruction must lie between writing m0 and its use.
__device__ __forceinline__ void load16_to_lds(const void* base, uint32_t byte_offset,
                                              uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(byte_offset),
               "s"(base), "s"(lds) : "m0");
}
__device__ __forceinline__ void load16_to_lds(const void* lane_address, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(lane_address),
               "s"(lds) : "m0");
}
// The same for 64 x 4 bytes.
__device__ __forceinline__ void load4_to_lds(const void* base, uint32_t byte_offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(byte_offset),
               "s"(base), "s"(lds) : "m0");
}

// Waits until at most N of this wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Every LDS access of this wave but the kYoung youngest has returned (they
// return in order), then all waves of the workgroup meet.
template <int kYoung = 0>
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" ::"n"(kYoung) : "memory");
}

// --------------------------------------------------------------------------
// Ragged groups (RowGroups in ep_gemm_index.h).
// --------------------------------------------------------------------------
__device__ __forceinline__ int32_t group_count(const RowGroups& g, int32_t e) {
  if (g.first == nullptr) return (int32_t)g.rows;
  if (g.capacity > 0) return min(max(g.count[e], 0), g.capacity);
  const int64_t lo = g.first[e], hi = g.first[e + 1];
  return (int32_t)(min(max(hi, (int64_t)0), g.rows) - min(max(lo, (int64_t)0), g.rows));
}
__device__ __forceinline__ int64_t group_first(const RowGroups& g, int32_t e) {
  if (g.first == nullptr) return 0;
  if (g.capacity > 0) return (int64_t)e * g.capacity;
  return min(max((int64_t)g.first[e], (int64_t)0), g.rows);
}

struct Tile {
  int32_t e;       // group
  int32_t rows;    // rows of this tile, at most the tile height
  int64_t row0;    // first row in the operand
  int32_t col;     // column tile
};

// The tile of workgroup `block`, out of row tiles of `height` rows times
// `col_tiles` column tiles.  The number of row tiles is known only here, from
// the groups' counts: the grid is an upper bound and the surplus workgroups
// get false.  Workgroups go round robin to the 8 XCDs, so that each XCD takes
// one contiguous eighth of the tiles; within it, bands of kBand row tiles walk
// the columns together, so that what runs at one time on an XCD shares row
// panels and (row tiles of one group) matrix panels in its L2.  kOneGroup: bands
// are of row tiles of one group.
// A group's rows are shared out evenly among its row tiles, in steps of 16 (so
// that 257 rows make tiles of 144 and 113 rows and not of 256 and 1; a kernel
// skips a tile's blocks of 16 rows that it does not have).
// Every wave does the search by itself: its lanes hold E/64 groups each.
constexpr int kXcds = 8;
__device__ __forceinline__ int64_t uniform(int64_t v) {  // the same in every lane: to scalar registers
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int32_t)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int32_t)v));
}
template <int kBand, bool kOneGroup = false>
__device__ __forceinline__ bool find_tile(const RowGroups& g, int32_t height, int32_t col_tiles,
                                          uint32_t block, Tile& t) {
  const int lane = threadIdx.x & 63;
  const int per = (g.E + 63) / 64;
  int32_t mine = 0;
  for (int j = 0; j < per; ++j) {
    const int e = lane * per + j;
    if (e < g.E) mine += tiles_of(group_count(g, e), height);
  }
  const int32_t incl = wave_inclusive_sum(mine);
  const int32_t row_tiles = __builtin_amdgcn_readlane(incl, 63);
  const int64_t total = (int64_t)row_tiles * col_tiles;
  const int64_t share = (total + kXcds - 1) / kXcds;
  const int64_t in_share = block / kXcds;
  const int64_t id = (int64_t)(block % kXcds) * share + in_share;
  if (in_share >= share || id >= total) return false;
  constexpr int32_t kRows = kOneGroup ? 1 : kBand;
  const int64_t band_tiles = (int64_t)kRows * col_tiles;
  const int32_t band = (int32_t)(id / band_tiles);
  const int32_t rem = (int32_t)(id - band * band_tiles);
  const int32_t height_of_band = min(kRows, row_tiles - band * kRows);
  const int32_t target = band * kRows + rem % height_of_band;
  t.col = rem / height_of_band;
  // The last lane whose first row tile is not after the target holds it.
  const int32_t before = incl - mine;
  const uint64_t not_after = __builtin_amdgcn_ballot_w64(before <= target);
  const int owner = 63 - __builtin_clzll(not_after);
  int32_t left = target - before, e = lane * per;
  for (int j = 0; j < per; ++j) {
    if (e >= g.E - 1) break;
    const int32_t n = tiles_of(group_count(g, e), height);
    if (left < n) break;
    left -= n;
    ++e;
  }
  t.e = __builtin_amdgcn_readlane(e, owner);
  left = __builtin_amdgcn_readlane(left, owner);
  const int32_t count = group_count(g, t.e);
  const int32_t even = (tiles_of(count, tiles_of(count, height)) + 15) & ~15;
  if constexpr (kOneGroup) {
    const int32_t n = tiles_of(count, height), at = left * col_tiles + t.col, whole = kBand * col_tiles;
    const int32_t rest = at % whole, rows = min(kBand, n - at / whole * kBand);
    left = at / whole * kBand + rest % rows;
    t.col = rest / rows;
  }
  const int32_t each = min(height, even);
  t.rows = (int32_t)min((int64_t)each, count - (int64_t)left * each);
  t.row0 = group_first(g, t.e) + (int64_t)left * each;
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.row0 = uniform(t.row0);
  t.col = __builtin_amdgcn_readfirstlane(t.col);
  return t.rows > 0;
}

// A launch holds fewer than 2^32 threads.
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads < ((int64_t)1 << 32); }

// --------------------------------------------------------------------------
// One call's products.  `a` holds the rows that the groups own (for the
// weights' gradient, whose reduction runs over them, the rows of dy), `b` the
// matrices (there: the rows of x).  Leading dimensions are in elements.
// --------------------------------------------------------------------------
struct GemmArgs {
  RowGroups groups;
  const void* a;
  const void* b;
  int32_t lda, ldb;
  int32_t out_rows;    // weights' gradient only: rows of each group's result
  int32_t out_cols;    // columns of the result (swiglu forward: of the activated result)
  int32_t reduce;      // length of the reduction (not for the weights' gradient)
  int64_t b_stride;    // elements from one group's matrix to the next
  int32_t act;
  const void* bias;      // forward: [E, columns of the product]
  const void* residual;  // forward: [rows, out_cols]
  void* preact;          // forward: written, may be NULL; rows' gradient: read
  void* out;
  void* bias_grad;       // weights' gradient: [E, out_rows] or NULL
  bool grad_f32;         // weights' gradient: fp32 results
  bool accumulate;       // weights' gradient: added to what is there
  // FP8: scales (fp32 per 128 channels, or 4 E8M0 bytes), one word per row and
  // 128 channels.
  const void* a_scales;
  const void* b_scales;
  int64_t a_scale_row, a_scale_step;  // words from row to row, and from 128 channels to the next
};

// --------------------------------------------------------------------------
// Element types and activations.
// --------------------------------------------------------------------------
template <bool kF16>
__device__ __forceinline__ float elem_at(const void* p, int64_t i) {
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  if constexpr (kF16) return (float)__builtin_bit_cast(_Float16, v);
  else return __uint_as_float((uint32_t)v << 16);
}
// fp32 -> bf16 or fp16, one rounding to nearest, ties to even.
template <bool kF16>
__device__ __forceinline__ uint16_t elem_rne(float f) {
  if constexpr (kF16) return __builtin_bit_cast(uint16_t, (_Float16)f);
  else return __builtin_bit_cast(uint16_t, (__bf16)f);
}
template <bool kF16>
__device__ __forceinline__ uint32_t elem_rne2(float lo, float hi) {
  return (uint32_t)elem_rne<kF16>(lo) | ((uint32_t)elem_rne<kF16>(hi) << 16);
}
template <bool kF16>
__device__ __forceinline__ float elem_low(uint32_t w) {
  if constexpr (kF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xFFFFu));
  else return __uint_as_float(w << 16);
}
template <bool kF16>
__device__ __forceinline__ float elem_high(uint32_t w) {
  if constexpr (kF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
  else return __uint_as_float(w & 0xFFFF0000u);
}

// 1 / (1 + exp(-z)) by the hardware's 2^x and reciprocal (each within an ulp
// of fp32; the argument's rounding adds |z| 2^-24: far below the rounding of
// the result to 16 bits).  exp(-z) overflows to infinity for z below -88, and
// the reciprocal is then 0.
// kExact: by expf and a correctly rounded quotient, where there is time for it.
template <bool kExact = false>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (kExact) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }
__device__ __forceinline__ float silu_slope(float z) {
  const float p = sigmoid(z);
  return p * (1.0f + z * (1.0f - p));
}
// d silu'(z) where there is time for it, rounded operation by operation as the formula
// stands: the gradient that an activation hands on in 16 bits is the one that the same
// formula gives in fp32 outside of a kernel.  (With multiply-adds one of 9000 fp16
// results went to the other neighbour, and the fp32 weights' gradient of 777 x 1000 x 504
// made of them was up to 2.8e-5 of its norm away.)
__device__ __forceinline__ float silu_backward_exact(float d, float z) {
#pragma clang fp contract(off)
  const float p = sigmoid<true>(z), q = z * (1.0f - p);
  return d * p * (1.0f + q);
}

// The lower tail of the normal distribution, without its exponential: h(a) of
//   Phi(-a) = bell h(a),  bell = exp(-a^2 / 2),  a = |z|,
// so that the tail keeps its digits all the way down.  h = t R(t), t = 1 / (1 + a / 4),
// R of degree 9, fitted here to the least largest relative error, 3e-9, over all a (h
// runs from 1/2 at 0 to 1 / (a sqrt(2 pi)) far out, which is R's value at t = 0 over
// a / 4).  In fp32 the tail is off by 1e-6 of itself up to a = 3 and by 2^-17 at 13,
// where the exponential's argument is rounded at 122 and a bf16 leaves its normal range.
// (1 + erf in fp32 is 0 at z = -6, and a fit of least absolute error, 1.5e-7, is off by
// 1% at -8.)  One exponential serves value and slope.  With the library's functions: the
// activation's own gradient, 8192 x 4096, 64 us by erfcf and expf, 47 by a true quotient
// and expf, 40 so, which is HBM's time; the rows' gradient through gelu of 1803 rows, 24
// experts, 392 x 520, 20 us by erff and expf, 16 so.
// kExact: the hardware's reciprocal improved by one step, where there is time for it.
template <bool kExact = false>
__device__ __forceinline__ float normal_tail(float a, float& bell) {
  const float d = fmaf(0.25f, a, 1.0f);
  float t = __builtin_amdgcn_rcpf(d);
  if constexpr (kExact) t = fmaf(fmaf(-d, t, 1.0f), t, t);
  bell = __builtin_amdgcn_exp2f(a * a * -0.72134752044448170f);
  float r = fmaf(t, 0.0209641105f, -0.0862399986f);
  r = fmaf(t, r, 0.105812593f);
  r = fmaf(t, r, -0.0423424627f);
  r = fmaf(t, r, 0.0702728241f);
  r = fmaf(t, r, 0.0565008422f);
  r = fmaf(t, r, 0.0821602460f);
  r = fmaf(t, r, 0.0933954401f);
  r = fmaf(t, r, 0.0997409440f);
  r = fmaf(t, r, 0.0997354605f);
  return t * r;
}
__device__ __forceinline__ float gelu(float z) {
  float bell;
  const float h = normal_tail(fabsf(z), bell);
  return z * (z < 0.0f ? bell * h : fmaf(-bell, h, 1.0f));
}
// Phi(z) + z phi(z) = g bell for z < 0 and 1 - g bell for z >= 0, g = h(a) - a / sqrt(2 pi).
template <bool kExact = false>
__device__ __forceinline__ float gelu_slope(float z) {
  float bell;
  const float a = fabsf(z), h = normal_tail<kExact>(a, bell), g = fmaf(a, -0.39894228040143268f, h);
  return z < 0.0f ? bell * g : fmaf(-bell, g, 1.0f);
}
__device__ __forceinline__ float act_value(int32_t act, float z) {
  switch (act) {
    case EP_ACT_RELU: return z < 0.0f ? 0.0f : z;  // a NaN stays one
    case EP_ACT_GELU: return gelu(z);
    case EP_ACT_SILU: return silu(z);
    default: return z;
  }
}
// d * act'(z)
template <bool kExact = false>
__device__ __forceinline__ float act_backward(int32_t act, float d, float z) {
  switch (act) {
    case EP_ACT_RELU: return z > 0.0f ? d : 0.0f;
    case EP_ACT_GELU: return d * gelu_slope<kExact>(z);
    case EP_ACT_SILU:
      if constexpr (kExact) return silu_backward_exact(d, z);
      else return d * silu_slope(z);
    default: return d;
  }
}

// --------------------------------------------------------------------------
// Epilogues: what becomes of a wave's TM x TN blocks of 16 x 16 sums (block
// (i, j), lane l: row l % 16, columns 4 (l / 16) .. + 3).
// --------------------------------------------------------------------------
enum Mode { kForward = 0, kRowsGrad = 1, kWeightsGrad = 2 };

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN, int kWaveBytes>
struct TileStore {
  static constexpr int kWaveCols = 16 * TN;
  static constexpr int kMask = 4 * TN < 16 ? 4 * TN - 1 : 15;  // 16-byte chunks of a row that change places
  static constexpr int kOutCols = kWaveCols * WN / (kGlu && kMode == kForward ? 2 : 1);

  // A wave hands its results to itself through its share of the ring, so that
  // a lane gets 8 neighbouring columns of a row, neighbouring lanes the next
  // ones, and every store covers whole cache lines.  16-byte chunk c of row r
  // lies at c ^ (r & 15) (as far as the row has chunks): the 16 rows that one
  // store instruction writes at the same column touch every bank once.
  static constexpr int kFit = kWaveBytes / (16 * kWaveCols * 4);  // blocks of rows that fit at once
  static constexpr int pass_blocks() {  // the largest part of TM that fits
    int n = kFit < TM ? kFit : TM;
    while (TM % n != 0) --n;
    return n;
  }
  static constexpr int kPassBlocks = pass_blocks();
  static_assert(TM % kPassBlocks == 0, "whole passes");

  static __device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = elem_low<kF16>(u[k]);
      v[2 * k + 1] = elem_high<kF16>(u[k]);
    }
  }
  static __device__ __forceinline__ void store8(void* p, int64_t i, const float* v) {
    u32x4 w;
    w.x = elem_rne2<kF16>(v[0], v[1]);
    w.y = elem_rne2<kF16>(v[2], v[3]);
    w.z = elem_rne2<kF16>(v[4], v[5]);
    w.w = elem_rne2<kF16>(v[6], v[7]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  }
  static __device__ __forceinline__ void fetch8(const char* own, int row, int col, float* v) {
    const int c = col >> 2;
    const f32x4 a = *reinterpret_cast<const f32x4*>(own + row * (kWaveCols * 4) + ((c ^ (row & kMask)) << 4));
    const f32x4 b = *reinterpret_cast<const f32x4*>(own + row * (kWaveCols * 4) + (((c + 1) ^ (row & kMask)) << 4));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }

  // `own`: the wave's kWaveBytes of LDS.
  static __device__ __forceinline__ void store_tile(const GemmArgs& g, const Tile& t, char* own, int wm,
                                                    int wn, const f32x4 (&acc)[TM][TN]) {
    const int lane = threadIdx.x & 63;
    constexpr int kLaneCols = kOutCols / WN / 8;  // lanes that share a row
    constexpr int kLaneRows = 64 / kLaneCols;     // rows of one pass of the loop below
    const int col_in = (lane % kLaneCols) * 8;
    const int col = t.col * kOutCols + wn * (kOutCols / WN) + col_in;
    const bool col_ok = col < g.out_cols;
    float bias[2][8] = {};
    if constexpr (kMode == kForward) {
      if (g.bias != nullptr && col_ok) {
        const int64_t at = (int64_t)t.e * (kGlu ? 2 * g.out_cols : g.out_cols) + col;
        load8(g.bias, at, bias[0]);
        if constexpr (kGlu) load8(g.bias, at + g.out_cols, bias[1]);
      }
    }
#pragma unroll
    for (int pass = 0; pass < TM / kPassBlocks; ++pass) {
#pragma unroll
      for (int i = 0; i < kPassBlocks; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int row = i * 16 + (lane & 15), c = j * 4 + (lane >> 4);
          *reinterpret_cast<f32x4*>(own + row * (kWaveCols * 4) + ((c ^ (row & kMask)) << 4)) =
              acc[pass * kPassBlocks + i][j];
        }
#pragma unroll 4
      for (int it = 0; it < 16 * kPassBlocks / kLaneRows; ++it) {
        const int r = it * kLaneRows + lane / kLaneCols;
        // block b of the wave is block b * WM + wm of the tile
        const int in_tile = (((pass * kPassBlocks + (r >> 4)) * WM + wm) << 4) + (r & 15);
        float v[8], u[8];
        fetch8(own, r, col_in, v);
        if constexpr (kGlu && kMode == kForward) fetch8(own, r, kWaveCols / 2 + col_in, u);
        if (in_tile < t.rows && col_ok) store_row(g, t, t.row0 + in_tile, col, v, u, bias);
      }
    }
  }

  // 8 results of one row: the products v (and u, the ups of swiglu's forward).
  static __device__ __forceinline__ void store_row(const GemmArgs& g, const Tile& t, int64_t row,
                                                   int col, float* v, float* u,
                                                   const float (*bias)[8]) {
    const int32_t n = g.out_cols;
    if constexpr (kMode == kForward) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += bias[0][k];
      if constexpr (kGlu) {
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] += bias[1][k];
        if (g.preact != nullptr) {
          store8(g.preact, row * 2 * n + col, v);
          store8(g.preact, row * 2 * n + n + col, u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = silu(v[k]) * u[k];
      } else {
        if (g.preact != nullptr) store8(g.preact, row * n + col, v);
        if (g.act != EP_ACT_NONE) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = act_value(g.act, v[k]);
        }
      }
      if (g.residual != nullptr) {
        float r[8];
        load8(g.residual, row * n + col, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += r[k];
      }
      store8(g.out, row * n + col, v);
    } else if constexpr (kMode == kRowsGrad) {
      float z[8];
      if constexpr (kGlu) {
        load8(g.preact, row * 2 * n + col, z);
        load8(g.preact, row * 2 * n + n + col, u);
        float dup[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dup[k] = v[k] * silu(z[k]);
          v[k] = v[k] * u[k] * silu_slope(z[k]);
        }
        store8(g.out, row * 2 * n + col, v);
        store8(g.out, row * 2 * n + n + col, dup);
      } else {
        if (g.act != EP_ACT_NONE) {
          load8(g.preact, row * n + col, z);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = act_backward(g.act, v[k], z[k]);
        }
        store8(g.out, row * n + col, v);
      }
    } else {
      const int64_t at = ((int64_t)t.e * g.out_rows + row) * n + col;
      if (g.grad_f32) {
        f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
        f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        if (g.accumulate) {
          a += p[0];
          b += p[1];
        }
        p[0] = a;
        p[1] = b;
      } else {
        if (g.accumulate) {
          load8(g.out, at, u);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += u[k];
        }
        store8(g.out, at, v);
      }
    }
  }
};

// Picks the kernel for a 16-bit product.
hipError_t launch_gemm(const GemmArgs& g, int mode, bool f16, hipStream_t stream);
// rows: about how many each group has.  wide: 64 x 64 tiles (the gradients' always are).
hipError_t launch_gemm_few(const GemmArgs& g, int mode, int64_t rows, bool wide, bool f16, hipStream_t stream);
hipError_t launch_gemm_fp8(const GemmArgs& g, bool mx, hipStream_t stream);
// launch_gemm_tile: `mode` 0 forward, 1 rows' gradient, 2 weights' gradient.
hipError_t launch_gemm_tile(const GemmArgs& g, int mode, bool f16, bool large, hipStream_t stream);

hipError_t launch_combine_grad(const void* dout, const void* y, const float* w, const ep_layout_t& L,
                               int32_t hidden, bool f16, void* dy, float* dw, hipStream_t stream);
hipError_t launch_act_grad(const void* dy, const void* z, int64_t rows, int32_t n, bool f16,
                           int32_t act, void* dz, hipStream_t stream);

}  // namespace ep
