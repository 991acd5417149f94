// ep_gemm_tile.hip -- bf16 and fp16 matrix products over ragged groups of rows,
// for groups of many rows: the experts' products, a dense layer's, and both
// kinds of gradients.
//
//   forward        out[r, n] = act(sum_k a[r, k] b[e, n, k] + bias[e, n]) + residual[r, n]
//   rows' gradient out[r, k] = (sum_n a[r, n] b[e, n, k]) act'(preact[r, k])
//   weights'       out[e, n, k] (+)= sum_{r in e} a[r, n] b[r, k]
//
// e is the group (expert) that row r belongs to.  The products are summed in
// fp32 by the matrix instructions and rounded once, after the epilogue.
//
// A workgroup of 4 waves makes one tile; each wave owns TM x TN blocks of 16 x
// 16 results.  The reduction is cut into stages of 32; a ring of 4 stages in LDS is
// filled by loads that need no registers, up to three stages ahead.  While the
// matrix instructions work on stage s, the matrix operand of stage s + 1 and
// the row operand's next fragments are read into registers, so one barrier a
// stage is the only time that they can stand still.
//
// The matrix operand takes the instruction's row side and the row operand its
// column side, so that a lane ends up with 4 neighbouring columns of one result
// row.  Where an operand has its reduction as the slow dimension, the
// transposing LDS read makes the fragments.
#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kStage = 32;  // reduction elements per stage (64 bytes)
constexpr int kSlots = 4;   // stages in the ring
constexpr int kWaves = 4;

template <bool kF16>
struct Frag;
template <>
struct Frag<false> {
  typedef bf16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<true> {
  typedef f16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// How `kSpan` rows (or columns) of an operand sit in a stage of LDS, and how
// they get there.
//  Reduction contiguous in memory: kSpan rows of 64 bytes, 16-byte chunk c of
//  row r at place c ^ ((r >> 2) & 3), so that the 16 lanes that read one chunk
//  of 16 neighbouring rows touch every bank once.
//  Reduction slow in memory: 32 rows of kSpan elements, pair p of 16-byte
//  chunks of row k at place p ^ f(k), f(k) = 4 * bit 3 of k + (k & 3): the
//  eight rows that one half wave of a transposing read touches lie in
//  different banks.
template <bool kContiguous, int kSpan>
struct Operand {
  static constexpr int kBytes = kSpan * kStage * 2;
  static constexpr int kLoads = kBytes / 1024 / kWaves;  // loads of a wave per stage
  static constexpr int kChunks = kSpan / 8;              // chunks per LDS row, slow reduction
  static_assert(kContiguous || kSpan >= 128, "the bank pattern spans 16 chunks");

  static __device__ __forceinline__ int swizzle(int k) { return ((k >> 3) & 1) * 4 + (k & 3); }

  // The row (contiguous) or reduction row (slow) of this lane's i-th load, and its chunk.
  static __device__ __forceinline__ int load_row(int i) {
    const int j = (threadIdx.x >> 6) * kLoads + i, lane = threadIdx.x & 63;
    return kContiguous ? j * 16 + (lane >> 2) : j * (64 / kChunks) + lane / kChunks;
  }
  static __device__ __forceinline__ int load_chunk(int i) {
    const int lane = threadIdx.x & 63, row = load_row(i);
    return kContiguous ? ((lane & 3) ^ ((row >> 2) & 3))
                       : ((lane % kChunks) ^ (swizzle(row) << 1));
  }
  static __device__ __forceinline__ uint32_t load_place(int i) {  // the wave's LDS offset
    return ((threadIdx.x >> 6) * kLoads + i) * 1024;
  }
};

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
struct TileGemm {
  static_assert(WM * WN == kWaves, "four waves");
  static constexpr int kRows = 16 * TM * WM;  // result rows of a tile
  static constexpr int kCols = 16 * TN * WN;  // product columns of a tile
  static constexpr bool kAContig = kMode != kWeightsGrad;
  static constexpr bool kBContig = kMode == kForward;
  typedef Operand<kAContig, kRows> A;
  typedef Operand<kBContig, kCols> B;
  typedef typename Frag<kF16>::type F;
  static constexpr int kStageBytes = A::kBytes + B::kBytes;
  static constexpr int kLoads = A::kLoads + B::kLoads;
  static constexpr int kAhead = 3;  // row fragments read ahead of their use
  static constexpr int kWaveCols = 16 * TN;
  static constexpr int kWaveBytes = kSlots * kStageBytes / kWaves;
  typedef TileStore<kMode, kF16, kGlu, TM, TN, WM, WN, kWaveBytes> Store;
  static constexpr int kOutCols = Store::kOutCols;

  const GemmArgs& g;
  char* const lds;
  uint32_t lds0;
  Tile t;
  int32_t reduce, stages, whole_stages;
  int32_t a_limit, b_limit;  // valid rows (contiguous) or columns (slow) of each operand
  const char *a0, *b0;       // first element of the operand of this tile
  int64_t a_step, b_step;    // bytes from one stage to the next
  uint32_t a_off[A::kLoads], b_off[B::kLoads];
  uint32_t a_read, b_read;
  int wm, wn, lane;
  int blocks;  // blocks of 16 rows of this wave that the tile has
  f32x4 acc[TM][TN];
  float bias_sum[2];
  bool bias_tile;
  F af[kAhead + 1], bf[2][TN];

  __device__ __forceinline__ TileGemm(const GemmArgs& args, char* smem) : g(args), lds(smem) {}

  // Row of the matrix operand that stands at place p of the tile's LDS rows:
  // for swiglu the first half of a wave's rows are gates, the second half the
  // ups of the same columns.
  __device__ __forceinline__ int matrix_row(int p) const {
    if constexpr (kGlu && kMode == kForward) {
      const int w = p / kWaveCols, in = p % kWaveCols, half = kWaveCols / 2;
      const int n = t.col * kOutCols + w * half + in % half;
      return min(n, g.out_cols - 1) + (in >= half ? g.out_cols : 0);
    } else {
      return min(t.col * kCols + p, g.out_cols - 1);
    }
  }

  __device__ __forceinline__ void setup() {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    lds0 = lds_address(lds);
    blocks = ((t.rows + 15) / 16 - wm + WM - 1) / WM;
    whole_stages = reduce / kStage;
    stages = (reduce + 2 * kStage - 1) / (2 * kStage) * 2;  // an even number: the last may be all zeros
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      const int row = A::load_row(i), chunk = A::load_chunk(i);
      if constexpr (kAContig) a_off[i] = (uint32_t)min(row, a_limit - 1) * (uint32_t)g.lda * 2u + chunk * 16;
      else a_off[i] = (uint32_t)row * (uint32_t)g.lda * 2u + min(chunk * 8, a_limit - 8) * 2;
    }
#pragma unroll
    for (int i = 0; i < B::kLoads; ++i) {
      const int row = B::load_row(i), chunk = B::load_chunk(i);
      if constexpr (kBContig) b_off[i] = (uint32_t)matrix_row(row) * (uint32_t)g.ldb * 2u + chunk * 16;
      else b_off[i] = (uint32_t)row * (uint32_t)g.ldb * 2u + min(chunk * 8, b_limit - 8) * 2;
    }
    a_step = kAContig ? kStage * 2 : (int64_t)kStage * g.lda * 2;
    b_step = kBContig ? kStage * 2 : (int64_t)kStage * g.ldb * 2;
    a_read = read_offset<A, kAContig>(wm * 16);
    b_read = A::kBytes + read_offset<B, kBContig>(wn * 16 * TN);
  }

  // LDS offset of this lane's part of the first fragment at row (column) w0.
  template <class Op, bool kContig>
  __device__ __forceinline__ uint32_t read_offset(int w0) const {
    const int q = lane >> 4, m = lane & 15;
    if constexpr (kContig) {
      return (w0 + m) * 64 + ((q ^ ((m >> 2) & 3)) << 4);
    } else {
      const int k = q * 8 + (m >> 2), gran = m & 3;
      return k * (Op::kChunks * 16) + (((w0 >> 3) ^ (Op::swizzle(k) << 1)) << 4) + ((gran >> 1) << 4) +
             ((gran & 1) << 3);
    }
  }

  // A wave's blocks of the row operand are every WM-th one of the tile, so that a
  // tile with few rows is shared by all waves; those of the other operand are
  // neighbours.
  template <class Op, bool kContig>
  __device__ __forceinline__ F read_fragment(uint32_t offset, int tile) const {
    if constexpr (kContig) {
      return *reinterpret_cast<const F*>(lds + offset + tile * 1024);
    } else {
      // Two transposing reads: reduction rows q*8 .. q*8+3, and the four after them.
      const uint32_t at = offset ^ (uint32_t)(tile << 5);
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(lds0 + at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds4*)(uintptr_t)(lds0 + at + 4 * Op::kChunks * 16));
      return __builtin_bit_cast(F, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }

  // Load j of a whole stage (the first A::kLoads are the row operand's).
  __device__ __forceinline__ void load_piece(int s, uint32_t slot, int j) const {
    const uint32_t at = lds0 + slot * kStageBytes;
    if (j < A::kLoads)
      load16_to_lds(a0 + s * a_step, a_off[j < A::kLoads ? j : 0],
                    __builtin_amdgcn_readfirstlane(at + A::load_place(j)));
    else
      load16_to_lds(b0 + s * b_step, b_off[j < A::kLoads ? 0 : j - A::kLoads],
                    __builtin_amdgcn_readfirstlane(at + A::kBytes + B::load_place(j - A::kLoads)));
  }
  // All loads of a stage; what lies past the reduction reads as zero.
  __device__ __forceinline__ void load_stage(int s, uint32_t slot) const {
    const int left = reduce - s * kStage;
    if (left >= kStage) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) load_piece(s, slot, j);
      return;
    }
    const uint32_t at = lds0 + slot * kStageBytes;
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      const int r = kAContig ? A::load_chunk(i) * 8 : A::load_row(i);
      const char* p = r < left ? a0 + s * a_step + a_off[i] : reinterpret_cast<const char*>(g_zero16);
      load16_to_lds(p, __builtin_amdgcn_readfirstlane(at + A::load_place(i)));
    }
#pragma unroll
    for (int i = 0; i < B::kLoads; ++i) {
      const int r = kBContig ? B::load_chunk(i) * 8 : B::load_row(i);
      const char* p = r < left ? b0 + s * b_step + b_off[i] : reinterpret_cast<const char*>(g_zero16);
      load16_to_lds(p, __builtin_amdgcn_readfirstlane(at + A::kBytes + B::load_place(i)));
    }
  }

  // Stage s.  Its matrix fragments are in the registers of `kSet` and its first
  // kAhead row fragments in af; the other row fragments are read while the
  // matrix instructions work, and so are the next stage's first ones.
  template <int kSet>
  __device__ __forceinline__ void step(int s) {
    // Stage s + 1 has landed, for every wave; and every wave is done with stage s - 1.
    if (s + 2 < stages) wait_loads<(kSlots - 3) * kLoads>();
    else wait_loads<0>();
    lds_barrier();
    const int ahead = s + kSlots - 1;
    const uint32_t slot = ahead % kSlots;
    const uint32_t base = (s % kSlots) * kStageBytes, next = ((s + 1) % kSlots) * kStageBytes;
    const bool whole = ahead < whole_stages;
    if (!whole && ahead < stages) load_stage(ahead, slot);
    if constexpr (kMode == kWeightsGrad) {
      if (bias_tile) add_to_bias(base);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (j * TM / kLoads == i && whole) load_piece(ahead, slot, j);
      // (past the last stage these read a slot whose contents nobody uses)
      constexpr int kRing = kAhead + 1;
      static_assert(2 * TM % kRing == 0, "two steps leave the ring where it was");
      const int f = i + kAhead;
      af[(kSet * TM + f) % kRing] = f < TM ? read_fragment<A, kAContig>(base + a_read, f * WM)
                                           : read_fragment<A, kAContig>(next + a_read, (f - TM) * WM);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (j * TM / TN == i) bf[1 - kSet][j] = read_fragment<B, kBContig>(next + b_read, j);
      const F a = af[(kSet * TM + i) % kRing];
      if (i < blocks) {
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Frag<kF16>::mfma(bf[kSet][j], a, acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Biases' gradient: the workgroups of the first column tile add up the rows of
  // dy that pass through their LDS, two columns and a part of the stage's rows
  // to a thread.
  static constexpr int kBiasParts = kWaves * 64 / (kRows / 2);
  __device__ __forceinline__ void add_to_bias(uint32_t base) {
    const int pair = threadIdx.x % (kRows / 2), part = threadIdx.x / (kRows / 2);
#pragma unroll
    for (int j = 0; j < kStage / kBiasParts; ++j) {
      const int k = part * (kStage / kBiasParts) + j;
      const uint32_t at = base + k * (A::kChunks * 16) + (((pair >> 2) ^ (A::swizzle(k) << 1)) << 4) +
                          (pair & 3) * 4;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(lds + at);
      bias_sum[0] += elem_low<kF16>(w);
      bias_sum[1] += elem_high<kF16>(w);
    }
  }
  // Called by all threads once the ring is free; the parts meet in LDS.
  __device__ __forceinline__ void store_bias() {
    float* sums = reinterpret_cast<float*>(lds);
    sums[threadIdx.x * 2] = bias_sum[0];
    sums[threadIdx.x * 2 + 1] = bias_sum[1];
    __syncthreads();
    for (int n = threadIdx.x; n < kRows && (int)t.row0 + n < g.out_rows; n += kWaves * 64) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < kBiasParts; ++p) s += sums[p * kRows + n];
      const int64_t at = (int64_t)t.e * g.out_rows + t.row0 + n;
      if (g.grad_f32) {
        float* p = static_cast<float*>(g.bias_grad) + at;
        *p = g.accumulate ? *p + s : s;
      } else {
        if (g.accumulate) s += elem_at<kF16>(g.bias_grad, at);
        static_cast<uint16_t*>(g.bias_grad)[at] = elem_rne<kF16>(s);
      }
    }
    __syncthreads();
  }

  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    bias_sum[0] = bias_sum[1] = 0.f;
    if (stages == 0) return;
    for (int s = 0; s < kSlots - 1 && s < stages; ++s) load_stage(s, s);
    wait_loads<0>();
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) af[i] = read_fragment<A, kAContig>(a_read, i * WM);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[0][j] = read_fragment<B, kBContig>(b_read, j);
    for (int s = 0; s < stages; s += 2) {
      step<0>(s);
      step<1>(s + 1);
    }
  }

  // Where the tile's operands lie; false for a workgroup without a tile.
  __device__ __forceinline__ bool place() {
    if constexpr (kMode == kWeightsGrad) {
      const int32_t rt = (g.out_rows + kRows - 1) / kRows, ct = (g.out_cols + kCols - 1) / kCols;
      // Every group's tiles are shared out among the XCDs, since the groups'
      // reductions may differ much in length.
      const int32_t share = (rt * ct + kXcds - 1) / kXcds;
      const int32_t in_share = blockIdx.x / kXcds;
      t.e = in_share / share;
      const int32_t rem = (int32_t)(blockIdx.x % kXcds) * share + in_share % share;
      if (t.e >= g.groups.E || rem >= rt * ct) return false;
      constexpr int32_t kBand = 4;
      const int32_t band = rem / (kBand * ct), in = rem - band * kBand * ct;
      const int32_t high = min(kBand, rt - band * kBand);
      t.row0 = (int64_t)(band * kBand + in % high) * kRows;
      t.col = in / high;
      t.rows = (int32_t)min((int64_t)kRows, g.out_rows - t.row0);
      bias_tile = g.bias_grad != nullptr && t.col == 0;
      const int64_t first = group_first(g.groups, t.e);
      reduce = __builtin_amdgcn_readfirstlane(group_count(g.groups, t.e));
      a_limit = g.out_rows - (int32_t)t.row0;
      b_limit = g.out_cols - t.col * kCols;
      a0 = static_cast<const char*>(g.a) + (first * g.lda + t.row0) * 2;
      b0 = static_cast<const char*>(g.b) + (first * g.ldb + (int64_t)t.col * kCols) * 2;
    } else {
      const int32_t ct = (g.out_cols + kOutCols - 1) / kOutCols;
      if (!find_tile<4>(g.groups, kRows, ct, blockIdx.x, t)) return false;
      reduce = g.reduce;
      a_limit = t.rows;
      a0 = static_cast<const char*>(g.a) + t.row0 * g.lda * 2;
      b0 = static_cast<const char*>(g.b) + t.e * g.b_stride * 2;
      if constexpr (kMode == kRowsGrad) {
        b_limit = g.out_cols - t.col * kCols;
        b0 += (int64_t)t.col * kCols * 2;
      }
    }
    return true;
  }

  __device__ __forceinline__ void run() {
    if (!place()) return;
    setup();
    accumulate();
    lds_barrier();  // every wave is done with the ring
    if constexpr (kMode == kWeightsGrad) {
      if (bias_tile) store_bias();
    }
    Store::store_tile(g, t, lds + (wm * WN + wn) * kWaveBytes, wm, wn, acc);
  }
};

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(kWaves * 64, TM * TN >= 64 ? 1 : 2) void gemm_tile_kernel(GemmArgs g) {
  typedef TileGemm<kMode, kF16, kGlu, TM, TN, WM, WN> G;
  __shared__ __align__(1024) char lds[kSlots * G::kStageBytes];
  G gemm(g, lds);
  gemm.run();
}

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  typedef TileGemm<kMode, kF16, kGlu, TM, TN, WM, WN> G;
  const int64_t ct = (g.out_cols + G::kOutCols - 1) / G::kOutCols;
  const int64_t rt = kMode == kWeightsGrad
                         ? (int64_t)g.groups.E * ((g.out_rows + G::kRows - 1) / G::kRows)
                         : max_row_tiles(g.groups, G::kRows);
  const int64_t rounds = kMode == kWeightsGrad ? (rt / g.groups.E * ct + kXcds - 1) / kXcds * g.groups.E
                                               : (rt * ct + kXcds - 1) / kXcds;
  const int64_t blocks = rounds * kXcds;
  if (!grid_fits(blocks, kWaves * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_tile_kernel<kMode, kF16, kGlu, TM, TN, WM, WN>
      <<<(uint32_t)blocks, kWaves * 64, 0, stream>>>(g);
  return hipGetLastError();
}

template <int kMode, bool kF16, bool kGlu>
hipError_t launch_size(const GemmArgs& g, bool large, hipStream_t stream) {
  return large ? launch<kMode, kF16, kGlu, 8, 8, 2, 2>(g, stream)
               : launch<kMode, kF16, kGlu, 4, 4, 2, 2>(g, stream);
}

template <bool kF16>
hipError_t launch_mode(const GemmArgs& g, int mode, bool large, hipStream_t stream) {
  const bool glu = g.act == EP_ACT_SWIGLU;
  if (mode == kWeightsGrad)
    return launch_size<kWeightsGrad, kF16, false>(g, large, stream);
  if (mode == kRowsGrad)
    return glu ? launch_size<kRowsGrad, kF16, true>(g, large, stream)
               : launch_size<kRowsGrad, kF16, false>(g, large, stream);
  return glu ? launch_size<kForward, kF16, true>(g, large, stream)
             : launch_size<kForward, kF16, false>(g, large, stream);
}

}  // namespace

hipError_t launch_gemm_tile(const GemmArgs& g, int mode, bool f16, bool large, hipStream_t stream) {
  return f16 ? launch_mode<true>(g, mode, large, stream) : launch_mode<false>(g, mode, large, stream);
}

// 256 x 256 tiles where the groups have the rows for them and there are enough
// tiles for every CU; 128 x 128 otherwise.
hipError_t launch_gemm(const GemmArgs& g, int mode, bool f16, hipStream_t stream) {
  const int64_t rows = mode == kWeightsGrad ? g.out_rows : g.groups.wanted / g.groups.E;
  const int64_t tiles = (int64_t)g.groups.E * ((rows + 255) / 256) * ((g.out_cols + 255) / 256);
  return launch_gemm_tile(g, mode, f16, rows >= 192 && tiles >= kChipCUs, stream);
}

}  // namespace ep
