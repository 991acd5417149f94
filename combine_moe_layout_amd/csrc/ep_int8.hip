// ep_int8.hip -- rows of bf16 or fp16 to 8-bit integers with one fp32 scale per row: dispatch's
// (every row goes to its token's receive rows) and of rows where they stand.
//
//   a = max(max|x|, 2^-100),  scale = a / 127 (one fp32 division),
//   code = the integer nearest to x / scale, ties to even
//
// A row that holds a NaN or an infinity gets a scale of NaN and codes of 0, so that whatever is
// computed from it is NaN.
//
// The quotient is that of real numbers: x times the scale's reciprocal is within 2^-16 of it, and
// where that is closer than 2^-14 to a border between two codes, the remainder x - code * scale,
// which one fused multiply-add gives exactly, decides (one wave in eight has such a place).
//
// Bound by HBM, as FP8 dispatch: one read of x, a row write for each of the token's pairs.  A row
// stays in its lanes' registers, 16 channels (two loads, one store of codes) to a vector, between
// its maximum and its codes.  65536 rows of 2048: 71 us (5.6 TB/s); dispatch of 8192 x 7168 to 8
// experts each: 97 us (6.0 TB/s).  Dispatch's stores go past the caches, those of rows where they
// stand do not: written past them, 1024 x 7168 rows and the product that reads them take 58 us
// together, 50 us as it is.
#include "ep_int8.h"

namespace ep {

namespace {

constexpr int kMaxLanes = 1024;
constexpr float kCodes = 127.0f;

typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;

// Larger of the magnitudes' bits, of both halves: the order of the bits is that of the values,
// with infinity above all of them and NaN above infinity.
__device__ __forceinline__ uint32_t max_magnitudes(uint32_t a, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}

// Codes of 16 values.
template <bool kF16>
__device__ __forceinline__ u32x4 encode16(const u32x4 (&x)[2], float scale, float inverse) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: a sum with it is rounded to integers
  float f[16], m[16], off = 0.0f;
  const uint32_t u[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = elem_low<kF16>(u[i]);
    f[2 * i + 1] = elem_high<kF16>(u[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = f[i] * inverse;
    m[i] = t + kMagic;
    off = fmaxf(off, fabsf(t - (m[i] - kMagic)));
  }
  if (__builtin_amdgcn_ballot_w64(off > 0.5f - 0x1p-14f) != 0) {
    const float half = 0.5f * scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float n = m[i] - kMagic, left = fmaf(-n, scale, f[i]);
      const bool odd = __float_as_uint(m[i]) & 1;
      if (left > half || (left == half && odd)) m[i] += 1.0f;
      else if (left < -half || (left == -half && odd)) m[i] -= 1.0f;
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b[4] = {__float_as_uint(m[4 * i]), __float_as_uint(m[4 * i + 1]), __float_as_uint(m[4 * i + 2]),
                           __float_as_uint(m[4 * i + 3])};
    w[i] = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  }
  return u32x4{w[0], w[1], w[2], w[3]};
}

// Whether a receive row is in use, by a layout's groups (E = 0: all rows are).
__device__ __forceinline__ bool row_used(const RowGroups& g, int64_t row) {
  if (g.first == nullptr) return true;
  if (g.capacity > 0) return row % g.capacity < group_count(g, (int32_t)(row / g.capacity));
  return row < g.first[g.E];
}

// lanes: threads of one row, whole waves; the block holds blockDim / lanes rows (one, if lanes >
// 64).  slots: a token's k receive rows, or NULL: the row itself.
template <bool kF16, int V>
__global__ __launch_bounds__(kMaxLanes) void int8_rows_kernel(const u32x4* __restrict__ x, int64_t rows,
                                                              int32_t hidden, int32_t lanes, int32_t k,
                                                              const int32_t* __restrict__ slots, RowGroups groups,
                                                              u32x4* __restrict__ codes,
                                                              float* __restrict__ scales) {
  __shared__ uint32_t part[kMaxLanes / 64];
  const int lane = threadIdx.x % lanes, local = threadIdx.x / lanes;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lanes) + local;
  if (row >= rows || (slots == nullptr && !row_used(groups, row))) return;  // all lanes of the row
  const int32_t vecs = hidden / 16;
  const u32x4* const from = x + row * vecs * 2;
  u32x4 in[V][2];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = lane + i * lanes;
    in[i][0] = in[i][1] = u32x4{0, 0, 0, 0};
    if (v < vecs) {
      in[i][0] = from[2 * v];
      in[i][1] = from[2 * v + 1];
    }
  }
  uint32_t both = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      both = max_magnitudes(both, in[i][h].x);
      both = max_magnitudes(both, in[i][h].y);
      both = max_magnitudes(both, in[i][h].z);
      both = max_magnitudes(both, in[i][h].w);
    }
  uint32_t most = reduce_max<64>(max(both & 0xFFFFu, both >> 16));
  if (lanes > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
    __syncthreads();
    for (int w = 0; w < lanes / 64; ++w) most = max(most, part[w]);
  }
  const float largest = elem_low<kF16>(most);
  const bool finite = largest <= 3.40282347e38f;
  float scale = fmaxf(largest, 0x1p-100f) / kCodes, inverse = 1.0f / scale;
  if (!finite) scale = __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = lane + i * lanes;
    u32x4 q = encode16<kF16>(in[i], scale, inverse);
    if (!finite) q = u32x4{0, 0, 0, 0};
    if (v >= vecs) continue;
    if (slots == nullptr) {
      codes[row * vecs + v] = q;
    } else {
      for (int j = 0; j < k; ++j) {
        const int32_t s = slots[row * k + j];
        if (s >= 0) store_nt(codes + (int64_t)s * vecs + v, q);
      }
    }
  }
  if (slots == nullptr) {
    if (lane == 0) scales[row] = scale;
  } else {
    for (int j = lane; j < k; j += lanes) {
      const int32_t s = slots[row * k + j];
      if (s >= 0) scales[s] = scale;
    }
  }
}

template <bool kF16>
hipError_t launch(const void* x, int64_t rows, int32_t hidden, int32_t k, const int32_t* slots,
                  const RowGroups& groups, void* codes, float* scales, hipStream_t stream) {
  const int vecs = hidden / 16;
  // Rows where they stand: two vectors to a lane beyond one wave's 64 (8192 x 7168: 30.5 us, 35.1 with one
  // and 34 with four; 65,536 x 2048: 71.5, 77.5 and 77).  Four, so that a row is one wave's and needs no
  // barrier, where that saves a second wave with half its lanes idle and there are rows enough: 65,536 x
  // 2064 and 2560 80 and 91.5 us (87 and 99 with two), 16,384 x 2560 26.4 (26.4); but 8192 x 2560 17.6
  // (16.6), 16 x 4096 7.2 (4.9), 65,536 x 3584 131 (122).  Dispatch: one as long as a workgroup holds the
  // row, for its k stores to be spread wide (8192 tokens of 4096 to 6 experts: 41 us, 64 with four).
  int vectors = 1;
  if (slots == nullptr && vecs > 64) vectors = vecs > 128 && vecs < 192 && rows >= 16384 ? 4 : 2;
  while ((vecs + vectors - 1) / vectors > kMaxLanes) vectors *= 2;
  const int lanes = ((vecs + vectors - 1) / vectors + 63) / 64 * 64;
  const int here = lanes == 64 ? 4 : 1;
  const int64_t blocks = (rows + here - 1) / here;
  if (!grid_fits(blocks, lanes * here)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  const auto run = [&](auto kernel) {
    kernel<<<(uint32_t)blocks, lanes * here, 0, stream>>>(static_cast<const u32x4*>(x), rows, hidden, lanes, k, slots,
                                                          groups, static_cast<u32x4*>(codes), scales);
  };
  if (vectors == 1) run(int8_rows_kernel<kF16, 1>);
  else if (vectors == 2) run(int8_rows_kernel<kF16, 2>);
  else run(int8_rows_kernel<kF16, 4>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch_int8(const void* x, const ep_layout_t& L, int32_t hidden, void* recv_x,
                                void* recv_scales, hipStream_t stream) {
  return launch<false>(x, L.num_tokens, hidden, L.num_topk, L.slot_idx, RowGroups{}, recv_x,
                       static_cast<float*>(recv_scales), stream);
}

hipError_t launch_quantize_int8(const void* x, const RowGroups& groups, int32_t n, bool f16, void* q,
                                float* scales, hipStream_t stream) {
  return f16 ? launch<true>(x, groups.rows, n, 1, nullptr, groups, q, scales, stream)
             : launch<false>(x, groups.rows, n, 1, nullptr, groups, q, scales, stream);
}

}  // namespace ep
