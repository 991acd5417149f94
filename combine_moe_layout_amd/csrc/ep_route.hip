// ep_route.hip -- the router's choice, and its gradient.
//
//   s = softmax(l) or sigmoid(l),  key = s + bias (without a bias: l, which orders alike)
//   groups of E / G experts: the topk_groups groups of the largest group scores stay
//   idx = the k largest keys, descending, ties to the lower index
//   w_j = scale s_j, or scale s_j / sum_i s_i over the chosen
//
// A logit of -inf or NaN (or a key of NaN or -inf) takes no part; +inf counts as the largest
// fp32 value.
//
// A token is L lanes of V neighbouring experts each, so a wave holds 64 / L tokens and
// nothing but the chosen (expert, logit) pairs goes through LDS.  A choice is a maximum over
// the token's lanes by DPP moves on order-preserving integers, and the lowest lane that has it
// (lanes are in the experts' order) owns it: the tie goes to the lower index by itself.
//
// The order is that of the keys as real numbers.  Logits are compared as they are; keys with
// scores in them are made in fp32 first, and where two that the result depends on are closer
// than fp32 can tell, the wave makes its tokens' keys again in fp64 (for random logits and
// biases about one token in 300 at 256 experts).
//
// Weights over the chosen are taken relative to the largest one, so that they are right also
// where every chosen score underflows.
#include "ep_route.h"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr float kMostF32 = 3.40282347e38f;

// Real numbers as integers of the same order (-0 as +0).
__device__ __forceinline__ int32_t order_of(float v) {
  const int32_t b = __builtin_bit_cast(int32_t, v + 0.0f);
  return b ^ (int32_t)((uint32_t)(b >> 31) >> 1);
}
__device__ __forceinline__ int64_t order_of(double v) {
  const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
  return b ^ (int64_t)((uint64_t)(b >> 63) >> 1);
}
__device__ __forceinline__ float value_of(int32_t o) {
  return __builtin_bit_cast(float, o ^ (int32_t)((uint32_t)(o >> 31) >> 1));
}
__device__ __forceinline__ double value_of(int64_t o) {
  return __builtin_bit_cast(double, o ^ (int64_t)((uint64_t)(o >> 63) >> 1));
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// --------------------------------------------------------------------------
// Logits.
// --------------------------------------------------------------------------
template <int kType>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (kType == EP_F32) return static_cast<const float*>(p)[i];
  else return elem_at<kType == EP_F16>(p, i);
}
__device__ __forceinline__ float usable(float l) {
  return l > -INFINITY ? fminf(l, kMostF32) : -INFINITY;  // (a comparison with NaN is false)
}
// Experts first .. first + V - 1 of token t; -inf past the last.  `whole`: E is a multiple of V.
template <int kType, int V>
__device__ __forceinline__ void load_logits(const void* p, int64_t t, int E, int first, bool whole, float (&l)[V]) {
  const int64_t at = t * E + first;
  if (whole) {
    if (first < E) {
      if constexpr (kType == EP_F32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at + i);
#pragma unroll
          for (int c = 0; c < 4; ++c) l[i + c] = v[c];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + i);
          l[i] = elem_low<kType == EP_F16>(v.x);
          l[i + 1] = elem_high<kType == EP_F16>(v.x);
          l[i + 2] = elem_low<kType == EP_F16>(v.y);
          l[i + 3] = elem_high<kType == EP_F16>(v.y);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = first + i < E ? logit_at<kType>(p, at + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = usable(l[i]);
}

struct Choice {
  int32_t expert;  // -1: none
  float logit;
};

// What a wave's own LDS accesses need before other lanes of it read them.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The largest logit of a token and the sum of exp(l - largest) over its experts; a token
// without usable logits gets a sum of 1.
template <typename R, int L, int V>
__device__ __forceinline__ void softmax_sums(const float (&l)[V], R& top, R& sum) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
  m = fmaxf(reduce_max<L>(m), -kMostF32);
  top = m;
  R s = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) s += exp_of((R)l[i] - top);
  s = reduce_sum<L>(s);
  sum = s > 0 ? s : 1;
}

// The choice with keys of type R (float, or double where float cannot tell), into
// `chosen`.  Returns whether two keys or group scores that decide are closer than float's
// rounding (never with double): then `chosen` may be wrong.
template <typename R, int L, int V>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&l)[V], const float* bias,
                                       int lane, R* shared, Choice* chosen) {
  using K = std::conditional_t<sizeof(R) == 4, int32_t, int64_t>;
  constexpr bool kFloat = sizeof(R) == 4;
  const R none = -INFINITY;
  const K none_key = order_of(none);
  // Rounding: a score is within 2^-21 of itself (exp, sum, quotient: a few steps of 2^-24
  // each), the bias adds half a step of the sum; twice that for a difference, and twice for a
  // sum of two.
  const auto near = [](R larger, R smaller, R factor) {
    return larger - smaller <= factor * (R)0x1p-20 * (1 + fabs(larger));
  };
  const int first = lane * V;
  const bool grouped = a.topk_groups < a.groups;
  R key[V];
  bool scored = bias != nullptr || (grouped && a.group_top == 2);
  if (scored) {
    R top = 0, sum = 1;
    if (a.softmax) softmax_sums<R, L, V>(l, top, sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const R s = a.softmax ? exp_of((R)l[i] - top) / sum : 1 / (1 + exp_of(-(R)l[i]));
      R k = s;
      if (bias != nullptr) k += (R)(first + i < a.E ? bias[first + i] : 0.0f);
      key[i] = l[i] > -INFINITY && k > none ? k : none;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = l[i];
  }
  bool close = false;
  uint32_t keep = (1u << V) - 1;  // experts in groups that stay
  if (grouped) {
    // A group's score: its largest key, or the sum of its two largest.
    const int n = a.E / a.groups;
    R* const score = shared;                 // [groups]
    const bool in_lanes = a.group_lanes > 0;  // a group is a power of two of whole lanes
    if (in_lanes) {
      R one = key[0], two = none;
#pragma unroll
      for (int i = 1; i < V; ++i) {
        two = fmax(two, fmin(one, key[i]));
        one = fmax(one, key[i]);
      }
      const auto merge = [&](auto step) {
        R a1, b1, a2, b2;
        exchange_any<decltype(step)::value>(one, a1, b1);
        exchange_any<decltype(step)::value>(two, a2, b2);
        one = fmax(a1, b1);
        two = fmax(fmin(a1, b1), fmax(a2, b2));
      };
      if (a.group_lanes > 1) merge(std::integral_constant<int, 0>());
      if (a.group_lanes > 2) merge(std::integral_constant<int, 1>());
      if (a.group_lanes > 4) merge(std::integral_constant<int, 2>());
      if (a.group_lanes > 8) merge(std::integral_constant<int, 3>());
      if (a.group_lanes > 16) merge(std::integral_constant<int, 4>());
      if (a.group_top == 2 && two > none) one += two;
      if (lane % a.group_lanes == 0 && first < a.E) score[first / n] = one;
      wave_lds_fence();
    } else {
      R* const keys = shared + a.groups;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (first + i < a.E) keys[first + i] = key[i];
      wave_lds_fence();
      for (int g = lane; g < a.groups; g += L) {
        R one = none, two = none;
        for (int i = 0; i < n; ++i) {
          const R k = keys[g * n + i];
          two = fmax(two, fmin(one, k));
          one = fmax(one, k);
        }
        if (a.group_top == 2 && two > none) one += two;
        score[g] = one;
      }
      wave_lds_fence();
    }
    // A group stays if fewer than topk_groups are ahead of it.  The last that stays looks how
    // far the best of those that do not is behind it.
    int last_group = -1;
    bool stays = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = min(first + i, a.E - 1) / n;
      if (g != last_group) {
        last_group = g;
        const R mine = score[g];
        int ahead = 0;
        R behind = none;
        for (int o = 0; o < a.groups; ++o) {
          const R other = score[o];
          const bool better = other > mine || (other == mine && o < g);
          ahead += better;
          if (!better && o != g) behind = fmax(behind, other);
        }
        stays = ahead < a.topk_groups;
        if (kFloat && scored && ahead == a.topk_groups - 1 && behind > none) close |= near(mine, behind, 2);
      }
      if (!stays) keep &= ~(1u << i);
    }
    wave_lds_fence();
  }
  const bool exact = bias == nullptr;  // by logits
  K order[V];
#pragma unroll
  for (int i = 0; i < V; ++i) order[i] = keep >> i & 1 ? order_of(exact ? (R)l[i] : key[i]) : none_key;
  K before = none_key;
  // One more than k, to see how far behind the first that is not chosen is.
  const int rounds = kFloat && !exact ? a.k + 1 : a.k;
  for (int j = 0; j < rounds; ++j) {
    K best = order[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = order[i] > best ? order[i] : best;
    const K all = reduce_max<L>(best);
    if (kFloat && !exact && j > 0 && all > none_key) close |= near(value_of(before), value_of(all), 1);
    before = all;
    const uint64_t have = __builtin_amdgcn_ballot_w64(best == all);
    const int seg = (threadIdx.x & 63) / L * L;
    const uint64_t mine = have >> seg & (~0ull >> (64 - L));
    if (lane == __builtin_ctzll(mine)) {
      int e = -1;
      float le = -INFINITY;
      bool open = true;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool hit = open && order[i] == all;
        if (hit) {
          e = first + i;
          le = l[i];
          order[i] = none_key;
          open = false;
        }
      }
      if (j < a.k) chosen[j] = all > none_key ? Choice{e, le} : Choice{-1, -INFINITY};
    }
  }
  return close;
}

// The weights' shares over the chosen, in lane j for choice j (0 past the last):
// renormalised softmax scores are exp(l - largest); sigmoid scores are taken relative to
// exp(largest) where that is negative.
template <int L>
__device__ __forceinline__ float share_of(const RouteArgs& a, const Choice& c) {
  const bool real = c.expert >= 0 && c.logit > -INFINITY;
  const float top = fmaxf(reduce_max<L>(real ? c.logit : -kMostF32), -kMostF32);
  float s = 0.0f;
  if (real) {
    if (a.softmax) s = expf(c.logit - top);
    else if (c.logit > 0.0f) s = 1.0f / (1.0f + expf(-c.logit));
    else s = expf(c.logit - fminf(top, 0.0f)) / (1.0f + expf(c.logit));
  }
  const float sum = reduce_sum<L>(s);
  return sum > 0.0f ? s / sum : 0.0f;
}
__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

template <int kType, int L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(const void* __restrict__ logits,
                                                         const float* __restrict__ bias, int64_t tokens,
                                                         RouteArgs a, int64_t* __restrict__ idx,
                                                         float* __restrict__ weights) {
  __shared__ Choice choices[kThreads];                    // k <= L of each token
  extern __shared__ __align__(16) double group_memory[];  // a.shared bytes of each token
  const int lane = threadIdx.x % L, local = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / L) + local;
  const int64_t from = t < tokens ? t : tokens - 1;  // (every lane takes part in every exchange)
  float l[V];
  load_logits<kType, V>(logits, from, a.E, lane * V, a.E % V == 0, l);
  Choice* const chosen = choices + local * L;
  char* const shared = reinterpret_cast<char*>(group_memory) + local * a.shared;
  const bool close = choose<float, L, V>(a, l, bias, lane, reinterpret_cast<float*>(shared), chosen);
  if (__builtin_amdgcn_ballot_w64(close) != 0)
    choose<double, L, V>(a, l, bias, lane, reinterpret_cast<double*>(shared), chosen);
  wave_lds_fence();
  const Choice c = lane < a.k ? chosen[lane] : Choice{-1, -INFINITY};
  float w;
  if (a.renormalize) {
    w = share_of<L>(a, c);
  } else if (a.softmax) {
    float top, sum;
    softmax_sums<float, L, V>(l, top, sum);
    w = expf(c.logit - top) / sum;
  } else {
    w = sigmoid_of(c.logit);
  }
  if (t < tokens && lane < a.k) {
    idx[t * a.k + lane] = c.expert;
    weights[t * a.k + lane] = c.expert >= 0 ? w * a.scale : 0.0f;
  }
}

// --------------------------------------------------------------------------
// The gradient by the logits, u_j the shares or scores of the chosen, dw their weights':
//   renormalised   g_j = scale u_j sum_i u_i (dw_j - dw_i)     (sigmoid: times 1 - s_j)
//   softmax        g_j = scale u_j dw_j, and every expert gets -p_e sum_i g_i
//   sigmoid        g_j = scale u_j dw_j (1 - s_j)
// scattered to the experts' places in the order of j, so ids that come twice add up.  The
// sum of differences keeps its digits where one choice has nearly all the weight.
// --------------------------------------------------------------------------
template <int kType, int L, int V>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(const float* __restrict__ dweights,
                                                              const void* __restrict__ logits,
                                                              const int64_t* __restrict__ idx, int64_t tokens,
                                                              RouteArgs a, void* __restrict__ dlogits) {
  constexpr int kTokens = kThreads / L;
  __shared__ float2 pairs[kThreads];  // (share, dw), then (expert, gradient)
  const int lane = threadIdx.x % L, local = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * kTokens + local;
  const int64_t from = t < tokens ? t : tokens - 1;
  float2* const mine = pairs + local * L;
  Choice c = {-1, -INFINITY};
  float dw = 0.0f;
  if (lane < a.k) {
    const int64_t e = idx[from * a.k + lane];
    if (e >= 0 && e < a.E) {
      c = Choice{(int32_t)e, usable(logit_at<kType>(logits, from * a.E + e))};
      dw = c.logit > -INFINITY ? dweights[from * a.k + lane] : 0.0f;
    }
  }
  float l[V];
  const bool dense = a.softmax && !a.renormalize;
  if (dense) load_logits<kType, V>(logits, from, a.E, lane * V, a.E % V == 0, l);
  float g, top = 0.0f, sum = 1.0f, mean = 0.0f;
  if (a.renormalize) {
    const float u = share_of<L>(a, c);
    mine[lane] = float2{u, dw};
    wave_lds_fence();
    g = 0.0f;
    for (int i = 0; i < a.k; ++i) g = fmaf(mine[i].x, dw - mine[i].y, g);
    g *= u * a.scale;
    wave_lds_fence();
  } else if (a.softmax) {
    softmax_sums<float, L, V>(l, top, sum);
    g = dw * (expf(c.logit - top) / sum) * a.scale;
    mean = reduce_sum<L>(g);
  } else {
    g = dw * sigmoid_of(c.logit) * a.scale;
  }
  if (!a.softmax) g = c.logit > -INFINITY ? g / (1.0f + expf(c.logit)) : 0.0f;
  mine[lane] = float2{__int_as_float(c.expert), g};
  wave_lds_fence();
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = dense ? -(expf(l[i] - top) / sum) * mean : 0.0f;
  const int first = lane * V;
  for (int j = 0; j < a.k; ++j) {
    const float2 p = mine[j];
    const int at = __float_as_int(p.x) - first;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] += at == i ? p.y : 0.0f;
  }
  if (t >= tokens) return;
  const int64_t to = t * a.E + first;
  if (a.E % V == 0) {
    if (first >= a.E) return;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if constexpr (kType == EP_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(dlogits) + to + i) = f32x4{d[i], d[i + 1], d[i + 2], d[i + 3]};
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + to + i) =
            uint2{elem_rne2<kType == EP_F16>(d[i], d[i + 1]), elem_rne2<kType == EP_F16>(d[i + 2], d[i + 3])};
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (first + i < a.E) {
        if constexpr (kType == EP_F32) static_cast<float*>(dlogits)[to + i] = d[i];
        else static_cast<uint16_t*>(dlogits)[to + i] = elem_rne<kType == EP_F16>(d[i]);
      }
  }
}

// Lanes of a token: four experts to a lane and at least a lane to a choice; past 64 lanes,
// eight or sixteen experts to a lane.
struct Shape {
  int lanes, experts;
};
Shape shape_of(const RouteArgs& a) {
  if (a.E > 512) return {64, 16};
  if (a.E > 256) return {64, 8};
  int lanes = 8;
  while (lanes * 4 < a.E || lanes < a.k) lanes *= 2;
  return {lanes, 4};
}

template <int kType, typename F>
hipError_t by_shape(const RouteArgs& a, F&& launch) {
  const Shape s = shape_of(a);
  using std::integral_constant;
  const integral_constant<int, kType> type;
  const integral_constant<int, 4> four;
  if (s.experts == 16) return launch(type, integral_constant<int, 64>(), integral_constant<int, 16>());
  if (s.experts == 8) return launch(type, integral_constant<int, 64>(), integral_constant<int, 8>());
  if (s.lanes == 64) return launch(type, integral_constant<int, 64>(), four);
  if (s.lanes == 32) return launch(type, integral_constant<int, 32>(), four);
  if (s.lanes == 16) return launch(type, integral_constant<int, 16>(), four);
  return launch(type, integral_constant<int, 8>(), four);
}
template <typename F>
hipError_t by_type(const RouteArgs& a, int32_t dtype, F&& launch) {
  if (dtype == EP_F32) return by_shape<EP_F32>(a, launch);
  if (dtype == EP_F16) return by_shape<EP_F16>(a, launch);
  return by_shape<EP_BF16>(a, launch);
}

}  // namespace

hipError_t launch_route(const void* logits, const float* bias, int64_t tokens, RouteArgs a, int32_t dtype,
                        int64_t* idx, float* weights, hipStream_t stream) {
  const Shape s = shape_of(a);
  if (a.topk_groups < a.groups) {
    // Groups of whole lanes, a power of two of them, meet by lane exchanges; others in LDS.
    const int n = a.E / a.groups, lanes = n / s.experts;
    if (n % s.experts == 0 && (lanes & (lanes - 1)) == 0) a.group_lanes = lanes;
    a.shared = (a.groups + (a.group_lanes > 0 ? 0 : a.E)) * (int32_t)sizeof(double);
  }
  return by_type(a, dtype, [&](auto type, auto L, auto V) -> hipError_t {
    // (half a workgroup where a token's groups take 16 KiB)
    const int threads = a.shared > (8 << 10) ? kThreads / 2 : kThreads, here = threads / decltype(L)::value;
    const int64_t blocks = (tokens + here - 1) / here;
    if (!grid_fits(blocks, threads)) return hipErrorInvalidValue;
    route_kernel<decltype(type)::value, decltype(L)::value, decltype(V)::value>
        <<<(uint32_t)blocks, threads, a.shared * here, stream>>>(logits, bias, tokens, a, idx, weights);
    return hipGetLastError();
  });
}

hipError_t launch_route_grad(const float* dweights, const void* logits, const int64_t* idx, int64_t tokens,
                             const RouteArgs& a, int32_t dtype, void* dlogits, hipStream_t stream) {
  return by_type(a, dtype, [&](auto type, auto L, auto V) -> hipError_t {
    constexpr int kTokens = kThreads / decltype(L)::value;
    const int64_t blocks = (tokens + kTokens - 1) / kTokens;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidValue;
    route_grad_kernel<decltype(type)::value, decltype(L)::value, decltype(V)::value>
        <<<(uint32_t)blocks, kThreads, 0, stream>>>(dweights, logits, idx, tokens, a, dlogits);
    return hipGetLastError();
  });
}

}  // namespace ep
