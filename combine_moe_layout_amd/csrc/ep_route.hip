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
// The order is that of the keys in fp64.  Logits are compared as they are.  Keys with scores in
// them are made in fp32 first; choices go on past the k-th while the next might belong before it,
// and where two candidates are closer than fp32 can tell (for random logits and biases at 256
// experts one token in 1000), the candidates' keys alone are made again in fp64.  Where that is
// not enough -- groups too close to tell, more candidates than lanes -- the wave does all of
// it in fp64.
//
// Weights over the chosen are taken relative to the largest one, so that they are right also
// where every chosen score underflows.
//
// Bound by the rounds of choosing: a dozen vector instructions of maximum, ballot and removal each,
// with lanes' keys sorted by fours beforehand.  8192 tokens, 256 experts, top-8, fp32: 6.8 us by
// logits, 10.5 with a bias, 12.3 with groups too (11.5 to 13.9 for other logits: a wave that goes to
// fp64 takes 2 us); the reading takes 1.8.  With every near pair redone in fp64 as a whole token, a
// bias took 14.1, where it now took 10.1.  65,536 tokens, 64 experts, top-6: 9.1 us, gradient 8.1.
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
// Experts first .. first + V - 1 of token t; -inf past the last.  `fours`: E is a multiple of 4.
template <int kType, int V>
__device__ __forceinline__ void load_logits(const void* p, int64_t t, int E, int first, bool fours, float (&l)[V]) {
  const int64_t at = t * E + first;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (fours && first + i < E) {
      if constexpr (kType == EP_F32) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at + i);
#pragma unroll
        for (int c = 0; c < 4; ++c) l[i + c] = v[c];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + i);
        l[i] = elem_low<kType == EP_F16>(v.x);
        l[i + 1] = elem_high<kType == EP_F16>(v.x);
        l[i + 2] = elem_low<kType == EP_F16>(v.y);
        l[i + 3] = elem_high<kType == EP_F16>(v.y);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) l[i + c] = first + i + c < E ? logit_at<kType>(p, at + i + c) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = usable(l[i]);
}
template <int V>
__device__ __forceinline__ void load_bias(const float* p, int E, int first, float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = p[min(first + i, E - 1)];
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

// 1 / (1 + exp(-l)), within 2^-22 of itself in float: the hardware's 2^x and reciprocal are each
// within 2^-23, the sum within 2^-24, and the slope takes a quarter of what the exponential is off.
__device__ __forceinline__ float score_sigmoid(float l) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l * -1.44269504088896341f));
}
__device__ __forceinline__ double score_sigmoid(double l) { return 1 / (1 + exp(-l)); }

// Whether two float keys may be in the other order in fp64.  A key is a score and half a step,
// 2^-24 of it, of its sum with the bias.  `unit` covers what two scores are off by: sigmoid scores
// 2^-22 each; softmax scores 2^-18.8 of themselves (the terms and additions, 22 at most, of the sum over
// all experts), two of which are at most 1 and at most twice the largest, 1 / sum.  Groups' scores of
// two keys: see sum_of_two.
__device__ __forceinline__ bool near(float unit, float larger, float smaller, float n) {
  return larger - smaller <= n * (unit + 0x1p-21f * fabsf(larger));
}
__device__ __forceinline__ float near_unit(const RouteArgs& a, float sum) {
  return a.softmax ? 0x1p-18f * fminf(1.0f, 2.0f / sum) : 0x1p-21f;
}

// A group's score of its two largest keys: their sum, in float half of it, which stays in float's range.
// The sum's roundings are 2^-24 (|one| + |two| + |sum|), at most 2^-23 (|two| + |sum|).  Where -two is at
// most 2 |sum| + c, that is 2^-23 (3 |sum| + c) for each of two groups, and `near` of the halves with 3/4
// of a unit and n = 2, 3 units and 2 * 2^-21 |sum| between the sums, has room for it: 1.5 * 2^-21 |sum|, and
// of the units what four scores leave (sigmoid 2^-21, so c = 1; softmax 1.8 units, so c = 2^22 units).
// Otherwise float cannot tell.
template <typename R>
__device__ __forceinline__ R sum_of_two(R one, R two, bool softmax, float unit, bool& unsure) {
  constexpr R kPart = sizeof(R) == 4 ? 0.5 : 1.0;
  if (!(two > -INFINITY)) return kPart * one;
  const R sum = kPart * one + kPart * two;
  if (sizeof(R) == 4 && -two > 4 * fabs(sum) + (softmax ? 0x1p22f * unit : 1.0f)) unsure = true;
  return sum;
}

// A lane's keys in fours, each sorted (neighbours change places, so equal keys stay in the experts'
// order): the best of a lane is the best of the fours' first.
template <typename K, int V>
struct LaneKeys {
  K key[V];
  uint32_t places[V / 4];  // where in its four each sorted key was, a byte each
  __device__ __forceinline__ void prepare() {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      int at[4] = {0, 1, 2, 3};
#pragma unroll
      for (int pass = 3; pass > 0; --pass)
#pragma unroll
        for (int i = 0; i < pass; ++i) {
          const K x = key[q + i], y = key[q + i + 1];
          const int p = at[i];
          const bool swap = y > x;
          key[q + i] = swap ? y : x;
          key[q + i + 1] = swap ? x : y;
          at[i] = swap ? at[i + 1] : p;
          at[i + 1] = swap ? p : at[i + 1];
        }
      places[q / 4] = at[0] | at[1] << 8 | at[2] << 16 | at[3] << 24;
    }
  }
  __device__ __forceinline__ K best() const {
    K k = key[0];
#pragma unroll
    for (int q = 4; q < V; q += 4) k = key[q] > k ? key[q] : k;
    return k;
  }
  // Takes the best key, `k`, out; returns its place in the lane.
  __device__ __forceinline__ int take(K k, K none) {
    int place = 0;
    bool open = true;
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const bool hit = V == 4 || (open && key[q] == k);
      open = open && !hit;
      place = hit ? q + (int)(places[q / 4] & 0xFF) : place;
      places[q / 4] = hit ? places[q / 4] >> 8 : places[q / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) key[q + i] = !hit ? key[q + i] : i < 3 ? key[q + i + 1] : none;
    }
    return place;
  }
};

// One round of choosing: the largest key of a token, and the lowest lane that has it.
template <int L, typename K>
__device__ __forceinline__ K best_of_token(K mine, bool& owner) {
  const K all = reduce_max<L>(mine);
  const uint64_t have = __builtin_amdgcn_ballot_w64(mine == all);
  const int lane = threadIdx.x & 63;
  if constexpr (L == 64) {
    owner = lane == (int)__builtin_ctzll(have);
  } else {  // lanes before this one in the token that have it too
    const uint64_t before = ((1ull << lane) - 1) & (~0ull << (lane / L * L));
    owner = mine == all && (have & before) == 0;
  }
  return all;
}

// The choice with keys of type R (float, or double where float cannot tell), into `chosen`.
// Returns whether float cannot (then `chosen` may be wrong); `wide`: L doubles of the token.
template <typename R, int L, int V>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&l)[V], const float* bias, const float (&bv)[V], int lane,
                                       R* shared, double* wide, int32_t* chosen) {
  using K = std::conditional_t<sizeof(R) == 4, int32_t, int64_t>;
  constexpr bool kFloat = sizeof(R) == 4;
  const R none = -INFINITY;
  const K none_key = order_of(none);
  const int first = lane * V;
  const bool grouped = a.topk_groups < a.groups, exact = bias == nullptr;  // exact: by logits
  LaneKeys<K, V> keys;
  uint32_t keep = (1u << V) - 1;  // experts in groups that stay
  bool unsure = false;
  R key[V];
  const bool scored = !exact || (grouped && a.group_top == 2);
  float unit = 0.0f;
  if (scored) {
    R top = 0, sum = 1;
    if (a.softmax) softmax_sums<R, L, V>(l, top, sum);
    unit = near_unit(a, (float)sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      R k = a.softmax ? exp_of((R)l[i] - top) / sum : score_sigmoid((R)l[i]);
      if (!exact) k += (R)bv[i];
      key[i] = l[i] > -INFINITY && k > none ? k : none;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = l[i];
  }
  if (grouped) {
    R* const score = shared;  // [groups]: the largest key, or the sum of the two largest
    const float group_unit = a.group_top == 2 ? 0.75f * unit : unit, group_n = a.group_top == 2 ? 2.0f : 1.0f;
    // Whether group g stays: fewer than topk_groups are ahead of it.  The last that stays looks
    // how far the best of those that do not is behind it.
    const auto stays = [&](int g, R mine) {
      int ahead = 0;
      R behind = none;
      for (int o = 0; o < a.groups; ++o) {
        const R other = score[o];
        const bool better = other > mine || (other == mine && o < g);
        ahead += better;
        if (!better && o != g) behind = fmax(behind, other);
      }
      if (kFloat && scored && ahead == a.topk_groups - 1 && behind > none)
        unsure |= near(group_unit, (float)mine, (float)behind, group_n);
      return ahead < a.topk_groups;
    };
    if (a.group_shift >= 0) {  // a group is 2^group_shift whole lanes
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
      if (a.group_shift > 0) merge(std::integral_constant<int, 0>());
      if (a.group_shift > 1) merge(std::integral_constant<int, 1>());
      if (a.group_shift > 2) merge(std::integral_constant<int, 2>());
      if (a.group_shift > 3) merge(std::integral_constant<int, 3>());
      if (a.group_shift > 4) merge(std::integral_constant<int, 4>());
      if (a.group_top == 2) one = sum_of_two(one, two, a.softmax, unit, unsure);
      const int g = lane >> a.group_shift;
      if (g < a.groups && lane == g << a.group_shift) score[g] = one;
      wave_lds_fence();
      if (!stays(g, one)) keep = 0;
    } else {
      const int n = a.E / a.groups;
      R* const all = shared + a.groups;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (first + i < a.E) all[first + i] = key[i];
      wave_lds_fence();
      for (int g = lane; g < a.groups; g += L) {
        R one = none, two = none;
        for (int i = 0; i < n; ++i) {
          const R k = all[g * n + i];
          two = fmax(two, fmin(one, k));
          one = fmax(one, k);
        }
        if (a.group_top == 2) one = sum_of_two(one, two, a.softmax, unit, unsure);
        score[g] = one;
      }
      wave_lds_fence();
      int group = -1;
      bool stay = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = min(first + i, a.E - 1) / n;
        if (g != group) {
          group = g;
          stay = stays(g, score[g]);
        }
        if (!stay) keep &= ~(1u << i);
      }
    }
    wave_lds_fence();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) keys.key[i] = keep >> i & 1 ? order_of(exact ? (R)l[i] : key[i]) : none_key;
  keys.prepare();
  bool owner;
  if (!kFloat || exact) {
    for (int j = 0; j < a.k; ++j) {
      const K all = best_of_token<L>(keys.best(), owner);
      if (owner) chosen[j] = all > none_key ? first + keys.take(all, none_key) : -1;
    }
    return unsure;
  }
  // The k largest, and those after them that may belong before the k-th in fp64.
  K kept = none_key, last = none_key;  // of choice `lane`, of choice k - 1
  int count = a.k;
  for (int j = 0;; ++j) {
    const K all = best_of_token<L>(keys.best(), owner);
    if (j >= a.k) {
      const bool more = all > none_key && near(unit, (float)value_of(last), (float)value_of(all), 1.0f);
      if (__builtin_amdgcn_ballot_w64(more) == 0) break;
      if (j >= L) {  // (L choices at most)
        unsure |= more;
        break;
      }
      if (!more) owner = false;
      count = more ? j + 1 : count;
    } else {
      last = all;
    }
    if (owner) chosen[j] = all > none_key ? first + keys.take(all, none_key) : -1;
    if (lane == j) kept = all;
  }
  const K before = (K)__shfl_up((int)kept, 1);
  const bool close = lane > 0 && lane < count && kept > none_key &&
                     near(unit, (float)value_of(before), (float)value_of(kept), 1.0f);
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(close) == 0, 1)) return unsure;
  // Again in fp64, for the candidates alone: a lane takes one and finds its place.
  double top = 0, sum = 1;
  if (a.softmax) softmax_sums<double, L, V>(l, top, sum);
  wave_lds_fence();
  const int e = lane < count ? chosen[lane] : -1;
  const int from = max(e, 0) / V;  // its logit is in that lane of the token, at place e % V
  float le = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float v = __shfl(l[i], from, L);
    le = max(e, 0) % V == i ? v : le;
  }
  double k = -INFINITY;
  if (e >= 0) k = (a.softmax ? exp((double)le - top) / sum : score_sigmoid((double)le)) + (double)bias[e];
  wide[lane] = k;
  wave_lds_fence();
  int place = 0;
  for (int i = 0; i < count; ++i) {
    const double other = wide[i];
    const int id = chosen[i];
    place += id >= 0 && (other > k || (other == k && id < e));
  }
  wave_lds_fence();
  if (e >= 0 && place < a.k) chosen[place] = e;  // (missing choices are behind all others already)
  return unsure;
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
  __shared__ int32_t choices[kThreads];                   // up to L of each token
  __shared__ double wide[kThreads];
  extern __shared__ __align__(16) double group_memory[];  // a.shared bytes of each token
  const int lane = threadIdx.x % L, local = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / L) + local;
  const int64_t from = t < tokens ? t : tokens - 1;  // (every lane takes part in every exchange)
  float bv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bv[i] = 0.0f;
  if (bias != nullptr) load_bias<V>(bias, a.E, lane * V, bv);
  float l[V];
  load_logits<kType, V>(logits, from, a.E, lane * V, a.E % 4 == 0, l);
  int32_t* const chosen = choices + local * L;
  char* const shared = reinterpret_cast<char*>(group_memory) + local * a.shared;
  const bool unsure = choose<float, L, V>(a, l, bias, bv, lane, reinterpret_cast<float*>(shared), wide + local * L, chosen);
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(unsure) != 0, 0))
    choose<double, L, V>(a, l, bias, bv, lane, reinterpret_cast<double*>(shared), wide + local * L, chosen);
  wave_lds_fence();
  Choice c = {lane < a.k ? chosen[lane] : -1, -INFINITY};
  if (c.expert >= 0) c.logit = usable(logit_at<kType>(logits, from * a.E + c.expert));
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
//   softmax        g_j = scale u_j (sum_i u_i (dw_j - dw_i) + q dw_j),  q = the shares of those not
//                  chosen, each of which gets -scale p_e sum_i u_i dw_i
//   sigmoid        g_j = scale u_j dw_j (1 - s_j)
// brought to the experts' places through LDS; an id that comes twice has its sum in order.  Sums of
// differences, and q as a sum of its own, keep their digits where the chosen have nearly all the weight.
// --------------------------------------------------------------------------
// kDense: softmax without renormalisation.  (65,536 tokens of 64 experts: 10.7 us, the others 8.1; in one
// kernel 11.1 and 8.4.)
template <bool kDense, int kType, int L, int V>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(const float* __restrict__ dweights,
                                                              const void* __restrict__ logits,
                                                              const int64_t* __restrict__ idx, int64_t tokens,
                                                              RouteArgs a, void* __restrict__ dlogits) {
  constexpr int kTokens = kThreads / L;
  __shared__ float2 pairs[kThreads];  // (share, dw), then (expert, gradient)
  __shared__ __align__(16) float rows[kThreads * V];
  const int lane = threadIdx.x % L, local = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * kTokens + local;
  const int64_t from = t < tokens ? t : tokens - 1;
  float2* const mine = pairs + local * L;
  // (One branch: behind one for each load the kernel's arguments came one by one too, 0.4 us.)
  Choice c = {-1, -INFINITY};
  float dw = 0.0f;
  if (lane < a.k) {
    const int64_t pair = from * a.k + lane, e = idx[pair];
    const float given = dweights[pair];
    const bool known = e >= 0 && e < a.E;
    const float logit = usable(logit_at<kType>(logits, from * a.E + (known ? e : 0)));
    if (known) c = Choice{(int32_t)e, logit};
    if (c.logit > -INFINITY) dw = given;
  }
  // The sum of `v` over an expert's entries, and whether this is the first of them.
  const auto by_expert = [&](float v, bool& first_entry) {
    mine[lane] = float2{__int_as_float(c.expert), v};
    wave_lds_fence();
    float total = 0.0f;
    first_entry = c.expert >= 0;
    for (int j = 0; j < a.k; ++j) {
      const float2 p = mine[j];
      const bool same = __float_as_int(p.x) == c.expert;
      total += same ? p.y : 0.0f;
      first_entry = first_entry && !(same && j < lane);
    }
    return total;
  };
  // sum_i u_i (dw - dw_i) of lanes' pairs
  const auto differences = [&](float u, float dw_of) {
    mine[lane] = float2{u, dw_of};
    wave_lds_fence();
    float sum = 0.0f;
    for (int i = 0; i < a.k; ++i) sum = fmaf(mine[i].x, dw_of - mine[i].y, sum);
    wave_lds_fence();
    return sum;
  };
  float* const row = rows + local * (L * V);
  const auto clear_row = [&] {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<f32x4*>(row + lane * V + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  float others[V];  // kDense: gradients of the experts that are not chosen
  float g;
  bool first_entry;
  if constexpr (kDense) {
    clear_row();
    const float total = by_expert(dw, first_entry);
    if (first_entry) row[c.expert] = 1.0f;
    load_logits<kType, V>(logits, from, a.E, lane * V, a.E % 4 == 0, others);
    float top, sum, rest = 0.0f;
    softmax_sums<float, L, V>(others, top, sum);
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      others[i] = row[lane * V + i] != 0.0f ? 0.0f : expf(others[i] - top) / sum;
      rest += others[i];
    }
    rest = reduce_sum<L>(rest);
    const float u = first_entry ? expf(c.logit - top) / sum : 0.0f;
    const float mean = reduce_sum<L>(u * total) * a.scale;
    g = fmaf(rest, total, differences(u, total)) * u * a.scale;
#pragma unroll
    for (int i = 0; i < V; ++i) others[i] *= -mean;
  } else {
    if (a.renormalize) {
      const float u = share_of<L>(a, c);
      g = differences(u, dw) * (u * a.scale);
    } else {
      g = dw * sigmoid_of(c.logit) * a.scale;
    }
    if (!a.softmax) g = c.logit > -INFINITY ? g / (1.0f + expf(c.logit)) : 0.0f;
    clear_row();
    g = by_expert(g, first_entry);
  }
  if (first_entry) row[c.expert] = g;
  wave_lds_fence();
  const int first = lane * V;
  const int64_t to = t * a.E + first;
  if (t >= tokens) return;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    f32x4 d = *reinterpret_cast<const f32x4*>(row + first + i);
    if constexpr (kDense) {
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) d[c4] += others[i + c4];
    }
    if (first + i >= a.E) continue;
    if (a.E % 4 == 0) {
      if constexpr (kType == EP_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(dlogits) + to + i) = d;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + to + i) =
            uint2{elem_rne2<kType == EP_F16>(d[0], d[1]), elem_rne2<kType == EP_F16>(d[2], d[3])};
      }
    } else {
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4)
        if (first + i + c4 < a.E) {
          if constexpr (kType == EP_F32) static_cast<float*>(dlogits)[to + i + c4] = d[c4];
          else static_cast<uint16_t*>(dlogits)[to + i + c4] = elem_rne<kType == EP_F16>(d[c4]);
        }
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
    if (n % s.experts == 0 && (lanes & (lanes - 1)) == 0) a.group_shift = __builtin_ctz(lanes);
    a.shared = (a.groups + (a.group_shift >= 0 ? 0 : a.E)) * (int32_t)sizeof(double);
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
    const auto run = [&](auto kernel) {
      kernel<<<(uint32_t)blocks, kThreads, 0, stream>>>(dweights, logits, idx, tokens, a, dlogits);
    };
    if (a.softmax && !a.renormalize)
      run(route_grad_kernel<true, decltype(type)::value, decltype(L)::value, decltype(V)::value>);
    else
      run(route_grad_kernel<false, decltype(type)::value, decltype(L)::value, decltype(V)::value>);
    return hipGetLastError();
  });
}

}  // namespace ep
