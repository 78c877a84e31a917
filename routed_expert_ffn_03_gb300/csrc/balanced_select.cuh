// balanced_select.cuh - one token's experts by a warp: scores with a bias for balance, limited to groups of experts.
//
//   s_e = softmax or sigmoid of the logits,  c_e = s_e + b_e;  a group's score: its largest c, or the sum of its two largest;
//   the `keep` best groups stay, and of their experts the k with the largest c (without a bias: logits) are selected.
//
// Experts are chosen as if scores were compared in 64 bits, so that the choice does not depend on how fp32 rounds an
// exponential.  Scores are fp32 first, with a bound on their error; only where two neighbours in the order are closer than
// that are they computed again in fp64: of one token in some thousands, for the candidates alone, one a lane.  (fp64 runs at a
// 64th of fp32's rate: all of 256 scores take 4 us.)  Where that does not decide it (a group's own best that close, more
// candidates than lanes, scores that underflow) all of the token's scores are.
#pragma once
#include "group_sort.cuh"
#include "route.cuh"

namespace moe {

constexpr int MAX_EXPERTS = 1024;

// What a block keeps of the bias and the groups: biases as they count (NaN and -inf: the expert is masked; +inf: the largest
// finite), and each expert's group.
struct BalancedTables {
  float bias[MAX_EXPERTS];
  uint8_t group[MAX_EXPERTS];
  int set;   // whether any bias is not 0
};

__device__ __forceinline__ void balanced_tables(const BalancedRouteArgs& a, BalancedTables& tab) {
  const int size = a.E / a.groups;
  bool set = false;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    const float b = a.bias ? clean(__ldg(a.bias + e)) : 0.f;
    tab.bias[e] = b;
    tab.group[e] = (uint8_t)(e / size);
    set |= b != 0.f;
  }
  set = __syncthreads_or(set);
  if (threadIdx.x == 0) tab.set = set;
}
// Whether different logits have different scores (the largest being m): a sigmoid near 1 and a softmax beside an infinite logit have not.
__device__ __forceinline__ bool scores_tell(const BalancedRouteArgs& a, float m) { return m < (a.kind == 1 ? 20.f : 1e30f); }
// Whether a token's experts are ordered by their biased scores.  Without a bias, and with biases that are all 0 (as training starts;
// there 16-bit logits are often equal), they are ordered by their logits, which is the scores' order.  Groups' scores likewise, where
// they are not sums.
__device__ __forceinline__ bool by_biased(const BalancedRouteArgs& a, const BalancedTables& tab, float m) {
  return a.bias && (tab.set || !scores_tell(a, m));
}

__device__ __forceinline__ float key_value(uint32_t k) { return k ? key_logit(k) : -INFINITY; }
__device__ __forceinline__ float warp_max_f(float v) { return key_value(__reduce_max_sync(0xffffffffu, v > -INFINITY ? logit_key(v) : 0u)); }

// order-preserving key of a number (not NaN; -0 below +0), two instructions
__device__ __forceinline__ uint32_t quick_key(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
// e^x within 2 + 1.2 |x| steps, and 1 / x within one; results below 2^-126 are 0
__device__ __forceinline__ float quick_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float quick_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Each register's two largest keys over the warp, all registers at once: the first steps of the butterfly halve the registers instead
// of reducing each (NV = 8: 60 instructions, where two reductions a register take 240).  Lane register_lane(r) receives register r's.
template <int NV>
__device__ __forceinline__ void two_largest(const uint32_t (&key)[NV], int lane, uint32_t& b1, uint32_t& b2) {
  uint32_t x1[NV], x2[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x1[i] = key[i];
    x2[i] = 0;
  }
  int o = 16;
#pragma unroll
  for (int n = NV / 2; n >= 1; n /= 2, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t k1 = upper ? x1[i + n] : x1[i], s1 = upper ? x1[i] : x1[i + n];
      const uint32_t r1 = __shfl_xor_sync(0xffffffffu, s1, o);
      if (n == NV / 2) {
        x2[i] = min(k1, r1);
      } else {
        const uint32_t k2 = upper ? x2[i + n] : x2[i], s2 = upper ? x2[i] : x2[i + n];
        x2[i] = max(min(k1, r1), max(k2, __shfl_xor_sync(0xffffffffu, s2, o)));
      }
      x1[i] = max(k1, r1);
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) {
    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, x1[0], o), r2 = __shfl_xor_sync(0xffffffffu, x2[0], o);
    x2[0] = max(min(x1[0], r1), max(x2[0], r2));
    x1[0] = max(x1[0], r1);
  }
  b1 = x1[0];
  b2 = x2[0];
}
template <int NV>
__device__ __forceinline__ int register_lane(int r) {   // the s-th step, across lanes 16 >> s, chose by bit log2(NV) - 1 - s
  return NV == 4 ? r << 3 : NV == 8 ? r << 2 : NV == 16 ? r << 1 : r;
}

// the kept groups as bits: the best of lane g's score of group g (-inf: none), equal ones the lower first
__device__ __forceinline__ unsigned kept_groups(double score, int groups, int keep, int lane) {
  int rank = 0;
  for (int q = 0; q < groups; ++q) {
    const double o = __shfl_sync(0xffffffffu, score, q);
    rank += o > score || (o == score && q < lane);
  }
  return __ballot_sync(0xffffffffu, lane < groups && rank < keep && score > -INFINITY);
}

// sum over the token's experts of e^(l - m), in 64 bits
static __device__ __noinline__ double exact_total(const BalancedRouteArgs& a, long long t, int lane, float m) {
  double z = 0.0;
  for (int e = lane; e < a.E; e += 32) {
    const float l = logit_of(a, t, e);
    if (l > -INFINITY) z += exp((double)l - (double)m);
  }
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
__device__ __forceinline__ double exact_score(const BalancedRouteArgs& a, float l, float m, double z) {
  return a.kind == 1 ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
}

// The whole selection in 64 bits: lane j < k receives the j-th expert, or -1.
template <int NV>
static __device__ __noinline__ int exact_select(const BalancedRouteArgs& a, const BalancedTables& tab, long long t, int lane, float m) {
  double c[NV];
  const double z = a.kind == 0 ? exact_total(a, t, lane, m) : 1.0;
  const bool by_bias = by_biased(a, tab, m), scores = by_bias || a.top2 || !scores_tell(a, m);
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    c[i] = -INFINITY;
    if (e < a.E) {
      const float l = logit_of(a, t, e), b = tab.bias[e];
      if (l > -INFINITY && b > -INFINITY) c[i] = scores ? exact_score(a, l, m, z) + (double)b : (double)l;
    }
  }
  unsigned kept = ~0u;
  if (a.keep < a.groups) {
    double score = -INFINITY;
    for (int g = 0; g < a.groups; ++g) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && tab.group[e] == g) {
          b2 = fmax(b2, fmin(b1, c[i]));
          b1 = fmax(b1, c[i]);
        }
      }
      for (int o = 16; o; o >>= 1) {
        const double x1 = __shfl_xor_sync(0xffffffffu, b1, o), x2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = fmax(fmax(b2, x2), fmin(b1, x1));
        b1 = fmax(b1, x1);
      }
      if (lane == g) score = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
    kept = kept_groups(score, a.groups, a.keep, lane);
  }
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.E || !((kept >> (tab.group[e] & 31)) & 1u)) c[i] = -INFINITY;
    else if (!by_bias && c[i] > -INFINITY) c[i] = logit_of(a, t, e);
  }
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = 0x7fffffff;
    for (int i = 0; i < NV; ++i)
      if (c[i] > best) {
        best = c[i];
        at = lane + 32 * i;
      }
    for (int o = 16; o; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > -INFINITY)) break;   // uniform
    if (lane == j) mine = at;
    if ((at & 31) == lane) c[at >> 5] = -INFINITY;
  }
  return mine;
}

constexpr int UNSETTLED = -2;

// Which `need` of the groups `open` stay, where fp32 leaves it so, by the 64-bit scores of each one's best one or two experts (all of the
// token's scores in 64 bits take some 10 us).  NO_GROUPS where a group's own best are too close to tell, too.
constexpr unsigned NO_GROUPS = 0;
static __device__ __noinline__ unsigned settle_groups(const BalancedRouteArgs& a, const BalancedTables& tab, long long t, int lane, unsigned open,
                                                      int need, float m, float inv, float err) {
  const int size = a.E / a.groups, best = a.top2 ? 2 : 1;
  auto apart = [&](float p, float q) { return p - q > 2.f * err + 0x1p-22f * fmaxf(fabsf(p), fabsf(q)); };
  int my_e[2] = {-1, -1};
  for (unsigned left = open; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    int e[2] = {-1, -1};
    float c[3] = {-INFINITY, -INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
    bool skipped = false;
    // the best one or two, and the best of the others; one of the same logit and bias as the least of those does not change the score, as
    // long as the best is no less than they are
    for (int r = 0; r <= best; ++r) {
      uint32_t key = 0;
      int at = 0x7fffffff;
      for (int q = g * size + lane; q < (g + 1) * size; q += 32) {
        const float x = logit_of(a, t, q), y = tab.bias[q];
        if (!(x > -INFINITY) || !(y > -INFINITY) || q == e[0] || q == e[1]) continue;
        if (r == best && x == l[best - 1] && y == b[best - 1]) {
          skipped = true;
          continue;
        }
        const uint32_t k = logit_key((a.kind == 1 ? quick_inverse(1.f + quick_exp(-x)) : quick_exp(x - m) * inv) + y);
        if (k > key) {
          key = k;
          at = q;
        }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, key);
      if (top == 0) break;   // uniform
      at = (int)__reduce_min_sync(0xffffffffu, key == top ? (unsigned)at : 0x7fffffffu);
      c[r] = key_value(top);
      if (r < best) {
        e[r] = at;
        l[r] = logit_of(a, t, at);
        b[r] = tab.bias[at];
      }
    }
    skipped = __any_sync(0xffffffffu, skipped);
    if ((c[best] > -INFINITY && !apart(c[best - 1], c[best])) ||
        (best == 2 && skipped && !apart(c[0], c[1]) && !(l[0] == l[1] && b[0] == b[1])))
      return NO_GROUPS;
    if (lane == g) {
      my_e[0] = e[0];
      my_e[1] = e[1];
    }
  }
  // (without a bias the softmax's sum is common to all)
  const double z = a.kind == 0 && tab.set ? exact_total(a, t, lane, m) : 1.0;
  double score = -INFINITY;
  for (int i = 0; i < best; ++i)
    if (my_e[i] >= 0) {
      const double v = exact_score(a, logit_of(a, t, my_e[i]), m, z) + (double)tab.bias[my_e[i]];
      score = i ? score + v : v;
    }
  int rank = 0;
  for (unsigned left = open; left; left &= left - 1) {
    const int q = __ffs(left) - 1;
    const double o = __shfl_sync(0xffffffffu, score, q);
    rank += o > score || (o == score && q < lane);
  }
  return __ballot_sync(0xffffffffu, ((open >> lane) & 1u) && rank < need);
}

// The order of a token's selected experts (lane j: the j-th, e; -1 from n on), where their keys leave it open.  The candidates, one a lane:
// the selected, and the others that are not below the least of them by more than the errors; those of the last one's logit and bias
// are left out where all the selected are no less than it (of equal ones the lower was taken).  By fp32 values first; where those are closer than their errors, and not of the
// same logit and bias, by 64 bits.  All lanes UNSETTLED where there are more candidates than lanes.
static __device__ __noinline__ int settle(const BalancedRouteArgs& a, const BalancedTables& tab, long long t, int lane, int e, unsigned kept,
                                          float m, float inv, float err) {
  const bool by_bias = by_biased(a, tab, m);
  auto score = [&](float l, float b) {
    return by_bias ? (a.kind == 1 ? quick_inverse(1.f + quick_exp(-l)) : quick_exp(l - m) * inv) + b : l;
  };
  const int n = __popc(__ballot_sync(0xffffffffu, e >= 0));
  const float my_l = e >= 0 ? logit_of(a, t, e) : INFINITY, my_b = e >= 0 ? tab.bias[e] : 0.f;
  const float l_last = __shfl_sync(0xffffffffu, my_l, n - 1), b_last = __shfl_sync(0xffffffffu, my_b, n - 1);
  const float least = -warp_max_f(e >= 0 ? -score(my_l, my_b) : -INFINITY);
  const float limit = least - (by_bias ? 2.f * err + 0x1p-21f * fabsf(least) : 0.f);
  if (!(limit > -INFINITY)) return UNSETTLED;
  const float c_last = score(l_last, b_last);
  const bool above = __all_sync(0xffffffffu, e < 0 || (my_l == l_last && my_b == b_last) ||
                                                 score(my_l, my_b) - c_last > (by_bias ? 2.f * err + 0x1p-21f * fmaxf(fabsf(c_last), fabsf(least)) : 0.f));
  int count = n;
  for (int i0 = 0; i0 < a.E; i0 += 32) {
    const int q = i0 + lane;
    const unsigned selected = __reduce_or_sync(0xffffffffu, lane < n && (e >> 5) == (i0 >> 5) ? 1u << (e & 31) : 0u);
    bool in = false;
    if (q < a.E && !((selected >> lane) & 1u) && ((kept >> (tab.group[q] & 31)) & 1u)) {
      const float l = logit_of(a, t, q), c = score(l, tab.bias[q]);
      in = l > -INFINITY && c >= limit && !(above && l == l_last && tab.bias[q] == b_last);
    }
    unsigned who = __ballot_sync(0xffffffffu, in);
    for (; who && count <= 32; who &= who - 1, ++count)
      if (lane == count) e = i0 + __ffs(who) - 1;
  }
  if (count > 32) return UNSETTLED;
  const bool live = lane < count;
  const float l = live ? logit_of(a, t, e) : -INFINITY, b = live ? tab.bias[e] : 0.f;
  double v = live ? score(l, b) : -INFINITY;
  auto order = [&]() {   // this lane's place among the candidates
    int rank = 0;
    for (int q = 0; q < count; ++q) {
      const double o = __shfl_sync(0xffffffffu, v, q);
      const int oe = __shfl_sync(0xffffffffu, e, q);
      rank += o > v || (o == v && oe < e);
    }
    return rank;
  };
  int rank = order();
  if (by_bias) {
    bool close = false;
    const float f = (float)v;
    for (int q = 0; q < count; ++q) {
      const float o = __shfl_sync(0xffffffffu, f, q), ol = __shfl_sync(0xffffffffu, l, q), ob = __shfl_sync(0xffffffffu, b, q);
      close |= q != lane && !(fabsf(o - f) > 2.f * err + 0x1p-22f * fabsf(o)) && !(ol == l && ob == b);
    }
    if (__any_sync(0xffffffffu, live && close)) {
      const double z = a.kind == 0 ? exact_total(a, t, lane, m) : 1.0;
      if (live) v = exact_score(a, l, m, z) + (double)b;
      rank = order();
    }
  }
  int from = -1;
  for (int q = 0; q < count; ++q)
    if (__shfl_sync(0xffffffffu, rank, q) == lane) from = q;
  const int sorted = __shfl_sync(0xffffffffu, e, max(from, 0));
  return from >= 0 && lane < a.k ? sorted : -1;
}

// kept_groups of fp32 scores by rounds of the warp's maximum (or minimum, where fewer groups go than stay); and the least kept and the
// largest other score (-inf: none).
__device__ __forceinline__ unsigned kept_by_rounds(float score, int groups, int keep, int lane, float& last, float& next) {
  const uint32_t key = lane < groups && score > -INFINITY ? logit_key(score) : 0u;
  unsigned kept = 0;
  if (2 * keep <= groups) {
    uint32_t rest = key, b = 0;
    for (int j = 0; j < keep; ++j) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, rest);
      if (best == 0) break;   // uniform
      b = best;
      const int who = __ffs(__ballot_sync(0xffffffffu, rest == best)) - 1;
      kept |= 1u << who;
      if (lane == who) rest = 0;
    }
    last = key_value(b);
    next = key_value(__reduce_max_sync(0xffffffffu, rest));
  } else {
    uint32_t rest = lane < groups ? key : 0xffffffffu, b = 0;
    unsigned gone = 0;
    for (int j = keep; j < groups; ++j) {
      b = __reduce_min_sync(0xffffffffu, rest);
      const int who = 31 - __clz(__ballot_sync(0xffffffffu, rest == b));   // of equal ones the last goes first
      gone |= 1u << who;
      if (lane == who) rest = 0xffffffffu;
    }
    kept = __ballot_sync(0xffffffffu, key != 0) & ~gone;
    last = key_value(__reduce_min_sync(0xffffffffu, key && ((kept >> lane) & 1u) ? key : 0xffffffffu));
    next = key_value(b);
  }
  return kept;
}

// The first n <= 33 keys in descending order (0: none left), lane j the j-th and `last` the 33rd; each key is unique.  A round takes
// the largest of the lanes' firsts, and the lane that held it steps to its second and third; where a lane gave all three, the
// warp starts again with rounds in which that lane looks through its keys.
template <int NV>
__device__ __forceinline__ uint32_t ordered_keys(const uint32_t (&key)[NV], int n, int lane, uint32_t& behind) {
  uint32_t b1 = 0, b2 = 0, b3 = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t x = min(b1, key[i]), y = min(b2, x);
    b1 = max(b1, key[i]);
    b2 = max(b2, x);
    b3 = max(b3, y);
  }
  const bool three = b3 != 0;
  const uint32_t best0 = b1;
  behind = 0;
  for (int j = 0; j < n; ++j) {
    const uint32_t b = __reduce_max_sync(0xffffffffu, b1);
    if (lane == j) mine = b;
    if (j == n - 1) behind = b;
    if (b1 == b) {
      b1 = b2;
      b2 = b3;
      b3 = 0;
    }
  }
  if (NV > 3 && __any_sync(0xffffffffu, three && b1 == 0)) {
    uint32_t best = best0, floor = 0xffffffffu;   // this lane's keys from `floor` on are taken
    mine = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t b = __reduce_max_sync(0xffffffffu, best);
      if (lane == j) mine = b;
      if (j == n - 1) behind = b;
      if (best == b && b) {
        floor = b;
        best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = max(best, key[i] < floor ? key[i] : 0u);
      }
    }
  }
  return mine;
}

// A group's score from its two largest.  Biases near the type's limits (the lowest value as a mask) would leave fp32 with it, and a
// group at -inf counts as empty; those that meet at the limit are told apart in 64 bits, as any that are close.
__device__ __forceinline__ float group_sum(float b1, float b2) {
  constexpr float MOST = 3.402823466e38f;
  return fminf(fmaxf(b1 + b2, -MOST), MOST);
}

// The selection of token t: lane j < k receives the j-th expert (-1: none) and its weight.  x: lane l's logits of experts
// l + 32 i (-inf, NaN: masked; -inf past the experts).
template <int NV>
__device__ __forceinline__ void balanced_token(const BalancedRouteArgs& a, const BalancedTables& tab, long long t, int lane,
                                               float (&x)[NV], int& my_e, float& my_w) {
  const bool limited = a.keep < a.groups;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);   // (NaN is passed over; no comparison below takes it)
  float m = warp_max_f(top);   // the largest logit
  if (m == INFINITY) {
    m = 3.402823466e38f;
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = x[i] == INFINITY ? m : x[i];
  }
  const bool by_bias = by_biased(a, tab, m), by_score = by_bias || (limited && (a.top2 || !scores_tell(a, m)));   // else logits are compared
  float inv = 1.f, err = 0.f;        // softmax: one over the sum; the scores' absolute error
  uint32_t key[NV];                  // by which experts are compared
  if (a.kind == 0 && (by_score || !a.renorm)) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float p = x[i] > -INFINITY ? quick_exp(x[i] - m) : 0.f;
      key[i] = __float_as_uint(p);
      z += p;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    inv = 1.f / z;
    // e^-d is within 2 + 1.2 d steps of itself, 2 steps of the largest; so are the sum's terms, and its NV + 5 additions
    // and two products a step each
    err = (NV + 20) * 0x1p-23f * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float c = __uint_as_float(key[i]) * inv + tab.bias[lane + 32 * i];
      key[i] = x[i] > -INFINITY && c > -INFINITY ? quick_key(c) : 0u;
    }
  } else if (by_score && a.kind == 1) {
    // the derivative by e^-l is s (1 - s): 2 + 1.2 |l| steps of it are 0.6 steps of 1 for l >= 0, and 2 + 1.2 |m| of the largest score
    // where all logits are below 0; the sum and the division two more
    err = 0x1p-23f * (4.f + 2.f * fmaxf(-m, 0.f)) / (1.f + __expf(-m));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float c = quick_inverse(1.f + quick_exp(-x[i])) + tab.bias[lane + 32 * i];
      key[i] = x[i] > -INFINITY && c > -INFINITY ? quick_key(c) : 0u;   // (c is never -0)
    }
  }
  if (!by_score) {   // (with a bias here it is 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = x[i] > -INFINITY ? logit_key(x[i]) : 0u;
  }
  // sigmoids below 2^-100 lose bits
  bool doubt = by_score && a.kind == 1 && m < -69.f && m > -INFINITY;
  unsigned kept = ~0u;
  if (limited) {
    float score = -INFINITY;
    auto finish = [&](int g, uint32_t b1, uint32_t b2) {   // a group's score from the lanes' two largest
      const uint32_t w1 = __reduce_max_sync(0xffffffffu, b1);
      float v = key_value(w1);
      if (a.top2 && w1) {
        const int first = __ffs(__ballot_sync(0xffffffffu, b1 == w1)) - 1;
        const uint32_t w2 = __reduce_max_sync(0xffffffffu, lane == first ? b2 : b1);
        if (w2) v = group_sum(v, key_value(w2));
      }
      if (lane == g) score = v;
    };
    const int size = a.E / a.groups, per = size / 32;
    const bool whole = size % 32 == 0;   // a group is whole registers
    if (whole) {
      uint32_t r1, r2, b1 = 0, b2 = 0;
      two_largest<NV>(key, lane, r1, r2);
      for (int q = 0; q < per; ++q) {
        const int from = register_lane<NV>((lane * per + q) & (NV - 1));
        const uint32_t o1 = __shfl_sync(0xffffffffu, r1, from), o2 = __shfl_sync(0xffffffffu, r2, from);
        b2 = max(min(b1, o1), max(b2, o2));
        b1 = max(b1, o1);
      }
      if (lane < a.groups) {
        score = key_value(b1);
        if (a.top2 && b2) score = group_sum(score, key_value(b2));
      }
    } else {
      for (int g = 0; g < a.groups; ++g) {
        uint32_t b1 = 0, b2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t k = (unsigned)(lane + 32 * i - g * size) < (unsigned)size ? key[i] : 0u;
          b2 = max(b2, min(b1, k));
          b1 = max(b1, k);
        }
        finish(g, b1, b2);
      }
    }
    float last, next;
    kept = kept_by_rounds(score, a.groups, a.keep, lane, last, next);
    // two scores a group, and the roundings of their sums with the biases and each other
    const float near = 4.f * err + 0x1p-21f * fmaxf(fabsf(last), fabsf(next));
    if (by_score && next > -INFINITY && !(last - next > near) && !doubt) {
      const bool in = (kept >> lane) & 1u;
      const unsigned sure = __ballot_sync(0xffffffffu, in && score - next > near);
      const unsigned open = __ballot_sync(0xffffffffu, lane < a.groups && score > -INFINITY && (in ? !(score - next > near) : !(last - score > near)));
      const unsigned more = settle_groups(a, tab, t, lane, open, __popc(kept) - __popc(sure), m, inv, err);
      doubt = more == NO_GROUPS;
      kept = sure | more;
    }
    unsigned stay = kept;   // by register, whole groups
    if (whole && per > 1) {
      stay = 0;
      for (int g = 0; g < a.groups; ++g)
        if ((kept >> g) & 1u) stay |= ((1u << per) - 1u) << (g * per);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (whole) {
        if (!((stay >> i) & 1u)) key[i] = 0;
      } else if (!((kept >> (tab.group[min(lane + 32 * i, MAX_EXPERTS - 1)] & 31)) & 1u)) {
        key[i] = 0;
      }
      if (by_score && !by_bias && key[i]) key[i] = logit_key(x[i]);
    }
  }
  int e = -1;
  if (!doubt) {
    // Keys to order by carry the expert in their low bits, a lower one larger, so each is unique, and a round needs no search for its
    // expert.  Above them stands the biased score in steps of 2^-23 (E > 256: 2^-22, 2^-21) of the scores' range, or the leading bits of the logit,
    // which hold a 16-bit one whole.  Where two neighbours could be the other way round, the candidates' values decide.
    constexpr int ID = NV == 4 ? 7 : NV == 8 ? 8 : NV == 16 ? 9 : 10, FIXED = 31 - ID < 23 ? 31 - ID : 23;
    constexpr uint32_t LOW = (1u << ID) - 1;
    float steps = 0.f, spread = 0.f;   // steps of one; the largest magnitude, to whose rounding the scores are known
    if (by_bias) {
      uint32_t hi = 0, lo = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hi = max(hi, key[i]);
        lo = min(lo, key[i] - 1u);   // (none: the largest)
      }
      hi = __reduce_max_sync(0xffffffffu, hi);
      lo = __reduce_min_sync(0xffffffffu, lo) + 1u;
      const float base = key_logit(lo), range = key_logit(hi) - base;
      spread = fmaxf(fabsf(base), fabsf(key_logit(hi)));
      // (a range beyond fp32, or none: all keys the same)
      // (8 below the field's end: the quick division may be 2 steps of fp32 above the quotient, which is 2 of the field's, and a key past
      // its end would be the least of all)
      steps = range > 1e-30f && range < 1e30f ? __fdividef((float)((1 << FIXED) - 8), range) : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float c = __uint_as_float(key[i] ^ (~(uint32_t)((int)key[i] >> 31) | 0x80000000u));
        key[i] = key[i] ? 0x80000000u | ((__float_as_uint(fmaf(c - base, steps, 8388608.f)) & 0x7fffffu) << ID) | (LOW - lane - 32 * i) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = key[i] ? (key[i] & ~LOW) | (LOW - lane - 32 * i) : 0u;
    }
    uint32_t behind;
    uint32_t mine = ordered_keys<NV>(key, a.k + 1, lane, behind);
    if (lane >= a.k) mine = 0;
    if (mine) e = (int)(LOW - (mine & LOW));
    if (by_bias || a.dtype == GT_FP32) {
      uint32_t after = __shfl_down_sync(0xffffffffu, mine, 1);
      if (lane + 1 >= a.k) after = behind;
      // scores: nearer than their errors, and two steps; logits: the same leading bits
      const float apart = (float)((mine >> ID) - (after >> ID)), least = by_bias ? 2.f + steps * (2.f * err + 0x1p-21f * spread) : 0.f;
      if (__any_sync(0xffffffffu, mine && after && !(apart > least))) {
        e = settle(a, tab, t, lane, e, kept, m, inv, err);
        doubt = __any_sync(0xffffffffu, e == UNSETTLED);
      }
    }
  }
  if (doubt) e = exact_select<NV>(a, tab, t, lane, m);
  // weights of the selected alone
  const float l = e >= 0 ? logit_of(a, t, e) : 0.f;
  float w = 0.f;
  if (a.renorm) {
    float num;
    if (a.kind == 1 && !__any_sync(0xffffffffu, e >= 0 && l < -60.f)) {
      num = e >= 0 ? __fdividef(1.f, 1.f + expf(-l)) : 0.f;
    } else {
      // e^(z - largest z) with z the logit or its log sigmoid, so that scores that would all underflow still give weights that sum
      // to the factor
      const float z = a.kind == 1 ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
      const float z0 = warp_max_f(e >= 0 ? z : -INFINITY);
      num = e >= 0 ? expf(z - z0) : 0.f;
    }
    float den = num;
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (e >= 0) w = __fdividef(num, den);
  } else if (e >= 0) {
    const float d = expf(-fabsf(l));
    w = a.kind == 1 ? (l >= 0.f ? 1.f : d) / (1.f + d) : expf(l - m) * inv;
  }
  my_e = e;
  my_w = w * a.factor;
}

}  // namespace moe
