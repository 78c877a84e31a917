// balanced_select.cuh - one token's experts by a warp: scores with a bias for balance, limited to groups of experts.
//
//   s_e = softmax or sigmoid of the logits,  c_e = s_e + b_e;  a group's score: its largest c, or the sum of its two largest;
//   the `keep` best groups stay, and of their experts the k with the largest c (without a bias: logits) are selected.
//
// Experts are chosen as if scores were compared in 64 bits, so that the choice does not depend on how fp32 rounds an
// exponential.  Scores are fp32 first, with a bound on their error; only where two neighbours in the order are closer than
// that are they computed again in fp64: of one token in some thousands, for the candidates alone, one a lane.  (fp64 runs at a
// 64th of fp32's rate: all of 256 scores take 4 us.)  Where that does not decide it (groups that close, more
// candidates than lanes, scores that underflow) all of the token's scores are.
#pragma once
#include "group_route.h"
#include "grouped.h"
#include "route.cuh"

namespace moe {

constexpr int MAX_EXPERTS = 1024;

// What a block keeps of the bias and the groups: biases as they count (NaN and -inf: the expert is masked; +inf: the largest
// finite), and each expert's group.
struct BalancedTables {
  float bias[MAX_EXPERTS];
  uint8_t group[MAX_EXPERTS];
};

__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }
__device__ __forceinline__ float load_logit(const void* p, long long i, int dtype) {
  if (dtype == GT_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return dtype == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ float logit_of(const GroupRouteArgs& a, long long t, int e) {
  return clean(load_logit(a.logits, t * a.ld + e, a.dtype));
}

__device__ __forceinline__ void balanced_tables(const GroupRouteArgs& a, BalancedTables& tab) {
  const int size = a.E / a.groups;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    tab.bias[e] = a.bias ? clean(__ldg(a.bias + e)) : 0.f;
    tab.group[e] = (uint8_t)(e / size);
  }
}

__device__ __forceinline__ float key_value(uint32_t k) { return k ? key_logit(k) : -INFINITY; }
__device__ __forceinline__ float warp_max_f(float v) { return key_value(__reduce_max_sync(0xffffffffu, v > -INFINITY ? logit_key(v) : 0u)); }

// the kept groups as bits: the best of lane g's score of group g (-inf: none), equal ones the lower first
template <typename T>
__device__ __forceinline__ unsigned kept_groups(T score, int groups, int keep, int lane) {
  int rank = 0;
  for (int q = 0; q < groups; ++q) {
    const T o = __shfl_sync(0xffffffffu, score, q);
    rank += o > score || (o == score && q < lane);
  }
  return __ballot_sync(0xffffffffu, lane < groups && rank < keep && score > (T)-INFINITY);
}

// sum over the token's experts of e^(l - m), in 64 bits
static __device__ __noinline__ double exact_total(const GroupRouteArgs& a, long long t, int lane, float m) {
  double z = 0.0;
  for (int e = lane; e < a.E; e += 32) {
    const float l = logit_of(a, t, e);
    if (l > -INFINITY) z += exp((double)l - (double)m);
  }
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
__device__ __forceinline__ double exact_score(const GroupRouteArgs& a, float l, float m, double z) {
  return a.kind == 1 ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
}

// The whole selection in 64 bits: lane j < k receives the j-th expert, or -1.
template <int NV>
static __device__ __noinline__ int exact_select(const GroupRouteArgs& a, const BalancedTables& tab, long long t, int lane, float m) {
  double c[NV];
  const double z = a.kind == 0 ? exact_total(a, t, lane, m) : 1.0;
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    c[i] = -INFINITY;
    if (e < a.E) {
      const float l = logit_of(a, t, e), b = tab.bias[e];
      if (l > -INFINITY && b > -INFINITY) c[i] = exact_score(a, l, m, z) + (double)b;
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
  // without a bias logits are compared, as their scores' order is theirs
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.E || !((kept >> (tab.group[e] & 31)) & 1u)) c[i] = -INFINITY;
    else if (!a.bias && c[i] > -INFINITY) c[i] = logit_of(a, t, e);
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

// The selection of token t: lane j < k receives the j-th expert (-1: none) and its weight.  x: lane l's logits of experts
// l + 32 i, cleaned (-inf: masked, or past the experts).
template <int NV>
__device__ __forceinline__ void balanced_token(const GroupRouteArgs& a, const BalancedTables& tab, long long t, int lane,
                                               const float (&x)[NV], int& my_e, float& my_w) {
  const bool limited = a.keep < a.groups, scores = a.bias || limited || !a.renorm;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
  const float m = warp_max_f(top);   // the largest logit
  float inv = 1.f, err = 0.f;        // softmax: one over the sum; the scores' absolute error
  if (scores) {
    if (a.kind == 0) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) z += x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      inv = 1.f / z;
      // each of NV + 5 additions, the exponential and two products a step; e^-d is off by d 2^-24 of itself for the rounding of d,
      // at most 0.37 2^-24
      err = (NV + 17) * 0x1p-23f * inv;
    } else {
      err = 0x1p-21f / (1.f + expf(-m));   // exponential, sum and division: four steps of the largest score at most
    }
  }
  // keys by which experts are compared: scores with the bias, or logits
  uint32_t key[NV];
  const bool by_score = a.bias || limited;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = 0;
    if (x[i] > -INFINITY) {
      float c = x[i];
      if (by_score) {
        const float s = a.kind == 1 ? __fdividef(1.f, 1.f + expf(-x[i])) : expf(x[i] - m) * inv;
        c = s + tab.bias[lane + 32 * i];
      }
      if (c > -INFINITY) key[i] = logit_key(c);
    }
  }
  // scores below 2^-100 lose bits
  bool doubt = by_score && a.kind == 1 && m < -69.f && m > -INFINITY;
  if (limited) {
    float score = -INFINITY;
    auto finish = [&](int g, uint32_t b1, uint32_t b2) {   // a group's score from the lanes' two largest
      const uint32_t w1 = __reduce_max_sync(0xffffffffu, b1);
      float v = key_value(w1);
      if (a.top2 && w1) {
        const int first = __ffs(__ballot_sync(0xffffffffu, b1 == w1)) - 1;
        const uint32_t w2 = __reduce_max_sync(0xffffffffu, lane == first ? b2 : b1);
        if (w2) v += key_value(w2);
      }
      if (lane == g) score = v;
    };
    const int size = a.E / a.groups;
    if (size % 32 == 0) {   // a group is whole registers
      uint32_t b1 = 0, b2 = 0;
      int left = size / 32, g = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (g < a.groups) {
          b2 = max(b2, min(b1, key[i]));
          b1 = max(b1, key[i]);
          if (--left == 0) {
            finish(g++, b1, b2);
            b1 = b2 = 0;
            left = size / 32;
          }
        }
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
    const unsigned kept = kept_groups(score, a.groups, a.keep, lane);
    const bool in = (kept >> lane) & 1u;
    const float last = -warp_max_f(in ? -score : -INFINITY), next = warp_max_f(lane < a.groups && !in ? score : -INFINITY);
    // two scores a group, and the roundings of their sums with the biases and each other
    doubt |= next > -INFINITY && !(last - next > 4.f * err + 0x1p-21f * fmaxf(fabsf(last), fabsf(next)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = min(lane + 32 * i, MAX_EXPERTS - 1);
      if (!((kept >> (tab.group[e] & 31)) & 1u)) key[i] = 0;
      else if (!a.bias && key[i]) key[i] = logit_key(x[i]);
    }
  }
  int e = -1;
  if (!doubt) {
    // the k best and the one behind them
    uint32_t mine = 0, behind = 0, best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) best = max(best, key[i]);
    for (int j = 0; j <= a.k; ++j) {
      const uint32_t b = __reduce_max_sync(0xffffffffu, best);
      if (b == 0) break;   // uniform
      if (j == a.k) {
        behind = b;
        break;
      }
      int id = 0x7fffffff;
      if (best == b) {
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == b) id = lane + 32 * i;
      }
      id = (int)__reduce_min_sync(0xffffffffu, (unsigned)id);
      if (lane == j) {
        mine = b;
        e = id;
      }
      if ((id & 31) == lane) {
        best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (lane + 32 * i == id) key[i] = 0;
          best = max(best, key[i]);
        }
      }
    }
    if (a.bias) {
      // neighbours in the order whose scores are closer than their errors, and not the same logit and bias
      const float c = key_value(mine), b = e >= 0 ? tab.bias[e] : 0.f, l = e >= 0 ? logit_of(a, t, e) : -INFINITY;
      uint32_t after = __shfl_down_sync(0xffffffffu, mine, 1);
      const float la = __shfl_down_sync(0xffffffffu, l, 1), ba = __shfl_down_sync(0xffffffffu, b, 1);
      const bool inner = lane + 1 < a.k;
      if (!inner) after = behind;
      const float ca = key_value(after);
      const float gap = 2.f * err + 0x1p-23f * fmaxf(fabsf(c), fabsf(ca));
      const bool close = lane < a.k && mine && after && !(c - ca > gap) && !(inner && l == la && b == ba);
      if (__any_sync(0xffffffffu, close)) {
        // candidates: the selected, and the others within the error of the last of them, one a lane
        const int n = __popc(__ballot_sync(0xffffffffu, mine != 0));
        const float c_last = __shfl_sync(0xffffffffu, c, n - 1);
        const float limit = c_last - 2.f * err - 0x1p-22f * fabsf(c_last);
        int count = n;
        doubt = !(limit > -INFINITY);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          unsigned who = __ballot_sync(0xffffffffu, key[i] != 0 && key_value(key[i]) >= limit);
          for (; who && count <= 32; who &= who - 1, ++count)
            if (lane == count) e = 32 * i + __ffs(who) - 1;
        }
        doubt |= count > 32;
        if (!doubt) {
          const double z = a.kind == 0 ? exact_total(a, t, lane, m) : 1.0;
          double v = -INFINITY;
          if (lane < count) v = exact_score(a, logit_of(a, t, e), m, z) + (double)tab.bias[e];
          int rank = 0, from = -1;
          for (int q = 0; q < count; ++q) {
            const double o = __shfl_sync(0xffffffffu, v, q);
            const int oe = __shfl_sync(0xffffffffu, e, q);
            rank += o > v || (o == v && oe < e);
          }
          for (int q = 0; q < count; ++q)
            if (__shfl_sync(0xffffffffu, rank, q) == lane) from = q;
          const int sorted = __shfl_sync(0xffffffffu, e, max(from, 0));
          e = from >= 0 && lane < a.k ? sorted : -1;
        }
      }
    }
  }
  if (doubt) e = exact_select<NV>(a, tab, t, lane, m);
  // weights: of the selected alone by e^(z - largest z) with z the logit or its log sigmoid, so that scores that would all
  // underflow still give weights that sum to the factor
  const float l = e >= 0 ? logit_of(a, t, e) : 0.f;
  float w = 0.f;
  if (a.renorm) {
    const float z = a.kind == 1 ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
    const float z0 = warp_max_f(e >= 0 ? z : -INFINITY);
    const float num = e >= 0 ? expf(z - z0) : 0.f;
    float den = num;
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (e >= 0) w = num / den;
  } else if (e >= 0) {
    const float d = expf(-fabsf(l));
    w = a.kind == 1 ? (l >= 0.f ? 1.f : d) / (1.f + d) : expf(l - m) * inv;
  }
  my_e = e;
  my_w = w * a.factor;
}

}  // namespace moe
