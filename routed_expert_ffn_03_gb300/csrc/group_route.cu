// group_route.cu - router selection of a batch from its logits, pairs grouped by expert.
//
// Two kernels.  The first takes a slice of the tokens per block: each warp selects one
// token's k experts (k rounds of two warp reductions over order-preserving keys of the
// logits) and writes ids and weights, and the block counts its pairs by expert.  The second
// takes the same slices: a block sums the counts of the blocks before it, scans the
// experts' totals into offsets, and places its pairs in order (a stable counting sort: no
// atomic decides a position, so the same logits give the same arrays).
#include "common.cuh"
#include "group_route.h"
#include "grouped.h"
#include "route.cuh"

namespace moe {

namespace {

constexpr int GR_THREADS = 256;
constexpr int GR_WARPS = GR_THREADS / 32;
constexpr int GR_MAX_BLOCKS = 128;

__device__ __forceinline__ float load_logit(const void* p, long long i, int dtype) {
  if (dtype == GT_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return dtype == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}

// k rounds: the largest key not yet taken, then the least id holding it (ids ascend with
// the register index inside a lane, and a lane keeps the first of its equal keys).  Keys at
// or below `none` are never selected.  Lane j < k receives the j-th id (-1: none left) and key.
template <int NV>
__device__ __forceinline__ void select_keys(const uint32_t (&key)[NV], uint32_t none, int k, int lane, int& my_e,
                                            uint32_t& my_key) {
  uint32_t taken = 0u, lk = none;
  int le = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (key[i] > lk) {
      lk = key[i];
      le = lane + 32 * i;
    }
  my_e = -1;
  my_key = none;
  for (int j = 0; j < k; ++j) {
    const uint32_t bk = __reduce_max_sync(0xffffffffu, lk);
    if (bk == none) break;   // uniform
    const int be = (int)__reduce_min_sync(0xffffffffu, lk == bk ? (uint32_t)le : 0xffffffffu);
    if (lane == j) {
      my_e = be;
      my_key = bk;
    }
    if (le == be) {
      taken |= 1u << ((be - lane) >> 5);
      lk = none;
      le = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!((taken >> i) & 1u) && key[i] > lk) {
          lk = key[i];
          le = lane + 32 * i;
        }
    }
  }
}

template <int NV>
__device__ __forceinline__ void token_topk(const GroupRouteArgs& a, long long t, int lane, int& my_e, uint32_t& my_key) {
  uint32_t key[NV];
  const uint32_t none = logit_key(-INFINITY);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    float x = e < a.E ? load_logit(a.logits, t * a.ld + e, a.dtype) : -INFINITY;
    x = x != x ? -INFINITY : fminf(x, 3.402823466e38f);
    key[i] = logit_key(x);
  }
  select_keys<NV>(key, none, a.k, lane, my_e, my_key);
}

// one token by one warp: its ids and weights
__device__ __forceinline__ int route_token(const GroupRouteArgs& a, long long t, int lane) {
  int e;
  uint32_t key;
  if (a.E <= 128) token_topk<4>(a, t, lane, e, key);
  else if (a.E <= 256) token_topk<8>(a, t, lane, e, key);
  else if (a.E <= 512) token_topk<16>(a, t, lane, e, key);
  else token_topk<32>(a, t, lane, e, key);
  // softmax over the selected logits, or over their log sigmoids: exp(z_j - z_0) / sum, the
  // first being the largest of both
  const float l = key_logit(key);
  float z = l;
  if (a.kind == 1) z = fminf(l, 0.f) - log1pf(expf(-fabsf(l)));
  const float z0 = __shfl_sync(0xffffffffu, z, 0);
  const float num = lane < a.k && e >= 0 ? expf(z - z0) : 0.f;
  float den = num;
#pragma unroll
  for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (lane < a.k) {
    a.idx[t * a.k + lane] = e;
    a.weights[t * a.k + lane] = e >= 0 ? num / den : 0.f;
  }
  return e;
}

__global__ void __launch_bounds__(GR_THREADS) group_select_kernel(GroupRouteArgs a) {
  __shared__ int hist[1024];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) hist[e] = 0;
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * a.per_block, t1 = min(t0 + a.per_block, (long long)a.T);
  for (long long t = t0 + warp; t < t1; t += GR_WARPS) {
    const int e = route_token(a, t, lane);
    if (lane < a.k && e >= 0) atomicAdd(&hist[e], 1);   // a count: its order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) a.hist[(long long)blockIdx.x * a.E + e] = hist[e];
}

__global__ void __launch_bounds__(GR_THREADS) group_place_kernel(GroupRouteArgs a) {
  __shared__ int next[GR_WARPS][1024];   // per warp: count by expert, then the next position
  __shared__ int wsum[GR_WARPS + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  for (int i = tid; i < GR_WARPS * 1024; i += GR_THREADS) (&next[0][0])[i] = 0;
  // expert 4 tid + q: its pairs in earlier blocks and in all of them
  int before[4] = {0, 0, 0, 0}, all[4] = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * tid + q;
    if (e < a.E)
      for (int b = 0; b < a.blocks; ++b) {
        const int c = __ldcg(a.hist + (long long)b * a.E + e);
        all[q] += c;
        if (b < (int)blockIdx.x) before[q] += c;
      }
  }
  const int mine = all[0] + all[1] + all[2] + all[3];
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int off = inc - mine;
  for (int w = 0; w < warp; ++w) off += wsum[w];
  int total = 0;
  for (int w = 0; w < GR_WARPS; ++w) total += wsum[w];

  // this warp's share of the block's pairs
  const long long P = (long long)a.T * a.k;
  const long long p0 = min((long long)blockIdx.x * a.per_block * a.k, P), p1 = min(p0 + (long long)a.per_block * a.k, P);
  const long long share = ((p1 - p0 + GR_WARPS - 1) / GR_WARPS + 31) / 32 * 32;
  const long long q0 = min(p0 + warp * share, p1), q1 = min(q0 + share, p1);
  for (long long i = q0 + lane; i < q1; i += 32) {
    const int e = __ldcg(a.idx + i);
    if (e >= 0) atomicAdd(&next[warp][e], 1);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 4 * tid + q;
    if (e < a.E) {
      int pos = off + before[q];
      for (int w = 0; w < GR_WARPS; ++w) {
        const int c = next[w][e];
        next[w][e] = pos;
        pos += c;
      }
      if (blockIdx.x == 0) a.offsets[e] = off;
    }
    off += all[q];
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[a.E] = total;
  __syncthreads();
  for (long long i0 = q0; i0 < q1; i0 += 32) {
    const long long i = i0 + lane;
    const int e = i < q1 ? __ldcg(a.idx + i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int r = __popc(same & ((1u << lane) - 1u));
      const int pos = next[warp][e] + r;
      a.pairs[pos] = (int)i;
      a.rows[pos] = (int)(i / a.k);
    }
    __syncwarp();
    if (e >= 0 && lane == 31 - __clz(same)) next[warp][e] += __popc(same);
    __syncwarp();
  }
  // no pair stands behind the last group
  for (long long i = max(p0, (long long)total) + tid; i < p1; i += GR_THREADS) {
    a.pairs[i] = -1;
    a.rows[i] = -1;
  }
}

}  // namespace

GroupRoutePlan group_route_plan(int T, int E, int k) {
  GroupRoutePlan p;
  p.per_block = (T + GR_MAX_BLOCKS - 1) / GR_MAX_BLOCKS;
  if (p.per_block < 32) p.per_block = 32;
  p.blocks = (T + p.per_block - 1) / p.per_block;
  p.workspace = (size_t)p.blocks * E * sizeof(int);
  return p;
}

cudaError_t launch_group_route(GroupRouteArgs a, cudaStream_t s) {
  group_select_kernel<<<a.blocks, GR_THREADS, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  group_place_kernel<<<a.blocks, GR_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
