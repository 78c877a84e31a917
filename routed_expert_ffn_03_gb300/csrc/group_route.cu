// group_route.cu - router selection of a batch from its logits, pairs grouped by expert.
//
// A block takes a slice of the tokens; each warp selects two tokens' experts at a time over order-preserving keys of the
// logits, writes ids and weights, and the block counts its
// pairs by expert.  Then a block sums the counts of the blocks before it, scans the experts' totals into offsets,
// and places its pairs in order: a stable counting sort, in which no atomic decides a position, so the same logits give
// the same arrays.  Up to 512 tokens are one cluster of one launch; more are two launches over one block of 32 warps an SM,
// the second waiting for the first on the device.  Bound: issue while selecting (about 350 instructions a token, 2.4 us for
// 32 tokens an SM), latency while placing: 16384 tokens of 256 bf16 logits, k = 8, take 19.6 us (10 MB, 1.5 us at the
// memory's rate), of which 8 are two launches' of any size; one token 4.8 us.
#include "group_sort.cuh"
#include "route.cuh"

namespace moe {

namespace {

// Keys carry the expert in their low 10 bits, a lower one larger, so each is unique and none is 0 but the masked ones.  16-bit
// logits fit the 22 bits above whole; of fp32 logits those are the leading ones.
template <int NV>
__device__ __forceinline__ void token_keys(const GroupRouteArgs& a, int lane, const float (&l)[NV], uint32_t (&key)[NV]) {
  constexpr uint32_t inf = 0xff800000u;   // key of +inf, which counts as the one below
  auto keys = [&](auto value) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = value(l[i]);
      const bool live = x > -INFINITY && lane + 32 * i < a.E;   // NaN is not
      key[i] = live ? (min(logit_key(x), inf - 1u) & ~1023u) | (uint32_t)(1023 - lane - 32 * i) : 0u;
    }
  };
  if (a.dtype == GT_BF16) keys([](float x) { return __uint_as_float(__float_as_uint(x) << 16); });
  else if (a.dtype == GT_FP16) keys([](float x) { return __half2float(__ushort_as_half((unsigned short)__float_as_uint(x))); });
  else keys([](float x) { return x; });
}

// The first n of the keys in descending order, lane j the j-th (0: none), for n <= FEW: each round takes the largest of the
// lanes' firsts, and the lane that held it steps to its second and third.  ok is false where a lane gave all three (one
// token in 20 for 8 of 256).  U tokens side by side, as each round waits for the one before.  (A sorting network over the
// warp takes twice the instructions: 20.8 and 19.6 us for 16384 tokens.)
constexpr int FEW = 10;
template <int NV, int U>
__device__ __forceinline__ void few_keys(const uint32_t (&key)[U][NV], int n, int lane, uint32_t (&mine)[U], bool (&ok)[U]) {
  uint32_t b1[U], b2[U], b3[U];
  bool three[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    b1[u] = b2[u] = b3[u] = mine[u] = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t x = min(b1[u], key[u][i]), y = min(b2[u], x);
      b1[u] = max(b1[u], key[u][i]);
      b2[u] = max(b2[u], x);
      b3[u] = max(b3[u], y);
    }
    three[u] = b3[u] != 0;
  }
#pragma unroll
  for (int j = 0; j < FEW; ++j) {
    if (j >= n) break;   // uniform
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t b = __reduce_max_sync(0xffffffffu, b1[u]);
      if (lane == j) mine[u] = b;
      if (b1[u] == b) {
        b1[u] = b2[u];
        b2[u] = b3[u];
        b3[u] = 0;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) ok[u] = !__any_sync(0xffffffffu, three[u] && b1[u] == 0);
}

// The same for any n <= 32 by rounds: the warp's largest key is the next, and the lane that held it looks for its next.
template <int NV>
__device__ __forceinline__ uint32_t rounds_of_keys(uint32_t (&key)[NV], int n, int lane) {
  uint32_t best = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) best = max(best, key[i]);
  for (int j = 0; j < n; ++j) {
    const uint32_t b = __reduce_max_sync(0xffffffffu, best);
    if (b == 0) break;   // uniform
    if (lane == j) mine = b;
    if (best == b) {
      best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (key[i] == b) key[i] = 0;
        best = max(best, key[i]);
      }
    }
  }
  return mine;
}

// The k best of one token from its sorted keys: lane j < k receives the j-th id (-1: none left).  Of fp32 logits one more
// key than k shows whether two neighbours in the order share their leading bits (1 or 2 tokens in 100 of random ones).  Among
// the k they are then ordered by their whole keys; if the k-th and the one behind it share them, or the latter is not
// known (k = 32), the token is selected again from whole keys, with a second maximum for the id.
template <int NV>
__device__ __forceinline__ int token_topk(const GroupRouteArgs& a, long long t, int lane, uint32_t mine) {
  int e = lane < a.k && mine ? 1023 - (int)(mine & 1023u) : -1;
  if (a.dtype == GT_FP32) {
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const unsigned doubt = __ballot_sync(0xffffffffu, lane < a.k && mine && (lane < 31 ? (mine ^ next) < 1024u : a.E > 32));
    if (doubt && !(doubt >> (a.k - 1))) {
      const uint32_t whole = e >= 0 ? logit_key(logit_of(a, t, e)) : 0u;
      int rank = 0;
      for (int i = 0; i < a.k; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, whole, i);
        const int oe = __shfl_sync(0xffffffffu, e, i);
        rank += o > whole || (o == whole && (oe < e || (oe == e && i < lane)));   // (the last: places left empty keep theirs)
      }
      int from = lane;
      for (int i = 0; i < a.k; ++i)
        if (__shfl_sync(0xffffffffu, rank, i) == lane) from = i;
      e = __shfl_sync(0xffffffffu, e, from);
    } else if (doubt) {
      uint32_t taken = 0;
      e = -1;
      for (int j = 0; j < a.k; ++j) {
        uint32_t lk = 0;
        int le = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int ee = lane + 32 * i;
          const float x = ee < a.E && !((taken >> i) & 1u) ? logit_of(a, t, ee) : -INFINITY;
          if (x > -INFINITY && logit_key(x) > lk) {   // ascending ids: the first of equal keys stays
            lk = logit_key(x);
            le = ee;
          }
        }
        const uint32_t bk = __reduce_max_sync(0xffffffffu, lk);
        if (bk == 0) break;
        const int be = (int)__reduce_min_sync(0xffffffffu, lk == bk ? (uint32_t)le : 0xffffffffu);
        if (lane == j) e = be;
        if (le == be && lk == bk) taken |= 1u << ((be - lane) >> 5);
      }
    }
  }
  return e;
}

// U tokens by one warp, t and every GR_WARPS-th behind it up to t1: their ids and weights, and their pairs by expert into hist
template <int NV, int U>
__device__ __forceinline__ void route_tokens(const GroupRouteArgs& a, long long t, long long t1, int lane, float (&l)[U][NV],
                                             int* hist) {
  uint32_t key[U][NV], mine[U];
  bool ok[U];
  const int n = a.dtype == GT_FP32 ? min(a.k + 1, 32) : a.k;
#pragma unroll
  for (int u = 0; u < U; ++u) token_keys<NV>(a, lane, l[u], key[u]);
  if (n <= FEW) few_keys<NV, U>(key, n, lane, mine, ok);
  float z[U], num[U], den[U];
  int e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tt = t + u * GR_WARPS;
    e[u] = -1;
    z[u] = 0.f;
    if (tt >= t1) continue;
    if (n > FEW || !ok[u]) mine[u] = rounds_of_keys<NV>(key[u], n, lane);
    e[u] = token_topk<NV>(a, tt, lane, mine[u]);
    // softmax over the selected logits, or over their log sigmoids: exp(z_j - z_0) / sum, the first being the largest
    // of both; a 16-bit logit stands in its key whole (+inf as a large value)
    float l = 0.f;
    if (e[u] >= 0)
      l = a.dtype == GT_FP32 ? logit_of(a, tt, e[u]) : key_logit(mine[u] >> 31 ? mine[u] & ~1023u : mine[u] | 1023u);
    z[u] = a.kind == 1 ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float z0 = __shfl_sync(0xffffffffu, z[u], 0);
    den[u] = num[u] = lane < a.k && e[u] >= 0 ? expf(z[u] - z0) : 0.f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) den[u] += __shfl_xor_sync(0xffffffffu, den[u], o);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tt = t + u * GR_WARPS;
    if (lane < a.k && tt < t1) {
      a.idx[tt * a.k + lane] = e[u];
      a.weights[tt * a.k + lane] = e[u] >= 0 ? num[u] / den[u] : 0.f;
      if (e[u] >= 0) atomicAdd(&hist[e[u]], 1);   // a count: its order does not matter
    }
  }
}

// this block's tokens; and its pairs by expert into hist (shared)
template <int NV>
__device__ __forceinline__ void select_tokens(const GroupRouteArgs& a, int* hist) {
  constexpr int U = NV <= 8 ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) hist[e] = 0;
  __syncthreads();
  const long long t0 = min((long long)blockIdx.x * a.per_block, (long long)a.T), t1 = min(t0 + a.per_block, (long long)a.T);
  for (long long t = t0 + warp; t < t1; t += U * GR_WARPS) {
    float l[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) load_token<NV>(a, min(t + u * GR_WARPS, t1 - 1), lane, l[u]);
    route_tokens<NV, U>(a, t, t1, lane, l, hist);
  }
  __syncthreads();
}

// One launch: the blocks are one cluster, and read each other's counts.
template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) group_one_kernel(GroupRouteArgs a) {
  extern __shared__ int counts[];
  __shared__ int hist[1024], all[1024], before[1024];
  const Pairs s = block_pairs(a, counts);
  for (int i = threadIdx.x; i < s.W * a.E; i += GR_THREADS) counts[i] = 0;
  pdl_wait();
  select_tokens<NV>(a, hist);
  if (a.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  count_pairs(a, s);   // while the others arrive
  if (a.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int e = threadIdx.x, rank = a.blocks > 1 ? (int)cluster_rank() : 0;
  int sum = 0, mine = 0;
  if (e < a.E)
    for (int r = 0; r < a.blocks; ++r) {
      int c = hist[e];
      if (a.blocks > 1)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(map_rank(smem_u32(&hist[e]), r)) : "memory");
      if (r < rank) mine += c;
      sum += c;
    }
  all[e] = sum;
  before[e] = mine;
  if (a.blocks > 1) cluster_sync_all();   // the others read this block's counts until here
  else __syncthreads();
  place_pairs<false>(a, s, before, all, counts, nullptr);
}

// The counts leave by clusters, hist [clusters][E], with each block's share of its cluster's before it, [blocks][E] behind:
// the next kernel's blocks then read half of the rows (read one by one, they took half of that kernel's time).
template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) group_select_kernel(GroupRouteArgs a) {
  __shared__ int hist[1024];
  pdl_launch_dependents();
  pdl_wait();
  select_tokens<NV>(a, hist);
  cluster_sync_all();
  const int rank = (int)cluster_rank(), clusters = a.blocks / GR_CLUSTER;
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) {
    int before = 0, all = 0;
#pragma unroll
    for (int r = 0; r < GR_CLUSTER; ++r) {
      int c;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(map_rank(smem_u32(&hist[e]), r)) : "memory");
      if (r < rank) before += c;
      all += c;
    }
    a.hist[(long long)(clusters + blockIdx.x) * a.E + e] = before;
    if (rank == 0) a.hist[(long long)(blockIdx.x / GR_CLUSTER) * a.E + e] = all;
  }
  cluster_sync_all();   // the others read this block's counts until here
}

__global__ void __launch_bounds__(GR_THREADS, 1) group_place_kernel(GroupRouteArgs a) {
  extern __shared__ int counts[];
  __shared__ int all[1024], before[1024];
  const Pairs pairs = block_pairs(a, counts);
  for (int i = threadIdx.x; i < pairs.W * a.E; i += GR_THREADS) counts[i] = 0;
  all[threadIdx.x] = before[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait();
  count_pairs(a, pairs);
  // thread (part, e): an expert's counts of every parts-th cluster
  const int Ep = (a.E + 31) & ~31, parts = GR_THREADS / Ep, part = threadIdx.x / Ep, e = threadIdx.x % Ep;
  const int clusters = a.blocks / GR_CLUSTER, mine = blockIdx.x / GR_CLUSTER;
  if (part < parts && e < a.E) {
    int s = 0, p = part == 0 ? __ldcg(a.hist + (long long)(clusters + blockIdx.x) * a.E + e) : 0;
#pragma unroll 20
    for (int c = part; c < clusters; c += parts) {
      const int n = __ldcg(a.hist + (long long)c * a.E + e);
      s += n;
      if (c < mine) p += n;
    }
    atomicAdd(&all[e], s);
    atomicAdd(&before[e], p);
  }
  __syncthreads();
  place_pairs<false>(a, pairs, before, all, counts, nullptr);
}

template <int NV>
cudaError_t launch_as(const GroupRouteArgs& a, cudaStream_t s) {
  const int warps = GR_COUNTS / a.E < GR_WARPS ? GR_COUNTS / a.E : GR_WARPS;
  const size_t smem = (size_t)warps * a.E * sizeof(int);
  if (a.T <= one_launch(a.E)) return launch(group_one_kernel<NV>, a.blocks, a.blocks, smem, s, a);
  cudaError_t e = launch(group_select_kernel<NV>, a.blocks, GR_CLUSTER, 0, s, a);
  return e != cudaSuccess ? e : launch(group_place_kernel, a.blocks, 1, smem, s, a);
}

template <int NV>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(group_one_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, GR_COUNTS * 4);
}

}  // namespace

cudaError_t group_route_set_attributes() {
  cudaError_t e = set_attribute<4>();
  if (e == cudaSuccess) e = set_attribute<8>();
  if (e == cudaSuccess) e = set_attribute<16>();
  if (e == cudaSuccess) e = set_attribute<32>();
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(group_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GR_COUNTS * 4);
  return e;
}

GroupRoutePlan group_route_plan(int T, int E, int k) {
  constexpr int kBlocks = 152;   // one an SM; a constant, so that the workspace's size does not depend on the device
  GroupRoutePlan p;
  if (T <= one_launch(E)) {   // a token a warp, from eight blocks on more
    p.blocks = 1;
    while (p.blocks < 8 && p.blocks * GR_WARPS < T) p.blocks *= 2;   // (some may have no tokens)
    p.per_block = (T - 1) / p.blocks + 1;
    p.workspace = 0;
  } else {
    p.per_block = (T - 1) / kBlocks + 1;
    if (p.per_block < GR_WARPS) p.per_block = GR_WARPS;
    p.blocks = ((T - 1) / p.per_block + GR_CLUSTER) / GR_CLUSTER * GR_CLUSTER;   // (one may have none)
    p.workspace = (size_t)(p.blocks + p.blocks / GR_CLUSTER) * E * sizeof(int);
  }
  return p;
}

cudaError_t launch_group_route(const GroupRouteArgs& a, cudaStream_t s) {
  if (a.E <= 128) return launch_as<4>(a, s);
  if (a.E <= 256) return launch_as<8>(a, s);
  return a.E <= 512 ? launch_as<16>(a, s) : launch_as<32>(a, s);
}

}  // namespace moe
