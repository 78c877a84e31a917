// balanced_route.cu - router selection of a batch with a bias for balance and limits to groups of experts, pairs grouped by expert.
//
// As group_route.cu, with balanced_select.cuh's selection, a token a warp at a time.  Bound: issue while selecting, some 900 instructions a
// token: 16384 tokens of 256 bf16 logits in 8 groups of which 4 stay, k = 8, take 26 us for it and 11 for placing the pairs (the
// logits and what is written 11 MB, 1.6 us at the memory's rate); one token 7.5 us.
#include "balanced_select.cuh"
#include "group_sort.cuh"

namespace moe {

namespace {

// one token by a warp: its ids and weights, and its pairs by expert into hist
template <int NV>
__device__ __forceinline__ void route_balanced(const BalancedRouteArgs& a, const BalancedTables& tab, long long t, int lane, int* hist) {
  float l[NV];
  load_token<NV>(a, t, lane, l);
  auto values = [&](auto value) {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = lane + 32 * i < a.E ? value(l[i]) : -INFINITY;
  };
  if (a.dtype == GT_BF16) values([](float x) { return __uint_as_float(__float_as_uint(x) << 16); });
  else if (a.dtype == GT_FP16) values([](float x) { return __half2float(__ushort_as_half((unsigned short)__float_as_uint(x))); });
  int e;
  float w;
  balanced_token<NV>(a, tab, t, lane, l, e, w);
  if (lane < a.k) {
    a.idx[t * a.k + lane] = e;
    a.weights[t * a.k + lane] = e >= 0 ? w : 0.f;
    if (e >= 0) atomicAdd(&hist[e], 1);   // a count: its order does not matter
  }
}

// this block's tokens; and its pairs by expert into hist (shared)
template <int NV>
__device__ __forceinline__ void select_tokens(const BalancedRouteArgs& a, int* hist) {
  __shared__ BalancedTables tab;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) hist[e] = 0;
  balanced_tables(a, tab);
  __syncthreads();
  const long long t0 = min((long long)blockIdx.x * a.per_block, (long long)a.T), t1 = min(t0 + a.per_block, (long long)a.T);
  for (long long t = t0 + warp; t < t1; t += GR_WARPS) route_balanced<NV>(a, tab, t, lane, hist);
  __syncthreads();
}

// One launch: the blocks are one cluster, and read each other's counts.
template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) balanced_one_kernel(BalancedRouteArgs a) {
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
  place_pairs<true>(a, s, before, all, counts, a.places);
}

// The counts leave by clusters, hist [clusters][E], with each block's share of its cluster's before it, [blocks][E] behind:
// the next kernel's blocks then read half of the rows.
template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) balanced_select_kernel(BalancedRouteArgs a) {
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

__global__ void __launch_bounds__(GR_THREADS, 1) balanced_place_kernel(BalancedRouteArgs a) {
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
  place_pairs<true>(a, pairs, before, all, counts, a.places);
}

template <int NV>
cudaError_t launch_as(const BalancedRouteArgs& a, cudaStream_t s) {
  const int warps = GR_COUNTS / a.E < GR_WARPS ? GR_COUNTS / a.E : GR_WARPS;
  const size_t smem = (size_t)warps * a.E * sizeof(int);
  if (a.T <= one_launch(a.E)) return launch(balanced_one_kernel<NV>, a.blocks, a.blocks, smem, s, a);
  cudaError_t e = launch(balanced_select_kernel<NV>, a.blocks, GR_CLUSTER, 0, s, a);
  return e != cudaSuccess ? e : launch(balanced_place_kernel, a.blocks, 1, smem, s, a);
}

template <int NV>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(balanced_one_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, GR_COUNTS * 4);
}

}  // namespace

cudaError_t balanced_route_set_attributes() {
  cudaError_t e = set_attribute<4>();
  if (e == cudaSuccess) e = set_attribute<8>();
  if (e == cudaSuccess) e = set_attribute<16>();
  if (e == cudaSuccess) e = set_attribute<32>();
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(balanced_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GR_COUNTS * 4);
  return e;
}

cudaError_t launch_balanced_route(const BalancedRouteArgs& a, cudaStream_t s) {
  if (a.E <= 128) return launch_as<4>(a, s);
  if (a.E <= 256) return launch_as<8>(a, s);
  return a.E <= 512 ? launch_as<16>(a, s) : launch_as<32>(a, s);
}

}  // namespace moe
