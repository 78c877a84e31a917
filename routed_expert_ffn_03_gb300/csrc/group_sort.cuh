// group_sort.cuh - what the batch routing kernels share: a token's logits, and the counting sort of its pairs by expert.
#pragma once
#include "common.cuh"
#include "group_route.h"
#include "grouped.h"
#include "grouped_mma.cuh"

namespace moe {

constexpr int GR_THREADS = 1024;
constexpr int GR_WARPS = GR_THREADS / 32;
// Tokens of the one-launch form, a cluster of up to 8 blocks: one or two a warp.  512 of 256 experts: 10.2 us, in two launches
// 10.4, and 16 with the host's part; 1000: 15.0 and 10.4.  256 of 1000 experts, k = 32: 33 us, 1000 111 and 36.
constexpr int one_launch(int E) { return E <= 512 ? 512 : 256; }
constexpr int GR_CLUSTER = 2;         // blocks that add up their counts before they leave (4 do not fill every SM: 33 us, not 20)
constexpr int GR_COUNTS = 16384;      // counts by warp and expert that a block holds

__device__ __forceinline__ float load_logit(const void* p, long long i, int dtype) {
  if (dtype == GT_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
  return dtype == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}

__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }
__device__ __forceinline__ float logit_of(const GroupRouteArgs& a, long long t, int e) {
  return clean(load_logit(a.logits, t * a.ld + e, a.dtype));
}

// Lane l's logits of token t: experts l + 32 i.  The loads of each type stand together: a branch around each would run them
// one after another.
template <int NV>
__device__ __forceinline__ void load_token(const GroupRouteArgs& a, long long t, int lane, float (&l)[NV]) {
  if (a.dtype == GT_FP32) {
    const float* src = static_cast<const float*>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = lane + 32 * i < a.E ? __ldg(src + lane + 32 * i) : -INFINITY;
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = __uint_as_float(lane + 32 * i < a.E ? __ldg(src + lane + 32 * i) : 0u);   // raw
  }
}

// A block's pairs, shared out to W warps in runs of whole 32s; counts (shared) [W][E].
struct Pairs {
  int W;
  long long p0, p1, q0, q1;   // the block's, this warp's
  int* next;                  // this warp's row of counts
};
__device__ __forceinline__ Pairs block_pairs(const GroupRouteArgs& a, int* counts) {
  Pairs s;
  const int warp = threadIdx.x >> 5;
  s.W = min(GR_WARPS, GR_COUNTS / a.E);
  const long long P = (long long)a.T * a.k;
  s.p0 = min((long long)blockIdx.x * a.per_block * a.k, P);
  s.p1 = min(s.p0 + (long long)a.per_block * a.k, P);
  const long long share = ((s.p1 - s.p0 + s.W - 1) / s.W + 31) / 32 * 32;
  s.q0 = min(s.p0 + warp * share, s.p1);
  s.q1 = warp < s.W ? min(s.q0 + share, s.p1) : s.q0;
  s.next = counts + warp * a.E;
  return s;
}
// counts (zeros before) by warp and expert
__device__ __forceinline__ void count_pairs(const GroupRouteArgs& a, const Pairs& s) {
  for (long long i = s.q0 + (threadIdx.x & 31); i < s.q1; i += 32) {
    const int e = __ldcg(a.idx + i);
    if (e >= 0) atomicAdd(&s.next[e], 1);
  }
}
// Places this block's pairs (PLACES: and says where each stands).  before, all (shared, [E]): an expert's pairs in earlier blocks and in all of them.
template <bool PLACES>
__device__ __forceinline__ void place_pairs(const GroupRouteArgs& a, const Pairs& s, const int* before, const int* all, int* counts,
                                            int* places) {
  __shared__ int wsum[GR_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
  // offsets: an exclusive scan of all over the experts, thread e its own
  const int mine = tid < E ? all[tid] : 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int sums = wsum[lane];   // GR_WARPS == 32: every warp scans the warps' sums for itself
  const int own = sums;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += v;
  }
  const int off = inc - mine + __shfl_sync(0xffffffffu, sums - own, warp), total = __shfl_sync(0xffffffffu, sums, 31);
  if (tid < E) {   // counts become first positions
    if (blockIdx.x == 0) a.offsets[tid] = off;
    int pos = off + before[tid];
#pragma unroll 8
    for (int w = 0; w < s.W; ++w) {
      const int c = counts[w * E + tid];
      counts[w * E + tid] = pos;
      pos += c;
    }
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[E] = total;
  __syncthreads();
  for (long long i0 = s.q0; i0 < s.q1; i0 += 32) {
    const long long i = i0 + lane;
    const int e = i < s.q1 ? __ldcg(a.idx + i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    int pos = 0;
    if (e >= 0) pos = s.next[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (PLACES && i < s.q1) places[i] = e >= 0 ? pos : -1;
    if (e >= 0) {
      a.pairs[pos] = (int)i;
      a.rows[pos] = (int)((unsigned)i / (unsigned)a.k);
      if (lane == 31 - __clz(same)) s.next[e] = pos + 1;
    }
    __syncwarp();
  }
  // no pair stands behind the last group
  for (long long i = max(s.p0, (long long)total) + tid; i < s.p1; i += GR_THREADS) {
    a.pairs[i] = -1;
    a.rows[i] = -1;
  }
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), int blocks, int cluster, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(GR_THREADS);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace moe
