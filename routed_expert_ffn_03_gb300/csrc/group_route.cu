// group_route.cu - router selection of a batch from its logits, pairs grouped by expert.
//
// A block takes a slice of the tokens; each warp selects one token's k experts at a time (k rounds of two warp
// reductions over order-preserving keys of the logits), writes ids and weights, and the block counts its
// pairs by expert.  Then a block sums the counts of the blocks before it, scans the experts' totals into offsets,
// and places its pairs in order: a stable counting sort, in which no atomic decides a position, so the same logits give
// the same arrays.  Up to 64 tokens are one block of one launch; more are two launches over one block of 32 warps an SM, the
// second waiting for the first on the device.  Bound: latency (the rounds of a selection depend on one another): ROUTE_LATENCY
#include "common.cuh"
#include "group_route.h"
#include "grouped.h"
#include "route.cuh"

namespace moe {

namespace {

constexpr int GR_THREADS = 1024;
constexpr int GR_WARPS = GR_THREADS / 32;
constexpr int GR_ONE_BLOCK = 64;      // tokens of the one-launch form: two a warp
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

// The k best of one token, by one warp (lane l holds experts l + 32 i): lane j < k receives the j-th id (-1: none left).
// Keys carry the expert in their low 10 bits, a lower one larger, so each is unique and one warp maximum a round finds the
// next: only the lane that held it looks for its next best.  16-bit logits fit the 22 bits above; of fp32 logits
// those are the leading ones, so one more round shows whether two neighbours in the order share them, and such a token
// (1 or 2 in 100 of random ones) is selected again from whole keys, with a second maximum for the id.
template <int NV>
__device__ __forceinline__ int token_topk(const GroupRouteArgs& a, long long t, int lane) {
  uint32_t key[NV];
  uint32_t best = 0;   // 0: below every expert's
  float l[NV];   // the loads of each type together: a branch around each would run them one after another
  if (a.dtype == GT_FP32) {
    const float* src = static_cast<const float*>(a.logits) + t * a.ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = lane + 32 * i < a.E ? __ldg(src + lane + 32 * i) : -INFINITY;
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(a.logits) + t * a.ld;
    uint16_t raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = lane + 32 * i < a.E ? __ldg(src + lane + 32 * i) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = a.dtype == GT_BF16 ? bf16_bits_to_float(raw[i]) : __half2float(__ushort_as_half(raw[i]));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    const float x = e < a.E ? clean(l[i]) : -INFINITY;
    key[i] = x > -INFINITY ? (logit_key(x) & ~1023u) | (uint32_t)(1023 - e) : 0u;
    best = max(best, key[i]);
  }
  uint32_t mine = 0, last = ~0u;
  bool same = false;
  const int rounds = a.dtype == GT_FP32 ? min(a.k + 1, a.E) : a.k;
  for (int j = 0; j < rounds; ++j) {
    const uint32_t b = __reduce_max_sync(0xffffffffu, best);
    if (b == 0) break;   // uniform
    same |= (b ^ last) < 1024u;
    last = b;
    if (lane == j && j < a.k) mine = b;
    if (best == b) {
      best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (key[i] == b) key[i] = 0;
        best = max(best, key[i]);
      }
    }
  }
  int e = mine ? 1023 - (int)(mine & 1023u) : -1;
  if (a.dtype == GT_FP32 && same) {   // uniform
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
  return e;
}

// one token by one warp: its ids and weights
template <int NV>
__device__ __forceinline__ int route_token(const GroupRouteArgs& a, long long t, int lane) {
  const int e = token_topk<NV>(a, t, lane);
  // softmax over the selected logits, or over their log sigmoids: exp(z_j - z_0) / sum, the
  // first being the largest of both
  const float l = e >= 0 ? logit_of(a, t, e) : 0.f;
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

// this block's tokens; and its pairs by expert into hist (shared)
template <int NV>
__device__ __forceinline__ void select_tokens(const GroupRouteArgs& a, int* hist) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) hist[e] = 0;
  __syncthreads();
  const long long t0 = (long long)blockIdx.x * a.per_block, t1 = min(t0 + a.per_block, (long long)a.T);
  for (long long t = t0 + warp; t < t1; t += GR_WARPS) {
    const int e = route_token<NV>(a, t, lane);
    if (lane < a.k && e >= 0) atomicAdd(&hist[e], 1);   // a count: its order does not matter
  }
  __syncthreads();
}

// Places this block's pairs.  before, all (shared, [E]): an expert's pairs in earlier blocks and in all of them.
// counts (shared): [W][E], W warps each with a run of the pairs.
__device__ __forceinline__ void place_pairs(const GroupRouteArgs& a, const int* before, int* all, int* counts) {
  __shared__ int wsum[GR_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
  const int W = min(GR_WARPS, GR_COUNTS / E);
  // offsets: an exclusive scan of all over the experts, thread e its own
  const int mine = tid < E ? all[tid] : 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  for (int i = tid; i < W * E; i += GR_THREADS) counts[i] = 0;
  __syncthreads();
  int off = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < GR_WARPS; ++w) {
    if (w < warp) off += wsum[w];
    total += wsum[w];
  }
  if (tid < E) {
    all[tid] = off;
    if (blockIdx.x == 0) a.offsets[tid] = off;
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[E] = total;
  const long long P = (long long)a.T * a.k;
  const long long p0 = min((long long)blockIdx.x * a.per_block * a.k, P), p1 = min(p0 + (long long)a.per_block * a.k, P);
  const long long share = ((p1 - p0 + W - 1) / W + 31) / 32 * 32;
  const long long q0 = min(p0 + warp * share, p1), q1 = warp < W ? min(q0 + share, p1) : q0;
  int* next = counts + warp * E;
  for (long long i = q0 + lane; i < q1; i += 32) {
    const int e = __ldcg(a.idx + i);
    if (e >= 0) atomicAdd(&next[e], 1);
  }
  __syncthreads();
  if (tid < E) {   // counts become first positions
    int pos = all[tid] + before[tid];
    for (int w = 0; w < W; ++w) {
      const int c = counts[w * E + tid];
      counts[w * E + tid] = pos;
      pos += c;
    }
  }
  __syncthreads();
  for (long long i0 = q0; i0 < q1; i0 += 32) {
    const long long i = i0 + lane;
    const int e = i < q1 ? __ldcg(a.idx + i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    int pos = 0;
    if (e >= 0) pos = next[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0) {
      a.pairs[pos] = (int)i;
      a.rows[pos] = (int)(i / a.k);
      if (lane == 31 - __clz(same)) next[e] = pos + 1;
    }
    __syncwarp();
  }
  // no pair stands behind the last group
  for (long long i = max(p0, (long long)total) + tid; i < p1; i += GR_THREADS) {
    a.pairs[i] = -1;
    a.rows[i] = -1;
  }
}

template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) group_one_kernel(GroupRouteArgs a) {
  extern __shared__ int counts[];
  __shared__ int all[1024], before[1024];
  pdl_wait();
  select_tokens<NV>(a, all);
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) before[e] = 0;
  __syncthreads();
  place_pairs(a, before, all, counts);
}

template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) group_select_kernel(GroupRouteArgs a) {
  __shared__ int hist[1024];
  pdl_launch_dependents();
  pdl_wait();
  select_tokens<NV>(a, hist);
  for (int e = threadIdx.x; e < a.E; e += GR_THREADS) a.hist[(long long)blockIdx.x * a.E + e] = hist[e];
}

__global__ void __launch_bounds__(GR_THREADS, 1) group_place_kernel(GroupRouteArgs a) {
  extern __shared__ int counts[];
  __shared__ int all[1024], before[1024];
  all[threadIdx.x] = before[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait();
  // thread (part, e): an expert's counts of every parts-th block
  const int Ep = (a.E + 31) & ~31, parts = GR_THREADS / Ep, part = threadIdx.x / Ep, e = threadIdx.x % Ep;
  if (part < parts && e < a.E) {
    int s = 0, p = 0;
    // each block starts at another row, so that they do not all read the same lines at once
    const int n = (a.blocks - part + parts - 1) / parts, start = n > 0 ? (int)(blockIdx.x % n) : 0;
#pragma unroll 16
    for (int i = 0; i < n; ++i) {
      const int r = i + start < n ? i + start : i + start - n, b = part + r * parts;
      const int c = __ldcg(a.hist + (long long)b * a.E + e);
      s += c;
      if (b < (int)blockIdx.x) p += c;
    }
    atomicAdd(&all[e], s);
    atomicAdd(&before[e], p);
  }
  __syncthreads();
  place_pairs(a, before, all, counts);
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), int blocks, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(GR_THREADS);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

template <int NV>
cudaError_t launch_as(const GroupRouteArgs& a, cudaStream_t s) {
  const int warps = GR_COUNTS / a.E < GR_WARPS ? GR_COUNTS / a.E : GR_WARPS;
  const size_t smem = (size_t)warps * a.E * sizeof(int);
  if (a.blocks == 1) return launch(group_one_kernel<NV>, 1, smem, s, a);
  cudaError_t e = launch(group_select_kernel<NV>, a.blocks, 0, s, a);
  return e != cudaSuccess ? e : launch(group_place_kernel, a.blocks, smem, s, a);
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
  p.per_block = T <= GR_ONE_BLOCK ? T : (T + kBlocks - 1) / kBlocks;
  if (T > GR_ONE_BLOCK && p.per_block < GR_WARPS) p.per_block = GR_WARPS;
  p.blocks = (T + p.per_block - 1) / p.per_block;
  p.workspace = p.blocks > 1 ? (size_t)p.blocks * E * sizeof(int) : 0;
  return p;
}

cudaError_t launch_group_route(const GroupRouteArgs& a, cudaStream_t s) {
  if (a.E <= 128) return launch_as<4>(a, s);
  if (a.E <= 256) return launch_as<8>(a, s);
  return a.E <= 512 ? launch_as<16>(a, s) : launch_as<32>(a, s);
}

}  // namespace moe
