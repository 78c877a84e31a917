// group_route.cu - router selection of a batch from its logits, pairs grouped by expert.
//
// A block takes a slice of the tokens; each warp selects one token's k experts at a time (k rounds of two warp
// reductions over order-preserving keys of the logits), writes ids and weights, and the block counts its
// pairs by expert.  Then a block sums the counts of the blocks before it, scans the experts' totals into offsets,
// and places its pairs in order: a stable counting sort, in which no atomic decides a position, so the same logits give
// the same arrays.  Up to 64 tokens are one block of one launch; more are two launches over one block of 32 warps an SM, the
// second waiting for the first on the device.  Bound: the
// integer pipe while selecting (about 300 instructions a token), latency while placing: 16384 tokens of 256 bf16 logits,
// k = 8, take 21 us (13 selecting; 10 MB, 1.5 us at the memory's rate), one token 5.7 us.
#include "common.cuh"
#include "group_route.h"
#include "grouped.h"
#include "grouped_mma.cuh"
#include "route.cuh"

namespace moe {

namespace {

constexpr int GR_THREADS = 1024;
constexpr int GR_WARPS = GR_THREADS / 32;
constexpr int GR_ONE_BLOCK = 64;      // tokens of the one-launch form: two a warp
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

// Keys carry the expert in their low 10 bits, a lower one larger, so each is unique and none is 0 but the masked ones.  16-bit
// logits fit the 22 bits above whole; of fp32 logits those are the leading ones.
template <int NV>
__device__ __forceinline__ void token_keys(const GroupRouteArgs& a, int lane, const float (&l)[NV], uint32_t (&key)[NV]) {
  constexpr uint32_t inf = 0xff800000u;   // key of +inf, which counts as the one below
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float x = l[i];
    if (a.dtype == GT_BF16) x = __uint_as_float(__float_as_uint(x) << 16);
    if (a.dtype == GT_FP16) x = __half2float(__ushort_as_half((unsigned short)__float_as_uint(x)));
    const bool live = x > -INFINITY && lane + 32 * i < a.E;   // NaN is not
    key[i] = live ? (min(logit_key(x), inf - 1u) & ~1023u) | (uint32_t)(1023 - lane - 32 * i) : 0u;
  }
}

// one comparator of a sorting network over the warp: of the pair (lane, lane ^ j) the lower lane keeps the larger key where
// `down`, the smaller one otherwise
__device__ __forceinline__ uint32_t comparator(uint32_t v, int j, bool down, int lane) {
  const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
  return (((lane & j) == 0) == down) ? max(v, o) : min(v, o);
}

// The first n of the keys in descending order, lane j the j-th (0: none), for n <= SORTED: the lanes' largest and second
// keys are sorted over the warp (descending and ascending) and merged, 35 comparators in all, which is right unless some
// lane's third belongs to the n (one token in 20 for 8 of 256).  Returns false then.
constexpr int SORTED = 10;
template <int NV>
__device__ __forceinline__ bool sorted_keys(const uint32_t (&key)[NV], int n, int lane, uint32_t& mine) {
  uint32_t b1 = 0, b2 = 0, b3 = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t x = min(b1, key[i]), y = min(b2, x);
    b1 = max(b1, key[i]);
    b2 = max(b2, x);
    b3 = max(b3, y);
  }
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) {
      b1 = comparator(b1, j, (lane & k) == 0 || k == 32, lane);
      b2 = comparator(b2, j, !((lane & k) == 0 || k == 32), lane);
    }
  uint32_t v = max(b1, b2);   // one falling, one rising: the 32 largest of both, as a bitonic sequence
#pragma unroll
  for (int j = 16; j; j >>= 1) v = comparator(v, j, true, lane);
  mine = v;
  return !__any_sync(0xffffffffu, b3 > __shfl_sync(0xffffffffu, v, n - 1));
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

// The k best of one token, by one warp: lane j < k receives the j-th id (-1: none left).  Of fp32 logits one more key than k
// shows whether two neighbours in the order share their leading bits (1 or 2 tokens in 100 of random ones).  Among the
// k they are then ordered by their whole keys; if the k-th and the one behind it share them, or the latter is not
// known (k = 32), the token is selected again from whole keys, with a second maximum for the id.
template <int NV>
__device__ __forceinline__ int token_topk(const GroupRouteArgs& a, long long t, int lane, const float (&l)[NV]) {
  uint32_t key[NV], mine = 0;
  token_keys<NV>(a, lane, l, key);
  const int n = a.dtype == GT_FP32 ? min(a.k + 1, 32) : a.k;
  if (n > SORTED || !sorted_keys<NV>(key, n, lane, mine)) mine = rounds_of_keys<NV>(key, n, lane);
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

// one token by one warp: its ids and weights
template <int NV>
__device__ __forceinline__ int route_token(const GroupRouteArgs& a, long long t, int lane, const float (&logits)[NV]) {
  const int e = token_topk<NV>(a, t, lane, logits);
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
  const long long t0 = min((long long)blockIdx.x * a.per_block, (long long)a.T), t1 = min(t0 + a.per_block, (long long)a.T);
  float l[NV], ahead[NV];
  if (t0 + warp < t1) load_token<NV>(a, t0 + warp, lane, ahead);
  for (long long t = t0 + warp; t < t1; t += GR_WARPS) {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = ahead[i];
    if (NV <= 8 && t + GR_WARPS < t1) load_token<NV>(a, t + GR_WARPS, lane, ahead);   // while this token is selected
    const int e = route_token<NV>(a, t, lane, l);
    if (NV > 8 && t + GR_WARPS < t1) load_token<NV>(a, t + GR_WARPS, lane, ahead);
    if (lane < a.k && e >= 0) atomicAdd(&hist[e], 1);   // a count: its order does not matter
  }
  __syncthreads();
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
// Places this block's pairs.  before, all (shared, [E]): an expert's pairs in earlier blocks and in all of them.
__device__ __forceinline__ void place_pairs(const GroupRouteArgs& a, const Pairs& s, const int* before, const int* all, int* counts) {
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

template <int NV>
__global__ void __launch_bounds__(GR_THREADS, 1) group_one_kernel(GroupRouteArgs a) {
  extern __shared__ int counts[];
  __shared__ int all[1024], before[1024];
  const Pairs s = block_pairs(a, counts);
  for (int i = threadIdx.x; i < s.W * a.E; i += GR_THREADS) counts[i] = 0;
  before[threadIdx.x] = 0;
  pdl_wait();
  select_tokens<NV>(a, all);
  count_pairs(a, s);
  __syncthreads();
  place_pairs(a, s, before, all, counts);
}

// The counts leave by clusters, hist [clusters][E], with each block's share of its cluster's before it, [blocks][E] behind:
// the next kernel's blocks then read half of the rows (read one by one, they took half of that kernel's time).
template <int NV>
__global__ void __cluster_dims__(GR_CLUSTER, 1, 1) __launch_bounds__(GR_THREADS, 1) group_select_kernel(GroupRouteArgs a) {
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
  place_pairs(a, pairs, before, all, counts);
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
  p.per_block = T <= GR_ONE_BLOCK ? T : (T - 1) / kBlocks + 1;
  if (T > GR_ONE_BLOCK && p.per_block < GR_WARPS) p.per_block = GR_WARPS;
  p.blocks = (T - 1) / p.per_block + 1;
  if (T > GR_ONE_BLOCK) p.blocks = (p.blocks + GR_CLUSTER - 1) / GR_CLUSTER * GR_CLUSTER;   // some without tokens
  p.workspace = T > GR_ONE_BLOCK ? (size_t)(p.blocks + p.blocks / GR_CLUSTER) * E * sizeof(int) : 0;
  return p;
}

cudaError_t launch_group_route(const GroupRouteArgs& a, cudaStream_t s) {
  if (a.E <= 128) return launch_as<4>(a, s);
  if (a.E <= 256) return launch_as<8>(a, s);
  return a.E <= 512 ? launch_as<16>(a, s) : launch_as<32>(a, s);
}

}  // namespace moe
