// grouped_mma.cuh - tcgen05, TMA and cluster helpers of the grouped products.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "grouped.h"

namespace moe {

// ---------------------------------------------------------------- shared-memory operand tiles
// Both layouts are 128-byte swizzled, as the TMA writes them, in 16-bit elements:
//   K-major: rows of 64 contracted elements (128 B); 8 rows make a 1024 B group, groups along
//     the rows follow each other.  A K = 16 step is 32 B further.
//   MN-major: 64 contracted rows of 64 elements of the other dimension (128 B each, 8 KB in
//     all), slabs of 64 elements following each other.  A K = 16 step is 16 rows = 2048 B further.
constexpr uint32_t SLAB_BYTES = 64 * 128;
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, bool mn_major) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(mn_major ? SLAB_BYTES >> 4 : 1) << 16;   // MN-major: slab to slab
  d |= (uint64_t)(1024 >> 4) << 32;                        // 8-row group to 8-row group
  d |= (uint64_t)1 << 46;                                  // descriptor version
  d |= (uint64_t)2 << 61;                                  // 128-byte swizzle
  return d;
}
// kind::f16 with fp32 sums; A and B both bf16 or both fp16
__host__ __device__ __forceinline__ uint32_t idesc_16(bool bf16, bool a_mn, bool b_mn, int M, int N) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// kind::f8f6f4 with fp32 sums, A and B e4m3, both K-major; a step is K = 32, the same 32 B
__host__ __device__ __forceinline__ uint32_t idesc_8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// true in one lane of the warp (all of it calls)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

template <int CG>
__device__ __forceinline__ void umma(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool acc) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void umma_8(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool acc) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// every mma issued so far by this thread arrives, when done, on the barrier: of this block, or at the same
// place in both blocks of the pair
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void umma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void umma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// 32 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// g sigma(g), by e^-|g|: the quick division gives 0 where 1 + e^-g is past 2^126, and e^-g is infinite past that, where the
// result is still a number of its type.  The exact division costs 0.6% of the Mixtral-shaped gate/up product of 1001 tokens (372
// and 374 us).
__device__ __forceinline__ float silu(float g) {
  const float e = expf(-fabsf(g));
  return g * ((g < 0.f ? e : 1.f) / (1.f + e));
}

// The same with a quick division, whose denominator is 1 to 2 here: within three steps of fp32, and fewer instructions where the
// products are as quick as their epilogue (8 bits).
__device__ __forceinline__ float silu_quick(float g) {
  const float e = expf(-fabsf(g));
  return g * __fdividef(g < 0.f ? e : 1.f, 1.f + e);
}

// two results rounded to a 16-bit type
__device__ __forceinline__ uint32_t pack_out(float lo, float hi, int dtype) {
  if (dtype == GT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- tiles
// The want-th tile of up to nt_rows rows over the groups, by one warp: its group and rows (e = -1: there is none).  Each lane
// counts a run of consecutive groups.
__device__ __forceinline__ void find_tile(const GroupedProblem& p, int nt_rows, int want, int lane, int& e, int& r0, int& r1) {
  const int run = (p.groups + 31) / 32, g0 = lane * run, g1 = min(g0 + run, p.groups);
  int mine = 0;
#pragma unroll 8
  for (int g = g0; g < g1; ++g) {
    int a, b;
    group_range(p.offsets, g, p.m, a, b);
    mine += (b - a + nt_rows - 1) / nt_rows;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  const int before = inc - mine;
  const unsigned who = __ballot_sync(0xffffffffu, want >= before && want < inc);
  e = -1;
  r0 = r1 = 0;
  if (!who) return;
  const int l = __ffs(who) - 1;
  if (lane == l) {
    int left = want - before;
    for (int g = g0; g < g1; ++g) {
      int a, b;
      group_range(p.offsets, g, p.m, a, b);
      const int nt = (b - a + nt_rows - 1) / nt_rows;
      if (left < nt) {
        e = g;
        r0 = a + left * nt_rows;
        r1 = min(b, r0 + nt_rows);
        break;
      }
      left -= nt;
    }
  }
  e = __shfl_sync(0xffffffffu, e, l);
  r0 = __shfl_sync(0xffffffffu, r0, l);
  r1 = __shfl_sync(0xffffffffu, r1, l);
}

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on a barrier of another block.  It announces that tensor memory has been read (ordered by the fences around that), or
// that rows of this block's own shared memory have been cleared, which the fence to the async proxy in front of it has made
// visible to the tensor core that reads them there.  A release at cluster scope would add a round trip through L2 to each
// (clearing: DeepSeek-V3-shaped weight gradient 335 and 410 us, Mixtral-shaped 650 and 697).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Every wait of the grouped kernels is bounded: by WaitLimit, as a rule about a second, far beyond any part of a tile, and where
// a warp waits across more steps of 64 elements, by 30 times what one takes for each of them on top.
constexpr unsigned long long WAIT_STEP = 16384;
// after a wait ran out: long enough for every copy and product in flight to end
constexpr long long DRAIN_CYCLES = 100000000ll;
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const WaitLimit& limit, unsigned long long steps = 0) {
  return mbar_wait_bounded(bar, parity, limit.cycles + steps * WAIT_STEP);
}
// Arrivals on the barrier of a stage's operands, n of them.  Under a bound of no cycles it is one more, which never comes: the
// hardware suspends a waiting thread for longer than the operands take, so a short bound alone would not run out.
__device__ __forceinline__ uint32_t stage_arrivals(const WaitLimit& limit, uint32_t n) { return n + (limit.cycles == 0); }
__device__ __forceinline__ void report_wait(const WaitLimit& limit) {
  *reinterpret_cast<volatile uint32_t*>(limit.status) = ST_TIMEOUT;
  __threadfence_system();
}
__device__ __forceinline__ void drain_time() {
  const long long t0 = clock64();
  while (clock64() - t0 < DRAIN_CYCLES) __nanosleep(1000);
}

// ---------------------------------------------------------------- tensor-map loads (128-byte swizzled tiles)
// CG = 2: the barrier may be the pair's first block's (a cluster address)
template <int CG>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* m, int a, int b, int c, int d, int e,
                                       uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(m), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(m), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(bar)
        : "memory");
}
// four rows named by number (a tensor map of one-row boxes; a number outside the tensor gives zeros)
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* m, int x, int4 r, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5, %6}], [%7];" ::"r"(dst),
      "l"(m), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
      : "memory");
}
// a box of shared memory to global memory, as a bulk group of this thread; the first to leave L2, which the
// operands need (3% of a weight gradient bound by its results)
__device__ __forceinline__ void tma_store_3d(uint32_t src, const CUtensorMap* m, int x, int y, int z) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(m),
      "r"(x), "r"(y), "r"(z), "r"(src), "l"(policy)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

}  // namespace moe
