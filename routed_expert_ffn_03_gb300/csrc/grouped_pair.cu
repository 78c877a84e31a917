// grouped_pair.cu - grouped 16-bit products on the tensor cores, one tile per pair of SMs.
//
//   forward:          D^T[f][t] = sum_k W_e[f][k] x[t][k]      f: 256 features, t: up to 256 of a group's rows
//   weight gradient:  dW_e[n][k] = sum_i dy[i][n] x[i][k]      n: 256, k: 256, i: a group's rows
//
// Both are one tcgen05 product of a pair of blocks (cta_group::2, M = 256): each block stages its
// 128 rows of the first factor and its half of the second in shared memory, and holds its
// 128 rows of the result in tensor memory.  The weights are the first factor of the forward
// product, so that a group's rows are the N of the instruction, which takes any multiple
// of 32: a group of 40 rows costs 64 columns and not a tile of 128 or 256 (with the rows as M it would).
// The pair halves what each SM fetches: 64 contracted elements take 32 KB for 512
// tensor cycles, where single blocks of 128 x 256 would take 48 KB.
//
// Persistent pairs walk the tiles; the warps of a block have fixed roles:
//   warp 0      copies operands by TMA into a ring of 6 stages (64 contracted elements each), in forward products the weights;
//   warp 1      of the first block issues the products for both;
//   warps 2..9  read finished results from tensor memory and store them, while the next
//               tile's products run into the other half of the 512 columns;
//   warp 10     in forward products copies the rows.  Where a weight gradient's group ends inside a step, it clears the rows
//               behind it in both factors, so that nothing of a neighbour enters a sum (zeros in one factor
//               alone would let the other's NaN through).
// Copies are issued by an elected thread of a warp that walks its loop together, and by two warps, as each instruction counts:
// from a branch of single lanes of one warp the Mixtral-shaped gate/up product takes 440 us for 1001 tokens and 682 for 2048
// instead of 385 and 587, the fp32 weight gradient 716 instead of 663.
// Rows named by number are copied side by side by a kernel of their own first (memory bound; 1% of a
// Mixtral-shaped gate/up product's time) and then come as tiles.  Measured against that, for the Mixtral-shaped down
// product of 8192 tokens (1160 us from tiles): TMA gather 4014 us (~76 cycles an instruction of 4 rows), cp.async by
// 4 warps into the same stages 1379 to 2072 us (its shared-memory writes wait behind the tensor core's reads).
// 16384 rows over 8 groups, k = 14336, n = 4096: 513 cycles a step, the tensor core's own; 1100 us, 1750 TFLOP/s, and up to
// 1250 in a long row of them, where the card's power limit holds the clock down.
// Tiles of a group go rows first within bands of 8 row tiles, so the pairs at work share
// weights and rows in L2.
#include "grouped.h"
#include "grouped_mma.cuh"

namespace moe {

namespace {

enum : int { GP_NK = 0, GP_KN = 1, GP_SWIGLU = 2, GP_WGRAD = 3, GP_NK8 = 4, GP_SWIGLU8 = 5 };
template <int MODE>
constexpr bool GP_IS_8 = MODE == GP_NK8 || MODE == GP_SWIGLU8;
template <int MODE>
constexpr bool GP_IS_SWIGLU = MODE == GP_SWIGLU || MODE == GP_SWIGLU8;
template <int MODE>
constexpr int GP_STEP = GP_IS_8<MODE> ? 128 : 64;   // contracted elements of a stage: 128 bytes

// stages of the ring, and per storing warp one box of results on its way out (weight gradient).  5 stages and two boxes
// were 8% slower (Mixtral-shaped, fp32 results: 765 and 711 us).
constexpr int GP_STAGES = 6;
constexpr int GP_OP = 128 * 128;                 // bytes of one factor's half stage: 128 rows x 64 elements
constexpr int GP_STAGE = 2 * GP_OP;
constexpr int GP_EPI_WARPS = 8;
constexpr int GP_CLEAR_WARP = 2 + GP_EPI_WARPS, GP_ROW_WARP = GP_CLEAR_WARP;   // weight gradient; forward
constexpr int GP_THREADS = (GP_CLEAR_WARP + 1) * 32;
constexpr int GP_MAX_GROUPS = 1024;
// The tensor core's running sum drops bits at every step (K = 16) instead of rounding, always towards zero, which costs about
// 2e-8 of the result a step: 1.3e-6 after 1024 elements, where fp32 sums rounded
// at every step are off by 3e-7.  fp32 results are therefore summed in parts of 8 stages (512 elements), which
// the storing warps add up in registers, rounding to nearest, while the next part's products run: 4 to 6e-7.  With swiglu the
// errors of gate and up add up, and parts are 4 stages: 6.9e-7 instead of 1.3e-6, for 7% more time (415 and 445 us for
// 1001 Mixtral-shaped tokens; in a weight gradient 4 stages would cost 8%).
// 16-bit results are summed in one go up to GP_LONG stages (16384 elements: 2e-5, a 24th of an fp16 half step) and in
// parts beyond, where the error would go on growing: an fp16 half step at 400 thousand elements.  Parts cost a forward product
// 3% there (4096 rows in 4 groups, n = 4096, k = 16448: 326 and 338 us; with swiglu 6%), a weight gradient 1%.
// In 8 bits a step is K = 32, a stage and a part twice the elements.  Where every step loses all that it can (2^-23 of the sum), 32
// steps cost 2e-6 and 1024 cost 8e-5, measured.
template <int MODE>
constexpr int GP_PART = GP_IS_SWIGLU<MODE> ? 4 : 8;
constexpr int GP_LONG = 256;
enum : int { GP_OUT_16 = 0, GP_OUT_16_LONG = 1, GP_OUT_32 = 2 };   // results, and whether contractions past GP_LONG may come
constexpr int GP_BAND = 8;                       // row tiles of a band
constexpr int GP_OUT = 4096;                     // a warp's box of results: 32 rows of 128 bytes
constexpr int GP_OFF_OUT = GP_STAGES * GP_STAGE;      // weight gradient
constexpr int GP_OFF_TAB = GP_OFF_OUT;           // forward: first tile of each group [groups + 1]
constexpr int GP_OFF_SCAN = GP_OFF_TAB + (GP_MAX_GROUPS + 2) * 4;
constexpr int GP_OFF_BAR = GP_OFF_OUT + GP_EPI_WARPS * GP_OUT;
constexpr int GP_BARS = 4 * GP_STAGES + 4;
constexpr int GP_SMEM = GP_OFF_BAR + GP_BARS * 8 + 16 + 1024;   // and 1024 to align the stages
static_assert(GP_OFF_SCAN % 8 == 0 && GP_OFF_SCAN + GP_THREADS / 32 * 8 <= GP_OFF_BAR && GP_SMEM <= 227 * 1024, "shared memory");

struct PairArgs {
  GroupedProblem p;
  int nft, nkt;        // forward: feature tiles; weight gradient: n tiles and k tiles
  int max_tiles;       // the most that m rows can make
  WaitLimit wait;
  bool wide;           // results can be stored as 4-byte pairs (forward) or by TMA (weight gradient)
  bool by_16;          // swiglu: W_e in boxes of 16 rows
};

struct Tile {
  int e, f0;           // group; first feature (forward), first n (weight gradient)
  int r0, rows;        // forward: the tile's rows; weight gradient: the group's rows
  int n;               // columns of the product: rows rounded up to 32, or 256
  int c0;              // weight gradient: first k
  int nkb;             // steps of 64
};

__device__ __forceinline__ void store1(void* d, long long at, float v, int t) {
  if (t == GT_FP32) static_cast<float*>(d)[at] = v;
  else if (t == GT_BF16) static_cast<__nv_bfloat16*>(d)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(d)[at] = __float2half_rn(v);
}

// stores without a branch around each
__device__ __forceinline__ void store32_if(bool live, void* at, uint32_t v) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.b32 [%0], %1;\n}\n" ::"l"(at), "r"(v),
               "r"((uint32_t)live)
               : "memory");
}
__device__ __forceinline__ void store16_if(bool live, void* at, uint32_t v) {
  asm volatile("{\n .reg .pred p;\n .reg .b16 l, h;\n setp.ne.u32 p, %2, 0;\n mov.b32 {l, h}, %1;\n @p st.global.b16 [%0], l;\n}\n" ::"l"(at),
               "r"(v), "r"((uint32_t)live)
               : "memory");
}

// the tile with number `t` (first[g] = first tile of group g)
template <int MODE>
__device__ __forceinline__ Tile decode(const PairArgs& a, const int* first, int t) {
  Tile T;
  const GroupedProblem& p = a.p;
  if (MODE == GP_WGRAD) {
    const int per = a.nft * a.nkt;
    T.e = t / per;
    int i = t - T.e * per;
    const int band = i / (GP_BAND * a.nkt), in = i - band * GP_BAND * a.nkt;
    const int h = min(GP_BAND, a.nft - band * GP_BAND);
    T.f0 = (band * GP_BAND + in % h) * 256;
    T.c0 = in / h * 256;
    int r1;
    group_range(p.offsets, T.e, p.m, T.r0, r1);
    T.rows = r1 - T.r0;
    T.n = 256;
    T.nkb = (T.rows + 63) / 64;
    return T;
  }
  int lo = 0, hi = p.groups;   // last group whose first tile is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  T.e = lo;
  int r1;
  group_range(p.offsets, lo, p.m, T.r0, r1);
  const int R = r1 - T.r0, nt = (R + 255) / 256;
  const int i = t - first[lo];
  const int band = i / (GP_BAND * a.nft), in = i - band * GP_BAND * a.nft;
  const int h = min(GP_BAND, nt - band * GP_BAND);
  const int rt = band * GP_BAND + in % h;
  T.f0 = in / h * (GP_IS_SWIGLU<MODE> ? 128 : 256);
  // the group's 32s of rows in even parts: a tile of few rows would wait for its weights
  const int units = (R + 31) / 32, base = units / nt, more = units - base * nt;
  const int at = (rt * base + min(rt, more)) * 32;
  T.rows = min(R - at, (base + (rt < more)) * 32);
  T.r0 += at;
  T.n = (T.rows + 31) & ~31;
  T.c0 = 0;
  T.nkb = (p.k + GP_STEP<MODE> - 1) / GP_STEP<MODE>;
  return T;
}

template <int MODE, int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GP_THREADS, 1)
    grouped_pair_kernel(const __grid_constant__ PairArgs a, const __grid_constant__ GroupedMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const GroupedProblem& p = a.p;
  constexpr bool WG = MODE == GP_WGRAD, SW = GP_IS_SWIGLU<MODE>, F32 = OUT == GP_OUT_32, F8 = GP_IS_8<MODE>;
  constexpr int STEP = GP_STEP<MODE>;
  constexpr bool PARTS = OUT != GP_OUT_16;   // sums in registers

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + GP_OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + GP_OFF_BAR + GP_BARS * 8);
  volatile int* s_abort = reinterpret_cast<int*>(smem + GP_OFF_BAR + GP_BARS * 8 + 4);
  int* first = reinterpret_cast<int*>(smem + GP_OFF_TAB);
  long long* scan = reinterpret_cast<long long*>(smem + GP_OFF_SCAN);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * GP_STAGES;
  const uint32_t land0 = empty0 + 8 * GP_STAGES, ready0 = land0 + 8 * GP_STAGES;
  const uint32_t tfull0 = ready0 + 8 * GP_STAGES, tempty0 = tfull0 + 16;

  if (tid == 0) {
    for (int s = 0; s < GP_STAGES; ++s) {
      mbar_init(full0 + 8 * s, stage_arrivals(a.wait, 1));   // first block's: its own arrival, both blocks' bytes
      mbar_init(empty0 + 8 * s, 1);    // the products that read the stage
      mbar_init(land0 + 8 * s, 1);     // this block's tiles of a step that has rows to clear
      mbar_init(ready0 + 8 * s, 2);    // first block's: both blocks have cleared theirs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * GP_EPI_WARPS);   // first block's: the storing warps of both
    }
    *s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b[0]);
  }
  pdl_wait();   // the copy of named rows, where there is one (and through it all work before)
  // first tile of each group: thread i scans groups 4 i .. 4 i + 3
  int total;
  if (WG) {
    total = p.groups * a.nft * a.nkt;
  } else {
    long long nt[4], mine = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int g = 4 * tid + q;
      int r0 = 0, r1 = 0;
      if (g < p.groups) group_range(p.offsets, g, p.m, r0, r1);
      nt[q] = (r1 - r0 + 255ll) / 256 * a.nft;
      mine += nt[q];
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long long off = inc - mine, all = 0;
#pragma unroll
    for (int w = 0; w < GP_THREADS / 32; ++w) {
      if (w < warp) off += scan[w];
      all += scan[w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (4 * tid + q < p.groups) first[4 * tid + q] = (int)off;
      off += nt[q];
    }
    // more than m rows can make: the offsets are not non-decreasing, and nothing is done
    total = all <= a.max_tiles ? (int)all : 0;
  }
  umma_fence_before();
  __syncthreads();
  cluster_sync_all();   // barriers of both blocks exist before either signals the other
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;
  // steps of a part of a tile's sum
  auto part_steps = [](int nkb) { return F32 || (PARTS && nkb > GP_LONG) ? GP_PART<MODE> : max(nkb, 1); };
  // whether the group ends inside step kb
  auto clears = [&](const Tile& T, int kb) { return WG && T.rows - kb * 64 < 64; };
  const int pair = blockIdx.x >> 1, npair = gridDim.x >> 1;
  const uint32_t s0 = smem_u32(smem);

  if (warp == 0 || (!WG && warp == GP_ROW_WARP)) {
    // ---------------------------------------------------------------- copies
    // As with the products below, the warp walks the loop together and one elected thread issues.  Forward: warp 0 the weights,
    // warp 10 the rows.
    const bool leader = elect_one(), weights = warp == 0;
    const uint32_t pair_full0 = __shfl_sync(0xffffffffu, map_rank(full0, 0), 0), base = __shfl_sync(0xffffffffu, s0, 0);
    const int side = __shfl_sync(0xffffffffu, (int)rank, 0);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = pair; t < total && ok; t += npair) {
      const Tile T = decode<MODE>(a, first, t);
      const int nkb = __shfl_sync(0xffffffffu, T.nkb, 0), half = __shfl_sync(0xffffffffu, T.n, 0) / 2;   // rows of B in each block
      const int e = __shfl_sync(0xffffffffu, T.e, 0), r0 = __shfl_sync(0xffffffffu, T.r0, 0);
      const int f0 = __shfl_sync(0xffffffffu, T.f0, 0), c0 = __shfl_sync(0xffffffffu, T.c0, 0);
      const int f = f0 + side * (SW ? 64 : 128), fb = c0 + side * 128, rb = r0 + side * half;
      const uint32_t bytes = GP_OP + (WG ? GP_OP : half * 128);   // of a step, in each block
      for (int kb = 0; kb < nkb; ++kb) {
        ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ph ^ 1, a.wait));
        if (!ok) break;
        // a step whose rows behind the group are to be cleared is announced to the block's own warp 10
        const bool clear = clears(T, kb);
        const uint32_t bar = (clear ? land0 : pair_full0) + 8 * s;
        const uint32_t da = base + s * GP_STAGE, db = da + GP_OP;
        if (leader) {
          if (weights) {
            if (clear) mbar_arrive_expect_tx(bar, bytes);
            if (side == 0) {
              if (clear) mbar_arrive(full0 + 8 * s);
              else mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
            }
          }
          if (WG) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tma_2d<2>(da + h * SLAB_BYTES, &maps.a, f + h * 64, r0 + kb * 64, bar);
              tma_2d<2>(db + h * SLAB_BYTES, &maps.b[0], fb + h * 64, r0 + kb * 64, bar);
            }
          } else if (weights) {
            if (MODE == GP_NK || MODE == GP_NK8) tma_3d<2>(da, &maps.a, kb * STEP, f, e, bar);
            if (SW && !a.by_16) tma_5d<2>(da, &maps.a, kb * STEP, 0, 0, f / 16, e, bar);
            if (SW && a.by_16)   // gate and up in turn, 16 rows each
              for (int i = 0; i < 8; ++i)
                tma_3d<2>(da + i * 2048, &maps.a, kb * STEP, f + (i >> 1) * 16 + (i & 1) * (p.n / 2), e, bar);
            if (MODE == GP_KN) {
              tma_3d<2>(da, &maps.a, f, kb * 64, e, bar);
              tma_3d<2>(da + SLAB_BYTES, &maps.a, f + 64, kb * 64, e, bar);
            }
          } else {
            // the half's rows, a multiple of 16, in boxes of 128, 64, 32 and 16
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int box = 16 << i, before = half & ~(2 * box - 1);
              if (half & box) tma_2d<2>(db + before * 128, &maps.b[i], kb * STEP, rb + before, bar);
            }
          }
        }
        __syncwarp();
        if (++s == GP_STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // the first block's products signal this block's barriers: they have all done so before it may exit
    for (int i = 0; i < GP_STAGES && ok; ++i) {
      ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ph ^ 1, a.wait));
      if (++s == GP_STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    // One elected thread issues, but the warp walks the loop together: the operands of the instructions then
    // sit in uniform registers.  Issued inside a lane's own branch each of them is moved there first, some 90 cycles
    // an instruction, and a step takes 650 cycles instead of the tensor core's 512.
    if (rank == 0) {
      const bool leader = elect_one();
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0, ready_ph = 0;   // ready_ph: a bit per stage, as not every step uses its barrier
      bool ok = true;
      constexpr bool a_mn = MODE == GP_KN || WG, b_mn = WG;
      constexpr uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
      const uint32_t base = __shfl_sync(0xffffffffu, s0, 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t da0 = sw128_desc(base, a_mn), db0 = sw128_desc(base + GP_OP, b_mn);
      const uint32_t idesc0 = F8 ? idesc_8(256, 0) : idesc_16(p.dtype == GT_BF16, a_mn, b_mn, 256, 0);
      Tile T{};
      if (pair < total) T = decode<MODE>(a, first, pair);
      for (int t = pair; t < total && ok; t += npair) {
        const int nkb = __shfl_sync(0xffffffffu, T.nkb, 0), n = __shfl_sync(0xffffffffu, T.n, 0);
        const int last_rows = __shfl_sync(0xffffffffu, T.rows, 0) - (nkb - 1) * 64;
        const uint32_t idesc = idesc0 | ((uint32_t)(n >> 3) << 17);
        if (t + npair < total) T = decode<MODE>(a, first, t + npair);   // while this tile's products are queued
        const int steps = part_steps(nkb);
        for (int kb0 = 0; kb0 < nkb && ok; kb0 += steps) {
          const int kb1 = min(kb0 + steps, nkb);
          ok = __all_sync(0xffffffffu, wait_bar(tempty0 + 8 * acc, aph ^ 1, a.wait));
          umma_fence_after();
          const uint32_t dst = tm + acc * 256;
          for (int kb = kb0; kb < kb1 && ok; ++kb) {
            ok = __all_sync(0xffffffffu, wait_bar(full0 + 8 * s, ph, a.wait));
            if (WG && kb == nkb - 1 && last_rows < 64) {   // rows behind the group are being cleared
              ok = __all_sync(0xffffffffu, ok && wait_bar(ready0 + 8 * s, (ready_ph >> s) & 1, a.wait));
              ready_ph ^= 1u << s;
            }
            if (!ok) break;
            umma_fence_after();
            const uint64_t da = da0 + (uint32_t)(s * (GP_STAGE >> 4)), db = db0 + (uint32_t)(s * (GP_STAGE >> 4));
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (F8) umma_8<2>(dst, da + kk * a_step, db + kk * b_step, idesc, kb > kb0 || kk > 0);
                else umma<2>(dst, da + kk * a_step, db + kk * b_step, idesc, kb > kb0 || kk > 0);
              }
              umma_commit_pair(empty0 + 8 * s);
            }
            __syncwarp();
            if (++s == GP_STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          if (leader) umma_commit_pair(tfull0 + 8 * acc);
          __syncwarp();
          if (++acc == 2) {
            acc = 0;
            aph ^= 1;
          }
        }
      }
      if (!ok && lane == 0) *s_abort = 1;
    }
  } else if (warp == GP_CLEAR_WARP) {
    // ---------------------------------------------------------------- rows behind a group
    if (WG) {
      int s = 0;
      uint32_t land_ph = 0;
      unsigned long long steps = 0;   // that the ring may still have to take until the next one that is cleared
      bool ok = true;
      for (int t = pair; t < total && ok; t += npair) {
        const Tile T = decode<MODE>(a, first, t);
        if (T.nkb == 0) continue;
        s = (s + T.nkb - 1) % GP_STAGES;   // the tile's last step
        steps += T.nkb;
        if (clears(T, T.nkb - 1)) {
          ok = __all_sync(0xffffffffu, wait_bar(land0 + 8 * s, (land_ph >> s) & 1, a.wait, steps));
          steps = 0;
          land_ph ^= 1u << s;
          if (!ok) break;
          uint8_t* st = smem + s * GP_STAGE;
          const uint4 z = make_uint4(0, 0, 0, 0);
          for (int r = T.rows - (T.nkb - 1) * 64 + (lane >> 3); r < 64; r += 4) {   // 8 lanes a row, 4 slabs
            uint4* d = reinterpret_cast<uint4*>(st + r * 128 + (lane & 7) * 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q * SLAB_BYTES / 16] = z;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(ready0 + 8 * s, 0));
        }
        s = (s + 1) % GP_STAGES;
      }
      if (!ok && lane == 0) *s_abort = 1;
    }
  } else {
    // ---------------------------------------------------------------- results
    const int quarter = warp & 3, part = (warp - 2) >> 2;   // TMEM lanes this warp may read; which half of the columns
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    const int n_out = SW ? p.n / 2 : p.n;
    auto release = [&]() {   // this warp has read result `acc`
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(tempty0 + 8 * acc, 0));
      if (++acc == 2) {
        acc = 0;
        aph ^= 1;
      }
    };
    for (int t = pair; t < total; t += npair) {
      const Tile T = decode<MODE>(a, first, t);
      if (T.nkb == 0 && !WG) continue;
      // this warp's q-th run of 32 columns: its runs alternate with the other warp's of the same lanes, by twos where a
      // box of 16-bit results is made of two
      auto run_at = [&](int q) { return WG && PARTS && !F32 ? (q >> 1) * 128 + part * 64 + (q & 1) * 32 : part * 32 + 64 * q; };
      float sum[PARTS ? 4 : 1][32];
      uint32_t td = 0;
      // 8 bits: the scales of this lane's row of W_e and of its column of each run, loaded while the products run (where they are
      // wanted, a run waits two round trips for them: Mixtral-shaped gate/up of 2002 rows 200 and 195 us, 875 rows, n = 7680, k = 448 20.7 and
      // 19.4)
      float ws = 0.f, xs[F8 ? 4 : 1];
      if (F8) {
        const int f = SW ? T.f0 + (int)rank * 64 + quarter * 16 + (lane & 15) : T.f0 + (int)rank * 128 + quarter * 32 + lane;
        if (f < n_out) ws = __ldg(p.b_scale + (long long)T.e * p.n + (SW && lane >= 16 ? n_out : 0) + f);
#pragma unroll
        for (int q = 0; q < (F8 ? 4 : 1); ++q) {
          const int c = run_at(q) + lane;
          xs[q] = c < T.rows ? row_scale(p, T.r0 + c) : 0.f;
        }
      }
      if (PARTS) {
#pragma unroll
        for (int q = 0; q < (PARTS ? 4 : 1); ++q)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[q][i] = 0.f;
        for (int kb = 0; kb < T.nkb && ok; kb += part_steps(T.nkb)) {
          ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * acc, aph, a.wait));
          if (!ok) break;
          umma_fence_after();
#pragma unroll
          for (int q = 0; q < (PARTS ? 4 : 1); ++q) {
            const int c = run_at(q);
            if (c < T.n) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {   // by 16: the sums fill the registers
                float v[16];
                tmem_ld16(tmem + acc * 256 + ((uint32_t)(quarter * 32) << 16) + c + 16 * h, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[q][16 * h + i] += v[i];
              }
            }
          }
          release();
        }
        if (!ok) break;
      } else if (T.nkb > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * acc, aph, a.wait));
        if (!ok) break;
        umma_fence_after();
        td = tmem + acc * 256 + ((uint32_t)(quarter * 32) << 16);
      }
      if (WG && a.wide) {
        // boxes of 32 rows x 128 bytes, by way of shared memory (128-byte swizzled, so that 8 lanes' 16-byte
        // stores meet 32 banks): each goes out as full lines, where a thread's own row would be written in
        // 16-byte pieces.  TMA leaves out what lies behind n and k.
        constexpr int cols = F32 ? 32 : 64;
        const int n0 = T.f0 + (int)rank * 128 + quarter * 32;
        uint8_t* out = smem + GP_OFF_OUT + (warp - 2) * GP_OUT;
#pragma unroll
        for (int q = 0; q < 128 / cols; ++q) {
          const int c = (2 * q + part) * cols;
          if (n0 >= p.n || T.c0 + c >= p.k) break;
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the box before has left
          __syncwarp();
          uint8_t* row = out + lane * 128;
          if (F32) {
            const float(&v)[32] = sum[F32 ? q : 0];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(row + ((i ^ (lane & 7)) << 4)) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[32];
              if (PARTS) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = sum[PARTS ? 2 * q + h : 0][i];
              } else if (T.nkb > 0) {
                tmem_ld32(td + c + 32 * h, v);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(row + (((4 * h + i) ^ (lane & 7)) << 4)) =
                    make_uint4(pack_out(v[8 * i], v[8 * i + 1], p.out_dtype), pack_out(v[8 * i + 2], v[8 * i + 3], p.out_dtype),
                               pack_out(v[8 * i + 4], v[8 * i + 5], p.out_dtype), pack_out(v[8 * i + 6], v[8 * i + 7], p.out_dtype));
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tma_store_3d(smem_u32(out), &maps.d, T.c0 + c, n0, T.e);
        }
      } else
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = run_at(q);
        if (c >= T.n) break;
        float v[32];
        if (PARTS) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = sum[PARTS ? q : 0][i];
        } else if (WG && T.nkb == 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        } else {
          tmem_ld32(td + c, v);
        }
        const float col_scale = F8 ? xs[F8 ? q : 0] : 0.f;
        if (F8) {
          // one after the other, as the scales' own product may be past fp32 where the result is not (with swiglu the columns' follow
          // where a lane has its column's gate and up)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] *= ws;
            if (!SW) v[i] *= __shfl_sync(0xffffffffu, col_scale, i);
          }
        }
        if (WG) {
          // lane: row n of dw; columns: k
          const int n = T.f0 + (int)rank * 128 + quarter * 32 + lane, k = T.c0 + c;
          if (n < p.n) {
            const long long at = (long long)T.e * p.d_stride + (long long)n * p.ldd + k;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (k + i < p.k) store1(p.d, at + i, v[i], p.out_dtype);
          }
        } else {
          // lane: feature; columns: rows c .. c + 31 of the tile
          constexpr int el = F32 ? 4 : 2;
          const long long pitch = p.ldd * el;
          long long my_off = -1;   // out rows by number: lane i finds that of column c + i
          if (p.d_rows && c + lane < T.rows) {
            const long long r = __ldg(p.d_rows + T.r0 + c + lane);
            if (r >= 0 && r < p.d_nrows) my_off = r * pitch;
          }
          // feature f of columns i + sub, i = 0 .. 31 in steps: where it goes, or null
          const int sub = SW ? lane >> 4 : !F32 && a.wide ? lane & 1 : 0;
          const int f = SW ? T.f0 + (int)rank * 64 + quarter * 16 + (lane & 15) : T.f0 + (int)rank * 128 + quarter * 32 + lane;
          char* d = static_cast<char*>(p.d) + (long long)(!SW && !F32 && a.wide ? f & ~1 : f) * el;
          char* first_col = d + ((long long)T.r0 + c + sub) * pitch;
          const int cols = f < n_out ? T.rows - c - sub : 0;
          auto place = [&](int i, bool& live) -> char* {
            if (!p.d_rows) {
              live = i < cols;
              return first_col + i * pitch;
            }
            const long long off = __shfl_sync(0xffffffffu, my_off, i + sub);
            live = off >= 0 && f < n_out;
            return d + off;
          };
          if (SW) {
            // lanes 0..15 hold gate, 16..31 up of the same 16 features: columns i and i + 1 are
            // exchanged so that the lower lanes finish column i and the upper ones column i + 1
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float mine = lane < 16 ? v[i] : v[i + 1];
              const float other = __shfl_xor_sync(0xffffffffu, lane < 16 ? v[i + 1] : v[i], 16);
              float g = lane < 16 ? mine : other, u = lane < 16 ? other : mine;
              if (F8) {
                const float s = __shfl_sync(0xffffffffu, col_scale, i + sub);
                g *= s;
                u *= s;
              }
              const float h = (F8 ? silu_quick(g) : silu(g)) * u;
              bool live;
              char* at = place(i, live);
              if (F32) store32_if(live, at, __float_as_uint(h));
              else store16_if(live, at, pack_out(h, h, p.out_dtype));
            }
          } else if (!F32 && a.wide) {
            // lanes 2 j and 2 j + 1 exchange columns i and i + 1: the even lane stores column i of both
            // features in one word, the odd lane column i + 1 (n is even: both features or neither)
            const bool odd = lane & 1;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
              bool live;
              char* at = place(i, live);
              store32_if(live, at, odd ? pack_out(other, v[i + 1], p.out_dtype) : pack_out(v[i], other, p.out_dtype));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              bool live;
              char* at = place(i, live);
              if (F32) store32_if(live, at, __float_as_uint(v[i]));
              else store16_if(live, at, pack_out(v[i], v[i], p.out_dtype));
            }
          }
        }
      }
      if (!PARTS && T.nkb > 0) release();
    }
    if (WG && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) *s_abort = 1;
  }
  umma_fence_before();
  __syncthreads();
  if (*s_abort) {   // a wait ran out: report, and let what is in flight end before the memory goes
    if (tid == 0) report_wait(a.wait);
    drain_time();
  }
  cluster_sync_all();   // the peer reads and signals this block's memory until here
  umma_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

template <int MODE, int OUT>
cudaError_t launch_as(const PairArgs& a, const GroupedMaps& m, unsigned pairs, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(2 * pairs);
  c.blockDim = dim3(GP_THREADS);
  c.dynamicSmemBytes = GP_SMEM;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, grouped_pair_kernel<MODE, OUT>, a, m);
}

template <int MODE>
cudaError_t launch_mode(const PairArgs& a, const GroupedMaps& m, unsigned pairs, cudaStream_t s) {
  if (a.p.out_dtype == GT_FP32) return launch_as<MODE, GP_OUT_32>(a, m, pairs, s);
  // (of a weight gradient the longest that a group can be: shorter ones are summed in one go there too)
  const long long longest = MODE == GP_WGRAD ? a.p.m : a.p.k;
  return longest > GP_LONG * GP_STEP<MODE> ? launch_as<MODE, GP_OUT_16_LONG>(a, m, pairs, s) : launch_as<MODE, GP_OUT_16>(a, m, pairs, s);
}

template <int MODE, int OUT>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(grouped_pair_kernel<MODE, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, GP_SMEM);
}
template <int MODE>
cudaError_t set_attributes() {
  cudaError_t e = set_attribute<MODE, GP_OUT_16>();
  if (e == cudaSuccess) e = set_attribute<MODE, GP_OUT_16_LONG>();
  return e == cudaSuccess ? set_attribute<MODE, GP_OUT_32>() : e;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t grouped_pair_set_attributes() {
  cudaError_t e = set_attributes<GP_NK>();
  if (e == cudaSuccess) e = set_attributes<GP_KN>();
  if (e == cudaSuccess) e = set_attributes<GP_SWIGLU>();
  if (e == cudaSuccess) e = set_attributes<GP_WGRAD>();
  if (e == cudaSuccess) e = set_attributes<GP_NK8>();
  if (e == cudaSuccess) e = set_attributes<GP_SWIGLU8>();
  return e;
}

bool grouped_maps(const GroupedProblem& p, bool wgrad, bool few, GroupedMaps* m) {
  const size_t el = p.eight ? 1 : 2;
  const uint32_t wide = 128 / (uint32_t)el;   // elements of a box
  const uint64_t lda = p.lda * el, ldb = p.ldb * el;
  CUtensorMap *ma = m ? &m->a : nullptr, *mb = m ? m->b : nullptr;
  auto map_b = [&](int i) { return mb ? mb + i : nullptr; };
  if (p.a_nrows < 1 || p.a_nrows > 0x7fffffffLL) return false;
  if (wgrad) {
    if (p.b_nrows < 1 || p.b_nrows > 0x7fffffffLL) return false;
    const uint64_t da[] = {(uint64_t)p.n, (uint64_t)p.a_nrows}, db[] = {(uint64_t)p.k, (uint64_t)p.b_nrows};
    const uint32_t tile[] = {64, 64};
    return tensor_map(ma, p.a, 2, 2, da, &lda, tile) && tensor_map(map_b(0), p.b, 2, 2, db, &ldb, tile);
  }
  const uint64_t n = p.n, k = p.k, E = p.groups;
  // one expert: any step to the next; several on top of one another are not a tensor
  const uint64_t rows = p.kn ? k : n, step = p.groups > 1 ? p.b_stride * el : rows * ldb;
  if (step == 0) return false;
  bool ok;
  if (p.swiglu && n / 2 % 16 == 0) {   // a tile's alternating runs of 16 rows of gate and up in one box
    const uint64_t h = n / 2, d[] = {k, 16, 2, h / 16, E}, st[] = {ldb, h * ldb, 16 * ldb, step};
    const uint32_t box[] = {wide, 16, 2, 4, 1};
    ok = tensor_map(ma, p.b, el, 5, d, st, box);
  } else {
    const uint64_t d[] = {p.kn ? n : k, p.kn ? k : n, E}, st[] = {ldb, step};
    const uint32_t box[] = {wide, p.swiglu ? 16u : p.kn ? 64u : 128u, 1};
    ok = tensor_map(ma, p.b, el, 3, d, st, box);
  }
  const uint64_t dx[] = {k, (uint64_t)p.a_nrows};
  if (few && p.a_rows) {
    const uint32_t one[] = {wide, 1};
    return ok && tensor_map(map_b(0), p.a, el, 2, dx, &lda, one);
  }
  for (int i = 0; i < (few ? 1 : 4) && ok; ++i) {
    const uint32_t tile[] = {wide, 16u << i};
    ok = tensor_map(map_b(i), p.a, el, 2, dx, &lda, tile);
  }
  return ok;
}

bool launch_grouped_pair(const GroupedProblem& p, bool wgrad, int num_sms, const WaitLimit& wait, cudaStream_t s,
                         cudaError_t* err) {
  GroupedMaps m;
  if (p.a_rows || p.b_rows || !grouped_maps(p, wgrad, false, &m)) return false;
  PairArgs a;
  a.p = p;
  a.wait = wait;
  a.by_16 = p.swiglu && p.n / 2 % 16 != 0;
  const int n_out = p.swiglu ? p.n / 2 : p.n;
  const size_t el = p.out_dtype == GT_FP32 ? 4 : 2;
  long long tiles;
  if (wgrad) {
    a.nft = (int)ceil_div(p.n, 256);
    a.nkt = (int)ceil_div(p.k, 256);
    tiles = (long long)p.groups * a.nft * a.nkt;
    const uint64_t d[] = {(uint64_t)p.k, (uint64_t)p.n, (uint64_t)p.groups};
    const uint64_t st[] = {p.ldd * el, p.groups > 1 ? p.d_stride * el : p.n * p.ldd * el};
    const uint32_t box[] = {128u / (uint32_t)el, 32, 1};
    a.wide = tensor_map(&m.d, p.d, el, 3, d, st, box);
  } else {
    a.nft = (int)ceil_div(n_out, p.swiglu ? 128 : 256);
    a.nkt = 1;
    tiles = (p.m / 256 + (p.m < p.groups ? p.m : p.groups)) * a.nft;
    a.wide = (uintptr_t)p.d % 4 == 0 && p.ldd % 2 == 0 && n_out % 2 == 0;
  }
  if (tiles > 0x3fffffff) return false;
  a.max_tiles = (int)tiles;
  const unsigned pairs = (unsigned)(tiles < num_sms / 2 ? tiles : num_sms / 2);
  if (wgrad) *err = launch_mode<GP_WGRAD>(a, m, pairs, s);
  else if (p.eight) *err = p.swiglu ? launch_mode<GP_SWIGLU8>(a, m, pairs, s) : launch_mode<GP_NK8>(a, m, pairs, s);
  else if (p.swiglu) *err = launch_mode<GP_SWIGLU>(a, m, pairs, s);
  else *err = p.kn ? launch_mode<GP_KN>(a, m, pairs, s) : launch_mode<GP_NK>(a, m, pairs, s);
  return true;
}

}  // namespace moe
