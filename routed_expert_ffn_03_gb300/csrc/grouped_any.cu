// grouped_any.cu - grouped 16-bit products for any stride, alignment and size.
//
// What the TMA kernels refuse (rows whose pitch or start is not a multiple of 16 bytes, odd widths, several experts
// on one matrix) is staged here by warps with plain loads, into the same swizzled shared-memory tiles,
// so the products still run on the tensor core.  A block takes one tile of 128 x 64 of a group and steps of 64
// contracted elements.  An operand word of 16 bytes that does not start on a 16-byte boundary is put together from the
// two aligned words around it (one of the two comes from L1: the neighbour lane's), unless those reach past the
// tensor's first or last byte: then it is read by elements.  Words behind the contracted length, rows of no group and row
// numbers outside their tensor are stored as zeros.  Warps:
//   warps 0..15  load (two steps ahead in registers) and store into a ring of 4 stages;
//   warp 16      issues the products, in parts of 256 elements in alternating results;
//   warps 16..19 add the parts up in fp32 registers.
// Then all warps store the tile by elements.
// Bound: the loads' latency and the staging's instructions: 141 TFLOP/s at 4096 rows, n = k = 4095, 8 groups (23
// with 64 x 64 tiles of the warp-level mma and element loads; 115 with 8 loading warps one step ahead).
#include "grouped.h"
#include "grouped_mma.cuh"

namespace moe {

namespace {

enum : int { GA_NK = 0, GA_KN = 1, GA_SWIGLU = 2, GA_WGRAD = 3 };
constexpr int GA_M = 128, GA_N = 64;             // tile: rows of the first factor and of the second
constexpr int GA_A = GA_M * 128, GA_B = GA_N * 128, GA_STAGE = GA_A + GA_B;   // bytes of a stage: 64 elements a row
constexpr int GA_STAGES = 4;
constexpr int GA_COPY_WARPS = 16, GA_EPI_WARPS = 4;
constexpr int GA_THREADS = (GA_COPY_WARPS + GA_EPI_WARPS) * 32;   // 20 warps have 96 registers a thread, 21 only 80
// 16-byte words of the factors that a thread stages
constexpr int GA_AW = GA_M * 8 / (GA_COPY_WARPS * 32), GA_BW = GA_N * 8 / (GA_COPY_WARPS * 32);
constexpr int GA_PART = 4;                      // stages of a part
constexpr int GA_SMEM = GA_STAGES * GA_STAGE + 256 + 1024;

struct AnyArgs {
  GroupedProblem p;
  WaitLimit wait;
};

// 8 elements at s (null: zeros), zeros from `left` on, as the two aligned words around them, or finished in the first
struct Word8 {
  uint4 a, b;
  int shift;   // bytes from a's first to the first wanted
};
__device__ __forceinline__ uint4 by_elements(const uint16_t* s, int n) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)__ldg(s + i) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_if(bool live, uintptr_t at) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " @p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(at), "r"((uint32_t)live));
  return v;
}
// N words of one factor.  lo, hi: the tensor's first byte and the one behind its last.  Where both aligned words of each of
// the warp's are inside the tensor, the loads stand side by side without a branch; else the words are read by elements.  PART:
// finish8 clears what is not wanted of a word, so such words load in the same way (a warp of an MN-major tile at the
// edge has one in every step; K-major ones meet them in the last step alone, and clearing costs the others 3%).
template <bool PART, int N>
__device__ __forceinline__ void load_words(const uint16_t* const (&s)[N], int left, uintptr_t lo, uintptr_t hi, Word8 (&w)[N]) {
  bool whole = true;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uintptr_t at = (uintptr_t)s[i] & ~(uintptr_t)15;
    whole = whole && (!s[i] || (PART && left <= 0) || ((PART || left >= 8) && at >= lo && at + 32 <= hi));
  }
  if (__all_sync(0xffffffffu, whole)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uintptr_t at = (uintptr_t)s[i] & ~(uintptr_t)15;
      w[i].shift = (int)((uintptr_t)s[i] & 15);
      w[i].a = load_if(s[i] != nullptr && (!PART || left > 0), at);
      w[i].b = load_if(s[i] != nullptr && (!PART || left > 0), at + 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i].shift = 0;
      w[i].a = w[i].b = make_uint4(0, 0, 0, 0);
      if (s[i] && left > 0) w[i].a = by_elements(s[i], min(left, 8));
    }
  }
}
template <bool PART>
__device__ __forceinline__ uint4 finish8(const Word8& w, int left) {
  const uint32_t v[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
  const int by = 8 * (w.shift & 3);
  const bool two = w.shift & 8, one = w.shift & 4;   // by halves: 8 bytes, then 4
  uint32_t x[6], y[5], r[4];
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = two ? v[i + 2] : v[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) y[i] = one ? x[i + 1] : x[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(y[i], y[i + 1], by);
  if (PART && left < 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = left >= 2 * i + 2 ? r[i] : left > 2 * i ? r[i] & 0xffffu : 0u;
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void store_out(void* d, long long at, float v, int t) {
  if (t == GT_FP32) static_cast<float*>(d)[at] = v;
  else if (t == GT_BF16) static_cast<__nv_bfloat16*>(d)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(d)[at] = __float2half_rn(v);
}

template <int MODE>
__global__ void __launch_bounds__(GA_THREADS, 1) grouped_any_kernel(const __grid_constant__ AnyArgs args) {
  constexpr bool WG = MODE == GA_WGRAD, SW = MODE == GA_SWIGLU;
  // factor A: W_e's features, or dw's k (weight gradient), so that a lane's neighbour is its neighbour in the result; factor
  // B: the group's rows, or dw's n.  MN-major: the contracted dimension is not the contiguous one.
  constexpr bool a_mn = WG || MODE == GA_KN, b_mn = WG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const GroupedProblem& p = args.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_out = SW ? p.n / 2 : p.n;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + GA_STAGES * GA_STAGE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * GA_STAGES + 4);
  int* s_tile = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* s_abort = s_tile + 3;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * GA_STAGES, tfull0 = empty0 + 8 * GA_STAGES, tempty0 = tfull0 + 16;
  if (tid == 0) {
    for (int s = 0; s < GA_STAGES; ++s) {
      mbar_init(full0 + 8 * s, stage_arrivals(args.wait, GA_COPY_WARPS));
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, GA_EPI_WARPS);
    }
    *s_abort = 0;
    mbar_fence_init();
  }
  if (warp == GA_COPY_WARPS) tmem_alloc<1>(smem_u32(tmem_slot), 2 * GA_N);

  // the tile: forward (group, row tile) x feature tile; weight gradient group x k tile x n tile
  int e, r0, r1, a0, b0 = 0;
  if (WG) {
    const int tb = (p.n + GA_N - 1) / GA_N, per = (p.k + GA_M - 1) / GA_M * tb;
    e = blockIdx.x / per;
    a0 = blockIdx.x % per / tb * GA_M;
    b0 = blockIdx.x % per % tb * GA_N;
    group_range(p.offsets, e, p.m, r0, r1);
  } else {
    constexpr int F = SW ? GA_M / 2 : GA_M;
    const int ta = (n_out + F - 1) / F;
    a0 = blockIdx.x % ta * F;
    if (warp == 0) {
      find_tile(p, GA_N, blockIdx.x / ta, lane, e, r0, r1);
      if (lane == 0) {
        s_tile[0] = e;
        s_tile[1] = r0;
        s_tile[2] = r1;
      }
    }
  }
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!WG) {
    e = s_tile[0];
    r0 = s_tile[1];
    r1 = s_tile[2];
  }
  const int rows = r1 - r0;
  const int kdim = e < 0 ? 0 : WG ? rows : p.k, nkb = (kdim + 63) / 64;
  const int cols = WG ? GA_N : (rows + 15) & ~15;   // columns of the product

  if (warp < GA_COPY_WARPS) {
    // ---------------------------------------------------------------- staging
    // K-major: thread: word c of rows r + step i.  MN-major: word c (in slabs of 8) of contracted rows r + step i.
    const uintptr_t a_lo = (uintptr_t)p.b, b_lo = (uintptr_t)p.a;
    const uintptr_t a_hi = a_lo + 2 * (WG ? (p.b_nrows - 1) * p.ldb + p.k
                                          : (p.groups - 1) * p.b_stride + ((p.kn ? p.k : p.n) - 1) * p.ldb + (p.kn ? p.n : p.k));
    const uintptr_t b_hi = b_lo + 2 * ((p.a_nrows - 1) * p.lda + (WG ? p.n : p.k));
    const int ca = a_mn ? tid & 15 : tid & 7, ra = a_mn ? tid >> 4 : tid >> 3;
    const int cb = tid & 7, rb = tid >> 3;
    constexpr int step_a = GA_COPY_WARPS * 32 / (a_mn ? 16 : 8), step_b = GA_COPY_WARPS * 32 / 8;
    const uint16_t* a_row[GA_AW];   // K-major: the rows' starts, null for a row of zeros
    const uint16_t* b_row[GA_BW];
    const uint16_t* w = p.b + (WG ? 0 : (long long)e * p.b_stride);
    auto row_at = [&](const uint16_t* base, const int* list, long long i, long long n, long long ld) -> const uint16_t* {
      const long long row = list ? __ldg(list + i) : i;
      return row >= 0 && row < n ? base + row * ld : nullptr;
    };
#pragma unroll
    for (int i = 0; i < GA_AW; ++i) {
      const int r = ra + step_a * i, f = SW ? a0 + (r >> 5) * 16 + (r & 15) : a0 + r;   // swiglu: 16 rows of gate, then 16 of up
      a_row[i] = !a_mn && f < n_out ? w + (long long)(SW && (r & 16) ? f + n_out : f) * p.ldb : nullptr;
    }
#pragma unroll
    for (int i = 0; i < GA_BW; ++i) {
      const int r = rb + step_b * i;
      b_row[i] = !b_mn && r < rows ? row_at(p.a, p.a_rows, r0 + r, p.a_nrows, p.lda) : nullptr;
    }
    auto left_a = [&](int kb) { return a_mn ? (WG ? p.k : n_out) - a0 - ca * 8 : kdim - kb * 64 - ca * 8; };
    auto left_b = [&](int kb) { return b_mn ? p.n - b0 - cb * 8 : kdim - kb * 64 - cb * 8; };
    auto load = [&](int kb, Word8 (&va)[GA_AW], Word8 (&vb)[GA_BW]) {
      const uint16_t* s[GA_AW];
#pragma unroll
      for (int i = 0; i < GA_AW; ++i) {
        if (a_mn) {
          const int k = kb * 64 + ra + step_a * i;
          const uint16_t* row = nullptr;
          if (k < kdim) row = WG ? row_at(p.b, p.b_rows, r0 + k, p.b_nrows, p.ldb) : w + (long long)k * p.ldb;
          s[i] = row ? row + a0 + ca * 8 : nullptr;
        } else {
          s[i] = a_row[i] ? a_row[i] + kb * 64 + ca * 8 : nullptr;
        }
      }
      load_words<a_mn>(s, left_a(kb), a_lo, a_hi, va);
      const uint16_t* t[GA_BW];
#pragma unroll
      for (int i = 0; i < GA_BW; ++i) {
        if (b_mn) {
          const int k = kb * 64 + rb + step_b * i;
          const uint16_t* row = k < kdim ? row_at(p.a, p.a_rows, r0 + k, p.a_nrows, p.lda) : nullptr;
          t[i] = row ? row + b0 + cb * 8 : nullptr;
        } else {
          t[i] = b_row[i] ? b_row[i] + kb * 64 + cb * 8 : nullptr;
        }
      }
      load_words<b_mn>(t, left_b(kb), b_lo, b_hi, vb);
    };
    const uint32_t at_a = (a_mn ? (ca >> 3) * SLAB_BYTES : 0) + ra * 128 + (((ca & 7) ^ (ra & 7)) << 4);
    const uint32_t at_b = rb * 128 + ((cb ^ (rb & 7)) << 4);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    // step kb's words, and then those of step kb + 2 in the same registers
    auto step = [&](int kb, Word8 (&va)[GA_AW], Word8 (&vb)[GA_BW]) {
      ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ph ^ 1, args.wait));
      if (!ok) return;
      uint8_t* st = smem + s * GA_STAGE;
#pragma unroll
      for (int i = 0; i < GA_AW; ++i) *reinterpret_cast<uint4*>(st + at_a + i * step_a * 128) = finish8<a_mn>(va[i], left_a(kb));
#pragma unroll
      for (int i = 0; i < GA_BW; ++i) *reinterpret_cast<uint4*>(st + GA_A + at_b + i * step_b * 128) = finish8<b_mn>(vb[i], left_b(kb));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(full0 + 8 * s);
      if (kb + 2 < nkb) load(kb + 2, va, vb);
      if (++s == GA_STAGES) {
        s = 0;
        ph ^= 1;
      }
    };
    Word8 va0[GA_AW], vb0[GA_BW], va1[GA_AW], vb1[GA_BW];
    if (nkb > 0) load(0, va0, vb0);
    if (nkb > 1) load(1, va1, vb1);
    for (int kb = 0; kb < nkb && ok; kb += 2) {
      step(kb, va0, vb0);
      if (ok && kb + 1 < nkb) step(kb + 1, va1, vb1);
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else {
    // ---------------------------------------------------------------- products and results
    const int quarter = warp & 3;   // of the TMEM lanes
    const uint32_t td = tmem + ((uint32_t)(quarter * 32) << 16);
    float sum[GA_N];
#pragma unroll
    for (int i = 0; i < GA_N; ++i) sum[i] = 0.f;
    int racc = 0;
    uint32_t raph = 0;
    bool ok = true;
    auto add_part = [&]() {
      ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * racc, raph, args.wait));
      if (!ok) return;
      umma_fence_after();
#pragma unroll
      for (int c = 0; c < GA_N; c += 16) {
        if (c < cols) {
          float v[16];
          tmem_ld16(td + racc * GA_N + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] += v[i];
        }
      }
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * racc);
      if (++racc == 2) {
        racc = 0;
        raph ^= 1;
      }
    };
    if (warp == GA_COPY_WARPS) {   // issues a part's products, then adds up the part before
      const bool leader = elect_one();
      constexpr uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
      const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t da0 = sw128_desc(base, a_mn), db0 = sw128_desc(base + GA_A, b_mn);
      const uint32_t idesc = idesc_16(p.dtype == GT_BF16, a_mn, b_mn, GA_M, __shfl_sync(0xffffffffu, cols, 0));
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      for (int k0 = 0; k0 < nkb && ok; k0 += GA_PART) {
        const int k1 = min(k0 + GA_PART, nkb);
        ok = __all_sync(0xffffffffu, wait_bar(tempty0 + 8 * acc, aph ^ 1, args.wait));
        umma_fence_after();
        for (int kb = k0; kb < k1 && ok; ++kb) {
          ok = __all_sync(0xffffffffu, wait_bar(full0 + 8 * s, ph, args.wait));
          if (!ok) break;
          umma_fence_after();
          const uint32_t off = s * (GA_STAGE >> 4);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma<1>(tm + acc * GA_N, da0 + off + kk * a_step, db0 + off + kk * b_step, idesc, kb > k0 || kk > 0);
            umma_commit(empty0 + 8 * s);
          }
          __syncwarp();
          if (++s == GA_STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (leader) umma_commit(tfull0 + 8 * acc);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          aph ^= 1;
        }
        if (k0 > 0) add_part();
      }
      if (ok && nkb > 0) add_part();
    } else {
      for (int k0 = 0; k0 < nkb && ok; k0 += GA_PART) add_part();
    }
    if (!ok && lane == 0) *s_abort = 1;
    // the sums, [column][feature], over the stages: all products have ended
    float* part = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
#pragma unroll
    for (int i = 0; i < GA_N; ++i)
      if (i < cols) part[i * GA_M] = sum[i];
  }
  umma_fence_before();
  __syncthreads();
  if (*s_abort) {   // a wait ran out: report, and let what is in flight end before the memory goes
    if (tid == 0) report_wait(args.wait);
    drain_time();
  } else if (e >= 0) {
    // stored by all warps in a short loop, neighbours along a row: unrolled over the columns in registers the code
    // runs once a tile and is fetched that often (124 rows in 19 groups, 1699 columns with swiglu, k = 103: 46 and 23 us)
    const float* part = reinterpret_cast<const float*>(smem);
    constexpr int F = SW ? GA_M / 2 : GA_M;
    const int columns = WG ? min(GA_N, p.n - b0) : rows, left = (WG ? p.k : n_out) - a0;
    for (int i = tid; i < columns * F; i += GA_THREADS) {
      const int c = i / F, f = i % F;
      if (f >= left) continue;
      if (WG) {
        store_out(p.d, (long long)e * p.d_stride + (long long)(b0 + c) * p.ldd + a0 + f, part[c * GA_M + f], p.out_dtype);
      } else {
        const long long row = p.d_rows ? __ldg(p.d_rows + r0 + c) : r0 + c;
        float v = part[c * GA_M + (SW ? (f >> 4) * 32 + (f & 15) : f)];
        if (SW) v = silu(v) * part[c * GA_M + (f >> 4) * 32 + (f & 15) + 16];
        if (row >= 0 && row < p.d_nrows) store_out(p.d, row * p.ldd + a0 + f, v, p.out_dtype);
      }
    }
  }
  umma_fence_after();
  if (warp == GA_COPY_WARPS) tmem_dealloc<1>(tmem, 2 * GA_N);
}

template <int MODE>
cudaError_t launch_mode(const AnyArgs& a, unsigned blocks, cudaStream_t s) {
  grouped_any_kernel<MODE><<<blocks, GA_THREADS, GA_SMEM, s>>>(a);
  return cudaGetLastError();
}
template <int MODE>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(grouped_any_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, GA_SMEM);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t grouped_any_set_attributes() {
  cudaError_t e = set_attribute<GA_NK>();
  if (e == cudaSuccess) e = set_attribute<GA_KN>();
  if (e == cudaSuccess) e = set_attribute<GA_SWIGLU>();
  if (e == cudaSuccess) e = set_attribute<GA_WGRAD>();
  return e;
}

cudaError_t launch_grouped_any(const GroupedProblem& p, bool wgrad, const WaitLimit& wait, cudaStream_t s) {
  // forward: every group can end inside a tile, so m rows make at most m / 64 + min(groups, m) row tiles
  const long long blocks =
      wgrad ? (long long)p.groups * ceil_div(p.k, GA_M) * ceil_div(p.n, GA_N)
            : (p.m / GA_N + (p.m < p.groups ? p.m : p.groups)) * ceil_div(p.swiglu ? p.n / 2 : p.n, p.swiglu ? GA_M / 2 : GA_M);
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const AnyArgs a{p, wait};
  if (wgrad) return launch_mode<GA_WGRAD>(a, (unsigned)blocks, s);
  if (p.swiglu) return launch_mode<GA_SWIGLU>(a, (unsigned)blocks, s);
  return p.kn ? launch_mode<GA_KN>(a, (unsigned)blocks, s) : launch_mode<GA_NK>(a, (unsigned)blocks, s);
}

}  // namespace moe
