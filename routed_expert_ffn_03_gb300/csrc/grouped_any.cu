// grouped_any.cu - grouped 16-bit products for any stride, alignment and size.
//
// D_e = A_e B_e^T for every group e (see GroupedProblem): a block takes one 64 x 64 tile of
// one group and walks the contracted dimension in steps of 32 with plain loads, so nothing
// is asked of strides or addresses.  Elements are read along whichever dimension is
// contiguous and stored in shared memory with the contracted dimension contiguous; rows
// and columns outside the group, and row numbers outside their array, are stored as zeros.
// Each of 4 warps multiplies a 32 x 32 quarter with mma m16n8k16 (fp32 sums).
#include "common.cuh"
#include "grouped.h"

namespace moe {

namespace {

constexpr int GA_T = 64;        // tile rows and columns
constexpr int GA_K = 32;        // contracted elements per step
constexpr int GA_LD = GA_K + 8; // shared row: 20 words, so a fragment's 8 rows x 4 words hit 32 banks
constexpr int GA_THREADS = 128;

enum : int { GA_NK = 0, GA_KN = 1, GA_SWIGLU = 2, GA_WGRAD = 3 };

template <bool BF>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ void store_out(void* d, long long at, float v, int t) {
  if (t == GT_FP32) static_cast<float*>(d)[at] = v;
  else if (t == GT_BF16) static_cast<__nv_bfloat16*>(d)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(d)[at] = __float2half_rn(v);
}

template <int MODE, bool BF>
__global__ void __launch_bounds__(GA_THREADS) grouped_any_kernel(GroupedProblem p) {
  constexpr bool WG = MODE == GA_WGRAD, SW = MODE == GA_SWIGLU;
  constexpr int NB = SW ? 2 : 1;
  __shared__ __align__(16) uint16_t as[GA_T * GA_LD];
  __shared__ __align__(16) uint16_t bs[NB][GA_T * GA_LD];
  __shared__ int s_tile[4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_out = SW ? p.n / 2 : p.n;

  // the tile: forward (group, row tile) x column tile; weight gradient group x row tile x column tile
  int r0, r1, e, a0, b0;
  if (WG) {
    const int ta = (p.n + GA_T - 1) / GA_T, tb = (p.k + GA_T - 1) / GA_T;
    const int per = ta * tb;
    e = blockIdx.x / per;
    a0 = (blockIdx.x % per) / tb * GA_T;
    b0 = (blockIdx.x % per) % tb * GA_T;
    group_range(p.offsets, e, p.m, r0, r1);
  } else {
    const int tb = (n_out + GA_T - 1) / GA_T;
    const int want = blockIdx.x / tb;
    b0 = blockIdx.x % tb * GA_T;
    if (warp == 0) {   // the want-th row tile over the groups
      int before = 0, found = -1, fr0 = 0, fr1 = 0;
      for (int g0 = 0; g0 < p.groups && found < 0; g0 += 32) {
        int gr0 = 0, gr1 = 0;
        if (g0 + lane < p.groups) group_range(p.offsets, g0 + lane, p.m, gr0, gr1);
        const int nt = (gr1 - gr0) / GA_T + ((gr1 - gr0) % GA_T != 0);
        int inc = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const bool mine = want >= before + inc - nt && want < before + inc;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
          const int l = __ffs(who) - 1;
          found = g0 + l;
          fr0 = __shfl_sync(0xffffffffu, gr0 + (want - before - inc + nt) * GA_T, l);
          fr1 = __shfl_sync(0xffffffffu, gr1, l);
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        s_tile[0] = found;
        s_tile[1] = fr0;
        s_tile[2] = fr1;
      }
    }
    __syncthreads();
    e = s_tile[0];
    if (e < 0) return;
    r0 = s_tile[1];
    r1 = min(s_tile[2], r0 + GA_T);
    a0 = 0;
  }

  const int kdim = WG ? r1 - r0 : p.k;   // contracted length
  const int am = WG ? p.n - a0 : r1 - r0;   // rows of A left from the tile's first
  const int bm = (WG ? p.k : n_out) - b0;   // rows of B left
  float acc[NB][2][4][4];
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[x][i][j][q] = 0.f;

  const long long wbase = WG ? 0 : (long long)e * p.b_stride;
  for (int k0 = 0; k0 < kdim; k0 += GA_K) {
    uint16_t va[GA_T * GA_K / GA_THREADS], vb[NB][GA_T * GA_K / GA_THREADS];
#pragma unroll
    for (int i = 0; i < GA_T * GA_K / GA_THREADS; ++i) {
      const int kc = tid & 31, rc = (tid >> 5) + 4 * i;   // contracted dimension contiguous
      const int mm = tid & 63, km = (tid >> 6) + 2 * i;   // the other one contiguous
      uint16_t v = 0;
      if (WG) {
        if (mm < am && k0 + km < kdim) {
          const long long row = p.a_rows ? __ldg(p.a_rows + r0 + k0 + km) : r0 + k0 + km;
          if (row >= 0 && row < p.a_nrows) v = __ldg(p.a + row * p.lda + a0 + mm);
        }
      } else if (rc < am && k0 + kc < kdim) {
        const long long row = p.a_rows ? __ldg(p.a_rows + r0 + rc) : r0 + rc;
        if (row >= 0 && row < p.a_nrows) v = __ldg(p.a + row * p.lda + k0 + kc);
      }
      va[i] = v;
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        v = 0;
        if (WG) {
          if (mm < bm && k0 + km < kdim) {
            const long long row = p.b_rows ? __ldg(p.b_rows + r0 + k0 + km) : r0 + k0 + km;
            if (row >= 0 && row < p.b_nrows) v = __ldg(p.b + row * p.ldb + b0 + mm);
          }
        } else if (MODE == GA_KN) {
          if (mm < bm && k0 + km < kdim) v = __ldg(p.b + wbase + (long long)(k0 + km) * p.ldb + b0 + mm);
        } else if (rc < bm && k0 + kc < kdim) {
          v = __ldg(p.b + wbase + (long long)(b0 + rc + x * n_out) * p.ldb + k0 + kc);
        }
        vb[x][i] = v;
      }
    }
    __syncthreads();   // the step before has been multiplied
#pragma unroll
    for (int i = 0; i < GA_T * GA_K / GA_THREADS; ++i) {
      const int kc = tid & 31, rc = (tid >> 5) + 4 * i;
      const int mm = tid & 63, km = (tid >> 6) + 2 * i;
      as[WG ? mm * GA_LD + km : rc * GA_LD + kc] = va[i];
#pragma unroll
      for (int x = 0; x < NB; ++x) bs[x][WG || MODE == GA_KN ? mm * GA_LD + km : rc * GA_LD + kc] = vb[x][i];
    }
    __syncthreads();
    const int g = lane >> 2, t = lane & 3, m0 = (warp >> 1) * 32, n0 = (warp & 1) * 32;
#pragma unroll
    for (int kk = 0; kk < GA_K; kk += 16) {
      uint32_t af[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          af[i][q] = *reinterpret_cast<const uint32_t*>(as + (m0 + i * 16 + g + (q & 1) * 8) * GA_LD + kk + 2 * t +
                                                        (q >> 1) * 8);
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint16_t* br = bs[x] + (n0 + j * 8 + g) * GA_LD + kk + 2 * t;
          const uint32_t bf0 = *reinterpret_cast<const uint32_t*>(br);
          const uint32_t bf1 = *reinterpret_cast<const uint32_t*>(br + 8);
#pragma unroll
          for (int i = 0; i < 2; ++i) mma16<BF>(acc[x][i][j], af[i], bf0, bf1);
        }
    }
  }

  const int g = lane >> 2, t = lane & 3, m0 = (warp >> 1) * 32, n0 = (warp & 1) * 32;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m0 + i * 16 + g + h * 8;
      if (r >= am) continue;
      long long at;
      if (WG) {
        at = (long long)e * p.d_stride + (long long)(a0 + r) * p.ldd;
      } else {
        const long long row = p.d_rows ? __ldg(p.d_rows + r0 + r) : r0 + r;
        if (row < 0 || row >= p.d_nrows) continue;
        at = row * p.ldd;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c = n0 + j * 8 + 2 * t + q;
          if (c >= bm) continue;
          float v = acc[0][i][j][2 * h + q];
          if (SW) v = v / (1.f + expf(-v)) * acc[NB - 1][i][j][2 * h + q];
          store_out(p.d, at + b0 + c, v, p.out_dtype);
        }
    }
}

template <int MODE>
cudaError_t launch_mode(const GroupedProblem& p, unsigned blocks, cudaStream_t s) {
  if (p.dtype == GT_BF16) grouped_any_kernel<MODE, true><<<blocks, GA_THREADS, 0, s>>>(p);
  else grouped_any_kernel<MODE, false><<<blocks, GA_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

long long tiles(long long v) { return (v + GA_T - 1) / GA_T; }

}  // namespace

cudaError_t launch_grouped_any(const GroupedProblem& p, bool wgrad, cudaStream_t s) {
  // forward: every group can end inside a tile, so there are at most m / 64 + min(groups, m) row tiles
  const long long blocks = wgrad ? (long long)p.groups * tiles(p.n) * tiles(p.k)
                                 : (p.m / GA_T + (p.m < p.groups ? p.m : p.groups)) * tiles(p.swiglu ? p.n / 2 : p.n);
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (wgrad) return launch_mode<GA_WGRAD>(p, (unsigned)blocks, s);
  if (p.swiglu) return launch_mode<GA_SWIGLU>(p, (unsigned)blocks, s);
  return p.kn ? launch_mode<GA_KN>(p, (unsigned)blocks, s) : launch_mode<GA_NK>(p, (unsigned)blocks, s);
}

}  // namespace moe
