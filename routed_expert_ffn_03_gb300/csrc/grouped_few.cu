// grouped_few.cu - grouped 16-bit products of few rows: the weights' bytes are the time.
//
//   D^T[f][t] = sum_k W_e[f][k] x[t][k],   128 features a block, up to NT of a group's rows
//
// With a few rows a group every weight is read once and multiplied a handful of times (bound: memory), so what counts
// is that all SMs read evenly and keep enough in flight.  A tile is 128 features of one block's tensor core
// (M = 128, the rows as N: 16 columns cost next to nothing), and a cluster of C blocks shares the contracted dimension
// of a tile, so that few tiles still make several blocks an SM.  Two blocks share an SM: one computes
// its start (finding its group takes two memory round trips) while the other streams.  Warps:
//   warp 0      copies W_e tiles by TMA into a ring;
//   warp 6      the rows (named by number: gather, 4 rows an instruction, cheap at 16 rows and not for many);
//   warp 1      issues the products, in parts of 256 elements in alternating results;
//   warps 2..5  add the parts up in fp32 registers (the tensor core's own running sum truncates at each step).
// Then the cluster adds its blocks' sums in rank order through distributed shared memory (no workspace, no
// atomics, the same bits every time) and each block stores its share.
// DeepSeek-V3-shaped layer: gate/up of one token (470 MB) 74 us, 0.93 of the memory's rate; down of four tokens (0.9 GB)
// 129 us (the pair kernel: 79 and 138).
#include "grouped.h"
#include "grouped_mma.cuh"

namespace moe {

namespace {

enum : int { GF_NK = 0, GF_KN = 1, GF_SWIGLU = 2 };
constexpr int GF_ROW_WARP = 6;
constexpr int GF_THREADS = (GF_ROW_WARP + 1) * 32;
constexpr int GF_A = 128 * 128;       // bytes of a W_e tile: 128 features x 64 elements
constexpr int GF_PART = 4;            // stages of a part (8 are no faster)

constexpr int gf_stages(int nt) { return nt == 16 ? 6 : nt == 32 ? 5 : 4; }   // two blocks an SM
constexpr int gf_stage_bytes(int nt) { return GF_A + nt * 128; }
constexpr int gf_smem(int nt) { return gf_stages(nt) * gf_stage_bytes(nt) + 256 + 1024; }

struct FewArgs {
  GroupedProblem p;
  int nft;              // feature tiles
  int cluster;
  WaitLimit wait;
  bool wide;            // 16-bit results can be stored in pairs
  bool by_16;           // swiglu: W_e in boxes of 16 rows
};

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int MODE, int NT>
__global__ void __launch_bounds__(GF_THREADS, 2)
    grouped_few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ GroupedMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  constexpr int STAGES = NT == 16 ? 6 : NT == 32 ? 5 : 4, STAGE = GF_A + NT * 128;
  constexpr int COLS = NT == 16 ? 32 : 2 * NT;      // two results
  constexpr bool SW = MODE == GF_SWIGLU;
  const GroupedProblem& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.cluster, rank = C > 1 ? (int)cluster_rank() : 0;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + STAGES * STAGE + 160);
  int* s_tile = reinterpret_cast<int*>(smem + STAGES * STAGE + 176);
  volatile int* s_abort = s_tile + 4;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, tfull0 = empty0 + 8 * STAGES, tempty0 = tfull0 + 16;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, stage_arrivals(a.wait, 1));
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 4);
    }
    *s_abort = 0;
    mbar_fence_init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b[0]);
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), COLS);
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x / C;
  if (warp == 0) {
    int e, r0, r1;
    find_tile(p, NT, tile / a.nft, lane, e, r0, r1);
    if (lane == 0) {
      s_tile[0] = e;
      s_tile[1] = r0;
      s_tile[2] = r1;
    }
  }
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int e = s_tile[0], r0 = s_tile[1], rows = s_tile[2] - r0;
  const bool work = e >= 0;                       // the same in every block of the cluster
  const int f0 = tile % a.nft * (SW ? 64 : 128);  // first feature (with swiglu: of gate and of up)
  const int n = (rows + 15) & ~15;                // columns of the product
  const int nkb = (p.k + 63) / 64, kb0 = (int)((long long)nkb * rank / C), kb1 = (int)((long long)nkb * (rank + 1) / C);
  const int n_out = SW ? p.n / 2 : p.n;

  float sum[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) sum[i] = 0.f;
  if (work && warp == 0) {
    // the warp walks the loop together and one elected thread issues: the operands sit in uniform registers
    const bool leader = elect_one();
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), bar0 = __shfl_sync(0xffffffffu, full0, 0);
    const int ue = __shfl_sync(0xffffffffu, e, 0), uf = __shfl_sync(0xffffffffu, f0, 0), un = __shfl_sync(0xffffffffu, n, 0);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ph ^ 1, a.wait));
      if (!ok) break;
      const uint32_t bar = bar0 + 8 * s, da = base + s * STAGE;
      if (leader) {
        mbar_arrive_expect_tx(bar, GF_A + un * 128);
        if (MODE == GF_NK) tma_3d<1>(da, &maps.a, kb * 64, uf, ue, bar);
        if (SW && !a.by_16) tma_5d<1>(da, &maps.a, kb * 64, 0, 0, uf / 16, ue, bar);
        if (SW && a.by_16)   // gate and up in turn, 16 rows each
          for (int i = 0; i < 8; ++i) tma_3d<1>(da + i * 2048, &maps.a, kb * 64, uf + (i >> 1) * 16 + (i & 1) * (p.n / 2), ue, bar);
        if (MODE == GF_KN) {
          tma_3d<1>(da, &maps.a, uf, kb * 64, ue, bar);
          tma_3d<1>(da + SLAB_BYTES, &maps.a, uf + 64, kb * 64, ue, bar);
        }
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (work && warp == GF_ROW_WARP) {
    int4 gr = make_int4(0, 0, 0, 0);
    if (p.a_rows && lane < n / 4) {   // lane i gathers rows 4 i .. 4 i + 3; a number outside x gives zeros
      int r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 4 * lane + q, none = (int)p.a_nrows;
        const int v = i < rows ? __ldg(p.a_rows + r0 + i) : none;
        r[q] = v >= 0 && v < none ? v : none;
      }
      gr = make_int4(r[0], r[1], r[2], r[3]);
    }
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ph ^ 1, a.wait));
      if (!ok) break;
      const uint32_t bar = full0 + 8 * s, db = smem_u32(smem) + s * STAGE + GF_A;
      if (p.a_rows) {
        if (lane < n / 4) tma_gather4(db + lane * 512, &maps.b[0], kb * 64, gr, bar);
      } else if (lane < n / 16) {
        tma_2d<1>(db + lane * 2048, &maps.b[0], kb * 64, r0 + lane * 16, bar);
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (work && warp == 1) {
    const bool leader = elect_one();
    constexpr bool a_mn = MODE == GF_KN;
    constexpr uint32_t a_step = (a_mn ? 2048 : 32) >> 4;
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t da0 = sw128_desc(base, a_mn), db0 = sw128_desc(base + GF_A, false);
    const uint32_t idesc = idesc_16(p.dtype == GT_BF16, a_mn, false, 128, __shfl_sync(0xffffffffu, n, 0));
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (int k0 = kb0; k0 < kb1 && ok; k0 += GF_PART) {
      const int k1 = min(k0 + GF_PART, kb1);
      ok = __all_sync(0xffffffffu, wait_bar(tempty0 + 8 * acc, aph ^ 1, a.wait));
      umma_fence_after();
      for (int kb = k0; kb < k1 && ok; ++kb) {
        ok = __all_sync(0xffffffffu, wait_bar(full0 + 8 * s, ph, a.wait));
        if (!ok) break;
        umma_fence_after();
        const uint64_t da = da0 + (uint32_t)(s * (STAGE >> 4)), db = db0 + (uint32_t)(s * (STAGE >> 4));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma<1>(tm + acc * NT, da + kk * a_step, db + kk * 2, idesc, kb > k0 || kk > 0);
          umma_commit(empty0 + 8 * s);
        }
        __syncwarp();
        if (++s == STAGES) {
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
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (work) {
    const uint32_t td = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int k0 = kb0; k0 < kb1; k0 += GF_PART) {
      ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * acc, aph, a.wait));
      if (!ok) break;
      umma_fence_after();
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        if (c < n) {
          float v[16];
          tmem_ld16(td + acc * NT + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] += v[i];
        }
      }
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
    // this block's sums, [column][feature], over the stages (all copies and products into them have ended)
    if (ok) {
      float* part = reinterpret_cast<float*>(smem);
      const int f = (warp & 3) * 32 + lane;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i < rows) part[i * 128 + f] = sum[i];
    }
  }
  umma_fence_before();
  __syncthreads();
  if (*s_abort) {   // a wait ran out: report, and let what is in flight end before the memory goes
    if (tid == 0) report_wait(a.wait);
    drain_time();
  }
  if (C > 1) cluster_sync_all();
  if (work && !*s_abort) {
    constexpr int per_row = SW ? 32 : 64;     // feature pairs of a row
    const int items = rows * per_row;
    for (int i = rank * GF_THREADS + tid; i < items; i += C * GF_THREADS) {
      const int t = i / per_row, j = i - t * per_row;
      // features 2 j, 2 j + 1; with swiglu gate and up lie in alternating runs of 16
      const int f = SW ? (2 * j >> 4) * 32 + (2 * j & 15) : 2 * j;
      const uint32_t at = smem_u32(smem) + (t * 128 + f) * 4;
      float2 v = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
      for (int r = 0; r < C; ++r) {
        const uint32_t q = C > 1 ? map_rank(at, r) : at;
        const float2 w = ld_cluster2(q);
        v.x += w.x;
        v.y += w.y;
        if (SW) {
          const float2 x = ld_cluster2(q + 64);
          u.x += x.x;
          u.y += x.y;
        }
      }
      if (SW) {
        v.x = silu(v.x) * u.x;
        v.y = silu(v.y) * u.y;
      }
      const long long row = p.d_rows ? __ldg(p.d_rows + r0 + t) : r0 + t;
      const int fo = f0 + 2 * j;
      if (row < 0 || row >= p.d_nrows || fo >= n_out) continue;
      const long long out = row * p.ldd + fo;
      if (p.out_dtype == GT_FP32) {
        float* d = static_cast<float*>(p.d) + out;
        d[0] = v.x;
        if (fo + 1 < n_out) d[1] = v.y;
      } else {
        const uint32_t w = pack_out(v.x, v.y, p.out_dtype);
        uint16_t* d = static_cast<uint16_t*>(p.d) + out;
        if (a.wide) {
          *reinterpret_cast<uint32_t*>(d) = w;
        } else {
          d[0] = (uint16_t)w;
          if (fo + 1 < n_out) d[1] = (uint16_t)(w >> 16);
        }
      }
    }
  }
  if (C > 1) cluster_sync_all();   // the others read this block's sums until here
  else __syncthreads();
  umma_fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, COLS);
}

template <int MODE, int NT>
cudaError_t launch_as(const FewArgs& a, const GroupedMaps& m, unsigned tiles, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(tiles * a.cluster);
  c.blockDim = dim3(GF_THREADS);
  c.dynamicSmemBytes = gf_smem(NT);
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, grouped_few_kernel<MODE, NT>, a, m);
}

template <int MODE>
cudaError_t launch_mode(const FewArgs& a, const GroupedMaps& m, int nt, unsigned tiles, cudaStream_t s) {
  if (nt == 16) return launch_as<MODE, 16>(a, m, tiles, s);
  return nt == 32 ? launch_as<MODE, 32>(a, m, tiles, s) : launch_as<MODE, 64>(a, m, tiles, s);
}

template <int MODE, int NT>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(grouped_few_kernel<MODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, gf_smem(NT));
}
template <int MODE>
cudaError_t set_attributes() {
  cudaError_t e = set_attribute<MODE, 16>();
  if (e == cudaSuccess) e = set_attribute<MODE, 32>();
  return e == cudaSuccess ? set_attribute<MODE, 64>() : e;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t grouped_few_set_attributes() {
  cudaError_t e = set_attributes<GF_NK>();
  if (e == cudaSuccess) e = set_attributes<GF_KN>();
  return e == cudaSuccess ? set_attributes<GF_SWIGLU>() : e;
}

bool launch_grouped_few(const GroupedProblem& p, int nt, int cluster, const WaitLimit& wait, cudaStream_t s, cudaError_t* err) {
  GroupedMaps m;
  if (!grouped_maps(p, false, true, &m)) return false;
  FewArgs a;
  a.p = p;
  a.wait = wait;
  const int n_out = p.swiglu ? p.n / 2 : p.n;
  a.nft = (int)ceil_div(n_out, p.swiglu ? 64 : 128);
  a.cluster = cluster;
  a.by_16 = p.swiglu && p.n / 2 % 16 != 0;
  a.wide = (uintptr_t)p.d % 4 == 0 && p.ldd % 2 == 0 && n_out % 2 == 0;
  const long long tiles = (p.m / nt + (p.m < p.groups ? p.m : p.groups)) * a.nft;   // the most that m rows can make
  if (tiles * cluster > 0x3fffffff) return false;
  *err = p.swiglu ? launch_mode<GF_SWIGLU>(a, m, nt, (unsigned)tiles, s)
         : p.kn   ? launch_mode<GF_KN>(a, m, nt, (unsigned)tiles, s)
                  : launch_mode<GF_NK>(a, m, nt, (unsigned)tiles, s);
  return true;
}

}  // namespace moe
