// rms_norm.cu - root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its gradient.
//
//   h = round(x + residual)  (to the residual's type; x without one),  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd g
//   8 bits: scale = max(max|y| / 448, 2^-100) (by the fp32 inverse of 448), q = e4m3(y / scale)
//   gradient: n = h rstd, d = dy g:  dh = rstd (d - n mean(d n)) + dsum,  dg = sum over rows of dy n
//
// What is stored is what is normalised, so that the gradient, which reads the stored sum, is that of what was computed.
// One pass: a row stays in registers between its sum of squares and its output; the largest |h g| is found along with the sum of
// squares (rstd is the same for all of the row), so 8 bits cost no second reduction.  Sums are fp32.  Bound: memory.
#include "rms_norm.h"
#include "rows_io.cuh"

namespace moe {

namespace {

constexpr float E4M3_INVERSE = 1.f / 448.f;   // of the largest e4m3
constexpr float LEAST_SCALE = 7.888609052210118e-31f;   // 2^-100: its inverse is a number, and a row of zeros stays zeros
constexpr int ROW_WARPS = 8;                            // rows of a block where a warp takes a row

// Sum of a and maximum of b over the row's threads: LANES of a warp, or the block (0).
template <int LANES>
__device__ __forceinline__ void row_reduce(float& a, float& b) {
#pragma unroll
  for (int o = LANES ? LANES / 2 : 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  if (LANES) return;
  __shared__ float2 part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) part[warp] = make_float2(a, b);
  __syncthreads();
  const float2 p = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  a = warp_sum(p.x);
  b = warp_max(p.y);
}

// Rows of any length and alignment, element by element.
template <int NC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ROW_WARPS : 1024) rms_norm_kernel(const NormArgs a) {
  constexpr bool VEC = false;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, stride = WARP ? 32 : blockDim.x;
  const long long t = WARP ? (long long)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.T) return;   // whole warps
  auto row = [&](const void* p, long long ld, int type) { return static_cast<const char*>(p) + t * ld * (type == GT_FP32 ? 4 : 2); };
  float h[NC * CHUNK], g[NC * CHUNK];
  load_row<NC, VEC>(row(a.x, a.ldx, a.x_type), a.x_type, a.H, tid, stride, h);
  if (a.residual) {
    load_row<NC, VEC>(row(a.residual, a.ld_res, a.res_type), a.res_type, a.H, tid, stride, g);
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) h[j] = round_to(h[j] + g[j], a.res_type);
    store_row<NC, VEC>(const_cast<char*>(row(a.sum, a.ld_sum, a.res_type)), a.res_type, a.H, tid, stride, h);
  }
  float ss = 0.f, top = 0.f, rstd = 1.f;
  if (a.norm) {
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) ss = fmaf(h[j], h[j], ss);
  }
  if (a.gain) {
    load_row<NC, VEC>(a.gain, a.gain_type, a.H, tid, stride, g);
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) h[j] *= g[j];
  }
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) top = fmaxf(top, fabsf(h[j]));
  row_reduce<WARP ? 32 : 0>(ss, top);
  if (a.norm) rstd = rsqrtf(ss / (float)a.H + a.eps);
  if (tid == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) h[j] *= rstd;
  if (a.out)
    store_row<NC, VEC>(const_cast<char*>(row(a.out, a.ldo, a.out_type)), a.out_type, a.H, tid, stride, h);
  if (a.out8) {
    const float scale = fmaxf(top * rstd * E4M3_INVERSE, LEAST_SCALE);
    store_e4m3<NC>(a.out8 + t * a.ldo8, a.H, tid, stride, h, scale);
    if (tid == 0) a.scale[t] = scale;
  }
}

// Aligned rows, types known: the row stays in registers as it lies (h in the type it was rounded to), half of what fp32 takes, so
// that more of them are in flight; it is made fp32 twice instead.
// 8192 rows of 7168 (bf16, gain, 8 bits out): with a residual 69.5 us, 0.87 of the memory's rate; without 50, of which 24 instructions an
// element fill 0.76 of the issue slots.
template <int XT, int HT, bool RES, int NC, int LANES, int MAXT>
__global__ void __launch_bounds__(MAXT, NC == 8 ? 2 : 1) rms_norm_words_kernel(const NormArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int tid = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x, stride = LANES ? LANES : blockDim.x;
  const long long at = LANES ? ((long long)blockIdx.x * (32 * ROW_WARPS) + threadIdx.x) / (LANES ? LANES : 1) : blockIdx.x;
  if (LANES && at - (threadIdx.x & 31) / (LANES ? LANES : 1) >= a.T) return;   // whole warps
  // (rows behind the last, in a warp that has others before them, are read as the last and not written)
  const bool live = at < a.T;
  const long long t = live ? at : a.T - 1;
  auto row = [&](const void* p, long long ld, int type) { return static_cast<const char*>(p) + t * ld * (type == GT_FP32 ? 4 : 2); };
  const int n = a.H / CHUNK;
  Word<true, HT> h[NC];
  {
    Word<true, XT> x[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) x[i].load(row(a.x, a.ldx, XT), 0, tid + i * stride, tid + i * stride < n);
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < NC; ++i) h[i].load(row(a.residual, a.ld_res, HT), 0, tid + i * stride, tid + i * stride < n);
      char* sum = const_cast<char*>(row(a.sum, a.ld_sum, HT));
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float v[CHUNK];
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) v[j] = x[i].get(j) + h[i].get(j);
        h[i].set(v);
        if (tid + i * stride < n && live) h[i].store(sum, tid + i * stride);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < Word<true, XT>::REGS; ++q) h[i].r[q] = x[i].r[q];
    }
  }
  float ss = 0.f, top = 0.f, rstd = 1.f;
  // chunk i of y / rstd
  auto scaled = [&](int i, float (&v)[CHUNK]) {
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) v[j] = h[i].get(j);
    if (a.gain && tid + i * stride < n) {
      float g[CHUNK];
      chunk_of<false>(a.gain, tid + i * stride, a.gain_type, g);
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) v[j] *= g[j];
    }
  };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (a.norm) {
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) ss = fmaf(h[i].get(j), h[i].get(j), ss);
    }
    if (a.out8) {
      if (HT != GT_FP32 && !a.gain) {
        top = fmaxf(top, h[i].largest());
      } else {
        float v[CHUNK];
        scaled(i, v);
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) top = fmaxf(top, fabsf(v[j]));
      }
    }
  }
  row_reduce<LANES>(ss, top);
  if (LANES && !live) return;
  if (a.norm) rstd = rsqrtf(ss / (float)a.H + a.eps);
  if (tid == 0 && a.rstd) a.rstd[t] = rstd;
  const float scale = fmaxf(top * rstd * E4M3_INVERSE, LEAST_SCALE);
  // the quotient itself: 16-bit values, and products of two, often lie on a border between two e4m3 numbers, where rstd and the scale
  // in one factor give the wrong one (3 values in 10000 of a bf16 row without a gain)
  const Divisor by(scale);
  if (tid == 0 && a.out8) a.scale[t] = scale;
  char* out = const_cast<char*>(row(a.out, a.ldo, a.out_type));
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tid + i * stride;
    if (c >= n) break;
    float v[CHUNK];
    scaled(i, v);
    if (a.norm) {
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) v[j] *= rstd;
    }
    if (a.out8) reinterpret_cast<uint2*>(a.out8 + t * a.ldo8)[c] = e4m3_chunk(v, by);
    if (a.out) put_chunk(out, c, a.out_type, v);
  }
}

// The gradient.  A thread has the same columns in every row, so the gain's gradient adds up in registers: over a block's rows
// first, then over the blocks by a kernel of its own, in a fixed order.
template <int NC, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ROW_WARPS : 1024) rms_norm_grad_kernel(const NormGradArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, stride = WARP ? 32 : blockDim.x;
  const long long first = WARP ? (long long)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  const long long step = (long long)gridDim.x * (WARP ? ROW_WARPS : 1);
  __shared__ float part[2][32];
  float dg[NC * CHUNK];
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) dg[j] = 0.f;
  int turn = 0;
  for (long long t = first; t < a.T; t += step, turn ^= 1) {
    auto row = [&](const void* p, long long ld, int type) { return static_cast<const char*>(p) + t * ld * (type == GT_FP32 ? 4 : 2); };
    float n[NC * CHUNK], d[NC * CHUNK];
    load_row<NC, VEC>(row(a.h, a.ld_h, a.h_type), a.h_type, a.H, tid, stride, n);
    load_row<NC, VEC>(row(a.dy, a.ld_dy, a.dy_type), a.dy_type, a.H, tid, stride, d);
    const float rstd = __ldg(a.rstd + t);
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) {
      n[j] *= rstd;
      dg[j] = fmaf(d[j], n[j], dg[j]);
    }
    float g[NC * CHUNK];
    if (a.gain) {
      load_row<NC, VEC>(a.gain, a.gain_type, a.H, tid, stride, g);
#pragma unroll
      for (int j = 0; j < NC * CHUNK; ++j) d[j] *= g[j];
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) dot = fmaf(d[j], n[j], dot);
    dot = warp_sum(dot);
    if (!WARP) {
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      if (lane == 0) part[turn][warp] = dot;   // (two in turn: the one before may still be read)
      __syncthreads();
      dot = warp_sum(lane < (int)(blockDim.x >> 5) ? part[turn][lane] : 0.f);
    }
    dot /= (float)a.H;
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) d[j] = rstd * fmaf(-n[j], dot, d[j]);
    if (a.dsum) {
      load_row<NC, VEC>(row(a.dsum, a.ld_dsum, a.dsum_type), a.dsum_type, a.H, tid, stride, g);
#pragma unroll
      for (int j = 0; j < NC * CHUNK; ++j) d[j] += g[j];
    }
    store_row<NC, VEC>(const_cast<char*>(row(a.dh, a.ld_dh, a.dh_type)), a.dh_type, a.H, tid, stride, d);
  }
  if (!a.dgain) return;
  float* out = a.partial + (long long)blockIdx.x * a.H;
  if (WARP) {   // the warps' sums in order
    extern __shared__ float sums[];   // [ROW_WARPS][H]
    float* mine = sums + (threadIdx.x >> 5) * a.H;
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) {
      const int e = element_of<NC, VEC>(j, tid, stride);
      if (e < a.H) mine[e] = dg[j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.H; e += blockDim.x) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < ROW_WARPS; ++w) s += sums[w * a.H + e];
      out[e] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC * CHUNK; ++j) {
      const int e = element_of<NC, VEC>(j, tid, stride);
      if (e < a.H) out[e] = dg[j];
    }
  }
}

// Aligned rows of a block: two blocks an SM (one where two rows do not fit twice), the rows of dy, h and dsum copied ahead into a
// ring of `stages` in shared memory, so that they arrive while the row before them waits for its sum.  Everything of a stage is
// read before the barrier of its row's sum, so behind it the stage is filled again.  8191 rows of 4096 (bf16 dy, fp32 h, dsum and dh): 70 us,
// 0.98 of the memory's rate; with one block of 512 threads an SM 78, with rows loaded into registers 86.
struct GradRing {
  int stages;
  uint32_t dy_bytes, h_bytes, dsum_bytes;   // of a row
  WaitLimit wait;
};
constexpr int RING_MAX = 8;
template <bool NARROW>
struct RingWords {   // 8 elements as they lie, of 16 bits (NARROW) or a type known at run time
  uint32_t r[NARROW ? 4 : 8];
  __device__ __forceinline__ void load(const uint8_t* row, int c, int type) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
    const bool wide = !NARROW && type == GT_FP32;
    const uint4 lo = p[wide ? 2 * c : c];
    r[0] = lo.x, r[1] = lo.y, r[2] = lo.z, r[3] = lo.w;
    if constexpr (!NARROW) {
      const uint4 hi = wide ? p[2 * c + 1] : lo;
      r[4] = hi.x, r[5] = hi.y, r[6] = hi.z, r[7] = hi.w;
    }
  }
  __device__ __forceinline__ void values(int type, float (&v)[CHUNK]) const {
    if (!NARROW && type == GT_FP32) {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) v[i] = __uint_as_float(r[NARROW ? 0 : i]);
    } else {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const float2 f = two_16(r[i / 2], type);
        v[i] = i % 2 ? f.y : f.x;
      }
    }
  }
};
template <int NC, int PER_SM, int MAXT, bool NARROW, bool KEEP>
__global__ void __launch_bounds__(MAXT, PER_SM) rms_norm_grad_ring_kernel(const NormGradArgs a, const GradRing ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part[2][32];
  __shared__ uint64_t bars[RING_MAX];
  __shared__ int gave_up[2];   // by the row's turn, as the sums
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, stride = blockDim.x, n = a.H / CHUNK;
  const uint32_t stage = ring.dy_bytes + ring.h_bytes + ring.dsum_bytes, bytes = stage;
  if (tid == 0) {
    for (int s = 0; s < ring.stages; ++s) mbar_init(smem_u32(bars + s), 1 + (ring.wait.cycles == 0));
    gave_up[0] = gave_up[1] = 0;
    mbar_fence_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  auto fill = [&](long long t, int s) {   // thread 0
    const uint32_t bar = smem_u32(bars + s), at = smem_u32(smem) + s * stage;
    auto row = [&](const void* p, long long ld, uint32_t row_bytes) {
      return static_cast<const char*>(p) + t * ld * (row_bytes / (uint32_t)a.H);
    };
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(at, row(a.dy, a.ld_dy, ring.dy_bytes), ring.dy_bytes, bar);
    bulk_g2s(at + ring.dy_bytes, row(a.h, a.ld_h, ring.h_bytes), ring.h_bytes, bar);
    if (a.dsum) bulk_g2s(at + ring.dy_bytes + ring.h_bytes, row(a.dsum, a.ld_dsum, ring.dsum_bytes), ring.dsum_bytes, bar);
  };
  const long long first = blockIdx.x, step = gridDim.x;
  if (tid == 0)
    for (int s = 0; s < ring.stages; ++s)
      if (first + s * step < a.T) fill(first + s * step, s);
  // The gain: in registers, or behind the stages (it is read twice a row, and little of L1 is left to read it from).
  uint4* gains = reinterpret_cast<uint4*>(smem + ring.stages * stage);
  float kept[KEEP ? NC * CHUNK : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float v[CHUNK];
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) v[j] = 1.f;
      if (a.gain && tid + i * stride < n) chunk_of<false>(a.gain, tid + i * stride, a.gain_type, v);
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) kept[i * CHUNK + j] = v[j];
    }
  } else {
    if (a.gain)
      for (int i = tid; i < n * (a.gain_type == GT_FP32 ? 2 : 1); i += stride) gains[i] = __ldg(static_cast<const uint4*>(a.gain) + i);
    __syncthreads();
  }
  float dg[NC * CHUNK];
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) dg[j] = 0.f;
  int s = 0, turn = 0;
  uint32_t parity = 0;
  float next_rstd = first < a.T ? __ldg(a.rstd + first) : 0.f;   // a row ahead, as all of the row waits for it
  for (long long t = first; t < a.T; t += step, turn ^= 1) {
    const float rstd = next_rstd;
    if (t + step < a.T) next_rstd = __ldg(a.rstd + t + step);
    if (!mbar_wait_bounded(smem_u32(bars + s), parity, ring.wait.cycles)) gave_up[turn] = 1;
    const uint8_t* at = smem + s * stage;
    RingWords<NARROW> y[NC], h[NC], ds[NC];
    float dot = 0.f;
    // n and d of chunk i; made twice, as the words take half the registers (16-bit rows)
    auto values = [&](int i, float (&yv)[CHUNK], float (&nv)[CHUNK], float (&d)[CHUNK]) {
      y[i].values(a.dy_type, yv);
      h[i].values(a.h_type, nv);
      float g[CHUNK];
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) g[j] = KEEP ? kept[KEEP ? i * CHUNK + j : 0] : 1.f;
      if (!KEEP && a.gain) chunk_of<true>(gains, tid + i * stride, a.gain_type, g);
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) {
        nv[j] *= rstd;
        d[j] = yv[j] * g[j];
      }
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tid + i * stride;
      if (c < n) {
        y[i].load(at, c, a.dy_type);
        h[i].load(at + ring.dy_bytes, c, a.h_type);
        if (a.dsum) ds[i].load(at + ring.dy_bytes + ring.h_bytes, c, a.dsum_type);
        float yv[CHUNK], nv[CHUNK], d[CHUNK];
        values(i, yv, nv, d);
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) {
          dg[i * CHUNK + j] = fmaf(yv[j], nv[j], dg[i * CHUNK + j]);
          dot = fmaf(d[j], nv[j], dot);
        }
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) part[turn][warp] = dot;   // (two in turn: the one before may still be read)
    __syncthreads();
    if (gave_up[turn]) break;   // the same in all threads
    if (tid == 0 && t + ring.stages * step < a.T) fill(t + ring.stages * step, s);
    dot = warp_sum(lane < (stride >> 5) ? part[turn][lane] : 0.f) / (float)a.H;
    char* out = static_cast<char*>(a.dh) + t * a.ld_dh * (a.dh_type == GT_FP32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tid + i * stride;
      if (c < n) {
        float v[CHUNK], yv[CHUNK], nv[CHUNK], d[CHUNK];
        values(i, yv, nv, d);
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) v[j] = rstd * fmaf(-nv[j], dot, d[j]);
        if (a.dsum) {
          ds[i].values(a.dsum_type, yv);
#pragma unroll
          for (int j = 0; j < CHUNK; ++j) v[j] += yv[j];
        }
        put_chunk(out, c, a.dh_type, v);
      }
    }
    if (++s == ring.stages) {
      s = 0;
      parity ^= 1;
    }
  }
  if (gave_up[turn]) {   // a wait ran out: report, and let the copies in flight end before the memory goes
    if (tid == 0) {
      *reinterpret_cast<volatile uint32_t*>(ring.wait.status) = ST_TIMEOUT;
      __threadfence_system();
    }
    const long long t0 = clock64();
    while (clock64() - t0 < 100000000ll) __nanosleep(1000);
    return;
  }
  if (!a.dgain) return;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (tid + i * stride < n) {
      float* out = a.partial + (long long)blockIdx.x * a.H + (tid + i * stride) * CHUNK;
      reinterpret_cast<float4*>(out)[0] = make_float4(dg[i * CHUNK], dg[i * CHUNK + 1], dg[i * CHUNK + 2], dg[i * CHUNK + 3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(dg[i * CHUNK + 4], dg[i * CHUNK + 5], dg[i * CHUNK + 6], dg[i * CHUNK + 7]);
    }
}

// Aligned rows of up to WARP_H, a warp a row: the three rows' words loaded together, a row ahead (10182 rows of 64: 24 us a call
// with loads one after another, 13 so, 7.4 of them on the device).
struct RawChunk {   // 8 elements of a type known at run time, as they lie
  uint32_t r[8];
  __device__ __forceinline__ void load(const void* row, int c, int type, bool in) {
    const char* p = static_cast<const char*>(row) + (long long)c * (type == GT_FP32 ? 32 : 16);
    Word<true, GT_BF16> lo, hi;
    lo.load(p, 0, 0, in);
    hi.load(p, CHUNK, 0, in && type == GT_FP32);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = lo.r[i];
      r[4 + i] = hi.r[i];
    }
  }
  __device__ __forceinline__ void values(int type, float (&v)[CHUNK]) const {
    if (type == GT_FP32) {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) v[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const float2 f = two_16(r[i / 2], type);
        v[i] = i % 2 ? f.y : f.x;
      }
    }
  }
};
template <int NC>
__global__ void __launch_bounds__(32 * ROW_WARPS) rms_norm_grad_warp_kernel(const NormGradArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, n = a.H / CHUNK;
  const long long first = (long long)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5), step = (long long)gridDim.x * ROW_WARPS;
  float dg[NC * CHUNK], g[NC * CHUNK];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float v[CHUNK];
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) v[j] = 1.f;
    if (a.gain && lane + 32 * i < n) chunk_of<false>(a.gain, lane + 32 * i, a.gain_type, v);
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) {
      g[i * CHUNK + j] = v[j];
      dg[i * CHUNK + j] = 0.f;
    }
  }
  RawChunk y[NC], h[NC], ds[NC];
  float rstd = 0.f;
  auto load = [&](long long t) {
    auto row = [&](const void* p, long long ld, int type) { return static_cast<const char*>(p) + t * ld * (type == GT_FP32 ? 4 : 2); };
    const bool live = t < a.T;
    rstd = live ? __ldg(a.rstd + t) : 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + 32 * i;
      y[i].load(row(a.dy, a.ld_dy, a.dy_type), c, a.dy_type, live && c < n);
      h[i].load(row(a.h, a.ld_h, a.h_type), c, a.h_type, live && c < n);
      ds[i].load(row(a.dsum, a.ld_dsum, a.dsum_type), c, a.dsum_type, live && a.dsum && c < n);
    }
  };
  load(first);
  for (long long t = first; t < a.T; t += step) {
    float nv[NC * CHUNK], d[NC * CHUNK], s[NC * CHUNK], dot = 0.f;
    const float r = rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float yv[CHUNK], hv[CHUNK], sv[CHUNK];
      y[i].values(a.dy_type, yv);
      h[i].values(a.h_type, hv);
      ds[i].values(a.dsum_type, sv);
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) {
        const int k = i * CHUNK + j;
        nv[k] = hv[j] * r;
        dg[k] = fmaf(yv[j], nv[k], dg[k]);
        d[k] = yv[j] * g[k];
        dot = fmaf(d[k], nv[k], dot);
        s[k] = sv[j];
      }
    }
    load(t + step);
    dot = warp_sum(dot) / (float)a.H;
    char* out = static_cast<char*>(a.dh) + t * a.ld_dh * (a.dh_type == GT_FP32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (lane + 32 * i < n) {
        float v[CHUNK];
#pragma unroll
        for (int j = 0; j < CHUNK; ++j) v[j] = r * fmaf(-nv[i * CHUNK + j], dot, d[i * CHUNK + j]) + s[i * CHUNK + j];
        put_chunk(out, lane + 32 * i, a.dh_type, v);
      }
  }
  if (!a.dgain) return;
  extern __shared__ float sums[];   // [ROW_WARPS][H], the warps' in order
  float* mine = sums + (threadIdx.x >> 5) * a.H;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (lane + 32 * i < n)
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) mine[(lane + 32 * i) * CHUNK + j] = dg[i * CHUNK + j];
  __syncthreads();
  for (int e = threadIdx.x; e < a.H; e += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < ROW_WARPS; ++w) v += sums[w * a.H + e];
    a.partial[(long long)blockIdx.x * a.H + e] = v;
  }
}

// dgain = the blocks' sums: 32 columns a block, a warp every 32nd row (its loads all at once: 7.4 us for 304 rows of 4096, with 8 warps 8.0)
constexpr int SUM_PARTS = 32;
__global__ void __launch_bounds__(32 * SUM_PARTS) sum_blocks_kernel(const float* partial, float* out, int blocks, int H) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float part[SUM_PARTS][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float s = 0.f;
  if (e < H) {
#pragma unroll 10
    for (int b = w; b < blocks; b += SUM_PARTS) s += partial[(long long)b * H + e];
  }
  part[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w || e >= H) return;
#pragma unroll
  for (int q = 1; q < SUM_PARTS; ++q) s += part[q][threadIdx.x];
  out[e] = s;
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), long long blocks, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// How a row is shared out: by a warp or a block, `nc` runs of 8 elements a thread.
struct Share {
  bool warp;
  int nc, threads;
};
constexpr int WARP_H = 1024;   // the longest row of a warp
constexpr int RING_SMS = 152;   // a constant, as norm_grad_blocks
Share share_of(int H, int most_nc) {
  if (H <= WARP_H) return {true, H <= 256 ? 1 : H <= 512 ? 2 : 4, 32 * ROW_WARPS};
  int nc = 1;
  while (nc < 4 && (nc < most_nc || H > nc * CHUNK * 1024)) nc *= 2;
  return {false, nc, (H + nc * CHUNK * 32 - 1) / (nc * CHUNK * 32) * 32};
}

bool multiple(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }
size_t bytes_of(int type) { return type == GT_FP32 ? 4 : 2; }
// rows that can be read and written in chunks (p null: there are none)
bool chunks(const void* p, long long ld, int type) { return !p || (multiple(p, 16) && ld * bytes_of(type) % 16 == 0); }

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
  const bool vec = a.H % CHUNK == 0 && chunks(a.x, a.ldx, a.x_type) && chunks(a.residual, a.ld_res, a.res_type) &&
                   chunks(a.residual ? a.sum : nullptr, a.ld_sum, a.res_type) && chunks(a.gain, 0, a.gain_type) &&
                   chunks(a.out, a.ldo, a.out_type) && (!a.out8 || (multiple(a.out8, 8) && a.ldo8 % 8 == 0));
  using std::integral_constant;
  using True = std::true_type;
  using False = std::false_type;
  if (!vec) {
    const Share sh = share_of(a.H, 4);
    const long long blocks = sh.warp ? ((long long)a.T + ROW_WARPS - 1) / ROW_WARPS : a.T;
    auto go = [&](auto nc, auto w) {
      return launch(rms_norm_kernel<decltype(nc)::value, decltype(w)::value>, blocks, sh.threads, 0, s, a);
    };
    auto with = [&](auto nc) { return sh.warp ? go(nc, True{}) : go(nc, False{}); };
    return sh.nc == 1 ? with(integral_constant<int, 1>{}) : sh.nc == 2 ? with(integral_constant<int, 2>{}) : with(integral_constant<int, 4>{});
  }
  // A warp a row up to WARP_H, else a block: of few chunks a thread where there are fewer rows than SMs (latency), four otherwise.
  const bool warp = a.H <= WARP_H;
  const int lanes = a.H <= 64 ? 8 : a.H <= 128 ? 16 : 32;   // of a row, in a warp
  const bool few = a.T <= num_sms, eight = !few && !a.norm && a.x_type != GT_FP32 && a.H >= 4096;
  const int nc = warp ? (a.H <= 256 ? 1 : a.H <= 512 ? 2 : 4) : few && a.H <= 8192 ? 1 : eight ? 8 : 4;
  const int rows = 32 * ROW_WARPS / lanes;
  const long long blocks = warp ? ((long long)a.T + rows - 1) / rows : a.T;
  const int threads = warp ? 32 * ROW_WARPS : (a.H / CHUNK + nc * 32 - 1) / (nc * 32) * 32;
  auto types = [&](auto xt, auto ht, auto res) {
    auto go = [&](auto c, auto w, auto most) {
      return launch(rms_norm_words_kernel<decltype(xt)::value, decltype(ht)::value, decltype(res)::value, decltype(c)::value,
                                          decltype(w)::value, decltype(most)::value>,
                    blocks, threads, 0, s, a);
    };
    using W = integral_constant<int, 32 * ROW_WARPS>;
    using Block = integral_constant<int, 0>;
    if (warp) {
      if (lanes == 8) return go(integral_constant<int, 1>{}, integral_constant<int, 8>{}, W{});
      if (lanes == 16) return go(integral_constant<int, 1>{}, integral_constant<int, 16>{}, W{});
      return nc == 1   ? go(integral_constant<int, 1>{}, integral_constant<int, 32>{}, W{})
             : nc == 2 ? go(integral_constant<int, 2>{}, integral_constant<int, 32>{}, W{})
                       : go(integral_constant<int, 4>{}, integral_constant<int, 32>{}, W{});
    }
    if (nc == 1) return go(integral_constant<int, 1>{}, Block{}, integral_constant<int, 1024>{});
    if constexpr (!decltype(res)::value && decltype(xt)::value != GT_FP32) {   // (rows as they are)
      if (nc == 8) return go(integral_constant<int, 8>{}, Block{}, integral_constant<int, 512>{});
    }
    return threads <= 512 ? go(integral_constant<int, 4>{}, Block{}, integral_constant<int, 512>{})
                          : go(integral_constant<int, 4>{}, Block{}, integral_constant<int, 1024>{});
  };
  auto of = [](int type, auto f) {
    if (type == GT_FP32) return f(integral_constant<int, GT_FP32>{});
    return type == GT_BF16 ? f(integral_constant<int, GT_BF16>{}) : f(integral_constant<int, GT_FP16>{});
  };
  return of(a.x_type, [&](auto xt) {
    if (!a.residual) return types(xt, xt, False{});
    return of(a.res_type, [&](auto rt) { return types(xt, rt, True{}); });
  });
}

int norm_grad_blocks(int T, int H) {
  const bool warp = H <= WARP_H;
  const int most = 304, need = warp ? (int)(((long long)T + ROW_WARPS - 1) / ROW_WARPS) : T;
  return need < most ? need : most;
}

namespace {
constexpr size_t ring_bytes(int per_sm) { return (per_sm == 2 ? 110 : 226) * 1024; }
// The kernels: chunks a thread, blocks an SM, most threads, rows all of 16 bits, the gain in registers.
template <int NC, int PER_SM, int MAXT, bool NARROW, bool KEEP>
struct Ring {
  static cudaError_t attribute() {
    return cudaFuncSetAttribute(rms_norm_grad_ring_kernel<NC, PER_SM, MAXT, NARROW, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)ring_bytes(PER_SM));
  }
  static cudaError_t launch_it(const NormGradArgs& a, const GradRing& r, int& blocks, cudaStream_t s) {
    const int threads = (a.H / CHUNK + NC * 32 - 1) / (NC * 32) * 32, most = PER_SM * RING_SMS;
    if (blocks > most) blocks = most;
    return launch(rms_norm_grad_ring_kernel<NC, PER_SM, MAXT, NARROW, KEEP>, blocks, threads, (size_t)r.stages * (r.dy_bytes + r.h_bytes + r.dsum_bytes) + (a.gain && !KEEP ? a.H * bytes_of(a.gain_type) : 0), s, a, r);
  }
};
using Ring2048 = Ring<1, 2, 256, false, true>;
using Ring4096 = Ring<2, 2, 256, false, true>;
using Ring7168Narrow = Ring<2, 2, 448, true, false>;
using Ring8192 = Ring<2, 1, 512, false, true>;
using Ring16384 = Ring<4, 1, 512, false, false>;
}  // namespace

cudaError_t rms_norm_set_attributes() {
  cudaError_t e = Ring2048::attribute();
  if (e == cudaSuccess) e = Ring4096::attribute();
  if (e == cudaSuccess) e = Ring8192::attribute();
  if (e == cudaSuccess) e = Ring7168Narrow::attribute();
  return e == cudaSuccess ? Ring16384::attribute() : e;
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, const WaitLimit& wait, cudaStream_t s) {
  const bool vec = a.H % CHUNK == 0 && chunks(a.dy, a.ld_dy, a.dy_type) && chunks(a.h, a.ld_h, a.h_type) &&
                   chunks(a.gain, 0, a.gain_type) && chunks(a.dsum, a.ld_dsum, a.dsum_type) && chunks(a.dh, a.ld_dh, a.dh_type);
  int blocks = norm_grad_blocks(a.T, a.H);
  cudaError_t e;
  GradRing ring{0, (uint32_t)(a.H * bytes_of(a.dy_type)), (uint32_t)(a.H * bytes_of(a.h_type)),
                a.dsum ? (uint32_t)(a.H * bytes_of(a.dsum_type)) : 0u, wait};
  const size_t row = ring.dy_bytes + ring.h_bytes + ring.dsum_bytes;
  const bool narrow = a.dy_type != GT_FP32 && a.h_type != GT_FP32 && (!a.dsum || a.dsum_type != GT_FP32);
  const size_t gain = a.gain && a.H > (narrow ? 4096 : 8192) ? a.H * bytes_of(a.gain_type) : 0;   // (in shared memory)
  // (16-bit rows of 8192 would fit twice in shared memory, but leave 64 registers a thread of the 72 that 7168 takes: 160 bytes of spills)
  const int per_sm = a.H <= (narrow ? 7168 : 4096) && 2 * row + gain <= ring_bytes(2) ? 2 : 1;
  const size_t fit = (ring_bytes(per_sm) - gain) / row;   // (the gain takes 64 KB at most)
  ring.stages = fit < RING_MAX ? (int)fit : RING_MAX;
  if (vec && a.H > WARP_H && a.H <= 16384 && ring.stages >= 2) {
    if (per_sm == 2)
      e = a.H <= 2048   ? Ring2048::launch_it(a, ring, blocks, s)
          : a.H <= 4096 ? Ring4096::launch_it(a, ring, blocks, s)
                        : Ring7168Narrow::launch_it(a, ring, blocks, s);
    else
      e = a.H <= 8192 ? Ring8192::launch_it(a, ring, blocks, s) : Ring16384::launch_it(a, ring, blocks, s);
  } else if (vec && a.H <= WARP_H) {
    const size_t smem = a.dgain ? (size_t)ROW_WARPS * a.H * sizeof(float) : 0;   // 32 KB at most
    const int threads = 32 * ROW_WARPS;
    e = a.H <= 256   ? launch(rms_norm_grad_warp_kernel<1>, blocks, threads, smem, s, a)
        : a.H <= 512 ? launch(rms_norm_grad_warp_kernel<2>, blocks, threads, smem, s, a)
                     : launch(rms_norm_grad_warp_kernel<4>, blocks, threads, smem, s, a);
  } else {
    const Share sh = share_of(a.H, 1);
    const size_t smem = sh.warp && a.dgain ? (size_t)ROW_WARPS * a.H * sizeof(float) : 0;   // 32 KB at most
    auto go = [&](auto nc, auto v, auto w) {
      return launch(rms_norm_grad_kernel<decltype(nc)::value, decltype(v)::value, decltype(w)::value>, blocks, sh.threads, smem, s, a);
    };
    auto with = [&](auto nc) {
      using T = std::true_type;
      using F = std::false_type;
      return sh.warp ? go(nc, F{}, T{}) : vec ? go(nc, T{}, F{}) : go(nc, F{}, F{});
    };
    e = sh.nc == 1   ? with(std::integral_constant<int, 1>{})
        : sh.nc == 2 ? with(std::integral_constant<int, 2>{})
                     : with(std::integral_constant<int, 4>{});
  }
  if (e == cudaSuccess && a.dgain)
    e = launch(sum_blocks_kernel, (a.H + 31) / 32, 32 * SUM_PARTS, 0, s, (const float*)a.partial, a.dgain, blocks, a.H);
  return e;
}

}  // namespace moe
