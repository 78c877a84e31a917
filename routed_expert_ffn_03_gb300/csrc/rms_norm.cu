// rms_norm.cu - root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its gradient.
//
//   h = round(x + residual)  (to the residual's type; x without one),  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd g
//   8 bits: scale = max(max|y| / 448, 2^-100), q = e4m3(y / scale)
//   gradient: n = h rstd, d = dy g:  dh = rstd (d - n mean(d n)) + dsum,  dg = sum over rows of dy n
//
// What is stored is what is normalised, so that the gradient, which reads the stored sum, is that of what was computed.
// One pass: a row stays in registers between its sum of squares and its output; the largest |h g| is found along with the sum of
// squares (rstd is the same for all of the row), so 8 bits cost no second reduction.  Sums are fp32.  Bound: memory.
#include "rms_norm.h"
#include "rows_io.cuh"

namespace moe {

namespace {

constexpr float E4M3_MAX = 448.f;
constexpr float LEAST_SCALE = 7.888609052210118e-31f;   // 2^-100: its inverse is a number, and a row of zeros stays zeros
constexpr int ROW_WARPS = 8;                            // rows of a block where a warp takes a row

// Sum of a and maximum of b over the row's threads: a warp, or the block.
template <bool WARP>
__device__ __forceinline__ void row_reduce(float& a, float& b) {
  a = warp_sum(a);
  b = warp_max(b);
  if (WARP) return;
  __shared__ float2 part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) part[warp] = make_float2(a, b);
  __syncthreads();
  const float2 p = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  a = warp_sum(p.x);
  b = warp_max(p.y);
}

template <int NC, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ROW_WARPS : 1024) rms_norm_kernel(const NormArgs a) {
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
  row_reduce<WARP>(ss, top);
  if (a.norm) rstd = rsqrtf(ss / (float)a.H + a.eps);
  if (tid == 0 && a.rstd) a.rstd[t] = rstd;
#pragma unroll
  for (int j = 0; j < NC * CHUNK; ++j) h[j] *= rstd;
  if (a.out)
    store_row<NC, VEC>(const_cast<char*>(row(a.out, a.ldo, a.out_type)), a.out_type, a.H, tid, stride, h);
  if (a.out8) {
    const float scale = fmaxf(top * rstd / E4M3_MAX, LEAST_SCALE);
    store_e4m3<NC, VEC>(a.out8 + t * a.ldo8, a.H, tid, stride, h, scale);
    if (tid == 0) a.scale[t] = scale;
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

// dgain = the blocks' sums: 32 columns a block, 8 parts of the rows, each in order
constexpr int SUM_PARTS = 8;
__global__ void __launch_bounds__(32 * SUM_PARTS) sum_blocks_kernel(const float* partial, float* out, int blocks, int H) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float part[SUM_PARTS][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float s = 0.f;
  if (e < H) {
#pragma unroll 8
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
  const Share sh = share_of(a.H, a.T <= num_sms ? 1 : 4);
  const bool vec = a.H % CHUNK == 0 && chunks(a.x, a.ldx, a.x_type) && chunks(a.residual, a.ld_res, a.res_type) &&
                   chunks(a.residual ? a.sum : nullptr, a.ld_sum, a.res_type) && chunks(a.gain, 0, a.gain_type) &&
                   chunks(a.out, a.ldo, a.out_type) && (!a.out8 || (multiple(a.out8, 8) && a.ldo8 % 8 == 0));
  const long long blocks = sh.warp ? ((long long)a.T + ROW_WARPS - 1) / ROW_WARPS : a.T;
  auto go = [&](auto nc, auto v, auto w) {
    return launch(rms_norm_kernel<decltype(nc)::value, decltype(v)::value, decltype(w)::value>, blocks, sh.threads, 0, s, a);
  };
  auto with = [&](auto nc) {
    using T = std::true_type;
    using F = std::false_type;
    return sh.warp ? (vec ? go(nc, T{}, T{}) : go(nc, F{}, T{})) : vec ? go(nc, T{}, F{}) : go(nc, F{}, F{});
  };
  if (sh.nc == 1) return with(std::integral_constant<int, 1>{});
  return sh.nc == 2 ? with(std::integral_constant<int, 2>{}) : with(std::integral_constant<int, 4>{});
}

int norm_grad_blocks(int T, int H) {
  const bool warp = H <= WARP_H;
  const int most = 304, need = warp ? (int)(((long long)T + ROW_WARPS - 1) / ROW_WARPS) : T;
  return need < most ? need : most;
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  const Share sh = share_of(a.H, 1);
  const bool vec = a.H % CHUNK == 0 && chunks(a.dy, a.ld_dy, a.dy_type) && chunks(a.h, a.ld_h, a.h_type) &&
                   chunks(a.gain, 0, a.gain_type) && chunks(a.dsum, a.ld_dsum, a.dsum_type) && chunks(a.dh, a.ld_dh, a.dh_type);
  const int blocks = norm_grad_blocks(a.T, a.H);
  const size_t smem = sh.warp && a.dgain ? (size_t)ROW_WARPS * a.H * sizeof(float) : 0;   // 32 KB at most
  auto go = [&](auto nc, auto v, auto w) {
    return launch(rms_norm_grad_kernel<decltype(nc)::value, decltype(v)::value, decltype(w)::value>, blocks, sh.threads, smem, s, a);
  };
  auto with = [&](auto nc) {
    using T = std::true_type;
    using F = std::false_type;
    return sh.warp ? (vec ? go(nc, T{}, T{}) : go(nc, F{}, T{})) : vec ? go(nc, T{}, F{}) : go(nc, F{}, F{});
  };
  cudaError_t e = sh.nc == 1   ? with(std::integral_constant<int, 1>{})
                  : sh.nc == 2 ? with(std::integral_constant<int, 2>{})
                               : with(std::integral_constant<int, 4>{});
  if (e == cudaSuccess && a.dgain)
    e = launch(sum_blocks_kernel, (a.H + 31) / 32, 32 * SUM_PARTS, 0, s, (const float*)a.partial, a.dgain, blocks, a.H);
  return e;
}

}  // namespace moe
