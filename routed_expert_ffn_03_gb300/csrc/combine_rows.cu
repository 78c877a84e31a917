// combine_rows.cu - the weighted sum of a token's expert results, where the grouped products left them, and its gradient.
//
//   out[t] = sum_j weights[t][j] y[places[t][j]]  (+ residual[t])      in rank order, fp32, rounded once
//   dy[places[t][j]] = weights[t][j] dout[t],   dweights[t][j] = <dout[t], y[places[t][j]]>
//
// The rows are named by where they stand, so the products can leave them by expert (a scattering product takes up to 15% longer)
// and no copy puts them in order.  A place outside y is no row: it adds nothing, and its weight's gradient is 0; a weight of 0
// reads no row, as that of a masked pair was never written.  Bound: memory; a thread has eight rows' words in flight, loaded with
// predicates, not branches.  2049 tokens of 7168, k = 8, bf16: 47 us, 0.92 of the memory's rate (with a branch around each load 155); the
// gradient of 8192 tokens of 4096, k = 2: 53 us, 0.94 (137).
#include "combine_rows.h"
#include "rows_io.cuh"

namespace moe {

namespace {

constexpr int CR_THREADS = 256;
constexpr int CR_RANKS = 8;    // rows in flight, where k > 2
constexpr int CR_MAX_K = 32;

// The token's rows and weights into shared memory: offsets in elements, -1 for none.
__device__ __forceinline__ void token_rows(const float* weights, const int* places, long long t, int k, long long y_rows, long long ld,
                                           bool skip_zero, long long* off, float* w) {
  if (threadIdx.x < k) {
    const long long i = t * k + threadIdx.x, r = places ? __ldg(places + i) : i;
    const float weight = __ldg(weights + i);
    const bool in = r >= 0 && r < y_rows && (weight != 0.f || !skip_zero);
    off[threadIdx.x] = in ? r * ld : -1;
    w[threadIdx.x] = weight;
  }
  __syncthreads();
}

template <bool VEC>
__device__ __forceinline__ void store_word(void* p, long long off, int c, int type, const float (&v)[VEC ? CHUNK : 1]) {
  if constexpr (!VEC) {
    put_value(p, off + c, type, v[0]);
  } else if (type == GT_FP32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + off) + 2 * c;
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off)[c] =
        make_uint4(pack_16(v[0], v[1], type), pack_16(v[2], v[3], type), pack_16(v[4], v[5], type), pack_16(v[6], v[7], type));
  }
}

// A block: a token, and one of gridDim.y runs of its columns; RANKS rows at a time.
template <bool VEC, int YT, int OT, int RANKS>
__global__ void __launch_bounds__(CR_THREADS) combine_rows_kernel(const CombineRowsArgs a) {
  constexpr int N = VEC ? CHUNK : 1;
  __shared__ long long off[CR_MAX_K];
  __shared__ float weight[CR_MAX_K];
  pdl_launch_dependents();
  pdl_wait();
  const long long t = blockIdx.x;
  token_rows(a.weights, a.places, t, a.k, a.y_rows, a.ldy, true, off, weight);
  const int words = a.H / N;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < words; c += gridDim.y * blockDim.x) {
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
    Word<VEC, OT> res;
    res.load(a.residual, t * a.ld_res, c, a.residual != nullptr);
    for (int j0 = 0; j0 < a.k; j0 += RANKS) {
      Word<VEC, YT> v[RANKS];
#pragma unroll
      for (int j = 0; j < RANKS; ++j) {
        const long long o = j0 + j < a.k ? off[j0 + j] : -1;
        v[j].load(a.y, o, c, o >= 0);
      }
#pragma unroll
      for (int j = 0; j < RANKS; ++j) {
        const float w = j0 + j < a.k && off[j0 + j] >= 0 ? weight[j0 + j] : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w, v[j].get(i), sum[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += res.get(i);
    store_word<VEC>(a.out, t * a.ldo, c, OT, sum);
  }
}

// A block: a token, as the weights' gradients are sums over all of its columns; RANKS rows at a time.
template <bool VEC, int DT, int YT, int RANKS>
__global__ void __launch_bounds__(512) combine_grad_kernel(const CombineGradArgs a) {
  constexpr int N = VEC ? CHUNK : 1;
  __shared__ long long off[CR_MAX_K];
  __shared__ float weight[CR_MAX_K];
  __shared__ float part[16][CR_MAX_K];
  pdl_launch_dependents();
  pdl_wait();
  const long long t = blockIdx.x;
  token_rows(a.weights, a.places, t, a.k, a.y_rows, 1, false, off, weight);
  const int words = a.H / N, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j0 = 0; j0 < a.k; j0 += RANKS) {
    float dot[RANKS];
#pragma unroll
    for (int j = 0; j < RANKS; ++j) dot[j] = 0.f;
    for (int c = threadIdx.x; c < words; c += blockDim.x) {
      Word<VEC, DT> d;
      Word<VEC, YT> v[RANKS];
      d.load(a.dout, t * a.ld_dout, c, true);
#pragma unroll
      for (int j = 0; j < RANKS; ++j) {
        const long long o = j0 + j < a.k ? off[j0 + j] : -1;
        v[j].load(a.y, o * a.ldy, c, o >= 0);
      }
#pragma unroll
      for (int j = 0; j < RANKS; ++j) {
        if (j0 + j < a.k && off[j0 + j] >= 0) {
          const float w = weight[j0 + j];
          float o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j] = fmaf(d.get(i), v[j].get(i), dot[j]);
            o[i] = w * d.get(i);
          }
          store_word<VEC>(a.dy, off[j0 + j] * a.ld_dy, c, YT, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RANKS; ++j) {
      if (j0 + j >= a.k) break;
      const float s = warp_sum(dot[j]);
      if (lane == 0) part[warp][j0 + j] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < a.k) {   // the warps' sums in order
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += part[w][threadIdx.x];
    a.dweights[t * a.k + threadIdx.x] = s;
  }
}

template <typename A>
cudaError_t launch(void (*kernel)(A), dim3 grid, int threads, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a);
}

bool chunks(const void* p, long long ld, int type) {
  return !p || ((uintptr_t)p % 16 == 0 && ld * (type == GT_FP32 ? 4 : 2) % 16 == 0);
}
// f with vec, two types and the rows at a time (2 where there are no more, for their registers) as constants
template <typename F>
cudaError_t by_types(bool vec, int t0, int t1, int k, F f) {
  auto type = [](int t, auto g) {
    if (t == GT_FP32) return g(std::integral_constant<int, GT_FP32>{});
    return t == GT_BF16 ? g(std::integral_constant<int, GT_BF16>{}) : g(std::integral_constant<int, GT_FP16>{});
  };
  return type(t0, [&](auto a) {
    return type(t1, [&](auto b) {
      auto ranks = [&](auto v) {
        return k <= 2 ? f(v, a, b, std::integral_constant<int, 2>{}) : f(v, a, b, std::integral_constant<int, CR_RANKS>{});
      };
      return vec ? ranks(std::true_type{}) : ranks(std::false_type{});
    });
  });
}
int warps_of(long long words, int most) {
  const long long t = (words + 31) / 32 * 32;
  return t < most ? (int)t : most;
}

}  // namespace

cudaError_t launch_combine_rows(const CombineRowsArgs& a, cudaStream_t s) {
  const bool vec = a.H % CHUNK == 0 && chunks(a.y, a.ldy, a.y_type) && chunks(a.residual, a.ld_res, a.out_type) &&
                   chunks(a.out, a.ldo, a.out_type);
  const long long words = vec ? a.H / CHUNK : a.H;
  long long runs = (words + CR_THREADS - 1) / CR_THREADS;
  const int threads = warps_of((words + runs - 1) / runs, CR_THREADS);   // even runs
  if (runs > 65535) runs = 65535;
  const dim3 grid((unsigned)a.T, (unsigned)runs);
  return by_types(vec, a.y_type, a.out_type, a.k, [&](auto v, auto yt, auto ot, auto ranks) {
    return launch(combine_rows_kernel<decltype(v)::value, decltype(yt)::value, decltype(ot)::value, decltype(ranks)::value>, grid, threads, s, a);
  });
}

cudaError_t launch_combine_rows_grad(const CombineGradArgs& a, cudaStream_t s) {
  const bool vec = a.H % CHUNK == 0 && chunks(a.dout, a.ld_dout, a.dout_type) && chunks(a.y, a.ldy, a.y_type) &&
                   chunks(a.dy, a.ld_dy, a.dy_type);
  // Few tokens: a block's own latency counts; many: small blocks, whose chains of loads and sums overlap.  us by threads 128 / 256 /
  // 512 / 1024: 200 tokens of 7168, k = 8: 13 / 11 / 9.7 / 12; 2048: 81 / 78 / 77 / 87; 8192 of 4096, k = 2: 52 / 54 / 72 / 72.
  const int threads = warps_of(vec ? a.H / CHUNK : a.H, a.T <= 304 ? 512 : a.k <= 2 ? 128 : 256);
  const dim3 grid((unsigned)a.T);
  return by_types(vec, a.dout_type, a.y_type, a.k, [&](auto v, auto dt, auto yt, auto ranks) {
    return launch(combine_grad_kernel<decltype(v)::value, decltype(dt)::value, decltype(yt)::value, decltype(ranks)::value>, grid, threads, s, a);
  });
}

}  // namespace moe
