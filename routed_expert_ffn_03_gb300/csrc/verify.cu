// verify.cu - which drafted tokens stand, and the token drawn after them.
//
// Draft i with token t stands iff u_i q_i(t) < p_i(t); the token after the last that stands
// is drawn by inverting the running sum of max(p - q, 0) (or of p, when every draft stands).
// A probability x in [0, 1] is carried as the integer floor(x 2^60) in 64 bits, so sums are exact
// and the same in any order, and the token is the least v with cum(v) > floor(u total): an
// integer comparison, with u a 64-bit fraction.  fp32 values of 2^-36 and more lose nothing to the floor.
//
// One block per sequence: only the row that decides is read (bound: memory).
#include "common.cuh"
#include "grouped.h"
#include "verify.h"

namespace moe {

namespace {

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
typedef unsigned long long u64;

__device__ __forceinline__ float load_prob(const void* p, long long i, int dtype) {
  float x;
  if (dtype == GT_FP32) x = __ldg(static_cast<const float*>(p) + i);
  else {
    const uint16_t b = __ldg(static_cast<const uint16_t*>(p) + i);
    x = dtype == GT_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
  }
  return fminf(fmaxf(x, 0.f), 1.f);   // fmaxf(NaN, 0) = 0
}
__device__ __forceinline__ u64 fixed60(float x) { return __float2ull_rz(x * 1152921504606846976.f); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

struct Row {          // the row that decides
  const void *p, *q;  // q null: no residual
  int hot;            // one-hot draft to leave out, or -1
  int dtype;
  __device__ __forceinline__ u64 weight(int v) const {
    u64 w = fixed60(load_prob(p, v, dtype));
    if (q) {
      const u64 x = fixed60(load_prob(q, v, dtype));
      w = w > x ? w - x : 0;
    }
    return v == hot ? 0 : w;
  }
};

__global__ void __launch_bounds__(VF_THREADS) verify_kernel(VerifyArgs a) {
  __shared__ u64 part[VF_WARPS];
  __shared__ int s_token;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = a.lengths ? min(max(__ldg(a.lengths + b), 0), a.D) : a.D;
  const size_t el = a.dtype == GT_FP32 ? 4 : 2;
  const char* p = static_cast<const char*>(a.p) + (size_t)((long long)b * a.p_seq) * el;
  const char* q = a.q ? static_cast<const char*>(a.q) + (size_t)((long long)b * a.q_seq) * el : nullptr;

  // lane i: draft i (every warp alike)
  int tok = -1;
  bool stands = true;
  if (lane < L) {
    tok = __ldg(a.draft + (long long)b * a.D + lane);
    stands = false;
    if (tok >= 0 && tok < a.V) {
      const float pv = load_prob(p + (size_t)(lane * a.p_row) * el, tok, a.dtype);
      const float qv = q ? load_prob(q + (size_t)(lane * a.q_row) * el, tok, a.dtype) : 1.f;
      const float u = fminf(fmaxf(__ldg(a.u + (long long)b * (a.D + 1) + lane), 0.f), 1.f);
      stands = (double)u * (double)qv < (double)pv;   // exact: 24-bit factors
    }
  }
  const unsigned no = __ballot_sync(0xffffffffu, !stands);
  const int r = no ? __ffs(no) - 1 : L;
  const int rej = __shfl_sync(0xffffffffu, tok, r & 31);
  Row row;
  row.p = p + (size_t)(r * a.p_row) * el;
  row.q = r < L && q ? q + (size_t)(r * a.q_row) * el : nullptr;
  row.hot = r < L && !q ? rej : -1;
  row.dtype = a.dtype;

  const float uf = fminf(fmaxf(__ldg(a.u + (long long)b * (a.D + 1) + a.D), 0.f), 1.f);
  const u64 U = uf >= 1.f ? ~0ull : __float2ull_rz(uf * 18446744073709551616.f);
  const int seg = ((a.V + VF_WARPS - 1) / VF_WARPS + 31) / 32 * 32;
  const int v0 = min((long long)warp * seg, (long long)a.V), v1 = min((long long)v0 + seg, (long long)a.V);
  if (threadIdx.x == 0) s_token = -1;
  for (int pass = 0; pass < 2; ++pass) {
    u64 sum = 0;
    for (int v = v0 + lane; v < v1; v += 32) sum += row.weight(v);
    sum = warp_sum(sum);
    __syncthreads();
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    u64 total = 0, before = 0;
    for (int w = 0; w < VF_WARPS; ++w) {
      if (w == warp) before = total;
      total += part[w];
    }
    if (total) {
      const u64 thr = __umul64hi(U, total);   // floor(u total) < total
      if (before <= thr && thr < before + sum) {
        u64 run = before;
        for (int w0 = v0; w0 < v1; w0 += 32) {
          const u64 c = run + warp_scan(w0 + lane < v1 ? row.weight(w0 + lane) : 0, lane);
          const unsigned hit = __ballot_sync(0xffffffffu, c > thr);
          if (hit) {
            if (lane == 0) s_token = w0 + __ffs(hit) - 1;
            break;
          }
          run = __shfl_sync(0xffffffffu, c, 31);
        }
      }
      break;
    }
    if (!row.q && row.hot < 0) break;   // p itself is empty
    row.q = nullptr;                    // nothing left of the residual: draw from p
    row.hot = -1;
  }
  __syncthreads();
  if (threadIdx.x <= a.D) {
    const int i = threadIdx.x;
    a.tokens[(long long)b * (a.D + 1) + i] = i < r ? __ldg(a.draft + (long long)b * a.D + i) : i == r ? s_token : -1;
  }
  if (threadIdx.x == 0) a.accepted[b] = r;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  verify_kernel<<<a.B, VF_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
