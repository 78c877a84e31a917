// route_grad.cu - gradient of the routing weights by the logits.
//
// With v_j = factor dweights_j, over the selected experts e_j of a token:
//   softmax renormalised:  dl_j = r_j (v_j - sum r v),                r = softmax of the selected logits
//   sigmoid renormalised:  dl_j = (1 - s_j) r_j (v_j - sum r v),      r = s / sum s
//   sigmoid:               dl_j = v_j s_j (1 - s_j)
//   softmax over all:      dl_e = P_e ([e selected] v_e - sum_j P_j v_j)
// and 0 for the other experts.  The bias and the groups choose; no gradient passes through them.  A warp takes a token: one pass
// over its row.  Bound: memory (the result; with softmax over all the logits too).
#include "group_sort.cuh"
#include "rows_io.cuh"

namespace moe {

namespace {

constexpr int RG_WARPS = 8;

template <int NV, bool ALL>
__global__ void __launch_bounds__(32 * RG_WARPS) route_grad_kernel(const RouteGradArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * RG_WARPS + (threadIdx.x >> 5);
  if (t >= a.T) return;   // whole warps
  auto logit = [&](int e) { return clean(load_logit(a.logits, t * a.ld + e, a.dtype)); };
  int e = lane < a.k ? __ldg(a.idx + t * a.k + lane) : -1;
  if (e < 0 || e >= a.E) e = -1;
  const float v = e >= 0 ? a.factor * __ldg(a.dweights + t * a.k + lane) : 0.f;
  const float l = e >= 0 ? logit(e) : -INFINITY;
  const bool live = l > -INFINITY;
  float p[ALL ? NV : 1], d = 0.f, s = 0.f;
  if (ALL) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < (ALL ? NV : 1); ++i) {
      const int q = lane + 32 * i;
      p[i] = q < a.E ? logit(q) : -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < (ALL ? NV : 1); ++i) {
      p[i] = p[i] > -INFINITY ? expf(p[i] - m) : 0.f;
      z += p[i];
    }
    z = warp_sum(z);
    const float inv = z > 0.f ? 1.f / z : 0.f;
    const float mine = live ? expf(l - m) * inv : 0.f;
    s = warp_sum(mine * v);
    d = mine * (v - s);
    s *= inv;
  } else if (a.renorm) {
    const float z = a.kind == 1 ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
    const float z0 = warp_max(live ? z : -INFINITY), num = live ? expf(z - z0) : 0.f;
    const float den = warp_sum(num), r = live ? num / den : 0.f;
    d = r * (v - warp_sum(r * v));
    if (a.kind == 1 && live) d *= 1.f / (1.f + expf(l));
  } else if (live) {
    const float q = expf(-fabsf(l));
    d = v * (q / ((1.f + q) * (1.f + q)));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = lane + 32 * i;
    if (q < a.E) put_value(a.dlogits, t * a.ldd + q, a.out_type, ALL ? -p[ALL ? i : 0] * s : 0.f);
  }
  __syncwarp();   // the selected ones on top
  if (e >= 0) put_value(a.dlogits, t * a.ldd + e, a.out_type, d);
}

template <int NV>
cudaError_t launch_as(const RouteGradArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(((long long)a.T + RG_WARPS - 1) / RG_WARPS));
  c.blockDim = dim3(32 * RG_WARPS);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return a.kind == 0 && !a.renorm ? cudaLaunchKernelEx(&c, route_grad_kernel<NV, true>, a)
                                  : cudaLaunchKernelEx(&c, route_grad_kernel<NV, false>, a);
}

}  // namespace

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t s) {
  if (a.E <= 128) return launch_as<4>(a, s);
  if (a.E <= 256) return launch_as<8>(a, s);
  return a.E <= 512 ? launch_as<16>(a, s) : launch_as<32>(a, s);
}

}  // namespace moe
