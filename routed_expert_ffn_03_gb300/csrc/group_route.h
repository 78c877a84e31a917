// group_route.h - arguments and launcher of the batch routing kernels (internal).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

namespace moe {

struct GroupRouteArgs {
  const void* logits;
  long long ld;
  int dtype, T, E, k, kind;
  int* idx;
  float* weights;
  int *offsets, *rows, *pairs;
  int* hist;               // pairs by expert: of each cluster of blocks, then of a cluster's blocks before each
  int blocks, per_block;   // tokens per block
};
struct GroupRoutePlan {
  int blocks, per_block;
  size_t workspace;        // bytes of hist
};
GroupRoutePlan group_route_plan(int T, int E, int k);
cudaError_t launch_group_route(const GroupRouteArgs& a, cudaStream_t s);
cudaError_t group_route_set_attributes();

// The selection with a bias for balance, limited to groups of experts.
struct BalancedRouteArgs : GroupRouteArgs {
  bool top2, renorm;   // top2: a group's score is the sum of its two largest, not its largest
  const float* bias;   // [E] or null
  int groups, keep;
  float factor;
  int* places;         // [T][k]
};
cudaError_t launch_balanced_route(const BalancedRouteArgs& a, cudaStream_t s);
cudaError_t balanced_route_set_attributes();

// Gradient of its weights by the logits.
struct RouteGradArgs {
  const float* dweights;   // [T][k]
  const void* logits;
  const int* idx;          // [T][k]
  void* dlogits;
  long long ld, ldd;
  int dtype, out_type, T, E, k, kind;
  bool renorm;
  float factor;
};
cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t s);

}  // namespace moe
