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

}  // namespace moe
