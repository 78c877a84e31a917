// grouped.h - device arguments and launchers of the 16-bit grouped products (internal).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

enum : int { GT_BF16 = 0, GT_FP16 = 1, GT_FP32 = 2 };

// One grouped product D = A B^T per group, seen the same way by every kernel.
//   forward: A = sorted rows of x [m][k], B = W_e as n rows of k; D rows go to out rows
//   weight gradient: A = dy^T (n rows), B = x^T (k rows), contracted over the group's rows
struct GroupedProblem {
  const uint16_t* a;         // x, or dy
  const uint16_t* b;         // w, or x
  void* d;                   // out, or dw
  const int* offsets;        // [groups + 1]
  const int* a_rows;         // row numbers of a by sorted row, or null
  const int* b_rows;         // weight gradient: row numbers of b, or null
  const int* d_rows;         // forward: out rows by sorted row, or null
  long long a_nrows, lda;
  long long b_nrows, ldb, b_stride;   // b_nrows: weight gradient only; b_stride: forward only
  long long d_nrows, ldd, d_stride;   // d_nrows: forward only; d_stride: weight gradient only
  long long m;
  int groups, n, k;          // n: rows of W_e (gate and up together with swiglu)
  int dtype, out_dtype;
  int kn;                    // forward: W_e stored [k][n]
  int swiglu;
};

// Row range of group g, with offsets outside [0, m] taken as the nearer end and an end
// before its start as an empty group.
__device__ __forceinline__ void group_range(const int* offsets, int g, long long m, int& r0, int& r1) {
  const int hi = (int)m;
  r0 = min(max(__ldg(offsets + g), 0), hi);
  r1 = min(max(__ldg(offsets + g + 1), r0), hi);
}

cudaError_t launch_grouped_any(const GroupedProblem& p, bool wgrad, cudaStream_t s);

}  // namespace moe
