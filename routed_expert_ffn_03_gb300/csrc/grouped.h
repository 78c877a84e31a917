// grouped.h - device arguments and launchers of the 16-bit grouped products (internal).
#pragma once
#include <cuda.h>
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

#ifdef __CUDACC__
// Row range of group g, with offsets outside [0, m] taken as the nearer end and an end
// before its start as an empty group.
__device__ __forceinline__ void group_range(const int* offsets, int g, long long m, int& r0, int& r1) {
  const int hi = (int)m;
  r0 = min(max(__ldg(offsets + g), 0), hi);
  r1 = min(max(__ldg(offsets + g + 1), r0), hi);
}
#endif

// The bound of a kernel's waits, in SM cycles, and the host-visible word that one which runs out sets.
struct WaitLimit {
  uint32_t* status;
  unsigned long long cycles;
};

// For any strides and alignment.
cudaError_t launch_grouped_any(const GroupedProblem& p, bool wgrad, const WaitLimit& wait, cudaStream_t s);
cudaError_t grouped_any_set_attributes();

// A tensor map over elements of 2 or 4 bytes, 128-byte swizzled, zeros outside: dims and box in elements, innermost
// first; strides (of dims 1 ..) in bytes.  False where the hardware cannot address the tensor so (a base, stride or
// size it does not take).  m null: that alone is looked at, without the driver.
bool tensor_map(CUtensorMap* m, const void* base, size_t elem, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box);
// The maps of a product, 64 elements wide.  a: the first factor in tiles.  b: the second, forward in boxes of 16, 32, 64
// and 128 rows, weight gradient [0] in tiles of 64 rows; for the few-rows kernel only [0], of one row where rows are named
// by number.  d: weight gradient: the result, in boxes of 32 rows of 128 bytes (made by the launcher).
struct GroupedMaps {
  CUtensorMap a, b[4], d;
};
// False where TMA cannot take the operands as they lie.  m null: that alone is looked at, without the driver.
bool grouped_maps(const GroupedProblem& p, bool wgrad, bool few, GroupedMaps* m);

// Copy of the rows named by number: dst[i][0 .. ld_dst) = src[rows[i]][0 .. len), zeros behind len and for a number
// outside [0, nrows), for the sorted rows i that offsets cover.  src and dst 16-byte aligned, ld_src and ld_dst
// multiples of 8 elements, ld_dst >= len.
struct RowCopy {
  const uint16_t* src;
  uint16_t* dst;
  const int *rows, *offsets;
  long long nrows, ld_src, m;
  int groups, len, ld_dst;
};
cudaError_t launch_copy_rows(const RowCopy& c, int num_sms, cudaStream_t s);

// The tensor-core kernel over pairs of SMs; false (nothing launched) where TMA cannot take the operands.
bool launch_grouped_pair(const GroupedProblem& p, bool wgrad, int num_sms, const WaitLimit& wait, cudaStream_t s,
                         cudaError_t* err);
cudaError_t grouped_pair_set_attributes();

// The kernel for few rows a group, in tiles of nt = 16, 32 or 64 rows, `cluster` (1, 2, 4, 8) blocks to a tile; forward
// products only; reads rows by number where they are.  Otherwise as launch_grouped_pair.
bool launch_grouped_few(const GroupedProblem& p, int nt, int cluster, const WaitLimit& wait, cudaStream_t s, cudaError_t* err);
cudaError_t grouped_few_set_attributes();

}  // namespace moe
