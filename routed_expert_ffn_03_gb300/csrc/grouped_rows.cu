// grouped_rows.cu - the rows that a grouped product names by number, side by side.
//
// dst row i = src row rows[i] (zeros for a number outside the source), for the sorted rows of the groups only.  One
// pass over 16-byte words, 4 in flight a thread; bound: memory (2 x the rows' bytes; 2002 rows of 4096 in 10 us, mostly in L2).
#include "common.cuh"
#include "grouped.h"

namespace moe {

namespace {

constexpr int RC_THREADS = 256;
constexpr int RC_UNROLL = 4;

__global__ void __launch_bounds__(RC_THREADS) copy_rows_kernel(RowCopy c) {
  pdl_launch_dependents();   // its wait still covers this kernel's writes
  const long long lo = min(max((long long)__ldg(c.offsets), 0ll), c.m);
  const long long hi = min(max((long long)__ldg(c.offsets + c.groups), lo), c.m);
  const int words = c.ld_dst / 8;                     // 16-byte words of a row (its last one padded with zeros)
  const long long total = (hi - lo) * words, step = (long long)gridDim.x * RC_THREADS;
  for (long long i0 = (long long)blockIdx.x * RC_THREADS + threadIdx.x; i0 < total; i0 += RC_UNROLL * step) {
    uint4 v[RC_UNROLL];
    long long at[RC_UNROLL];
#pragma unroll
    for (int q = 0; q < RC_UNROLL; ++q) {
      const long long i = i0 + q * step;
      v[q] = make_uint4(0, 0, 0, 0);
      at[q] = -1;
      if (i < total) {
        const long long r = lo + i / words;
        const int w = (int)(i % words);
        const long long src = __ldg(c.rows + r);
        at[q] = r * words + w;
        // a word that reaches past the row's end stays inside the row's pitch, or the last row's allocation ends
        // with it: then only what is there is read
        if (src >= 0 && src < c.nrows) {
          const uint16_t* s = c.src + src * c.ld_src + w * 8;
          if (w * 8 + 8 <= c.len) v[q] = __ldg(reinterpret_cast<const uint4*>(s));
          else {
            uint16_t* h = reinterpret_cast<uint16_t*>(&v[q]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (w * 8 + j < c.len) h[j] = __ldg(s + j);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < RC_UNROLL; ++q)
      if (at[q] >= 0) reinterpret_cast<uint4*>(c.dst)[at[q]] = v[q];
  }
}

}  // namespace

cudaError_t launch_copy_rows(const RowCopy& c, int num_sms, cudaStream_t s) {
  const long long words = c.m * (c.ld_dst / 8), per = RC_THREADS * RC_UNROLL;
  long long blocks = (words + per - 1) / per;
  if (blocks > 8ll * num_sms) blocks = 8ll * num_sms;
  copy_rows_kernel<<<(unsigned)blocks, RC_THREADS, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace moe
