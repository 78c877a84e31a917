// grouped_rows.cu - the rows that a grouped product names by number, side by side.
//
// dst row i = src row rows[i] (zeros for a number outside the source), for the sorted rows of the groups only.  One
// pass over 16-byte words, a warp a run of 128 words of one row (a division a run, not a word), 4 in flight a thread.
// Bound: memory (2 x the rows' bytes; 2002 rows of 4096 in 3 us, mostly in L2; 6216 of 7168 in
// 17; with a division a word 11 and 29).
#include "common.cuh"
#include "grouped.h"

namespace moe {

namespace {

constexpr int RC_THREADS = 256;
constexpr int RC_RUN = 128;   // words

__global__ void __launch_bounds__(RC_THREADS) copy_rows_kernel(RowCopy c) {
  pdl_launch_dependents();   // its wait still covers this kernel's writes
  pdl_wait();
  const long long lo = min(max((long long)__ldg(c.offsets), 0ll), c.m);
  const long long hi = min(max((long long)__ldg(c.offsets + c.groups), lo), c.m);
  const int words = c.ld_dst / 8;                     // 16-byte words of a row (its last one padded with zeros)
  const int runs = (words + RC_RUN - 1) / RC_RUN, lane = threadIdx.x & 31;
  const long long total = (hi - lo) * runs, step = (long long)gridDim.x * (RC_THREADS / 32);
  for (long long i = (long long)blockIdx.x * (RC_THREADS / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const long long r = lo + (i <= 0xffffffffll ? (uint32_t)i / (uint32_t)runs : i / runs);
    const int w0 = (int)(i - (r - lo) * runs) * RC_RUN + lane;
    const long long src = __ldg(c.rows + r);
    const uint16_t* s = src >= 0 && src < c.nrows ? c.src + src * c.ld_src : nullptr;
    uint4* d = reinterpret_cast<uint4*>(c.dst) + r * words;
    uint4 v[RC_RUN / 32];
#pragma unroll
    for (int q = 0; q < RC_RUN / 32; ++q) {
      const int w = w0 + 32 * q;
      v[q] = make_uint4(0, 0, 0, 0);
      // a word that reaches past the row's end stays inside the row's pitch, or the last row's allocation ends
      // with it: then only what is there is read
      if (s && w * 8 + 8 <= c.len) {
        v[q] = __ldg(reinterpret_cast<const uint4*>(s) + w);
      } else if (s && w * 8 < c.len) {
        uint16_t* h = reinterpret_cast<uint16_t*>(&v[q]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (w * 8 + j < c.len) h[j] = __ldg(s + w * 8 + j);
      }
    }
#pragma unroll
    for (int q = 0; q < RC_RUN / 32; ++q)
      if (w0 + 32 * q < words) d[w0 + 32 * q] = v[q];
  }
}

}  // namespace

cudaError_t launch_copy_rows(const RowCopy& c, int num_sms, cudaStream_t s) {
  const long long runs = c.m * ((c.ld_dst / 8 + RC_RUN - 1) / RC_RUN), per = RC_THREADS / 32;
  long long blocks = (runs + per - 1) / per;
  if (blocks > 8ll * num_sms) blocks = 8ll * num_sms;
  cudaLaunchConfig_t l = {};
  l.gridDim = dim3((unsigned)blocks);
  l.blockDim = dim3(RC_THREADS);
  l.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  l.attrs = at;
  l.numAttrs = 1;
  return cudaLaunchKernelEx(&l, copy_rows_kernel, c);
}

}  // namespace moe
