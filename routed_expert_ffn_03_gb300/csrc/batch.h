// batch.h - what the entry points of the batch operators share (internal).
#pragma once
#include "../../include/moe.h"
#include "grouped.h"

namespace moe {

// What a device needs once: kernel attributes, its SM count, and the host-visible word that a kernel whose wait ran
// out sets.  Made by the first call on the device, kept for the life of the process.  batch_device: the current
// device's, set up; MOE_ETIMEOUT once a wait ran out there.
struct BatchDevice {
  int num_sms;
  WaitLimit wait;
};
moe_status batch_device(BatchDevice* out);

inline bool is_dtype(int t, bool fp32) { return t == MOE_T_BF16 || t == MOE_T_FP16 || (fp32 && t == MOE_T_FP32); }
inline size_t dtype_bytes(int t) { return t == MOE_T_FP32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// rows of `len` elements `ld` apart that do not overlap, all of them within 2^62 bytes
inline bool rows_fit(long long rows, long long ld, long long len) {
  return rows >= 0 && ld >= len && ld < (1ll << 40) && (rows == 0 || ld <= (1ll << 60) / rows);
}

inline moe_status done(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ECUDA;
}

}  // namespace moe
