// verify.h - arguments and launcher of the draft verification kernel (internal).
#pragma once
#include <cuda_runtime.h>

namespace moe {

struct VerifyArgs {
  const void *p, *q;       // q null: one-hot drafts
  const int *draft, *lengths;
  const float* u;
  int *accepted, *tokens;
  long long p_seq, p_row, q_seq, q_row;
  int B, D, V, dtype;
};
cudaError_t verify_set_attributes();
cudaError_t launch_verify(const VerifyArgs& a, int num_sms, cudaStream_t s);

}  // namespace moe
