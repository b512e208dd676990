// Typed linear map on the tensor cores (linear_tc.cu).
#pragma once

#include "linear.h"

namespace tpc {

constexpr int kLinTcEntries = 48;  // (output block, 64 columns) pairs of a call

// kernels that the product launches; 0: it has too many (output block, 64 columns) pairs
int linear_tc_launches(const LinRows& R);
// the row product; split = 3xTF32, else one TF32 pass; after: a kernel of the same call is
// the last work on the stream; more: another one follows (see chain.cuh)
cudaError_t linear_tc_rows(const LinRows& R, bool split, uint64_t limit, bool after, bool more, cudaStream_t st);
// first code recorded by an expired wait since the last read (0 = none); clears it
cudaError_t linear_tc_read_error(int* code);

}  // namespace tpc
