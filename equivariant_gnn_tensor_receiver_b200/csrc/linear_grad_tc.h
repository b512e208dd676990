// Weight gradient of the typed linear map on the tensor cores (linear_grad_tc.cu).
#pragma once

#include "linear.h"

namespace tpc {

constexpr int kLinGradTcEntries = 48;  // (path, channel tile) pairs of a call

// whether the (path, channel tile) pairs of a plan fit; whether the chunks of a call do as well
bool linear_grad_tc_plan(const LinPath* path, int n);
bool linear_grad_tc_supported(const LinPath* path, int n, int T, int64_t N);
// bytes of the partial tiles of a call
size_t linear_grad_tc_bytes(const LinPath* path, int n, int T, int64_t N);
// dW (and zeros for empty types); split = 3xTF32, else one TF32 pass; after: the same call's
// row product is the last work on the stream (see chain.cuh).  Two launches.
cudaError_t linear_grad_tc(const LinGrad& G, bool split, float* part, uint64_t limit, bool after, cudaStream_t st);
// first code recorded by an expired wait since the last read (0 = none); clears it
cudaError_t linear_grad_tc_read_error(int* code);

}  // namespace tpc
