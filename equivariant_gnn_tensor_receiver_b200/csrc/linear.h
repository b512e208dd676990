// Typed linear map: what the host plan and its kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tpconv.h"

namespace tpc {

constexpr int kLinBlocks = 12;             // blocks of an irreps string (plan.h)
constexpr int kLinPaths = 48;              // pairs of blocks (paths of a plan)
constexpr int kLinSources = 2 * kLinPaths; // with two operand pairs (double backward)

// One product of rows: out block `o` collects its sources
//   out[n, ooff + w d + m] = sum_s sum_k  x_s[n, off_s + k d + m] * B_s[type(n)][k][w],
//   B_s[k][w] = W_s[woff_s + k rk + w rw]   (a path's block or its transpose)
struct LinSource {
  int off;      // first column of the source block in its rows
  int k;        // channels
  int64_t woff; // weight block
  int rk, rw;   // strides of k and of the output channel
  int pair;     // 0: (x0, w0), 1: (x1, w1)
};
struct LinOut {
  int off, n, d;      // first column, channels, 2l+1
  int first, count;   // sources
};
struct LinRows {
  int n_out, n_src, T;
  int64_t N;
  int64_t wnumel;          // weights of one type
  int dim_src, dim_out;    // floats of a source row and of an output row
  const float *x[2], *w[2];
  float* out;
  const int *perm, *offsets;
  LinOut o[kLinBlocks];
  LinSource s[kLinSources];
};

// One weight gradient: dW[t][woff + u cout + w] = sum_{n in t, m} x[n, xoff + u d + m] g[n, goff + w d + m]
struct LinPath {
  int d, ci, co, xoff, goff;
  int i1, i3;
  int64_t woff;
};
struct LinGrad {
  int n_paths, T;
  int64_t N;
  int64_t wnumel;
  int dim_x, dim_g;
  const float *x, *g;
  float* dw;
  const int *perm, *offsets;
  LinPath p[kLinPaths];
};

// Tiles of `unit` nodes that n >= 0 nodes make.  (Unsigned: n + unit - 1 passes 2^31 for the largest graphs.)
__host__ __device__ constexpr int units_of(int n, int unit) {
  return int((unsigned(n) + unsigned(unit) - 1) / unsigned(unit));
}
static_assert(units_of(0x7fffffff, 120) == 17895698 && units_of(0x7fffffff, 0x7fffffff) == 1 && units_of(0, 9) == 0 &&
                  units_of(9, 9) == 1 && units_of(10, 9) == 2,
              "N goes up to 2^31 - 1");

// the nodes [b, e) of group t in perm; t == T is the group without a type
__device__ __forceinline__ void lin_group(const int* offsets, int T, int64_t N, int t, int* b, int* e) {
  const int n = int(N);
  const int lo = min(max(offsets[t], 0), n);
  *b = lo;
  *e = t < T ? min(max(offsets[t + 1], lo), n) : n;
}

}  // namespace tpc
