// Typed linear map of irreps features and its gradients: plan, C entry points and
// the kernels of the FP32 pipes (sm_100a).
//
//   out[n, i3, w, m] = sum_{p -> i3} sum_u W[type n][p][u][w] x[n, i1, u, m]
// is, per type and output block, a product of the (node, m) rows of that type with
// a small matrix: matrix products grouped by type, of ragged sizes.  dx is the same
// with the transposed blocks, dW[t] = sum over the rows of t of x^T g.  The double
// backward is made of the same two (the map is bilinear): d_g = lin(gg_x, W) +
// lin(x, gg_W) in one pass over two operand pairs, d_x = lin^T(g, gg_W),
// d_W = wgrad(gg_x, g).
//
// The group sizes live on the device (offsets), so the host launches an upper bound
// of row tiles and every CTA finds its type in the offsets; nothing is copied back.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "chain.cuh"
#include "irreps.h"
#include "linear_grad_tc.h"
#include "linear_tc.h"
#include "node_ops.h"

namespace tpc {
namespace {

constexpr int kTR = 64, kTC = 64, kTK = 16;  // tile of the FP32 kernels: rows, columns, depth

// Finds tile `tile` among the groups' tiles of `unit` nodes: its group, first node
// and node count (0: no such tile).  One warp; every lane returns the same.
__device__ __forceinline__ void find_tile(const int* offsets, int T, int64_t N, int groups, int unit, int tile, int* t,
                                          int* first, int* count) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  *t = 0, *first = 0, *count = 0;
  for (int t0 = 0; t0 < groups; t0 += 32) {
    const int k = t0 + lane;
    int b = 0, e = 0;
    if (k < groups) lin_group(offsets, T, N, k, &b, &e);
    // (units_of, with a signed division: the rows kernel gets 48 registers by it and not 40, and takes
    // 36 and not 40 us at 4096 nodes of 64x0e+64x1o+64x2e)
    const int q = (e - b) / unit, n = q + (q * unit < e - b);
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    const int lo = carry + s - n;
    const unsigned hit = __ballot_sync(0xffffffffu, tile >= lo && tile < lo + n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int base = __shfl_sync(0xffffffffu, b + (tile - lo) * unit, src);
      *t = t0 + src;
      *first = base;
      *count = min(unit, __shfl_sync(0xffffffffu, e, src) - base);
      return;
    }
    carry += __shfl_sync(0xffffffffu, s, 31);
  }
}

// ---- rows: out = x W ------------------------------------------------------------
// CTA: 64 (node, m) rows of one type x 64 output channels, depth 16 a step, a 4 x 4
// register tile per thread (FP32 pipes; bound by shared-memory reads and FFMA).
__global__ void __launch_bounds__(256) k_linear_rows(const __grid_constant__ LinRows P, int colt) {
  __shared__ float sa[kTK][kTR + 4], sb[kTK][kTC + 4];
  __shared__ int s_t, s_first, s_count;
  __shared__ int s_node[kTR];
  const LinOut& O = P.o[blockIdx.y / colt];
  const int c0 = (blockIdx.y % colt) * kTC;
  if (c0 >= O.n) return;
  const int d = O.d, unit = kTR / d;  // whole nodes only
  if (threadIdx.x < 32) {
    int t, f, c;
    find_tile(P.offsets, P.T, P.N, P.T + 1, unit, blockIdx.x, &t, &f, &c);
    if (threadIdx.x == 0) s_t = t, s_first = f, s_count = c;
  }
  __syncthreads();
  const int t = s_t, count = s_count;
  if (count <= 0) return;
  if (threadIdx.x < kTR) {
    int n = -1;
    if (int(threadIdx.x) < count) {
      n = P.perm[s_first + threadIdx.x];
      if (n < 0 || n >= P.N) n = -1;
    }
    s_node[threadIdx.x] = n;
  }
  __syncthreads();
  const int rows = count * d;
  float acc[4][4] = {};
  const int tr = (threadIdx.x / 16) * 4, tc = (threadIdx.x % 16) * 4;
  if (t < P.T) {
    for (int s = 0; s < O.count; ++s) {
      const LinSource& S = P.s[O.first + s];
      const float* x = P.x[S.pair];
      const float* w = P.w[S.pair] + int64_t(t) * P.wnumel + S.woff;
      for (int k0 = 0; k0 < S.k; k0 += kTK) {
        // a node's 16 x d floats are contiguous
        for (int i = threadIdx.x; i < unit * d * kTK; i += 256) {
          const int q = i / (d * kTK), j = i % (d * kTK), k = j / d, m = j % d;
          const int n = s_node[q];
          sa[k][q * d + m] = (n >= 0 && k0 + k < S.k) ? x[int64_t(n) * P.dim_src + S.off + (k0 + k) * d + m] : 0.f;
        }
        for (int i = threadIdx.x; i < kTK * kTC; i += 256) {
          // the faster index follows the weight's unit stride
          const int k = S.rw == 1 ? i / kTC : i % kTK, c = S.rw == 1 ? i % kTC : i / kTK;
          sb[k][c] = (k0 + k < S.k && c0 + c < O.n) ? w[int64_t(k0 + k) * S.rk + int64_t(c0 + c) * S.rw] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTK; ++k) {
          float a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = sa[k][tr + i], b[i] = sb[k][tc + i];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * b[j];
        }
        __syncthreads();
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tr + i;
    if (r >= rows) continue;
    const int n = s_node[r / d], m = r % d;
    if (n < 0) continue;
    float* o = P.out + int64_t(n) * P.dim_out + O.off + m;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + tc + j < O.n) o[int64_t(c0 + tc + j) * d] = acc[i][j];
  }
}

// ---- weight gradient: per type and path, x^T g over the type's rows ----------------
// The nodes of a type are cut into pieces of `unit`; CTA (piece, path tile) adds the
// piece's rows into a 64 x 64 tile and stores it as the piece's partial.  The reduce
// kernel adds a type's pieces in order.
// A piece of a wide plan, or of a plan of few tiles, has any number of rows, and one FP32
// chain over them loses 1.5e-5 of the sum at 262144 rows.  So a chain ends after kChain rows
// and is added to the piece's partial, which is this CTA's alone: roundings of 256 + rows / 256
// additions in a row, 1e-6 at 262144 rows.  Measured (dweight, device; in brackets one chain):
// 8192 nodes of 512x l <= 2 2.22 ms (2.25), 65536 of 64x l <= 2 750 us (722), 100000 of 1024x0e
// 17.7 ms (14.2: 48 registers hold five CTAs on an SM, 40 held six, and its 768 CTAs in one
// wave).  The second sums in registers: 80 of them, 2.79 ms for the first; in shared memory,
// with their errors carried along: 2.40 ms.
constexpr int kChain = 256;
static_assert(kChain % kTK == 0, "whole steps");
__global__ void __launch_bounds__(256) k_linear_grad(const __grid_constant__ LinGrad P, int unit, int tiles_u,
                                                     int tiles_w, float* __restrict__ part) {
  __shared__ float sa[kTK][kTR + 4], sb[kTK][kTC + 4];
  __shared__ int s_first, s_count;
  chain_next();
  const int per = tiles_u * tiles_w;
  const LinPath& Q = P.p[blockIdx.y / per];
  const int u0 = ((blockIdx.y % per) / tiles_w) * kTR, w0 = ((blockIdx.y % per) % tiles_w) * kTC;
  if (u0 >= Q.ci || w0 >= Q.co) return;
  if (threadIdx.x < 32) {
    int t, f, c;
    find_tile(P.offsets, P.T, P.N, P.T, unit, blockIdx.x, &t, &f, &c);
    if (threadIdx.x == 0) s_first = f, s_count = c;
  }
  __syncthreads();
  const int count = s_count, first = s_first;
  if (count <= 0) return;
  const int d = Q.d, rows = count * d;
  float acc[4][4] = {};
  const int tr = (threadIdx.x / 16) * 4, tc = (threadIdx.x % 16) * 4;
  float* o = part + int64_t(blockIdx.x) * P.wnumel + Q.woff;
  for (int r0 = 0; r0 < rows; r0 += kTK) {
    for (int i = threadIdx.x; i < kTK * kTR; i += 256) {
      const int k = i / kTR, c = i % kTR, r = r0 + k;
      float a = 0.f, b = 0.f;
      if (r < rows) {
        const int n = P.perm[first + r / d], m = r % d;
        if (n >= 0 && n < P.N) {
          if (u0 + c < Q.ci) a = P.x[int64_t(n) * P.dim_x + Q.xoff + int64_t(u0 + c) * d + m];
          if (w0 + c < Q.co) b = P.g[int64_t(n) * P.dim_g + Q.goff + int64_t(w0 + c) * d + m];
        }
      }
      sa[k][c] = a;
      sb[k][c] = b;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = sa[k][tr + i], b[i] = sb[k][tc + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * b[j];
    }
    __syncthreads();
    if ((r0 + kTK) % kChain != 0 && r0 + kTK < rows) continue;
    int co = Q.co;
    asm volatile("" : "+r"(co));  // (or 16 addresses are kept through the loop: 62 registers, not 48)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (u0 + tr + i < Q.ci && w0 + tc + j < co) {
          float* to = o + int64_t(u0 + tr + i) * co + w0 + tc + j;
          *to = r0 >= kChain ? *to + acc[i][j] : acc[i][j];
        }
        acc[i][j] = 0.f;
      }
  }
}

// dW[t][i] = sum of part[piece][i] over the pieces of type t = blockIdx.y, in order.  (Groups
// that overlap, from offsets that do not ascend, would have more than the workspace's pieces.)
__global__ void __launch_bounds__(256) k_linear_grad_reduce(const __grid_constant__ LinGrad P, int unit, int pieces,
                                                            const float* part) {
  __shared__ int s_lo, s_n;
  const int t = blockIdx.y;
  if (threadIdx.x < 32) {
    int before = 0, n = 0;
    for (int k = threadIdx.x; k <= t; k += 32) {
      int b, e;
      lin_group(P.offsets, P.T, P.N, k, &b, &e);
      const int c = units_of(e - b, unit);
      if (k < t) before += c;
      else n = c;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x == 0) s_lo = min(before, pieces), s_n = min(n, pieces - s_lo);
  }
  __syncthreads();
  chain_wait();
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < P.wnumel; i += 256LL * gridDim.x) {
    float s = 0.f;
    for (int k = 0; k < s_n; ++k) s += part[int64_t(s_lo + k) * P.wnumel + i];
    P.dw[int64_t(t) * P.wnumel + i] = s;
  }
}

// tiles of `unit` nodes over `groups` ragged groups of N nodes: an upper bound
int64_t tile_bound(int64_t N, int groups, int unit) { return N / unit + std::min<int64_t>(groups, N); }

constexpr int kSMs = 148;

}  // namespace
}  // namespace tpc

using namespace tpc;

struct tpconv_linear {
  int T, gemm;
  int n_in, n_out;
  int in_l[kLinBlocks], in_p[kLinBlocks], in_mul[kLinBlocks], in_off[kLinBlocks];
  int out_l[kLinBlocks], out_p[kLinBlocks], out_mul[kLinBlocks], out_off[kLinBlocks];
  int dim_in, dim_out, n_paths;
  int64_t wnumel;
  LinPath path[kLinPaths];
};

namespace {

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// pieces of the FP32 weight gradient: enough to fill the GPU about twice; nodes of a piece
int64_t grad_pieces(const tpconv_linear* p) {
  int cu = 1, cw = 1;
  for (int i = 0; i < p->n_paths; ++i) {
    cu = std::max(cu, ceil_div(p->path[i].ci, kTR));
    cw = std::max(cw, ceil_div(p->path[i].co, kTC));
  }
  return std::max<int64_t>(1, 2 * kSMs / std::max(1, p->n_paths * cu * cw));
}
int grad_unit(const tpconv_linear* p, int64_t N) {
  const int64_t want = grad_pieces(p);
  return int(std::max<int64_t>(16, (N + want - 1) / want));
}
// its partials for up to N nodes (tile_bound(n, T, grad_unit(p, n)) is within this for every n <= N)
size_t grad_partials(const tpconv_linear* p, int64_t N) {
  return size_t(std::min(N / 16, grad_pieces(p)) + std::min<int64_t>(p->T, N)) * size_t(p->wnumel) * 4;
}

// the row product of `transposed` (dx, d_x) or plain (out, d_g) blocks with one or two operand pairs
void fill_rows(const tpconv_linear* p, bool transposed, int pairs, LinRows* R) {
  std::memset(R, 0, sizeof(*R));
  R->T = p->T;
  R->wnumel = p->wnumel;
  R->n_out = transposed ? p->n_in : p->n_out;
  R->dim_src = transposed ? p->dim_out : p->dim_in;
  R->dim_out = transposed ? p->dim_in : p->dim_out;
  for (int b = 0; b < R->n_out; ++b) {
    LinOut& o = R->o[b];
    o.off = transposed ? p->in_off[b] : p->out_off[b];
    o.n = transposed ? p->in_mul[b] : p->out_mul[b];
    o.d = 2 * (transposed ? p->in_l[b] : p->out_l[b]) + 1;
    o.first = R->n_src;
    for (int q = 0; q < pairs; ++q)
      for (int i = 0; i < p->n_paths; ++i) {
        const LinPath& a = p->path[i];
        if ((transposed ? a.i1 : a.i3) != b) continue;
        LinSource& s = R->s[R->n_src++];
        s.off = transposed ? a.goff : a.xoff;
        s.k = transposed ? a.co : a.ci;
        s.woff = a.woff;
        s.rk = transposed ? 1 : a.co;
        s.rw = transposed ? a.co : 1;
        s.pair = q;
      }
    o.count = R->n_src - o.first;
  }
}

// multiply-adds of one pass over all paths, in millions
double mega_macs(const tpconv_linear* p, int64_t N) {
  double m = 0;
  for (int i = 0; i < p->n_paths; ++i) m += double(p->path[i].ci) * p->path[i].co * p->path[i].d;
  return m * 1e-6 * double(N);
}

// The weight gradient's small calls run on the FP32 pipes, as the rows' do.  Measured, FP32 /
// tensor cores in us: 64x0e+64x1o+64x2e, 64 nodes 14.4 / 16.5, 512 nodes 18.5 / 19.1 (8 types)
// and 18.5 / 22.6 (one); 128 channels up to l = 3, 32 nodes 16.5 / 18.5, 512 nodes 43 / 27.
// Up to how many nodes a call is small:
int64_t grad_small(const tpconv_linear* p) { return int64_t(std::min(512.0, 20 / std::max(mega_macs(p, 1), 1e-6))); }
// whether a call's weight gradient runs on the tensor cores
bool grad_on_tc(const tpconv_linear* p, int64_t N) {
  return p->gemm != TPCONV_GEMM_SIMT && N > grad_small(p) && linear_grad_tc_supported(p->path, p->n_paths, p->T, N);
}

// Whether a call's products are chained (chain.cuh).  Its tensor-core kernels take a whole SM
// for each CTA: chained, the next one's preparation hides in the tail of the one before; for
// more rows its early CTAs cost more than that.  Backward with 8 types, apart and chained in
// us: 64x0e+64x1o+64x2e, 4096 nodes 47 / 43, 8192 nodes 57 / 53, 16384 nodes 83 / 86, 262144
// nodes 599 / 809; 128x up to l = 3, 4096 nodes 98 / 100, 8192 nodes 151 / 151.  (The join
// of partial tiles, of small CTAs, is always chained.)
bool chained(const tpconv_linear* p, int64_t N) { return N * std::max(p->dim_in, p->dim_out) <= 5000000; }

// Small products run on the FP32 pipes whatever the mode (and are no less exact): the
// tensor-core kernel takes 8 to 9 us before its first tile is stored.  Measured, FP32 /
// tensor cores in us: 8 channels, 64 to 4096 nodes 8.3 / 12.4; 32 channels, 512 nodes
// 10.3 / 12.4, 1024 nodes 13 / 12.4; 64 channels, 32 nodes 18.4 / 12.3 (its depth is
// walked 16 channels a step).
// after, more: a kernel of the same call was the last work on the stream, another one follows.
cudaError_t rows_product(const tpconv_linear* p, const LinRows& R, NodePhase& ph, bool after, bool more,
                         cudaStream_t st) {
  int depth = 0;  // most channels that an output block sums over
  for (int b = 0; b < R.n_out; ++b) {
    int k = 0;
    for (int s = 0; s < R.o[b].count; ++s) k += R.s[R.o[b].first + s].k;
    depth = std::max(depth, k);
  }
  const bool small = depth <= 32 && mega_macs(p, R.N) <= 5;
  const int tc = p->gemm != TPCONV_GEMM_SIMT && !small ? linear_tc_launches(R) : 0;
  if (tc > 0) {
    ph.note(tc);
    return linear_tc_rows(R, p->gemm == TPCONV_GEMM_FP32, device_wait_limit(), after, more, st);
  }
  int colt = 1, dmax = 1;
  for (int b = 0; b < R.n_out; ++b) {
    colt = std::max(colt, ceil_div(R.o[b].n, kTC));
    dmax = std::max(dmax, R.o[b].d);
  }
  const int64_t tiles = tile_bound(R.N, R.T + 1, kTR / dmax);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  k_linear_rows<<<dim3(unsigned(tiles), unsigned(R.n_out * colt)), 256, 0, st>>>(R, colt);
  ph.note(1);
  return cudaGetLastError();
}

cudaError_t weight_gradient(const tpconv_linear* p, int64_t N, const int* perm, const int* offsets, const float* x,
                            const float* g, float* dw, float* part, NodePhase& ph, bool after,
                            cudaStream_t st) {
  if (p->wnumel == 0) return cudaSuccess;
  LinGrad G;
  std::memset(&G, 0, sizeof(G));
  G.n_paths = p->n_paths, G.T = p->T, G.N = N, G.wnumel = p->wnumel;
  G.dim_x = p->dim_in, G.dim_g = p->dim_out;
  G.x = x, G.g = g, G.dw = dw, G.perm = perm, G.offsets = offsets;
  std::copy(p->path, p->path + p->n_paths, G.p);
  if (grad_on_tc(p, N)) {
    ph.note(2);
    return linear_grad_tc(G, p->gemm == TPCONV_GEMM_FP32, part, device_wait_limit(), after, st);
  }
  int cu = 1, cw = 1;
  for (int i = 0; i < p->n_paths; ++i) {
    cu = std::max(cu, ceil_div(G.p[i].ci, kTR));
    cw = std::max(cw, ceil_div(G.p[i].co, kTC));
  }
  const int unit = grad_unit(p, N);
  const int64_t pieces = tile_bound(N, p->T, unit);
  const int64_t ny = int64_t(p->n_paths) * cu * cw;
  if (ny > 65535) return cudaErrorInvalidValue;
  k_linear_grad<<<dim3(unsigned(pieces), unsigned(ny)), 256, 0, st>>>(G, unit, cu, cw, part);
  cudaError_t e = cudaGetLastError();
  if (e) return e;
  const unsigned bx = unsigned(std::min<int64_t>((p->wnumel + 255) / 256, 1024));
  ph.note(2);
  return chain_launch(k_linear_grad_reduce, dim3(bx, unsigned(p->T)), 256, 0, st, G, unit, int(pieces),
                      static_cast<const float*>(part));
}

size_t ws_bytes(const tpconv_linear* p, int op, int64_t N) {
  if (op == TPCONV_OP_FORWARD || N == 0 || p->wnumel == 0) return 0;
  // of the kernel that the call runs; a workspace for N nodes holds for fewer, small calls included
  const bool tc = p->gemm != TPCONV_GEMM_SIMT && N > grad_small(p) && linear_grad_tc_plan(p->path, p->n_paths);
  const size_t fp32 = grad_partials(p, tc && grad_on_tc(p, N) ? grad_small(p) : N);
  return (std::max(fp32, tc ? linear_grad_tc_bytes(p->path, p->n_paths, p->T, N) : 0) + 255) & ~size_t(255);
}

bool floats_ok(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (q && misaligned(q, 4)) return false;
  return true;
}

int check_call(const tpconv_linear* p, int64_t N, const int* perm, const int* offsets, size_t need, const void* ws,
               size_t ws_n) {
  if (!p || N < 0 || N >= (int64_t(1) << 31)) return TPCONV_ERR_INVALID_ARG;
  if (N > 0 && (!perm || !offsets)) return TPCONV_ERR_INVALID_ARG;
  if (misaligned(perm, 4) || misaligned(offsets, 4)) return TPCONV_ERR_INVALID_ARG;
  if (ws_n < need) return TPCONV_ERR_WORKSPACE_TOO_SMALL;
  if (need && (!ws || misaligned(ws, 256))) return TPCONV_ERR_INVALID_ARG;
  return TPCONV_OK;
}
int status_of(cudaError_t e) { return e == cudaSuccess ? TPCONV_OK : TPCONV_ERR_CUDA; }

int create(tpconv_linear** out, const char* irreps_in, const char* irreps_out, int n_types, int gemm) {
  std::vector<Blk> bi, bo;
  int st = parse_irreps(irreps_in, bi);
  if (!st) st = parse_irreps(irreps_out, bo);
  if (st) return st;
  if (bi.size() > size_t(kLinBlocks) || bo.size() > size_t(kLinBlocks)) return TPCONV_ERR_UNSUPPORTED;
  tpconv_linear* p = new (std::nothrow) tpconv_linear();
  if (!p) return TPCONV_ERR_INTERNAL;
  std::memset(p, 0, sizeof(*p));
  p->T = n_types;
  p->gemm = gemm;
  p->n_in = int(bi.size());
  p->n_out = int(bo.size());
  for (int i = 0; i < p->n_in; ++i) {
    p->in_l[i] = bi[i].l, p->in_p[i] = bi[i].p, p->in_mul[i] = bi[i].mul, p->in_off[i] = p->dim_in;
    p->dim_in += bi[i].mul * (2 * bi[i].l + 1);
  }
  for (int i = 0; i < p->n_out; ++i) {
    p->out_l[i] = bo[i].l, p->out_p[i] = bo[i].p, p->out_mul[i] = bo[i].mul, p->out_off[i] = p->dim_out;
    p->dim_out += bo[i].mul * (2 * bo[i].l + 1);
  }
  for (int o = 0; o < p->n_out; ++o)
    for (int i = 0; i < p->n_in; ++i) {
      if (bi[i].l != bo[o].l || bi[i].p != bo[o].p) continue;
      if (p->n_paths >= kLinPaths) {
        delete p;
        return TPCONV_ERR_UNSUPPORTED;
      }
      LinPath& q = p->path[p->n_paths++];
      q.d = 2 * bi[i].l + 1, q.ci = bi[i].mul, q.co = bo[o].mul;
      q.xoff = p->in_off[i], q.goff = p->out_off[o], q.i1 = i, q.i3 = o;
      q.woff = p->wnumel;
      p->wnumel += int64_t(q.ci) * q.co;
    }
  // channels of a block: column tiles of a launch stay within the grid's limit
  for (int i = 0; i < p->n_in; ++i)
    if (p->in_mul[i] > 8192) st = TPCONV_ERR_UNSUPPORTED;
  for (int o = 0; o < p->n_out; ++o)
    if (p->out_mul[o] > 8192) st = TPCONV_ERR_UNSUPPORTED;
  int cu = 1, cw = 1;
  for (int i = 0; i < p->n_paths; ++i) {
    cu = std::max(cu, ceil_div(p->path[i].ci, kTR));
    cw = std::max(cw, ceil_div(p->path[i].co, kTC));
  }
  if (int64_t(p->n_paths) * cu * cw > 65535) st = TPCONV_ERR_UNSUPPORTED;
  if (st) {
    delete p;
    return st;
  }
  *out = p;
  return TPCONV_OK;
}

}  // namespace

extern "C" {

int tpconv_linear_create(tpconv_linear** out, const char* irreps_in, const char* irreps_out, int n_types, int gemm) {
  if (!out) return TPCONV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!irreps_in || !irreps_out || n_types < 1) return TPCONV_ERR_INVALID_ARG;
  if (n_types > TPCONV_MAX_TYPES) return TPCONV_ERR_UNSUPPORTED;
  if (gemm < TPCONV_GEMM_FP32 || gemm > TPCONV_GEMM_SIMT) return TPCONV_ERR_INVALID_ARG;
  if (gemm == 2) return TPCONV_ERR_UNSUPPORTED;  // no half-precision operand mode, as for tpconv_plan_create
  try {
    return create(out, irreps_in, irreps_out, n_types, gemm);
  } catch (...) {
    return TPCONV_ERR_INTERNAL;
  }
}

int tpconv_linear_destroy(tpconv_linear* plan) {
  delete plan;
  return TPCONV_OK;
}

int tpconv_linear_info(const tpconv_linear* plan, int* n_paths, int* dim_in, int* dim_out, int* n_types,
                       size_t* weight_numel) {
  if (!plan) return TPCONV_ERR_INVALID_ARG;
  if (n_paths) *n_paths = plan->n_paths;
  if (dim_in) *dim_in = plan->dim_in;
  if (dim_out) *dim_out = plan->dim_out;
  if (n_types) *n_types = plan->T;
  if (weight_numel) *weight_numel = size_t(plan->wnumel);
  return TPCONV_OK;
}

int tpconv_linear_path(const tpconv_linear* plan, int i, int* l, int* c_in, int* c_out, int* in_block, int* out_block,
                       size_t* weight_offset) {
  if (!plan || i < 0 || i >= plan->n_paths) return TPCONV_ERR_INVALID_ARG;
  const LinPath& q = plan->path[i];
  if (l) *l = (q.d - 1) / 2;
  if (c_in) *c_in = q.ci;
  if (c_out) *c_out = q.co;
  if (in_block) *in_block = q.i1;
  if (out_block) *out_block = q.i3;
  if (weight_offset) *weight_offset = size_t(q.woff);
  return TPCONV_OK;
}

int tpconv_linear_workspace_size(const tpconv_linear* plan, int op, int64_t N, size_t* bytes) {
  if (!plan || !bytes || N < 0 || N >= (int64_t(1) << 31) || op < TPCONV_OP_FORWARD || op > TPCONV_OP_DOUBLE_BACKWARD)
    return TPCONV_ERR_INVALID_ARG;
  *bytes = ws_bytes(plan, op, N);
  return TPCONV_OK;
}

int tpconv_linear_forward(const tpconv_linear* plan, int64_t N, const int32_t* perm, const int32_t* offsets,
                          const float* x, const float* weight, float* out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (!plan) return TPCONV_ERR_INVALID_ARG;
  int st = check_call(plan, N, perm, offsets, N < 0 ? 0 : ws_bytes(plan, TPCONV_OP_FORWARD, N), workspace, workspace_bytes);
  if (st) return st;
  if (N > 0 && (!x || !out || (!weight && plan->wnumel))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, out})) return TPCONV_ERR_INVALID_ARG;
  const size_t wb = size_t(plan->T) * size_t(plan->wnumel) * 4;
  const Span sp[] = {{out, size_t(N) * plan->dim_out * 4}, {x, size_t(N) * plan->dim_in * 4}, {weight, wb},
                     {perm, size_t(N) * 4}, {offsets, size_t(plan->T + 1) * 4}};
  if (overlapping(sp, 1, 5)) return TPCONV_ERR_INVALID_ARG;
  if (N == 0) return TPCONV_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NodePhase ph(TPCONV_PHASE_LINEAR, s);
  LinRows R;
  fill_rows(plan, false, 1, &R);
  R.N = N, R.x[0] = x, R.w[0] = weight, R.out = out, R.perm = perm, R.offsets = offsets;
  return status_of(rows_product(plan, R, ph, false, false, s));
}

int tpconv_linear_backward(const tpconv_linear* plan, int64_t N, const int32_t* perm, const int32_t* offsets,
                           const float* x, const float* weight, const float* g, float* dx, float* dweight,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan) return TPCONV_ERR_INVALID_ARG;
  const size_t need = (dweight && N > 0) ? ws_bytes(plan, TPCONV_OP_BACKWARD, N) : 0;
  int st = check_call(plan, N, perm, offsets, need, workspace, workspace_bytes);
  if (st) return st;
  if (N > 0 && (!g || (dx && !weight && plan->wnumel) || (dweight && !x))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, dx, dweight})) return TPCONV_ERR_INVALID_ARG;
  const size_t wb = size_t(plan->T) * size_t(plan->wnumel) * 4, rin = size_t(N) * plan->dim_in * 4;
  const Span sp[] = {{dx, rin}, {dweight, wb}, {workspace, need}, {x, rin}, {weight, wb},
                     {g, size_t(N) * plan->dim_out * 4}, {perm, size_t(N) * 4}, {offsets, size_t(plan->T + 1) * 4}};
  if (overlapping(sp, 3, 8)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) return (dweight && wb && cudaMemsetAsync(dweight, 0, wb, s)) ? TPCONV_ERR_CUDA : TPCONV_OK;
  NodePhase ph(TPCONV_PHASE_LINEAR, s);
  const bool chain = chained(plan, N);
  cudaError_t e = cudaSuccess;
  if (dx) {
    LinRows R;
    fill_rows(plan, true, 1, &R);
    R.N = N, R.x[0] = g, R.w[0] = weight, R.out = dx, R.perm = perm, R.offsets = offsets;
    e = rows_product(plan, R, ph, false, chain && dweight && plan->wnumel, s);
  }
  if (!e && dweight)
    e = weight_gradient(plan, N, perm, offsets, x, g, dweight, static_cast<float*>(workspace), ph, chain && dx, s);
  return status_of(e);
}

int tpconv_linear_double_backward(const tpconv_linear* plan, int64_t N, const int32_t* perm, const int32_t* offsets,
                                  const float* x, const float* weight, const float* g, const float* gg_x,
                                  const float* gg_weight, float* d_g, float* d_x, float* d_weight, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!plan) return TPCONV_ERR_INVALID_ARG;
  const size_t need = (d_weight && gg_x && N > 0) ? ws_bytes(plan, TPCONV_OP_DOUBLE_BACKWARD, N) : 0;
  int st = check_call(plan, N, perm, offsets, need, workspace, workspace_bytes);
  if (st) return st;
  const bool a = gg_x != nullptr, b = gg_weight != nullptr;
  if (N > 0 && ((d_g && ((a && !weight && plan->wnumel) || (b && !x))) || (!g && ((d_x && b) || (d_weight && a)))))
    return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, gg_x, gg_weight, d_g, d_x, d_weight})) return TPCONV_ERR_INVALID_ARG;
  const size_t wb = size_t(plan->T) * size_t(plan->wnumel) * 4, rin = size_t(N) * plan->dim_in * 4,
               rout = size_t(N) * plan->dim_out * 4;
  const Span sp[] = {{d_g, rout}, {d_x, rin}, {d_weight, wb}, {workspace, need}, {x, rin}, {weight, wb},
                     {g, rout}, {gg_x, rin}, {gg_weight, wb}, {perm, size_t(N) * 4}, {offsets, size_t(plan->T + 1) * 4}};
  if (overlapping(sp, 4, 11)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d_weight && wb && (N == 0 || !a) && cudaMemsetAsync(d_weight, 0, wb, s)) return TPCONV_ERR_CUDA;
  if (N == 0) return TPCONV_OK;
  NodePhase ph(TPCONV_PHASE_LINEAR, s);
  cudaError_t e = cudaSuccess;
  LinRows R;
  // products of this call, each but the last followed by another on the stream
  const bool chain = chained(plan, N);
  const bool p_g = d_g && (a || b), p_x = d_x && b, p_w = d_weight && a && plan->wnumel;
  if (d_g) {
    if (!a && !b) {
      e = cudaMemsetAsync(d_g, 0, rout, s);
    } else {
      fill_rows(plan, false, a && b ? 2 : 1, &R);
      R.N = N, R.out = d_g, R.perm = perm, R.offsets = offsets;
      R.x[0] = a ? gg_x : x, R.w[0] = a ? weight : gg_weight;
      R.x[1] = x, R.w[1] = gg_weight;
      e = rows_product(plan, R, ph, false, chain && (p_x || (p_w && !d_x)), s);
    }
  }
  if (!e && d_x) {
    if (!b) {
      e = cudaMemsetAsync(d_x, 0, rin, s);
    } else {
      fill_rows(plan, true, 1, &R);
      R.N = N, R.x[0] = g, R.w[0] = gg_weight, R.out = d_x, R.perm = perm, R.offsets = offsets;
      e = rows_product(plan, R, ph, chain && p_g, chain && p_w, s);
    }
  }
  if (!e && d_weight && a)
    e = weight_gradient(plan, N, perm, offsets, gg_x, g, d_weight, static_cast<float*>(workspace), ph,
                        chain && (p_x || (p_g && !d_x)), s);
  return status_of(e);
}

int tpconv_linear_device_status(const tpconv_linear* plan, void* stream, int* status) {
  if (!plan || !status) return TPCONV_ERR_INVALID_ARG;
  *status = TPCONV_OK;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return TPCONV_ERR_CUDA;
  int a = 0, b = 0;
  if (linear_tc_read_error(&a) != cudaSuccess || linear_grad_tc_read_error(&b) != cudaSuccess) return TPCONV_ERR_CUDA;
  if (a || b) *status = TPCONV_ERR_TIMEOUT;
  return TPCONV_OK;
}

}  // extern "C"
