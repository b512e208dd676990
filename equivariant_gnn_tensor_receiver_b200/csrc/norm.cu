// Layer norm of irreps features, its backward and double backward (sm_100a).
//
// Per node and block (C channels, D = 2l+1, S = C D entries):
//   xc = P x (P removes the channel mean for l = 0, identity for l > 0),
//   r = (<xc, xc> / S + eps)^-1/2,  h = r xc,  y = w h (+ b)
//   backward:  gh = w g,  dx = P r (gh - h <gh, h> / S),  dw_u = sum g h,  db_u = sum g
//   double backward of <gg_x, dx> + <gg_w, dw> + <gg_b, db>, with a = P gg_x:
//     A1 = <a, gh> / S,  A2 = <a, h> / S,  G2 = <gh, h> / S,  K = <gg_w g, h> / S,
//     t = r (a - h A2),  d_g = w t + gg_w h + gg_b,  d_w_u = sum g t,
//     d_x = P [r gg_w g - r^2 (gh A2 + a G2) - h (r^2 (A1 - 3 G2 A2) + r K)].
// The variance is that of the centred entries (a second sum over registers, not
// a difference of moments); sums and statistics are fp32.
//
// Bound: HBM.  Every pass reads each row tensor once and writes each row output
// once; a row stays in registers between the two.  A team of TL lanes owns whole
// rows, and lane i owns the same columns of every row it visits (element or
// 4-float vector i + TL j), so the per-column weights sit in shared memory once
// per CTA and the weight gradients accumulate in registers over the rows, one
// accumulator per column.  At the end the CTA adds its teams' accumulators in
// order into a partial row of the workspace, and k_norm_reduce sums the partial
// rows in a fixed order (no atomics: repeated calls agree bit for bit).
// A row's blocks are reduced together by masks on the lane's vectors, so any mix
// of blocks costs one pass.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/tpconv.h"
#include "irreps.h"
#include "node_ops.h"

namespace tpc {
namespace {

constexpr int kBlocksMax = 12;

struct NormDev {
  int nb, dim, nw, nbias;
  int off[kBlocksMax + 1];  // first column of a block; off[nb] = dim
  int d[kBlocksMax];        // 2l+1
  int woff[kBlocksMax];     // first weight of a block
  int boff[kBlocksMax];     // first bias of a block, or -1
  float inv[kBlocksMax];    // 1 / S
  float eps;
};

enum { kFwd = 0, kBwd = 1, kDbl = 2 };

struct NormArgs {
  const float *x, *w, *b, *g, *a, *al, *be;
  float *o0, *o1;   // y | dx | d_g, d_x
  float* part;      // partial rows of the weight gradients, or null
  int want_b;       // backward: partial rows of dbias too
  int64_t n;
};

template <int VEC>
struct Pack {
  float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Pack<VEC> ld(const float* p) {
  Pack<VEC> r;
  if constexpr (VEC == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    r.v[0] = q.x, r.v[1] = q.y, r.v[2] = q.z, r.v[3] = q.w;
  } else {
    r.v[0] = *p;
  }
  return r;
}
// rows are read once: streaming loads
template <int VEC>
__device__ __forceinline__ Pack<VEC> ld_row(const float* p) {
  Pack<VEC> r;
  if constexpr (VEC == 4) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(p));
    r.v[0] = q.x, r.v[1] = q.y, r.v[2] = q.z, r.v[3] = q.w;
  } else {
    r.v[0] = __ldcs(p);
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ void st_row(float* p, const Pack<VEC>& r) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
  else
    *p = r.v[0];
}

constexpr int kThreads(int TL) { return TL > 256 ? TL : (TL > 32 ? TL : 256); }

// Team sums of Q quantities per block.  val[q][j]: this lane's share of vector j
// for quantity q; on return the block's sum, in every lane that owns a vector of
// that block.  use(q, b): whether quantity q is wanted for block b (uniform).
template <int Q, int V, int TL, class Use>
__device__ __forceinline__ void block_sums(const NormDev& p, const int (&blk)[V], float (&val)[Q][V], float* red,
                                           Use use) {
  if constexpr (TL <= 32) {
    for (int b = 0; b < p.nb; ++b) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (!use(q, b)) continue;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) s += blk[j] == b ? val[q][j] : 0.f;
#pragma unroll
        for (int o = TL / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // a block's sum replaces the shares of its vectors, which no later block reads
#pragma unroll
        for (int j = 0; j < V; ++j) val[q][j] = blk[j] == b ? s : val[q][j];
      }
    }
  } else {
    constexpr int NW = TL / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* tot = red + NW * kBlocksMax * Q;
    for (int b = 0; b < p.nb; ++b) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (!use(q, b)) continue;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) s += blk[j] == b ? val[q][j] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) red[warp * (kBlocksMax * Q) + b * Q + q] = s;
      }
    }
    __syncthreads();
    if (threadIdx.x < p.nb * Q && use(int(threadIdx.x) % Q, int(threadIdx.x) / Q)) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += red[w * (kBlocksMax * Q) + threadIdx.x];
      tot[threadIdx.x] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (blk[j] >= 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (use(q, blk[j])) val[q][j] = tot[blk[j] * Q + q];
      }
  }
}

// floats of shared memory behind the column weights: reduction scratch
constexpr int kRedQ = 6;
template <int TL>
constexpr int red_floats() {
  return TL <= 32 ? 0 : (TL / 32 + 1) * kBlocksMax * kRedQ;
}

template <int MODE, int VEC, int V, int TL>
__global__ void __launch_bounds__(kThreads(TL)) k_norm(const __grid_constant__ NormDev p, const NormArgs A) {
  constexpr int TEAMS = kThreads(TL) / TL;
  constexpr int NACC = MODE == kBwd ? 2 : (MODE == kDbl ? 1 : 0);  // dw, db | d_w
  extern __shared__ float4 smem4[];
  float* sm = reinterpret_cast<float*>(smem4);
  const int dimp = (p.dim + 3) & ~3;
  float* sw = sm;                                    // weight of every column
  float* s1 = sm + dimp;                             // forward: bias; double backward: gg_w
  float* s2 = sm + 2 * dimp;                         // double backward: gg_b
  float* red = sm + (MODE == kDbl ? 3 : 2) * dimp;
  // per-column weights: block by block, so no search is needed
  for (int b = 0; b < p.nb; ++b) {
    const int d = p.d[b], n = p.off[b + 1] - p.off[b];
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int u = i / d, c = p.off[b] + i;
      sw[c] = A.w ? A.w[p.woff[b] + u] : 1.f;
      if constexpr (MODE == kFwd) s1[c] = (A.b && p.boff[b] >= 0) ? A.b[p.boff[b] + u] : 0.f;
      if constexpr (MODE == kDbl) {
        s1[c] = A.al ? A.al[p.woff[b] + u] : 0.f;
        s2[c] = (A.be && p.boff[b] >= 0) ? A.be[p.boff[b] + u] : 0.f;
      }
    }
  }
  __syncthreads();

  const int tl = threadIdx.x % TL, team = threadIdx.x / TL;
  int blk[V];       // block of vector j, -1 behind the row
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (tl + TL * j) * VEC;
    blk[j] = -1;
    if (c < p.dim)
      for (int b = 0; b < p.nb; ++b)
        if (c >= p.off[b]) blk[j] = b;
  }
  float inv[V];
  bool cen[V];  // l = 0: centred
#pragma unroll
  for (int j = 0; j < V; ++j) {
    inv[j] = blk[j] >= 0 ? p.inv[blk[j]] : 0.f;
    cen[j] = blk[j] >= 0 && p.d[blk[j]] == 1;
  }
  Pack<VEC> acc[NACC > 0 ? NACC : 1][V];
#pragma unroll
  for (int k = 0; k < (NACC > 0 ? NACC : 1); ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[k][j].v[e] = 0.f;

  // every lane runs the same number of rounds: the sums are collective
  const int64_t stride = int64_t(gridDim.x) * TEAMS;
  const int64_t rounds = (A.n + stride - 1) / stride;
  for (int64_t k = 0; k < rounds; ++k) {
    const int64_t row = k * stride + int64_t(blockIdx.x) * TEAMS + team;
    const bool on = row < A.n;
    const int64_t base = row * p.dim;
    Pack<VEC> x[V], g[MODE == kFwd ? 1 : V], a[MODE == kDbl ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (tl + TL * j) * VEC;
      const bool in = on && blk[j] >= 0;
      const Pack<VEC> zero = {};
      x[j] = in ? ld_row<VEC>(A.x + base + c) : zero;
      if constexpr (MODE != kFwd) g[j] = in ? ld_row<VEC>(A.g + base + c) : zero;
      if constexpr (MODE == kDbl) a[j] = (in && A.a) ? ld_row<VEC>(A.a + base + c) : zero;
    }
    // centre the scalars (x, and gg_x in the double backward)
    {
      constexpr int Q = MODE == kDbl ? 2 : 1;
      float s[Q][V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[0][j] = 0.f;
        if constexpr (Q == 2) s[1][j] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[0][j] += x[j].v[e];
          if constexpr (Q == 2) s[1][j] += a[j].v[e];
        }
      }
      block_sums<Q, V, TL>(p, blk, s, red, [&](int, int b) { return p.d[b] == 1; });
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[j].v[e] -= cen[j] ? s[0][j] * inv[j] : 0.f;
          if constexpr (Q == 2) a[j].v[e] -= cen[j] ? s[1][j] * inv[j] : 0.f;
        }
    }
    // x becomes h
    float r[V];
    {
      float s[1][V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[0][j] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0][j] += x[j].v[e] * x[j].v[e];
      }
      block_sums<1, V, TL>(p, blk, s, red, [](int, int) { return true; });
#pragma unroll
      for (int j = 0; j < V; ++j) {
        r[j] = 1.f / sqrtf(s[0][j] * inv[j] + p.eps);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j].v[e] *= r[j];
      }
    }
    if constexpr (MODE == kFwd) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (tl + TL * j) * VEC;
        if (!on || blk[j] < 0) continue;
        const Pack<VEC> w = ld<VEC>(sw + c), bb = ld<VEC>(s1 + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j].v[e] = w.v[e] * x[j].v[e] + bb.v[e];
        st_row<VEC>(A.o0 + base + c, x[j]);
      }
    } else if constexpr (MODE == kBwd) {
      float s[2][V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[0][j] = s[1][j] = 0.f;
        if (blk[j] < 0) continue;
        const Pack<VEC> w = ld<VEC>(sw + (tl + TL * j) * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          acc[0][j].v[e] += g[j].v[e] * x[j].v[e];
          acc[1][j].v[e] += g[j].v[e];
          g[j].v[e] = __fmul_rn(g[j].v[e], w.v[e]);  // (not fused into gh - mean: a lone scalar gives 0)
          s[0][j] += g[j].v[e] * x[j].v[e];
          s[1][j] += g[j].v[e];
        }
      }
      if (A.o0) {
        block_sums<2, V, TL>(p, blk, s, red, [&](int q, int b) { return q == 0 || p.d[b] == 1; });
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!on || blk[j] < 0) continue;
          const float c1 = s[0][j] * inv[j], mg = cen[j] ? s[1][j] * inv[j] : 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[j].v[e] = r[j] * (g[j].v[e] - mg - x[j].v[e] * c1);
          st_row<VEC>(A.o0 + base + (tl + TL * j) * VEC, x[j]);
        }
      }
    } else {
      float s[6][V];  // a.gh, a.h, gh.h, (al g).h, sum gh, sum al g
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int q = 0; q < 6; ++q) s[q][j] = 0.f;
        if (blk[j] < 0) continue;
        const Pack<VEC> w = ld<VEC>(sw + (tl + TL * j) * VEC), al = ld<VEC>(s1 + (tl + TL * j) * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float gh = __fmul_rn(w.v[e], g[j].v[e]), ag = __fmul_rn(al.v[e], g[j].v[e]);
          s[0][j] += a[j].v[e] * gh;
          s[1][j] += a[j].v[e] * x[j].v[e];
          s[2][j] += gh * x[j].v[e];
          s[3][j] += ag * x[j].v[e];
          s[4][j] += gh;
          s[5][j] += ag;
        }
      }
      block_sums<6, V, TL>(p, blk, s, red, [&](int q, int b) { return q < 4 || p.d[b] == 1; });
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!on || blk[j] < 0) continue;
        const int c = (tl + TL * j) * VEC;
        const Pack<VEC> w = ld<VEC>(sw + c), al = ld<VEC>(s1 + c), be = ld<VEC>(s2 + c);
        const float a1 = s[0][j] * inv[j], a2 = s[1][j] * inv[j], g2 = s[2][j] * inv[j], kk = s[3][j] * inv[j];
        const float mgh = cen[j] ? s[4][j] * inv[j] : 0.f, mag = cen[j] ? s[5][j] * inv[j] : 0.f;
        const float rr = r[j], ch = rr * (rr * (a1 - 3.f * g2 * a2) + kk);
        Pack<VEC> dg, dx;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float gh = __fmul_rn(w.v[e], g[j].v[e]), ag = __fmul_rn(al.v[e], g[j].v[e]);
          const float t = rr * (a[j].v[e] - x[j].v[e] * a2);
          acc[0][j].v[e] += g[j].v[e] * t;
          dg.v[e] = w.v[e] * t + al.v[e] * x[j].v[e] + be.v[e];
          dx.v[e] = rr * ((ag - mag) - rr * ((gh - mgh) * a2 + a[j].v[e] * g2)) - x[j].v[e] * ch;
        }
        if (A.o0) st_row<VEC>(A.o0 + base + c, dg);
        if (A.o1) st_row<VEC>(A.o1 + base + c, dx);
      }
    }
  }
  // partial rows of the weight gradients: the CTA's teams one after another
  if constexpr (MODE != kFwd) {
    if (!A.part) return;
    const int na = MODE == kBwd && A.want_b ? 2 : 1;
    for (int k = 0; k < na; ++k) {
      for (int t = 0; t < TEAMS; ++t) {
        __syncthreads();
        if (team != t) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (blk[j] < 0) continue;
          const int c = (tl + TL * j) * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float v = (NACC == 2 && k == 1) ? acc[NACC - 1][j].v[e] : acc[0][j].v[e];
            sw[c + e] = t == 0 ? v : sw[c + e] + v;
          }
        }
      }
      __syncthreads();
      float* dst = A.part + (int64_t(blockIdx.x) * na + k) * p.dim;
      for (int c = threadIdx.x; c < p.dim; c += blockDim.x) dst[c] = sw[c];
    }
  }
}

// dw[u] = sum over partial rows and m of column (u, m); db the same of the second
// rows.  One warp per weight; lane i adds rows i, i + 32, ... and the lanes are
// added by a tree: a fixed order.
__global__ void __launch_bounds__(256) k_norm_reduce(const __grid_constant__ NormDev p, const float* __restrict__ part,
                                                     int rows, int na, float* __restrict__ dw, float* __restrict__ db) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= p.nw) return;
  int b = 0;
  for (int k = 1; k < p.nb; ++k)
    if (i >= p.woff[k]) b = k;
  const int d = p.d[b], u = i - p.woff[b], c = p.off[b] + u * d;
  for (int k = 0; k < na; ++k) {
    float* o = k == 0 ? (dw ? dw + i : nullptr) : ((db && p.boff[b] >= 0) ? db + p.boff[b] + u : nullptr);
    if (!o) continue;
    float s = 0.f;
    for (int r = lane; r < rows; r += 32) {
      const float* q = part + (int64_t(r) * na + k) * p.dim + c;
      for (int m = 0; m < d; ++m) s += q[m];
    }
#pragma unroll
    for (int t = 16; t > 0; t >>= 1) s += __shfl_xor_sync(0xffffffffu, s, t);
    if (lane == 0) *o = s;
  }
}

constexpr int kSMs = 148;

struct Shape {
  int vec, v, tl;
};
// Lanes per row and vectors per lane: the narrowest team whose lanes hold at most
// five float4 of a row (16-byte rows and blocks), or at most eight single floats
// (other rows; twenty for the widest): the rows of a pass stay in registers.
Shape shape_of(int dim, bool vec4) {
  if (vec4) {
    const int nv = dim / 4;
    const int tl = nv <= 32 ? 8 : (nv <= 160 ? 32 : (nv <= 640 ? 128 : 512));
    const int need = (nv + tl - 1) / tl;
    return {4, need <= 2 ? 2 : (need <= 3 ? 3 : (need <= 4 ? 4 : 5)), tl};
  }
  const int tl = dim <= 32 ? 8 : (dim <= 256 ? 32 : (dim <= 1024 ? 128 : 512));
  const int need = (dim + tl - 1) / tl;
  return {1, need <= 2 ? 2 : (need <= 4 ? 4 : (need <= 8 ? 8 : 20)), tl};
}
int teams_of(int tl) { return kThreads(tl) / tl; }

// CTAs of a pass: enough to fill the GPU, but several rows to a team where the
// rows suffice, so that the weight columns in shared memory and the partial rows
// of the gradients are paid once for them.
int grid_of(int64_t n, int tl, int mode) {
  const int64_t ctas = (n + teams_of(tl) - 1) / teams_of(tl);
  const int per_sm = mode == kFwd ? 8 : 3;
  return int(std::max<int64_t>(1, std::min<int64_t>(ctas, int64_t(kSMs) * per_sm)));
}

template <int MODE, int VEC, int V, int TL>
cudaError_t launch(const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  const int dimp = (p.dim + 3) & ~3;
  const size_t sm = (size_t(MODE == kDbl ? 3 : 2) * dimp + red_floats<TL>()) * 4;
  if (sm > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k_norm<MODE, VEC, V, TL>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sm));
    if (e) return e;
  }
  k_norm<MODE, VEC, V, TL><<<grid, kThreads(TL), sm, st>>>(p, a);
  return cudaGetLastError();
}
template <int MODE, int VEC, int TL>
cudaError_t launch_v(int v, const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  if constexpr (VEC == 4) {
    switch (v) {
      case 2: return launch<MODE, 4, 2, TL>(p, a, grid, st);
      case 3: return launch<MODE, 4, 3, TL>(p, a, grid, st);
      case 4: return launch<MODE, 4, 4, TL>(p, a, grid, st);
      default: return launch<MODE, 4, 5, TL >= 32 ? TL : 32>(p, a, grid, st);  // (a team of 8 has at most 4)
    }
  } else {
    if (v == 2 && TL <= 32) return launch<MODE, 1, 2, TL <= 32 ? TL : 32>(p, a, grid, st);
    if (v == 4) return launch<MODE, 1, 4, TL>(p, a, grid, st);
    if (v == 8 && TL >= 32) return launch<MODE, 1, 8, TL >= 32 ? TL : 32>(p, a, grid, st);
    if (v == 20 && TL == 512) return launch<MODE, 1, 20, 512>(p, a, grid, st);
    return cudaErrorInvalidValue;
  }
}
template <int MODE, int VEC>
cudaError_t launch_tl(const Shape& s, const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  switch (s.tl) {
    case 8: return launch_v<MODE, VEC, 8>(s.v, p, a, grid, st);
    case 32: return launch_v<MODE, VEC, 32>(s.v, p, a, grid, st);
    case 128: return launch_v<MODE, VEC, 128>(s.v, p, a, grid, st);
    default: return launch_v<MODE, VEC, 512>(s.v, p, a, grid, st);
  }
}
template <int MODE>
cudaError_t launch_mode(const Shape& s, const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  return s.vec == 4 ? launch_tl<MODE, 4>(s, p, a, grid, st) : launch_tl<MODE, 1>(s, p, a, grid, st);
}

}  // namespace
}  // namespace tpc

using namespace tpc;

struct tpconv_norm {
  NormDev p;
  bool vec4;  // every block starts and ends on a multiple of 4 floats
};

namespace {

int status_of(cudaError_t e) { return e == cudaSuccess ? TPCONV_OK : TPCONV_ERR_CUDA; }

// workspace: the partial rows of dw (and db)
size_t partial_bytes(const tpconv_norm* plan, int op, int64_t N) {
  if (op == TPCONV_OP_FORWARD || N <= 0) return 0;
  const Shape s = shape_of(plan->p.dim, plan->vec4);
  const int mode = op == TPCONV_OP_BACKWARD ? kBwd : kDbl;
  return size_t(grid_of(N, s.tl, mode)) * (mode == kBwd ? 2 : 1) * plan->p.dim * 4;
}

bool rows16(const tpconv_norm* plan, std::initializer_list<const void*> ps) {
  if (!plan->vec4) return false;
  for (const void* q : ps)
    if (q && !aligned_to_16(q)) return false;
  return true;
}
bool floats_ok(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (q && misaligned(q, 4)) return false;
  return true;
}

}  // namespace

extern "C" {

int tpconv_norm_create(tpconv_norm** out, const char* irreps, double eps) {
  if (!out) return TPCONV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!irreps || !(eps > 0) || !std::isfinite(eps) || !(float(eps) > 0.f) || !std::isfinite(float(eps)))
    return TPCONV_ERR_INVALID_ARG;
  try {
    std::vector<Blk> b;
    const int st = parse_irreps(irreps, b);
    if (st) return st;
    static_assert(sizeof(NormDev) < 2048, "kernel parameter");
    if (b.size() > size_t(kBlocksMax)) return TPCONV_ERR_UNSUPPORTED;
    NormDev p;
    std::memset(&p, 0, sizeof(p));
    p.nb = int(b.size());
    p.eps = float(eps);
    bool vec4 = true;
    int64_t off = 0;
    for (int i = 0; i < p.nb; ++i) {
      const int d = 2 * b[i].l + 1;
      p.off[i] = int(off);
      p.d[i] = d;
      p.woff[i] = p.nw;
      p.boff[i] = (b[i].l == 0 && b[i].p == 1) ? p.nbias : -1;
      const int64_t s = int64_t(b[i].mul) * d;
      if (off + s > TPCONV_NORM_MAX_DIM) return TPCONV_ERR_UNSUPPORTED;
      p.inv[i] = float(1.0 / double(s));
      p.nw += b[i].mul;
      if (p.boff[i] >= 0) p.nbias += b[i].mul;
      vec4 = vec4 && s % 4 == 0;
      off += s;
    }
    p.off[p.nb] = p.dim = int(off);
    tpconv_norm* plan = new (std::nothrow) tpconv_norm();
    if (!plan) return TPCONV_ERR_INTERNAL;
    plan->p = p;
    plan->vec4 = vec4;
    *out = plan;
    return TPCONV_OK;
  } catch (...) {
    return TPCONV_ERR_INTERNAL;
  }
}

int tpconv_norm_destroy(tpconv_norm* plan) {
  delete plan;
  return TPCONV_OK;
}

int tpconv_norm_info(const tpconv_norm* plan, int* n_blocks, int* dim, int* weight_numel, int* bias_numel) {
  if (!plan) return TPCONV_ERR_INVALID_ARG;
  if (n_blocks) *n_blocks = plan->p.nb;
  if (dim) *dim = plan->p.dim;
  if (weight_numel) *weight_numel = plan->p.nw;
  if (bias_numel) *bias_numel = plan->p.nbias;
  return TPCONV_OK;
}

int tpconv_norm_workspace_size(const tpconv_norm* plan, int op, int64_t N, size_t* bytes) {
  if (!plan || !bytes || N < 0 || op < TPCONV_OP_FORWARD || op > TPCONV_OP_DOUBLE_BACKWARD)
    return TPCONV_ERR_INVALID_ARG;
  *bytes = (partial_bytes(plan, op, N) + 255) & ~size_t(255);
  return TPCONV_OK;
}

int tpconv_norm_forward(const tpconv_norm* plan, int64_t N, const float* x, const float* weight, const float* bias,
                        float* y, void* stream) {
  if (!plan || N < 0 || (N > 0 && (!x || !y))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, bias, y})) return TPCONV_ERR_INVALID_ARG;
  const NormDev& p = plan->p;
  const size_t rows = size_t(N) * p.dim * 4;
  const Span sp[] = {{y, rows}, {x, rows}, {weight, size_t(p.nw) * 4}, {bias, size_t(p.nbias) * 4}};
  if (overlapping(sp, 1, 4)) return TPCONV_ERR_INVALID_ARG;
  if (N == 0) return TPCONV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NodePhase ph(TPCONV_PHASE_NORM, st);
  const Shape s = shape_of(p.dim, rows16(plan, {x, y}));
  NormArgs a{};
  a.x = x, a.w = weight, a.b = bias, a.o0 = y, a.n = N;
  ph.note(1);
  return status_of(launch_mode<kFwd>(s, p, a, grid_of(N, s.tl, kFwd), st));
}

int tpconv_norm_backward(const tpconv_norm* plan, int64_t N, const float* x, const float* weight, const float* g,
                         float* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!plan || N < 0 || (N > 0 && (!x || !g))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, dx, dweight, dbias})) return TPCONV_ERR_INVALID_ARG;
  const NormDev& p = plan->p;
  const bool sums = dweight || dbias;
  const size_t need = sums ? partial_bytes(plan, TPCONV_OP_BACKWARD, N) : 0;
  if (workspace_bytes < need) return TPCONV_ERR_WORKSPACE_TOO_SMALL;
  if (need && (!workspace || misaligned(workspace, 256))) return TPCONV_ERR_INVALID_ARG;
  const size_t rows = size_t(N) * p.dim * 4, wb = size_t(p.nw) * 4;
  const Span sp[] = {{dx, rows}, {dweight, wb}, {dbias, size_t(p.nbias) * 4}, {workspace, need},
                     {x, rows},  {weight, wb},  {g, rows}};
  if (overlapping(sp, 4, 7)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, wb, st)) return TPCONV_ERR_CUDA;
    if (dbias && p.nbias && cudaMemsetAsync(dbias, 0, size_t(p.nbias) * 4, st)) return TPCONV_ERR_CUDA;
    return TPCONV_OK;
  }
  if (!dx && !sums) return TPCONV_OK;
  NodePhase ph(TPCONV_PHASE_NORM, st);
  const Shape s = shape_of(p.dim, rows16(plan, {x, g, dx}));
  const int grid = grid_of(N, s.tl, kBwd);
  NormArgs a{};
  a.x = x, a.w = weight, a.g = g, a.o0 = dx, a.n = N;
  a.want_b = dbias && p.nbias > 0;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = launch_mode<kBwd>(s, p, a, grid, st);
  ph.note(1);
  if (e == cudaSuccess && sums) {
    k_norm_reduce<<<(p.nw + 7) / 8, 256, 0, st>>>(p, a.part, grid, a.want_b ? 2 : 1, dweight, dbias);
    ph.note(1);
    e = cudaGetLastError();
  }
  return status_of(e);
}

int tpconv_norm_double_backward(const tpconv_norm* plan, int64_t N, const float* x, const float* weight,
                                const float* g, const float* gg_x, const float* gg_weight, const float* gg_bias,
                                float* d_g, float* d_x, float* d_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!plan || N < 0 || (N > 0 && (!x || !g))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, gg_x, gg_weight, gg_bias, d_g, d_x, d_weight})) return TPCONV_ERR_INVALID_ARG;
  const NormDev& p = plan->p;
  const size_t need = d_weight ? partial_bytes(plan, TPCONV_OP_DOUBLE_BACKWARD, N) : 0;
  if (workspace_bytes < need) return TPCONV_ERR_WORKSPACE_TOO_SMALL;
  if (need && (!workspace || misaligned(workspace, 256))) return TPCONV_ERR_INVALID_ARG;
  const size_t rows = size_t(N) * p.dim * 4, wb = size_t(p.nw) * 4;
  const Span sp[] = {{d_g, rows},  {d_x, rows}, {d_weight, wb}, {workspace, need},  {x, rows},
                     {weight, wb}, {g, rows},   {gg_x, rows},   {gg_weight, wb}, {gg_bias, size_t(p.nbias) * 4}};
  if (overlapping(sp, 4, 10)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (d_weight && cudaMemsetAsync(d_weight, 0, wb, st)) return TPCONV_ERR_CUDA;
    return TPCONV_OK;
  }
  if (!d_g && !d_x && !d_weight) return TPCONV_OK;
  NodePhase ph(TPCONV_PHASE_NORM, st);
  const Shape s = shape_of(p.dim, rows16(plan, {x, g, gg_x, d_g, d_x}));
  const int grid = grid_of(N, s.tl, kDbl);
  NormArgs a{};
  a.x = x, a.w = weight, a.g = g, a.a = gg_x, a.al = gg_weight, a.be = gg_bias, a.o0 = d_g, a.o1 = d_x, a.n = N;
  a.part = d_weight ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = launch_mode<kDbl>(s, p, a, grid, st);
  ph.note(1);
  if (e == cudaSuccess && d_weight) {
    k_norm_reduce<<<(p.nw + 7) / 8, 256, 0, st>>>(p, a.part, grid, 1, d_weight, nullptr);
    ph.note(1);
    e = cudaGetLastError();
  }
  return status_of(e);
}

}  // extern "C"
