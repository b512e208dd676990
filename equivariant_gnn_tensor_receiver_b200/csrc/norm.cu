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
// rows.  Each block of the row has lanes of its own, as many as its length asks for:
// lane i of a block's L lanes owns the elements (4-float vectors, where rows and
// blocks are 16-byte aligned) i + L j of it, in every row that the team visits.  A
// lane's sums are then one number each, a block's sum is a scan over its lanes (six
// shuffles, whatever the number of blocks), the per-column weights sit in shared
// memory once per CTA, and the weight gradients accumulate in registers over the
// rows.  At the end the CTA adds its teams' accumulators pairwise into a partial row
// of the workspace, and k_norm_reduce sums the partial rows in a fixed order (no
// atomics: repeated calls agree bit for bit).  (Lanes dealt out over the row without
// regard to blocks need a masked sum per block and quantity: 46 us against 25
// for the double backward of 20 011 rows of 37x0e+21x1o+5x2e+3x0o.)
//
// Measured (graph replays, warm; floor = bytes over 6.54 TB/s), 120 000 rows: 128x l<=3
// (2048 floats) forward 312 us (floor 301), backward 548 (451), double backward 843 (752);
// 32x l<=2 (288 floats) 52 (42), 90 (63; dx alone 82), 142 (106).  Blocks that do not start on 16 bytes
// (37x0e+21x1o+5x2e+3x0o, 128 floats, read 4 bytes at a time) 41 (19), 64 (28), 115 (47):
// there the instructions bound it (70 % of the issue slots; addresses, predicates and
// the sums' shuffles for four bytes at a time), not HBM.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/tpconv.h"
#include "chain.cuh"
#include "irreps.h"
#include "node_ops.h"

namespace tpc {
namespace {

constexpr int kBlocksMax = 12;

struct NormDev {
  int nb, dim, nw, nbias;
  int any0;                 // whether a block has l = 0
  int off[kBlocksMax + 1];  // first column of a block; off[nb] = dim
  int d[kBlocksMax];        // 2l+1
  int woff[kBlocksMax];     // first weight of a block
  int boff[kBlocksMax];     // first bias of a block, or -1
  int lane[kBlocksMax + 1]; // first lane of a block's lanes in a team
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
    r.v[0] = __ldg(p);  // (the sectors of unaligned pieces are shared between vectors)
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

// where a lane stands: its block (-1: none), the block's lanes in this warp, and for
// teams of several warps the warps that hold the block
struct Place {
  int b, first, last, w0, w1;
};

// Sums of Q quantities over the block of each lane, in every lane of the block.
template <int Q, int TL>
__device__ __forceinline__ void block_sums(const Place& at, float (&v)[Q], float* red) {
  const int lane = threadIdx.x & 31;
  constexpr int W = TL < 32 ? TL : 32;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float u = __shfl_up_sync(0xffffffffu, v[q], o);
      v[q] += lane - o >= at.first ? u : 0.f;
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q] = __shfl_sync(0xffffffffu, v[q], at.last);
  if constexpr (TL > 32) {
    // the parts of a block that several warps share: [warp][block][quantity]
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // the last sums have been read
    if (at.b >= 0 && lane == at.first) {
#pragma unroll
      for (int q = 0; q < Q; ++q) red[(warp * kBlocksMax + at.b) * Q + q] = v[q];
    }
    __syncthreads();
    if (at.b >= 0 && at.w1 > at.w0) {
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] = 0.f;
      for (int w = at.w0; w <= at.w1; ++w)
#pragma unroll
        for (int q = 0; q < Q; ++q) v[q] += red[(w * kBlocksMax + at.b) * Q + q];
    }
  }
}

// floats of shared memory behind the column weights: reduction scratch
constexpr int kRedQ = 6;
template <int TL>
constexpr int red_floats() {
  return TL <= 32 ? 0 : TL / 32 * kBlocksMax * kRedQ;
}

template <int MODE, int VEC, int V, int TL>
__global__ void __launch_bounds__(kThreads(TL)) k_norm(const __grid_constant__ NormDev p, const NormArgs A) {
  constexpr int TEAMS = kThreads(TL) / TL;
  constexpr int NACC = MODE == kBwd ? 2 : (MODE == kDbl ? 1 : 0);  // dw, db | d_w
  extern __shared__ float4 smem4[];
  float* sm = reinterpret_cast<float*>(smem4);
  if (MODE != kFwd && A.part) chain_next();
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
  Place at{-1, int(threadIdx.x & 31), int(threadIdx.x & 31), 0, 0};
  for (int b = 0; b < p.nb; ++b)
    if (tl >= p.lane[b] && tl < p.lane[b + 1]) at.b = b;
  int col = 0, left = 0, step = 1;  // first column, elements from there to the block's end, elements between vectors
  float inv = 0.f;
  bool cen = false;  // l = 0: centred
  if (at.b >= 0) {
    const int l0 = p.lane[at.b], l1 = p.lane[at.b + 1], base = int(threadIdx.x & 31) - tl % 32;
    at.first = base + max(l0 - (tl & ~31), 0);
    at.last = base + min(l1 - (tl & ~31), 32) - 1;
    at.w0 = l0 >> 5, at.w1 = (l1 - 1) >> 5;
    col = p.off[at.b] + (tl - l0) * VEC;
    left = p.off[at.b + 1] - col;
    step = (l1 - l0) * VEC;
    inv = p.inv[at.b];
    cen = p.d[at.b] == 1;
  }
  Pack<VEC> acc[NACC > 0 ? NACC : 1][V];
#pragma unroll
  for (int k = 0; k < (NACC > 0 ? NACC : 1); ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[k][j].v[e] = 0.f;
  const Pack<VEC> zero = {};

  // every lane runs the same number of rounds: the sums are collective
  const int64_t stride = int64_t(gridDim.x) * TEAMS;
  const int64_t rounds = (A.n + stride - 1) / stride;
  constexpr int NG = MODE == kFwd ? 1 : V, NA = MODE == kDbl ? V : 1;
  auto load = [&](int64_t k, Pack<VEC>(&x)[V], Pack<VEC>(&g)[NG], Pack<VEC>(&a)[NA]) {
    const int64_t row = k * stride + int64_t(blockIdx.x) * TEAMS + team, base = row * p.dim + col;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool in = row < A.n && j * step < left;
      x[j] = in ? ld_row<VEC>(A.x + base + j * step) : zero;
      if constexpr (MODE != kFwd) g[j] = in ? ld_row<VEC>(A.g + base + j * step) : zero;
      if constexpr (MODE == kDbl) a[j] = (in && A.a) ? ld_row<VEC>(A.a + base + j * step) : zero;
    }
  };
  // Rows of few floats a lane are read one round ahead: a warp's own latencies (the reads,
  // then the sums one after another) would leave HBM waiting.  120 000 rows of 128x l<=3,
  // without and with: backward 887 and 548 us, double backward 1244 and 843; 32x l<=2: 122
  // and 92, 170 and 144.  Not for single floats in the double backward: 122 without, 136 with.
  constexpr bool AHEAD = V * VEC <= 12 && (VEC == 4 || MODE != kDbl);
  Pack<VEC> nx[V], ng[NG], na[NA];
  if constexpr (AHEAD) load(0, nx, ng, na);
  for (int64_t k = 0; k < rounds; ++k) {
    const int64_t row = k * stride + int64_t(blockIdx.x) * TEAMS + team;
    const bool on = row < A.n;
    const int64_t base = row * p.dim + col;
    Pack<VEC> x[V], g[NG], a[NA];
    if constexpr (AHEAD) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] = nx[j];
        if constexpr (MODE != kFwd) g[j] = ng[j];
        if constexpr (MODE == kDbl) a[j] = na[j];
      }
      load(k + 1, nx, ng, na);
    } else {
      load(k, x, g, a);
    }
    // centre the scalars (x, and gg_x in the double backward); what lies behind a block stays 0
    if (p.any0) {
      constexpr int Q = MODE == kDbl ? 2 : 1;
      float s[Q] = {};
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[0] += x[j].v[e];
          if constexpr (Q == 2) s[1] += a[j].v[e];
        }
      block_sums<Q, TL>(at, s, red);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (cen && j * step < left) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x[j].v[e] -= s[0] * inv;
            if constexpr (Q == 2) a[j].v[e] -= s[1] * inv;
          }
        }
    }
    // x becomes h.  In the double backward, which divides by the root mean square up to
    // three times, the scalars' sum is taken again with their squares: what the rounding
    // of the mean left is removed from both.
    float r;
    {
      constexpr int Q = MODE == kDbl ? 2 : 1;
      float s[Q] = {};
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[0] += x[j].v[e] * x[j].v[e];
          if constexpr (Q == 2) s[1] += x[j].v[e];
        }
      block_sums<Q, TL>(at, s, red);
      float m = 0.f;
      if constexpr (Q == 2) m = cen ? s[1] * inv : 0.f;
      const float var = s[0] * inv - m * m;
      r = 1.f / sqrtf((var < 0.f ? 0.f : var) + p.eps);  // (a NaN stays)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * step < left) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[j].v[e] = (Q == 2 ? x[j].v[e] - m : x[j].v[e]) * r;
        }
    }
    if constexpr (MODE == kFwd) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = col + j * step;
        if (!on || j * step >= left) continue;
        const Pack<VEC> w = ld<VEC>(sw + c), bb = ld<VEC>(s1 + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j].v[e] = w.v[e] * x[j].v[e] + bb.v[e];
        st_row<VEC>(A.o0 + base + j * step, x[j]);
      }
    } else if constexpr (MODE == kBwd) {
      float s[2] = {};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * step >= left) continue;
        const Pack<VEC> w = ld<VEC>(sw + col + j * step);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          acc[0][j].v[e] += g[j].v[e] * x[j].v[e];
          acc[1][j].v[e] += g[j].v[e];
          g[j].v[e] = __fmul_rn(g[j].v[e], w.v[e]);  // (not fused into gh - mean: a lone scalar gives 0)
          s[0] += g[j].v[e] * x[j].v[e];
          s[1] += g[j].v[e];
        }
      }
      if (A.o0) {
        block_sums<2, TL>(at, s, red);
        const float c1 = s[0] * inv, mg = cen ? s[1] * inv : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!on || j * step >= left) continue;
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[j].v[e] = r * (g[j].v[e] - mg - x[j].v[e] * c1);
          st_row<VEC>(A.o0 + base + j * step, x[j]);
        }
      }
    } else {
      float s[6] = {};  // a.gh, a.h, gh.h, (al g).h, sum gh, sum al g
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j * step >= left) continue;
        const Pack<VEC> w = ld<VEC>(sw + col + j * step), al = ld<VEC>(s1 + col + j * step);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float gh = __fmul_rn(w.v[e], g[j].v[e]), ag = __fmul_rn(al.v[e], g[j].v[e]);
          s[0] += a[j].v[e] * gh;
          s[1] += a[j].v[e] * x[j].v[e];
          s[2] += gh * x[j].v[e];
          s[3] += ag * x[j].v[e];
          s[4] += gh;
          s[5] += ag;
        }
      }
      block_sums<6, TL>(at, s, red);
      const float a1 = s[0] * inv, a2 = s[1] * inv, g2 = s[2] * inv, kk = s[3] * inv;
      const float mgh = cen ? s[4] * inv : 0.f, mag = cen ? s[5] * inv : 0.f;
      const float ch = r * (r * (a1 - 3.f * g2 * a2) + kk);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!on || j * step >= left) continue;
        const int c = col + j * step;
        const Pack<VEC> w = ld<VEC>(sw + c), al = ld<VEC>(s1 + c), be = ld<VEC>(s2 + c);
        Pack<VEC> dg, dx;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float gh = __fmul_rn(w.v[e], g[j].v[e]), ag = __fmul_rn(al.v[e], g[j].v[e]);
          const float t = r * (a[j].v[e] - x[j].v[e] * a2);
          acc[0][j].v[e] += g[j].v[e] * t;
          dg.v[e] = w.v[e] * t + al.v[e] * x[j].v[e] + be.v[e];
          dx.v[e] = r * ((ag - mag) - r * ((gh - mgh) * a2 + a[j].v[e] * g2)) - x[j].v[e] * ch;
        }
        if (A.o0) st_row<VEC>(A.o0 + base + j * step, dg);
        if (A.o1) st_row<VEC>(A.o1 + base + j * step, dx);
      }
    }
  }
  // partial rows of the weight gradients: the CTA's teams added pairwise, in a fixed order
  if constexpr (MODE != kFwd) {
    if (!A.part) return;
    const int na = MODE == kBwd && A.want_b ? 2 : 1;
    // shared memory: one row of sums per team of the lower half (the weights are no longer needed)
    for (int half = TEAMS / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (team >= half && team < 2 * half) {
#pragma unroll
        for (int k = 0; k < NACC; ++k)
          if (k < na)
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (j * step < left) st_row<VEC>(sm + ((team - half) * na + k) * dimp + col + j * step, acc[k][j]);
      }
      __syncthreads();
      if (team < half) {
#pragma unroll
        for (int k = 0; k < NACC; ++k)
          if (k < na)
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (j * step < left) {
                const Pack<VEC> o = ld<VEC>(sm + (team * na + k) * dimp + col + j * step);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[k][j].v[e] += o.v[e];
              }
      }
    }
    if (team == 0) {
#pragma unroll
      for (int k = 0; k < NACC; ++k)
        if (k < na) {
          float* dst = A.part + (int64_t(blockIdx.x) * na + k) * dimp;
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j * step < left) st_row<VEC>(dst + col + j * step, acc[k][j]);
        }
    }
  }
}

// dw[u] = sum over partial rows and m of column (u, m); db the same of the second
// rows.  A CTA takes whole channels of one block, up to 32 columns: thread (x, y) adds
// rows y, y + 32, ... of column x (coalesced), the 32 sums of a column are added by a
// tree, then the 2l+1 columns of a channel: a fixed order.
__global__ void __launch_bounds__(1024) k_norm_reduce(const __grid_constant__ NormDev p, const float* part,
                                                      int rows, int na, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[32][33], col[32];
  const int dimp = (p.dim + 3) & ~3, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  int i = blockIdx.x, b = 0;
  for (;; ++b) {  // the block, and the CTA's channels u0 .. u0 + n - 1 of it
    const int n = 32 / p.d[b], c = (p.off[b + 1] - p.off[b]) / p.d[b], ctas = (c + n - 1) / n;
    if (i < ctas) break;
    i -= ctas;
  }
  const int d = p.d[b], per = 32 / d, mul = (p.off[b + 1] - p.off[b]) / d;
  const int u0 = i * per, n = min(per, mul - u0), c0 = p.off[b] + u0 * d;
  chain_wait();
  for (int k = 0; k < na; ++k) {
    float* o = k == 0 ? (dw ? dw + p.woff[b] : nullptr) : ((db && p.boff[b] >= 0) ? db + p.boff[b] : nullptr);
    if (!o) continue;
    float v = 0.f;
    if (x < n * d) {
      const float* q = part + int64_t(k) * dimp + c0 + x;
#pragma unroll 4
      for (int r = y; r < rows; r += 32) v += q[int64_t(r) * na * dimp];
    }
    s[y][x] = v;
    __syncthreads();
    float w = s[x][y];  // warp y: column y
#pragma unroll
    for (int t = 16; t > 0; t >>= 1) w += __shfl_xor_sync(0xffffffffu, w, t);
    if (x == 0) col[y] = w;
    __syncthreads();
    if (threadIdx.x < n) {
      float z = 0.f;
      for (int m = 0; m < d; ++m) z += col[threadIdx.x * d + m];
      o[u0 + threadIdx.x] = z;
    }
    __syncthreads();
  }
}

constexpr int kSMs = 148;

struct Shape {
  int vec, v, tl;
};
// Lanes per row and vectors per lane, and the blocks' lanes: the narrowest team whose
// lanes hold at most five float4 of a row (16-byte rows and blocks), or at most eight
// single floats (other rows), so that a pass's rows stay in registers; up to six float4
// or 24 floats for the widest rows.
Shape shape_of(NormDev& p, bool vec4) {
  static const int v4[] = {1, 2, 3, 4, 5, 6}, v1[] = {2, 4, 5, 8, 24};
  const int vec = vec4 ? 4 : 1, nv = vec4 ? 6 : 5, wide = nv - 1;
  for (int tl : {8, 32, 128, 512})
    for (int i = 0; i < nv; ++i) {
      if (i == wide && tl != 512) continue;
      const int v = vec4 ? v4[i] : v1[i];
      int lanes = 0;
      for (int b = 0; b < p.nb; ++b) {
        p.lane[b] = lanes;
        lanes += ((p.off[b + 1] - p.off[b]) / vec + v - 1) / v;
      }
      p.lane[p.nb] = lanes;
      if (lanes <= tl) return {vec, v, tl};
    }
  return {0, 0, 0};  // (not reached: at most 10240 floats and 12 blocks)
}
int teams_of(int tl) { return kThreads(tl) / tl; }

// CTAs of a pass.  Forward: as many as there are rows for, up to eight per SM.  The
// gradients: what their registers leave resident (512 threads per SM, 1024 of few
// floats a lane), and at least two rows to a team: the partial rows of the sums are
// paid once for them.
int grid_of(int64_t n, const Shape& s, int mode) {
  const int64_t teams = mode == kFwd ? n : (n + 1) / 2, ctas = (teams + teams_of(s.tl) - 1) / teams_of(s.tl);
  const int per_sm = mode == kFwd ? 8 : (s.vec * s.v <= 12 ? 1024 : 512) / kThreads(s.tl);
  return int(std::max<int64_t>(1, std::min<int64_t>(ctas, int64_t(kSMs) * per_sm)));
}

int reduce_grid(const NormDev& p) {
  int g = 0;
  for (int b = 0; b < p.nb; ++b) {
    const int n = 32 / p.d[b], c = (p.off[b + 1] - p.off[b]) / p.d[b];
    g += (c + n - 1) / n;
  }
  return g;
}

template <int MODE, int VEC, int V, int TL>
cudaError_t launch(const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  const int dimp = (p.dim + 3) & ~3;
  // the column weights and the reduction scratch; at the end the teams' sums
  const int sums = MODE == kFwd ? 0 : kThreads(TL) / TL / 2 * (MODE == kBwd ? 2 : 1);
  const size_t sm = std::max(size_t(MODE == kDbl ? 3 : 2) * dimp + red_floats<TL>(), size_t(sums) * dimp) * 4;
  if (sm > 48 * 1024) {
    // (the most a call may ask for, not this call's: another thread's call must not lower it)
    cudaError_t e = cudaFuncSetAttribute(k_norm<MODE, VEC, V, TL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         227 * 1024);
    if (e) return e;
  }
  k_norm<MODE, VEC, V, TL><<<grid, kThreads(TL), sm, st>>>(p, a);
  return cudaGetLastError();
}
template <int MODE, int VEC, int TL>
cudaError_t launch_v(int v, const NormDev& p, const NormArgs& a, int grid, cudaStream_t st) {
  if constexpr (VEC == 4) {
    switch (v) {
      case 1: return launch<MODE, 4, 1, TL>(p, a, grid, st);
      case 2: return launch<MODE, 4, 2, TL>(p, a, grid, st);
      case 3: return launch<MODE, 4, 3, TL>(p, a, grid, st);
      case 4: return launch<MODE, 4, 4, TL>(p, a, grid, st);
      case 5: return launch<MODE, 4, 5, TL>(p, a, grid, st);
      default: return launch<MODE, 4, 6, 512>(p, a, grid, st);  // (the widest team alone)
    }
  } else {
    switch (v) {
      case 2: return launch<MODE, 1, 2, TL>(p, a, grid, st);
      case 4: return launch<MODE, 1, 4, TL>(p, a, grid, st);
      case 5: return launch<MODE, 1, 5, TL>(p, a, grid, st);
      case 8: return launch<MODE, 1, 8, TL>(p, a, grid, st);
      default: return launch<MODE, 1, 24, 512>(p, a, grid, st);
    }
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
  // the grid grows with the teams of a CTA: the more of the two ways a call may run
  NormDev p = plan->p;
  const Shape s = shape_of(p, plan->vec4), s1 = shape_of(p, false);
  const int mode = op == TPCONV_OP_BACKWARD ? kBwd : kDbl;
  return size_t(std::max(grid_of(N, s, mode), grid_of(N, s1, mode))) * (mode == kBwd ? 2 : 1) * ((plan->p.dim + 3) & ~3) * 4;
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
      p.any0 |= d == 1;
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
  NormDev p = plan->p;
  const size_t rows = size_t(N) * p.dim * 4;
  const Span sp[] = {{y, rows}, {x, rows}, {weight, size_t(p.nw) * 4}, {bias, size_t(p.nbias) * 4}};
  if (overlapping(sp, 1, 4)) return TPCONV_ERR_INVALID_ARG;
  if (N == 0) return TPCONV_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NodePhase ph(TPCONV_PHASE_NORM, st);
  const Shape s = shape_of(p, rows16(plan, {x, y}));
  NormArgs a{};
  a.x = x, a.w = weight, a.b = bias, a.o0 = y, a.n = N;
  ph.note(1);
  return status_of(launch_mode<kFwd>(s, p, a, grid_of(N, s, kFwd), st));
}

int tpconv_norm_backward(const tpconv_norm* plan, int64_t N, const float* x, const float* weight, const float* g,
                         float* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!plan || N < 0 || (N > 0 && (!x || !g))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, dx, dweight, dbias})) return TPCONV_ERR_INVALID_ARG;
  NormDev p = plan->p;
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
  const Shape s = shape_of(p, rows16(plan, {x, g, dx}));
  const int grid = grid_of(N, s, kBwd);
  NormArgs a{};
  a.x = x, a.w = weight, a.g = g, a.o0 = dx, a.n = N;
  a.want_b = dbias && p.nbias > 0;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = launch_mode<kBwd>(s, p, a, grid, st);
  ph.note(1);
  if (e == cudaSuccess && sums) {
    e = chain_launch(k_norm_reduce, reduce_grid(p), 1024, 0, st, p, static_cast<const float*>(a.part), grid,
                     a.want_b ? 2 : 1, dweight, dbias);
    ph.note(1);
  }
  return status_of(e);
}

int tpconv_norm_double_backward(const tpconv_norm* plan, int64_t N, const float* x, const float* weight,
                                const float* g, const float* gg_x, const float* gg_weight, const float* gg_bias,
                                float* d_g, float* d_x, float* d_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!plan || N < 0 || (N > 0 && (!x || !g))) return TPCONV_ERR_INVALID_ARG;
  if (!floats_ok({x, weight, g, gg_x, gg_weight, gg_bias, d_g, d_x, d_weight})) return TPCONV_ERR_INVALID_ARG;
  NormDev p = plan->p;
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
  const Shape s = shape_of(p, rows16(plan, {x, g, gg_x, d_g, d_x}));
  const int grid = grid_of(N, s, kDbl);
  NormArgs a{};
  a.x = x, a.w = weight, a.g = g, a.a = gg_x, a.al = gg_weight, a.be = gg_bias, a.o0 = d_g, a.o1 = d_x, a.n = N;
  a.part = d_weight ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = launch_mode<kDbl>(s, p, a, grid, st);
  ph.note(1);
  if (e == cudaSuccess && d_weight) {
    e = chain_launch(k_norm_reduce, reduce_grid(p), 1024, 0, st, p, static_cast<const float*>(a.part), grid, 1, d_weight,
                     static_cast<float*>(nullptr));
    ph.note(1);
  }
  return status_of(e);
}

}  // extern "C"
