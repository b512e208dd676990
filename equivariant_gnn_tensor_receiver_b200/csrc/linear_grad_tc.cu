// Weight gradient of the typed linear map on the tensor cores (sm_100a: tcgen05
// with one operand in TMEM, bulk copies of node rows).
//
//   dW[t][u][w] = sum over the (node, m) rows of type t of x[n, u, m] g[n, w, m]
//
// per path, 128 input channels and 64 output channels: a product whose depth is the
// ragged row count of the type.  A chunk is the rows of 64, 16, 8 or 8 nodes
// (l = 0..3: 64, 48, 40, 56 rows); bulk copies gather the nodes' pieces of x and g by
// perm.  The A operand is x transposed: thread u reads its channel of every row (the
// lanes of a warp are 2l+1 floats apart: no bank conflicts), splits it (3xTF32) and
// stores hi and lo to TMEM, lane = u, column = row.  The B operand is g: thread w
// reads its channel and writes hi and lo into the K-major 128-byte-swizzled tile.  One
// thread issues A_lo B_hi + A_hi B_lo, then A_hi B_hi.  After kRound chunks the
// accumulator's bank is added into fp32 registers (round to nearest), which bounds
// the chain of tensor-core additions whatever the number of rows.
//
// The (path, channel tile) entries x types x chunks are cut into one equal share per
// CTA.  A type's rows that lie in one share are stored straight into dW; a share
// that begins or ends inside a type stores a partial tile (at most two per CTA), and
// k_linear_grad_join adds a type's partial tiles in the order of the CTAs: no
// atomics, the same bits every time.  It also clears the weights of empty types.
//
// Bound: HBM (x and g read once), next to shared memory: a row of 64 + 64 channels
// is 512 B from HBM and about 2.3 KB of shared-memory traffic.
// Warps 0-3 convert x, 4-7 convert g, 8-11 add finished banks and store, 12 issues
// copies, 13 MMAs.  Waits are bounded as in the row kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "linear_grad_tc.h"
#include "linear_tc_common.cuh"

namespace tpc {
namespace {

using namespace tc;

__device__ int g_linear_grad_error;  // first code recorded by an expired wait (0 = none)

constexpr int kMT = 128, kNT = 64;            // input and output channels of a tile
constexpr int kKMax = 64;                     // rows of a chunk, at most
constexpr int kRound = 3;                     // chunks accumulated in TMEM before they are added up
constexpr int kBTile = kNT * kKMax * 4;       // 16 KB: hi or lo of a B chunk
constexpr int kMaxStages = 6;
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 448;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 2 * kKMax, kTmemD = 256;

// nodes and rows of a chunk
__host__ __device__ constexpr int chunk_nodes(int d) { return d == 1 ? 64 : (d == 3 ? 16 : 8); }
__host__ __device__ inline int tiles_u(const LinPath& p) { return (p.ci + kMT - 1) / kMT; }
__host__ __device__ inline int tiles_w(const LinPath& p) { return (p.co + kNT - 1) / kNT; }
// cost of a chunk: the bytes it moves, in units of 1 KB
__host__ __device__ inline int chunk_cost(const LinPath& p, int u0, int w0) {
  const int cu = p.ci - u0 < kMT ? p.ci - u0 : kMT, cw = p.co - w0 < kNT ? p.co - w0 : kNT;
  return 1 + (cu + cw) * p.d * chunk_nodes(p.d) / 256;
}

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t afull[2], aempty[2], dfull[2], dempty[2], fin;
  uint32_t tmem;
  int abort;
  int total[4];  // chunks of all types for d = 1, 3, 5, 7
  int start_t, start_j;
};

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_grad_error, code);
}

// chunks of all types per degree: warp i (of the first four) for d = 2i + 1
__device__ __forceinline__ void count_chunks(const LinGrad& P, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= 4) return;
  const int unit = chunk_nodes(2 * warp + 1);
  int s = 0;
  for (int t = lane; t < P.T; t += 32) {
    int b, e;
    lin_group(P.offsets, P.T, P.N, t, &b, &e);
    s += (e - b + unit - 1) / unit;
  }
  s = __reduce_add_sync(0xffffffffu, s);
  if (lane == 0) total[warp] = s;
}
__device__ __forceinline__ int64_t total_cost(const LinGrad& P, const int* total) {
  int64_t c = 0;
  for (int p = 0; p < P.n_paths; ++p)
    for (int u = 0; u < tiles_u(P.p[p]); ++u)
      for (int w = 0; w < tiles_w(P.p[p]); ++w)
        c += int64_t(total[P.p[p].d >> 1]) * chunk_cost(P.p[p], u * kMT, w * kNT);
  return c;
}
__device__ __forceinline__ int64_t share_begin(int64_t total, int b, int ctas) { return total * b / ctas; }

// a run of chunks of one type in one entry
struct Piece {
  int p, u0, w0, t, first, nodes;
  int slot;  // partial tile, or -1: the type's rows are all here
};

struct Walk {
  const LinGrad& P;
  const Shared& sh;
  int64_t lo, hi, base = 0, left = 0;
  int p = -1, u = 0, w = 0;
  int t = 0, j = 0, gb = 0, ge = 0, n = 0;
  bool first_entry = true;

  __device__ Walk(const LinGrad& g, const Shared& s, int64_t total) : P(g), sh(s) {
    lo = share_begin(total, blockIdx.x, gridDim.x);
    hi = share_begin(total, blockIdx.x + 1, gridDim.x);
  }
  __device__ bool next_entry(int64_t* j0) {
    for (;;) {
      if (p < 0) {
        p = 0;
      } else {
        base += int64_t(sh.total[P.p[p].d >> 1]) * chunk_cost(P.p[p], u * kMT, w * kNT);
        if (++w >= tiles_w(P.p[p])) {
          w = 0;
          if (++u >= tiles_u(P.p[p])) u = 0, ++p;
        }
      }
      if (p >= P.n_paths || base >= hi) return false;
      const int c = chunk_cost(P.p[p], u * kMT, w * kNT);
      const int64_t all = sh.total[P.p[p].d >> 1];
      const int64_t a = lo <= base ? 0 : min((lo - base + c - 1) / c, all), b = min((hi - base + c - 1) / c, all);
      if (a < b) {
        left = b - a;
        *j0 = a;
        return true;
      }
    }
  }
  __device__ void load_group() {
    lin_group(P.offsets, P.T, P.N, t, &gb, &ge);
    const int unit = chunk_nodes(P.p[p].d);
    n = (ge - gb + unit - 1) / unit;
  }
  __device__ bool next(Piece* q) {
    if (left == 0) {
      int64_t j0;
      if (!next_entry(&j0)) return false;
      if (first_entry) {
        t = sh.start_t, j = sh.start_j;
        first_entry = false;
      } else {
        t = 0, j = 0;
      }
      load_group();
    }
    while (j >= n) {
      if (t + 1 >= P.T) return false;
      ++t, j = 0;
      load_group();
    }
    const int unit = chunk_nodes(P.p[p].d), c = int(min(int64_t(n - j), left));
    q->p = p, q->u0 = u * kMT, q->w0 = w * kNT, q->t = t;
    q->first = gb + j * unit;
    q->nodes = min(ge - q->first, c * unit);
    q->slot = (j == 0 && c == n) ? -1 : 2 * int(blockIdx.x) + (j == 0);
    j += c, left -= c;
    return true;
  }
};

// thread u: its channel of rows k0 .. k0+7 of the chunk (zeros at and behind kv)
template <int D>
__device__ __forceinline__ void read8(const float* col, int pitch, int k0, int kv, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + i;
    v[i] = k < kv ? col[(k / D) * pitch + k % D] : 0.f;
  }
}
template <int D, bool SPLIT>
__device__ __forceinline__ void convert_a(const float* raw, int u, int cu, int kv, uint32_t ta) {
  constexpr int ROWS = chunk_nodes(D) * D;
  const float* col = raw + min(u, cu - 1) * D;
  const int pitch = cu * D;
#pragma unroll 2
  for (int k0 = 0; k0 < ROWS; k0 += 8) {
    if (k0 >= kv) break;
    float v[8], h[8];
    read8<D>(col, pitch, k0, kv, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = rn_tf32(v[i]), v[i] = rn_tf32(v[i] - h[i]);
    tmem_st8(ta + k0, h);
    if (SPLIT) tmem_st8(ta + kKMax + k0, v);
  }
}
// thread (w, half): every second group of 8 rows of its channel, into the swizzled tile
template <int D, bool SPLIT>
__device__ __forceinline__ void convert_b(const float* raw, int w, int half, int cw, int kv, unsigned char* hi) {
  constexpr int ROWS = chunk_nodes(D) * D;
  const float* col = raw + min(w, cw - 1) * D;
  const int pitch = cw * D;
#pragma unroll 2
  for (int k0 = 8 * half; k0 < ROWS; k0 += 16) {
    if (k0 >= kv) break;
    float v[8], h[8];
    read8<D>(col, pitch, k0, w < cw ? kv : 0, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = rn_tf32(v[i]), v[i] = rn_tf32(v[i] - h[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = k0 / 4 + i;  // 16-byte column of the tile
      const int off = (j >> 3) * (kNT * 128) + w * 128 + (((j & 7) ^ (w & 7)) << 4);
      *reinterpret_cast<float4*>(hi + off) = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      if (SPLIT)
        *reinterpret_cast<float4*>(hi + kBTile + off) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_grad_tc(const __grid_constant__ LinGrad P, int stages, int stage_bytes, int g_offset,
                     float* __restrict__ part, uint64_t limit) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sB = base;  // 2 x (hi | lo)
  unsigned char* sRaw = base + 4 * kBTile;
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 256);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.afull[i], 256);
      mbar_init(&sh.aempty[i], 1);
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 128);
    }
    mbar_init(&sh.fin, 1);
    sh.abort = 0;
    sh.start_t = sh.start_j = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 13) tmem_alloc(&sh.tmem, kTmemCols);
  count_chunks(P, sh.total);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const int64_t total = total_cost(P, sh.total);
  if (warp == 0) {  // the type of the CTA's first chunk
    Walk w(P, sh, total);
    int64_t j0;
    if (w.next_entry(&j0)) {
      const int unit = chunk_nodes(P.p[w.p].d);
      int carry = 0;
      for (int t0 = 0; t0 < P.T; t0 += 32) {
        const int t = t0 + lane;
        int n = 0;
        if (t < P.T) {
          int b, e;
          lin_group(P.offsets, P.T, P.N, t, &b, &e);
          n = (e - b + unit - 1) / unit;
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += v;
        }
        const int64_t first = int64_t(carry) + s - n;
        if (j0 >= first && j0 < first + n) sh.start_t = t, sh.start_j = int(j0 - first);
        carry += __shfl_sync(0xffffffffu, s, 31);
      }
    }
  }
  __syncthreads();

  Walk walk(P, sh, total);
  Piece q;
  bool ok = true;
  int ci = 0;  // chunks so far
  if (warp < 8) {
    // ---- operands ----
    const bool is_a = warp < 4;
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
    const int t = threadIdx.x & 127;
    while (ok && walk.next(&q)) {
      const LinPath& L = P.p[q.p];
      const int cu = min(kMT, L.ci - q.u0), cw = min(kNT, L.co - q.w0), nq = chunk_nodes(L.d);
      for (int n0 = 0; n0 < q.nodes; n0 += nq, ++ci) {
        const int st = ci % stages, ab = ci & 1, kv = min(nq, q.nodes - n0) * L.d;
        if (ci >= 2 && !wait(&sh.aempty[ab], ((ci >> 1) + 1) & 1, limit, abort, 1)) ok = false;
        if (ok && !wait(&sh.full[st], (ci / stages) & 1, limit, abort, 2)) ok = false;
        if (!ok) break;
        const unsigned char* raw = sRaw + st * stage_bytes;
        if (is_a) {
          fence_after_sync();
          const float* rx = reinterpret_cast<const float*>(raw);
          const uint32_t ta = lane_base + kTmemA + ab * kTmemAStage;
          if (warp * 32 < cu) {  // (rows of the product behind the channels are not stored)
            switch (L.d) {
              case 1: convert_a<1, SPLIT>(rx, t, cu, kv, ta); break;
              case 3: convert_a<3, SPLIT>(rx, t, cu, kv, ta); break;
              case 5: convert_a<5, SPLIT>(rx, t, cu, kv, ta); break;
              default: convert_a<7, SPLIT>(rx, t, cu, kv, ta); break;
            }
          }
          mbar_arrive(&sh.empty[st]);
          tmem_wait_st();
          fence_before_sync();
        } else {
          const float* rg = reinterpret_cast<const float*>(raw + g_offset);
          unsigned char* hi = sB + ab * 2 * kBTile;
          switch (L.d) {
            case 1: convert_b<1, SPLIT>(rg, t & 63, t >> 6, cw, kv, hi); break;
            case 3: convert_b<3, SPLIT>(rg, t & 63, t >> 6, cw, kv, hi); break;
            case 5: convert_b<5, SPLIT>(rg, t & 63, t >> 6, cw, kv, hi); break;
            default: convert_b<7, SPLIT>(rg, t & 63, t >> 6, cw, kv, hi); break;
          }
          mbar_arrive(&sh.empty[st]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        mbar_arrive(&sh.afull[ab]);
      }
    }
  } else if (warp < 12) {
    // ---- finished banks to registers, pieces to memory ----
    const int r = threadIdx.x - 256;
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemD;
    int ri = 0;  // rounds so far
    while (ok && walk.next(&q)) {
      const LinPath& L = P.p[q.p];
      const int cu = min(kMT, L.ci - q.u0), cw = min(kNT, L.co - q.w0), nq = chunk_nodes(L.d);
      const int rounds = ((q.nodes + nq - 1) / nq + kRound - 1) / kRound;
      float acc[kNT];
#pragma unroll
      for (int i = 0; i < kNT; ++i) acc[i] = 0.f;
      for (int k = 0; k < rounds; ++k, ++ri) {
        const int db = ri & 1;
        if (!wait(&sh.dfull[db], (ri >> 1) & 1, limit, abort, 3)) {
          ok = false;
          break;
        }
        fence_after_sync();
        if ((warp & 3) * 32 < cu) {
#pragma unroll
          for (int c = 0; c < kNT; c += 16) {
            if (c < cw) {
              float v[16];
              tmem_ld16(lane_base + db * kNT + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
            }
          }
        }
        fence_before_sync();
        mbar_arrive(&sh.dempty[db]);
      }
      if (!ok || r >= cu) continue;
      float* dst = q.slot < 0 ? P.dw + int64_t(q.t) * P.wnumel + L.woff + int64_t(q.u0 + r) * L.co + q.w0
                              : part + (int64_t(q.slot) * kMT + r) * kNT;
#pragma unroll
      for (int i = 0; i < kNT; i += 4)
        if (i < cw) *reinterpret_cast<float4*>(dst + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
  } else if (warp == 12) {
    // ---- node rows to shared memory ----
    while (ok && walk.next(&q)) {
      const LinPath& L = P.p[q.p];
      const uint32_t bx = uint32_t(min(kMT, L.ci - q.u0) * L.d * 4), bg = uint32_t(min(kNT, L.co - q.w0) * L.d * 4);
      const float* x = P.x + L.xoff + q.u0 * L.d;
      const float* g = P.g + L.goff + q.w0 * L.d;
      const int nq = chunk_nodes(L.d);
      for (int n0 = 0; n0 < q.nodes; n0 += nq, ++ci) {
        const int st = ci % stages, cnt = min(nq, q.nodes - n0);
        int node[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = lane + 32 * i;
          node[i] = k < cnt ? P.perm[q.first + n0 + k] : 0;
          if (node[i] < 0 || node[i] >= P.N) node[i] = 0;
        }
        if (ci >= stages && !wait(&sh.empty[st], ((ci / stages) + 1) & 1, limit, abort, 4)) ok = false;
        ok = __all_sync(0xffffffffu, ok && !*abort);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sh.full[st], uint32_t(cnt) * (bx + bg));
        __syncwarp();
        const uint32_t dst = smem_u32(sRaw + st * stage_bytes);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = lane + 32 * i;
          if (k < cnt) {
            bulk_load(dst + k * bx, x + int64_t(node[i]) * P.dim_x, bx, &sh.full[st]);
            bulk_load(dst + g_offset + k * bg, g + int64_t(node[i]) * P.dim_g, bg, &sh.full[st]);
          }
        }
      }
    }
    if (*abort)
      for (int c = (ci > stages ? ci - stages : 0); c < ci; ++c)
        if (!mbar_wait_for(&sh.full[c % stages], (c / stages) & 1, kDrainLimitNs)) break;
  } else {
    // ---- MMAs ----
    int ri = 0;
    while (ok && walk.next(&q)) {
      const LinPath& L = P.p[q.p];
      const int cw = min(kNT, L.co - q.w0), nq = chunk_nodes(L.d);
      const uint32_t idesc = idesc_tf32(kMT, (cw + 15) & ~15);
      int in_round = 0;
      for (int n0 = 0; n0 < q.nodes; n0 += nq, ++ci) {
        const int ab = ci & 1, db = ri & 1, steps = (min(nq, q.nodes - n0) * L.d + 7) / 8;
        if (in_round == 0 && ri >= 2 && !wait(&sh.dempty[db], ((ri >> 1) + 1) & 1, limit, abort, 5)) ok = false;
        if (ok && !wait(&sh.afull[ab], (ci >> 1) & 1, limit, abort, 6)) ok = false;
        if (!ok) break;
        fence_after_sync();
        const bool last = ++in_round == kRound || n0 + nq >= q.nodes;
        if (lane == 0) {
          const uint32_t td = tmem + kTmemD + db * kNT;
          const uint32_t ah = tmem + kTmemA + ab * kTmemAStage, al = ah + kKMax;
          const uint32_t bh = smem_u32(sB + ab * 2 * kBTile), bl = bh + kBTile;
          auto off = [](int k) { return uint32_t((k >> 2) * (kNT * 128) + (k & 3) * 32); };
          uint32_t acc = in_round > 1;
          if (SPLIT)
            for (int k = 0; k < steps; ++k) {
              mma_tf32_ta(td, al + 8 * k, sw128_kmajor(bh + off(k)), idesc, acc);
              acc = 1;
              mma_tf32_ta(td, ah + 8 * k, sw128_kmajor(bl + off(k)), idesc, 1);
            }
          for (int k = 0; k < steps; ++k) {
            mma_tf32_ta(td, ah + 8 * k, sw128_kmajor(bh + off(k)), idesc, acc);
            acc = 1;
          }
          mma_commit(&sh.aempty[ab]);
          if (last) mma_commit(&sh.dfull[db]);
        }
        __syncwarp();
        if (last) in_round = 0, ++ri;
      }
    }
    if (lane == 0) {
      mma_commit(&sh.fin);
      mbar_wait_for(&sh.fin, 0, kDrainLimitNs);
    }
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 13) {
    fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// One (entry, type) per blockIdx.x, kJoinRows input channels per blockIdx.y: zeros
// for a type without nodes, the sum of the partial tiles in CTA order for one whose
// rows are spread over several shares, nothing otherwise.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(256) k_linear_grad_join(const __grid_constant__ LinGrad P, int ctas,
                                                          const float* __restrict__ part) {
  __shared__ int total[4];
  __shared__ int s_before, s_n;
  count_chunks(P, total);
  const int t = blockIdx.x % P.T;
  int e = blockIdx.x / P.T, p = 0;
  while (e >= tiles_u(P.p[p]) * tiles_w(P.p[p])) e -= tiles_u(P.p[p]) * tiles_w(P.p[p]), ++p;
  const LinPath& L = P.p[p];
  const int u0 = e / tiles_w(L) * kMT, w0 = e % tiles_w(L) * kNT;
  const int cu = min(kMT, L.ci - u0), cw = min(kNT, L.co - w0);
  if (threadIdx.x >= 128 && threadIdx.x < 160) {  // chunks of the types before t, and of t
    const int lane = threadIdx.x & 31, unit = chunk_nodes(L.d);
    int before = 0, n = 0;
    for (int k = lane; k <= t; k += 32) {
      int b, g;
      lin_group(P.offsets, P.T, P.N, k, &b, &g);
      const int c = (g - b + unit - 1) / unit;
      if (k < t) before += c;
      else n = c;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_before = before, s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  float* dw = P.dw + int64_t(t) * P.wnumel + L.woff + int64_t(u0) * L.co + w0;
  const int r0 = blockIdx.y * kJoinRows, r1 = min(cu, r0 + kJoinRows);
  int b0 = 0, b1 = -1;
  int64_t all = 0, seg = 0;
  const int c = chunk_cost(L, u0, w0);
  if (n > 0) {
    all = total_cost(P, total);
    int64_t begin = 0;  // cost before the entry
    for (int k = 0; k <= p; ++k)
      for (int u = 0; u < tiles_u(P.p[k]); ++u)
        for (int w = 0; w < tiles_w(P.p[k]); ++w)
          if (k < p || u * kMT < u0 || (u * kMT == u0 && w * kNT < w0))
            begin += int64_t(total[P.p[k].d >> 1]) * chunk_cost(P.p[k], u * kMT, w * kNT);
    seg = begin + int64_t(s_before) * c;
    // the share that holds the chunk whose cost begins at x
    auto owner = [&](int64_t x) {
      int b = int(x * ctas / all);
      while (b > 0 && x < share_begin(all, b, ctas)) --b;
      while (b + 1 < ctas && x >= share_begin(all, b + 1, ctas)) ++b;
      return b;
    };
    b0 = owner(seg);
    b1 = owner(seg + int64_t(n - 1) * c);
    if (b0 == b1) return;
  }
  for (int i = threadIdx.x; i < (r1 - r0) * cw; i += 256) {
    const int r = r0 + i / cw, w = i % cw;
    float s = 0.f;
    for (int b = b0; b <= b1; ++b) {
      if (b > b0) {  // a share narrower than a chunk's cost may hold none
        const int64_t k = (share_begin(all, b, ctas) - seg + c - 1) / c;
        if (seg + k * c >= share_begin(all, b + 1, ctas)) continue;
      }
      s += part[(int64_t(b == b0 ? 2 * b + 1 : 2 * b) * kMT + r) * kNT + w];
    }
    dw[int64_t(r) * L.co + w] = s;
  }
}

constexpr int kSMs = 148;

// one CTA per SM, or per chunk where there are fewer (an upper bound)
int ctas_of(const LinPath* path, int n, int T, int64_t N) {
  int64_t c = 0;
  for (int p = 0; p < n && c < kSMs; ++p)
    c += (N / chunk_nodes(path[p].d) + std::min<int64_t>(T, N)) * tiles_u(path[p]) * tiles_w(path[p]);
  return int(std::max<int64_t>(1, std::min<int64_t>(kSMs, c)));
}

}  // namespace

bool linear_grad_tc_supported(const LinGrad& G) {
  const auto bad = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  if (G.dim_x % 4 || G.dim_g % 4 || bad(G.x) || bad(G.g) || bad(G.dw)) return false;
  int entries = 0;
  for (int p = 0; p < G.n_paths; ++p) {
    const LinPath& L = G.p[p];
    if (L.ci % 4 || L.co % 4 || L.xoff % 4 || L.goff % 4) return false;
    entries += tiles_u(L) * tiles_w(L);
  }
  return entries <= kLinGradTcEntries;
}

size_t linear_grad_tc_bytes(const LinPath* path, int n, int T, int64_t N) {
  return size_t(2) * ctas_of(path, n, T, N) * kMT * kNT * 4;
}

cudaError_t linear_grad_tc(const LinGrad& G, bool split, float* part, uint64_t limit, cudaStream_t st) {
  int sx = 0, sg = 0, entries = 0;
  for (int p = 0; p < G.n_paths; ++p) {
    const LinPath& L = G.p[p];
    sx = std::max(sx, std::min(kMT, L.ci) * L.d * chunk_nodes(L.d) * 4);
    sg = std::max(sg, std::min(kNT, L.co) * L.d * chunk_nodes(L.d) * 4);
    entries += tiles_u(L) * tiles_w(L);
  }
  const int stage = (sx + sg + 127) & ~127;
  const int room = kSMemMax - 1024 - int(sizeof(Shared)) - 256 - 4 * kBTile;
  const int stages = std::min(kMaxStages, room / stage);
  if (stages < 2) return cudaErrorInvalidValue;
  const int sm = 1024 + 4 * kBTile + stages * stage;
  auto* k = split ? k_linear_grad_tc<true> : k_linear_grad_tc<false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
  if (e) return e;
  const int ctas = ctas_of(G.p, G.n_paths, G.T, G.N);
  k<<<ctas, kThreads, sm, st>>>(G, stages, stage, sx, part, limit);
  if ((e = cudaGetLastError())) return e;
  k_linear_grad_join<<<dim3(unsigned(entries * G.T), kMT / kJoinRows), 256, 0, st>>>(G, ctas, part);
  return cudaGetLastError();
}

cudaError_t linear_grad_tc_read_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_linear_grad_error, sizeof(int));
  if (e) return e;
  return *code ? cudaMemcpyToSymbol(g_linear_grad_error, &zero, sizeof(int)) : cudaSuccess;
}

}  // namespace tpc
