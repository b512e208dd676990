// Weight gradient of the typed linear map on the tensor cores (sm_100a: tcgen05
// with one operand in TMEM, bulk copies of node rows).
//
//   dW[t][u][w] = sum over the (node, m) rows of type t of x[n, u, m] g[n, w, m]
//
// per path, 128 input channels and 64 output channels: a product whose depth is the
// ragged row count of the type.  A chunk is the rows of 64, 21, 12 or 9 nodes
// (l = 0..3: 64, 63, 60, 63 rows, filled up with zeros); copy warps gather the nodes'
// pieces of x and g by perm, a bulk copy each (4-byte asynchronous copies where a block
// or tensor is not 16-byte aligned).  The A operand is x transposed: thread u reads its channel of every row (the
// lanes of a warp are 2l+1 floats apart: no bank conflicts), splits it (3xTF32) and
// stores hi and lo to TMEM, lane = u, column = row.  The B operand is g: thread w
// reads its channel and writes hi and lo into the K-major 128-byte-swizzled tile, lo
// as further columns.  One thread issues (D1 | D2) += A_hi (B_hi | B_lo) and
// D2 += A_lo B_hi.  After kRound chunks the accumulator's bank is added into fp32
// registers (round to nearest), which bounds the chain of tensor-core additions
// whatever the number of rows.
//
// The (path, channel tile) entries x types x chunks are cut into one equal share per
// CTA.  A type's rows that lie in one share are stored straight into dW; a share
// that begins or ends inside a type stores a partial tile (at most two per CTA), and
// k_linear_grad_join adds a type's partial tiles in the order of the CTAs: no
// atomics, the same bits every time.  It also clears the weights of empty types.
//
// Bound: HBM (x and g read once), next to shared memory: a row of 64 + 64 channels
// is 512 B from HBM and about 2.3 KB of shared-memory traffic.
// Two sets of warps convert every second chunk each (the latency of a chunk's steps is
// what bounds it): warps 0-3 and 8-11 x, 4-7 and 12-15 g; 16-23 add finished banks (32
// columns each) and store, 24-29 copy, 30 issues the MMAs.  Waits are bounded as in the
// row kernel.
// Measured (device, 3xTF32): 262144 nodes of 64x0e+64x1o+64x2e, 16 types: 302 us with the
// join (7), 4.0 TB/s, 0.61 of the measured copy rate; one set of converters: 469 us.
// No unit is near its limit (issue slots 51 %, tensor pipe 32 %, shared memory 31 %): the
// steps of a chunk, one after another, bound it.  The threads leave 64 registers each, and
// 3xTF32 spills 104 bytes of them (136 where pieces are not aligned).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>

#include "chain.cuh"
#include "linear_grad_tc.h"
#include "linear_tc_common.cuh"

namespace tpc {
namespace {

using namespace tc;

__device__ int g_linear_grad_error;  // first code recorded by an expired wait (0 = none)

constexpr int kSMs = 148;                     // CTAs of a call, at most
constexpr int kMT = 128, kNT = 64;            // input and output channels of a tile
constexpr int kKMax = 64;                     // rows of a chunk, at most
constexpr int kRound = 2;                     // chunks accumulated in TMEM before they are added up
constexpr int kBHalf = 2 * kNT * 128;         // 32 rows of B: 64 columns' hi and behind them their lo
constexpr int kBTile = 2 * kBHalf;
constexpr int kMaxStages = 4;                 // raw chunks, an even number
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 992;
constexpr int kCopyWarps = 6, kCopy = 32 * kCopyWarps;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 2 * kKMax, kTmemD = 256, kTmemDStage = 128;  // A: hi | lo, D: D1 | D2

// nodes and rows of a chunk
__host__ __device__ constexpr int chunk_nodes(int d) { return kKMax / d; }

// (path, 128 input channels, 64 output channels)
struct Entry {
  int d;            // 2l+1
  int xoff, goff;   // first columns in x and g
  int cu, cw;       // channels
  int co;           // output channels of the path: the pitch of its weight
  int64_t woff;     // first weight
};
struct Params {
  int n_entries, T, dim_x, dim_g;
  int64_t N, wnumel;
  const float *x, *g;
  float* dw;
  const int *perm, *offsets;
  int coef[4];  // cost of a chunk of d = 1, 3, 5, 7, summed over the entries
  Entry e[kLinGradTcEntries];
  Cut cut[kLinGradTcEntries];
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t afull[2], aempty[2], dfull[2], dempty[2], fin;
  uint32_t tmem;
  int abort;
  int total[4];  // chunks of all types for d = 1, 3, 5, 7
  WalkState walk[kThreads / 32];
  int node[2][64];
  int issued[kCopyWarps];
};

constexpr int kDynMax = kSMemMax - int(sizeof(Shared)) - 64;  // dynamic shared memory of a call, at most

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_grad_error, code);
}

__device__ __forceinline__ int total_cost(const Params& P, const int* total) {
  int c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c += total[i] * P.coef[i];
  return c;
}

// a run of chunks of one type in one entry
struct Piece {
  int e, t, end, nodes;  // (counted down to `end`: a step past it would pass 2^31 in the largest graphs)
  int slot;  // partial tile, or -1: the type's rows are all here
};

struct Walk {
  WalkState* w;
  const Cut* cuts;
  const int *total, *offs;
  int n, T;

  __device__ __forceinline__ bool next(Piece* q) {
    const Run r = next_run(w, cuts, n, total, offs, T);
    if (r.e < 0) return false;
    const bool begins = r.first == offs[r.t], ends = r.end == offs[r.t + 1];
    q->e = r.e, q->t = r.t, q->end = r.end, q->nodes = r.end - r.first;
    q->slot = begins && ends ? -1 : 2 * int(blockIdx.x) + begins;
    return true;
  }
};

// 16 rows from K0 of the thread's channel, split (zeros at and behind kv).  The pitch is
// hidden from the compiler, which would keep a register for every node's offset.
template <int D, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void read16(const float* col, int pitch, int k0, int kv, float (&h)[16], float (&l)[16]) {
  asm volatile("" : "+r"(pitch));
  const float* row = col + (k0 / D) * pitch;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int k = k0 + i;
    const float v = (WHOLE ? k < chunk_nodes(D) * D : k < kv) ? row[k % D] : 0.f;
    if (k % D == D - 1) row += pitch;
    tf32_split<SPLIT>(v, h[i], l[i]);
  }
}
template <int D, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void convert_a(const float* col, int pitch, int kv, uint32_t ta) {
#pragma unroll
  for (int k0 = 0; k0 < kKMax; k0 += 16) {
    if (!WHOLE && k0 >= kv) break;
    float h[16], l[16];
    read16<D, SPLIT, WHOLE>(col, pitch, k0, kv, h, l);
    tmem_st16(ta + k0, h);
    if (SPLIT) tmem_st16(ta + kKMax + k0, l);
  }
}
// thread (w, half): every second group of 16 rows of its channel, into the swizzled tile
template <int D, bool SPLIT, bool WHOLE, int HALF>
__device__ __forceinline__ void convert_b(const float* col, int pitch, int w, int n16, int kv, unsigned char* hi) {
#pragma unroll
  for (int k0 = 16 * HALF; k0 < kKMax; k0 += 32) {
    if (!WHOLE && k0 >= kv) break;
    float h[16], l[16];
    read16<D, SPLIT, WHOLE>(col, pitch, k0, kv, h, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = k0 / 4 + i;  // 16-byte column of the tile; the lo rows begin at a multiple of 16
      unsigned char* to = hi + (j >> 3) * kBHalf + w * 128 + (((j & 7) ^ (w & 7)) << 4);
      *reinterpret_cast<float4*>(to) = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
      if (SPLIT) *reinterpret_cast<float4*>(to + n16 * 128) = make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
    }
  }
}
// one chunk of an operand; whole chunks without a test per row.  Columns of B behind
// the channels repeat the last one: what they give is not stored.
template <int D, bool SPLIT>
__device__ __forceinline__ void chunk_a(const float* raw, int u, int cu, int kv, uint32_t ta) {
  const float* col = raw + min(u, cu - 1) * D;
  if (kv == chunk_nodes(D) * D)
    convert_a<D, SPLIT, true>(col, cu * D, kv, ta);
  else
    convert_a<D, SPLIT, false>(col, cu * D, kv, ta);
}
template <int D, bool SPLIT>
__device__ __forceinline__ void chunk_b(const float* raw, int t, int cw, int kv, unsigned char* hi) {
  const int w = t & 63, n16 = (cw + 15) & ~15;
  if (w >= n16) return;
  const float* col = raw + min(w, cw - 1) * D;
  if (kv == chunk_nodes(D) * D) {
    if (t < 64)
      convert_b<D, SPLIT, true, 0>(col, cw * D, w, n16, kv, hi);
    else
      convert_b<D, SPLIT, true, 1>(col, cw * D, w, n16, kv, hi);
  } else {
    if (t < 64)
      convert_b<D, SPLIT, false, 0>(col, cw * D, w, n16, kv, hi);
    else
      convert_b<D, SPLIT, false, 1>(col, cw * D, w, n16, kv, hi);
  }
}

template <bool SPLIT, int VEC>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_grad_tc(const __grid_constant__ Params P, int stages, int stage_bytes, int g_offset,
                     float* __restrict__ part, uint64_t limit) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sB = base;  // of each set
  unsigned char* sRaw = base + 2 * kBTile;
  Entry* E = reinterpret_cast<Entry*>(sRaw + stages * stage_bytes);
  Cut* cuts = reinterpret_cast<Cut*>(E + P.n_entries);
  int* offs = reinterpret_cast<int*>(cuts + P.n_entries);
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  chain_next();
  for (int i = threadIdx.x; i < P.n_entries * int(sizeof(Entry) / 4); i += kThreads)
    reinterpret_cast<int*>(E)[i] = reinterpret_cast<const int*>(P.e)[i];
  for (int i = threadIdx.x; i < P.n_entries * int(sizeof(Cut) / 4); i += kThreads)
    reinterpret_cast<int*>(cuts)[i] = reinterpret_cast<const int*>(P.cut)[i];
  load_offsets(offs, P.offsets, P.T, P.N);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh.full[s], VEC == 4 ? kCopyWarps : kCopy);
      mbar_init(&sh.empty[s], 256);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.afull[i], 256);
      mbar_init(&sh.aempty[i], 1);
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 256);
    }
    mbar_init(&sh.fin, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 30) tmem_alloc(&sh.tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem;
  if (warp < 4) {
    const int n = count_units(offs, P.T, chunk_nodes(2 * warp + 1));
    if (lane == 0) sh.total[warp] = n;
  }
  __syncthreads();

  walk_begin(&sh.walk[warp], total_cost(P, sh.total));
  Walk walk{&sh.walk[warp], cuts, sh.total, offs, P.n_entries, P.T};
  Piece q;
  bool ok = true;
  int ci = 0;  // chunks so far
  if (warp < 16) {
    // ---- operands: chunks of the set's parity ----
    const bool is_a = (warp & 7) < 4;
    const int set = warp >> 3;
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemA;
    const int t = threadIdx.x & 127;
    while (ok && walk.next(&q)) {
      const Entry& L = E[q.e];
      const int d = L.d, cu = L.cu, cw = L.cw, nq = chunk_nodes(d);
      const int end = ci + units_of(q.nodes, nq), tail = (q.nodes - (end - ci - 1) * nq) * d;  // rows of the last
      for (; ci < end; ++ci) {
        if ((ci & 1) != set) continue;
        const int st = ci % stages, ab = set, kv = ci + 1 < end ? nq * d : tail;
        if (ci >= 2 && !wait(&sh.aempty[ab], ((ci >> 1) + 1) & 1, limit, abort, 1)) ok = false;
        if (ok && !wait(&sh.full[st], (ci / stages) & 1, limit, abort, 2)) ok = false;
        if (!ok) break;
        const unsigned char* raw = sRaw + st * stage_bytes;
        if (is_a) {
          fence_after_sync();
          const float* rx = reinterpret_cast<const float*>(raw);
          const uint32_t ta = lane_base + ab * kTmemAStage;
          if ((warp & 3) * 32 < cu) {  // (rows of the product behind the channels are not stored)
            switch (d) {
              case 1: chunk_a<1, SPLIT>(rx, t, cu, kv, ta); break;
              case 3: chunk_a<3, SPLIT>(rx, t, cu, kv, ta); break;
              case 5: chunk_a<5, SPLIT>(rx, t, cu, kv, ta); break;
              default: chunk_a<7, SPLIT>(rx, t, cu, kv, ta); break;
            }
          }
          mbar_arrive(&sh.empty[st]);
          tmem_wait_st();
          fence_before_sync();
        } else {
          const float* rg = reinterpret_cast<const float*>(raw + g_offset);
          unsigned char* hi = sB + ab * kBTile;
          switch (d) {
            case 1: chunk_b<1, SPLIT>(rg, t, cw, kv, hi); break;
            case 3: chunk_b<3, SPLIT>(rg, t, cw, kv, hi); break;
            case 5: chunk_b<5, SPLIT>(rg, t, cw, kv, hi); break;
            default: chunk_b<7, SPLIT>(rg, t, cw, kv, hi); break;
          }
          mbar_arrive(&sh.empty[st]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        mbar_arrive(&sh.afull[ab]);
      }
    }
  } else if (warp < 24) {
    // ---- finished banks to registers, pieces to memory: a row and 32 columns a thread ----
    const int r = threadIdx.x & 127, c0 = 32 * ((warp - 16) >> 2);
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemD;
    int ri = 0;  // rounds so far
    while (ok && walk.next(&q)) {
      const Entry& L = E[q.e];
      const int cu = L.cu, cw = L.cw, nq = chunk_nodes(L.d);
      const int rounds = (units_of(q.nodes, nq) + kRound - 1) / kRound;
      const bool mine = (warp & 3) * 32 < cu && c0 < cw;
      float acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = 0.f;
      for (int k = 0; k < rounds; ++k, ++ri) {
        const int db = ri & 1;
        if (!wait(&sh.dfull[db], (ri >> 1) & 1, limit, abort, 3)) {
          ok = false;
          break;
        }
        fence_after_sync();
        if (mine) {
          const uint32_t td = lane_base + db * kTmemDStage + c0;
#pragma unroll
          for (int p = 0; p < (SPLIT ? 2 : 1); ++p)
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
              float v[16];
              tmem_ld16(td + p * ((cw + 15) & ~15) + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
            }
        }
        fence_before_sync();
        mbar_arrive(&sh.dempty[db]);
      }
      if (!ok || !mine || r >= cu) continue;
      if (q.slot >= 0) {  // a partial tile has room for all columns
        float4* dst = reinterpret_cast<float4*>(part + (int64_t(q.slot) * kMT + r) * kNT + c0);
#pragma unroll
        for (int i = 0; i < 32; i += 4) dst[i / 4] = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      } else {
        float* dst = P.dw + int64_t(q.t) * P.wnumel + L.woff + int64_t(r) * L.co + c0;
#pragma unroll
        for (int i = 0; i < 32; i += VEC) {
          if (c0 + i < cw) {
            if constexpr (VEC == 4)
              *reinterpret_cast<float4*>(dst + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            else
              dst[i] = acc[i];
          }
        }
      }
    }
  } else if (warp < 30) {
    // ---- node rows to shared memory, several chunks ahead ----
    const int r = threadIdx.x - 768;
    if constexpr (VEC == 4) {
      // a bulk copy per node and tensor, dealt out over the warps (issuing one takes some
      // 60 cycles): copy i of a chunk is node i / 2 of x or g
      static_assert(kCopy >= 2 * kKMax, "a copy a thread");
      const int w = warp - 24, i0 = lane * kCopyWarps + w;
      while (ok && walk.next(&q)) {
        const Entry& L = E[q.e];
        const int d = L.d, nq = chunk_nodes(d), lx = L.cu * d, lg = L.cw * d;
        const bool is_g = i0 & 1;
        const float* src = is_g ? P.g + L.goff : P.x + L.xoff;
        const int dim = is_g ? P.dim_g : P.dim_x;
        const uint32_t bytes = uint32_t(is_g ? lg : lx) * 4;
        auto node_of = [&](int k, int left) {  // of a chunk, from which on `left` nodes are left
          const int n = k < left ? P.perm[q.end - left + k] : 0;
          return n >= 0 && n < P.N ? n : 0;
        };
        const int k = i0 / 2;
        int node = k < nq ? node_of(k, q.nodes) : 0;  // of the next chunk, read while this one is copied
        for (int left = q.nodes; left > 0; left -= nq, ++ci) {
          const int st = ci % stages, cnt = min(nq, left);
          const float* from = src + int64_t(node) * dim;
          if (k < nq && left > nq) node = node_of(k, left - nq);
          if (r < 2) prefetch_nodes(P.perm, unsigned(q.end - left) + kPermAhead + 32 * r, P.N);
          const uint32_t mine = __reduce_add_sync(0xffffffffu, k < cnt ? bytes : 0u);
          if (ci >= stages && !wait(&sh.empty[st], ((ci / stages) + 1) & 1, limit, abort, 4)) ok = false;
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&sh.full[st], mine);
          __syncwarp();
          if (k < cnt)
            bulk_load(smem_u32(sRaw + st * stage_bytes) + (is_g ? g_offset : 0) + k * bytes, from, bytes, &sh.full[st]);
        }
      }
      if (lane == 0) sh.issued[w] = ci;
      asm volatile("bar.sync 1, 192;" ::: "memory");
      drain_ring(sh.full, stages, ci, sh.issued, kCopyWarps);
    } else {
      while (walk.next(&q)) {  // (a warp that gave up keeps passing the group's barriers)
        const Entry& L = E[q.e];
        const int d = L.d, nq = chunk_nodes(d), lx = L.cu * d, lg = L.cw * d;
        const float *x = P.x + L.xoff, *g = P.g + L.goff;
        // the nodes of the next chunk are read while this one is copied
        int node = r < min(nq, q.nodes) ? P.perm[q.end - q.nodes + r] : 0;
        for (int left = q.nodes; left > 0; left -= nq, ++ci) {
          const int st = ci % stages, cnt = min(nq, left);
          int* nodes = sh.node[ci & 1];
          if (r < 64) nodes[r] = (node >= 0 && node < P.N) ? node : 0;
          asm volatile("bar.sync 1, 192;" ::: "memory");
          node = r < nq && r < left - nq ? P.perm[q.end - left + nq + r] : 0;
          if (r < 2) prefetch_nodes(P.perm, unsigned(q.end - left) + kPermAhead + 32 * r, P.N);
          if (ok && ci >= stages && !wait(&sh.empty[st], ((ci / stages) + 1) & 1, limit, abort, 4)) ok = false;
          if (!ok) continue;
          const uint32_t dst = smem_u32(sRaw + st * stage_bytes);
          auto rows = [&](const float* src, int dim, int len, uint32_t to0) {
            const RowShare w(len, r, kCopy);
            for (int o = w.at; o < len; o += w.pieces)
              copy_rows(src + o, dim, nodes, w, cnt, to0 + (w.row * len + o) * 4, len * 4);
          };
          rows(x, P.dim_x, lx, dst);
          rows(g, P.dim_g, lg, dst + g_offset);
          copies_arrive(&sh.full[st]);
        }
      }
      copies_wait_all();  // no copy may be in flight when the CTA ends
    }
  } else {
    // ---- MMAs ----
    int ri = 0;
    while (ok && walk.next(&q)) {
      const Entry& L = E[q.e];
      const int d = L.d, nq = chunk_nodes(d);
      const int n16 = (L.cw + 15) & ~15;
      const uint32_t id1 = idesc_tf32(kMT, SPLIT ? 2 * n16 : n16), id2 = idesc_tf32(kMT, n16);
      int in_round = 0;
      for (int left = q.nodes; left > 0; left -= nq, ++ci) {
        const int ab = ci & 1, db = ri & 1, steps = (min(nq, left) * d + 7) / 8;
        if (in_round == 0 && ri >= 2 && !wait(&sh.dempty[db], ((ri >> 1) + 1) & 1, limit, abort, 5)) ok = false;
        if (ok && !wait(&sh.afull[ab], (ci >> 1) & 1, limit, abort, 6)) ok = false;
        if (!ok) break;
        fence_after_sync();
        const bool last = ++in_round == kRound || left <= nq;
        if (lane == 0) {
          const uint32_t td = tmem + kTmemD + db * kTmemDStage, a = tmem + kTmemA + ab * kTmemAStage;
          const uint64_t b = sw128_kmajor(smem_u32(sB + ab * kBTile));
#pragma unroll
          for (int k = 0; k < kKMax / 8; ++k) {
            if (k >= steps) break;
            const uint64_t bk = b + uint64_t((k >> 2) * (kBHalf / 16) + (k & 3) * 2);
            mma_tf32_ta(td, a + 8 * k, bk, id1, in_round > 1 || k > 0);
            if (SPLIT) mma_tf32_ta(td + n16, a + kKMax + 8 * k, bk, id2, 1);
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
  if (warp == 30) {
    fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
    chain_wait();
  }
}

// One (entry, type) per blockIdx.x, 16 input channels per blockIdx.y: zeros
// for a type without nodes, the sum of the partial tiles in CTA order for one whose
// rows are spread over several shares, nothing otherwise.
constexpr int kJoinRows = 16;  // 16 float4 of 64 columns a row: 256 threads
static_assert(kJoinRows * kNT / 4 == 256, "one float4 a thread");
__global__ void __launch_bounds__(256) k_linear_grad_join(const __grid_constant__ Params P, int ctas,
                                                          const float* part) {
  __shared__ int offs[TPCONV_MAX_TYPES + 2];
  __shared__ int total[4], s_slots, slot[kSMs];
  const int t = blockIdx.x % P.T, e = blockIdx.x / P.T, warp = threadIdx.x >> 5;
  const Entry& L = P.e[e];
  load_offsets(offs, P.offsets, P.T, P.N);
  __syncthreads();
  if (warp < 4) {
    const int n = count_units(offs, P.T, chunk_nodes(2 * warp + 1));
    if ((threadIdx.x & 31) == 0) total[warp] = n;
  }
  __syncthreads();
  chain_wait();
  const int r0 = blockIdx.y * kJoinRows, r1 = min(L.cu, r0 + kJoinRows), cw = L.cw;
  if (r0 >= r1) return;
  if (warp == 0) {
    // the slots of the type's pieces
    const int unit = chunk_nodes(L.d), n = group_units(offs, t, unit), c = P.cut[e].cost;
    int m = -1;
    if (n == 0) {
      m = 0;
    } else {
      const int all = total_cost(P, total);
      int seg = count_units(offs, t, unit) * c;  // cost before the type's first chunk
      for (int k = 0; k < e; ++k) seg += total[P.cut[k].which] * P.cut[k].cost;
      const int end = seg + (n - 1) * c;  // cost before its last chunk
      // the shares that hold the first and the last chunk
      const int per = all / ctas, more = all - per * ctas, wide = more * (per + 1);
      auto owner = [&](int x) { return x < wide ? x / (per + 1) : more + (x - wide) / max(per, 1); };
      // (within the CTAs whatever the offsets say: groups that overlap cost more than was planned for)
      const int first = min(max(owner(seg), 0), ctas - 1), last = min(max(owner(end), 0), ctas - 1);
      m = 0;
      for (int b0 = first; b0 <= last; b0 += 32) {
        const int b = b0 + threadIdx.x;
        bool has = b == first;
        if (b > first && b <= last) {  // a share narrower than a chunk's cost may hold none
          const int lo = per * b + min(b, more), hi = per * (b + 1) + min(b + 1, more);
          has = seg + (lo - seg + c - 1) / c * c < hi;
        }
        const unsigned mask = __ballot_sync(0xffffffffu, has);
        if (has) slot[m + __popc(mask & ((1u << threadIdx.x) - 1))] = 2 * b + (b == first);
        m += __popc(mask);
      }
      if (m == 1) m = -1;  // all in one share: stored by its CTA
    }
    if (threadIdx.x == 0) s_slots = m;
  }
  __syncthreads();
  const int m = s_slots;
  if (m < 0) return;
  // a float4 of the partial tiles a thread (their rows have room for 64 columns)
  const int r = r0 + (threadIdx.x >> 4), w = 4 * (threadIdx.x & 15);
  if (r >= r1 || w >= cw) return;
  const float* p0 = part + int64_t(r) * kNT + w;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int b = 0; b < m; ++b) {
    const float4 v = *reinterpret_cast<const float4*>(p0 + int64_t(slot[b]) * kMT * kNT);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  float* dw = P.dw + int64_t(t) * P.wnumel + L.woff + int64_t(r) * L.co + w;
  dw[0] = s.x;
  if (w + 1 < cw) dw[1] = s.y;
  if (w + 2 < cw) dw[2] = s.z;
  if (w + 3 < cw) dw[3] = s.w;
}

int tiles_u(const LinPath& p) { return (p.ci + kMT - 1) / kMT; }
int tiles_w(const LinPath& p) { return (p.co + kNT - 1) / kNT; }

// one CTA per SM, or per chunk where there are fewer (an upper bound)
int ctas_of(const LinPath* path, int n, int T, int64_t N) {
  int64_t c = 0;
  for (int p = 0; p < n && c < kSMs; ++p)
    c += (N / chunk_nodes(path[p].d) + std::min<int64_t>(T, N)) * tiles_u(path[p]) * tiles_w(path[p]);
  return int(std::max<int64_t>(1, std::min<int64_t>(kSMs, c)));
}

bool vec4(const LinGrad& G) {
  const auto bad = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  if (G.dim_x % 4 || G.dim_g % 4 || G.wnumel % 4 || bad(G.x) || bad(G.g) || bad(G.dw)) return false;
  for (int p = 0; p < G.n_paths; ++p) {
    const LinPath& L = G.p[p];
    if (L.ci % 4 || L.co % 4 || L.xoff % 4 || L.goff % 4 || L.woff % 4) return false;
  }
  return true;
}

}  // namespace

bool linear_grad_tc_plan(const LinPath* path, int n) {
  int entries = 0;
  for (int p = 0; p < n; ++p) entries += tiles_u(path[p]) * tiles_w(path[p]);
  return entries <= kLinGradTcEntries;
}

bool linear_grad_tc_supported(const LinPath* path, int n, int T, int64_t N) {
  int64_t chunks = 0;
  for (int p = 0; p < n; ++p) chunks += (N / chunk_nodes(path[p].d) + T) * tiles_u(path[p]) * tiles_w(path[p]);
  return linear_grad_tc_plan(path, n) && chunks < kMostCost;
}

size_t linear_grad_tc_bytes(const LinPath* path, int n, int T, int64_t N) {
  return size_t(2) * ctas_of(path, n, T, N) * kMT * kNT * 4;
}

cudaError_t linear_grad_tc(const LinGrad& G, bool split, float* part, uint64_t limit, bool after, cudaStream_t st) {
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.T = G.T, P.dim_x = G.dim_x, P.dim_g = G.dim_g, P.N = G.N, P.wnumel = G.wnumel;
  P.x = G.x, P.g = G.g, P.dw = G.dw, P.perm = G.perm, P.offsets = G.offsets;
  int sx = 0, sg = 0;
  for (int p = 0; p < G.n_paths; ++p) {
    const LinPath& L = G.p[p];
    for (int u0 = 0; u0 < L.ci; u0 += kMT)
      for (int w0 = 0; w0 < L.co; w0 += kNT) {
        Entry& E = P.e[P.n_entries++];
        E.d = L.d, E.xoff = L.xoff + u0 * L.d, E.goff = L.goff + w0 * L.d;
        E.cu = std::min(kMT, L.ci - u0), E.cw = std::min(kNT, L.co - w0), E.co = L.co;
        E.woff = L.woff + int64_t(u0) * L.co + w0;
        // the KB that a chunk moves, what any chunk takes, and more where the copies of a
        // chunk take long to issue (l = 0: 1.4 times the others)
        P.cut[P.n_entries - 1] = {16 + (E.cu + E.cw) * L.d * chunk_nodes(L.d) / 256 +
                                      std::max(0, 2 * chunk_nodes(L.d) - 40) / 4,
                                  chunk_nodes(L.d), L.d >> 1};
        sx = std::max(sx, E.cu * L.d * chunk_nodes(L.d) * 4);
        sg = std::max(sg, E.cw * L.d * chunk_nodes(L.d) * 4);
      }
  }
  const int shift = cost_shift(P.cut, P.n_entries, G.N, G.T);
  for (int i = 0; i < P.n_entries; ++i) {
    P.cut[i].cost = std::max(1, P.cut[i].cost >> shift);
    P.coef[P.cut[i].which] += P.cut[i].cost;
  }
  sx = (sx + 15) & ~15;
  const int stage = (sx + sg + 15) & ~15;
  const int fixed = 1024 + 2 * kBTile + P.n_entries * int(sizeof(Entry) + sizeof(Cut)) + (P.T + 2) * 4;
  // at most 32 KB of x and 16 KB of g: two stages always fit; an even number, so that a stage
  // belongs to one set of converters
  const int stages = std::min(kMaxStages, (kDynMax - fixed) / stage) & ~1;
  if (stages < 2) return cudaErrorInvalidValue;
  const int sm = fixed + stages * stage;
  const bool v = vec4(G);
  auto* k = split ? (v ? k_linear_grad_tc<true, 4> : k_linear_grad_tc<true, 1>)
                  : (v ? k_linear_grad_tc<false, 4> : k_linear_grad_tc<false, 1>);
  // (the most a call may ask for, not this call's: another thread's call must not lower it)
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynMax);
  if (e) return e;
  const int ctas = ctas_of(G.p, G.n_paths, G.T, G.N);
  if (after) {
    if ((e = chain_launch(k, ctas, kThreads, sm, st, P, stages, stage, sx, part, limit))) return e;
  } else {
    k<<<ctas, kThreads, sm, st>>>(P, stages, stage, sx, part, limit);
    if ((e = cudaGetLastError())) return e;
  }
  return chain_launch(k_linear_grad_join, dim3(unsigned(P.n_entries * G.T), kMT / kJoinRows), 256, 0, st, P, ctas,
                      static_cast<const float*>(part));
}

cudaError_t linear_grad_tc_read_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_linear_grad_error, sizeof(int));
  if (e) return e;
  return *code ? cudaMemcpyToSymbol(g_linear_grad_error, &zero, sizeof(int)) : cudaSuccess;
}

}  // namespace tpc
