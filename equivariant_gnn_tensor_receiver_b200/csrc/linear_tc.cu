// Typed linear map on the tensor cores: rows times the weight of their type
// (sm_100a: tcgen05 with the row operand in TMEM, gathers by asynchronous copies).
//
//   out[n, w, m] = sum_k x[n, k, m] B_t[k][w]     per (output block, 64 columns, type t)
//
// A tile is the (node, m) rows of up to 128 / (2l+1) nodes of one type, times 64
// output channels.  The weight of the (block, columns, type) is resident in shared
// memory, split once into TF32 hi and lo; the node rows are the only stream:
//   copy threads gather the nodes' contiguous pieces [64 channels][2l+1] by perm, 16
//   bytes a thread (4 where a block or tensor is not aligned for it), several chunks
//   ahead;
//   converter threads, one per row, read their row's channels (stride 2l+1), split
//   them (3xTF32, Ootomo & Yokota, 2022) and store hi and lo as the A operand in
//   TMEM: the transposition from [channel][m] to rows costs one shared-memory read
//   per element and no write;
//   one thread issues, 8 channels a step, (D1 | D2) += A_hi (B_hi | B_lo) as one product
//   of up to 128 columns, and D2 += A_lo B_hi: two instructions instead of three, and
//   the small products add up among themselves;
//   epilogue threads, one per row and 32 columns, lay D1 + D2 out as [channel][m] in
//   shared memory, and store the nodes' pieces, 16 bytes a thread.
// The pitch of a node in shared memory is 4 or 8 floats off a multiple of 32, which
// leaves at most two rows of a warp on a bank.
//
// Bound: HBM for up to 128 channels (each row read and written once: a node of
// 64 channels at l <= 2 moves 4.6 KB and takes 0.22 MFLOP in three TF32 products).
// With several 64-column tiles (more than 64 output channels) the rows are read
// once per column tile, at about the same time, so mostly from L2.
//
// One persistent CTA per SM takes an equal share of the (block, columns) x types x
// tiles list, in order, so that its weight changes rarely; the group sizes are read
// from the device.  Warps 0-7 convert (two per 32 rows, 32 channels each), 8-15 run the
// epilogue (two per 32 rows, 32 columns each), 16-20 copy, 21 issues the MMAs: with one
// warpgroup for each role their latencies, not the issue slots (36 % busy), bounded
// the tile.  (Bulk copies of a node's piece were tried in place of the copy threads: about
// 60 cycles of issue a copy, 2.5 times the time at 64 scalars a node.)
// Every wait is bounded by the call's limit; on expiry the kernel records it, stops
// issuing, waits (bounded) for its own copies and MMAs, frees TMEM and returns.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>

#include "linear_tc.h"
#include "linear_tc_common.cuh"

namespace tpc {
namespace {

using namespace tc;

__device__ int g_linear_error;  // first code recorded by an expired wait (0 = none)

constexpr int kSMs = 148;
constexpr int kNT = 64, kKC = 64;             // columns of a tile, channels of a chunk
constexpr int kMaxChunks = kLinTcChunks;      // chunks of a resident weight
// one chunk of a weight: 32 channels behind 32 channels, each the rows of up to 64 output
// channels' hi and behind them their lo, 128 bytes a row (K-major, 128-byte swizzle)
constexpr int kWHalf = 2 * kNT * 32 * 4;
constexpr int kWChunk = 2 * kWHalf;
constexpr int kRaw = 32928;                   // a raw chunk or an output tile (see node_pitch)
constexpr int kMaxStages = 4;
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 704, kCopy = 160;     // copy threads: whole rows of 16, 48, 80, 112 pieces fill them
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 128, kTmemD = 256, kTmemDStage = 128;  // A: 2 x (hi 64 | lo 64), D: 2 x (D1 | D2)

// nodes of a tile; floats of a node's 64 channels plus padding (multiple of 4)
__host__ __device__ constexpr int tile_of(int d) { return d == 1 ? 120 : 128 / d; }
__host__ __device__ constexpr int node_pitch(int d) { return kKC * d + (d == 1 || d == 3 ? 4 : 8); }
static_assert(tile_of(1) * node_pitch(1) * 4 <= kRaw && tile_of(3) * node_pitch(3) * 4 <= kRaw &&
                  tile_of(5) * node_pitch(5) * 4 <= kRaw && tile_of(7) * node_pitch(7) * 4 <= kRaw,
              "a tile fits its buffer");

constexpr int chunks_of(int k) { return (k + kKC - 1) / kKC; }
constexpr int col_tiles(int n) { return (n + kNT - 1) / kNT; }

// (output block, 64 columns)
struct Entry {
  int d, cost;       // 2l+1; cost of a tile: its chunks plus one
  int off, nw;       // first output column, channels
  int c0;            // first channel of the block
  int first, count;  // sources
  int pad;
};
struct Params {
  int n_entries, n_src, T, dim_src, dim_out;
  int64_t N, wnumel;
  const float *x[2], *w[2];
  float* out;
  const int *perm, *offsets;
  int coef[4];  // cost of a tile of d = 1, 3, 5, 7, summed over the entries
  Entry e[kLinTcEntries];
  LinSource s[kLinSources];
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t afull[2], aempty[2], dfull[2], dempty[2], wfull, wfree, fin;
  uint32_t tmem;
  int abort;
  int total[4];                    // tiles of all types for d = 1, 3, 5, 7
  int node_in[2][128], node_out[2][128];
};

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_error, code);
}

// ---- the CTA's share of the work -------------------------------------------------
// Entries in order, in each the tiles of the types; CTA b owns the tiles whose cost
// begins in its share.  Every warp walks the same list.
struct Item {
  int e, t, first, count;
  bool run;       // the first tile with this weight
  bool run_last;  // the last tile of this CTA with this weight
  bool zero;      // no product: a block without a source
};

struct Walk {
  const Entry* E;
  const int* offs;
  const int* total;
  int n_entries, T;
  int64_t lo, hi, base = 0;
  int left = 0;                // tiles of this share left in the entry
  int e = -1, unit = 1, t = 0;
  int at = 0, end = 0;         // the group's next node, its end
  bool fresh = true, empty = false;

  __device__ Walk(const Params& P, const Entry* entries, const int* o, const int* tot)
      : E(entries), offs(o), total(tot), n_entries(P.n_entries), T(P.T) {
    int64_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += int64_t(tot[i]) * P.coef[i];
    lo = share_begin(c, blockIdx.x, gridDim.x);
    hi = share_begin(c, blockIdx.x + 1, gridDim.x);
  }
  __device__ bool next_entry() {
    for (;;) {
      if (e >= 0) base += int64_t(total[E[e].d >> 1]) * E[e].cost;
      if (++e >= n_entries || base >= hi) {
        e = n_entries;
        return false;
      }
      const int c = E[e].cost;
      const int64_t n = total[E[e].d >> 1];
      const int64_t a = lo <= base ? 0 : min(div_cost(lo - base + c - 1, c), n),
                    b = min(div_cost(hi - base + c - 1, c), n);
      if (a < b) {
        left = int(b - a);
        unit = tile_of(E[e].d);
        empty = E[e].count == 0;
        int j;
        seek_unit(offs, T, unit, a, &t, &j);
        end = t < T ? offs[t + 1] : 0;
        at = t < T ? offs[t] + j * unit : 0;
        fresh = true;
        return true;
      }
    }
  }
  __device__ bool next(Item* it) {
    if (left == 0 && !next_entry()) return false;
    while (at >= end) {
      if (t + 1 >= T) return false;
      ++t, fresh = true;
      at = offs[t], end = offs[t + 1];
    }
    it->e = e, it->t = t;
    it->first = at;
    it->count = min(unit, end - at);
    it->run = fresh;
    it->zero = empty;
    fresh = false;
    at += unit, --left;
    it->run_last = left == 0 || at >= end;
    return true;
  }
};

// a node's row m, channels k0 .. k0+15 of the raw chunk (zeros at and behind kc)
template <int D, bool WHOLE>
__device__ __forceinline__ void read_row16(const float* row, int k0, int kc, float (&v)[16]) {
  if constexpr (D == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(row + k0 + 4 * i);
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = k0 + i < kc ? v[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (WHOLE || k0 + i < kc) ? row[(k0 + i) * D] : 0.f;
  }
}
template <int D, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void convert16(const float* row, int k0, int kc, uint32_t ta) {
  float v[16], h[16];
  read_row16<D, WHOLE>(row, k0, kc, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) tf32_split<SPLIT>(v[i], h[i], v[i]);
  tmem_st16(ta + k0, h);
  if (SPLIT) tmem_st16(ta + kKC + k0, v);
}
// 32 channels of one chunk of the thread's row: raw -> hi (and lo) in TMEM
template <int D, bool SPLIT>
__device__ __forceinline__ void convert(const float* raw, int r, int first, int kc, uint32_t ta) {
  constexpr int ROWS = tile_of(D) * D;
  const int rr = r < ROWS ? r : ROWS - 1;
  const float* row = raw + (rr / D) * node_pitch(D) + rr % D;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    if (first + i + 16 <= kc)
      convert16<D, SPLIT, true>(row, first + i, kc, ta);
    else if (first + i < kc)
      convert16<D, SPLIT, false>(row, first + i, kc, ta);
  }
}
template <int D, bool SPLIT>
__device__ __forceinline__ void lay_out(uint32_t td, float* stage, int r, int first, int nw) {
  constexpr int ROWS = tile_of(D) * D;
  float* row = stage + (r / D) * node_pitch(D) + r % D;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    const int c = first + i;
    if (c >= nw) break;
    float v[16];
    tmem_ld16(td + c, v);
    if (SPLIT) {
      float w[16];
      tmem_ld16(td + ((nw + 15) & ~15) + c, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] += w[i];
    }
    if (r < ROWS) {
      if constexpr (D == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(row + c + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) row[(c + i) * D] = v[i];
      }
    }
  }
}

template <bool SPLIT, int VEC>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ Params P, int chunks, int stages, int outs, uint64_t limit) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sW = base;
  float* sRaw = reinterpret_cast<float*>(base + chunks * kWChunk);
  float* sOut = sRaw + stages * (kRaw / 4);
  LinSource* S = reinterpret_cast<LinSource*>(sOut + outs * (kRaw / 4));
  Entry* E = reinterpret_cast<Entry*>(S + P.n_src);
  int* offs = reinterpret_cast<int*>(E + P.n_entries);
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the lists to shared memory: a walk through kernel parameters misses the constant cache at every step
  for (int i = threadIdx.x; i < P.n_src * int(sizeof(LinSource) / 4); i += kThreads)
    reinterpret_cast<int*>(S)[i] = reinterpret_cast<const int*>(P.s)[i];
  for (int i = threadIdx.x; i < P.n_entries * int(sizeof(Entry) / 4); i += kThreads)
    reinterpret_cast<int*>(E)[i] = reinterpret_cast<const int*>(P.e)[i];
  load_offsets(offs, P.offsets, P.T, P.N);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh.full[s], kCopy);
      mbar_init(&sh.empty[s], 256);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.afull[i], 256);
      mbar_init(&sh.aempty[i], 1);
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 256);
    }
    mbar_init(&sh.wfull, 512);
    mbar_init(&sh.wfree, 1);
    mbar_init(&sh.fin, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 21) tmem_alloc(&sh.tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem;
  if (warp < 4) {
    const int n = count_units(offs, P.T, tile_of(2 * warp + 1));
    if (lane == 0) sh.total[warp] = n;
  }
  __syncthreads();

  Walk walk(P, E, offs, sh.total);
  Item it;
  // the weight of a run, by the converter and epilogue threads: thread (n, q0) takes four channels at a time
  auto load_weight = [&](const Entry& O, int t) {
    const int n = threadIdx.x & 63, n16 = (O.nw + 15) & ~15;
    int c = 0;
    for (int s = 0; s < O.count; ++s) {
      const LinSource& Q = S[O.first + s];
      const float* w = P.w[Q.pair] + int64_t(t) * P.wnumel + Q.woff + int64_t(O.c0 + n) * Q.rw;
      for (int k0 = 0; k0 < Q.k; k0 += kKC, ++c) {
        unsigned char* hi = sW + c * kWChunk;
        const int kc = min(kKC, Q.k - k0);
        float v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int k = 4 * (int(threadIdx.x >> 6) + 8 * i) + f;
            v[i][f] = (n < O.nw && k < kc) ? __ldg(w + int64_t(k0 + k) * Q.rk) : 0.f;
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int q = (threadIdx.x >> 6) + 8 * i;
          float h[4], l[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) tf32_split<SPLIT>(v[i][f], h[f], l[f]);
          // (the lo rows begin at a multiple of 16: the same swizzle)
          const int off = (q >> 3) * kWHalf + n * 128 + (((q & 7) ^ (n & 7)) << 4);
          if (n < n16) {
            *reinterpret_cast<float4*>(hi + off) = make_float4(h[0], h[1], h[2], h[3]);
            if (SPLIT) *reinterpret_cast<float4*>(hi + off + n16 * 128) = make_float4(l[0], l[1], l[2], l[3]);
          }
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive(&sh.wfull);
  };

  if (warp < 8) {
    // ---- rows to TMEM ----
    const int r = threadIdx.x & 127, half = 32 * (warp >> 2);
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemA;
    int ci = 0, wrun = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const Entry& O = E[it.e];
      if (it.run) {
        // the MMAs of the previous weight have completed
        if (wrun > 0 && !wait(&sh.wfree, (wrun - 1) & 1, limit, abort, 1)) break;
        load_weight(O, it.t);
        ++wrun;
      }
      for (int s = 0; ok && s < O.count; ++s) {
        const int K = S[O.first + s].k;
        for (int k0 = 0; k0 < K; k0 += kKC, ++ci) {
          const int st = ci % stages, ab = ci & 1, kc = min(kKC, K - k0);
          if (ci >= 2 && !wait(&sh.aempty[ab], ((ci >> 1) + 1) & 1, limit, abort, 2)) ok = false;
          if (ok && !wait(&sh.full[st], (ci / stages) & 1, limit, abort, 3)) ok = false;
          if (!ok) break;
          fence_after_sync();
          const float* raw = sRaw + st * (kRaw / 4);
          const uint32_t ta = lane_base + ab * kTmemAStage;
          switch (O.d) {
            case 1: convert<1, SPLIT>(raw, r, half, kc, ta); break;
            case 3: convert<3, SPLIT>(raw, r, half, kc, ta); break;
            case 5: convert<5, SPLIT>(raw, r, half, kc, ta); break;
            default: convert<7, SPLIT>(raw, r, half, kc, ta); break;
          }
          mbar_arrive(&sh.empty[st]);
          tmem_wait_st();
          fence_before_sync();
          mbar_arrive(&sh.afull[ab]);
        }
      }
    }
  } else if (warp < 16) {
    // ---- epilogue ----
    const int et = threadIdx.x - 256, r = et & 127, half = 32 * ((warp - 8) >> 2);
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemD;
    int ti = 0, oi = 0, wrun = 0;
    bool ok = true;  // a warp that gave up keeps passing the group's barriers
    auto node_of = [&](const Item& q) { return half == 0 && r < q.count ? P.perm[q.first + r] : -1; };
    Item ahead;
    bool more = walk.next(&ahead);
    int node = more ? node_of(ahead) : -1;
    // this CTA's share of the nodes without a type: zero rows, a warp each
    {
      const int b = offs[P.T], nz = max(int(P.N) - b, 0);
      const int z0 = b + int(share_begin(nz, blockIdx.x, gridDim.x)), z1 = b + int(share_begin(nz, blockIdx.x + 1, gridDim.x));
      for (int i = z0 + (warp - 8); i < z1; i += 8) {
        const int n = P.perm[i];
        if (n < 0 || n >= P.N) continue;
        float* dst = P.out + int64_t(n) * P.dim_out;
        for (int c = lane * VEC; c < P.dim_out; c += 32 * VEC) {
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(dst + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          else
            dst[c] = 0.f;
        }
      }
    }
    while (more) {
      it = ahead;
      const int cur = node;
      more = walk.next(&ahead);
      if (more) node = node_of(ahead);  // read a tile ahead: its latency is that of HBM
      const Entry& O = E[it.e];
      const int db = ti & 1;
      float* stage = sOut + (outs == 2 ? oi & 1 : 0) * (kRaw / 4);
      if (!it.zero && it.run) {
        if (ok && wrun > 0) ok = wait(&sh.wfree, (wrun - 1) & 1, limit, abort, 9);
        if (ok) load_weight(O, it.t);
        ++wrun;
      }
      if (outs == 1) asm volatile("bar.sync 1, 256;" ::: "memory");  // the last tile has been read
      if (half == 0) sh.node_out[oi & 1][r] = (cur >= 0 && cur < P.N) ? cur : -1;
      if (!it.zero) {
        if (ok) ok = wait(&sh.dfull[db], (ti >> 1) & 1, limit, abort, 4);
        if (ok) {
          fence_after_sync();
          const uint32_t td = lane_base + db * kTmemDStage;
          switch (O.d) {
            case 1: lay_out<1, SPLIT>(td, stage, r, half, O.nw); break;
            case 3: lay_out<3, SPLIT>(td, stage, r, half, O.nw); break;
            case 5: lay_out<5, SPLIT>(td, stage, r, half, O.nw); break;
            default: lay_out<7, SPLIT>(td, stage, r, half, O.nw); break;
          }
          fence_before_sync();
          mbar_arrive(&sh.dempty[db]);
        }
        ++ti;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (ok) {
        const int pitch = node_pitch(O.d), dim = P.dim_out;
        float* out = P.out + O.off;
        const int* nodes = sh.node_out[oi & 1];
        const int n = O.nw * O.d / VEC;
        const RowShare w(n, et, 256);
        for (int o = w.at; o < n; o += w.pieces) {
          const float* src = stage + w.row * pitch + o * VEC;
#pragma unroll 4
          for (int q = w.row; q < it.count; q += w.rows, src += w.rows * pitch) {
            const int node = nodes[q];
            float* dst = out + int64_t(node) * dim + o * VEC;
            if constexpr (VEC == 4) {
              const float4 v = it.zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(src);
              if (node >= 0) *reinterpret_cast<float4*>(dst) = v;
            } else {
              const float v = it.zero ? 0.f : *src;
              if (node >= 0) *dst = v;
            }
          }
        }
      }
      ++oi;
    }
  } else if (warp < 21) {
    // ---- node rows to shared memory, several chunks ahead ----
    const int r = threadIdx.x - 512;
    int ci = 0, ni = 0;
    bool ok = true, more = false;
    auto next_item = [&](Item* q) {  // the next tile with a product
      bool m;
      do m = walk.next(q);
      while (m && q->zero);
      return m;
    };
    auto node_of = [&](const Item& q) { return r < q.count ? P.perm[q.first + r] : 0; };
    more = next_item(&it);
    int node = more ? node_of(it) : 0;
    while (more) {  // (a warp that gave up keeps passing the group's barriers)
      const Item cur = it;
      const Entry& O = E[cur.e];
      int* nodes = sh.node_in[ni & 1];
      ++ni;
      if (r < 128) nodes[r] = (node >= 0 && node < P.N) ? node : 0;  // (a wrong node's row is not stored)
      more = next_item(&it);
      if (more) node = node_of(it);  // read while this tile is copied
      asm volatile("bar.sync 2, 160;" ::: "memory");
      for (int s = 0; ok && s < O.count; ++s) {
        const LinSource& Q = S[O.first + s];
        const float* x = P.x[Q.pair] + Q.off;
        for (int k0 = 0; k0 < Q.k; k0 += kKC, ++ci) {
          const int st = ci % stages, pitch = node_pitch(O.d);
          if (ci >= stages && !wait(&sh.empty[st], ((ci / stages) + 1) & 1, limit, abort, 5)) ok = false;
          if (!ok) break;
          const uint32_t dst = smem_u32(sRaw + st * (kRaw / 4));
          const int n = min(kKC, Q.k - k0) * O.d / VEC;
          const RowShare w(n, r, kCopy);
          for (int o = w.at; o < n; o += w.pieces) {
            const float* src = x + k0 * O.d + o * VEC;
            uint32_t to = dst + (w.row * pitch + o * VEC) * 4;
#pragma unroll 4
            for (int q = w.row; q < cur.count; q += w.rows, to += w.rows * pitch * 4)
              copy_async<VEC>(to, src + int64_t(nodes[q]) * P.dim_src);
          }
          copies_arrive(&sh.full[st]);
        }
      }
    }
    copies_wait_all();  // no copy may be in flight when the CTA ends
  } else {
    // ---- MMAs ----
    int ci = 0, ti = 0, wrun = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const Entry& O = E[it.e];
      const int db = ti & 1;
      const int n16 = (O.nw + 15) & ~15;
      const uint32_t id1 = idesc_tf32(128, SPLIT ? 2 * n16 : n16), id2 = idesc_tf32(128, n16);
      const uint32_t td = tmem + kTmemD + db * kTmemDStage;
      if (it.run && !wait(&sh.wfull, wrun & 1, limit, abort, 6)) break;
      if (it.run) ++wrun;
      if (ti >= 2 && !wait(&sh.dempty[db], ((ti >> 1) + 1) & 1, limit, abort, 7)) break;
      int wc = 0;
      for (int s = 0; ok && s < O.count; ++s) {
        const int K = S[O.first + s].k;
        for (int k0 = 0; k0 < K; k0 += kKC, ++ci, ++wc) {
          const int ab = ci & 1, steps = (min(kKC, K - k0) + 7) / 8;
          if (!wait(&sh.afull[ab], (ci >> 1) & 1, limit, abort, 8)) {
            ok = false;
            break;
          }
          fence_after_sync();
          if (lane == 0) {
            const uint32_t a = tmem + kTmemA + ab * kTmemAStage;
            const uint64_t b = sw128_kmajor(smem_u32(sW + wc * kWChunk));
#pragma unroll
            for (int k = 0; k < kKC / 8; ++k) {
              if (k >= steps) break;
              // (the descriptor's address field counts 16 bytes: 32 bytes a step)
              const uint64_t bk = b + uint64_t((k >> 2) * (kWHalf / 16) + (k & 3) * 2);
              mma_tf32_ta(td, a + 8 * k, bk, id1, wc > 0 || k > 0);
              if (SPLIT) mma_tf32_ta(td + n16, a + kKC + 8 * k, bk, id2, 1);
            }
            mma_commit(&sh.aempty[ab]);
          }
          __syncwarp();
        }
      }
      if (ok && lane == 0) {
        mma_commit(&sh.dfull[db]);
        if (it.run_last) mma_commit(&sh.wfree);
      }
      __syncwarp();
      ++ti;
    }
    if (lane == 0) {
      mma_commit(&sh.fin);
      mbar_wait_for(&sh.fin, 0, kDrainLimitNs);  // no MMA may be in flight when TMEM is freed
    }
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 21) {
    fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// the shape of a call: chunks of its widest weight, shared memory behind it
struct Shape {
  int chunks, entries, stages, outs, bytes;
};
Shape shape_of(const LinRows& R) {
  Shape h{0, 0, 0, 0, 0};
  for (int b = 0; b < R.n_out; ++b) {
    const LinOut& O = R.o[b];
    int c = 0;
    for (int s = 0; s < O.count; ++s) c += chunks_of(R.s[O.first + s].k);
    h.chunks = std::max(h.chunks, c);
    h.entries += col_tiles(O.n);
  }
  const int lists = R.n_src * int(sizeof(LinSource)) + h.entries * int(sizeof(Entry)) + (R.T + 2) * 4;
  // the weight, then as many raw stages (two to four) and output buffers (one or two) as fit
  const int fixed = 1024 + h.chunks * kWChunk + lists;
  const int room = (kSMemMax - int(sizeof(Shared)) - 64 - fixed) / kRaw;
  h.outs = room >= 5 ? 2 : 1;
  h.stages = std::min(kMaxStages, room - h.outs);
  h.bytes = fixed + (h.stages + h.outs) * kRaw;
  return h;
}

bool vec4(const LinRows& R) {
  const auto bad = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  if (R.dim_src % 4 || R.dim_out % 4 || bad(R.out)) return false;
  for (int b = 0; b < R.n_out; ++b) {
    const LinOut& O = R.o[b];
    if (O.n % 4 || O.off % 4) return false;
    for (int s = 0; s < O.count; ++s) {
      const LinSource& S = R.s[O.first + s];
      if (S.k % 4 || S.off % 4 || bad(R.x[S.pair])) return false;
    }
  }
  return true;
}

}  // namespace

bool linear_tc_supported(const LinRows& R) {
  const Shape h = shape_of(R);
  return h.chunks <= kMaxChunks && h.entries <= kLinTcEntries && h.stages >= 2;
}

cudaError_t linear_tc_rows(const LinRows& R, bool split, uint64_t limit, cudaStream_t st) {
  const Shape h = shape_of(R);
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.n_src = R.n_src, P.T = R.T, P.dim_src = R.dim_src, P.dim_out = R.dim_out, P.N = R.N, P.wnumel = R.wnumel;
  for (int i = 0; i < 2; ++i) P.x[i] = R.x[i], P.w[i] = R.w[i];
  P.out = R.out, P.perm = R.perm, P.offsets = R.offsets;
  std::copy(R.s, R.s + R.n_src, P.s);
  int64_t tiles = 0;
  for (int b = 0; b < R.n_out; ++b) {
    const LinOut& O = R.o[b];
    int cost = 1;
    for (int s = 0; s < O.count; ++s) cost += chunks_of(R.s[O.first + s].k);
    for (int c0 = 0; c0 < O.n; c0 += kNT) {
      P.e[P.n_entries++] = {O.d, cost, O.off + c0 * O.d, std::min(kNT, O.n - c0), c0, O.first, O.count, 0};
      P.coef[O.d >> 1] += cost;
    }
    tiles += (R.N / tile_of(O.d) + std::min<int64_t>(R.T, R.N)) * col_tiles(O.n);
  }
  const bool v = vec4(R);
  auto* k = split ? (v ? k_linear_tc<true, 4> : k_linear_tc<true, 1>) : (v ? k_linear_tc<false, 4> : k_linear_tc<false, 1>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, h.bytes);
  if (e) return e;
  k<<<unsigned(std::min<int64_t>(kSMs, tiles)), kThreads, h.bytes, st>>>(P, h.chunks, h.stages, h.outs, limit);
  return cudaGetLastError();
}

cudaError_t linear_tc_read_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_linear_error, sizeof(int));
  if (e) return e;
  return *code ? cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(int)) : cudaSuccess;
}

}  // namespace tpc
