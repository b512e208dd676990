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
//   one thread issues D += A_lo B_hi + A_hi B_lo, then A_hi B_hi (the small products
//   first, while the accumulator is small);
//   epilogue threads, one per row, lay D out as [channel][m] in shared memory, and
//   store the nodes' pieces, 16 bytes a thread.
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
// from the device.  Warps 0-3 convert, 4-7 run the epilogue, 8-11 copy, 12 issues the
// MMAs.  (Bulk copies of a node's piece were tried in place of the copy threads: about
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
constexpr int kWHalf = kNT * kKC * 4;         // hi or lo of one chunk: 16 KB
constexpr int kWChunk = 2 * kWHalf;
constexpr int kRaw = 32928;                   // a raw chunk or an output tile (see node_pitch)
constexpr int kMaxStages = 4;
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 416;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 128, kTmemD = 256;  // A: 2 x (hi 64 | lo 64), D: 2 x 64

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
  int total[4];                    // tiles of all groups for d = 1, 3, 5, 7
  int node_in[2][128], node_out[2][128];
};

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_error, code);
}

// ---- the CTA's share of the work -------------------------------------------------
// Entries in order, in each the tiles of groups 0..T; CTA b owns the tiles whose cost
// begins in its share.  Every warp walks the same list.
struct Item {
  int e, t, first, count;
  bool run;       // the first tile with this weight
  bool run_last;  // the last tile of this CTA with this weight
  bool zero;      // no product: a group without a type, or a block without a source
};

struct Walk {
  const Entry* E;
  const int* offs;
  const int* total;
  int n_entries, T;
  int64_t lo, hi, base = 0, left = 0;
  int e = -1, unit = 1, t = 0, j = 0, tiles = 0;
  bool fresh = true;

  __device__ Walk(const Params& P, const Entry* entries, const int* o, const int* tot)
      : E(entries), offs(o), total(tot), n_entries(P.n_entries), T(P.T) {
    int64_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += int64_t(tot[i]) * P.coef[i];
    lo = share_begin(c, blockIdx.x, gridDim.x);
    hi = share_begin(c, blockIdx.x + 1, gridDim.x);
  }
  __device__ bool next(Item* it) {
    if (left == 0) {
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
          left = b - a;
          unit = tile_of(E[e].d);
          seek_unit(offs, T + 1, unit, a, &t, &j);
          tiles = t <= T ? group_units(offs, t, unit) : 0;
          fresh = true;
          break;
        }
      }
    }
    while (j >= tiles) {
      if (t >= T) return false;
      ++t, j = 0, fresh = true;
      tiles = group_units(offs, t, unit);
    }
    it->e = e, it->t = t;
    it->first = offs[t] + j * unit;
    it->count = min(unit, offs[t + 1] - it->first);
    it->run = fresh;
    it->zero = t >= T || E[e].count == 0;
    fresh = false;
    ++j, --left;
    it->run_last = left == 0 || j >= tiles;
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
// one chunk of the thread's row: raw -> hi (and lo) in TMEM
template <int D, bool SPLIT>
__device__ __forceinline__ void convert(const float* raw, int r, int kc, uint32_t ta) {
  constexpr int ROWS = tile_of(D) * D;
  const int rr = r < ROWS ? r : ROWS - 1;
  const float* row = raw + (rr / D) * node_pitch(D) + rr % D;
  if (kc == kKC) {
#pragma unroll
    for (int k0 = 0; k0 < kKC; k0 += 16) convert16<D, SPLIT, true>(row, k0, kc, ta);
  } else {
    for (int k0 = 0; k0 < kc; k0 += 16) convert16<D, SPLIT, false>(row, k0, kc, ta);
  }
}
template <int D>
__device__ __forceinline__ void lay_out(uint32_t td, float* stage, int r, int nw) {
  constexpr int ROWS = tile_of(D) * D;
  float* row = stage + (r / D) * node_pitch(D) + r % D;
#pragma unroll
  for (int c = 0; c < kNT; c += 16) {
    if (c >= nw) break;
    float v[16];
    tmem_ld16(td + c, v);
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

// one chunk's products: 8 channels a step, each operand's hi and lo
__device__ __forceinline__ void issue(uint32_t td, uint32_t a, uint64_t bh, uint64_t bl, uint32_t idesc, int k,
                                      uint32_t acc, bool cross) {
  // (the descriptors' address field counts 16 bytes: 32 bytes a step, 8 KB behind 32 channels)
  const uint64_t step = uint64_t((k >> 2) * (kNT * 128 / 16) + (k & 3) * 2);
  if (cross) {
    mma_tf32_ta(td, a + kKC + 8 * k, bh + step, idesc, acc);
    mma_tf32_ta(td, a + 8 * k, bl + step, idesc, 1);
  } else {
    mma_tf32_ta(td, a + 8 * k, bh + step, idesc, acc);
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
      mbar_init(&sh.full[s], 128);
      mbar_init(&sh.empty[s], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.afull[i], 128);
      mbar_init(&sh.aempty[i], 1);
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 128);
    }
    mbar_init(&sh.wfull, 256);
    mbar_init(&sh.wfree, 1);
    mbar_init(&sh.fin, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(&sh.tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem;
  if (warp < 4) {
    const int n = count_units(offs, P.T + 1, tile_of(2 * warp + 1));
    if (lane == 0) sh.total[warp] = n;
  }
  __syncthreads();

  Walk walk(P, E, offs, sh.total);
  Item it;
  // the weight of a run, by the converter and epilogue threads: thread (n, q0) takes four channels at a time
  auto load_weight = [&](const Entry& O, int t) {
    const int n = threadIdx.x & 63;
    int c = 0;
    for (int s = 0; s < O.count; ++s) {
      const LinSource& Q = S[O.first + s];
      const float* w = P.w[Q.pair] + int64_t(t) * P.wnumel + Q.woff + int64_t(O.c0 + n) * Q.rw;
      for (int k0 = 0; k0 < Q.k; k0 += kKC, ++c) {
        unsigned char* hi = sW + c * kWChunk;
        const int kc = min(kKC, Q.k - k0);
        float v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const int k = 4 * (int(threadIdx.x >> 6) + 4 * i) + f;
            v[i][f] = (n < O.nw && k < kc) ? __ldg(w + int64_t(k0 + k) * Q.rk) : 0.f;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = (threadIdx.x >> 6) + 4 * i;
          float h[4], l[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) tf32_split<SPLIT>(v[i][f], h[f], l[f]);
          const int off = (q >> 3) * (kNT * 128) + n * 128 + (((q & 7) ^ (n & 7)) << 4);
          *reinterpret_cast<float4*>(hi + off) = make_float4(h[0], h[1], h[2], h[3]);
          if (SPLIT) *reinterpret_cast<float4*>(hi + kWHalf + off) = make_float4(l[0], l[1], l[2], l[3]);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive(&sh.wfull);
  };

  if (warp < 4) {
    // ---- rows to TMEM ----
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + (uint32_t(warp * 32) << 16) + kTmemA;
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
            case 1: convert<1, SPLIT>(raw, r, kc, ta); break;
            case 3: convert<3, SPLIT>(raw, r, kc, ta); break;
            case 5: convert<5, SPLIT>(raw, r, kc, ta); break;
            default: convert<7, SPLIT>(raw, r, kc, ta); break;
          }
          mbar_arrive(&sh.empty[st]);
          tmem_wait_st();
          fence_before_sync();
          mbar_arrive(&sh.afull[ab]);
        }
      }
    }
  } else if (warp < 8) {
    // ---- epilogue ----
    const int r = threadIdx.x - 128;
    const uint32_t lane_base = tmem + (uint32_t((warp - 4) * 32) << 16) + kTmemD;
    int ti = 0, oi = 0, wrun = 0;
    bool ok = true;  // a warp that gave up keeps passing the group's barriers
    while (walk.next(&it)) {
      const Entry& O = E[it.e];
      const int db = ti & 1;
      float* stage = sOut + (outs == 2 ? oi & 1 : 0) * (kRaw / 4);
      int node = r < it.count ? P.perm[it.first + r] : -1;
      if (!it.zero && it.run) {
        if (ok && wrun > 0) ok = wait(&sh.wfree, (wrun - 1) & 1, limit, abort, 9);
        if (ok) load_weight(O, it.t);
        ++wrun;
      }
      if (outs == 1) asm volatile("bar.sync 1, 128;" ::: "memory");  // the last tile has been read
      sh.node_out[oi & 1][r] = (node >= 0 && node < P.N) ? node : -1;
      if (!it.zero) {
        if (ok) ok = wait(&sh.dfull[db], (ti >> 1) & 1, limit, abort, 4);
        if (ok) {
          fence_after_sync();
          const uint32_t td = lane_base + db * kNT;
          switch (O.d) {
            case 1: lay_out<1>(td, stage, r, O.nw); break;
            case 3: lay_out<3>(td, stage, r, O.nw); break;
            case 5: lay_out<5>(td, stage, r, O.nw); break;
            default: lay_out<7>(td, stage, r, O.nw); break;
          }
          fence_before_sync();
          mbar_arrive(&sh.dempty[db]);
        }
        ++ti;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) {
        const int pitch = node_pitch(O.d);
        float* out = P.out + O.off;
        const int* nodes = sh.node_out[oi & 1];
#pragma unroll 4
        for (Pieces<VEC> p(it.count, O.nw * O.d, r, 128); p.valid(); p.advance()) {
          const int n = nodes[p.q];
          if (n < 0) continue;
          float* dst = out + int64_t(n) * P.dim_out + p.o * VEC;
          const float* src = stage + p.q * pitch + p.o * VEC;
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(dst) = it.zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(src);
          else
            *dst = it.zero ? 0.f : *src;
        }
      }
      ++oi;
    }
  } else if (warp < 12) {
    // ---- node rows to shared memory, several chunks ahead ----
    const int r = threadIdx.x - 256;
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
      nodes[r] = (node >= 0 && node < P.N) ? node : 0;  // (a wrong node's row is not stored)
      more = next_item(&it);
      if (more) node = node_of(it);  // read while this tile is copied
      asm volatile("bar.sync 2, 128;" ::: "memory");
      for (int s = 0; ok && s < O.count; ++s) {
        const LinSource& Q = S[O.first + s];
        const float* x = P.x[Q.pair] + Q.off;
        for (int k0 = 0; k0 < Q.k; k0 += kKC, ++ci) {
          const int st = ci % stages, pitch = node_pitch(O.d);
          if (ci >= stages && !wait(&sh.empty[st], ((ci / stages) + 1) & 1, limit, abort, 5)) ok = false;
          if (!ok) break;
          const uint32_t dst = smem_u32(sRaw + st * (kRaw / 4));
#pragma unroll 4
          for (Pieces<VEC> p(cur.count, min(kKC, Q.k - k0) * O.d, r, 128); p.valid(); p.advance())
            copy_async<VEC>(dst + (p.q * pitch + p.o * VEC) * 4,
                            x + int64_t(nodes[p.q]) * P.dim_src + k0 * O.d + p.o * VEC);
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
      const uint32_t idesc = idesc_tf32(128, (O.nw + 15) & ~15);
      const uint32_t td = tmem + kTmemD + db * kNT;
      if (it.run && !wait(&sh.wfull, wrun & 1, limit, abort, 6)) break;
      if (it.run) ++wrun;
      if (ti >= 2 && !wait(&sh.dempty[db], ((ti >> 1) + 1) & 1, limit, abort, 7)) break;
      uint32_t acc = 0;
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
            const uint64_t bh = sw128_kmajor(smem_u32(sW + wc * kWChunk)), bl = sw128_kmajor(smem_u32(sW + wc * kWChunk + kWHalf));
            if (SPLIT) {
              if (steps == 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) issue(td, a, bh, bl, idesc, k, k > 0 ? 1u : acc, true);
              } else {
                for (int k = 0; k < steps; ++k) issue(td, a, bh, bl, idesc, k, k > 0 ? 1u : acc, true);
              }
              acc = 1;
            }
            if (steps == 8) {
#pragma unroll
              for (int k = 0; k < 8; ++k) issue(td, a, bh, bl, idesc, k, k > 0 ? 1u : acc, false);
            } else {
              for (int k = 0; k < steps; ++k) issue(td, a, bh, bl, idesc, k, k > 0 ? 1u : acc, false);
            }
            acc = 1;
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
  if (warp == 12) {
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
    tiles += (R.N / tile_of(O.d) + std::min<int64_t>(R.T + 1, R.N)) * col_tiles(O.n);
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
