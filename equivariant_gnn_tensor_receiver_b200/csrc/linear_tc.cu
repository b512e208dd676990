// Typed linear map on the tensor cores: rows times the weight of their type
// (sm_100a: tcgen05 with the row operand in TMEM, gathers by asynchronous copies).
//
//   out[n, w, m] = sum_k x[n, k, m] B_t[k][w]     per (output block, 64 columns, type t)
//
// A tile is the (node, m) rows of up to 128 / (2l+1) nodes of one type, times 64
// output channels.  The weight of the (block, columns, type) is resident in shared
// memory, split once into TF32 hi and lo; the node rows are the only stream:
//   copy warps gather the nodes' contiguous pieces [64 channels][2l+1] by perm, a bulk
//   copy a node (4-byte asynchronous copies where a block or tensor is not 16-byte
//   aligned), several chunks ahead;
//   converter threads, one per row, read their row's channels (stride 2l+1), split
//   them (3xTF32, Ootomo & Yokota, 2022) and store hi and lo as the A operand in
//   TMEM: the transposition from [channel][m] to rows costs one shared-memory read
//   per element and no write;
//   one thread issues, 8 channels a step, (D1 | D2) += A_hi (B_hi | B_lo) as one product
//   of up to 128 columns, and D2 += A_lo B_hi: two instructions instead of three, and
//   the small products add up among themselves;
//   epilogue threads, one per row, lay D1 + D2 out as [channel][m] in shared memory, and
//   bulk copies store the nodes' pieces (threads, where they are not aligned or added).
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
// from the device.  What bounds a tile is the latency of its steps, not the issue
// slots, so two pipelines take every second tile each, with buffers and barriers of
// their own, and share the weight: warps 0-3 and 4-7 convert, 8-11 and 12-15 run the
// epilogue, 21 and 22 issue the MMAs; 16-20 copy for both.
// (Issuing a bulk copy takes some 60 cycles, so the nodes are dealt out over the warps.
// Stores from registers held four warps for 5500 cycles a tile, waiting for the memory
// pipe to take them: 306 us against 270 at 262144 nodes of 64x0e+64x1o+64x2e, where equal
// shares took 270; both warpgroups of a role on one tile: 340 us.)
// Measured (device, 3xTF32): 262144 nodes of 64x0e+64x1o+64x2e, 16 types: 242 us, 4.99 TB/s,
// 0.76 of the measured copy rate; 4096 nodes of it: 21 us, most of it the latency of a
// CTA's first tile (weight, rows, product, store one after another).
// A sum over more than 160 channels runs in several passes that add to the output.
// Every wait is bounded by the call's limit; on expiry the kernel records it, stops
// issuing, waits (bounded) for its own copies and MMAs, frees TMEM and returns.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "chain.cuh"
#include "linear_tc.h"
#include "linear_tc_common.cuh"

namespace tpc {
namespace {

using namespace tc;

__device__ int g_linear_error;  // first code recorded by an expired wait (0 = none)

constexpr int kSMs = 148;
constexpr int kNT = 64, kKC = 64;             // columns of a tile, channels of a chunk
// 32 channels of a weight: the rows of up to 64 output channels' hi and behind them their
// lo, 128 bytes a row (K-major, 128-byte swizzle)
constexpr int kWHalf = 2 * kNT * 32 * 4;
constexpr int kMaxHalves = 5;                 // of a resident weight: 160 channels
constexpr int kRaw = 32928;                   // a raw chunk or an output tile (see node_pitch)
constexpr int kMaxStages = 2;                 // raw chunks of a pipeline
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 736, kCopyWarps = 5, kCopy = 32 * kCopyWarps;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 128, kTmemD = 256, kTmemDStage = 128;  // A: 2 x (hi 64 | lo 64), D: 2 x (D1 | D2)

// nodes of a tile; floats of a node's 64 channels plus padding (multiple of 4)
__host__ __device__ constexpr int tile_of(int d) { return d == 1 ? 120 : 128 / d; }
__host__ __device__ constexpr int node_pitch(int d) { return kKC * d + (d == 1 || d == 3 ? 4 : 8); }
static_assert(tile_of(1) * node_pitch(1) * 4 <= kRaw && tile_of(3) * node_pitch(3) * 4 <= kRaw &&
                  tile_of(5) * node_pitch(5) * 4 <= kRaw && tile_of(7) * node_pitch(7) * 4 <= kRaw,
              "a tile fits its buffer");

__host__ __device__ constexpr int chunks_of(int k) { return (k + kKC - 1) / kKC; }
__host__ __device__ constexpr int halves_of(int k) { return (k + 31) / 32; }
constexpr int col_tiles(int n) { return (n + kNT - 1) / kNT; }

// (output block, 64 columns)
struct Entry {
  int d;             // 2l+1
  int off, nw;       // first output column, channels
  int c0;            // first channel of the block
  int first, count;  // sources
  int pad;
};
static_assert(sizeof(Entry) % 4 == 0 && sizeof(Cut) % 4 == 0 && sizeof(LinSource) % 8 == 0, "copied by words");
struct Params {
  int n_entries, n_src, T, dim_src, dim_out;
  int64_t N, wnumel;
  const float *x[2], *w[2];
  float* out;
  const int *perm, *offsets;
  int coef[4];     // cost of a tile of d = 1, 3, 5, 7, summed over the entries
  int accumulate;  // add to the output (and leave the rows without a type alone)
  Entry e[kLinTcEntries];
  Cut cut[kLinTcEntries];  // cost of a tile: by its chunks
  LinSource s[kLinSources];
};

struct Shared {
  uint64_t full[2][kMaxStages], empty[2][kMaxStages];
  uint64_t afull[2], aempty[2], dfull[2], dempty[2], wfull, wfree, fin;
  uint32_t tmem;
  int abort;
  int total[4];                    // tiles of all types for d = 1, 3, 5, 7
  WalkState walk[kThreads / 32];
  int node_in[2][128], node_out[2][128];
  int issued[2][kCopyWarps];
};

constexpr int kDynMax = kSMemMax - int(sizeof(Shared)) - 64;  // dynamic shared memory of a call, at most

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_error, code);
}

// ---- the CTA's tiles ---------------------------------------------------------------
struct Item {
  int e, t, first, count;
  bool run;       // the first tile with this weight
  bool run_last;  // the last tile of this CTA with this weight
  bool zero;      // no product: a block without a source
};

struct Walk {
  WalkState* w;
  const Entry* E;
  const Cut* cuts;
  const int *total, *offs;
  int n, T;
  int e = 0, t = 0, at = 0, end = 0, unit = 1;
  bool zero = false;

  __device__ __forceinline__ bool next(Item* it) {
    const bool fresh = at >= end;
    if (fresh) {
      const Run r = next_run(w, cuts, n, total, offs, T);
      if (r.e < 0) return false;
      e = r.e, t = r.t, at = r.first, end = r.end;
      unit = cuts[e].nodes;
      zero = E[e].count == 0;
    }
    it->e = e, it->t = t, it->first = at;
    it->count = min(unit, end - at);
    it->run = fresh;
    it->zero = zero;
    at += it->count;
    it->run_last = at >= end;
    return true;
  }
};

// 16 channels of a node's row m: raw -> hi (and lo) in TMEM, zeros at and behind n
template <int D, bool SPLIT, bool WHOLE>
__device__ __forceinline__ void convert16(const float* row, int n, uint32_t ta) {
  float v[16], h[16];
  if constexpr (D == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(row + 4 * i);
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (WHOLE || i < n) ? row[i * D] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) tf32_split<SPLIT>((D > 1 || WHOLE || i < n) ? v[i] : 0.f, h[i], v[i]);
  tmem_st16(ta, h);
  if (SPLIT) tmem_st16(ta + kKC, v);
}
// one chunk of the thread's row
template <int D, bool SPLIT>
__device__ __forceinline__ void convert(const float* raw, int r, int kc, uint32_t ta) {
  constexpr int ROWS = tile_of(D) * D;
  const int rr = r < ROWS ? r : ROWS - 1;
  const float* row = raw + (rr / D) * node_pitch(D) + rr % D;
  int k0 = 0;
#pragma unroll 1
  for (; k0 + 16 <= kc; k0 += 16, row += 16 * D) convert16<D, SPLIT, true>(row, 16, ta + k0);
  if (k0 < kc) convert16<D, SPLIT, false>(row, kc - k0, ta + k0);
}
template <int D, bool SPLIT>
__device__ __forceinline__ void lay_out(uint32_t td, float* stage, int r, int nw) {
  constexpr int ROWS = tile_of(D) * D;
  float* row = stage + (r / D) * node_pitch(D) + r % D;
#pragma unroll 1
  for (int c = 0; c < nw; c += 16, row += 16 * D) {
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
          *reinterpret_cast<float4*>(row + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) row[i * D] = v[i];
      }
    }
  }
}

struct One {
  float x;
  __device__ __forceinline__ One operator+(const One& o) const { return {x + o.x}; }
};
struct __align__(16) Four {
  float x, y, z, w;
  __device__ __forceinline__ Four operator+(const Four& o) const { return {x + o.x, y + o.y, z + o.z, w + o.w}; }
};

template <bool SPLIT, int VEC>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ Params P, int halves, int stages, int more, uint64_t limit) {
  using Pack = std::conditional_t<VEC == 4, Four, One>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sW = base;
  float* sRaw = reinterpret_cast<float*>(base + halves * kWHalf);
  float* sOut = sRaw + 2 * stages * (kRaw / 4);
  LinSource* S = reinterpret_cast<LinSource*>(sOut + 2 * (kRaw / 4));
  Entry* E = reinterpret_cast<Entry*>(S + P.n_src);
  Cut* cuts = reinterpret_cast<Cut*>(E + P.n_entries);
  int* offs = reinterpret_cast<int*>(cuts + P.n_entries);
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (more) chain_next();
  // the lists to shared memory: a walk through kernel parameters misses the constant cache at every step
  for (int i = threadIdx.x; i < P.n_src * int(sizeof(LinSource) / 4); i += kThreads)
    reinterpret_cast<int*>(S)[i] = reinterpret_cast<const int*>(P.s)[i];
  for (int i = threadIdx.x; i < P.n_entries * int(sizeof(Entry) / 4); i += kThreads)
    reinterpret_cast<int*>(E)[i] = reinterpret_cast<const int*>(P.e)[i];
  for (int i = threadIdx.x; i < P.n_entries * int(sizeof(Cut) / 4); i += kThreads)
    reinterpret_cast<int*>(cuts)[i] = reinterpret_cast<const int*>(P.cut)[i];
  load_offsets(offs, P.offsets, P.T, P.N);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < kMaxStages; ++s) {
        mbar_init(&sh.full[i][s], VEC == 4 ? kCopyWarps : kCopy);
        mbar_init(&sh.empty[i][s], 128);
      }
      mbar_init(&sh.afull[i], 128);
      mbar_init(&sh.aempty[i], 1);
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 128);
    }
    mbar_init(&sh.wfull, 512);
    mbar_init(&sh.wfree, 2);
    mbar_init(&sh.fin, 2);
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

  {
    int c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c += sh.total[i] * P.coef[i];
    walk_begin(&sh.walk[warp], c);
  }
  Walk walk{&sh.walk[warp], E, cuts, sh.total, offs, P.n_entries, P.T};
  Item it;
  // the weight of a run, by the converter and epilogue threads: thread (n, q0) takes four channels at a time
  auto load_weight = [&](const Entry& O, int t) {
    const int n = threadIdx.x & 63, n16 = (O.nw + 15) & ~15;
    unsigned char* hi = sW;
    for (int s = 0; s < O.count; ++s) {
      const LinSource& Q = S[O.first + s];
      const float* w = P.w[Q.pair] + int64_t(t) * P.wnumel + Q.woff + int64_t(O.c0 + n) * Q.rw;
      for (int k0 = 0; k0 < Q.k; k0 += kKC) {
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
          if (n < n16 && q < 8 * halves_of(kc)) {
            *reinterpret_cast<float4*>(hi + off) = make_float4(h[0], h[1], h[2], h[3]);
            if (SPLIT) *reinterpret_cast<float4*>(hi + off + n16 * 128) = make_float4(l[0], l[1], l[2], l[3]);
          }
        }
        hi += halves_of(kc) * kWHalf;
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive(&sh.wfull);
  };

  if (warp < 8) {
    // ---- rows to TMEM: tiles of the set's parity ----
    const int r = threadIdx.x & 127, set = warp >> 2;
    const uint32_t ta = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemA + set * kTmemAStage;
    int ci = 0, ti = 0, wrun = 0;  // the set's chunks, all tiles, all runs
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
      if ((ti++ & 1) != set) continue;
      for (int s = 0; ok && s < O.count; ++s) {
        const int K = S[O.first + s].k;
        for (int k0 = 0; k0 < K; k0 += kKC, ++ci) {
          const int st = ci % stages, kc = min(kKC, K - k0);
          if (ci >= 1 && !wait(&sh.aempty[set], (ci - 1) & 1, limit, abort, 2)) ok = false;
          if (ok && !wait(&sh.full[set][st], (ci / stages) & 1, limit, abort, 3)) ok = false;
          if (!ok) break;
          fence_after_sync();
          const float* raw = sRaw + (set * stages + st) * (kRaw / 4);
          switch (O.d) {
            case 1: convert<1, SPLIT>(raw, r, kc, ta); break;
            case 3: convert<3, SPLIT>(raw, r, kc, ta); break;
            case 5: convert<5, SPLIT>(raw, r, kc, ta); break;
            default: convert<7, SPLIT>(raw, r, kc, ta); break;
          }
          mbar_arrive(&sh.empty[set][st]);
          tmem_wait_st();
          fence_before_sync();
          mbar_arrive(&sh.afull[set]);
        }
      }
    }
  } else if (warp < 16) {
    // ---- epilogue: tiles of the set's parity ----
    const int r = threadIdx.x & 127, set = (warp - 8) >> 2;
    const uint32_t td = tmem + (uint32_t((warp & 3) * 32) << 16) + kTmemD + set * kTmemDStage;
    float* stage = sOut + set * (kRaw / 4);
    int* nodes = sh.node_out[set];
    int ti = 0, di = 0, wrun = 0;  // tiles, tiles with a product
    bool ok = true;  // a warp that gave up keeps passing the set's barriers
    auto bar = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory"); };
    // the next tile of the set; on the way, its part of the weights of new runs
    auto next_item = [&](int* d) {
      for (;;) {
        if (!walk.next(&it)) return false;
        *d = di;
        if (!it.zero) ++di;
        if (!it.zero && it.run) {
          if (ok && wrun > 0) ok = wait(&sh.wfree, (wrun - 1) & 1, limit, abort, 9);
          if (ok) load_weight(E[it.e], it.t);
          ++wrun;
        }
        // a tile with a product goes to the set of its accumulator
        if (it.zero ? (ti++ & 1) == set : (*d & 1) == set) return true;
      }
    };
    // this CTA's share of the nodes without a type: zero rows, a warp each
    if (!P.accumulate) {
      const int b = offs[P.T], nz = max(int(P.N) - b, 0);
      const int z0 = b + share_begin(nz, blockIdx.x, gridDim.x), z1 = b + share_begin(nz, blockIdx.x + 1, gridDim.x);
      for (unsigned i = z0 + (warp - 8); i < unsigned(z1); i += 8) {  // (i passes 2^31 behind the largest graphs)
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
    // bulk copies of whole pieces (16-byte aligned ones, stored and not added): the warps of the set
    // take every fourth node each
    const bool bulk = VEC == 4 && !P.accumulate;
    const int mine = bulk ? lane * 4 + (warp & 3) : r;
    auto node_of = [&](const Item& q) { return mine < q.count ? P.perm[q.first + mine] : -1; };
    int d;
    bool more = next_item(&d);
    int node = more ? node_of(it) : -1;
    while (more) {
      const Item cur = it;
      const Entry& O = E[cur.e];
      if (bulk) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      bar();  // the set's last tile has been read
      if (!cur.zero) {
        if (ok) ok = wait(&sh.dfull[set], (d >> 1) & 1, limit, abort, 4);
        if (ok) {
          fence_after_sync();
          switch (O.d) {
            case 1: lay_out<1, SPLIT>(td, stage, r, O.nw); break;
            case 3: lay_out<3, SPLIT>(td, stage, r, O.nw); break;
            case 5: lay_out<5, SPLIT>(td, stage, r, O.nw); break;
            default: lay_out<7, SPLIT>(td, stage, r, O.nw); break;
          }
          fence_before_sync();
          mbar_arrive(&sh.dempty[set]);
        }
      }
      const int out_node = (node >= 0 && node < P.N) ? node : -1;
      if (bulk) {
        if (cur.zero)
          for (int i = r; i < tile_of(O.d) * node_pitch(O.d) / 4; i += 128)
            reinterpret_cast<float4*>(stage)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      } else {
        nodes[r] = out_node;
      }
      bar();
      if (bulk) {
        if (ok && out_node >= 0)
          bulk_store(P.out + int64_t(out_node) * P.dim_out + O.off, smem_u32(stage + mine * node_pitch(O.d)),
                     uint32_t(O.nw * O.d * 4));
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      more = next_item(&d);
      if (more) node = node_of(it);  // read while this tile is stored
      if (ok && !bulk) {
        const int pitch = node_pitch(O.d), dim = P.dim_out, n = O.nw * O.d / VEC;
        const RowShare w(n, r, 128);
        for (int o = w.at; o < n; o += w.pieces) {
          const float* src = stage + w.row * pitch + o * VEC;
          float* out = P.out + O.off + o * VEC;
          // Four rows at a time, read before any is stored: the compiler cannot tell the
          // stores from the reads, and would wait for each.
          auto put = [&](int m, Pack v) {
            if (m < 0) return;
            Pack* dst = reinterpret_cast<Pack*>(out + int64_t(m) * dim);
            if (P.accumulate) v = v + *dst;
            *dst = v;
          };
          int q = w.row;
          const int rp = w.rows * pitch;
          if (!cur.zero)
            for (; q + 3 * w.rows < cur.count; q += 4 * w.rows, src += 4 * rp) {
              int m[4];
              Pack v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                m[i] = nodes[q + i * w.rows];
                v[i] = *reinterpret_cast<const Pack*>(src + i * rp);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) put(m[i], v[i]);
            }
          for (; q < cur.count; q += w.rows, src += rp)
            put(nodes[q], cur.zero ? Pack{} : *reinterpret_cast<const Pack*>(src));
        }
      }
    }
    if (bulk) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp < 21) {
    // ---- node rows to shared memory, several chunks ahead ----
    int ci[2] = {0, 0}, ni = 0;  // chunks of each pipeline, tiles
    bool ok = true, more = false;
    auto next_item = [&](Item* q) {  // the next tile with a product
      bool m;
      do m = walk.next(q);
      while (m && q->zero);
      return m;
    };
    if constexpr (VEC == 4) {
      // a bulk copy per node, every fifth node a warp: issuing one takes some 60 cycles
      const int w = warp - 16, r = lane * kCopyWarps + w;
      auto node_of = [&](const Item& q) {
        const int n = r < q.count ? P.perm[q.first + r] : 0;
        return n >= 0 && n < P.N ? n : 0;  // (a wrong node's row is not stored)
      };
      more = next_item(&it);
      int node = more ? node_of(it) : 0;
      while (ok && more) {
        const Item cur = it;
        const Entry& O = E[cur.e];
        const int set = ni++ & 1, pitch = node_pitch(O.d) * 4;
        const int64_t row = int64_t(node) * P.dim_src;
        more = next_item(&it);
        if (more) {
          node = node_of(it);  // read while this tile is copied
          if (r < 4) prefetch_nodes(P.perm, unsigned(it.first) + kPermAhead + 32 * r, P.N);
        }
        const uint32_t mine = cur.count > w ? uint32_t(cur.count - w + kCopyWarps - 1) / kCopyWarps : 0;
        for (int s = 0; ok && s < O.count; ++s) {
          const LinSource& Q = S[O.first + s];
          const float* x = P.x[Q.pair] + row + Q.off;
          for (int k0 = 0; k0 < Q.k; k0 += kKC) {
            const int c = ci[set], st = c % stages;
            const uint32_t bytes = uint32_t(min(kKC, Q.k - k0) * O.d * 4);
            if (c >= stages && !wait(&sh.empty[set][st], ((c / stages) + 1) & 1, limit, abort, 5)) ok = false;
            if (!ok) break;
            ci[set] = c + 1;
            if (lane == 0) mbar_expect_tx(&sh.full[set][st], bytes * mine);
            __syncwarp();
            if (r < cur.count)
              bulk_load(smem_u32(sRaw + (set * stages + st) * (kRaw / 4)) + r * pitch, x + k0 * O.d, bytes,
                        &sh.full[set][st]);
          }
        }
      }
      if (lane == 0) sh.issued[0][w] = ci[0], sh.issued[1][w] = ci[1];
      asm volatile("bar.sync 3, 160;" ::: "memory");
#pragma unroll
      for (int set = 0; set < 2; ++set) drain_ring(sh.full[set], stages, ci[set], sh.issued[set], kCopyWarps);
    } else {
      const int r = threadIdx.x - 512;
      auto node_of = [&](const Item& q) { return r < q.count ? P.perm[q.first + r] : 0; };
      more = next_item(&it);
      int node = more ? node_of(it) : 0;
      while (more) {  // (a warp that gave up keeps passing the group's barriers)
        const Item cur = it;
        const Entry& O = E[cur.e];
        const int set = ni & 1;
        int* nodes = sh.node_in[set];
        ++ni;
        if (r < 128) nodes[r] = (node >= 0 && node < P.N) ? node : 0;  // (a wrong node's row is not stored)
        more = next_item(&it);
        if (more) {
          node = node_of(it);  // read while this tile is copied
          if (r < 4) prefetch_nodes(P.perm, unsigned(it.first) + kPermAhead + 32 * r, P.N);
        }
        asm volatile("bar.sync 3, 160;" ::: "memory");
        for (int s = 0; ok && s < O.count; ++s) {
          const LinSource& Q = S[O.first + s];
          const float* x = P.x[Q.pair] + Q.off;
          for (int k0 = 0; k0 < Q.k; k0 += kKC) {
            const int c = set ? ci[1]++ : ci[0]++, st = c % stages, pitch = node_pitch(O.d);
            if (c >= stages && !wait(&sh.empty[set][st], ((c / stages) + 1) & 1, limit, abort, 5)) ok = false;
            if (!ok) break;
            const uint32_t dst = smem_u32(sRaw + (set * stages + st) * (kRaw / 4));
            const int n = min(kKC, Q.k - k0) * O.d;
            const RowShare w(n, r, kCopy);
            for (int o = w.at; o < n; o += w.pieces) {
              const float* src = x + k0 * O.d + o;
              uint32_t to = dst + (w.row * pitch + o) * 4;
              copy_rows(src, P.dim_src, nodes, w, cur.count, to, pitch * 4);
            }
            copies_arrive(&sh.full[set][st]);
          }
        }
      }
      copies_wait_all();  // no copy may be in flight when the CTA ends
    }
  } else {
    // ---- MMAs: tiles of the warp's parity ----
    const int set = warp - 21;
    int ci = 0, ti = 0, wrun = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const Entry& O = E[it.e];
      // every run in turn, with or without a tile: an arrival at wfree must not run ahead of its phase
      if (it.run && !wait(&sh.wfull, wrun++ & 1, limit, abort, 6)) break;
      if ((ti & 1) == set) {
        const int n16 = (O.nw + 15) & ~15;
        const uint32_t id1 = idesc_tf32(128, SPLIT ? 2 * n16 : n16), id2 = idesc_tf32(128, n16);
        const uint32_t td = tmem + kTmemD + set * kTmemDStage;
        if (ti >= 2 && !wait(&sh.dempty[set], ((ti >> 1) + 1) & 1, limit, abort, 7)) break;
        uint32_t wo = 0;  // the chunk's place in the weight
        for (int s = 0; ok && s < O.count; ++s) {
          const int K = S[O.first + s].k;
          for (int k0 = 0; k0 < K; k0 += kKC, ++ci) {
            const int kc = min(kKC, K - k0), steps = (kc + 7) / 8;
            if (!wait(&sh.afull[set], ci & 1, limit, abort, 8)) {
              ok = false;
              break;
            }
            fence_after_sync();
            if (lane == 0) {
              const uint32_t a = tmem + kTmemA + set * kTmemAStage;
              const uint64_t b = sw128_kmajor(smem_u32(sW) + wo);
#pragma unroll
              for (int k = 0; k < kKC / 8; ++k) {
                if (k >= steps) break;
                // (the descriptor's address field counts 16 bytes: 32 bytes a step)
                const uint64_t bk = b + uint64_t((k >> 2) * (kWHalf / 16) + (k & 3) * 2);
                mma_tf32_ta(td, a + 8 * k, bk, id1, wo > 0 || k > 0);
                if (SPLIT) mma_tf32_ta(td + n16, a + kKC + 8 * k, bk, id2, 1);
              }
              mma_commit(&sh.aempty[set]);
            }
            __syncwarp();
            wo += halves_of(kc) * kWHalf;
          }
        }
        if (ok && lane == 0) mma_commit(&sh.dfull[set]);
      }
      // the weight is free once both warps' products with it have completed
      if (ok && it.run_last && lane == 0) mma_commit(&sh.wfree);
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
    chain_wait();
  }
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

// the passes of an output block: its sources' chunks in order, as many as a weight holds
int passes_of(const LinRows& R, const LinOut& O) {
  int pass = 0, halves = 0;
  for (int s = 0; s < O.count; ++s) {
    const int K = R.s[O.first + s].k;
    for (int c = 0; c < chunks_of(K); ++c) {
      const int h = halves_of(std::min(kKC, K - c * kKC));
      if (halves + h > kMaxHalves) ++pass, halves = 0;
      halves += h;
    }
  }
  return pass + 1;
}

}  // namespace

int linear_tc_launches(const LinRows& R) {
  int entries = 0, passes = 1;
  int64_t tiles = 0;
  for (int b = 0; b < R.n_out; ++b) {
    entries += col_tiles(R.o[b].n);
    tiles += (R.N / tile_of(R.o[b].d) + R.T) * col_tiles(R.o[b].n);
    passes = std::max(passes, passes_of(R, R.o[b]));
  }
  return entries <= kLinTcEntries && tiles < kMostCost ? passes : 0;
}

cudaError_t linear_tc_rows(const LinRows& R, bool split, uint64_t limit, bool after, bool more, cudaStream_t st) {
  const bool v = vec4(R);
  auto* kernel = split ? (v ? k_linear_tc<true, 4> : k_linear_tc<true, 1>)
                       : (v ? k_linear_tc<false, 4> : k_linear_tc<false, 1>);
  const int passes = linear_tc_launches(R);
  for (int pass = 0; pass < passes; ++pass) {
    Params P;
    std::memset(&P, 0, sizeof(P));
    P.T = R.T, P.dim_src = R.dim_src, P.dim_out = R.dim_out, P.N = R.N, P.wnumel = R.wnumel;
    for (int i = 0; i < 2; ++i) P.x[i] = R.x[i], P.w[i] = R.w[i];
    P.out = R.out, P.perm = R.perm, P.offsets = R.offsets, P.accumulate = pass > 0;
    int64_t tiles = 0;
    int most = 0;
    for (int b = 0; b < R.n_out; ++b) {
      const LinOut& O = R.o[b];
      // the pass's chunks of the block's sources, neighbours together
      const int first = P.n_src;
      int chunks = 0, halves = 0, at = 0, cur = 0;
      for (int s = 0; s < O.count; ++s) {
        const LinSource& S = R.s[O.first + s];
        int lo = -1, hi = -1;
        for (int c = 0; c < chunks_of(S.k); ++c) {
          const int h = halves_of(std::min(kKC, S.k - c * kKC));
          if (cur + h > kMaxHalves) ++at, cur = 0;
          cur += h;
          if (at != pass) continue;
          if (lo < 0) lo = c;
          hi = c + 1;
          ++chunks;
          halves += h;
        }
        if (lo < 0) continue;
        LinSource& q = P.s[P.n_src++];
        q = S;
        q.off += lo * kKC * O.d, q.woff += int64_t(lo) * kKC * S.rk;
        q.k = std::min(S.k, hi * kKC) - lo * kKC;
      }
      if (pass > 0 && chunks == 0) continue;
      most = std::max(most, halves);
      for (int c0 = 0; c0 < O.n; c0 += kNT) {
        // (measured, l = 0..2: 1.2, 1.05 and 1 times: the more nodes, the more copies to issue)
        P.cut[P.n_entries] = {10 * (chunks + 1) + chunks * tile_of(O.d) / 30, tile_of(O.d), O.d >> 1};
        P.e[P.n_entries++] = {O.d, O.off + c0 * O.d, std::min(kNT, O.n - c0), c0, first, P.n_src - first, 0};
      }
      tiles += (R.N / tile_of(O.d) + std::min<int64_t>(R.T, R.N)) * col_tiles(O.n);
    }
    const int shift = cost_shift(P.cut, P.n_entries, R.N, R.T);
    for (int i = 0; i < P.n_entries; ++i) {
      P.cut[i].cost = std::max(1, P.cut[i].cost >> shift);
      P.coef[P.cut[i].which] += P.cut[i].cost;
    }
    // shared memory: the weight, and for each pipeline an output tile and as many raw chunks (one or two) as fit
    const int fixed = 1024 + most * kWHalf + 2 * kRaw + P.n_src * int(sizeof(LinSource)) +
                      P.n_entries * int(sizeof(Entry) + sizeof(Cut)) + (P.T + 2) * 4;
    static_assert(1024 + kMaxHalves * kWHalf + 4 * kRaw + kLinSources * int(sizeof(LinSource)) +
                          kLinTcEntries * int(sizeof(Entry) + sizeof(Cut)) + (TPCONV_MAX_TYPES + 2) * 4 <=
                      kDynMax,
                  "a raw chunk always fits");
    const int stages = std::min(kMaxStages, (kDynMax - fixed) / (2 * kRaw));
    const int bytes = fixed + 2 * stages * kRaw;
    // (the most a call may ask for, not this call's: another thread's call must not lower it)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynMax);
    if (e) return e;
    const unsigned grid = unsigned(std::min<int64_t>(kSMs, tiles));
    const int next = more && pass == passes - 1;
    if (after && pass == 0) {  // (a later pass reads what the one before wrote)
      e = chain_launch(kernel, grid, kThreads, bytes, st, P, most, stages, next, limit);
    } else {
      kernel<<<grid, kThreads, bytes, st>>>(P, most, stages, next, limit);
      e = cudaGetLastError();
    }
    if (e) return e;
  }
  return cudaSuccess;
}

cudaError_t linear_tc_read_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_linear_error, sizeof(int));
  if (e) return e;
  return *code ? cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(int)) : cudaSuccess;
}

}  // namespace tpc
