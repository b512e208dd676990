// Typed linear map on the tensor cores: rows times the weight of their type
// (sm_100a: tcgen05 with the row operand in TMEM, bulk copies of node rows).
//
//   out[n, w, m] = sum_k x[n, k, m] B_t[k][w]     per (output block, 64 columns, type t)
//
// A tile is the (node, m) rows of up to 128 / (2l+1) nodes of one type, times 64
// output channels.  The weight of the (block, columns, type) is resident in shared
// memory, split once into TF32 hi and lo; the node rows are the only stream:
//   bulk copies gather the nodes' contiguous pieces [64 channels][2l+1] by perm;
//   converter threads, one per row, read their row's channels (stride 2l+1), split
//   them (3xTF32, Ootomo & Yokota, 2022: a_hi = rn_tf32(a), a_lo = rn_tf32(a - a_hi))
//   and store hi and lo as the A operand in TMEM: the transposition from [channel][m]
//   to rows costs one shared-memory read per element and no write;
//   one thread issues D += A_lo B_hi + A_hi B_lo, then A_hi B_hi (the small products
//   first, while the accumulator is small);
//   epilogue threads, one per row, lay D out as [channel][m] and bulk copies scatter
//   the nodes' pieces by perm.
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
// from the device.  Warps 0-3 convert, 4-7 run the epilogue, 8 issues copies, 9 MMAs.
// Every wait is bounded by the call's limit; on expiry the kernel records it, stops
// issuing, waits (bounded) for its own copies and MMAs, frees TMEM and returns.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "linear_tc.h"
#include "linear_tc_common.cuh"

namespace tpc {
namespace {

using namespace tc;

__device__ int g_linear_error;  // first code recorded by an expired wait (0 = none)

constexpr int kNT = 64, kKC = 64;             // columns of a tile, channels of a chunk
constexpr int kMaxChunks = kLinTcChunks;      // chunks of a resident weight
constexpr int kWChunk = 2 * kNT * kKC * 4;    // hi and lo of one chunk: 32 KB
constexpr int kRaw = 33024;                   // a raw chunk or an output tile (see node_pitch)
constexpr int kMaxStages = 4;
constexpr int kSMemMax = 227 * 1024;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 0, kTmemAStage = 128, kTmemD = 256;  // A: 2 x (hi 64 | lo 64), D: 2 x 64

// nodes of a tile; floats of a node's 64 channels plus padding (multiple of 4)
__host__ __device__ constexpr int tile_of(int d) { return d == 1 ? 120 : 128 / d; }
__host__ __device__ constexpr int node_pitch(int d) { return kKC * d + (d == 1 || d == 3 ? 4 : 8); }
static_assert(tile_of(1) * node_pitch(1) * 4 <= kRaw && tile_of(3) * node_pitch(3) * 4 <= kRaw &&
                  tile_of(5) * node_pitch(5) * 4 <= kRaw && tile_of(7) * node_pitch(7) * 4 <= kRaw,
              "a tile fits its buffer");

__host__ __device__ inline int chunks_of(int k) { return (k + kKC - 1) / kKC; }
__host__ __device__ inline int col_tiles(int n) { return (n + kNT - 1) / kNT; }

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t afull[2], aempty[2], dfull[2], dempty[2];
  uint64_t wfull, wfree, fin;
};
struct Shared {
  Bars b;
  uint32_t tmem;
  int abort;
  int total[4];                   // tiles of all groups for d = 1, 3, 5, 7
  int start_t, start_j;           // group and tile of the CTA's first item
};

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort, int code) {
  return wait_or_abort(b, parity, limit, abort, &g_linear_error, code);
}

// ---- the CTA's share of the work -------------------------------------------------
// Entries (output block, 64 columns) in order, in each the tiles of groups 0..T; a
// tile costs its chunks plus one; CTA b owns the tiles whose cost begins in its share.
struct Item {
  int ob, c0, d, t, first, count;
  bool run;       // the first tile with this weight
  bool zero;      // no product: a group without a type, or a block without a source
  bool run_last;  // the last tile of this CTA with this weight
};

struct Walk {
  const LinRows& P;
  const Shared& sh;
  int64_t lo, hi, base = 0;
  int ob = -1, ct = 0, d = 1;
  int64_t left = 0;
  int t = 0, j = 0, gb = 0, ge = 0, tiles = 0;
  bool first_entry = true, fresh = true;

  __device__ Walk(const LinRows& p, const Shared& s, int64_t total) : P(p), sh(s) {
    lo = total * blockIdx.x / gridDim.x;
    hi = total * (blockIdx.x + 1) / gridDim.x;
  }
  __device__ static int cost(const LinRows& P, int ob) {
    int c = 1;
    for (int s = 0; s < P.o[ob].count; ++s) c += chunks_of(P.s[P.o[ob].first + s].k);
    return c;
  }
  __device__ static int64_t total_cost(const LinRows& P, const Shared& s) {
    int64_t c = 0;
    for (int b = 0; b < P.n_out; ++b) c += int64_t(s.total[P.o[b].d >> 1]) * cost(P, b) * col_tiles(P.o[b].n);
    return c;
  }
  // moves to the next entry with tiles of this CTA; its first tile index in *j0
  __device__ bool next_entry(int64_t* j0) {
    for (;;) {
      if (ob < 0) {
        ob = 0;
      } else {
        base += int64_t(sh.total[d >> 1]) * cost(P, ob);
        if (++ct >= col_tiles(P.o[ob].n)) ++ob, ct = 0;
      }
      if (ob >= P.n_out || base >= hi) return false;
      d = P.o[ob].d;
      const int c = cost(P, ob);
      const int64_t n = sh.total[d >> 1];
      const int64_t a = lo <= base ? 0 : min((lo - base + c - 1) / c, n), b = min((hi - base + c - 1) / c, n);
      if (a < b) {
        left = b - a;
        *j0 = a;
        return true;
      }
    }
  }

  __device__ void load_group() {
    lin_group(P.offsets, P.T, P.N, t, &gb, &ge);
    tiles = (ge - gb + tile_of(d) - 1) / tile_of(d);
  }
  __device__ bool next(Item* it) {
    if (left == 0) {
      int64_t j0;
      if (!next_entry(&j0)) return false;
      if (first_entry) {
        t = sh.start_t, j = sh.start_j;  // found once for the CTA's first tile
        first_entry = false;
      } else {
        t = 0, j = 0;
      }
      fresh = true;
      load_group();
    }
    while (j >= tiles) {
      if (t >= P.T) return false;  // (offsets that change under the call)
      ++t, j = 0;
      fresh = true;
      load_group();
    }
    it->ob = ob, it->c0 = ct * kNT, it->d = d, it->t = t;
    it->first = gb + j * tile_of(d);
    it->count = min(tile_of(d), ge - it->first);
    it->run = fresh;
    it->zero = t >= P.T || P.o[ob].count == 0;
    fresh = false;
    ++j, --left;
    it->run_last = left == 0 || j >= tiles;
    return true;
  }
};

// a node's row m, channels k0 .. k0+15 of the raw chunk (zeros at and behind kc)
template <int D>
__device__ __forceinline__ void read_row16(const float* row, int k0, int kc, float (&v)[16]) {
  if constexpr (D == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + 4 * i < kc) q = *reinterpret_cast<const float4*>(row + k0 + 4 * i);
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = k0 + i < kc ? row[(k0 + i) * D] : 0.f;
  }
}
// one chunk of the thread's row: raw -> hi (and lo) in TMEM
template <int D, bool SPLIT>
__device__ __forceinline__ void convert(const float* raw, int r, int kc, uint32_t ta) {
  constexpr int ROWS = tile_of(D) * D;
  const int rr = r < ROWS ? r : ROWS - 1;
  const float* row = raw + (rr / D) * node_pitch(D) + rr % D;
  for (int k0 = 0; k0 < kc; k0 += 16) {
    float v[16], h[16];
    read_row16<D>(row, k0, kc, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      h[i] = rn_tf32(v[i]);
      v[i] = rn_tf32(v[i] - h[i]);
    }
    tmem_st16(ta + k0, h);
    if (SPLIT) tmem_st16(ta + kKC + k0, v);
  }
}
template <int D>
__device__ __forceinline__ void lay_out16(float* stage, int r, int c, const float (&v)[16]) {
  constexpr int ROWS = tile_of(D) * D;
  if (r >= ROWS) return;
  float* row = stage + (r / D) * node_pitch(D) + r % D;
  if constexpr (D == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(row + c + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) row[(c + i) * D] = v[i];
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ LinRows P, int chunks, int stages, int outs, uint64_t limit) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sW = base;
  float* sRaw = reinterpret_cast<float*>(base + chunks * kWChunk);
  float* sOut = reinterpret_cast<float*>(base + chunks * kWChunk + stages * kRaw);
  __shared__ Shared sh;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh.b.full[s], 1);
      mbar_init(&sh.b.empty[s], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.b.afull[i], 128);
      mbar_init(&sh.b.aempty[i], 1);
      mbar_init(&sh.b.dfull[i], 1);
      mbar_init(&sh.b.dempty[i], 128);
    }
    mbar_init(&sh.b.wfull, 128);
    mbar_init(&sh.b.wfree, 1);
    mbar_init(&sh.b.fin, 1);
    sh.abort = 0;
    sh.start_t = sh.start_j = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc(&sh.tmem, kTmemCols);
  // tiles of all groups per degree: warp i for d = 2i + 1
  if (warp < 4) {
    const int d = 2 * warp + 1, unit = tile_of(d);
    int s = 0;
    for (int t = lane; t <= P.T; t += 32) {
      int b, e;
      lin_group(P.offsets, P.T, P.N, t, &b, &e);
      s += (e - b + unit - 1) / unit;
    }
    s = __reduce_add_sync(0xffffffffu, s);
    if (lane == 0) sh.total[warp] = s;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const int64_t total = Walk::total_cost(P, sh);
  // the group of the CTA's first tile
  if (warp == 0) {
    Walk w(P, sh, total);
    int64_t j0;
    if (w.next_entry(&j0)) {
      const int unit = tile_of(w.d);
      int carry = 0;
      for (int t0 = 0; t0 <= P.T; t0 += 32) {
        const int t = t0 + lane;
        int n = 0;
        if (t <= P.T) {
          int b, e;
          lin_group(P.offsets, P.T, P.N, t, &b, &e);
          n = (e - b + unit - 1) / unit;
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += u;
        }
        const int64_t first = int64_t(carry) + s - n;
        if (j0 >= first && j0 < first + n) sh.start_t = t, sh.start_j = int(j0 - first);
        carry += __shfl_sync(0xffffffffu, s, 31);
      }
    }
  }
  __syncthreads();

  Walk walk(P, sh, total);
  Item it;
  if (warp < 4) {
    // ---- weights, and rows to TMEM ----
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + (uint32_t(warp * 32) << 16);
    int ci = 0, wrun = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const LinOut& O = P.o[it.ob];
      if (it.run) {
        // the MMAs of the previous weight have completed
        if (wrun > 0 && !wait(&sh.b.wfree, (wrun - 1) & 1, limit, abort, 1)) break;
        const int nw = min(kNT, O.n - it.c0), n = threadIdx.x & 63;
        int c = 0;
        for (int s = 0; s < O.count; ++s) {
          const LinSource& S = P.s[O.first + s];
          const float* w = P.w[S.pair] + int64_t(it.t) * P.wnumel + S.woff + int64_t(it.c0 + n) * S.rw;
          for (int k0 = 0; k0 < S.k; k0 += kKC, ++c) {
            unsigned char* hi = sW + c * kWChunk;
            const int kc = min(kKC, S.k - k0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int q = (threadIdx.x >> 6) + 2 * i;  // channels 4q .. 4q+3
              float v[4], h[4], l[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = (n < nw && 4 * q + e < kc) ? __ldg(w + int64_t(k0 + 4 * q + e) * S.rk) : 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = rn_tf32(v[e]), l[e] = rn_tf32(v[e] - h[e]);
              const int off = (q >> 3) * (kNT * 128) + n * 128 + (((q & 7) ^ (n & 7)) << 4);
              *reinterpret_cast<float4*>(hi + off) = make_float4(h[0], h[1], h[2], h[3]);
              if (SPLIT) *reinterpret_cast<float4*>(hi + kNT * kKC * 4 + off) = make_float4(l[0], l[1], l[2], l[3]);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&sh.b.wfull);
        ++wrun;
      }
      for (int s = 0; ok && s < O.count; ++s) {
        const int K = P.s[O.first + s].k;
        for (int k0 = 0; k0 < K; k0 += kKC, ++ci) {
          const int st = ci % stages, ab = ci & 1, kc = min(kKC, K - k0);
          if (ci >= 2 && !wait(&sh.b.aempty[ab], ((ci >> 1) + 1) & 1, limit, abort, 2)) ok = false;
          if (ok && !wait(&sh.b.full[st], (ci / stages) & 1, limit, abort, 3)) ok = false;
          if (!ok) break;
          fence_after_sync();
          const float* raw = sRaw + st * (kRaw / 4);
          const uint32_t ta = lane_base + kTmemA + ab * kTmemAStage;
          switch (it.d) {
            case 1: convert<1, SPLIT>(raw, r, kc, ta); break;
            case 3: convert<3, SPLIT>(raw, r, kc, ta); break;
            case 5: convert<5, SPLIT>(raw, r, kc, ta); break;
            default: convert<7, SPLIT>(raw, r, kc, ta); break;
          }
          mbar_arrive(&sh.b.empty[st]);
          tmem_wait_st();
          fence_before_sync();
          mbar_arrive(&sh.b.afull[ab]);
        }
      }
    }
  } else if (warp < 8) {
    // ---- epilogue ----
    const int r = threadIdx.x - 128;
    const uint32_t lane_base = tmem + (uint32_t((warp - 4) * 32) << 16);
    int ti = 0, oi = 0;
    bool ok = true;  // a warp that gave up keeps passing the group's barriers
    while (walk.next(&it)) {
      const LinOut& O = P.o[it.ob];
      const int db = ti & 1, nw = min(kNT, O.n - it.c0);
      float* stage = sOut + (oi % outs) * (kRaw / 4);
      // the copies that read this buffer two (one) tiles ago have read it
      if (outs == 1)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      else
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok && !it.zero) {
        ok = wait(&sh.b.dfull[db], (ti >> 1) & 1, limit, abort, 4);
        if (ok) {
          fence_after_sync();
          for (int c = 0; c < nw; c += 16) {
            float v[16];
            tmem_ld16(lane_base + kTmemD + db * kNT + c, v);
            switch (it.d) {
              case 1: lay_out16<1>(stage, r, c, v); break;
              case 3: lay_out16<3>(stage, r, c, v); break;
              case 5: lay_out16<5>(stage, r, c, v); break;
              default: lay_out16<7>(stage, r, c, v); break;
            }
          }
          fence_before_sync();
          mbar_arrive(&sh.b.dempty[db]);
        }
      } else if (ok) {
        for (int i = r; i < tile_of(it.d) * node_pitch(it.d) / 4; i += 128)
          reinterpret_cast<float4*>(stage)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (!it.zero) ++ti;
      ++oi;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok && !*abort && r < it.count) {
        const int n = P.perm[it.first + r];
        if (n >= 0 && n < P.N)
          bulk_store(P.out + int64_t(n) * P.dim_out + O.off + it.c0 * it.d,
                     smem_u32(stage + r * node_pitch(it.d)), uint32_t(nw * it.d * 4));
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp == 8) {
    // ---- node rows to shared memory ----
    int ci = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const LinOut& O = P.o[it.ob];
      int node[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = lane + 32 * i;
        node[i] = q < it.count ? P.perm[it.first + q] : 0;
        if (node[i] < 0 || node[i] >= P.N) node[i] = 0;  // (its row is not stored)
      }
      for (int s = 0; ok && s < O.count; ++s) {
        const LinSource& S = P.s[O.first + s];
        for (int k0 = 0; k0 < S.k; k0 += kKC, ++ci) {
          const int st = ci % stages;
          const uint32_t bytes = uint32_t(min(kKC, S.k - k0) * it.d * 4);
          if (ci >= stages && !wait(&sh.b.empty[st], ((ci / stages) + 1) & 1, limit, abort, 5)) ok = false;
          ok = __all_sync(0xffffffffu, ok && !*abort);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&sh.b.full[st], bytes * it.count);
          __syncwarp();
          const float* x = P.x[S.pair] + S.off + k0 * it.d;
          const uint32_t dst = smem_u32(sRaw + st * (kRaw / 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int q = lane + 32 * i;
            if (q < it.count)
              bulk_load(dst + q * node_pitch(it.d) * 4, x + int64_t(node[i]) * P.dim_src, bytes, &sh.b.full[st]);
          }
        }
      }
    }
    // no copy may be in flight when the CTA ends
    if (*abort)
      for (int c = (ci > stages ? ci - stages : 0); c < ci; ++c)
        if (!mbar_wait_for(&sh.b.full[c % stages], (c / stages) & 1, kDrainLimitNs)) break;
  } else {
    // ---- MMAs ----
    int ci = 0, ti = 0, wrun = 0;
    bool ok = true;
    while (ok && walk.next(&it)) {
      if (it.zero) continue;
      const LinOut& O = P.o[it.ob];
      const int db = ti & 1, nw = min(kNT, O.n - it.c0);
      const uint32_t idesc = idesc_tf32(128, (nw + 15) & ~15);
      const uint32_t td = tmem + kTmemD + db * kNT;
      if (it.run && !wait(&sh.b.wfull, wrun & 1, limit, abort, 6)) break;
      if (it.run) ++wrun;
      if (ti >= 2 && !wait(&sh.b.dempty[db], ((ti >> 1) + 1) & 1, limit, abort, 7)) break;
      uint32_t acc = 0;
      int wc = 0;
      for (int s = 0; ok && s < O.count; ++s) {
        const int K = P.s[O.first + s].k;
        for (int k0 = 0; k0 < K; k0 += kKC, ++ci, ++wc) {
          const int ab = ci & 1, steps = (min(kKC, K - k0) + 7) / 8;
          if (!wait(&sh.b.afull[ab], (ci >> 1) & 1, limit, abort, 8)) {
            ok = false;
            break;
          }
          fence_after_sync();
          if (lane == 0) {
            const uint32_t ah = tmem + kTmemA + ab * kTmemAStage, al = ah + kKC;
            const uint32_t bh = smem_u32(sW + wc * kWChunk), bl = bh + kNT * kKC * 4;
            auto off = [](int k) { return uint32_t((k >> 2) * (kNT * 128) + (k & 3) * 32); };
            if (SPLIT) {
              for (int k = 0; k < steps; ++k) {
                mma_tf32_ta(td, al + 8 * k, sw128_kmajor(bh + off(k)), idesc, acc);
                acc = 1;
                mma_tf32_ta(td, ah + 8 * k, sw128_kmajor(bl + off(k)), idesc, 1);
              }
            }
            for (int k = 0; k < steps; ++k) {
              mma_tf32_ta(td, ah + 8 * k, sw128_kmajor(bh + off(k)), idesc, acc);
              acc = 1;
            }
            mma_commit(&sh.b.aempty[ab]);
          }
          __syncwarp();
        }
      }
      if (ok && lane == 0) {
        mma_commit(&sh.b.dfull[db]);
        if (it.run_last) mma_commit(&sh.b.wfree);
      }
      __syncwarp();
      ++ti;
    }
    if (lane == 0) {
      mma_commit(&sh.b.fin);
      mbar_wait_for(&sh.b.fin, 0, kDrainLimitNs);  // no MMA may be in flight when TMEM is freed
    }
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kSMs = 148;

}  // namespace

bool linear_tc_supported(const LinRows& R) {
  const auto bad = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
  if (R.dim_src % 4 || R.dim_out % 4 || bad(R.out)) return false;
  int entries = 0;
  for (int b = 0; b < R.n_out; ++b) {
    const LinOut& O = R.o[b];
    if (O.n % 4 || O.off % 4) return false;
    entries += col_tiles(O.n);
    int c = 0;
    for (int s = 0; s < O.count; ++s) {
      const LinSource& S = R.s[O.first + s];
      if (S.k % 4 || S.off % 4 || bad(R.x[S.pair])) return false;
      c += chunks_of(S.k);
    }
    if (c > kMaxChunks) return false;
  }
  return entries <= kLinTcEntries;
}

cudaError_t linear_tc_rows(const LinRows& R, bool split, uint64_t limit, cudaStream_t st) {
  int chunks = 0;
  int64_t tiles = 0;
  for (int b = 0; b < R.n_out; ++b) {
    const LinOut& O = R.o[b];
    int c = 0;
    for (int s = 0; s < O.count; ++s) c += chunks_of(R.s[O.first + s].k);
    chunks = std::max(chunks, c);
    tiles += (R.N / tile_of(O.d) + std::min<int64_t>(R.T + 1, R.N)) * col_tiles(O.n);
  }
  // shared memory: the weight, then as many raw stages (two to four) and output buffers (one or two) as fit
  const int room = (kSMemMax - 1024 - int(sizeof(Shared)) - 256 - chunks * kWChunk) / kRaw;
  const int outs = room >= 5 ? 2 : 1, stages = std::min(kMaxStages, room - outs);
  if (stages < 2) return cudaErrorInvalidValue;
  const int sm = 1024 + chunks * kWChunk + (stages + outs) * kRaw;
  auto* k = split ? k_linear_tc<true> : k_linear_tc<false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
  if (e) return e;
  k<<<unsigned(std::min<int64_t>(kSMs, tiles)), kThreads, sm, st>>>(R, chunks, stages, outs, limit);
  return cudaGetLastError();
}

cudaError_t linear_tc_read_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_linear_error, sizeof(int));
  if (e) return e;
  return *code ? cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(int)) : cudaSuccess;
}

}  // namespace tpc
