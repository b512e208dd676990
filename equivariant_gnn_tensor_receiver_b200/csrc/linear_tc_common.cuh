// Device helpers shared by the tensor-core kernels of the typed linear map.
#pragma once

#include "linear.h"
#include "tc_common.cuh"

namespace tpc {
namespace tc {

// D (+)= A B with A in TMEM (lane = row, one column per K element), B through a shared-memory descriptor
__device__ __forceinline__ void mma_tf32_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// 16 fp32 per lane into consecutive TMEM columns of the warp's lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// TF32 halves of a: hi = a rounded to nearest (ties away from zero), lo = the exact
// remainder, of which the tensor core reads the first 11 bits.  By integer
// arithmetic: the conversion instruction runs at a quarter of the rate, and two a
// value were what bounded the kernels.  (Infinities and NaN end as NaN through lo.)
__device__ __forceinline__ float tf32_hi(float a) {
  return __uint_as_float((__float_as_uint(a) + 0x1000u) & 0xffffe000u);
}
// hi (and lo) of one operand value: SPLIT as above, else the value rounded to TF32
template <bool SPLIT>
__device__ __forceinline__ void tf32_split(float a, float& hi, float& lo) {
  if constexpr (SPLIT) {
    hi = tf32_hi(a);
    lo = a - hi;
  } else {
    hi = rn_tf32(a);
    lo = 0.f;
  }
}

// asynchronous copies of one float to shared memory, and their arrival on a barrier
__device__ __forceinline__ void copy_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Brings the node ids some tiles ahead into L2: a tile's copies are issued in less time than
// HBM answers, so that reading the ids one tile ahead alone would bound them.
constexpr int kPermAhead = 512;
__device__ __forceinline__ void prefetch_nodes(const int* perm, unsigned at, int64_t N) {
  if (at < N) asm volatile("prefetch.global.L2 [%0];" ::"l"(perm + at));
}

// untiled bulk copies: both addresses and the size are multiples of 16 bytes
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
// The ring's copy warps arrive on a stage's barrier with the bytes of their own bulk
// copies.  At the end (after an abort the warps may have stopped at different chunks) the
// arrivals that a warp left out are made up for, and the last chunks are waited for,
// bounded: no copy is in flight when the CTA ends.  issued: the chunks of each of the
// `warps` copy warps, written before a barrier of theirs.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int chunk, const volatile int* issued, int warps) {
  int m = chunk;
  for (int w = 0; w < warps; ++w) m = max(m, issued[w]);
  if ((threadIdx.x & 31) == 0)
    for (int c = chunk; c < m; ++c) mbar_arrive(&full[c % stages]);
  for (int c = max(m - stages, 0); c < m; ++c)
    if (!mbar_wait_for(&full[c % stages], (c / stages) & 1, kDrainLimitNs)) break;
}

// How `threads` threads share rows of `n` pieces (of one or four floats): as many whole rows at a time as
// fit (or, for longer rows, the pieces of one row in turn); a thread keeps its place
// in the row, so that a step costs an addition and not a division.
struct RowShare {
  int row, at;       // this thread's first row and piece
  int rows, pieces;  // rows, or pieces of one row, that a step covers
  __device__ __forceinline__ RowShare(int n, int thread, int threads) {
    const int r = threads / n;
    rows = r > 0 ? r : 1;
    pieces = r > 0 ? n : threads;
    row = r > 0 ? thread / n : 0;
    at = r > 0 ? thread - row * n : thread;
    if (row >= rows) at = n;  // a thread left over
  }
};

// one piece of rows w.row, w.row + w.rows, ... < count: row q of node nodes[q] at src (+ its
// node's offset) to to + (q - w.row) pitch bytes; the ids of four rows are read at a time, as
// no read is moved across a copy
__device__ __forceinline__ void copy_rows(const float* src, int dim, const int* nodes, const RowShare& w, int count,
                                          uint32_t to, int pitch) {
  for (int q = w.row; q < count; q += 4 * w.rows, to += 4 * w.rows * pitch) {
    int n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = q + i * w.rows < count ? nodes[q + i * w.rows] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n[i] >= 0) copy_async(to + i * w.rows * pitch, src + int64_t(n[i]) * dim);
  }
}

__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait that also ends when another role gave up; the same answer for the
// whole warp.  A wait that takes longer than the limit is recorded in *error and
// raises the CTA's abort flag, even when its phase completes in the end (a single
// try may sleep past a short limit).
__device__ __forceinline__ bool wait_or_abort(uint64_t* b, uint32_t parity, uint64_t limit, volatile int* abort,
                                              int* error, int code) {
  bool ok = mbar_test(b, parity);
  if (!ok) {
    const uint64_t t0 = global_ns();
    for (;;) {
      ok = mbar_try(b, parity);
      if (global_ns() - t0 > limit) {
        atomicCAS(error, 0, code);
        *abort = 1;
        ok = false;
        break;
      }
      if (ok || *abort) break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// ---- ragged groups ---------------------------------------------------------------
// offs[0 .. T + 1] in shared memory: where each group begins (clamped to [0, N]), N at
// the end; group T holds the nodes without a type.
__device__ __forceinline__ void load_offsets(int* offs, const int* offsets, int T, int64_t N) {
  for (int t = threadIdx.x; t <= T + 1; t += blockDim.x)
    offs[t] = t <= T ? min(max(offsets[t], 0), int(N)) : int(N);
}
__device__ __forceinline__ int group_units(const int* offs, int t, int unit) {
  const int n = offs[t + 1] - offs[t];
  return n > 0 ? units_of(n, unit) : 0;
}
// units of the first `groups` groups; one warp, the same answer in every lane
__device__ __forceinline__ int count_units(const int* offs, int groups, int unit) {
  int s = 0;
  for (int t = threadIdx.x & 31; t < groups; t += 32) s += group_units(offs, t, unit);
  return __reduce_add_sync(0xffffffffu, s);
}
// the group of unit `at`, and its index there
__device__ __forceinline__ void seek_unit(const int* offs, int groups, int unit, int at, int* t, int* j) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  *t = groups, *j = 0;
  for (int t0 = 0; t0 < groups; t0 += 32) {
    const int n = t0 + lane < groups ? group_units(offs, t0 + lane, unit) : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    const int first = carry + s - n;
    const unsigned hit = __ballot_sync(0xffffffffu, at >= first && at < first + n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      *t = t0 + src;
      *j = at - __shfl_sync(0xffffffffu, first, src);
      return;
    }
    carry += __shfl_sync(0xffffffffu, s, 31);
  }
}

// The first cost of share b of `shares` equal ones.  Costs are 32-bit (the host scales
// them to a total below 2^31): the walks are short, and 64-bit divisions made them the
// longest part of a small call.
__device__ __forceinline__ int share_begin(int total, int b, int shares) {
  const int q = total / shares;
  return q * b + min(b, total - q * shares);
}

// ---- a CTA's share of a list of work ----------------------------------------------
// Entries in order, in each the units (tiles or chunks of `nodes` consecutive nodes) of
// the types; share b owns the units whose cost begins in it, and meets them as runs:
// nodes [first, end) of one type in one entry.  Every warp walks the same list by
// itself; where it stands between two runs is kept in shared memory (a register copy in
// every role cost more than the walk: 600 cycles a tile), and next_run is one function.
struct Cut {
  int cost, nodes, which;  // of a unit; which: index of the unit kind's total
};
struct Run {
  int e, t, first, end;  // e < 0: no more
};
struct WalkState {
  int base, lo, hi;    // cost before the entry, the share's costs
  int left, e, t, at;  // units of the share left in the entry, entry, type, next node
};
__device__ __forceinline__ void walk_begin(WalkState* w, int total) {
  if ((threadIdx.x & 31) == 0) {
    w->base = 0;
    w->lo = share_begin(total, blockIdx.x, gridDim.x);
    w->hi = share_begin(total, blockIdx.x + 1, gridDim.x);
    w->left = 0, w->e = -1, w->t = 0, w->at = 0;
  }
  __syncwarp();
}
static __device__ __noinline__ Run next_run(WalkState* w, const Cut* cuts, int n_cuts, const int* total,
                                            const int* offs, int T) {
  WalkState s = *w;
  __syncwarp();
  if (s.e >= n_cuts) return {-1, 0, 0, 0};
  if (s.left == 0) {
    for (;;) {
      if (s.e >= 0) s.base += total[cuts[s.e].which] * cuts[s.e].cost;
      if (++s.e >= n_cuts || s.base >= s.hi) {
        if ((threadIdx.x & 31) == 0) w->e = n_cuts, w->left = 0, w->base = s.hi;
        __syncwarp();
        return {-1, 0, 0, 0};
      }
      const int c = cuts[s.e].cost;
      const int n = total[cuts[s.e].which];
      const int a = s.lo <= s.base ? 0 : min((s.lo - s.base + c - 1) / c, n), b = min((s.hi - s.base + c - 1) / c, n);
      if (a < b) {
        s.left = b - a;
        int j;
        seek_unit(offs, T, cuts[s.e].nodes, a, &s.t, &j);
        s.at = s.t < T ? offs[s.t] + j * cuts[s.e].nodes : 0;
        break;
      }
    }
  } else {
    ++s.t;
    s.at = s.t < T ? offs[s.t] : 0;
  }
  const int nodes = cuts[s.e].nodes;
  while (s.t < T && s.at >= offs[s.t + 1]) {
    ++s.t;
    s.at = s.t < T ? offs[s.t] : 0;
  }
  Run r{-1, 0, 0, 0};
  if (s.t < T) {
    const int end = offs[s.t + 1], all = units_of(end - s.at, nodes);
    const bool whole = all <= s.left;  // (the whole tiles alone end below 2^31)
    r = {s.e, s.t, s.at, whole ? end : s.at + s.left * nodes};
    s.left -= whole ? all : s.left;
  }
  if ((threadIdx.x & 31) == 0) *w = s;
  __syncwarp();
  return r;
}

// The most that a list may cost, and so the most units it may have: a call with more runs on the FP32 pipes.  (48 paths between 1x1o blocks and 940 million nodes have more.)
constexpr int64_t kMostCost = (int64_t(1) << 31) - (1 << 20);

// how far the costs of a list are to be shifted down (to 1 at least) for a total below 2^31
inline int cost_shift(const Cut* cuts, int n, int64_t nodes, int T) {
  for (int s = 0;; ++s) {
    int64_t total = 0;
    for (int i = 0; i < n; ++i)
      total += (nodes / cuts[i].nodes + T) * (cuts[i].cost >> s > 1 ? cuts[i].cost >> s : 1);
    if (total < kMostCost || s == 31) return s;
  }
}

}  // namespace tc
}  // namespace tpc
