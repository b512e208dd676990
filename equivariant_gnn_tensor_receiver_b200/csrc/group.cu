// Nodes grouped by type: a stable counting sort with one digit (sm_100a).
//
//   perm    = node ids by key, ascending inside a key (key = type, or n_types for
//             any other value), offsets[t] = number of nodes with a key below t.
//
// The N ids are cut into tiles of consecutive nodes, worked on up to 8192 at a time.  A
// tile's warps own consecutive pieces of up to 256; the lanes of a warp that hold the same key
// find each other (match) and their ranks follow from the lane order, so a node's place is
//   offsets[key] + nodes of that key in earlier tiles + in earlier warps + rank:
// no atomics decide an order, and the result is the stable one.
// Up to kSingle nodes run as one tile in one launch (the call's latency is all);
// more run as two launches: histograms per tile (shared-memory atomics: a count has no
// order), then every tile adds up the histograms before its own (a table of
// (n_types + 1) x tiles ints that stays in L2) and scatters.  Work: 4 bytes read twice
// and 4 written per node.
// Measured (device): 1.2 M nodes of 89 types 27 us, of which the second launch takes 22; the
// bytes alone are 2 us.  Its warps wait for global memory (the table of histograms, the
// types), for matches and shared memory, and at barriers, in about equal parts, a third of the
// issue slots used; 32 registers a thread spill 56 bytes.  Up to 8192 nodes 8.3 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/tpconv.h"
#include "chain.cuh"
#include "node_ops.h"

namespace tpc {
namespace {

constexpr int kWarps = 32;                 // of a CTA
constexpr int kKeys = TPCONV_MAX_TYPES + 1;
constexpr int kSteps = 8;                  // nodes of a lane at a time, at most
constexpr int kStep = 32 * kWarps;         // nodes of a CTA in a step
constexpr int kSingle = kStep * kSteps;    // nodes handled by one CTA alone
constexpr int kMaxTiles = 296;             // two CTAs of 1024 threads per SM: one wave

// the keys of the lane's nodes first, first + 32, ... of `steps` steps; -1 behind n
__device__ __forceinline__ void load_keys(const int* type, int64_t first, int64_t n, int steps, int T,
                                          int (&key)[kSteps]) {
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t p = first + 32 * i;
    const bool in = i < steps && p < n;
    const int t = in ? type[p] : 0;
    key[i] = in ? ((t >= 0 && t < T) ? t : T) : -1;
  }
}

__global__ void __launch_bounds__(kWarps * 32) k_group_count(int64_t N, int64_t tile, int steps, int T, int tiles,
                                                             const int* __restrict__ type, int* __restrict__ hist) {
  chain_next();
  __shared__ int cnt[4][kKeys];  // (copies: less contention on a common type)
  const int K = T + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 4 * kKeys; i += blockDim.x) cnt[i / kKeys][i % kKeys] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * tile, t1 = min(t0 + tile, N);
  for (int64_t s = t0; s < t1; s += kStep * steps) {
    int key[kSteps];
    load_keys(type, s + warp * 32 * steps + lane, t1, steps, T, key);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (key[i] >= 0) atomicAdd(&cnt[warp & 3][key[i]], 1);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < K; k += blockDim.x)
    hist[int64_t(k) * tiles + blockIdx.x] = cnt[0][k] + cnt[1][k] + cnt[2][k] + cnt[3][k];
}

// place of every node of one tile.  tiles == 1: the tile is everything and no
// histogram table is read.
__global__ void __launch_bounds__(kWarps * 32, 2) k_group_place(int64_t N, int64_t tile, int steps, int T, int tiles,
                                                             const int* __restrict__ type,
                                                             const int* hist, int* __restrict__ perm,
                                                             int* __restrict__ offsets) {
  extern __shared__ int cnt[];  // [kWarps][K] counts, then cursors; [K] next place, [K] totals
  const int K = T + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* place = cnt + kWarps * K;
  int* total = place + K;
  const int64_t t0 = blockIdx.x * tile, t1 = min(t0 + tile, N);
  if (tiles > 1) {
    chain_wait();
    // key by key, the warps' lanes add up the tiles' histograms
    for (int k = warp; k < K; k += kWarps) {
      int b = 0, s = 0;
#pragma unroll 8
      for (int t = lane; t < tiles; t += 32) {
        const int h = hist[int64_t(k) * tiles + t];
        s += h;
        b += t < int(blockIdx.x) ? h : 0;
      }
      s = __reduce_add_sync(0xffffffffu, s);
      b = __reduce_add_sync(0xffffffffu, b);
      if (lane == 0) place[k] = b, total[k] = s;
    }
  } else {
    for (int k = threadIdx.x; k < K; k += blockDim.x) place[k] = total[k] = 0;
    __syncthreads();
    for (int64_t s = t0; s < t1; s += kStep * steps) {
      int key[kSteps];
      load_keys(type, s + warp * 32 * steps + lane, t1, steps, T, key);
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (key[i] >= 0) atomicAdd(&total[key[i]], 1);
    }
  }
  __syncthreads();
  if (warp == 0) {  // exclusive scan of the totals over the keys
    int carry = 0;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int k = k0 + lane;
      const int v = k < K ? total[k] : 0;
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      if (k < K) {
        const int first = carry + s - v;
        if (blockIdx.x == 0) offsets[k] = first;  // offsets[T] = first node of no group
        place[k] += first;
      }
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
  }
  int* mine = cnt + warp * K;
  for (int64_t s = t0; s < t1; s += kStep * steps) {
    const int64_t first = s + warp * 32 * steps + lane;
    int key[kSteps], rank[kSteps];
    load_keys(type, first, t1, steps, T, key);
    for (int k = lane; k < K; k += 32) mine[k] = 0;
    __syncwarp();
    // ranks inside the warp's piece
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i >= steps) break;
      const unsigned peers = __match_any_sync(0xffffffffu, key[i]);
      const int before = __popc(peers & ((1u << lane) - 1));
      rank[i] = key[i] >= 0 ? mine[key[i]] + before : 0;
      __syncwarp();
      if (key[i] >= 0 && before == 0) mine[key[i]] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += blockDim.x) {
      int at = place[k];
#pragma unroll 8
      for (int w = 0; w < kWarps; ++w) {
        const int c = cnt[w * K + k];
        cnt[w * K + k] = at;
        at += c;
      }
      place[k] = at;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (key[i] >= 0) perm[mine[key[i]] + rank[i]] = int(first + 32 * i);
    __syncthreads();
  }
}

// steps of a CTA at a time, and nodes of a tile (a multiple of those steps)
int steps_of(int64_t N) {
  return int(std::min<int64_t>(kSteps, (N + int64_t(kMaxTiles) * kStep - 1) / (int64_t(kMaxTiles) * kStep)));
}
int64_t tile_nodes(int64_t N) {
  const int64_t sub = int64_t(kStep) * steps_of(N);
  return ((N + kMaxTiles - 1) / kMaxTiles + sub - 1) / sub * sub;
}

size_t place_smem(int T) { return size_t(kWarps + 2) * (T + 1) * 4; }
static_assert((kWarps + 2) * kKeys * 4 <= 48 * 1024, "the counters fit the default shared memory");

bool group_args(int64_t N, int n_types) {
  return N >= 0 && N < (int64_t(1) << 31) && n_types >= 1 && n_types <= TPCONV_MAX_TYPES;
}
size_t group_bytes(int64_t N, int T) {
  if (N <= kSingle) return 0;
  const int64_t tile = tile_nodes(N), tiles = (N + tile - 1) / tile;
  return (size_t(tiles) * (T + 1) * 4 + 255) & ~size_t(255);
}

}  // namespace
}  // namespace tpc

using namespace tpc;

extern "C" {

int tpconv_group_workspace_size(int64_t N, int n_types, size_t* bytes) {
  if (!bytes || !group_args(N, n_types)) return TPCONV_ERR_INVALID_ARG;
  *bytes = group_bytes(N, n_types);
  return TPCONV_OK;
}

int tpconv_group_nodes(int64_t N, int n_types, const int32_t* type, int32_t* perm, int32_t* offsets, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!group_args(N, n_types) || !offsets || (N > 0 && (!type || !perm))) return TPCONV_ERR_INVALID_ARG;
  if (misaligned(type, 4) || misaligned(perm, 4) || misaligned(offsets, 4)) return TPCONV_ERR_INVALID_ARG;
  const size_t need = group_bytes(N, n_types);
  if (workspace_bytes < need) return TPCONV_ERR_WORKSPACE_TOO_SMALL;
  if (need && (!workspace || misaligned(workspace, 256))) return TPCONV_ERR_INVALID_ARG;
  const Span sp[] = {{perm, size_t(N) * 4}, {offsets, size_t(n_types + 1) * 4}, {workspace, need},
                     {type, size_t(N) * 4}};
  if (overlapping(sp, 3, 4)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NodePhase ph(TPCONV_PHASE_GROUP, st);
  if (N <= kSingle) {
    k_group_place<<<1, kWarps * 32, place_smem(n_types), st>>>(
        N, kSingle, int(std::max<int64_t>(1, (N + kStep - 1) / kStep)), n_types, 1, type, nullptr, perm, offsets);
    ph.note(1);
  } else {
    const int64_t tile = tile_nodes(N);
    const int tiles = int((N + tile - 1) / tile);
    int* hist = static_cast<int*>(workspace);
    k_group_count<<<tiles, kWarps * 32, 0, st>>>(N, tile, steps_of(N), n_types, tiles, type, hist);
    if (cudaGetLastError()) return TPCONV_ERR_CUDA;
    ph.note(2);
    if (chain_launch(k_group_place, tiles, kWarps * 32, place_smem(n_types), st, N, tile, steps_of(N), n_types, tiles,
                     type, static_cast<const int*>(hist), perm, offsets))
      return TPCONV_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? TPCONV_OK : TPCONV_ERR_CUDA;
}

}  // extern "C"
