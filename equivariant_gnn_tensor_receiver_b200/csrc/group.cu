// Nodes grouped by type: a stable counting sort with one digit (sm_100a).
//
//   perm    = node ids by key, ascending inside a key (key = type, or n_types for
//             any other value), offsets[t] = number of nodes with a key below t.
//
// The N ids are cut into tiles of consecutive nodes.  A tile's warps own
// consecutive pieces of it; the lanes of a warp that hold the same key find each
// other (match) and their ranks follow from the lane order, so a node's place is
//   offsets[key] + nodes of that key in earlier tiles + in earlier warps + rank:
// no atomics decide an order, and the result is the stable one.
// Up to kSingle nodes run as one tile in one launch (the call's latency is all);
// more run as two launches: histograms per tile, then every tile adds up the
// histograms before its own (a table of tiles x (n_types + 1) ints that stays in
// L2) and scatters.  Work: 4 bytes read twice and 4 written per node.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/tpconv.h"
#include "node_ops.h"

namespace tpc {
namespace {

constexpr int kWarps = 32;                 // of a CTA
constexpr int kKeys = TPCONV_MAX_TYPES + 1;
constexpr int kSingle = 8192;              // nodes handled by one CTA alone
constexpr int kTile = 4096;                // nodes of a tile otherwise (at least)
constexpr int kMaxTiles = 592;

__device__ __forceinline__ int key_of(const int* type, int64_t i, int T) {
  const int t = type[i];
  return (t >= 0 && t < T) ? t : T;
}

// nodes of a tile for N nodes: a multiple of 32 * kWarps
inline int64_t tile_nodes(int64_t N) {
  int64_t per = (N + kMaxTiles - 1) / kMaxTiles;
  per = std::max<int64_t>(per, kTile);
  return (per + 32 * kWarps - 1) / (32 * kWarps) * (32 * kWarps);
}

// cnt[warp][key] = nodes of that key in the warp's piece [w0, w1) of the tile
__device__ __forceinline__ void count_piece(const int* type, int64_t w0, int64_t w1, int T, int* mine) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = w0; i < w1; i += 32) {
    const int64_t n = i + lane;
    const bool in = n < w1;
    const int k = in ? key_of(type, n, T) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, k);
    if (in && lane == __ffs(peers) - 1) mine[k] += __popc(peers);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kWarps * 32) k_group_count(int64_t N, int64_t tile, int T,
                                                             const int* __restrict__ type, int* __restrict__ hist) {
  extern __shared__ int cnt[];  // [kWarps][T + 1]
  const int K = T + 1, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * K; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * tile, piece = tile / kWarps;
  const int64_t w0 = min(t0 + warp * piece, N), w1 = min(t0 + (warp + 1) * piece, N);
  count_piece(type, w0, w1, T, cnt + warp * K);
  __syncthreads();
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    int s = 0;
    for (int w = 0; w < kWarps; ++w) s += cnt[w * K + k];
    hist[int64_t(blockIdx.x) * K + k] = s;
  }
}

// place of every node of one tile.  tiles == 1: the tile is everything and no
// histogram table is read.
__global__ void __launch_bounds__(kWarps * 32) k_group_place(int64_t N, int64_t tile, int T, int tiles,
                                                             const int* __restrict__ type,
                                                             const int* __restrict__ hist, int* __restrict__ perm,
                                                             int* __restrict__ offsets) {
  extern __shared__ int cnt[];  // [kWarps][K] counts, then cursors; [K] before, [K] totals
  const int K = T + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* before = cnt + kWarps * K;
  int* total = before + K;
  for (int i = threadIdx.x; i < (kWarps + 2) * K; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * tile, piece = tile / kWarps;
  const int64_t w0 = min(t0 + warp * piece, N), w1 = min(t0 + (warp + 1) * piece, N);
  count_piece(type, w0, w1, T, cnt + warp * K);
  if (tiles > 1) {
    // key by key, the warps' lanes add up the tiles' histograms
    for (int k = warp; k < K; k += kWarps) {
      int b = 0, s = 0;
      for (int t = lane; t < tiles; t += 32) {
        const int h = hist[int64_t(t) * K + k];
        s += h;
        if (t < int(blockIdx.x)) b += h;
      }
      s = __reduce_add_sync(0xffffffffu, s);
      b = __reduce_add_sync(0xffffffffu, b);
      if (lane == 0) before[k] = b, total[k] = s;
    }
  }
  __syncthreads();
  if (tiles == 1) {
    for (int k = threadIdx.x; k < K; k += blockDim.x) {
      int s = 0;
      for (int w = 0; w < kWarps; ++w) s += cnt[w * K + k];
      total[k] = s;
    }
    __syncthreads();
  }
  // exclusive scan of the totals over the keys (one warp), then the cursors
  if (warp == 0) {
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
        before[k] += first;
      }
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    int s = before[k];
    for (int w = 0; w < kWarps; ++w) {
      const int c = cnt[w * K + k];
      cnt[w * K + k] = s;
      s += c;
    }
  }
  __syncthreads();
  int* cur = cnt + warp * K;
  for (int64_t i = w0; i < w1; i += 32) {
    const int64_t n = i + lane;
    const bool in = n < w1;
    const int k = in ? key_of(type, n, T) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, k);
    const int rank = __popc(peers & ((1u << lane) - 1));
    if (in) perm[cur[k] + rank] = int(n);
    __syncwarp();
    if (in && rank == 0) cur[k] += __popc(peers);
    __syncwarp();
  }
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
    k_group_place<<<1, kWarps * 32, place_smem(n_types), st>>>(N, kSingle, n_types, 1, type, nullptr, perm, offsets);
    ph.note(1);
  } else {
    const int64_t tile = tile_nodes(N);
    const int tiles = int((N + tile - 1) / tile);
    int* hist = static_cast<int*>(workspace);
    k_group_count<<<tiles, kWarps * 32, size_t(kWarps) * (n_types + 1) * 4, st>>>(N, tile, n_types, type, hist);
    if (cudaGetLastError()) return TPCONV_ERR_CUDA;
    k_group_place<<<tiles, kWarps * 32, place_smem(n_types), st>>>(N, tile, n_types, tiles, type, hist, perm, offsets);
    ph.note(2);
  }
  return cudaGetLastError() == cudaSuccess ? TPCONV_OK : TPCONV_ERR_CUDA;
}

}  // extern "C"
