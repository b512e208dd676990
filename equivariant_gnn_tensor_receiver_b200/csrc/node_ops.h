// What the node operators (grouping, typed linear map, layer norm) share with
// the library's core: launch counts and timing of a phase, the device-wait
// limit, and host checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tpc {

// Counts `launches` kernels of a phase and, with profiling enabled, brackets
// the scope with events on the stream (implemented in tpconv.cu).
class NodePhase {
 public:
  NodePhase(int phase, cudaStream_t st);
  ~NodePhase();
  void note(int64_t launches);
  NodePhase(const NodePhase&) = delete;
  NodePhase& operator=(const NodePhase&) = delete;

 private:
  int phase_;
  void* scope_;
};

uint64_t device_wait_limit();  // ns, tpconv_set_wait_limit

struct Span {
  const void* p;
  size_t bytes;
};
// whether any of the first n_out spans overlaps another span (null or empty spans never do)
inline bool overlapping(const Span* s, int n_out, int n) {
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j || !s[i].p || !s[j].p || !s[i].bytes || !s[j].bytes) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = reinterpret_cast<uintptr_t>(s[j].p);
      if (a < b + s[j].bytes && b < a + s[i].bytes) return true;
    }
  return false;
}
inline bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
inline bool aligned_to_16(const void* p) { return !misaligned(p, 16); }

}  // namespace tpc
