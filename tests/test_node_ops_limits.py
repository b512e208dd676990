"""Host side of the node operators at the limits of their contract (no GPU)."""

import os
import subprocess

import pytest

PLANS = [("64x0e+64x1o+64x2e", 10, "fp32"), ("128x0e+128x1o+128x2e+128x3o", 89, "fp32"), ("8x0e+8x1o", 4, "fp32"),
         ("512x0e+512x1o+512x2e", 3, "fp32"), ("64x0e+64x1o+64x2e", 256, "simt"), ("37x0e+21x1o", 7, "tf32"),
         ("1x0e", 1, "fp32")]


@pytest.fixture(scope="module")
def T():
    from equivariant_gnn_tensor_receiver_b200 import build
    build.build(verbose=False)
    import equivariant_gnn_tensor_receiver_b200 as T
    return T


@pytest.mark.parametrize("irr,n_types,gemm", PLANS)
def test_linear_workspace_for_more_nodes_holds_for_fewer(T, irr, n_types, gemm):
    p = T.LinearPlan(irr, irr, n_types=n_types, gemm=gemm)
    ns = sorted(set(list(range(0, 1200)) + [round(1.07 ** k) for k in range(100, 317)] + [2 ** 31 - 1]))
    for op in (T.OP_BACKWARD, T.OP_DOUBLE_BACKWARD):
        sizes = [T._lib.tpconv_linear_workspace_size(p, op, n) for n in ns]
        assert sizes == sorted(sizes) and sizes[0] == 0


def test_linear_workspace_is_that_of_the_kernel_that_runs(T):
    """the tensor-core gradient's partial tiles (two of 32 KB per CTA, 148 CTAs), or what small calls need on the
    FP32 pipes: not the FP32 kernel's partials for all nodes"""
    size = T._lib.tpconv_linear_workspace_size
    tiles = 2 * 148 * 128 * 64 * 4
    wide = T.LinearPlan("128x0e+128x1o+128x2e+128x3o", "128x0e+128x1o+128x2e+128x3o", n_types=89)
    # small calls: up to 20 M multiply-adds, 76 nodes: at most 4 whole pieces and 76 ragged ones
    assert size(wide, 1, 8192) == max(tiles, 80 * wide.weight_numel * 4)
    wider = T.LinearPlan("256x0e+256x1o+256x2e+256x3o", "256x0e+256x1o+256x2e+256x3o", n_types=16)
    assert size(wider, 1, 262144) <= 20 << 20
    layer = T.LinearPlan("64x0e+64x1o+64x2e", "64x0e+64x1o+64x2e", n_types=10)
    assert size(layer, 1, 64) <= 1 << 20 and size(layer, 1, 4096) == tiles


MOST_CHUNKS = r"""
#include <cstdio>
#include <vector>
#include "linear_grad_tc.h"
#include "linear_tc.h"
int main() {
  for (int d : {1, 3, 5, 7})
    for (long long N : {1000LL, 400000000LL, 1000000000LL, (1LL << 31) - 1}) {
      std::vector<tpc::LinPath> p(48);
      for (auto& q : p) q = {d, 1, 1, 0, 0, 0, 0, 0};
      static tpc::LinRows R;
      R = {};
      R.n_out = 12, R.T = 3, R.N = N;
      for (int b = 0; b < 12; ++b) R.o[b] = {0, 256, d, 0, 0};
      std::printf("%d %lld %d %d\n", d, N, int(tpc::linear_grad_tc_supported(p.data(), 48, 3, N)),
                  tpc::linear_tc_launches(R));
    }
}
"""


def test_calls_of_too_many_chunks_leave_the_tensor_cores(T, tmp_path):
    """The tensor-core kernels share out their chunks by 32-bit costs, at least one a chunk: calls with more chunks
    (48 paths and hundreds of millions of nodes) are given to the FP32 kernels."""
    from equivariant_gnn_tensor_receiver_b200 import build as B
    src, exe = tmp_path / "most.cu", tmp_path / "most"
    src.write_text(MOST_CHUNKS)
    objs = [os.path.join(B.BUILD, f + ".cu.o") for f in ("linear_grad_tc", "linear_tc")]
    subprocess.run([B.NVCC, *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, str(src), *objs, "-o",
                    str(exe)], check=True, capture_output=True, timeout=300)
    got = [tuple(map(int, r.split())) for r in subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                                                              timeout=60).stdout.splitlines()]
    assert len(got) == 16
    for d, n, grad, rows in got:
        assert grad == (48 * (n // (64 // d) + 3) < 2 ** 31 - 2 ** 20)
        assert (rows > 0) == (48 * (n // (120 if d == 1 else 128 // d) + 3) < 2 ** 31 - 2 ** 20)
