"""Host side of the node operators at the limits of their contract (no GPU)."""

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
