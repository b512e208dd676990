"""Node operators at the limits of their contract, on the device: the largest graphs, long sums, caller-owned
buffers on explicit streams.  Tolerances stand beside each test."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import equivariant_gnn_tensor_receiver_b200 as T
    T.lib()
    return T


@pytest.mark.parametrize("gemm", ["fp32", "simt"])
def test_linear_of_the_most_nodes(T, gemm):
    """2^31 - 1 nodes, nearly all of one type, some of no type behind them: counts of tiles and the steps past the
    last node stay below 2^31.  Small whole numbers, so every product and sum is exact."""
    import torch
    n, few = 2 ** 31 - 1, 1000
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    types = torch.ones(n, dtype=torch.int32, device="cuda")
    types[3:7] = 0
    types[-5:] = -1
    G = T.NodeGroups(types, 2)
    assert G.offsets.tolist() == [0, 4, n - 5]
    assert G.perm[:6].tolist() == [3, 4, 5, 6, 0, 1] and G.perm[-6:].tolist() == list(range(n - 6, n))
    p = T.LinearPlan("1x0e", "1x0e", n_types=2, gemm=gemm)
    w = torch.tensor([[3.0], [2.0]], device="cuda")
    x = torch.randint(1, 100, (n, 1), device="cuda", dtype=torch.int8).float()
    want = x * 2
    want[3:7] = 3 * x[3:7]
    want[-5:] = 0
    out = torch.full_like(x, -1)
    T.linear_forward(p, G, x, w, out=out)
    assert torch.equal(out, want)
    del want
    g = out.zero_()
    g[:few], g[-few:] = 1, 2
    r = T.linear_backward(p, G, x, w, g)
    some = torch.cat((x[:few], 2 * x[-few:-5]))[:, 0]
    a = x[3:7].sum()
    assert r["dweight"].tolist() == [[a.item()], [(some.sum() - a).item()]]
    dx = r["dx"]
    assert (dx[:few, 0] == torch.where(types[:few] == 0, 3.0, 2.0)).all() and (dx[-few:-5] == 4).all()
    assert not dx[-5:].any() and not dx[few:-few].any()
    assert T._lib.tpconv_linear_device_status(p) == 0
    del x, g, out, dx, r, G, types
    torch.cuda.empty_cache()
