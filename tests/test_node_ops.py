"""Host side of the node operators (no GPU): plans, workspace sizes and the refusals of every entry point.
The C entry points check their arguments before any device work, so a refused call needs no device; the
pointers below are host addresses that only ever get compared."""

import ctypes

import numpy as np
import pytest

from oracle import node as O

INVALID, BAD_IRREPS, UNSUPPORTED, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def T():
    from equivariant_gnn_tensor_receiver_b200 import build
    build.build(verbose=False)
    import equivariant_gnn_tensor_receiver_b200 as T
    return T


@pytest.mark.parametrize("irr", [("64x0e+64x1o+64x2e",) * 2, ("37x0e+21x1o+5x2e", "50x0e+19x1o"),
                                 ("2x0e+3x0e+1x2e", "2x2e+5x0e+2x0o"), ("4x1o", "4x1e")])
def test_linear_plan_matches_oracle(T, irr):
    p = T.LinearPlan(*irr, n_types=3)
    paths, numel = O.linear_paths(*irr)
    assert (p.weight_numel, p.dim_in, p.dim_out) == (numel, O.blocks(irr[0])[1], O.blocks(irr[1])[1])
    assert [(q["c_in"], q["c_out"], 2 * q["l"] + 1, q["weight_offset"]) for q in p.paths] == [
        (i[1], o[1], i[2], k) for i, o, k in paths]


@pytest.mark.parametrize("irreps", ["64x0e+64x1o+64x2e", "3x0o+2x0e+5x3o+1x0e", "4096x0e"])
def test_norm_plan_matches_oracle(T, irreps):
    p = T.NormPlan(irreps)
    assert (p.weight_numel, p.bias_numel) == O.norm_sizes(irreps) and p.dim == O.blocks(irreps)[1]


def status(T, f):
    with pytest.raises(T.TPConvError) as e:
        f()
    return e.value.status


def test_plans_refuse(T):
    assert status(T, lambda: T.LinearPlan("8x0e+8xe", "8x0e")) == BAD_IRREPS
    assert status(T, lambda: T.LinearPlan("8x0e", "")) == BAD_IRREPS
    assert status(T, lambda: T.LinearPlan("8x4e", "8x0e")) == UNSUPPORTED
    assert status(T, lambda: T.LinearPlan("8x0e", "8x0e", n_types=0)) == INVALID
    assert status(T, lambda: T.LinearPlan("8x0e", "8x0e", n_types=257)) == UNSUPPORTED
    assert status(T, lambda: T.LinearPlan("8193x0e", "8x0e")) == UNSUPPORTED
    assert status(T, lambda: T.LinearPlan("+".join(["1x0e"] * 8), "+".join(["1x0e"] * 8))) == UNSUPPORTED  # 64 paths
    assert T.LinearPlan("+".join(["1x0e"] * 6), "+".join(["1x0e"] * 8)).n_paths == 48
    assert status(T, lambda: T.NormPlan("8x0")) == BAD_IRREPS
    assert status(T, lambda: T.NormPlan("8x4e")) == UNSUPPORTED
    assert status(T, lambda: T.NormPlan("10241x0e")) == UNSUPPORTED
    assert T.NormPlan("10240x0e").dim == 10240
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-60):
        assert status(T, lambda: T.NormPlan("8x0e", eps=eps)) == INVALID
    h = ctypes.c_void_p()
    assert T.lib().tpconv_linear_create(ctypes.byref(h), b"8x0e", b"8x0e", 1, 2) == UNSUPPORTED  # no half mode
    assert T.lib().tpconv_linear_create(None, b"8x0e", b"8x0e", 1, 0) == INVALID


def test_workspace_is_bounded(T):
    L = T._lib
    p = T.LinearPlan("64x0e+64x1o+64x2e", "64x0e+64x1o+64x2e", n_types=16)
    assert L.tpconv_linear_workspace_size(p, 0, 10 ** 6) <= 1 << 20
    sizes = [L.tpconv_linear_workspace_size(p, 1, n) for n in (0, 1, 4096, 10 ** 6, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] == 0 and sizes[-1] <= 256 << 20
    q = T.NormPlan("64x0e+64x1o+64x2e")
    sizes = [L.tpconv_norm_workspace_size(q, 1, n) for n in (0, 1, 4096, 10 ** 6, 2 ** 40)]
    assert sizes == sorted(sizes) and sizes[-1] <= 8 << 20
    assert L.tpconv_group_workspace_size(100, 10) == 0
    assert L.tpconv_group_workspace_size(2 ** 31 - 1, 256) <= 1 << 20
    for f in (lambda: L.tpconv_linear_workspace_size(p, 3, 10), lambda: L.tpconv_linear_workspace_size(p, 0, -1),
              lambda: L.tpconv_norm_workspace_size(q, -1, 10), lambda: L.tpconv_group_workspace_size(2 ** 31, 10),
              lambda: L.tpconv_group_workspace_size(10, 0), lambda: L.tpconv_group_workspace_size(10, 257)):
        assert status(T, f) == INVALID


class Mem:
    """disjoint, 256-byte aligned host ranges standing for device buffers"""

    def __init__(self):
        self.keep = []

    def __call__(self, nbytes, shift=0):
        a = np.zeros(nbytes + 512, dtype=np.uint8)
        self.keep.append(a)
        return ctypes.c_void_p((a.ctypes.data + 255) // 256 * 256 + shift)


def test_group_refuses(T):
    m, f = Mem(), T.lib().tpconv_group_nodes
    t, p, o = m(4 * 100), m(4 * 100), m(4 * 11)
    assert f(-1, 10, t, p, o, None, 0, None) == INVALID
    assert f(100, 0, t, p, o, None, 0, None) == INVALID
    assert f(100, 257, t, p, o, None, 0, None) == INVALID
    assert f(2 ** 31, 10, t, p, o, None, 0, None) == INVALID
    assert f(100, 10, None, p, o, None, 0, None) == INVALID
    assert f(100, 10, t, None, o, None, 0, None) == INVALID
    assert f(100, 10, t, p, None, None, 0, None) == INVALID
    assert f(100, 10, t, t, o, None, 0, None) == INVALID          # in place
    assert f(100, 10, t, p, p, None, 0, None) == INVALID
    assert f(100, 10, m(400, 2), p, o, None, 0, None) == INVALID  # misaligned
    assert f(100_000, 10, m(4 * 100_000), m(4 * 100_000), o, None, 0, None) == WS


def test_norm_refuses(T):
    m, L = Mem(), T.lib()
    q = T.NormPlan("4x0e+4x1o")
    h, n = q.handle, 10
    row = lambda: m(4 * 16 * n)  # noqa: E731
    x, y, w, b = row(), row(), m(32), m(16)
    assert L.tpconv_norm_forward(None, n, x, w, b, y, None) == INVALID
    assert L.tpconv_norm_forward(h, -1, x, w, b, y, None) == INVALID
    assert L.tpconv_norm_forward(h, n, None, w, b, y, None) == INVALID
    assert L.tpconv_norm_forward(h, n, x, w, b, None, None) == INVALID
    assert L.tpconv_norm_forward(h, n, x, w, b, x, None) == INVALID
    assert L.tpconv_norm_forward(h, n, x, y, b, y, None) == INVALID
    assert L.tpconv_norm_forward(h, n, m(4 * 16 * n, 2), w, b, y, None) == INVALID
    g, dx, dw, db = row(), row(), m(32), m(16)
    ws = m(1 << 20)
    big = ctypes.c_size_t(1 << 20)
    assert L.tpconv_norm_backward(h, n, x, w, None, dx, dw, db, ws, big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, dx, dw, db, None, 0, None) == WS
    assert L.tpconv_norm_backward(h, n, x, w, g, dx, dw, db, None, big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, dx, dw, db, m(1 << 20, 16), big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, g, dw, db, ws, big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, dx, w, db, ws, big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, dx, dw, dw, ws, big, None) == INVALID
    assert L.tpconv_norm_backward(h, n, x, w, g, ws, dw, db, ws, big, None) == INVALID
    a, dg = row(), row()
    assert L.tpconv_norm_double_backward(h, n, x, w, None, a, None, None, dg, dx, dw, ws, big, None) == INVALID
    assert L.tpconv_norm_double_backward(h, n, x, w, g, a, None, None, dg, dg, dw, ws, big, None) == INVALID
    assert L.tpconv_norm_double_backward(h, n, x, w, g, a, None, None, a, dx, dw, ws, big, None) == INVALID
    assert L.tpconv_norm_double_backward(h, n, x, w, g, a, None, None, dg, dx, dw, ws, 0, None) == WS


def test_linear_refuses(T):
    m, L = Mem(), T.lib()
    q = T.LinearPlan("4x0e+4x1o", "8x0e+4x1o", n_types=2)
    h, n = q.handle, 10
    x, out, w = m(4 * 16 * n), m(4 * 20 * n), m(4 * 2 * q.weight_numel)
    perm, off = m(4 * n), m(12)
    ws, big = m(1 << 22), ctypes.c_size_t(1 << 22)
    fwd = L.tpconv_linear_forward
    assert fwd(None, n, perm, off, x, w, out, ws, big, None) == INVALID
    assert fwd(h, -1, perm, off, x, w, out, ws, big, None) == INVALID
    assert fwd(h, 2 ** 31, perm, off, x, w, out, ws, big, None) == INVALID
    assert fwd(h, n, None, off, x, w, out, ws, big, None) == INVALID
    assert fwd(h, n, perm, None, x, w, out, ws, big, None) == INVALID
    assert fwd(h, n, perm, off, None, w, out, ws, big, None) == INVALID
    assert fwd(h, n, perm, off, x, None, out, ws, big, None) == INVALID
    assert fwd(h, n, perm, off, x, w, None, ws, big, None) == INVALID
    assert fwd(h, n, perm, off, x, w, x, ws, big, None) == INVALID
    assert fwd(h, n, perm, off, x, w, perm, ws, big, None) == INVALID
    g, dx, dw = m(4 * 20 * n), m(4 * 16 * n), m(4 * 2 * q.weight_numel)
    bwd = L.tpconv_linear_backward
    assert bwd(h, n, perm, off, x, w, None, dx, dw, ws, big, None) == INVALID
    assert bwd(h, n, perm, off, None, w, g, dx, dw, ws, big, None) == INVALID
    assert bwd(h, n, perm, off, x, w, g, dx, dw, None, 0, None) == WS
    assert bwd(h, n, perm, off, x, w, g, dx, dw, m(1 << 22, 16), big, None) == INVALID
    assert bwd(h, n, perm, off, x, w, g, x, dw, ws, big, None) == INVALID
    assert bwd(h, n, perm, off, x, w, g, dx, w, ws, big, None) == INVALID
    a, al, dg = m(4 * 16 * n), m(4 * 2 * q.weight_numel), m(4 * 20 * n)
    dbl = L.tpconv_linear_double_backward
    assert dbl(h, n, perm, off, x, w, None, a, al, dg, dx, dw, ws, big, None) == INVALID
    assert dbl(h, n, perm, off, None, w, g, a, al, dg, dx, dw, ws, big, None) == INVALID
    assert dbl(h, n, perm, off, x, None, g, a, al, dg, dx, dw, ws, big, None) == INVALID
    assert dbl(h, n, perm, off, x, w, g, a, al, g, dx, dw, ws, big, None) == INVALID
    assert dbl(h, n, perm, off, x, w, g, a, al, dg, dx, al, ws, big, None) == INVALID
    assert dbl(h, n, perm, off, x, w, g, a, al, dg, dx, dw, None, 0, None) == WS


def test_python_layer_refuses_host_tensors(T):
    import torch
    q = T.NormPlan("4x0e")
    with pytest.raises(ValueError):
        T.norm_forward(q, torch.zeros(3, 4))
    with pytest.raises(ValueError):
        T.NodeGroups(torch.zeros(3, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        T.linear_forward(T.LinearPlan("4x0e", "4x0e"), None, torch.zeros(3, 4), torch.zeros(1, 16))


def test_streams_of_another_device_are_refused():
    """(a stand-in for the stream: the check is the host's)"""
    from types import SimpleNamespace
    from equivariant_gnn_tensor_receiver_b200 import node
    with pytest.raises(ValueError, match="stream"):
        node._on(0, SimpleNamespace(device_index=1, cuda_stream=0))
    assert isinstance(node._on(1, SimpleNamespace(device_index=1, cuda_stream=0)), node._There)
